// scan_bwd.cu -- gated linear recurrence: backward pass.
//
// With m_t = alpha_t lam_t the adjoint runs from the last token to the first,
//     lam_t = dO_t + m_{t+1},   m_t = alpha_t lam_t,
// again a recurrence of maps m -> A m + H with the same A, split and joined as in the forward
// (scan_impl.cuh).  dg_t = m_t h_{t-1} reads h from the forward's output, so nothing is
// recomputed and every element is read and written once: 10 (plain), 12 (tied) or 16 (gate)
// bytes per token and channel in bf16.  HBM bounds it.
#include "scan_impl.cuh"

namespace gdr {

namespace {

constexpr int kSeg = 4;
constexpr int kTile = kScanWarps * kSeg;

template <typename IO, typename GT>
struct BwdParams {
    const IO* v; const GT* g; const GT* beta; const IO* o; const IO* dO;
    const float *h0, *dh_final;
    IO* dv; GT* dg; GT* dbeta;
    float* dh0;
    int* status;
    Seqs q;
    int D, L, slabs, reverse;
};

template <typename IO, typename GT, int kWrite, int VEC, bool kSeqs>
__global__ void __launch_bounds__(kScanThreads)
scan_bwd_kernel(const BwdParams<IO, GT> p, const int cluster) {
    __shared__ ScanShared<VEC> sh;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = blockIdx.x % cluster;
    const int unit = blockIdx.x / cluster;
    const int slab = unit % p.slabs, row = unit / p.slabs;
    const int c = (slab * 32 + lane) * VEC;
    const bool on = c < p.D;
    const int L = p.L;
    const size_t row0 = (size_t)row * L;

    if (kSeqs && blockIdx.x == 0) check_cu(p.q, p.status, tid, kScanThreads);
    if (kSeqs && rank == 0 && p.dh0 && on) {  // the state passes an empty sequence unchanged
        for (int s = wid; s < p.q.n; s += kScanWarps) {
            if (p.q.begin(s) != p.q.end(s)) continue;
            float x[VEC] = {};
            if (p.dh_final) load_f<float, VEC>(p.dh_final + (size_t)s * p.D + c, x);
            store_vec<float, VEC>(p.dh0 + (size_t)s * p.D + c, x);
        }
    }

    float carry[VEC] = {}, h0_row[VEC] = {};
    if (!kSeqs && on) {
        if (p.dh_final) load_f<float, VEC>(p.dh_final + (size_t)row * p.D + c, carry);
        if (p.h0) load_f<float, VEC>(p.h0 + (size_t)row * p.D + c, h0_row);
    }

    Vec<IO, VEC> rv[kSeg], ro[kSeg], rd[kSeg];
    Vec<GT, VEC> rg[kSeg], rb[kSeg];
    // place i of the adjoint's order: the forward's, backwards
    auto place = [&](int i) { return p.reverse ? i : L - 1 - i; };
    auto fetch = [&](int first) {
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            if (!on || first + i >= L) continue;
            const size_t at = (row0 + place(first + i)) * p.D + c;
            rg[i] = load_vec<GT, VEC>(p.g + at);
            rd[i] = load_vec<IO, VEC>(p.dO + at);
            if constexpr (kWrite != GDR_WRITE_PLAIN) rv[i] = load_vec<IO, VEC>(p.v + at);
            if constexpr (kWrite == GDR_WRITE_GATE) rb[i] = load_vec<GT, VEC>(p.beta + at);
            if (first + i + 1 < L)  // h of the token before, in the forward's order
                ro[i] = load_vec<IO, VEC>(p.o + (row0 + place(first + i + 1)) * p.D + c);
        }
    };

    const int stride = cluster * kTile;
    int first = rank * kTile + wid * kSeg;
    int step = 0;
    for (int base = 0; base < L; base += stride, first += stride, ++step) {
        const int n = min(kSeg, L - first);
        fetch(first);
        Marks m{0u, 0u, 0};  // start: the forward's last token of a sequence, end: its first
        if constexpr (kSeqs)
            m = find_marks<kSeg>(p.q, [&](int i) { return place(first + i); }, n, !p.reverse, lane);
        float a[kSeg][VEC], d[kSeg][VEC];
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            const bool in = i < n && on;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                a[i][j] = in ? expf(to_f(rg[i].x[j])) : 1.f;
                d[i][j] = in ? to_f(rd[i].x[j]) : 0.f;
            }
            if (kSeqs && (m.start >> i & 1u) && p.dh_final) {
                const int s = __shfl_sync(0xffffffffu, m.seq, i);
                float x[VEC] = {};
                if (on) load_f<float, VEC>(p.dh_final + (size_t)s * p.D + c, x);
#pragma unroll
                for (int j = 0; j < VEC; ++j) d[i][j] += x[j];
            }
        }
        Run<VEC> run;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float A = 1.f, H = 0.f;
#pragma unroll
            for (int i = 0; i < kSeg; ++i) {
                H = a[i][j] * (kSeqs && (m.start >> i & 1u) ? d[i][j] : d[i][j] + H);
                A *= a[i][j];
            }
            run.A[j] = kSeqs && m.start ? kReset : A;
            run.H[j] = H;
        }
        float mu[VEC];
        join_runs(sh, run, step, cluster, rank, wid, lane, carry, mu);
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            const bool ends = kSeqs ? (m.end >> i & 1u) : first + i == L - 1;
            const int s = kSeqs ? __shfl_sync(0xffffffffu, m.seq, i) : row;
            float lam[VEC], hp[VEC] = {}, out[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                lam[j] = kSeqs && (m.start >> i & 1u) ? d[i][j] : d[i][j] + mu[j];
                mu[j] = a[i][j] * lam[j];
            }
            if (i >= n || !on) continue;
            const size_t at = (row0 + place(first + i)) * p.D + c;
            if (!ends) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) hp[j] = to_f(ro[i].x[j]);
            } else if (!kSeqs) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) hp[j] = h0_row[j];
            } else if (p.h0) {
                load_f<float, VEC>(p.h0 + (size_t)s * p.D + c, hp);
            }
            if (ends && p.dh0) store_vec<float, VEC>(p.dh0 + (size_t)s * p.D + c, mu);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                out[j] = mu[j] * (kWrite == GDR_WRITE_TIED ? hp[j] - to_f(rv[i].x[j]) : hp[j]);
            store_vec<GT, VEC>(p.dg + at, out);
            if constexpr (kWrite == GDR_WRITE_GATE) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) out[j] = lam[j] * to_f(rv[i].x[j]);
                store_vec<GT, VEC>(p.dbeta + at, out);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if constexpr (kWrite == GDR_WRITE_GATE) out[j] = lam[j] * to_f(rb[i].x[j]);
                else if constexpr (kWrite == GDR_WRITE_TIED) out[j] = -expm1f(to_f(rg[i].x[j])) * lam[j];
                else out[j] = lam[j];
            }
            store_vec<IO, VEC>(p.dv + at, out);
        }
    }
}

template <typename IO, typename GT, int kWrite, int VEC>
gdr_status bwd_launch(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    const bool seqs = scan_one_row(a, x.cu);
    BwdParams<IO, GT> p;
    p.v = static_cast<const IO*>(x.v);
    p.g = static_cast<const GT*>(x.g);
    p.beta = static_cast<const GT*>(x.beta);
    p.o = static_cast<const IO*>(x.o_in);
    p.dO = static_cast<const IO*>(x.dO);
    p.h0 = x.h0;
    p.dh_final = x.dh_final;
    p.dv = static_cast<IO*>(x.dv);
    p.dg = static_cast<GT*>(x.dg);
    p.dbeta = static_cast<GT*>(x.dbeta);
    p.dh0 = x.dh0;
    p.status = a.status;
    p.q = Seqs{x.cu, a.n_seqs, a.T, a.B * a.T};
    p.D = a.D;
    p.L = seqs ? a.B * a.T : a.T;
    p.slabs = (a.D + 32 * VEC - 1) / (32 * VEC);
    p.reverse = a.reverse;
    const long long units = (long long)p.slabs * (seqs ? 1 : a.B);
    return seqs ? scan_launch(scan_bwd_kernel<IO, GT, kWrite, VEC, true>, p, units, p.L, kTile, st)
                : scan_launch(scan_bwd_kernel<IO, GT, kWrite, VEC, false>, p, units, p.L, kTile, st);
}

struct Bwd {
    template <typename IO, typename GT, int kWrite>
    static gdr_status go(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
        return a.D % 2 ? bwd_launch<IO, GT, kWrite, 1>(a, x, st)
                       : bwd_launch<IO, GT, kWrite, 2>(a, x, st);
    }
};

}  // namespace

gdr_status launch_scan_bwd(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    if (a.B * (long long)a.T == 0) {
        const size_t bytes = sizeof(float) * (size_t)a.n_seqs * a.D;
        if (!x.dh0 || x.dh0 == x.dh_final) return GDR_OK;
        const cudaError_t e = x.dh_final ? cudaMemcpyAsync(x.dh0, x.dh_final, bytes,
                                                           cudaMemcpyDeviceToDevice, st)
                                         : cudaMemsetAsync(x.dh0, 0, bytes, st);
        return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
    }
    return scan_dispatch<Bwd>(a, x, st);
}

}  // namespace gdr
