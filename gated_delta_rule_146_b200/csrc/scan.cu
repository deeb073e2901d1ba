// scan.cu -- gated linear recurrence: forward over whole sequences, and one token.
//
//     h_t = alpha_t h_{t-1} + b_t,   alpha = exp(g),   b = v | beta v | (1 - alpha) v,   o = h
//
// Every element is read and written once (6 bytes per token and channel in bf16, 8 with beta),
// for five operations: HBM bounds it.  The split is described in scan_impl.cuh.
#include "scan_impl.cuh"

namespace gdr {

namespace {

constexpr int kSeg = 8;  // tokens of a lane's run
constexpr int kTile = kScanWarps * kSeg;

template <typename IO, typename GT>
struct FwdParams {
    const IO* v; const GT* g; const GT* beta;
    const float* h0;
    IO* o;
    float* h_final;
    int* status;
    Seqs q;
    int D, L, slabs, reverse;  // L: tokens of a row
};

// alpha and b of one element
template <int kWrite>
__device__ __forceinline__ void decay_write(float g, float v, float beta, float& a, float& b) {
    if constexpr (kWrite == GDR_WRITE_TIED) {
        const float em = expm1f(g);  // 1 - alpha without cancellation
        a = 1.f + em;
        b = -em * v;
    } else {
        a = expf(g);
        b = kWrite == GDR_WRITE_GATE ? beta * v : v;
    }
}

// kSeqs: one row holds all sequences, whose starts reset the state; else a row is a sequence.
template <typename IO, typename GT, int kWrite, int VEC, bool kSeqs>
__global__ void __launch_bounds__(kScanThreads)
scan_fwd_kernel(const FwdParams<IO, GT> p, const int cluster) {
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
    if (kSeqs && rank == 0 && p.h_final && on) {  // empty sequences keep their state
        for (int s = wid; s < p.q.n; s += kScanWarps) {
            if (p.q.begin(s) != p.q.end(s)) continue;
            float x[VEC] = {};
            if (p.h0) load_f<float, VEC>(p.h0 + (size_t)s * p.D + c, x);
            store_vec<float, VEC>(p.h_final + (size_t)s * p.D + c, x);
        }
    }

    float carry[VEC] = {};
    if (!kSeqs && p.h0 && on) load_f<float, VEC>(p.h0 + (size_t)row * p.D + c, carry);

    Vec<IO, VEC> rv[kSeg];
    Vec<GT, VEC> rg[kSeg], rb[kSeg];
    auto place = [&](int i) { return p.reverse ? L - 1 - i : i; };
    auto fetch = [&](int first) {
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            if (!on || first + i >= L) continue;
            const size_t at = (row0 + place(first + i)) * p.D + c;
            rv[i] = load_vec<IO, VEC>(p.v + at);
            rg[i] = load_vec<GT, VEC>(p.g + at);
            if constexpr (kWrite == GDR_WRITE_GATE) rb[i] = load_vec<GT, VEC>(p.beta + at);
        }
    };

    const int stride = cluster * kTile;
    int first = rank * kTile + wid * kSeg;
    fetch(first);
    int step = 0;
    for (int base = 0; base < L; base += stride, first += stride, ++step) {
        const int n = min(kSeg, L - first);  // tokens of this lane's run (may be <= 0)
        float a[kSeg][VEC], b[kSeg][VEC];
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (i < n && on)
                    decay_write<kWrite>(to_f(rg[i].x[j]), to_f(rv[i].x[j]),
                                        kWrite == GDR_WRITE_GATE ? to_f(rb[i].x[j]) : 0.f,
                                        a[i][j], b[i][j]);
                else { a[i][j] = 1.f; b[i][j] = 0.f; }
            }
        }
        fetch(first + stride);

        Marks m{0u, 0u, 0};
        if constexpr (kSeqs) {
            m = find_marks<kSeg>(p.q, [&](int i) { return place(first + i); }, n, p.reverse, lane);
            if (m.start && p.h0) {  // b at a start takes the initial state in
#pragma unroll
                for (int i = 0; i < kSeg; ++i) {
                    if (!(m.start >> i & 1u)) continue;
                    const int s = __shfl_sync(0xffffffffu, m.seq, i);
                    float x[VEC] = {};
                    if (on) load_f<float, VEC>(p.h0 + (size_t)s * p.D + c, x);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) b[i][j] = fmaf(a[i][j], x[j], b[i][j]);
                }
            }
        }
        Run<VEC> run;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float A = 1.f, H = 0.f;
#pragma unroll
            for (int i = 0; i < kSeg; ++i) {
                H = kSeqs && (m.start >> i & 1u) ? b[i][j] : fmaf(a[i][j], H, b[i][j]);
                A *= a[i][j];
            }
            run.A[j] = kSeqs && m.start ? kReset : A;
            run.H[j] = H;
        }
        float h[VEC];
        join_runs(sh, run, step, cluster, rank, wid, lane, carry, h);
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                h[j] = kSeqs && (m.start >> i & 1u) ? b[i][j] : fmaf(a[i][j], h[j], b[i][j]);
            if (i < n && on) store_vec<IO, VEC>(p.o + (row0 + place(first + i)) * p.D + c, h);
            if (kSeqs && (m.end >> i & 1u) && p.h_final) {
                const int s = __shfl_sync(0xffffffffu, m.seq, i);
                if (on) store_vec<float, VEC>(p.h_final + (size_t)s * p.D + c, h);
            }
        }
    }
    if (!kSeqs && p.h_final && rank == 0 && wid == 0 && on)
        store_vec<float, VEC>(p.h_final + (size_t)row * p.D + c, carry);
}

template <typename IO, typename GT, int kWrite, int VEC>
gdr_status fwd_launch(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    const bool seqs = scan_one_row(a, x.cu);
    FwdParams<IO, GT> p;
    p.v = static_cast<const IO*>(x.v);
    p.g = static_cast<const GT*>(x.g);
    p.beta = static_cast<const GT*>(x.beta);
    p.h0 = x.h0;
    p.o = static_cast<IO*>(x.o);
    p.h_final = x.h_final;
    p.status = a.status;
    p.q = Seqs{x.cu, a.n_seqs, a.T, a.B * a.T};
    p.D = a.D;
    p.L = seqs ? a.B * a.T : a.T;
    p.slabs = (a.D + 32 * VEC - 1) / (32 * VEC);
    p.reverse = a.reverse;
    const long long units = (long long)p.slabs * (seqs ? 1 : a.B);
    return seqs ? scan_launch(scan_fwd_kernel<IO, GT, kWrite, VEC, true>, p, units, p.L, kTile, st)
                : scan_launch(scan_fwd_kernel<IO, GT, kWrite, VEC, false>, p, units, p.L, kTile, st);
}

template <typename IO, typename GT, int kWrite>
gdr_status fwd_vec(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    return a.D % 2 ? fwd_launch<IO, GT, kWrite, 1>(a, x, st) : fwd_launch<IO, GT, kWrite, 2>(a, x, st);
}

struct Fwd {
    template <typename IO, typename GT, int kWrite>
    static gdr_status go(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
        return fwd_vec<IO, GT, kWrite>(a, x, st);
    }
};

// ---- one token ------------------------------------------------------------------------------
// Streams the fp32 state once: 14 bytes per channel in bf16 (16 with beta).
template <typename IO, typename GT, int kWrite, int VEC>
__global__ void __launch_bounds__(256)
scan_step_kernel(const IO* __restrict__ v, const GT* __restrict__ g, const GT* __restrict__ beta,
                 const float* h, float* h_out, IO* __restrict__ o, long long n) {
    const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * VEC;
    if (at >= n) return;
    float fh[VEC], fv[VEC], fg[VEC], fb[VEC] = {};
    load_f<float, VEC>(h + at, fh);
    load_f<IO, VEC>(v + at, fv);
    load_f<GT, VEC>(g + at, fg);
    if constexpr (kWrite == GDR_WRITE_GATE) load_f<GT, VEC>(beta + at, fb);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float a, b;
        decay_write<kWrite>(fg[j], fv[j], fb[j], a, b);
        fh[j] = fmaf(a, fh[j], b);
    }
    store_vec<float, VEC>(h_out + at, fh);
    store_vec<IO, VEC>(o + at, fh);
}

struct Step {
    template <typename IO, typename GT, int kWrite>
    static gdr_status go(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
        const long long n = (long long)a.B * a.D;  // the rows join: only the end can be ragged
        const IO* v = static_cast<const IO*>(x.v);
        const GT *g = static_cast<const GT*>(x.g), *b = static_cast<const GT*>(x.beta);
        IO* o = static_cast<IO*>(x.o);
        const int vec = n % 4 ? 1 : 4;
        const long long blocks = (n / vec + 255) / 256;
        if (vec == 4)
            scan_step_kernel<IO, GT, kWrite, 4><<<(unsigned)blocks, 256, 0, st>>>(
                v, g, b, x.h0, x.h_final, o, n);
        else
            scan_step_kernel<IO, GT, kWrite, 1><<<(unsigned)blocks, 256, 0, st>>>(
                v, g, b, x.h0, x.h_final, o, n);
        return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
    }
};

}  // namespace

int scan_cluster(long long units, long long tiles) {
    int c = 1;
    while (c < kScanMaxCluster && units * c < 2 * 148 && tiles >= 2 * c) c *= 2;
    return c;
}

gdr_status launch_scan_fwd(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    if (a.B * (long long)a.T == 0) {  // every state stays
        const size_t bytes = sizeof(float) * (size_t)a.n_seqs * a.D;
        if (!x.h_final || x.h_final == x.h0) return GDR_OK;
        const cudaError_t e = x.h0 ? cudaMemcpyAsync(x.h_final, x.h0, bytes,
                                                     cudaMemcpyDeviceToDevice, st)
                                   : cudaMemsetAsync(x.h_final, 0, bytes, st);
        return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
    }
    return scan_dispatch<Fwd>(a, x, st);
}

gdr_status launch_scan_step(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    return scan_dispatch<Step>(a, x, st);
}

}  // namespace gdr
