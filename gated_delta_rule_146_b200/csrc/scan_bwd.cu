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

constexpr int kStages = 4;
constexpr int kSeg = 4;                    // tokens of a warp's run
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

// Where a warp's tokens of each tensor lie in a stage: g, dO, o of the token before, v, beta.
template <typename IO, typename GT, int kWrite>
struct Stage {
    static constexpr int kG = Rows<GT, kSeg>::kBytes, kI = Rows<IO, kSeg>::kBytes;
    static constexpr int dO = kG, o = dO + kI, v = o + kI, beta = v + kI;
    static constexpr int kBytes = v + (kWrite == GDR_WRITE_PLAIN ? 0 : kI) +
                                  (kWrite == GDR_WRITE_GATE ? kG : 0);
};

struct Elements {
    F2 a[kSeg], d[kSeg];           // alpha; dO, with dh_final at a sequence's last token
    Marks m;                       // start: the last token of a sequence, end: its first
};

template <typename IO, typename GT, int kWrite, Copy kCopy, bool kSeqs>
__global__ void __launch_bounds__(kScanThreads, 2)
scan_bwd_kernel(const BwdParams<IO, GT> p, const int cluster) {
    extern __shared__ __align__(128) char stages[];
    __shared__ ScanShared sh;
    using St = Stage<IO, GT, kWrite>;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = blockIdx.x % cluster;
    const int unit = blockIdx.x / cluster;
    const int slab = unit % p.slabs, row = unit / p.slabs;
    const int left = p.D - slab * kSlab;
    const int c = slab * kSlab + 2 * lane, mine = left - 2 * lane;
    const int L = p.L, D = p.D;
    // the adjoint's order: the forward's, backwards
    const int origin = p.reverse ? 0 : L - 1, dir = p.reverse ? 1 : -1;

    scan_open(sh, cluster);
    if (kSeqs && blockIdx.x == 0) check_cu(p.q, p.status, tid, kScanThreads);
    if (kSeqs && rank == 0 && p.dh0) {  // the state's gradient passes an empty sequence unchanged
        for (int s = wid; s < p.q.n; s += kScanWarps) {
            if (p.q.begin(s) != p.q.end(s)) continue;
            F2 x = f2(0.f);
            if (p.dh_final) x = load_state<kCopy>(p.dh_final + (size_t)s * D + c, mine);
            store_pair<float, kCopy>(p.dh0 + (size_t)s * D + c, x, mine);
        }
    }

    const size_t base = (size_t)row * L * D + slab * kSlab;
    const int stride = cluster * kTile, first0 = rank * kTile + wid * kSeg;
    const int steps = (int)(((long long)L + stride - 1) / stride);
    const long long hop = (long long)dir * stride * D;
    char* const buf = stages + wid * kStages * St::kBytes;
    Feed<GT, kCopy, kSeg> fg, fb;
    Feed<IO, kCopy, kSeg> fd, fo, fv;
    fg.open(p.g + base, origin, dir, first0, D, left, lane);
    fd.open(p.dO + base, origin, dir, first0, D, left, lane);
    fo.open(p.o + base, origin, dir, first0 + 1, D, left, lane);
    if constexpr (kWrite != GDR_WRITE_PLAIN) fv.open(p.v + base, origin, dir, first0, D, left, lane);
    if constexpr (kWrite == GDR_WRITE_GATE) fb.open(p.beta + base, origin, dir, first0, D, left, lane);
    auto feed = [&](int k) {
        char* s = buf + k % kStages * St::kBytes;
        const int place = k < steps ? first0 + k * stride : L;
        fg.tile(s, place, L, hop);
        fd.tile(s + St::dO, place, L, hop);
        fo.tile(s + St::o, place + 1, L, hop);
        if constexpr (kWrite != GDR_WRITE_PLAIN) fv.tile(s + St::v, place, L, hop);
        if constexpr (kWrite == GDR_WRITE_GATE) fb.tile(s + St::beta, place, L, hop);
        copy_commit();
    };
    // a tile's stage is read until the tile is finished, a step after it was formed
#pragma unroll
    for (int k = 0; k < kStages - 2; ++k) feed(k);

    F2 carry = f2(0.f), h0_row = f2(0.f);
    if (!kSeqs) {
        if (p.dh_final) carry = load_state<kCopy>(p.dh_final + (size_t)row * D + c, mine);
        if (p.h0) h0_row = load_state<kCopy>(p.h0 + (size_t)row * D + c, mine);
    }
    Here here{0, 0};
    auto form = [&](int k, Elements& e) {
        copy_wait<kStages - 3>();
        __syncwarp();
        feed(k + kStages - 2);
        const char* s = buf + k % kStages * St::kBytes;
        if constexpr (kSeqs) {
            const int first = first0 + k * stride;
            e.m = find_marks(p.q, here, origin, dir, first, min(kSeg, L - first), lane);
        }
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            e.a[i] = exp2ch(Rows<GT, kSeg>::read(s, i, lane));
            e.d[i] = Rows<IO, kSeg>::read(s + St::dO, i, lane);
            if (kSeqs && (e.m.start >> i & 1u) && p.dh_final) {
                const int q = __shfl_sync(0xffffffffu, e.m.seq, i);
                e.d[i] = add2(e.d[i], load_state<kCopy>(p.dh_final + (size_t)q * D + c, mine));
            }
        }
        Run run{e.a[0], mul2(e.a[0], e.d[0])};
#pragma unroll
        for (int i = 1; i < kSeg; ++i) {
            const F2 y = add2(e.d[i], run.H);
            run.H = mul2(e.a[i], kSeqs ? pick2(e.m.start >> i & 1u, e.d[i], y) : y);
            run.A = mul2(run.A, e.a[i]);
        }
        if (kSeqs && e.m.start) run.A = f2(kReset);
        sh.warp[k & 3][wid][lane] = run;
    };

    const long long next = (long long)dir * D;
    long long out = (long long)base + (origin + (long long)dir * first0) * D + 2 * lane;
    auto finish = [&](int k, const Elements& e, F2 mu) {
        const char* s = buf + k % kStages * St::kBytes;
        const int first = first0 + k * stride, n = L - first;
        long long at = out;
        out += hop;
#pragma unroll
        for (int i = 0; i < kSeg; ++i, at += next) {
            const bool ends = kSeqs ? (e.m.end >> i & 1u) : first + i == L - 1;
            const int q = !kSeqs ? row : ends ? __shfl_sync(0xffffffffu, e.m.seq, i) : 0;
            const F2 sum = add2(e.d[i], mu);
            const F2 lam = kSeqs ? pick2(e.m.start >> i & 1u, e.d[i], sum) : sum;
            mu = mul2(e.a[i], lam);
            if (i >= n) continue;
            F2 hp = Rows<IO, kSeg>::read(s + St::o, i, lane);
            if (ends) {
                hp = h0_row;
                if (kSeqs && p.h0) hp = load_state<kCopy>(p.h0 + (size_t)q * D + c, mine);
                if (p.dh0) store_pair<float, kCopy>(p.dh0 + (size_t)q * D + c, mu, mine);
            }
            if constexpr (kWrite == GDR_WRITE_PLAIN) {
                store_pair<IO, kCopy>(p.dv + at, lam, mine);
            } else {
                const F2 v = Rows<IO, kSeg>::read(s + St::v, i, lane);
                if constexpr (kWrite == GDR_WRITE_GATE) {
                    store_pair<GT, kCopy>(p.dbeta + at, mul2(lam, v), mine);
                    store_pair<IO, kCopy>(
                        p.dv + at, mul2(lam, Rows<GT, kSeg>::read(s + St::beta, i, lane)), mine);
                } else {
                    hp = add2(hp, f2(-v.lo(), -v.hi()));
                    const F2 w = one_minus(Rows<GT, kSeg>::read(s, i, lane), e.a[i]);
                    store_pair<IO, kCopy>(p.dv + at, mul2(w, lam), mine);
                }
            }
            store_pair<GT, kCopy>(p.dg + at, mul2(mu, hp), mine);
        }
    };
    const bool ok = scan_walk<kSeqs, Elements>(sh, steps, cluster, rank, wid, lane, carry, form, finish);
    if (!ok && p.status) atomicCAS(p.status, (int)GDR_OK, (int)GDR_ERR_TIMEOUT);
    scan_close(cluster);
}

template <typename IO, typename GT, int kWrite, Copy kCopy>
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
    p.slabs = (a.D + kSlab - 1) / kSlab;
    p.reverse = a.reverse;
    const long long units = (long long)p.slabs * (seqs ? 1 : a.B);
    const size_t smem = (size_t)kScanWarps * kStages * Stage<IO, GT, kWrite>::kBytes;
    return seqs ? scan_launch(scan_bwd_kernel<IO, GT, kWrite, kCopy, true>, p, units, p.L, kTile, smem, st)
                : scan_launch(scan_bwd_kernel<IO, GT, kWrite, kCopy, false>, p, units, p.L, kTile, smem, st);
}

struct Bwd {
    template <typename IO, typename GT, int kWrite>
    static gdr_status go(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
        const Copy copy = scan_copy(a);
        if (copy == kCopy16) return bwd_launch<IO, GT, kWrite, kCopy16>(a, x, st);
        if constexpr (sizeof(IO) == sizeof(GT)) {
            if (copy == kCopyPair) return bwd_launch<IO, GT, kWrite, kCopyPair>(a, x, st);
        }
        return bwd_launch<IO, GT, kWrite, kCopyOne>(a, x, st);
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
