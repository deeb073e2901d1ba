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
    float a[kSeg][2], d[kSeg][2];  // alpha; dO, with dh_final at a sequence's last token
    Run before;
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

    if (kSeqs && blockIdx.x == 0) check_cu(p.q, p.status, tid, kScanThreads);
    if (kSeqs && rank == 0 && p.dh0) {  // the state's gradient passes an empty sequence unchanged
        for (int s = wid; s < p.q.n; s += kScanWarps) {
            if (p.q.begin(s) != p.q.end(s)) continue;
            float x[2] = {};
            if (p.dh_final) load_state<kCopy>(p.dh_final + (size_t)s * D + c, x, mine);
            store_pair<float, kCopy>(p.dh0 + (size_t)s * D + c, x, mine);
        }
    }

    const size_t base = (size_t)row * L * D + slab * kSlab;
    char* const buf = stages + wid * kStages * St::kBytes;
    auto feed = [&](int first, int stage) {
        char* s = buf + stage * St::kBytes;
        feed_rows<GT, kCopy, kSeg>(s, p.g + base, origin, dir, first, L, D, left, lane);
        feed_rows<IO, kCopy, kSeg>(s + St::dO, p.dO + base, origin, dir, first, L, D, left, lane);
        feed_rows<IO, kCopy, kSeg>(s + St::o, p.o + base, origin, dir, first + 1, L, D, left, lane);
        if constexpr (kWrite != GDR_WRITE_PLAIN)
            feed_rows<IO, kCopy, kSeg>(s + St::v, p.v + base, origin, dir, first, L, D, left, lane);
        if constexpr (kWrite == GDR_WRITE_GATE)
            feed_rows<GT, kCopy, kSeg>(s + St::beta, p.beta + base, origin, dir, first, L, D, left,
                                       lane);
        copy_commit();
    };

    const int stride = cluster * kTile;
    const int steps = (int)(((long long)L + stride - 1) / stride);
    const int first0 = rank * kTile + wid * kSeg;
    auto place = [&](int k) {
        const long long f = first0 + (long long)k * stride;
        return (int)(f < L ? f : L);
    };
    // a tile's stage is read until the tile is finished, a step after it was formed
#pragma unroll
    for (int k = 0; k < kStages - 2; ++k) feed(place(k), k);

    Here here{0, 0};
    auto form = [&](int k, Elements& e) {
        copy_wait<kStages - 3>();
        __syncwarp();
        feed(place(k + kStages - 2), (k + kStages - 2) % kStages);
        const char* s = buf + (k % kStages) * St::kBytes;
        if constexpr (kSeqs) {
            const int first = place(k);
            e.m = find_marks(p.q, here, origin, dir, first, min(kSeg, L - first), lane);
        }
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            float g[2];
            Rows<GT, kSeg>::read(s, i, lane, g);
            Rows<IO, kSeg>::read(s + St::dO, i, lane, e.d[i]);
#pragma unroll
            for (int j = 0; j < 2; ++j) e.a[i][j] = expf(g[j]);
            if (kSeqs && (e.m.start >> i & 1u) && p.dh_final) {
                const int q = __shfl_sync(0xffffffffu, e.m.seq, i);
                float x[2];
                load_state<kCopy>(p.dh_final + (size_t)q * D + c, x, mine);
#pragma unroll
                for (int j = 0; j < 2; ++j) e.d[i][j] += x[j];
            }
        }
        Run run;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float A = 1.f, H = 0.f;
#pragma unroll
            for (int i = 0; i < kSeg; ++i) {
                H = e.a[i][j] * (kSeqs && (e.m.start >> i & 1u) ? e.d[i][j] : e.d[i][j] + H);
                A *= e.a[i][j];
            }
            run.A[j] = kSeqs && e.m.start ? kReset : A;
            run.H[j] = H;
        }
        sh.warp[k & 1][wid][lane] = run;
    };

    float carry[2] = {}, h0_row[2] = {};
    if (!kSeqs) {
        if (p.dh_final) load_state<kCopy>(p.dh_final + (size_t)row * D + c, carry, mine);
        if (p.h0) load_state<kCopy>(p.h0 + (size_t)row * D + c, h0_row, mine);
    }

    auto cl = cooperative_groups::this_cluster();
    Run whole;
    auto publish = [&](int k, Elements& e) {
        join_block<kSeqs>(sh.warp[k & 1], wid, lane, e.before, whole);
        if (cluster > 1) {
            if (wid < cluster) *cl.map_shared_rank(&sh.block[k & 3][rank][lane], wid) = whole;
            cl.barrier_arrive();
        }
    };
    auto finish = [&](int k, const Elements& e, const Run& tile) {
        float mu[2];
        if (cluster == 1) {
            mu[0] = carry[0];
            mu[1] = carry[1];
            run_apply<kSeqs>(tile, carry);
        } else {
            for (int r = 0; r < cluster; ++r) {
                if (r == rank) { mu[0] = carry[0]; mu[1] = carry[1]; }
                run_apply<kSeqs>(sh.block[k & 3][r][lane], carry);
            }
        }
        run_apply<kSeqs>(e.before, mu);
        const char* s = buf + (k % kStages) * St::kBytes;
        const int first = place(k), n = min(kSeg, L - first);
        const long long next = (long long)dir * D;
        long long at = (long long)base + (long long)(origin + dir * first) * D + 2 * lane;
#pragma unroll
        for (int i = 0; i < kSeg; ++i, at += next) {
            const bool ends = kSeqs ? (e.m.end >> i & 1u) : first + i == L - 1;
            const int q = !kSeqs ? row : ends ? __shfl_sync(0xffffffffu, e.m.seq, i) : 0;
            float lam[2], hp[2], out[2], v[2], w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                lam[j] = kSeqs && (e.m.start >> i & 1u) ? e.d[i][j] : e.d[i][j] + mu[j];
                mu[j] = e.a[i][j] * lam[j];
            }
            if (i >= n) continue;
            Rows<IO, kSeg>::read(s + St::o, i, lane, hp);
            if (ends) {
                hp[0] = h0_row[0];
                hp[1] = h0_row[1];
                if (kSeqs && p.h0) load_state<kCopy>(p.h0 + (size_t)q * D + c, hp, mine);
                if (p.dh0) store_pair<float, kCopy>(p.dh0 + (size_t)q * D + c, mu, mine);
            }
            if constexpr (kWrite != GDR_WRITE_PLAIN) Rows<IO, kSeg>::read(s + St::v, i, lane, v);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                out[j] = mu[j] * (kWrite == GDR_WRITE_TIED ? hp[j] - v[j] : hp[j]);
            store_pair<GT, kCopy>(p.dg + at, out, mine);
            if constexpr (kWrite == GDR_WRITE_GATE) {
                Rows<GT, kSeg>::read(s + St::beta, i, lane, w);
#pragma unroll
                for (int j = 0; j < 2; ++j) out[j] = lam[j] * v[j];
                store_pair<GT, kCopy>(p.dbeta + at, out, mine);
            } else if constexpr (kWrite == GDR_WRITE_TIED) {
                Rows<GT, kSeg>::read(s, i, lane, w);
#pragma unroll
                for (int j = 0; j < 2; ++j) w[j] = -expm1f(w[j]);
            } else {
                w[0] = w[1] = 1.f;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) out[j] = kWrite == GDR_WRITE_PLAIN ? lam[j] : w[j] * lam[j];
            store_pair<IO, kCopy>(p.dv + at, out, mine);
        }
    };

    // the forward's walk (scan.cu)
    auto turn = [&](int k, Elements& now, Elements& next) {
        const Run tile = whole;
        if (k + 1 < steps) {
            form(k + 1, next);
            __syncthreads();
        }
        if (cluster > 1) cl.barrier_wait();
        if (k + 1 < steps) publish(k + 1, next);
        finish(k, now, tile);
    };
    Elements even, odd;
    form(0, even);
    __syncthreads();
    publish(0, even);
    for (int k = 0; k < steps; k += 2) {
        turn(k, even, odd);
        if (k + 1 < steps) turn(k + 1, odd, even);
    }
    copy_wait<0>();
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
