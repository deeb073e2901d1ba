// scan_impl.cuh -- what the forward and the backward kernel of the gated linear recurrence
// share: the split of a row over threads, warps and blocks, and the joining of its pieces.
//
// A recurrence x <- a x + b over a run of tokens is the map x -> A x + H (A the product of the
// decays, H the run's result from zero), and maps compose.  A block owns a slab of 32 * VEC
// channels of one row and walks it in tiles of kWarps * kSeg tokens: a lane keeps kSeg tokens of
// its channels in registers, forms its run's (A, H), and the block's warps join theirs through
// shared memory, in order.  Where rows and channels give too few blocks, the P blocks of a
// cluster take P neighbouring tiles at once and join through distributed shared memory: one
// cluster barrier a step, no other wait between blocks, and every join in a fixed order.
//
// A run that holds the start of a sequence ignores what comes in.  Its A is kReset (decays are
// never negative) and the join selects H, so that infinities and NaN of the sequence before
// do not pass, as they would through a product with zero.
#pragma once

#include <cooperative_groups.h>

#include "layer.cuh"

namespace gdr {

constexpr int kScanWarps = 8;
constexpr int kScanThreads = 32 * kScanWarps;
constexpr int kScanMaxCluster = 8;
constexpr float kReset = -1.f;

template <int VEC>
struct alignas(8 * VEC) Run {
    float A[VEC], H[VEC];
};

// x after the run, from x before it
__device__ __forceinline__ float run_apply(float A, float H, float x) {
    return A < 0.f ? H : fmaf(A, x, H);
}

template <int VEC>
__device__ __forceinline__ void run_apply(const Run<VEC>& r, float (&x)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = run_apply(r.A[j], r.H[j], x[j]);
}

// f followed by r, into f
template <int VEC>
__device__ __forceinline__ void run_join(Run<VEC>& f, const Run<VEC>& r) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        f.H[j] = run_apply(r.A[j], r.H[j], f.H[j]);
        f.A[j] = (r.A[j] < 0.f || f.A[j] < 0.f) ? kReset : f.A[j] * r.A[j];
    }
}

template <int VEC>
struct ScanShared {
    Run<VEC> warp[2][kScanWarps][32];          // runs of the block's warps, by step parity
    Run<VEC> block[2][kScanMaxCluster][32];    // runs of the cluster's blocks
};

// Joins this step's runs.  `mine`: the lane's run; `carry`: the channels' state before the
// step's first token, which becomes the state after its last; returns in x the state before
// the lane's run.  Two parities keep a step's reads apart from the next one's writes: a block
// writes a parity again only behind the barrier that follows every read of it.
template <int VEC>
__device__ __forceinline__ void join_runs(ScanShared<VEC>& sh, const Run<VEC>& mine, int step,
                                          int cluster, int rank, int wid, int lane,
                                          float (&carry)[VEC], float (&x)[VEC]) {
    const int par = step & 1;
    sh.warp[par][wid][lane] = mine;
    __syncthreads();
    if (cluster == 1) {
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) {
            if (w == wid) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[j] = carry[j];
            }
            run_apply(sh.warp[par][w][lane], carry);
        }
        return;
    }
    auto cl = cooperative_groups::this_cluster();
    if (wid < cluster) {  // warp k tells block k
        Run<VEC> all = sh.warp[par][0][lane];
#pragma unroll
        for (int w = 1; w < kScanWarps; ++w) run_join(all, sh.warp[par][w][lane]);
        *cl.map_shared_rank(&sh.block[par][rank][lane], wid) = all;
    }
    cl.sync();
    for (int k = 0; k < cluster; ++k) {
        if (k == rank) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[j] = carry[j];
        }
        run_apply(sh.block[par][k][lane], carry);
    }
    for (int w = 0; w < wid; ++w) run_apply(sh.warp[par][w][lane], x);
}

// Which of the warp's tokens start or end a sequence, in the kernel's order, and (in lane i)
// the sequence of token i.
struct Marks {
    unsigned start, end;
    int seq;
};

// tok(i): the token at place i of the warp's run, n of them; `flip`: the order is that of
// decreasing tokens.
template <int kSeg, typename F>
__device__ __forceinline__ Marks find_marks(const Seqs& q, F tok, int n, bool flip, int lane) {
    bool lo = false, hi = false;
    int s = 0;
    if (lane < kSeg && lane < n) {
        const int t = tok(lane);
        s = q.of(t);
        lo = t == q.begin(s);
        hi = t == q.end(s) - 1;
    }
    Marks m;
    const unsigned l = __ballot_sync(0xffffffffu, lo), h = __ballot_sync(0xffffffffu, hi);
    m.start = flip ? h : l;
    m.end = flip ? l : h;
    m.seq = s;
    return m;
}

// ---- launching ---------------------------------------------------------------------------------

// Whether one row of the kernel holds all sequences: packed ones, and rows too short for a
// block's tile each.
inline bool scan_one_row(const gdr_scan_args& a, const int32_t* cu) { return cu || a.T < 64; }

// Blocks of a cluster: as few as fill the GPU (units: slabs times rows; tiles of a row).
int scan_cluster(long long units, long long tiles);

template <typename P>
gdr_status scan_launch(void (*kernel)(P, int), const P& p, long long units, int L, int tile,
                       cudaStream_t st) {
    int cluster = scan_cluster(units, (L + tile - 1) / tile);
    if (units * cluster > 0x7fffffffLL) return GDR_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(kScanThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, cluster) == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

template <typename Op, typename IO, typename GT>
gdr_status scan_dispatch_write(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    switch (a.write) {
        case GDR_WRITE_GATE: return Op::template go<IO, GT, GDR_WRITE_GATE>(a, x, st);
        case GDR_WRITE_TIED: return Op::template go<IO, GT, GDR_WRITE_TIED>(a, x, st);
        default: return Op::template go<IO, GT, GDR_WRITE_PLAIN>(a, x, st);
    }
}

template <typename Op>
gdr_status scan_dispatch(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (a.io_dtype == GDR_BF16)
        return a.gate_dtype == GDR_BF16 ? scan_dispatch_write<Op, bf, bf>(a, x, st)
                                        : scan_dispatch_write<Op, bf, float>(a, x, st);
    return a.gate_dtype == GDR_BF16 ? scan_dispatch_write<Op, float, bf>(a, x, st)
                                    : scan_dispatch_write<Op, float, float>(a, x, st);
}

}  // namespace gdr
