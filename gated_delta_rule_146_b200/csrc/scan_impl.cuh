// scan_impl.cuh -- what the forward and the backward kernel of the gated linear recurrence
// share: the split of a row over lanes, warps and blocks, the feeding of its tokens, and the
// joining of its pieces.
//
// A recurrence x <- a x + b over a run of tokens is the map x -> A x + H (A the product of the
// decays, H the run's result from zero), and maps compose.  A block owns a slab of 64 channels
// of one row, two per lane, and walks it in tiles of kScanWarps * kSeg tokens: a warp takes
// kSeg tokens and forms its run's (A, H); the block's warps join theirs through shared memory,
// in order.  Where rows and channels give too few blocks, the blocks of a cluster take
// neighbouring tiles at once and join through distributed shared memory.  There is no other wait
// between blocks, no workspace, and every join has a fixed order.
//
// The walk is a pipeline.  A warp's tokens arrive by asynchronous copies, kStages - 1 tiles
// ahead, into shared memory of its own; the runs of tile k + 1 are formed and handed over before
// the elements of tile k are finished, so that neither the block's barrier nor the cluster's is
// waited for right after it was reached.
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
constexpr int kSlab = 64;                      // channels of a block
constexpr float kReset = -1.f;

// The map of a run, for a lane's two channels.
struct alignas(16) Run {
    float A[2], H[2];
};

template <bool kSeqs>
__device__ __forceinline__ void run_apply(const Run& r, float (&x)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float y = fmaf(r.A[j], x[j], r.H[j]);
        x[j] = kSeqs && r.A[j] < 0.f ? r.H[j] : y;
    }
}

// f followed by r, into f
template <bool kSeqs>
__device__ __forceinline__ void run_join(Run& f, const Run& r) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const bool stop = kSeqs && r.A[j] < 0.f;
        f.H[j] = stop ? r.H[j] : fmaf(r.A[j], f.H[j], r.H[j]);
        f.A[j] = stop || (kSeqs && f.A[j] < 0.f) ? kReset : f.A[j] * r.A[j];
    }
}

__device__ __forceinline__ Run run_none() { return Run{{1.f, 1.f}, {0.f, 0.f}}; }

struct ScanShared {
    Run warp[2][kScanWarps][32];         // runs of the block's warps, by tile parity
    // runs of the cluster's blocks, by tile modulo four.  A block writes tile k + 1 once every
    // block has handed over tile k, which it does before it reads tile k - 1: the slot written
    // is neither of these
    Run block[4][kScanMaxCluster][32];
};

// Joins the block's runs of one tile (all written, behind a block barrier): the map of the
// warps before this one, and that of the whole tile.
template <bool kSeqs>
__device__ __forceinline__ void join_block(const Run (&warp)[kScanWarps][32], int wid, int lane,
                                           Run& before, Run& all) {
    all = run_none();
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) {
        if (w == wid) before = all;
        run_join<kSeqs>(all, warp[w][lane]);
    }
}

// ---- feeding -----------------------------------------------------------------------------------
// How rows are copied: 16 bytes a lane where rows are whole 16-byte words; a lane's own two
// channels (4 or 8 bytes) where D is even; else through registers, one element at a time.
enum Copy { kCopy16, kCopyPair, kCopyOne };

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool in) {
    const int n = in ? kBytes : 0;  // the rest of the word is zero
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A warp's kSeg rows of 64 channels of one tensor in shared memory.
template <typename E, int kSeg>
struct Rows {
    static constexpr int kBytes = kSeg * kSlab * (int)sizeof(E);
    static __device__ __forceinline__ void read(const char* p, int i, int lane, float (&f)[2]) {
        const char* q = p + i * kSlab * (int)sizeof(E) + lane * 2 * (int)sizeof(E);
        if constexpr (sizeof(E) == 2) {
            const uint32_t r = *reinterpret_cast<const uint32_t*>(q);
            f[0] = __uint_as_float(r << 16);
            f[1] = __uint_as_float(r & 0xffff0000u);
        } else {
            const float2 r = *reinterpret_cast<const float2*>(q);
            f[0] = r.x;
            f[1] = r.y;
        }
    }
};

// Copies places [first, first + kSeg) of a row's order into p; places at or behind L are zero.
// src: the slab's first channel of the row's first token; place 0 is token `origin`, and the
// order goes up or (dir = -1) down the tokens.
template <typename E, Copy kCopy, int kSeg>
__device__ __forceinline__ void feed_rows(char* p, const E* src, int origin, int dir, int first,
                                          int L, int D, int left, int lane) {
    if constexpr (kCopy == kCopy16) {
        constexpr int kChunks = kSlab * (int)sizeof(E) / 16;  // of a row
        constexpr int kRows = 32 / kChunks;                   // rows of one pass of the warp
        constexpr int kEls = 16 / (int)sizeof(E);
        const int row = lane / kChunks, col = (lane % kChunks) * kEls;
        const E* at = src + (long long)(origin + dir * (first + row)) * D + col;
        const long long next = (long long)dir * kRows * D;
        uint32_t dst = (uint32_t)__cvta_generic_to_shared(p) + (uint32_t)lane * 16;
#pragma unroll
        for (int m = 0; m < kSeg / kRows; ++m) {
            const bool in = col < left && first + row + m * kRows < L;
            copy_async<16>(dst + m * 512, in ? at : src, in);
            at += next;
        }
    } else if constexpr (kCopy == kCopyPair) {
        const E* at = src + (long long)(origin + dir * first) * D + 2 * lane;
        const long long next = (long long)dir * D;
        uint32_t dst = (uint32_t)__cvta_generic_to_shared(p) + (uint32_t)(lane * 2 * sizeof(E));
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            const bool in = 2 * lane < left && first + i < L;
            copy_async<2 * (int)sizeof(E)>(dst + i * kSlab * (int)sizeof(E), in ? at : src, in);
            at += next;
        }
    } else {
        const E* at = src + (long long)(origin + dir * first) * D + 2 * lane;
        const long long next = (long long)dir * D;
        E r[kSeg][2];
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                r[i][j] = 2 * lane + j < left && first + i < L ? at[j] : from_f<E>(0.f);
            at += next;
        }
        E* q = reinterpret_cast<E*>(p);
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) q[i * kSlab + 2 * lane + j] = r[i][j];
        }
    }
}

// Writes a lane's two channels of one token (left: channels from the lane's first on).
template <typename E, Copy kCopy>
__device__ __forceinline__ void store_pair(E* p, const float (&f)[2], int left) {
    if constexpr (kCopy != kCopyOne) {
        if (left > 0) store_vec<E, 2>(p, f);
    } else {
        if (left > 0) p[0] = from_f<E>(f[0]);
        if (left > 1) p[1] = from_f<E>(f[1]);
    }
}

// A lane's two channels of a state row.
template <Copy kCopy>
__device__ __forceinline__ void load_state(const float* p, float (&f)[2], int left) {
    f[0] = f[1] = 0.f;
    if constexpr (kCopy != kCopyOne) {
        if (left > 0) load_f<float, 2>(p, f);
    } else {
        if (left > 0) f[0] = p[0];
        if (left > 1) f[1] = p[1];
    }
}

// ---- sequences of a row ------------------------------------------------------------------------

// Which of a warp's tokens start or end a sequence, in the kernel's order, and (in lane i) the
// sequence of token i.
struct Marks {
    unsigned start, end;
    int seq;
};

// The sequence met last, so that runs inside one sequence need no search.
struct Here {
    int b, e;
};

__device__ __forceinline__ Marks find_marks(const Seqs& q, Here& here, int origin, int dir,
                                            int first, int n, int lane) {
    Marks m{0u, 0u, 0};
    if (n <= 0) return m;
    const int x = origin + dir * first, y = origin + dir * (first + n - 1);
    if (min(x, y) > here.b && max(x, y) < here.e - 1) return m;
    bool lo = false, hi = false;
    if (lane < n) {
        const int t = origin + dir * (first + lane);
        m.seq = q.of(t);
        here.b = q.begin(m.seq);
        here.e = q.end(m.seq);
        lo = t == here.b;
        hi = t == here.e - 1;
    }
    const unsigned l = __ballot_sync(0xffffffffu, lo), h = __ballot_sync(0xffffffffu, hi);
    m.start = dir > 0 ? l : h;
    m.end = dir > 0 ? h : l;
    here.b = __shfl_sync(0xffffffffu, here.b, n - 1);
    here.e = __shfl_sync(0xffffffffu, here.e, n - 1);
    return m;
}

// ---- launching ---------------------------------------------------------------------------------

// Whether one row of the kernel holds all sequences: packed ones, and rows that would not fill
// a block's tile each.
inline bool scan_one_row(const gdr_scan_args& a, const int32_t* cu) { return cu || a.T < 64; }

// The widest copy that both types allow.  (Mixed types with rows of odd words are rare enough to
// go element by element.)
inline Copy scan_copy(const gdr_scan_args& a) {
    const bool mixed = a.io_dtype != a.gate_dtype, f32 = !mixed && a.io_dtype == GDR_F32;
    return a.D % (f32 ? 4 : 8) == 0 ? kCopy16 : a.D % 2 == 0 && !mixed ? kCopyPair : kCopyOne;
}

// Blocks of a cluster: as few as fill the GPU (units: slabs times rows; tiles of a row).
int scan_cluster(long long units, long long tiles);

template <typename P>
gdr_status scan_launch(void (*kernel)(P, int), const P& p, long long units, int L, int tile,
                       size_t smem, cudaStream_t st) {
    const int cluster = scan_cluster(units, ((long long)L + tile - 1) / tile);
    if (units * cluster > 0x7fffffffLL) return GDR_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return GDR_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = smem;
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
