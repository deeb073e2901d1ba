// scan_impl.cuh -- what the forward and the backward kernel of the gated linear recurrence
// share: the split of a row over lanes, warps and blocks, the feeding of its tokens, and the
// joining of its pieces.
//
// A recurrence x <- a x + b over a run of tokens is the map x -> A x + H (A the product of the
// decays, H the run's result from zero), and maps compose.  A block owns a slab of 64 / kGroups
// channels of one row, two per lane, and walks it in tiles.  A lane takes kSeg tokens of a tile;
// the kGroups groups of lanes of a warp take runs that follow one another, and so do the warps.
// Runs are formed, (A, H), and joined in order: a warp's by shuffles, a block's through shared
// memory.  Where rows and channels give too few blocks, the blocks of a cluster take neighbouring
// tiles at once and join through distributed shared memory; and with groups, slabs are narrower and
// tiles longer, for more blocks and fewer steps.  There is no other wait between blocks, no
// workspace, and every join has a fixed order.
//
// The walk is a pipeline.  A warp's tokens arrive by asynchronous copies, two tiles ahead, into
// shared memory of its own, and it forms the run of tile k + 1 before it finishes tile k.  In a
// single block every warp then carries the state along the runs by itself: two blocks on an SM
// cover each other's barriers.  In a cluster the way to the other blocks is long, and the work
// around it is taken off the workers: one warp, the publisher, joins the block's runs and sends
// them to all blocks; another, the folder, carries the state along and leaves every worker the
// state before its run.
//
// A run that holds the start of a sequence ignores what comes in.  Its A is kReset (decays are
// never negative) and the join selects H, so that infinities and NaN of the sequence before
// do not pass, as they would through a product with zero.
#pragma once

#include "layer.cuh"
#include "tc_ptx.cuh"

namespace gdr {

using namespace tc;

constexpr int kScanMaxCluster = 8;             // a warp hands the block's run to one block
constexpr int kSlab = 64;                      // channels of a block without groups
constexpr float kReset = -1.f;
#ifndef GDR_SCAN_WAIT_NS   // (the test of a wait that runs out takes a shorter one)
#define GDR_SCAN_WAIT_NS 2000000000ull
#endif
constexpr uint64_t kScanWaitNs = GDR_SCAN_WAIT_NS;

// 1 - e^g given a = e^g: the series of e^g - 1 near zero (|g| < 1/2; the term left out is below
// 2^-26 of the sum), the difference elsewhere.
__device__ __forceinline__ F2 one_minus(F2 g, F2 a) {
    F2 q = fma2(g, f2(1.f / 40320), f2(1.f / 5040));
    q = fma2(q, g, f2(1.f / 720));
    q = fma2(q, g, f2(1.f / 120));
    q = fma2(q, g, f2(1.f / 24));
    q = fma2(q, g, f2(1.f / 6));
    q = fma2(q, g, f2(0.5f));
    q = fma2(q, g, f2(1.f));
    q = mul2(q, g);
    return f2(fabsf(g.lo()) < 0.5f ? -q.lo() : 1.f - a.lo(), fabsf(g.hi()) < 0.5f ? -q.hi() : 1.f - a.hi());
}

// ---- runs ----------------------------------------------------------------------------------------
// The map of a run, for a lane's two channels.
struct alignas(16) Run {
    F2 A, H;
};

// x after the run
template <bool kSeqs>
__device__ __forceinline__ F2 run_apply(const Run& r, F2 x) {
    const F2 y = fma2(r.A, x, r.H);
    return kSeqs ? pick2(r.A.lo() < 0.f, r.H, y) : y;
}

// f followed by r
template <bool kSeqs>
__device__ __forceinline__ Run run_join(const Run& f, const Run& r) {
    Run o;
    o.H = run_apply<kSeqs>(r, f.H);
    o.A = mul2(f.A, r.A);
    if (kSeqs) o.A = pick2(r.A.lo() < 0.f || f.A.lo() < 0.f, f2(kReset), o.A);
    return o;
}

// A warp's joined runs, behind the groups' own: what came before a group in its warp.
template <int kGroups, bool kSeqs>
__device__ __forceinline__ Run join_groups(Run& run, int lane) {
    constexpr int n = 32 / kGroups;
    auto up = [&](const Run& r, int by) {
        return Run{F2{__shfl_up_sync(0xffffffffu, r.A.v, by)}, F2{__shfl_up_sync(0xffffffffu, r.H.v, by)}};
    };
#pragma unroll
    for (int by = n; by < 32; by *= 2) {
        const Run f = up(run, by);
        if (lane >= by) run = run_join<kSeqs>(f, run);
    }
    const Run before = up(run, n);
    return lane >= n ? before : Run{f2(1.f), f2(0.f)};
}

// In a single block runs go by tile modulo four: between the readings of tile k, behind the
// barrier of its step, and the writing of tile k + 4 lies another step's barrier.  In a cluster
// they go by tile parity: a worker forms tile k + 2 once it has the state of tile k, and the folder
// has read that tile's runs by then.  Blocks' runs go by tile modulo four: a block sends tile j
// when its workers have the states of tile j - 2, for which every block has sent tile j - 2, and so
// has folded tile j - 4.
//
// A block whose wait has run out is late, and stays so.  Its folder then neither waits nor arms a
// barrier; it hands NaN to the workers and keeps it as the state, so that every value that misses a
// run is NaN and no wrong one is written.  Its publisher sends nothing more, since it is no longer
// bound to the order above; the other blocks miss its runs and become late in turn.
template <int kWarps, bool kCluster>
struct alignas(128) ScanShared {
    Run run[kCluster ? 2 : 4][kWarps][32];
    F2 before[kCluster ? 2 : 1][kCluster ? kWarps : 1][32];
    Run block[kCluster ? 4 : 1][kScanMaxCluster][32];
    alignas(128) uint64_t full[4];   // bytes of block[] that have come
    volatile int late;
};

// A single block's walk over the row's tiles.  E holds a lane's elements of a tile; form(k, e)
// makes them and returns the run, finish(k, e, x) uses them with the state x before it.  `carry`
// goes from the state before the row's first token to the one behind its last.
template <bool kSeqs, typename E, int kWarps, typename Form, typename Finish>
__device__ __forceinline__ void scan_walk(ScanShared<kWarps, false>& sh, int steps, int wid, int lane,
                                          F2& carry, Form form, Finish finish) {
    auto turn = [&](int k, E& now, E& next) {
        if (k + 1 < steps) sh.run[(k + 1) & 3][wid][lane] = form(k + 1, next);
        __syncthreads();
        F2 x = carry;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == wid) x = carry;
            carry = run_apply<kSeqs>(sh.run[k & 3][w][lane], carry);
        }
        finish(k, now, x);
    };
    E even, odd;
    sh.run[0][wid][lane] = form(0, even);
    __syncthreads();
    for (int k = 0; k < steps; k += 2) {
        turn(k, even, odd);
        if (k + 1 < steps) turn(k + 1, odd, even);
    }
}

// The blocks' named barriers: tile k's runs are formed (kFormed + parity), the states before them
// are there (kFolded + parity).
enum { kFormed = 1, kFolded = 3 };
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Waits, for two seconds at most, until every block's run of tile k is here.
__device__ __forceinline__ bool runs_here(uint64_t* bar_, uint32_t parity) {
    const uint32_t bar = smem_u32(bar_);
    auto ready = [&](uint32_t ns) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(ns) : "memory");
        return ok != 0;
    };
    if (ready(1000u)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!ready(1000000u))
        if (globaltimer_ns() - t0 > kScanWaitNs) return false;
    return true;
}

// A worker's walk in a cluster.  form returns the warp's joined runs in the last group, e.before
// what came before the lane's group.
template <int kGroups, bool kSeqs, typename E, int kWarps, typename Form, typename Finish>
__device__ __forceinline__ void scan_work(ScanShared<kWarps, true>& sh, int steps, int wid, int lane,
                                          Form form, Finish finish) {
    const int formed = blockDim.x, folded = 32 * (kWarps + 1);
    constexpr int n = 32 / kGroups;
    auto give = [&](int k, E& e) {
        const Run run = form(k, e);
        if (lane >= 32 - n) sh.run[k & 1][wid][lane - (32 - n)] = run;
        bar_arrive(kFormed + (k & 1), formed);
    };
    auto turn = [&](int k, E& now, E& next) {
        if (k + 1 < steps) give(k + 1, next);
        bar_sync(kFolded + (k & 1), folded);
        F2 x = sh.before[k & 1][wid][lane % n];
        if (kGroups > 1) x = run_apply<kSeqs>(now.before, x);
        finish(k, now, x);
    };
    E even, odd;
    give(0, even);
    for (int k = 0; k < steps; k += 2) {
        turn(k, even, odd);
        if (k + 1 < steps) turn(k + 1, odd, even);
    }
}

// The folder's walk.  False if a wait ran out; the walk then goes on, late, so that all threads meet
// at the barriers.
template <int kGroups, bool kSeqs, int kWarps>
__device__ __forceinline__ bool scan_fold(ScanShared<kWarps, true>& sh, int steps, int cluster, int rank,
                                          int lane, F2& carry) {
    bool ok = true;
    for (int k = 0; k < steps; ++k) {
        const int par = k & 1;
        bar_sync(kFormed + par, blockDim.x);
        uint64_t* full = &sh.full[k & 3];
        if (ok && lane == 0)
            mbar_expect_tx(full, (uint32_t)cluster * (32 / kGroups) * sizeof(Run));
        // the maps from the block's first token to every worker, while the other blocks' runs come
        Run to[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) to[w] = sh.run[par][w][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) to[w] = run_join<kSeqs>(to[w - 1], to[w]);
        if (ok) ok = __all_sync(0xffffffffu, runs_here(full, (uint32_t)(k >> 2) & 1u));
        if (!ok) {
            sh.late = 1;
            __threadfence_block();  // before a worker overwrites what the publisher may be reading
            carry = f2(__int_as_float(0x7fffffff));
        }
        F2 x = carry;
        Run blocks[kScanMaxCluster];
#pragma unroll
        for (int r = 0; r < kScanMaxCluster; ++r) blocks[r] = sh.block[k & 3][r][lane];
#pragma unroll
        for (int r = 0; r < kScanMaxCluster; ++r) {
            if (r == rank) x = carry;
            if (r < cluster && ok) carry = run_apply<kSeqs>(blocks[r], carry);
        }
        sh.before[par][0][lane] = x;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) sh.before[par][w][lane] = run_apply<kSeqs>(to[w - 1], x);
        bar_arrive(kFolded + par, 32 * (kWarps + 1));
    }
    return ok;
}

// The publisher's walk: joins the block's runs of every tile and sends them to all blocks.
template <int kGroups, bool kSeqs, int kWarps>
__device__ __forceinline__ void scan_publish(ScanShared<kWarps, true>& sh, int steps, int cluster, int rank,
                                             int lane) {
    for (int k = 0; k < steps; ++k) {
        bar_sync(kFormed + (k & 1), blockDim.x);
        const Run(&r)[kWarps][32] = sh.run[k & 1];
        Run all = r[0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) all = run_join<kSeqs>(all, r[w][lane]);
        const uint32_t to = smem_u32(&sh.block[k & 3][rank][lane]), bar = smem_u32(&sh.full[k & 3]);
        __threadfence_block();
        if (lane >= 32 / kGroups || sh.late) continue;
        for (int b = 0; b < cluster; ++b)
            asm volatile(
                "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                ::"r"(cluster_map(to, b)), "f"(all.A.lo()), "f"(all.A.hi()), "f"(all.H.lo()),
                "f"(all.H.hi()), "r"(cluster_map(bar, b))
                : "memory");
    }
}

// The blocks of a cluster start together, their barriers ready, and end together, so that nothing
// is sent to a block that is gone.  A late block has not waited for what was sent to it: its folder
// stays until that has come.
template <int kWarps, bool kCluster>
__device__ __forceinline__ void scan_open(ScanShared<kWarps, kCluster>& sh) {
    if (!kCluster) return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&sh.full[i], 1);
        sh.late = 0;
        mbar_init_fence();
    }
    __syncwarp();
    cluster_sync_all();
}
template <bool kCluster>
__device__ __forceinline__ void scan_close(bool late = false) {
    if (!kCluster) return;
    __syncwarp();
    cluster_sync_all();
    if (late) __nanosleep(1000000u);
}

// ---- feeding -----------------------------------------------------------------------------------
// How rows are copied: 16 bytes a lane where rows are whole 16-byte words; a lane's own two
// channels (4 or 8 bytes) where D is even; else through registers, one element at a time.
enum Copy { kCopy16, kCopyPair, kCopyOne };

// A warp's kSeg * kGroups rows of kSlab / kGroups channels of one tensor in shared memory, the rows
// of a group behind a row's width of padding, so that the groups read different banks.
template <typename E, int kSeg, int kGroups>
struct Rows {
    static constexpr int kRow = kSlab / kGroups * (int)sizeof(E);
    static constexpr int kPad = kGroups > 1 ? kRow : 0;
    static constexpr int kBytes = kGroups * (kSeg * kRow + kPad);
    static __device__ __forceinline__ F2 read(const char* p, int i, int lane) {
        constexpr int n = 32 / kGroups;
        const char* q = p + lane / n * (kSeg * kRow + kPad) + i * kRow + lane % n * 2 * (int)sizeof(E);
        if constexpr (sizeof(E) == 2) {
            const uint32_t r = *reinterpret_cast<const uint32_t*>(q);
            return f2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
        } else {
            return F2{*reinterpret_cast<const uint64_t*>(q)};
        }
    }
};

// Copies a warp's rows of one tensor, tile after tile.  Place 0 of a row's order is token
// `origin`, and the order goes up or (dir = -1) down the tokens; places at or behind L are zero.
template <typename E, Copy kCopy, int kSeg, int kGroups>
struct Feed {
    using R = Rows<E, kSeg, kGroups>;
    static constexpr int kWidth = kSlab / kGroups;            // channels
    static constexpr int kEls = kCopy == kCopy16 ? 16 / (int)sizeof(E) : 2;
    static constexpr int kPerRow = kWidth / kEls;             // lanes of a row
    static constexpr int kRows = 32 / kPerRow;                // rows of one pass of the warp
    static constexpr int kPasses = kSeg * kGroups / kRows;
    static_assert(kSeg * kGroups % kRows == 0 && (kSeg % kRows == 0 || kRows % kSeg == 0),
                  "a pass copies whole rows of a run, or of several");
    const E* at;        // the lane's part of its first row of the next tile
    long long pass;     // elements from a pass to the next
    uint32_t dst;       // the lane's place in a stage
    int row, left;

    static __device__ __forceinline__ constexpr int pass_bytes(int m) {
        return m * kRows * R::kRow + m * kRows / kSeg * R::kPad;
    }
    // src: the slab's first channel of the row's first token; `first`: the place of the warp's
    // first row; left: channels of the slab
    __device__ __forceinline__ void open(const E* src, int origin, int dir, long long first, int D,
                                         int channels, int lane) {
        row = lane / kPerRow;
        const int col = lane % kPerRow * kEls;
        left = channels < kWidth ? channels - col : kWidth;
        at = src + (origin + dir * (first + row)) * D + col;
        pass = (long long)dir * kRows * D;
        dst = (uint32_t)(row * R::kRow + row / kSeg * R::kPad + col * (int)sizeof(E));
    }
    // `place`: the tile's first row of this warp; hop: elements to the next tile
    __device__ __forceinline__ void tile(char* stage, int place, int L, long long hop) {
        const E* p = at;
        at += hop;
        if constexpr (kCopy == kCopyOne) {
            E r[kPasses][2];
#pragma unroll
            for (int m = 0; m < kPasses; ++m) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    r[m][j] = j < left && place + row + m * kRows < L ? p[j] : from_f<E>(0.f);
                p += pass;
            }
#pragma unroll
            for (int m = 0; m < kPasses; ++m) {
                E* q = reinterpret_cast<E*>(stage + dst + pass_bytes(m));
                q[0] = r[m][0];
                q[1] = r[m][1];
            }
        } else {
            const uint32_t q = smem_u32(stage) + dst;
#pragma unroll
            for (int m = 0; m < kPasses; ++m) {
                copy_async<kEls * (int)sizeof(E)>(q + pass_bytes(m), p,
                                                  left > 0 && place + row + m * kRows < L);
                p += pass;
            }
        }
    }
};

// Writes a lane's two channels of one token (left: channels from the lane's first on).
template <typename E, Copy kCopy>
__device__ __forceinline__ void store_pair(E* p, F2 f, int left) {
    if constexpr (kCopy != kCopyOne) {
        const float x[2] = {f.lo(), f.hi()};
        if (left > 0) store_vec<E, 2>(p, x);
    } else {
        if (left > 0) p[0] = from_f<E>(f.lo());
        if (left > 1) p[1] = from_f<E>(f.hi());
    }
}

// A lane's two channels of a state row, which may be the row that the kernel writes.
template <Copy kCopy>
__device__ __forceinline__ F2 load_state(const float* p, int left) {
    float f[2] = {0.f, 0.f};
    if constexpr (kCopy != kCopyOne) {
        if (left > 0) {
            const Vec<float, 2> v = load_in_place<float, 2>(p);
            f[0] = v.x[0];
            f[1] = v.x[1];
        }
    } else {
        if (left > 0) f[0] = p[0];
        if (left > 1) f[1] = p[1];
    }
    return f2(f[0], f[1]);
}

// ---- sequences of a row ------------------------------------------------------------------------

// Bounds of up to this many sequences are kept in shared memory.
constexpr int kCuShared = 1024;
constexpr size_t kCuBytes = sizeof(int32_t) * (kCuShared + 32);

// The call's sequences, with their bounds in shared memory if they fit.  All threads of the block.
__device__ __forceinline__ Seqs share_cu(Seqs q, int32_t* room) {
    if (q.cu && q.n <= kCuShared) {
        for (int s = threadIdx.x; s <= q.n; s += blockDim.x) room[s] = q.cu[s];
        q.cu = room;
    }
    __syncthreads();
    return q;
}

// Calls f(s) in all lanes of a warp for the warp's share of the empty sequences.
template <typename F>
__device__ __forceinline__ void each_empty(const Seqs& q, int wid, int warps, int lane, F f) {
    if (!q.cu) return;  // rows of at least a token
    for (long long s0 = wid * 32; s0 < q.n; s0 += warps * 32) {
        const int s = (int)s0 + lane;
        unsigned m = __ballot_sync(0xffffffffu, s0 + lane < q.n && q.begin(s) == q.end(s));
        for (; m; m &= m - 1) f((int)s0 + __ffs(m) - 1);
    }
}

// Which of a warp's rows start or end a sequence, in the kernel's order, and (in lane i) the
// sequence of row i.
struct Marks {
    unsigned start, end;
    int seq;
    __device__ __forceinline__ bool any() const { return (start | end) != 0; }
};

// The sequence met last, so that rows inside one sequence need no search.
struct Here {
    int b, e;
};

// n rows from place `first` on
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

// A lane's share of the marks: whether token i of its run starts or ends a sequence, and that
// sequence.  All lanes of the warp.
template <int kSeg>
struct Mark {
    unsigned start, end;  // of the lane's run
    int base;
    __device__ __forceinline__ Mark(const Marks& m, int group) : base(group * kSeg) {
        start = m.start >> base;
        end = m.end >> base;
    }
    __device__ __forceinline__ bool starts(int i) const { return start >> i & 1u; }
    __device__ __forceinline__ bool ends(int i) const { return end >> i & 1u; }
    __device__ __forceinline__ int seq(const Marks& m, int i) const {
        return __shfl_sync(0xffffffffu, m.seq, base + i);
    }
    __device__ __forceinline__ bool any_start() const { return (start & ((1u << kSeg) - 1)) != 0; }
};

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

// How a call is laid out.  Many slabs of 64 channels: a block each, two on an SM (cluster 0).  Few:
// clusters, one block on an SM, of slabs so wide (groups) and of so many blocks that the walk takes
// the fewest steps; a step takes about the same time in all of them.  The blocks of a cluster are
// in one part of the GPU: the occupancy query counts 148 clusters of 1 block, 74 of 2, 45 of 3, 33
// of 4, 26 of 5, 22 of 6 and 15 of 7 or 8.
struct ScanPlan {
    int groups, cluster;
};
inline ScanPlan scan_plan(int D, long long rows, long long L, int block_rows, int single_from) {
    static const unsigned char most[kScanMaxCluster + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
    if ((D + kSlab - 1) / kSlab * rows >= single_from) return {1, 0};
    ScanPlan best{1, 0};
    long long fewest = -1;
    for (int g = 1; g <= 4; g *= 2) {
        const long long units = (D + kSlab / g - 1) / (kSlab / g) * rows;
        for (int c = 1; c <= kScanMaxCluster; ++c) {
            if (units > most[c]) break;
            const long long stride = (long long)block_rows * g * c, steps = (L + stride - 1) / stride;
            if (fewest < 0 || steps < fewest) { fewest = steps; best = {g, c}; }
        }
    }
    return best;
}

template <typename P>
gdr_status scan_launch(void (*kernel)(P, int), const P& p, long long units, int cluster, int threads,
                       size_t smem, cudaStream_t st) {
    if (units * cluster > 0x7fffffffLL) return GDR_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return GDR_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(threads);
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

template <typename Op, typename IO>
gdr_status scan_dispatch_gate(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    return a.gate_dtype == GDR_BF16 ? scan_dispatch_write<Op, IO, __nv_bfloat16>(a, x, st)
                                    : scan_dispatch_write<Op, IO, float>(a, x, st);
}

template <int kValue>
struct Int {
    static constexpr int value = kValue;
};

}  // namespace gdr
