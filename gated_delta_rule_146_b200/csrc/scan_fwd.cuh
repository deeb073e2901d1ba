// scan_fwd.cuh -- gated linear recurrence: the forward kernel over whole sequences.
//
//     h_t = alpha_t h_{t-1} + b_t,   alpha = exp(g),   b = v | beta v | (1 - alpha) v,   o = h
//
// Every element is read and written once (6 bytes per token and channel in bf16, 8 with beta),
// for about twenty instructions a pair of channels: HBM bounds it.  8 x 4096 x 2048 in bf16 with
// beta takes 86 us, 95 % of the copy rate; tied (98 to 102 us, 62 %) the instructions of 1 - e^g
// bound it.  Clusters come to 75 % (131072 x 1024, plain: 164 us): with one block on an SM nothing
// covers the barriers and dependent instructions of a step, at 55 % of the issue slots of the 128
// SMs they fill.  Packed sequences add the work at their bounds (32768 x 1024: 47 us as one, 65 in
// 32).  The split is described in scan_impl.cuh.
#pragma once

#include "scan_impl.cuh"

namespace gdr {

namespace {

// Two tiles ahead.  More bytes in flight cost: with three tiles ahead the training shape takes 97
// instead of 86 us (beta given), with one 95.
constexpr int kStages = 3;

// Tokens of a warp's run: eight in bf16, four where fp32 doubles the bytes of a tile.
template <typename IO, typename GT>
constexpr int seg_of = sizeof(IO) + sizeof(GT) > 4 ? 4 : 8;

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

template <typename IO, typename GT, int kWrite, int kGroups>
constexpr int stage_bytes = Rows<IO, seg_of<IO, GT>, kGroups>::kBytes +
                            (kWrite == GDR_WRITE_GATE ? 2 : 1) * Rows<GT, seg_of<IO, GT>, kGroups>::kBytes;

// A lane's elements of a tile, from the forming of its run to the output.
template <int kSeg>
struct Elements {
    F2 a[kSeg], b[kSeg];
    Run before;   // what came before the lane's group in its warp
    Marks m;
};

// kSeqs: one row holds all sequences, whose starts reset the state; else a row is a sequence.
// kLayout: 0 for a single block, else the groups of lanes of a block in a cluster.
template <typename IO, typename GT, int kWrite, Copy kCopy, bool kSeqs, int kLayout, int kWarps>
__global__ void __launch_bounds__(32 * (kWarps + 2 * (kLayout > 0)), kLayout > 0 ? 1 : 2)
scan_fwd_kernel(const FwdParams<IO, GT> p, const int cluster) {
    extern __shared__ __align__(128) char smem[];
    constexpr bool kCluster = kLayout > 0;
    constexpr int kGroups = kCluster ? kLayout : 1, kLanes = 32 / kGroups;
    using Shared = ScanShared<kWarps, kCluster>;
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    char* const stages = smem + sizeof(sh) + (kSeqs ? kCuBytes : 0);
    constexpr int kSeg = seg_of<IO, GT>, kRows = kGroups * kSeg, kTile = kWarps * kRows;
    constexpr int kStage = stage_bytes<IO, GT, kWrite, kGroups>, kWidth = kSlab / kGroups;
    using RowsIO = Rows<IO, kSeg, kGroups>;
    using RowsGT = Rows<GT, kSeg, kGroups>;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = blockIdx.x % cluster;
    const int unit = blockIdx.x / cluster;
    const int slab = unit % p.slabs, row = unit / p.slabs;
    const int left = p.D - slab * kWidth;      // channels from the slab's first on
    const int group = lane / kLanes, c = slab * kWidth + 2 * (lane % kLanes), mine = p.D - c;
    const int L = p.L, D = p.D;
    const int origin = p.reverse ? L - 1 : 0, dir = p.reverse ? -1 : 1;

    F2 carry = f2(0.f);  // the folder's; read before any block can write h_final
    if (!kSeqs && (!kCluster || wid == kWarps) && p.h0)
        carry = load_state<kCopy>(p.h0 + (size_t)row * D + c, mine);
    Seqs seqs = p.q;
    if constexpr (kSeqs) seqs = share_cu(p.q, reinterpret_cast<int32_t*>(smem + sizeof(sh)));
    scan_open(sh);
    if (kSeqs && blockIdx.x == 0) check_cu(seqs, p.status, tid, 32 * (kWarps + 2 * kCluster));
    if (kSeqs && rank == 0 && p.h_final)  // empty sequences keep their state
        each_empty(seqs, wid, kWarps + 2 * kCluster, lane, [&](int s) {
            const F2 x = p.h0 ? load_state<kCopy>(p.h0 + (size_t)s * D + c, mine) : f2(0.f);
            store_pair<float, kCopy>(p.h_final + (size_t)s * D + c, x, mine);
        });

    const size_t base = (size_t)row * L * D + slab * kWidth;
    const int stride = cluster * kTile, first0 = rank * kTile + wid * kRows;
    const int steps = (int)(((long long)L + stride - 1) / stride);
    const long long hop = (long long)dir * stride * D;  // elements from a tile to the next
    char* const buf = stages + wid * kStages * kStage;
    Feed<IO, kCopy, kSeg, kGroups> fv;
    Feed<GT, kCopy, kSeg, kGroups> fg, fb;
    fv.open(p.v + base, origin, dir, first0, D, left, lane);
    fg.open(p.g + base, origin, dir, first0, D, left, lane);
    if constexpr (kWrite == GDR_WRITE_GATE) fb.open(p.beta + base, origin, dir, first0, D, left, lane);
    // The tiles walk on past L by at most kStages steps: L is bounded so that no place overflows.
    auto feed = [&](int k, int stage) {
        char* s = buf + stage * kStage;
        const int place = k < steps ? first0 + k * stride : L;
        fv.tile(s, place, L, hop);
        fg.tile(s + RowsIO::kBytes, place, L, hop);
        if constexpr (kWrite == GDR_WRITE_GATE)
            fb.tile(s + RowsIO::kBytes + RowsGT::kBytes, place, L, hop);
        copy_commit();
    };
    if constexpr (kCluster) if (wid >= kWarps) {
        bool ok = true;
        if (wid > kWarps) {
            scan_publish<kGroups, kSeqs>(sh, steps, cluster, rank, lane);
        } else {
            ok = scan_fold<kGroups, kSeqs>(sh, steps, cluster, rank, lane, carry);
            if (!ok && p.status && lane == 0) atomicCAS(p.status, (int)GDR_OK, (int)GDR_ERR_TIMEOUT);
            if (!kSeqs && p.h_final && rank == 0 && group == 0)
                store_pair<float, kCopy>(p.h_final + (size_t)row * D + c, carry, mine);
        }
        scan_close<kCluster>(!ok);
        return;
    }
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) feed(k, k);

    Here here{0, 0};
    int stage = 0;  // of the next tile to be formed
    auto form = [&](int k, Elements<kSeg>& e) -> Run {
        copy_wait<kStages - 2>();
        __syncwarp();
        // into the stage of the tile before: every lane has read it
        feed(k + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        const char* s = buf + stage * kStage;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if constexpr (kSeqs) {
            const int first = first0 + k * stride;
            e.m = find_marks(seqs, here, origin, dir, first, min(kRows, L - first), lane);
        }
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            const F2 v = RowsIO::read(s, i, lane), g = RowsGT::read(s + RowsIO::kBytes, i, lane);
            e.a[i] = exp2ch(g);
            if constexpr (kWrite == GDR_WRITE_GATE)
                e.b[i] = mul2(RowsGT::read(s + RowsIO::kBytes + RowsGT::kBytes, i, lane), v);
            else if constexpr (kWrite == GDR_WRITE_TIED)
                e.b[i] = mul2(one_minus(g, e.a[i]), v);
            else
                e.b[i] = v;
        }
        const Mark<kSeg> mark(e.m, group);
        if (kSeqs && e.m.start && p.h0) {  // b at a start takes the initial state in
#pragma unroll
            for (int i = 0; i < kSeg; ++i) {
                const int q = mark.seq(e.m, i);
                if (mark.starts(i))
                    e.b[i] = fma2(e.a[i], load_state<kCopy>(p.h0 + (size_t)q * D + c, mine), e.b[i]);
            }
        }
        Run run{e.a[0], e.b[0]};
        if (!kSeqs || !e.m.start) {
#pragma unroll
            for (int i = 1; i < kSeg; ++i) {
                run.H = fma2(e.a[i], run.H, e.b[i]);
                run.A = mul2(run.A, e.a[i]);
            }
        } else {
#pragma unroll
            for (int i = 1; i < kSeg; ++i) {
                run.H = pick2(mark.starts(i), e.b[i], fma2(e.a[i], run.H, e.b[i]));
                run.A = mul2(run.A, e.a[i]);
            }
            if (mark.any_start()) run.A = f2(kReset);
        }
        if constexpr (kGroups > 1) e.before = join_groups<kGroups, kSeqs>(run, lane);
        return run;
    };

    const long long next = (long long)dir * D;
    IO* out = p.o + base + (origin + (long long)dir * (first0 + group * kSeg)) * D + 2 * (lane % kLanes);
    auto finish = [&](int k, const Elements<kSeg>& e, F2 h) {
        const int rest = L - (first0 + k * stride), n = rest - group * kSeg;
        IO* q = out;
        out += hop;
        if (rest >= kRows && !(kSeqs && e.m.any())) {
#pragma unroll
            for (int i = 0; i < kSeg; ++i, q += next) {
                h = fma2(e.a[i], h, e.b[i]);
                store_pair<IO, kCopy>(q, h, mine);
            }
            return;
        }
        const Mark<kSeg> mark(e.m, group);
#pragma unroll
        for (int i = 0; i < kSeg; ++i, q += next) {
            const F2 y = fma2(e.a[i], h, e.b[i]);
            h = kSeqs ? pick2(mark.starts(i), e.b[i], y) : y;
            if (i < n) store_pair<IO, kCopy>(q, h, mine);
            if (kSeqs && e.m.end && p.h_final) {
                const int s = mark.seq(e.m, i);
                if (mark.ends(i)) store_pair<float, kCopy>(p.h_final + (size_t)s * D + c, h, mine);
            }
        }
    };
    if constexpr (kCluster) {
        scan_work<kGroups, kSeqs, Elements<kSeg>>(sh, steps, wid, lane, form, finish);
    } else {
        scan_walk<kSeqs, Elements<kSeg>>(sh, steps, wid, lane, carry, form, finish);
        if (!kSeqs && p.h_final && wid == 0)
            store_pair<float, kCopy>(p.h_final + (size_t)row * D + c, carry, mine);
    }
    copy_wait<0>();
    scan_close<kCluster>();
}

// Slabs times rows from which single blocks are faster than clusters of one: with 128 of them and
// beta 100 us against 118 (2 x 8192 x 4096 in bf16), with 75 of them 43 against 41 (15 x 2677 x
// 296), and copied one by one 96 against 147 (15 x 2677 x 291).
constexpr int kSingleFrom = 112, kSingleOne = 75;

template <typename IO, typename GT, int kWrite, Copy kCopy>
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
    p.reverse = a.reverse;
    constexpr int kSeg = seg_of<IO, GT>;
    constexpr int kWide = 14;  // workers: with the two other warps 128 registers a thread (16: 96)
    const long long rows = seqs ? 1 : a.B;
    const ScanPlan plan = scan_plan(a.D, rows, p.L, kWide * kSeg,
                                    kCopy == kCopyOne ? kSingleOne : kSingleFrom);
    const int width = kSlab / plan.groups;
    p.slabs = (a.D + width - 1) / width;
    auto launch = [&](auto kernel, int warps, int threads, size_t stage, size_t shared) {
        return scan_launch(kernel, p, rows * p.slabs, plan.cluster ? plan.cluster : 1, threads,
                           warps * kStages * stage + shared + (seqs ? kCuBytes : 0), st);
    };
    auto in_cluster = [&](auto groups) {
        constexpr int g = decltype(groups)::value;
        constexpr size_t kStage = stage_bytes<IO, GT, kWrite, g>, kShared = sizeof(ScanShared<kWide, true>);
        return seqs ? launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, true, g, kWide>, kWide,
                             32 * (kWide + 2), kStage, kShared)
                    : launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, false, g, kWide>, kWide,
                             32 * (kWide + 2), kStage, kShared);
    };
    if (plan.cluster) {
        if (plan.groups == 1) return in_cluster(Int<1>{});
        if (plan.groups == 2) return in_cluster(Int<2>{});
        return in_cluster(Int<4>{});
    }
    constexpr size_t kStage = stage_bytes<IO, GT, kWrite, 1>, kShared = sizeof(ScanShared<8, false>);
    return seqs ? launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, true, 0, 8>, 8, 256, kStage, kShared)
                : launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, false, 0, 8>, 8, 256, kStage, kShared);
}

struct Fwd {
    template <typename IO, typename GT, int kWrite>
    static gdr_status go(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
        const Copy copy = scan_copy(a);
        if (copy == kCopy16) return fwd_launch<IO, GT, kWrite, kCopy16>(a, x, st);
        if constexpr (sizeof(IO) == sizeof(GT)) {
            if (copy == kCopyPair) return fwd_launch<IO, GT, kWrite, kCopyPair>(a, x, st);
        }
        return fwd_launch<IO, GT, kWrite, kCopyOne>(a, x, st);
    }
};

}  // namespace

// The forward for one type of v and o: a translation unit each.
template <typename IO>
gdr_status scan_fwd_io(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    return scan_dispatch_gate<Fwd, IO>(a, x, st);
}

}  // namespace gdr
