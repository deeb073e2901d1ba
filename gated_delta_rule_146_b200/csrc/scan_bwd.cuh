// scan_bwd.cuh -- gated linear recurrence: backward pass.
//
// With m_t = alpha_t lam_t the adjoint runs from the last token to the first,
//     lam_t = dO_t + m_{t+1},   m_t = alpha_t lam_t,
// again a recurrence of maps m -> A m + H with the same A, split and joined as in the forward
// (scan_impl.cuh).  dg_t = m_t h_{t-1} reads h from the forward's output, so nothing is
// recomputed and every element is read and written once: 10 (plain), 12 (tied) or 16 (gate)
// bytes per token and channel in bf16.  HBM bounds it: 8 x 4096 x 2048 in bf16 with beta takes 174
// to 182 us, 90 to 94 % of the copy rate.  Clusters wait at the barriers of a step and on dependent
// instructions (52 % of the issue slots of the 120 SMs they fill): 49157 packed tokens x 768, plain,
// 143 us, 40 %.
#pragma once

#include "scan_impl.cuh"

namespace gdr {

namespace {

// Stages of the two rings.  The second is a step ahead; how far the first may be was measured on
// 8 x 4096 x 2048 in bf16: plain 120 us one tile ahead, 136 two; with beta 211 and 186 (two tiles
// ahead leave room for one block on an SM instead of two).  More bytes in flight than the memory
// system takes in order cost time.
template <int kWrite>
constexpr int early_stages = kWrite == GDR_WRITE_GATE ? 3 : 2;
constexpr int kLateStages = 2;

// Tokens of a warp's run: eight in single blocks in bf16, four where fp32 doubles the bytes or the
// sixteen warps of a cluster's block share the registers.
template <typename IO, typename GT>
constexpr int seg_of(bool cluster) { return !cluster && sizeof(IO) + sizeof(GT) == 4 ? 8 : 4; }

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

// A warp's tokens in shared memory, in two rings: g and dO of a tile are read when its run is
// formed, o of the token before, v and beta a step later, when it is finished.
template <typename IO, typename GT, int kWrite, int kSeg, int kGroups>
struct Ring {
    static constexpr int kG = Rows<GT, kSeg, kGroups>::kBytes, kI = Rows<IO, kSeg, kGroups>::kBytes;
    static constexpr int kEarly = kG + kI;
    static constexpr int v = kI, beta = v + kI;  // behind o
    static constexpr int kLate = kWrite == GDR_WRITE_GATE ? beta + kG
                               : kWrite == GDR_WRITE_TIED ? beta : v;
    static constexpr int kEarlyStages = early_stages<kWrite>;
    static constexpr int kBytes = kEarlyStages * kEarly + kLateStages * kLate;
};

template <int kWrite, int kSeg>
struct Elements {
    F2 a[kSeg], d[kSeg];           // alpha; dO, with dh_final at a sequence's last token
    F2 w[kWrite == GDR_WRITE_TIED ? kSeg : 1];
    Run before;                    // what came before the lane's group in its warp
    Marks m;                       // start: the last token of a sequence, end: its first
};

// kLayout: 0 for a single block, else the groups of lanes of a block in a cluster.
template <typename IO, typename GT, int kWrite, Copy kCopy, bool kSeqs, int kLayout, int kWarps>
__global__ void __launch_bounds__(32 * (kWarps + 2 * (kLayout > 0)), kLayout > 0 ? 1 : 2)
scan_bwd_kernel(const BwdParams<IO, GT> p, const int cluster) {
    extern __shared__ __align__(128) char smem[];
    constexpr bool kCluster = kLayout > 0;
    constexpr int kGroups = kCluster ? kLayout : 1, kLanes = 32 / kGroups;
    using Shared = ScanShared<kWarps, kCluster>;
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    char* const stages = smem + sizeof(sh) + (kSeqs ? kCuBytes : 0);
    constexpr int kSeg = seg_of<IO, GT>(kCluster), kRows = kGroups * kSeg, kTile = kWarps * kRows;
    constexpr int kWidth = kSlab / kGroups;
    using RowsIO = Rows<IO, kSeg, kGroups>;
    using RowsGT = Rows<GT, kSeg, kGroups>;
    using R = Ring<IO, GT, kWrite, kSeg, kGroups>;
    constexpr int kEarlyStages = R::kEarlyStages;
    using Els = Elements<kWrite, kSeg>;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = blockIdx.x % cluster;
    const int unit = blockIdx.x / cluster;
    const int slab = unit % p.slabs, row = unit / p.slabs;
    const int left = p.D - slab * kWidth;      // channels from the slab's first on
    const int group = lane / kLanes, c = slab * kWidth + 2 * (lane % kLanes), mine = p.D - c;
    const int L = p.L, D = p.D;
    // the adjoint's order: the forward's, backwards
    const int origin = p.reverse ? 0 : L - 1, dir = p.reverse ? 1 : -1;

    F2 carry = f2(0.f), h0_row = f2(0.f);  // the folder's, the workers'
    if (!kSeqs && (!kCluster || wid == kWarps) && p.dh_final)
        carry = load_state<kCopy>(p.dh_final + (size_t)row * D + c, mine);
    Seqs seqs = p.q;
    if constexpr (kSeqs) seqs = share_cu(p.q, reinterpret_cast<int32_t*>(smem + sizeof(sh)));
    scan_open(sh);
    if (kSeqs && blockIdx.x == 0) check_cu(seqs, p.status, tid, 32 * (kWarps + 2 * kCluster));
    if (kSeqs && rank == 0 && p.dh0)  // the state's gradient passes an empty sequence unchanged
        each_empty(seqs, wid, kWarps + 2 * kCluster, lane, [&](int s) {
            const F2 x = p.dh_final ? load_state<kCopy>(p.dh_final + (size_t)s * D + c, mine) : f2(0.f);
            store_pair<float, kCopy>(p.dh0 + (size_t)s * D + c, x, mine);
        });

    const size_t base = (size_t)row * L * D + slab * kWidth;
    const int stride = cluster * kTile, first0 = rank * kTile + wid * kRows;
    const int steps = (int)(((long long)L + stride - 1) / stride);
    const long long hop = (long long)dir * stride * D;
    char* const early = stages + wid * R::kBytes;
    char* const late = early + kEarlyStages * R::kEarly;
    Feed<GT, kCopy, kSeg, kGroups> fg, fb;
    Feed<IO, kCopy, kSeg, kGroups> fd, fo, fv;
    fg.open(p.g + base, origin, dir, first0, D, left, lane);
    fd.open(p.dO + base, origin, dir, first0, D, left, lane);
    fo.open(p.o + base, origin, dir, first0 + 1, D, left, lane);
    if constexpr (kWrite != GDR_WRITE_PLAIN) fv.open(p.v + base, origin, dir, first0, D, left, lane);
    if constexpr (kWrite == GDR_WRITE_GATE) fb.open(p.beta + base, origin, dir, first0, D, left, lane);
    auto place_of = [&](int k) { return k < steps ? first0 + k * stride : L; };
    auto feed_early = [&](int k, int stage) {
        char* s = early + stage * R::kEarly;
        fg.tile(s, place_of(k), L, hop);
        fd.tile(s + R::kG, place_of(k), L, hop);
    };
    auto feed_late = [&](int k, int stage) {
        char* s = late + stage * R::kLate;
        fo.tile(s, place_of(k) + 1, L, hop);
        if constexpr (kWrite != GDR_WRITE_PLAIN) fv.tile(s + R::v, place_of(k), L, hop);
        if constexpr (kWrite == GDR_WRITE_GATE) fb.tile(s + R::beta, place_of(k), L, hop);
    };
    if constexpr (kCluster) if (wid >= kWarps) {
        bool ok = true;
        if (wid > kWarps) {
            scan_publish<kGroups, kSeqs>(sh, steps, cluster, rank, lane);
        } else {
            ok = scan_fold<kGroups, kSeqs>(sh, steps, cluster, rank, lane, carry);
            if (!ok && p.status && lane == 0) atomicCAS(p.status, (int)GDR_OK, (int)GDR_ERR_TIMEOUT);
        }
        scan_close<kCluster>(!ok);
        return;
    }
    // copy group k: the first ring's tile k, with the second's kEarlyStages - 1 tiles behind it
#pragma unroll
    for (int k = 0; k < kEarlyStages - 1; ++k) {
        feed_early(k, k);
        copy_commit();
    }

    if (!kSeqs && p.h0) h0_row = load_state<kCopy>(p.h0 + (size_t)row * D + c, mine);
    Here here{0, 0};
    int stage = 0;  // of the next tile to be formed
    auto form = [&](int k, Els& e) -> Run {
        copy_wait<kEarlyStages - 2>();
        __syncwarp();
        // into the stages of tiles k - 1 and k - 2, which every lane has read
        feed_early(k + kEarlyStages - 1, stage == 0 ? kEarlyStages - 1 : stage - 1);
        feed_late(k, k & 1);
        copy_commit();
        const char* s = early + stage * R::kEarly;
        stage = stage == kEarlyStages - 1 ? 0 : stage + 1;
        if constexpr (kSeqs) {
            const int first = first0 + k * stride;
            e.m = find_marks(seqs, here, origin, dir, first, min(kRows, L - first), lane);
        }
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            const F2 g = RowsGT::read(s, i, lane);
            e.a[i] = exp2ch(g);
            if constexpr (kWrite == GDR_WRITE_TIED) e.w[i] = one_minus(g, e.a[i]);
            e.d[i] = RowsIO::read(s + R::kG, i, lane);
        }
        const Mark<kSeg> mark(e.m, group);
        if (kSeqs && e.m.start && p.dh_final) {
#pragma unroll
            for (int i = 0; i < kSeg; ++i) {
                const int q = mark.seq(e.m, i);
                if (mark.starts(i))
                    e.d[i] = add2(e.d[i], load_state<kCopy>(p.dh_final + (size_t)q * D + c, mine));
            }
        }
        Run run{e.a[0], mul2(e.a[0], e.d[0])};
        if (!kSeqs || !e.m.start) {
#pragma unroll
            for (int i = 1; i < kSeg; ++i) {
                run.H = mul2(e.a[i], add2(e.d[i], run.H));
                run.A = mul2(run.A, e.a[i]);
            }
        } else {
#pragma unroll
            for (int i = 1; i < kSeg; ++i) {
                run.H = mul2(e.a[i], pick2(mark.starts(i), e.d[i], add2(e.d[i], run.H)));
                run.A = mul2(run.A, e.a[i]);
            }
            if (mark.any_start()) run.A = f2(kReset);
        }
        if constexpr (kGroups > 1) e.before = join_groups<kGroups, kSeqs>(run, lane);
        return run;
    };

    const long long next = (long long)dir * D;
    long long out = (long long)base + (origin + (long long)dir * (first0 + group * kSeg)) * D +
                    2 * (lane % kLanes);
    auto finish = [&](int k, const Els& e, F2 mu) {
        // the second ring's tile k came in the group before the last; behind the last tile nothing
        // was formed
        if (k + 1 == steps) copy_wait<0>(); else copy_wait<1>();
        __syncwarp();
        const char* s = late + (k & 1) * R::kLate;
        const int rest = L - (first0 + k * stride), n = rest - group * kSeg;
        long long at = out;
        out += hop;
        // the gradients of token i of the run, at element `at`, h of the token before being hp
        auto element = [&](int i, F2 lam, F2 hp) {
            if constexpr (kWrite == GDR_WRITE_PLAIN) {
                store_pair<IO, kCopy>(p.dv + at, lam, mine);
            } else {
                const F2 v = RowsIO::read(s + R::v, i, lane);
                if constexpr (kWrite == GDR_WRITE_GATE) {
                    store_pair<GT, kCopy>(p.dbeta + at, mul2(lam, v), mine);
                    store_pair<IO, kCopy>(
                        p.dv + at, mul2(lam, RowsGT::read(s + R::beta, i, lane)), mine);
                } else {
                    hp = add2(hp, f2(-v.lo(), -v.hi()));
                    store_pair<IO, kCopy>(p.dv + at, mul2(e.w[i], lam), mine);
                }
            }
            store_pair<GT, kCopy>(p.dg + at, mul2(mu, hp), mine);
        };
        if (kSeqs ? rest >= kRows && !e.m.any() : rest > kRows) {  // no sequence ends here
#pragma unroll
            for (int i = 0; i < kSeg; ++i, at += next) {
                const F2 lam = add2(e.d[i], mu);
                mu = mul2(e.a[i], lam);
                element(i, lam, RowsIO::read(s, i, lane));
            }
            return;
        }
        const Mark<kSeg> mark(e.m, group);
#pragma unroll
        for (int i = 0; i < kSeg; ++i, at += next) {
            const bool ends = kSeqs ? mark.ends(i) : i == n - 1;
            const int q = kSeqs ? mark.seq(e.m, i) : row;
            const F2 sum = add2(e.d[i], mu);
            const F2 lam = kSeqs ? pick2(mark.starts(i), e.d[i], sum) : sum;
            mu = mul2(e.a[i], lam);
            if (i >= n) continue;
            F2 hp = RowsIO::read(s, i, lane);
            if (ends) {
                hp = h0_row;
                if (kSeqs && p.h0) hp = load_state<kCopy>(p.h0 + (size_t)q * D + c, mine);
                if (p.dh0) store_pair<float, kCopy>(p.dh0 + (size_t)q * D + c, mu, mine);
            }
            element(i, lam, hp);
        }
    };
    if constexpr (kCluster) {
        scan_work<kGroups, kSeqs, Els>(sh, steps, wid, lane, form, finish);
    } else {
        scan_walk<kSeqs, Els>(sh, steps, wid, lane, carry, form, finish);
    }
    copy_wait<0>();
    scan_close<kCluster>();
}

// Slabs times rows from which single blocks are faster than clusters of one.  With beta: with 128
// of them 172 us against 196 (2 x 8192 x 4096 in bf16), with 75 of them 68 against 59 (15 x 2677 x
// 296), copied one by one 168 against 211 (15 x 2677 x 291).  Tied, with 128 of them: 209 against
// 168 (4 x 8192 x 2048).
template <int kWrite>
constexpr int kSingleFrom = kWrite == GDR_WRITE_GATE ? 112 : 149;
constexpr int kSingleOne = 75;

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
    p.reverse = a.reverse;
    // 16 warps' rings fit an SM's shared memory in bf16 only
    constexpr int kWide = sizeof(IO) + sizeof(GT) == 4 ? 16 : 8;
    const long long rows = seqs ? 1 : a.B;
    const ScanPlan plan = scan_plan(a.D, rows, p.L, kWide * seg_of<IO, GT>(true),
                                    kCopy == kCopyOne ? kSingleOne : kSingleFrom<kWrite>);
    const int width = kSlab / plan.groups;
    p.slabs = (a.D + width - 1) / width;
    auto launch = [&](auto kernel, int warps, int threads, size_t ring, size_t shared) {
        return scan_launch(kernel, p, rows * p.slabs, plan.cluster ? plan.cluster : 1, threads,
                           warps * ring + shared + (seqs ? kCuBytes : 0), st);
    };
    auto in_cluster = [&](auto groups) {
        constexpr int g = decltype(groups)::value;
        constexpr size_t kRing = Ring<IO, GT, kWrite, seg_of<IO, GT>(true), g>::kBytes;
        constexpr size_t kShared = sizeof(ScanShared<kWide, true>);
        return seqs ? launch(scan_bwd_kernel<IO, GT, kWrite, kCopy, true, g, kWide>, kWide,
                             32 * (kWide + 2), kRing, kShared)
                    : launch(scan_bwd_kernel<IO, GT, kWrite, kCopy, false, g, kWide>, kWide,
                             32 * (kWide + 2), kRing, kShared);
    };
    if (plan.cluster) {
        if (plan.groups == 1) return in_cluster(Int<1>{});
        if (plan.groups == 2) return in_cluster(Int<2>{});
        return in_cluster(Int<4>{});
    }
    constexpr size_t kRing = Ring<IO, GT, kWrite, seg_of<IO, GT>(false), 1>::kBytes;
    constexpr size_t kShared = sizeof(ScanShared<8, false>);
    return seqs ? launch(scan_bwd_kernel<IO, GT, kWrite, kCopy, true, 0, 8>, 8, 256, kRing, kShared)
                : launch(scan_bwd_kernel<IO, GT, kWrite, kCopy, false, 0, 8>, 8, 256, kRing, kShared);
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

// The backward for one type of v and o: a translation unit each.
template <typename IO>
gdr_status scan_bwd_io(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    return scan_dispatch_gate<Bwd, IO>(a, x, st);
}

}  // namespace gdr
