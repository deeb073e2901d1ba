// norm.cu -- group norm of every token's heads with an activation or a gate: forward, backward;
// and the dispatch of the per-sequence form (norm_seq.cu).
//
//     n = (x - mean) rstd (or x rstd), u = n w + b, y = u act(z) | act(u)
//     dx = rstd (q - mean(q) - n mean(q n)),  q = du w      (mean(q) with centering only)
//
// A group's channels stay in one warp's registers: the statistics are two passes over registers
// (sums of squares about the mean, no cancellation), the tensors are read and written once: 4 or
// 6 (gate) bytes per element forward, 6 or 10 backward in bf16.  HBM bounds both with a gate: 8 x
// 4096 x 16 x 128 in bf16 takes 66 us forward and 113 to 119 backward, 94 and 86 to 91 % of the copy
// rate.  Without one: 59 and 100 us (54 and 84 without centering), 69 and 61 %: the activation waits
// for the row's statistics, so that a row is one chain of dependent instructions and shuffles.
//
// Each lane group keeps one head, so that weights, and in the backward the sums for dw and db,
// stay in registers over all its rows; the sums are joined over the block, then over the blocks
// by a second kernel, in a fixed order.
#include "norm_impl.cuh"

namespace gdr {

namespace {

// How the rows (token, head) are dealt out.  A slot is one lane group of one block; slot i takes
// rows i, i + slots, ...; slots is a multiple of H, so a slot's head stays.
struct Deal {
    int blocks;
    int used;          // lane groups of a block that take part
    long long slots;
    int part_rows;     // rows of partial sums
};

Deal deal(const gdr_norm_args& a, int groups, int resident, int per_slot) {
    const long long rows = (long long)a.B * a.T * a.H, most_blocks = 148LL * resident;
    Deal d;
    // the blocks fill the GPU once; a slot takes at least `per_slot` rows where there are so many,
    // so that partial sums stay a small share of the traffic
    if (a.H <= groups) {
        d.used = groups / a.H * a.H;
        const long long per = (long long)d.used * per_slot, b = (rows + per - 1) / per;
        d.blocks = (int)(b < 1 ? 1 : b > most_blocks ? most_blocks : b);
        d.slots = (long long)d.blocks * d.used;
        d.part_rows = d.blocks;
    } else {
        d.used = groups;
        long long per_head = rows / a.H / per_slot;
        const long long most = most_blocks * groups / a.H;
        if (per_head > most) per_head = most;
        if (per_head < 1) per_head = 1;
        d.slots = per_head * a.H;
        d.blocks = (int)((d.slots + groups - 1) / groups);
        d.part_rows = a.shared_weight ? d.blocks : (int)per_head;
    }
    return d;
}

// The row's centred values and 1 / deviation.
template <typename S>
__device__ __forceinline__ float token_stats(Pairs<S>& x, int l, int d, int center, float eps) {
    const float inv = 1.f / d;
    if (center) centre<S>(x, group_sum<S::LPG>(lane_sum<S>(x)) * inv, l, d);
    return rsqrtf(group_sum<S::LPG>(lane_squares<S>(x)) * inv + eps);
}

template <typename S>
__global__ void __launch_bounds__(kNormThreads, S::kResident)
norm_token_fwd(const NormParams<typename S::IO> p, int used, long long slots) {
    extern __shared__ __align__(16) char smem[];
    const int g = threadIdx.x / S::LPG, l = threadIdx.x % S::LPG;
    const long long slot = (long long)blockIdx.x * used + g;
    const bool on = g < used && slot < slots;
    const int head = (int)(slot % p.H);
    const Pairs<S> w = load_affine<S>(p.w, 1.f, head, l, p.d, p.shared);
    const Pairs<S> b = load_affine<S>(p.b, 0.f, head, l, p.d, p.shared);
    const bool gate = p.z != nullptr;
    const typename S::IO* const src[2] = {p.x, p.z};
    const size_t hop = (size_t)slots * p.d;
    size_t at = (size_t)slot * p.d;
    // the slot's rows, and the most a slot of the block has: every lane takes part in the group sums
    // until then
    const int mine = on && slot < p.rows ? (int)((p.rows - 1 - slot) / slots) + 1 : 0;
    const long long slot0 = (long long)blockIdx.x * used;
    const int most = slot0 < p.rows ? (int)((p.rows - 1 - slot0) / slots) + 1 : 0;
    Ring<S, 2> ring(smem, l, p.d, gate ? 2 : 1, (long long)hop);
    ring.open(src, mine ? at : 0, mine);
    for (int i = 0; i < most; ++i, at += hop) {
        Raw<S> raw[2];
        ring.take(src, raw);
        Pairs<S> x = widen<S>(raw[0]);
        const float rstd = token_stats<S>(x, l, p.d, p.center, p.eps);
        if (i < mine)
            with_form(p.act, gate, [&](auto form) {
                store_row<S>(p.y + at, l, p.d, norm_rows<S>(form, x, w, b, raw[1], rstd));
            });
    }
    copy_wait<0>();
}

template <typename S, bool kBias>
__global__ void __launch_bounds__(kNormThreads, S::kResidentSums)
norm_token_bwd(const NormParams<typename S::IO> p, int used, long long slots) {
    extern __shared__ __align__(16) char smem[];
    const int g = threadIdx.x / S::LPG, l = threadIdx.x % S::LPG;
    const long long slot = (long long)blockIdx.x * used + g;
    const bool on = g < used && slot < slots;
    const int head = (int)(slot % p.H);
    const Pairs<S> w = load_affine<S>(p.w, 1.f, head, l, p.d, p.shared);
    const Pairs<S> b = load_affine<S>(p.b, 0.f, head, l, p.d, p.shared);
    Pairs<S> dw = fill<S>(0.f), db = fill<S>(0.f);
    const bool gate = p.z != nullptr;
    const float inv = 1.f / p.d;
    const typename S::IO* const src[3] = {p.x, p.dy, p.z};
    const size_t hop = (size_t)slots * p.d;
    size_t at = (size_t)slot * p.d;
    // the slot's rows, and the most a slot of the block has: every lane takes part in the group sums
    // until then
    const int mine = on && slot < p.rows ? (int)((p.rows - 1 - slot) / slots) + 1 : 0;
    const long long slot0 = (long long)blockIdx.x * used;
    const int most = slot0 < p.rows ? (int)((p.rows - 1 - slot0) / slots) + 1 : 0;
    Ring<S, 3> ring(smem, l, p.d, gate ? 3 : 2, (long long)hop);
    ring.open(src, mine ? at : 0, mine);
    for (int i = 0; i < most; ++i, at += hop) {
        Raw<S> raw[3];
        ring.take(src, raw);
        const bool in = i < mine;
        Pairs<S> x = widen<S>(raw[0]);
        float rstd = token_stats<S>(x, l, p.d, p.center, p.eps);
        if (!in) rstd = 0.f;  // zeros throughout: nothing for the sums
        Back<S> o;
        with_form(p.act, gate, [&](auto form) {
            o = back_rows<S, true, kBias>(form, x, raw[1], raw[2], w, b, rstd, dw, db);
        });
        const float mq = p.center ? group_sum<S::LPG>(o.s1) * inv : 0.f;
        const float mqn = group_sum<S::LPG>(o.s2) * inv;
        if (in) {
            store_row<S>(p.dx + at, l, p.d, back_dx<S>(o, rstd, mq, mqn));
            if (gate) store_row<S>(p.dz + at, l, p.d, o.dz);
        }
    }
    copy_wait<0>();
    let_follow();
    if (!p.part) return;

    // sums over the block's lane groups of one head (of all, for a shared weight)
    constexpr int kCh = S::LPG * S::VEC;
    float* const sh = reinterpret_cast<float*>(smem);  // in the rings' place
    static_assert(sizeof(float) * S::kGroups * kCh <= Ring<S, 3>::kBytes, "the rings are larger");
    const int heads = p.shared ? 1 : p.H <= S::kGroups ? p.H : 0;
    for (int which = 0; which < 1 + kBias; ++which) {
#pragma unroll
        for (int k = 0; k < S::NV; ++k) {
            if (heads == 0) {  // more heads than lane groups: nothing to join
                if (!on) continue;
#pragma unroll
                for (int j = 0; j < S::VEC; ++j) {
                    const int c = (k * S::LPG + l) * S::VEC + j;
                    const F2 v = which ? db.f[k][j / 2] : dw.f[k][j / 2];
                    if (c < p.d)
                        p.part[(((size_t)(slot / p.H) * 2 + which) * p.H + head) * p.d + c] =
                            j & 1 ? v.hi() : v.lo();
                }
                continue;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < S::VEC / 2; ++j) {
                const F2 v = which ? db.f[k][j] : dw.f[k][j];
                sh[g * kCh + l * S::VEC + 2 * j] = on ? v.lo() : 0.f;
                sh[g * kCh + l * S::VEC + 2 * j + 1] = on ? v.hi() : 0.f;
            }
            __syncthreads();
            for (int i = threadIdx.x; i < heads * kCh; i += kNormThreads) {
                const int h = i / kCh, c = k * kCh + i % kCh;
                if (c >= p.d) continue;
                float v = 0.f;
                for (int gg = h; gg < used; gg += heads) v += sh[gg * kCh + i % kCh];
                p.part[(((size_t)blockIdx.x * 2 + which) * heads + h) * p.d + c] = v;
            }
        }
    }
}

// 32 channels of one head a block (all heads for a shared weight); its 32 warps over the rows.
__global__ void __launch_bounds__(1024)
norm_reduce_kernel(const float* part, int rows, int H, int d, float* dw, float* db) {
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, h = blockIdx.y, which = blockIdx.z;
    float* out = which ? db : dw;
    wait_before();
    if (!out) return;
    float v = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int r = wid; r < rows; r += 32) v += part[(((size_t)r * 2 + which) * H + h) * d + c];
    }
    sh[wid][lane] = v;
    __syncthreads();
    if (wid == 0 && c < d) {
#pragma unroll 8
        for (int k = 1; k < 32; ++k) v += sh[k][lane];
        out[(size_t)h * d + c] = v;
    }
}

// Rows a lane group takes at least, where there are so many.
constexpr int kPerSlot = 8;

struct TokenFwd {
    template <typename S>
    static void go(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
        const Deal d = deal(a, S::kGroups, S::kResident, 1);
        norm_launch<Ring<S, 2>::kBytes>(norm_token_fwd<S>, d.blocks, st,
                                        norm_params<typename S::IO>(a, x), d.used, d.slots);
    }
};

struct TokenBwd {
    template <typename S>
    static void go(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
        const bool bias = x.b || x.db;
        const Deal d = deal(a, S::kGroups, S::kResidentSums, kPerSlot);
        auto p = norm_params<typename S::IO>(a, x);
        if (!x.dw && !x.db) p.part = nullptr;
        if (bias)
            norm_launch<Ring<S, 3>::kBytes>(norm_token_bwd<S, true>, d.blocks, st, p, d.used, d.slots);
        else
            norm_launch<Ring<S, 3>::kBytes>(norm_token_bwd<S, false>, d.blocks, st, p, d.used, d.slots);
        if (p.part) launch_norm_reduce(a, x.ws, d.part_rows, x.dw, x.db, st);
    }
};

struct TokenBwdSize {
    template <typename S>
    static void go(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t) {
        *reinterpret_cast<int*>(x.ws) = deal(a, S::kGroups, S::kResidentSums, kPerSlot).part_rows;
    }
};

}  // namespace

void launch_norm_reduce(const gdr_norm_args& a, const float* part, int rows, float* dw,
                              float* db, cudaStream_t st) {
    const int H = a.shared_weight ? 1 : a.H;
    launch_follower(norm_reduce_kernel, dim3((a.d + 31) / 32, H, 2), dim3(1024), 0, st, part, rows, H,
                    a.d, dw, db);
}

bool norm_supported(const gdr_norm_args& a) {
    const int v = a.io_dtype == GDR_BF16 ? 8 : 4;
    return a.d <= (a.d % v == 0 ? 1024 : 256) && a.H <= 65535;
}

size_t norm_fwd_workspace(const gdr_norm_args& a) {
    return a.per_sequence ? norm_seq_fwd_workspace(a) : 0;
}

size_t norm_bwd_workspace(const gdr_norm_args& a) {
    if (a.per_sequence) return norm_seq_bwd_workspace(a);
    int part_rows = 0;
    NormPtrs x{};
    x.ws = reinterpret_cast<float*>(&part_rows);
    norm_shape<TokenBwdSize>(a, x, nullptr);
    return align_up(sizeof(float) * 2 * (size_t)part_rows * (a.shared_weight ? 1 : a.H) * a.d, 256);
}

gdr_status launch_norm_fwd(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    if (a.per_sequence) return launch_norm_seq_fwd(a, x, st);
    if ((long long)a.B * a.T == 0) return GDR_OK;
    return norm_dispatch<TokenFwd>(a, x, st);
}

gdr_status launch_norm_bwd(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    return a.per_sequence ? launch_norm_seq_bwd(a, x, st) : norm_dispatch<TokenBwd>(a, x, st);
}

}  // namespace gdr
