// norm_seq.cu -- group norm with statistics over all tokens of a sequence: forward, backward.
//
// A group is one head's channels over a whole sequence, more than a block can hold, so each
// direction is two passes over the tensors with the sums joined between them: sums of every
// (tile of tokens, head), their join per (sequence, head), then the elements.  The second pass
// reads x again: from L2 where the tensors fit there.  16 segments of 2048 tokens x 12 x 64 in bf16
// take 45 us forward and 60 backward (bytes read once: 15 and 23), the backward's two passes at 64 %
// of the issue slots.  8 x 4096 x 16 x 128, beyond L2, takes 165 us backward with a gate, at the rate
// of two passes' bytes (163), and 104 us forward without one: the statistics pass 47, where its bytes
// take 20 (its many short blocks load, join and end), and the second 54, where they take 41.
//
// A tile may meet several sequences.  Tile i and sequence s have the piece number i + s: along
// the token axis each step goes to the next tile or to the next sequence, so the numbers are
// distinct and a sequence's pieces lie side by side, whatever the lengths.  A block takes its
// tile's sequences one after the other, so the first pass slows down where they are shorter than
// its tile: 32768 tokens x 16 x 64 take 57 us forward and 78 backward in sequences of 1024, 250 and
// 320 in sequences of 8, 1540 and 1990 in sequences of one.
//
// Variances: each piece's sum of squares is taken about the piece's own mean, from registers,
// and pieces are joined pairwise with the difference of their means, so that no large squares
// cancel.  Every join has a fixed order.
#include "norm_impl.cuh"

namespace gdr {

namespace {

__device__ __forceinline__ float block_sum(float x, float* sh) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kNormWarps; ++i) v += sh[i];
    return v;
}

// Two sums over a block behind one barrier, in two buffers by turns: behind a call's barrier all
// threads have read the call before it, so the next one may overwrite that.  (Against two sums of
// block_sum: 166 instead of 174 us on the shape above.  The statistics pass gains nothing by it.)
__device__ __forceinline__ float2 block_sums(float x, float y, float2 (*sh)[kNormWarps], int& turn) {
    x = warp_sum(x);
    y = warp_sum(y);
    float2* const mine = sh[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kNormWarps; ++i) {
        v.x += mine[i].x;
        v.y += mine[i].y;
    }
    return v;
}

// Tokens a lane group holds at once in the statistics pass.
template <typename S>
constexpr int kHold = S::NV >= 8 ? 1 : 8 / S::NV;

// part[(tile + s) * H + h] = (mean, sum of squares about it) of the piece's values; without
// centering (0, sum of squares).
template <typename S>
__global__ void __launch_bounds__(kNormThreads, 3)
norm_seq_stats(const NormParams<typename S::IO> p) {
    constexpr int kTokens = S::kGroups * kHold<S>;
    __shared__ float sh[kNormWarps];
    const int g = threadIdx.x / S::LPG, l = threadIdx.x % S::LPG;
    const int tile = blockIdx.x / p.H, h = blockIdx.x % p.H;
    if (blockIdx.x == 0) check_cu(p.q, p.status, threadIdx.x, kNormThreads);
    const int t0 = (int)min((long long)p.q.total, (long long)tile * kTokens);
    const int t1 = (int)min((long long)p.q.total, (long long)t0 + kTokens);
    Raw<S> x[kHold<S>];
#pragma unroll
    for (int i = 0; i < kHold<S>; ++i) {
        const int t = t0 + g + i * S::kGroups;
        x[i] = load_row<S>(p.x + ((size_t)(t < t1 ? t : t0) * p.H + h) * p.d, l, p.d, t < t1);
    }
    let_follow();
    for (int s = p.q.of(t0); s < p.q.n; ++s) {
        const int b = p.q.begin(s), e = p.q.end(s);
        if (b >= t1) break;
        const int lo = max(b, t0), hi = min(e, t1);
        if (lo >= hi) continue;
        float mean = 0.f;
        if (p.center) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kHold<S>; ++i) {
                const int t = t0 + g + i * S::kGroups;
                if (t >= lo && t < hi) v += lane_sum<S>(widen<S>(x[i]));
            }
            mean = block_sum(v, sh) / ((float)(hi - lo) * p.d);
        }
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kHold<S>; ++i) {
            const int t = t0 + g + i * S::kGroups;
            if (t < lo || t >= hi) continue;
            Pairs<S> f = widen<S>(x[i]);
            centre<S>(f, mean, l, p.d);
            v += lane_squares<S>(f);
        }
        v = block_sum(v, sh);
        if (threadIdx.x == 0)
            reinterpret_cast<float2*>(p.part)[((size_t)tile + s) * p.H + h] = make_float2(mean, v);
    }
}

// One warp per (sequence, head): joins the pieces' (mean, sum of squares).
__global__ void __launch_bounds__(128)
norm_seq_join_stats(Seqs q, int H, int d, int tokens, float eps, const float2* part, float2* stats) {
    const long long unit = (long long)blockIdx.x * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    wait_before();
    let_follow();
    if (unit >= (long long)q.n * H) return;
    const int s = (int)(unit / H), h = (int)(unit % H);
    const int b = q.begin(s), e = q.end(s);
    float n = 0.f, mean = 0.f, m2 = 0.f;
    auto join = [&](float nb, float mb, float sb) {
        if (nb == 0.f) return;
        const float all = n + nb, diff = mb - mean, f = nb / all;
        mean = fmaf(diff, f, mean);
        m2 += sb + diff * diff * n * f;
        n = all;
    };
    if (b < e) {
        for (int i = b / tokens + lane; i <= (e - 1) / tokens; i += 32) {
            const float2 v = part[((size_t)i + s) * H + h];
            const long long lo = max((long long)b, (long long)i * tokens);
            const long long hi = min((long long)e, (long long)i * tokens + tokens);
            join((float)(hi - lo) * d, v.x, v.y);
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float nb = __shfl_down_sync(0xffffffffu, n, o);
        const float mb = __shfl_down_sync(0xffffffffu, mean, o);
        const float sb = __shfl_down_sync(0xffffffffu, m2, o);
        if (lane + o < 32) join(nb, mb, sb);
    }
    if (lane == 0)
        stats[unit] = make_float2(mean, rsqrtf((n > 0.f ? m2 / n : 0.f) + eps));
}

// The sequence of token t, not before s.
__device__ __forceinline__ int seq_from(const Seqs& q, int s, int t) {
    while (s + 1 < q.n && t >= q.end(s)) ++s;
    return s;
}

// The second pass visits the tiles backwards: the first one's last tiles are still in L2.
template <typename S>
__global__ void __launch_bounds__(kNormThreads, S::kResident)
norm_seq_apply(const NormParams<typename S::IO> p, int tokens) {
    extern __shared__ __align__(16) char smem[];
    const int g = threadIdx.x / S::LPG, l = threadIdx.x % S::LPG;
    const int block = gridDim.x - 1 - blockIdx.x, tile = block / p.H, h = block % p.H;
    const int t0 = (int)min((long long)p.q.total, (long long)tile * tokens);
    const int t1 = (int)min((long long)p.q.total, (long long)t0 + tokens);
    const Pairs<S> w = load_affine<S>(p.w, 1.f, h, l, p.d, p.shared);
    const Pairs<S> b = load_affine<S>(p.b, 0.f, h, l, p.d, p.shared);
    const bool gate = p.z != nullptr;
    const typename S::IO* const src[2] = {p.x, p.z};
    const size_t hop = (size_t)S::kGroups * p.H * p.d;
    const int mine = t0 + g < t1 ? (t1 - 1 - (t0 + g)) / S::kGroups + 1 : 0;
    size_t at = mine ? ((size_t)(t0 + g) * p.H + h) * p.d : 0;
    Ring<S, 2> ring(smem, l, p.d, gate ? 2 : 1, (long long)hop);
    ring.open(src, at, mine);
    int s = t0 + g < t1 ? p.q.of(t0 + g) : 0;
    wait_before();  // for the statistics; the tensors are the caller's
    int end = t0;   // of the sequence whose statistics are at hand
    float2 st{};
    for (int t = t0 + g; t < t1; t += S::kGroups, at += hop) {
        Raw<S> raw[2];
        ring.take(src, raw);
        if (t >= end) {
            s = seq_from(p.q, s, t);
            end = s + 1 < p.q.n ? p.q.end(s) : t1;
            st = reinterpret_cast<const float2*>(p.stats)[(size_t)s * p.H + h];
        }
        Pairs<S> x = widen<S>(raw[0]);
        centre<S>(x, st.x, l, p.d);
        with_form(p.act, gate, [&](auto form) {
            store_row<S>(p.y + at, l, p.d, norm_rows<S>(form, x, w, b, raw[1], st.y));
        });
    }
    copy_wait<0>();
}

// First pass of the backward: dz, the tile's sums for dw and db, and per piece the sums of q
// and q n.
template <typename S>
__global__ void __launch_bounds__(kNormThreads, S::kResident)
norm_seq_bwd_sums(const NormParams<typename S::IO> p, int tokens, float2* pieces) {
    extern __shared__ __align__(16) char smem[];
    constexpr int kCh = S::LPG * S::VEC;
    __shared__ float2 sh[2][kNormWarps];
    int turn = 0;
    const int g = threadIdx.x / S::LPG, l = threadIdx.x % S::LPG;
    const int tile = blockIdx.x / p.H, h = blockIdx.x % p.H;
    if (blockIdx.x == 0) check_cu(p.q, p.status, threadIdx.x, kNormThreads);
    const int t0 = (int)min((long long)p.q.total, (long long)tile * tokens);
    const int t1 = (int)min((long long)p.q.total, (long long)t0 + tokens);
    const Pairs<S> w = load_affine<S>(p.w, 1.f, h, l, p.d, p.shared);
    const Pairs<S> b = load_affine<S>(p.b, 0.f, h, l, p.d, p.shared);
    Pairs<S> dw = fill<S>(0.f), db = fill<S>(0.f);
    const bool gate = p.z != nullptr;
    const typename S::IO* const src[3] = {p.x, p.dy, p.z};
    const size_t hop = (size_t)S::kGroups * p.H * p.d;
    Ring<S, 3> ring(smem, l, p.d, gate ? 3 : 2, (long long)hop);
    for (int s = t0 < t1 ? p.q.of(t0) : p.q.n; s < p.q.n; ++s) {
        const int sb = p.q.begin(s), se = p.q.end(s);
        if (sb >= t1) break;
        const int lo = max(sb, t0), hi = min(se, t1);
        if (lo >= hi) continue;
        const float2 st = __ldg(reinterpret_cast<const float2*>(p.stats) + (size_t)s * p.H + h);
        float s1 = 0.f, s2 = 0.f;
        const int mine = lo + g < hi ? (hi - 1 - (lo + g)) / S::kGroups + 1 : 0;
        size_t at = mine ? ((size_t)(lo + g) * p.H + h) * p.d : 0;
        ring.open(src, at, mine);
        for (int t = lo + g; t < hi; t += S::kGroups, at += hop) {
            Raw<S> raw[3];
            ring.take(src, raw);
            Pairs<S> x = widen<S>(raw[0]);
            centre<S>(x, st.x, l, p.d);
            Back<S> o;
            with_form(p.act, gate, [&](auto form) {
                o = back_rows<S, true, true>(form, x, raw[1], raw[2], w, b, st.y, dw, db);
            });
            s1 += o.s1;
            s2 += o.s2;
            if (gate) store_row<S>(p.dz + at, l, p.d, o.dz);
        }
        const float2 sums = block_sums(s1, s2, sh, turn);
        if (threadIdx.x == 0) pieces[((size_t)tile + s) * p.H + h] = sums;
    }
    copy_wait<0>();
    let_follow();
    float* const shw = reinterpret_cast<float*>(smem);  // in the rings' place
    static_assert(sizeof(float) * S::kGroups * kCh <= Ring<S, 3>::kBytes, "the rings are larger");
    if (!p.part) return;
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int k = 0; k < S::NV; ++k) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < S::VEC / 2; ++j) {
                const F2 v = which ? db.f[k][j] : dw.f[k][j];
                shw[g * kCh + l * S::VEC + 2 * j] = v.lo();
                shw[g * kCh + l * S::VEC + 2 * j + 1] = v.hi();
            }
            __syncthreads();
            for (int i = threadIdx.x; i < kCh; i += kNormThreads) {
                const int c = k * kCh + i;
                if (c >= p.d) continue;
                float v = 0.f;
                for (int gg = 0; gg < S::kGroups; ++gg) v += shw[gg * kCh + i];
                const size_t row = p.shared ? ((size_t)blockIdx.x * 2 + which)
                                            : (((size_t)tile * 2 + which) * p.H + h);
                p.part[row * p.d + c] = v;
            }
        }
    }
}

// One warp per (sequence, head): means of q and q n over the group.
__global__ void __launch_bounds__(128)
norm_seq_join_sums(Seqs q, int H, int d, int tokens, int center, const float2* pieces,
                   float2* means) {
    const long long unit = (long long)blockIdx.x * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    wait_before();
    let_follow();
    if (unit >= (long long)q.n * H) return;
    const int s = (int)(unit / H), h = (int)(unit % H);
    const int b = q.begin(s), e = q.end(s);
    if (b >= e) return;
    float s1 = 0.f, s2 = 0.f;
    for (int i = b / tokens + lane; i <= (e - 1) / tokens; i += 32) {
        const float2 v = pieces[((size_t)i + s) * H + h];
        s1 += v.x;
        s2 += v.y;
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    const float n = (float)(e - b) * d;
    if (lane == 0) means[unit] = make_float2(center ? s1 / n : 0.f, s2 / n);
}

template <typename S>
__global__ void __launch_bounds__(kNormThreads, S::kResident)
norm_seq_bwd_apply(const NormParams<typename S::IO> p, int tokens,
                   const float2* means) {
    extern __shared__ __align__(16) char smem[];
    const int g = threadIdx.x / S::LPG, l = threadIdx.x % S::LPG;
    const int block = gridDim.x - 1 - blockIdx.x, tile = block / p.H, h = block % p.H;
    const int t0 = (int)min((long long)p.q.total, (long long)tile * tokens);
    const int t1 = (int)min((long long)p.q.total, (long long)t0 + tokens);
    const Pairs<S> w = load_affine<S>(p.w, 1.f, h, l, p.d, p.shared);
    const Pairs<S> b = load_affine<S>(p.b, 0.f, h, l, p.d, p.shared);
    Pairs<S> none;
    const bool gate = p.z != nullptr;
    const typename S::IO* const src[3] = {p.x, p.dy, p.z};
    const size_t hop = (size_t)S::kGroups * p.H * p.d;
    const int mine = t0 + g < t1 ? (t1 - 1 - (t0 + g)) / S::kGroups + 1 : 0;
    size_t at = mine ? ((size_t)(t0 + g) * p.H + h) * p.d : 0;
    Ring<S, 3> ring(smem, l, p.d, gate ? 3 : 2, (long long)hop);
    ring.open(src, at, mine);
    int s = t0 + g < t1 ? p.q.of(t0 + g) : 0;
    wait_before();  // for the means; the tensors and statistics are the caller's
    int end = t0;   // of the sequence whose statistics are at hand
    float2 st{}, m{};
    for (int t = t0 + g; t < t1; t += S::kGroups, at += hop) {
        Raw<S> raw[3];
        ring.take(src, raw);
        if (t >= end) {
            s = seq_from(p.q, s, t);
            end = s + 1 < p.q.n ? p.q.end(s) : t1;
            st = __ldg(reinterpret_cast<const float2*>(p.stats) + (size_t)s * p.H + h);
            m = means[(size_t)s * p.H + h];
        }
        Pairs<S> x = widen<S>(raw[0]);
        centre<S>(x, st.x, l, p.d);
        with_form(p.act, gate, [&](auto form) {
            const Back<S> o = back_rows<S, false, true>(form, x, raw[1], raw[2], w, b, st.y, none, none);
            store_row<S>(p.dx + at, l, p.d, back_dx<S>(o, st.y, m.x, m.y));
        });
    }
    copy_wait<0>();
}

// ---- launching ---------------------------------------------------------------------------------

// Tokens of a tile in the statistics pass: what a block holds in registers.
int stats_tile(const gdr_norm_args& a) {
    const int v = a.io_dtype == GDR_BF16 ? 8 : 4;
    const int n = a.d % v ? (a.d + 1) / 2 : a.d / v;   // vectors of a row
    const int nv = n <= 32 ? 1 : n <= 64 ? 2 : n <= 128 ? 4 : 8;
    return norm_groups(a) * (8 / nv);
}

// Tokens of a tile in the other passes: as many as make the blocks (a tile and head each) one wave
// of three on an SM, in whole passes of the block's lane groups.
int apply_tile(const gdr_norm_args& a) {
    const int g = norm_groups(a);
    const long long tokens = (long long)a.B * a.T;
    const long long tiles = 148 * 3 / a.H > 0 ? 148 * 3 / a.H : 1;
    const long long per = (tokens + tiles * g - 1) / (tiles * g);
    return (int)(per < 1 ? 1 : per > 256 ? 256 : per) * g;
}

long long tiles_of(const gdr_norm_args& a, int tile) {
    return ((long long)a.B * a.T + tile - 1) / tile;
}

size_t pair_bytes(long long rows, int H) {
    return align_up(sizeof(float2) * (size_t)rows * H, 256);
}

struct SeqStats {
    template <typename S>
    static void go(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
        norm_seq_stats<S><<<(unsigned)(tiles_of(a, stats_tile(a)) * a.H), kNormThreads, 0, st>>>(
            norm_params<typename S::IO>(a, x));
    }
};

struct SeqApply {
    template <typename S>
    static void go(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
        const int tile = apply_tile(a);
        norm_launch<Ring<S, 2>::kBytes, true>(norm_seq_apply<S>, tiles_of(a, tile) * a.H, st,
                                        norm_params<typename S::IO>(a, x), tile);
    }
};

unsigned unit_blocks(const gdr_norm_args& a) {
    return (unsigned)(((long long)a.n_seqs * a.H + 3) / 4);
}

struct SeqBwd {
    template <typename S>
    static void go(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
        const int tile = apply_tile(a);
        const long long tiles = tiles_of(a, tile);
        const long long blocks = tiles * a.H;
        auto p = norm_params<typename S::IO>(a, x);
        char* ws = reinterpret_cast<char*>(x.ws);
        float2* pieces = reinterpret_cast<float2*>(ws);
        float2* means = reinterpret_cast<float2*>(ws + pair_bytes(tiles + a.n_seqs, a.H));
        p.part = reinterpret_cast<float*>(ws + pair_bytes(tiles + a.n_seqs, a.H) +
                                          pair_bytes(a.n_seqs, a.H));
        if (!x.dw && !x.db) p.part = nullptr;
        if (tiles) {
            norm_launch<Ring<S, 3>::kBytes>(norm_seq_bwd_sums<S>, blocks, st, p, tile, pieces);
            launch_follower(norm_seq_join_sums, dim3(unit_blocks(a)), dim3(128), 0, st, p.q, a.H, a.d,
                            tile, a.center, pieces, means);
            norm_launch<Ring<S, 3>::kBytes, true>(norm_seq_bwd_apply<S>, blocks, st, p, tile,
                                            (const float2*)means);
        }
        if (p.part)
            launch_norm_reduce(a, p.part, (int)(a.shared_weight ? tiles * a.H : tiles), x.dw, x.db,
                               st);
    }
};

}  // namespace

size_t norm_seq_fwd_workspace(const gdr_norm_args& a) {
    return pair_bytes(tiles_of(a, stats_tile(a)) + a.n_seqs, a.H) + pair_bytes(a.n_seqs, a.H);
}

size_t norm_seq_bwd_workspace(const gdr_norm_args& a) {
    const long long tiles = tiles_of(a, apply_tile(a));
    return pair_bytes(tiles + a.n_seqs, a.H) + pair_bytes(a.n_seqs, a.H) +
           align_up(sizeof(float) * 2 * (size_t)tiles * a.H * a.d, 256);
}

gdr_status launch_norm_seq_fwd(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    const int tile = stats_tile(a);
    const long long tiles = tiles_of(a, tile);
    NormPtrs y = x;
    const float2* part = reinterpret_cast<const float2*>(x.ws);
    if (!y.stats)
        y.stats = reinterpret_cast<float*>(reinterpret_cast<char*>(x.ws) +
                                           pair_bytes(tiles + a.n_seqs, a.H));
    y.stats_in = y.stats;
    if (tiles && norm_dispatch<SeqStats>(a, y, st) != GDR_OK) return GDR_ERR_CUDA;
    if (launch_follower(norm_seq_join_stats, dim3(unit_blocks(a)), dim3(128), 0, st,
                        Seqs{x.cu, a.n_seqs, a.T, a.B * a.T}, a.H, a.d, tile, a.eps, part,
                        reinterpret_cast<float2*>(y.stats)) != cudaSuccess)
        return GDR_ERR_CUDA;
    return tiles ? norm_dispatch<SeqApply>(a, y, st) : GDR_OK;
}

gdr_status launch_norm_seq_bwd(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    return norm_dispatch<SeqBwd>(a, x, st);
}

}  // namespace gdr
