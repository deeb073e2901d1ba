// conv.cu -- short causal depthwise convolution with an activation: forward, backward, one token.
//
//     p_t = bias + sum_{j < W} w[W-1-j] x_{t-j},   y_t = act(p_t)
//
// A thread owns N neighbouring channels (8 bytes of a row) and walks a run of tokens with the last
// W inputs in registers, so that every input is read once (and W - 1 more at the start of each
// run, which the cache serves).  Tokens arrive by asynchronous copies, two batches of four ahead,
// in shared memory of the thread's own, which takes no registers and no barrier.  Channels go in
// pairs through packed fp32 arithmetic, and the activation costs one exponential and one
// reciprocal in place of an IEEE division.
//
// HBM bounds the forward (4 bytes per token and channel in bf16): 65537 x 4096 takes 182 us, 90 %
// of the copy rate.  The backward (6 bytes) comes to 60 %: 8 x 4096 x 2048 takes 100 to 102 us, its
// 24 instructions an element waiting on one another in the 16 warps that its registers allow.  In
// fp32 these 8 x 4096 x 2048 take 100 to 106 us forward and 160 backward (82 and 76 %).
//
// The backward forms p again from x.  dx_t gathers dp of the W - 1 tokens behind it, so a run
// reads that far ahead; the gradients of weights and bias are summed over the run in registers,
// over a block's runs in shared memory, and over the blocks by a second kernel, always in the
// same order.
#include "layer.cuh"

namespace gdr {

namespace {

constexpr int kConvWarps = 4;
constexpr int kConvThreads = 32 * kConvWarps;

// Results in bf16 do not show the coarser sigmoid's error (layer.cuh); fp32 ones do where p is large
// and exact.  The fine one costs fp32 2 to 4 % (8 x 4096 x 2048: 102 -> 106 us, backward 156 -> 160).
template <typename IO>
constexpr bool kFine = sizeof(IO) == 4;

template <typename IO>
struct ConvParams {
    const IO* x; const IO* state; const IO* dy;
    const float* w; const float* bias;
    IO* y; IO* state_out; IO* dx; IO* dstate;
    float* part;              // [blocks over tokens][W + 1][D]
    int* status;
    Seqs q;
    int D, reverse;
    int run, slabs, across;   // tokens of a warp's run, slabs of channels, slabs of a block
};

// The tokens of one sequence in scan order: place 0 is its first token there.
struct Span {
    int b, e, reverse;
    __device__ __forceinline__ int token(int i) const { return reverse ? e - 1 - i : b + i; }
};

// A run [t0, t1) of the token axis meets sequences s = of(t0), of(t0) + 1, ...  Within one, the
// tokens of the run are places [i0, i1).
__device__ __forceinline__ void run_places(const Span& sp, int t0, int t1, int& i0, int& i1) {
    const int lo = max(t0, sp.b), hi = min(t1, sp.e);
    i0 = sp.reverse ? sp.e - hi : lo - sp.b;
    i1 = sp.reverse ? sp.e - lo : hi - sp.b;
}

// N channels as they lie in memory.  kWhole: rows are whole vectors of N; else element by element,
// `left` channels from the thread's first one on.
template <typename IO, int N, bool kWhole>
__device__ __forceinline__ Vec<IO, N> fetch(const IO* p, int left) {
    if constexpr (kWhole) {
        return load_vec<IO, N>(p);
    } else {
        Vec<IO, N> v;
#pragma unroll
        for (int j = 0; j < N; ++j) v.x[j] = j < left ? p[j] : from_f<IO>(0.f);
        return v;
    }
}
template <typename IO, int N, bool kWhole>
__device__ __forceinline__ void put(IO* p, const F2 (&f)[N / 2], int left) {
    Vec<IO, N> v;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) set_pair(v, j, f[j]);
    if constexpr (kWhole) {
        store_raw(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < left) p[j] = v.x[j];
    }
}
template <typename IO, int N>
__device__ __forceinline__ void pairs(const Vec<IO, N>& v, F2 (&f)[N / 2]) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) f[j] = pair_of(v, j);
}

// x at place i of a sequence, from its state where i < 0
template <typename IO, int W, int N, bool kWhole>
__device__ __forceinline__ void fetch_place(const ConvParams<IO>& p, const Span& sp, int s, int i,
                                            int c, F2 (&f)[N / 2]) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) f[j] = f2(0.f);
    if (i >= 0)
        pairs(fetch<IO, N, kWhole>(p.x + (size_t)sp.token(i) * p.D + c, p.D - c), f);
    else if (p.state)
        pairs(fetch<IO, N, kWhole>(p.state + ((size_t)s * (W - 1) + (W - 1 + i)) * p.D + c, p.D - c), f);
}

template <int W, int N>
__device__ __forceinline__ void load_weights(const float* w, const float* bias, int c, int D,
                                             F2 (&wr)[W][N / 2], F2 (&br)[N / 2]) {
    auto at = [&](int ch, int k) { return ch < D ? __ldg(w + (size_t)ch * W + k) : 0.f; };
    auto b = [&](int ch) { return bias && ch < D ? __ldg(bias + ch) : 0.f; };
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
#pragma unroll
        for (int k = 0; k < W; ++k) wr[k][j] = f2(at(c + 2 * j, k), at(c + 2 * j + 1, k));
        br[j] = f2(b(c + 2 * j), b(c + 2 * j + 1));
    }
}

// A thread's next tokens of kT tensors: batches of kBatch tokens in a ring of kStages.
constexpr int kBatch = 4, kStages = 3;
template <typename IO, int N, bool kWhole, int kT>
struct Ring {
    using V = Vec<IO, N>;
    static constexpr int kBytes = kStages * kT * kBatch * kConvThreads * (int)sizeof(V);
    V* slot;              // the thread's first
    const IO* at[kT];     // the next token to be fetched
    int ask, have, n;     // batches asked for and used, tokens in all

    __device__ __forceinline__ V* place(int stage, int t, int u) {
        return slot + ((stage * kT + t) * kBatch + u) * kConvThreads;
    }
    __device__ __forceinline__ void next(long long hop, int left) {
        const int rest = n - ask * kBatch;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (u >= rest) break;
                V* to = place(ask % kStages, t, u);
                if constexpr (kWhole) copy_async<(int)sizeof(V)>(smem_u32(to), at[t], true);
                else *to = fetch<IO, N, false>(at[t], left);
                at[t] += hop;
            }
        }
        ++ask;
        copy_commit();
    }
    // `tokens` of them, from those at at[] on
    __device__ __forceinline__ void open(char* smem, int thread, int tokens, long long hop, int left) {
        slot = reinterpret_cast<V*>(smem) + thread;
        ask = have = 0;
        n = tokens;
        copy_wait<0>();
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) next(hop, left);
    }
    // the next batch; the one behind the last asked for is asked for
    __device__ __forceinline__ void take(V (&v)[kT][kBatch], long long hop, int left) {
        copy_wait<kStages - 2>();
#pragma unroll
        for (int t = 0; t < kT; ++t) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) v[t][u] = *place(have % kStages, t, u);
        }
        ++have;
        next(hop, left);
    }
};

// What a warp works on: a slab of channels and a run of tokens.  A block's warps take `across`
// neighbouring slabs, of as many runs as that leaves, and blocks go over the slabs first, so that
// what runs together reads long pieces of rows.
struct Where {
    long long warp, warps, tokens_block;
    int slab, across, col, line;  // the warp's column and line in the block
    __device__ __forceinline__ Where(int slabs, int across_, int wid) : across(across_) {
        const int columns = (slabs + across - 1) / across, lines = kConvWarps / across;
        col = wid % across;
        line = wid / across;
        tokens_block = blockIdx.x / columns;
        slab = blockIdx.x % columns * across + col;
        warp = tokens_block * lines + line;
        warps = (long long)(gridDim.x / columns) * lines;
    }
};

template <typename IO, int W, int N, bool kWhole, int kAct>
__global__ void __launch_bounds__(kConvThreads)
conv_fwd_kernel(const ConvParams<IO> p) {
    constexpr int P = N / 2;
    __shared__ __align__(16) char smem[Ring<IO, N, kWhole, 1>::kBytes];
    const int lane = threadIdx.x, wid = threadIdx.y;
    const Where me(p.slabs, p.across, wid);
    const int c = (me.slab * 32 + lane) * N, left = p.D - c;
    if (blockIdx.x == 0) check_cu(p.q, p.status, wid * 32 + lane, kConvThreads);
    if (left <= 0) return;

    if (p.state_out) {  // the last W - 1 inputs of every sequence
        for (long long s = me.warp; s < p.q.n; s += me.warps) {
            const Span sp{p.q.begin((int)s), p.q.end((int)s), p.reverse};
            const int len = max(sp.e - sp.b, 0);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                F2 f[P];
                fetch_place<IO, W, N, kWhole>(p, sp, (int)s, len - (W - 1) + k, c, f);
                put<IO, N, kWhole>(p.state_out + ((size_t)s * (W - 1) + k) * p.D + c, f, left);
            }
        }
    }
    const long long first = me.warp * p.run;
    if (first >= p.q.total) return;
    const int t0 = (int)first, t1 = (int)min((long long)p.q.total, first + p.run);

    F2 w[W][P], bias[P];
    load_weights<W, N>(p.w, p.bias, c, p.D, w, bias);
    const long long hop = p.reverse ? -(long long)p.D : p.D;
    for (int s = p.q.of(t0); s < p.q.n; ++s) {
        const Span sp{p.q.begin(s), p.q.end(s), p.reverse};
        if (sp.b >= t1) break;
        int i0, i1;
        run_places(sp, t0, t1, i0, i1);
        if (i0 >= i1) continue;
        F2 x[W - 1][P];  // places i - (W - 1) .. i - 1
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            fetch_place<IO, W, N, kWhole>(p, sp, s, i0 - (W - 1) + k, c, x[k]);
        const IO* in = p.x + (size_t)sp.token(i0) * p.D + c;
        IO* out = p.y + (size_t)sp.token(i0) * p.D + c;
        auto step = [&](const Vec<IO, N>& v) {
            F2 now[P], y[P];
            pairs(v, now);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                F2 a = fma2(w[W - 1][j], now[j], bias[j]);
#pragma unroll
                for (int k = 0; k < W - 1; ++k) a = fma2(w[k][j], x[k][j], a);
                y[j] = act2<kAct, kFine<IO>>(a);
#pragma unroll
                for (int k = 0; k < W - 2; ++k) x[k][j] = x[k + 1][j];
                x[W - 2][j] = now[j];
            }
            put<IO, N, kWhole>(out, y, left);
            out += hop;
        };
        Ring<IO, N, kWhole, 1> ring;
        ring.at[0] = in;
        ring.open(smem, wid * 32 + lane, i1 - i0, hop, left);
        for (int i = i0; i < i1; i += kBatch) {
            Vec<IO, N> v[1][kBatch];
            ring.take(v, hop, left);
            if (i + kBatch <= i1) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) step(v[0][u]);
            } else {
#pragma unroll
                for (int u = 0; u < kBatch - 1; ++u)
                    if (i + u < i1) step(v[0][u]);
            }
        }
    }
}

// Blocks on an SM: five spill (115 instead of 100 to 102 us).
constexpr int kBwdResident = 4;

template <typename IO, int W, int N, bool kWhole, int kAct>
__global__ void __launch_bounds__(kConvThreads, kBwdResident)
conv_bwd_kernel(const ConvParams<IO> p) {
    constexpr int P = N / 2;
    union Shared {
        char ring[Ring<IO, N, kWhole, 2>::kBytes];
        float sums[kConvWarps][32 * N];
    };
    __shared__ __align__(16) Shared smem;
    auto& sh = smem.sums;
    const int lane = threadIdx.x, wid = threadIdx.y;
    const Where me(p.slabs, p.across, wid);
    const int c = (me.slab * 32 + lane) * N, left = p.D - c;
    if (blockIdx.x == 0) check_cu(p.q, p.status, wid * 32 + lane, kConvThreads);
    if (p.dstate && left > 0) {  // nothing reads an empty sequence's state
        for (long long s = me.warp; s < p.q.n; s += me.warps) {
            if (p.q.begin((int)s) < p.q.end((int)s)) continue;
            F2 z[P];
#pragma unroll
            for (int j = 0; j < P; ++j) z[j] = f2(0.f);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                put<IO, N, kWhole>(p.dstate + ((size_t)s * (W - 1) + k) * p.D + c, z, left);
        }
    }
    const long long first = me.warp * p.run;
    const int t0 = (int)min((long long)p.q.total, first);
    const int t1 = (int)min((long long)p.q.total, first + p.run);

    F2 dw[W][P], db[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        db[j] = f2(0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][j] = f2(0.f);
    }
    if (left > 0 && t0 < t1) {
        F2 w[W][P], bias[P];
        load_weights<W, N>(p.w, p.bias, c, p.D, w, bias);
        const long long hop = p.reverse ? -(long long)p.D : p.D;
        for (int s = p.q.of(t0); s < p.q.n; ++s) {
            const Span sp{p.q.begin(s), p.q.end(s), p.reverse};
            if (sp.b >= t1) break;
            int i0, i1;
            run_places(sp, t0, t1, i0, i1);
            if (i0 >= i1) continue;
            const int len = sp.e - sp.b;
            F2 x[W - 1][P], dp[W - 1][P];  // places i - (W - 1) .. i - 1
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                fetch_place<IO, W, N, kWhole>(p, sp, s, i0 - (W - 1) + k, c, x[k]);
#pragma unroll
                for (int j = 0; j < P; ++j) dp[k][j] = f2(0.f);
            }
            // A step brings dp of place i in and dx of place i - (W - 1) out; `own`: the run's
            // token, which counts for dw and db; past: behind the sequence's end, where dp is zero.
            F2 dx[P];
            auto step = [&](const Vec<IO, N>& vx, const Vec<IO, N>& vdy, bool own, bool past) {
                F2 xi[P], d[P];
                pairs(vx, xi);
                pairs(vdy, d);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    F2 a = fma2(w[W - 1][j], xi[j], bias[j]), v, g;
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) a = fma2(w[k][j], x[k][j], a);
                    act2_both<kAct, kFine<IO>>(a, v, g);
                    d[j] = past ? f2(0.f) : mul2(d[j], g);
                    if (own) {
                        db[j] = add2(db[j], d[j]);
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dw[k][j] = fma2(d[j], x[k][j], dw[k][j]);
                        dw[W - 1][j] = fma2(d[j], xi[j], dw[W - 1][j]);
                    }
                    // dx_out = sum_k w[W-1-k] dp_{out + k}
                    F2 sum = mul2(w[0][j], d[j]);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) sum = fma2(w[W - 1 - k][j], dp[k][j], sum);
                    dx[j] = sum;
#pragma unroll
                    for (int k = 0; k < W - 2; ++k) { x[k][j] = x[k + 1][j]; dp[k][j] = dp[k + 1][j]; }
                    x[W - 2][j] = xi[j];
                    dp[W - 2][j] = d[j];
                }
            };
            auto any = [&](int i) {
                const bool past = i >= len;
                Vec<IO, N> vx{}, vdy{};
                if (!past) {
                    const size_t at = (size_t)sp.token(i) * p.D + c;
                    vx = fetch<IO, N, kWhole>(p.x + at, left);
                    vdy = fetch<IO, N, kWhole>(p.dy + at, left);
                }
                step(vx, vdy, i < i1, past);
                const int out = i - (W - 1);
                if (out < i0 && i0 > 0) return;  // another run's
                if (out >= 0)
                    put<IO, N, kWhole>(p.dx + (size_t)sp.token(out) * p.D + c, dx, left);
                else if (p.dstate)
                    put<IO, N, kWhole>(p.dstate + ((size_t)s * (W - 1) + (W - 1 + out)) * p.D + c, dx, left);
            };
            int i = i0;
            for (; i < min(i0 + W - 1, i1); ++i) any(i);
            if (i + kBatch <= i1) {  // the run's own tokens, dx of its own tokens
                const size_t at = (size_t)sp.token(i) * p.D + c;
                IO* out = p.dx + (size_t)sp.token(i - (W - 1)) * p.D + c;
                Ring<IO, N, kWhole, 2> ring;
                ring.at[0] = p.x + at;
                ring.at[1] = p.dy + at;
                ring.open(smem.ring, wid * 32 + lane, (i1 - i) / kBatch * kBatch, hop, left);
                for (; i + kBatch <= i1; i += kBatch) {
                    Vec<IO, N> v[2][kBatch];
                    ring.take(v, hop, left);
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        step(v[0][u], v[1][u], true, false);
                        put<IO, N, kWhole>(out, dx, left);
                        out += hop;
                    }
                }
            }
            for (; i < i1 + W - 1; ++i) any(i);
        }
    }
    let_follow();
    // the block's runs, then one row of partial sums a block, in the rings' place
    copy_wait<0>();
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const F2 v = k < W ? dw[k < W ? k : 0][j] : db[j];
            sh[wid][lane * N + 2 * j] = v.lo();
            sh[wid][lane * N + 2 * j + 1] = v.hi();
        }
        __syncthreads();
        if (me.line == 0) {
            for (int i = lane; i < 32 * N; i += 32) {
                const int ch = me.slab * 32 * N + i;
                if (ch >= p.D) break;
                float v = 0.f;
                for (int g = me.col; g < kConvWarps; g += me.across) v += sh[g][i];
                p.part[((size_t)me.tokens_block * (W + 1) + k) * p.D + ch] = v;
            }
        }
    }
}

// dw, dbias from the partial sums: 32 channels a block, its 8 warps over the rows.
template <int W>
__global__ void __launch_bounds__(256)
conv_reduce_kernel(const float* part, int rows, int D, float* dw, float* dbias) {
    __shared__ float sh[8][32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    wait_before();
    float v = 0.f;
    if (c < D)
#pragma unroll 4
        for (int r = wid; r < rows; r += 8) v += part[((size_t)r * (W + 1) + k) * D + c];
    sh[wid][lane] = v;
    __syncthreads();
    if (wid != 0 || c >= D) return;
#pragma unroll
    for (int g = 1; g < 8; ++g) v += sh[g][lane];
    if (k < W) dw[(size_t)c * W + k] = v;
    else if (dbias) dbias[c] = v;
}

template <typename IO, int W, int N, bool kWhole, int kAct>
__global__ void __launch_bounds__(128)
conv_step_kernel(const IO* __restrict__ x, const float* __restrict__ w,
                 const float* __restrict__ bias, const IO* state, IO* state_out,
                 IO* __restrict__ y, int D) {
    constexpr int P = N / 2;
    const int c = (blockIdx.x * 128 + threadIdx.x) * N, left = D - c;
    if (left <= 0) return;
    const size_t n = blockIdx.y;
    const IO* st = state + n * (W - 1) * D + c;
    // the state may be updated in place: all of it is read before any of it is written
    F2 win[W][P], wr[W][P], b[P];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Vec<IO, N> v;
        if constexpr (kWhole) {
            v = load_in_place<IO, N>(st + (size_t)k * D);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) v.x[j] = j < left ? st[(size_t)k * D + j] : from_f<IO>(0.f);
        }
        pairs(v, win[k]);
    }
    pairs(fetch<IO, N, kWhole>(x + n * D + c, left), win[W - 1]);
    load_weights<W, N>(w, bias, c, D, wr, b);
    F2 out[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        F2 a = fma2(wr[W - 1][j], win[W - 1][j], b[j]);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) a = fma2(wr[k][j], win[k][j], a);
        out[j] = act2<kAct, kFine<IO>>(a);
    }
    put<IO, N, kWhole>(y + n * D + c, out, left);
    IO* so = state_out + n * (W - 1) * D + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) put<IO, N, kWhole>(so + (size_t)k * D, win[k + 1], left);
}

// ---- launching ---------------------------------------------------------------------------------

// Channels of a thread: four where rows are whole vectors of four, else two.
int conv_channels(const gdr_conv_args& a) { return a.D % 4 ? 2 : 4; }

struct ConvGrid {
    int run, slabs, across;  // as in ConvParams
    unsigned rows, blocks;   // blocks over the tokens, blocks
};

// A run is long enough that the W - 1 extra tokens read at its ends cost little, and short enough
// that `resident` blocks on an SM are there where the tokens suffice.
ConvGrid conv_grid(const gdr_conv_args& a, int across, int resident, int most) {
    ConvGrid g;
    const int per_slab = 32 * conv_channels(a);
    const long long tokens = (long long)a.B * a.T;
    g.slabs = (a.D + per_slab - 1) / per_slab;
    while (across > g.slabs) across /= 2;
    g.across = across;
    const int columns = (g.slabs + across - 1) / across, lines = kConvWarps / across;
    const long long rows = 148 * resident / columns > 0 ? 148 * resident / columns : 1;
    const long long run = (tokens + rows * lines - 1) / (rows * lines);
    g.run = (int)(run < 8 ? 8 : run > most ? most : run);
    const long long per = (long long)g.run * lines;
    g.rows = (unsigned)((tokens + per - 1) / per);
    if (g.rows == 0) g.rows = 1;
    g.blocks = g.rows * (unsigned)columns;
    return g;
}
// Measured on 65537 x 4096 (forward) and 8 x 4096 x 2048 (backward) in bf16.  Forward: a block's
// warps on four neighbouring slabs 186 us, on four runs of one slab 190; runs of up to 64, 128, 256
// tokens 195, 186, 198.  Backward: one slab 98 us, four 104; runs of up to 32, 64, 128, 256 tokens
// 131, 108, 100, 98.  (Each series on one box and build, which differ by a few percent.)
ConvGrid fwd_grid(const gdr_conv_args& a) { return conv_grid(a, 4, 8, 128); }
ConvGrid bwd_grid(const gdr_conv_args& a) { return conv_grid(a, 1, kBwdResident, 256); }

template <typename IO>
ConvParams<IO> conv_params(const gdr_conv_args& a, const ConvPtrs& x, const ConvGrid& g) {
    ConvParams<IO> p;
    p.x = static_cast<const IO*>(x.x);
    p.state = static_cast<const IO*>(x.state);
    p.dy = static_cast<const IO*>(x.dy);
    p.w = x.w;
    p.bias = x.bias;
    p.y = static_cast<IO*>(x.y);
    p.state_out = static_cast<IO*>(x.state_out);
    p.dx = static_cast<IO*>(x.dx);
    p.dstate = static_cast<IO*>(x.dstate);
    p.part = x.ws;
    p.status = a.status;
    p.q = Seqs{x.cu, a.n_seqs, a.T, a.B * a.T};
    p.D = a.D;
    p.reverse = a.reverse;
    p.run = g.run;
    p.slabs = (int)g.slabs;
    p.across = g.across;
    return p;
}

struct ConvFwd {
    template <typename IO, int W, int N, bool kWhole, int kAct>
    static void go(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
        const ConvGrid g = fwd_grid(a);
        conv_fwd_kernel<IO, W, N, kWhole, kAct><<<g.blocks, dim3(32, kConvWarps), 0, st>>>(
            conv_params<IO>(a, x, g));
    }
};

struct ConvBwd {
    template <typename IO, int W, int N, bool kWhole, int kAct>
    static void go(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
        const ConvGrid g = bwd_grid(a);
        conv_bwd_kernel<IO, W, N, kWhole, kAct><<<g.blocks, dim3(32, kConvWarps), 0, st>>>(
            conv_params<IO>(a, x, g));
        launch_follower(conv_reduce_kernel<W>, dim3((a.D + 31) / 32, W + 1), dim3(256), 0, st, x.ws,
                        (int)g.rows, a.D, x.dw, x.dbias);
    }
};

struct ConvStep {
    template <typename IO, int W, int N, bool kWhole, int kAct>
    static void go(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
        const unsigned bx = (unsigned)((a.D + 128 * N - 1) / (128 * N));
        for (int n0 = 0; n0 < a.B; n0 += 65535) {  // a grid's second dimension ends at 65535
            const int n = a.B - n0 < 65535 ? a.B - n0 : 65535;
            const size_t row = (size_t)n0 * a.D, srow = row * (W - 1);
            conv_step_kernel<IO, W, N, kWhole, kAct><<<dim3(bx, n), 128, 0, st>>>(
                static_cast<const IO*>(x.x) + row, x.w, x.bias,
                static_cast<const IO*>(x.state) + srow, static_cast<IO*>(x.state_out) + srow,
                static_cast<IO*>(x.y) + row, a.D);
        }
    }
};

template <typename Op, typename IO, int W, int kAct>
void conv_vectors(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    if (a.D % 4 == 0) Op::template go<IO, W, 4, true, kAct>(a, x, st);
    else if (a.D % 2 == 0) Op::template go<IO, W, 2, true, kAct>(a, x, st);
    else Op::template go<IO, W, 2, false, kAct>(a, x, st);
}

template <typename Op, typename IO, int W>
void conv_act(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    if (a.activation == GDR_ACT_SILU) conv_vectors<Op, IO, W, GDR_ACT_SILU>(a, x, st);
    else conv_vectors<Op, IO, W, GDR_ACT_NONE>(a, x, st);
}

template <typename Op, typename IO>
void conv_width(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    switch (a.width) {
        case 2: conv_act<Op, IO, 2>(a, x, st); break;
        case 3: conv_act<Op, IO, 3>(a, x, st); break;
        default: conv_act<Op, IO, 4>(a, x, st);
    }
}

template <typename Op>
gdr_status conv_dispatch(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    if (a.io_dtype == GDR_BF16) conv_width<Op, __nv_bfloat16>(a, x, st);
    else conv_width<Op, float>(a, x, st);
    return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

}  // namespace

size_t conv_bwd_workspace(const gdr_conv_args& a) {
    const ConvGrid g = bwd_grid(a);
    return align_up(sizeof(float) * (size_t)g.rows * (a.width + 1) * a.D, 256);
}

gdr_status launch_conv_fwd(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    return conv_dispatch<ConvFwd>(a, x, st);
}

gdr_status launch_conv_bwd(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    return conv_dispatch<ConvBwd>(a, x, st);
}

gdr_status launch_conv_step(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    return conv_dispatch<ConvStep>(a, x, st);
}

}  // namespace gdr
