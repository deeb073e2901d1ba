// conv.cu -- short causal depthwise convolution with an activation: forward, backward, one token.
//
//     p_t = bias + sum_{j < W} w[W-1-j] x_{t-j},   y_t = act(p_t)
//
// A thread owns VEC neighbouring channels and walks a run of tokens with the last W inputs in
// registers, so that every input is read once (and W - 1 more at the start of each run, which
// the cache serves).  The activation is one exponential and one division per element; HBM bounds
// all three kernels: 4 bytes per token and channel forward and 6 backward, in bf16.
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

template <typename IO>
struct ConvParams {
    const IO* x; const IO* state; const IO* dy;
    const float* w; const float* bias;
    IO* y; IO* state_out; IO* dx; IO* dstate;
    float* part;              // [blocks over tokens][W + 1][D]
    int* status;
    Seqs q;
    int D, act, reverse;
    int run;                  // tokens of a warp's run
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

// x at place i of a sequence, from its state where i < 0
template <typename IO, int W, int VEC>
__device__ __forceinline__ void load_place(const ConvParams<IO>& p, const Span& sp, int s, int i,
                                           int c, float (&f)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = 0.f;
    if (i >= 0) load_f<IO, VEC>(p.x + (size_t)sp.token(i) * p.D + c, f);
    else if (p.state) load_f<IO, VEC>(p.state + ((size_t)s * (W - 1) + (W - 1 + i)) * p.D + c, f);
}

template <int W, int VEC>
__device__ __forceinline__ void load_weights(const float* w, const float* bias, int c,
                                             float (&wr)[W][VEC], float (&br)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
#pragma unroll
        for (int k = 0; k < W; ++k) wr[k][j] = __ldg(w + (size_t)(c + j) * W + k);
        br[j] = bias ? __ldg(bias + c + j) : 0.f;
    }
}

template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(kConvThreads)
conv_fwd_kernel(const ConvParams<IO> p) {
    const int lane = threadIdx.x, wid = threadIdx.y;
    const int c = (blockIdx.y * 32 + lane) * VEC;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        check_cu(p.q, p.status, wid * 32 + lane, kConvThreads);
    if (c >= p.D) return;
    const long long warp = (long long)blockIdx.x * kConvWarps + wid;
    const long long warps = (long long)gridDim.x * kConvWarps;

    if (p.state_out) {  // the last W - 1 inputs of every sequence
        for (long long s = warp; s < p.q.n; s += warps) {
            const Span sp{p.q.begin((int)s), p.q.end((int)s), p.reverse};
            const int len = max(sp.e - sp.b, 0);
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                float f[VEC];
                load_place<IO, W, VEC>(p, sp, (int)s, len - (W - 1) + k, c, f);
                store_vec<IO, VEC>(p.state_out + ((size_t)s * (W - 1) + k) * p.D + c, f);
            }
        }
    }
    const long long first = warp * p.run;
    if (first >= p.q.total) return;
    const int t0 = (int)first, t1 = (int)min((long long)p.q.total, first + p.run);

    float w[W][VEC], bias[VEC];
    load_weights<W, VEC>(p.w, p.bias, c, w, bias);
    for (int s = p.q.of(t0); s < p.q.n; ++s) {
        const Span sp{p.q.begin(s), p.q.end(s), p.reverse};
        if (sp.b >= t1) break;
        int i0, i1;
        run_places(sp, t0, t1, i0, i1);
        if (i0 >= i1) continue;
        float x[W][VEC];  // x[k]: place i - (W - 1) + k
#pragma unroll
        for (int k = 1; k < W; ++k)
            load_place<IO, W, VEC>(p, sp, s, i0 - W + k, c, x[k]);
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
            const size_t at = (size_t)sp.token(i) * p.D + c;
#pragma unroll
            for (int k = 0; k + 1 < W; ++k) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[k][j] = x[k + 1][j];
            }
            load_f<IO, VEC>(p.x + at, x[W - 1]);
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float a = bias[j];
#pragma unroll
                for (int k = 0; k < W; ++k) a = fmaf(w[k][j], x[k][j], a);
                y[j] = act_f(a, p.act);
            }
            store_vec<IO, VEC>(p.y + at, y);
        }
    }
}

template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(kConvThreads)
conv_bwd_kernel(const ConvParams<IO> p) {
    __shared__ float sh[kConvWarps][32 * VEC];
    const int lane = threadIdx.x, wid = threadIdx.y;
    const int c = (blockIdx.y * 32 + lane) * VEC;
    const bool on = c < p.D;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        check_cu(p.q, p.status, wid * 32 + lane, kConvThreads);
    const long long warp = (long long)blockIdx.x * kConvWarps + wid;
    const long long warps = (long long)gridDim.x * kConvWarps;
    if (p.dstate && on) {  // nothing reads an empty sequence's state
        for (long long s = warp; s < p.q.n; s += warps) {
            if (p.q.begin((int)s) < p.q.end((int)s)) continue;
            const float z[VEC] = {};
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                store_vec<IO, VEC>(p.dstate + ((size_t)s * (W - 1) + k) * p.D + c, z);
        }
    }
    const long long first = warp * p.run;
    const int t0 = (int)min((long long)p.q.total, first);
    const int t1 = (int)min((long long)p.q.total, first + p.run);

    float dw[W][VEC] = {}, db[VEC] = {};
    if (on && t0 < t1) {
        float w[W][VEC], bias[VEC];
        load_weights<W, VEC>(p.w, p.bias, c, w, bias);
        for (int s = p.q.of(t0); s < p.q.n; ++s) {
            const Span sp{p.q.begin(s), p.q.end(s), p.reverse};
            if (sp.b >= t1) break;
            int i0, i1;
            run_places(sp, t0, t1, i0, i1);
            if (i0 >= i1) continue;
            const int len = sp.e - sp.b;
            float x[W][VEC], dp[W][VEC];  // places i - (W - 1) .. i
#pragma unroll
            for (int k = 1; k < W; ++k) {
                load_place<IO, W, VEC>(p, sp, s, i0 - W + k, c, x[k]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) dp[k][j] = 0.f;
            }
            // each step brings dp of place i in and dx of place i - (W - 1) out: places ahead
            // of the run's end complete its last tokens, zeros behind the sequence's
            const int first_out = i0 == 0 ? -(W - 1) : i0;
#pragma unroll 2
            for (int i = i0; i < i1 + W - 1; ++i) {
#pragma unroll
                for (int k = 0; k + 1 < W; ++k) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) { x[k][j] = x[k + 1][j]; dp[k][j] = dp[k + 1][j]; }
                }
                if (i < len) {
                    const size_t at = (size_t)sp.token(i) * p.D + c;
                    float dy[VEC];
                    load_f<IO, VEC>(p.x + at, x[W - 1]);
                    load_f<IO, VEC>(p.dy + at, dy);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        float a = bias[j], v, d;
#pragma unroll
                        for (int k = 0; k < W; ++k) a = fmaf(w[k][j], x[k][j], a);
                        act_both(a, p.act, v, d);
                        dp[W - 1][j] = dy[j] * d;
                    }
                    if (i < i1) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            db[j] += dp[W - 1][j];
#pragma unroll
                            for (int k = 0; k < W; ++k) dw[k][j] = fmaf(dp[W - 1][j], x[k][j], dw[k][j]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) dp[W - 1][j] = 0.f;
                }
                const int out = i - (W - 1);
                if (out < first_out) continue;
                float dx[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    dx[j] = 0.f;  // dx_out = sum_j w[W-1-j] dp_{out + j}
#pragma unroll
                    for (int k = 0; k < W; ++k) dx[j] = fmaf(w[W - 1 - k][j], dp[k][j], dx[j]);
                }
                if (out >= 0) store_vec<IO, VEC>(p.dx + (size_t)sp.token(out) * p.D + c, dx);
                else if (p.dstate)
                    store_vec<IO, VEC>(p.dstate + ((size_t)s * (W - 1) + (W - 1 + out)) * p.D + c, dx);
            }
        }
    }
    // the block's runs, then one row of partial sums a block
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            float v = db[j];
#pragma unroll
            for (int kk = 0; kk < W; ++kk) v = kk == k ? dw[kk][j] : v;
            sh[wid][lane * VEC + j] = v;
        }
        __syncthreads();
        for (int i = wid * 32 + lane; i < 32 * VEC; i += kConvThreads) {
            const int ch = blockIdx.y * 32 * VEC + i;
            if (ch >= p.D) break;
            float v = 0.f;
#pragma unroll
            for (int g = 0; g < kConvWarps; ++g) v += sh[g][i];
            p.part[((size_t)blockIdx.x * (W + 1) + k) * p.D + ch] = v;
        }
    }
}

// dw, dbias from the partial sums: 32 channels a block, its 8 warps over the rows.
template <int W>
__global__ void __launch_bounds__(256)
conv_reduce_kernel(const float* __restrict__ part, int rows, int D, float* __restrict__ dw,
                   float* __restrict__ dbias) {
    __shared__ float sh[8][32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    float v = 0.f;
    if (c < D)
        for (int r = wid; r < rows; r += 8) v += part[((size_t)r * (W + 1) + k) * D + c];
    sh[wid][lane] = v;
    __syncthreads();
    if (wid != 0 || c >= D) return;
#pragma unroll
    for (int g = 1; g < 8; ++g) v += sh[g][lane];
    if (k < W) dw[(size_t)c * W + k] = v;
    else if (dbias) dbias[c] = v;
}

template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(128)
conv_step_kernel(const IO* __restrict__ x, const float* __restrict__ w,
                 const float* __restrict__ bias, const IO* state, IO* state_out,
                 IO* __restrict__ y, int D, int act) {
    const int c = (blockIdx.x * 128 + threadIdx.x) * VEC;
    if (c >= D) return;
    const size_t n = blockIdx.y + (size_t)blockIdx.z * gridDim.y;
    float win[W][VEC], wr[W][VEC], b[VEC], out[VEC];
    const IO* st = state + n * (W - 1) * D + c;
    // the state may be updated in place: all of it is read before any of it is written
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) win[k][j] = 0.f;
        Vec<IO, VEC> v;
        using R = typename RawOf<sizeof(IO) * VEC>::T;
        const R r = *reinterpret_cast<const R*>(st + (size_t)k * D);
        memcpy(&v, &r, sizeof(R));
#pragma unroll
        for (int j = 0; j < VEC; ++j) win[k][j] = to_f(v.x[j]);
    }
    load_f<IO, VEC>(x + n * D + c, win[W - 1]);
    load_weights<W, VEC>(w, bias, c, wr, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float a = b[j];
#pragma unroll
        for (int k = 0; k < W; ++k) a = fmaf(wr[k][j], win[k][j], a);
        out[j] = act_f(a, act);
    }
    store_vec<IO, VEC>(y + n * D + c, out);
    IO* so = state_out + n * (W - 1) * D + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_vec<IO, VEC>(so + (size_t)k * D, win[k + 1]);
}

// ---- launching ---------------------------------------------------------------------------------

// Channels of a thread: 8 bytes where rows are whole 8-byte words, else one element.
int conv_vec(const gdr_conv_args& a) {
    const int v = a.io_dtype == GDR_BF16 ? 4 : 2;
    return a.D % v ? 1 : v;
}

// Tokens of a warp's run: long enough that the W - 1 extra tokens read at its ends cost little,
// short enough that the warps fill the GPU.
int conv_run(const gdr_conv_args& a, int vec, int most) {
    const long long slabs = (a.D + 32 * vec - 1) / (32 * vec);
    const long long tokens = (long long)a.B * a.T;
    long long run = tokens * slabs / (148 * 32);
    return (int)(run < 8 ? 8 : run > most ? most : run);
}

struct ConvGrid {
    int vec, run;
    unsigned blocks, slabs;
};

ConvGrid conv_grid(const gdr_conv_args& a, int most) {
    ConvGrid g;
    g.vec = conv_vec(a);
    g.run = conv_run(a, g.vec, most);
    const long long per = (long long)g.run * kConvWarps;
    g.blocks = (unsigned)(((long long)a.B * a.T + per - 1) / per);
    if (g.blocks == 0) g.blocks = 1;
    g.slabs = (unsigned)((a.D + 32 * g.vec - 1) / (32 * g.vec));
    return g;
}

constexpr int kFwdRun = 64, kBwdRun = 256;

template <typename IO>
ConvParams<IO> conv_params(const gdr_conv_args& a, const ConvPtrs& x, int run) {
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
    p.act = a.activation;
    p.reverse = a.reverse;
    p.run = run;
    return p;
}

struct ConvFwd {
    template <typename IO, int W, int VEC>
    static void go(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
        const ConvGrid g = conv_grid(a, kFwdRun);
        conv_fwd_kernel<IO, W, VEC><<<dim3(g.blocks, g.slabs), dim3(32, kConvWarps), 0, st>>>(
            conv_params<IO>(a, x, g.run));
    }
};

struct ConvBwd {
    template <typename IO, int W, int VEC>
    static void go(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
        const ConvGrid g = conv_grid(a, kBwdRun);
        conv_bwd_kernel<IO, W, VEC><<<dim3(g.blocks, g.slabs), dim3(32, kConvWarps), 0, st>>>(
            conv_params<IO>(a, x, g.run));
        conv_reduce_kernel<W><<<dim3((a.D + 31) / 32, W + 1), 256, 0, st>>>(
            x.ws, (int)g.blocks, a.D, x.dw, x.dbias);
    }
};

struct ConvStep {
    template <typename IO, int W, int VEC>
    static void go(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
        const unsigned bx = (unsigned)((a.D + 128 * VEC - 1) / (128 * VEC));
        for (int n0 = 0; n0 < a.B; n0 += 65535) {  // a grid's second dimension ends at 65535
            const int n = a.B - n0 < 65535 ? a.B - n0 : 65535;
            const size_t row = (size_t)n0 * a.D, srow = row * (W - 1);
            conv_step_kernel<IO, W, VEC><<<dim3(bx, n), 128, 0, st>>>(
                static_cast<const IO*>(x.x) + row, x.w, x.bias,
                static_cast<const IO*>(x.state) + srow, static_cast<IO*>(x.state_out) + srow,
                static_cast<IO*>(x.y) + row, a.D, a.activation);
        }
    }
};

template <typename Op, typename IO, int VEC>
void conv_width(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    switch (a.width) {
        case 2: Op::template go<IO, 2, VEC>(a, x, st); break;
        case 3: Op::template go<IO, 3, VEC>(a, x, st); break;
        default: Op::template go<IO, 4, VEC>(a, x, st);
    }
}

template <typename Op>
gdr_status conv_dispatch(const gdr_conv_args& a, const ConvPtrs& x, cudaStream_t st) {
    const bool one = conv_vec(a) == 1;
    if (a.io_dtype == GDR_BF16) {
        if (one) conv_width<Op, __nv_bfloat16, 1>(a, x, st);
        else conv_width<Op, __nv_bfloat16, 4>(a, x, st);
    } else {
        if (one) conv_width<Op, float, 1>(a, x, st);
        else conv_width<Op, float, 2>(a, x, st);
    }
    return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

}  // namespace

size_t conv_bwd_workspace(const gdr_conv_args& a) {
    const ConvGrid g = conv_grid(a, kBwdRun);
    return align_up(sizeof(float) * (size_t)g.blocks * (a.width + 1) * a.D, 256);
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
