// norm_impl.cuh -- what the kernels of the group norm share: how a group's channels lie in a
// warp, sums over them, and the formulas of one element.
//
// The d channels of one token's head are spread over LPG lanes, NV vectors of VEC channels each:
// 16 bytes where rows are whole such words, else two elements, read one by one.  A warp so holds
// 32 / LPG heads and reads whole lines of a tensor.  Channels go in pairs through packed fp32
// arithmetic; lanes behind the last channel hold zeros.
#pragma once

#include "layer.cuh"

namespace gdr {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;

template <typename IO_, bool kWhole_, int LPG_, int NV_>
struct Shape {
    using IO = IO_;
    static constexpr bool kWhole = kWhole_;
    static constexpr int VEC = kWhole ? 16 / (int)sizeof(IO) : 2, LPG = LPG_, NV = NV_;
    static constexpr int kGroups = kNormThreads / LPG;  // heads a block holds at once
    // results in bf16, or of rounded sums, do not show the coarser sigmoid's error (layer.cuh)
    static constexpr bool kFine = sizeof(IO) == 4;
    // rows of a lane group on their way at once, and blocks on an SM that the registers allow
    static constexpr int kStages = NV == 1 ? 3 : 2;
    static constexpr int kResident = NV == 1 ? 3 : NV == 2 ? 2 : 1;
    // of the per-token backward: with its sums in registers two blocks are faster than three that
    // spill a little (8 x 4096 x 16 x 128 in bf16, gated: 113 us against 129)
    static constexpr int kResidentSums = NV <= 2 ? 2 : 1;
};

template <typename IO>
struct NormParams {
    const IO *x, *z, *dy;
    const float *w, *b;
    IO *y, *dx, *dz;
    const float* stats;   // [n_seqs][H][2], per sequence
    float* part;          // partial sums
    int* status;
    Seqs q;
    int H, d, center, act, shared;
    float eps;
    long long rows;       // tokens times heads
};

template <int LPG>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = LPG / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One lane's channels of a row, as they lie in memory.
template <typename S>
struct Raw {
    Vec<typename S::IO, S::VEC> v[S::NV];
};
// The same in fp32.
template <typename S>
struct Pairs {
    F2 f[S::NV][S::VEC / 2];
};

template <typename S>
__device__ __forceinline__ Raw<S> load_row(const typename S::IO* p, int l, int d, bool on) {
    using IO = typename S::IO;
    Raw<S> r;
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = (k * S::LPG + l) * S::VEC;
        if (S::kWhole && on && c < d) {
            r.v[k] = load_vec<IO, S::VEC>(p + c);
        } else {
#pragma unroll
            for (int j = 0; j < S::VEC; ++j)
                r.v[k].x[j] = !S::kWhole && on && c + j < d ? p[c + j] : from_f<IO>(0.f);
        }
    }
    return r;
}

// A lane's next rows of kT tensors, on their way into shared memory of its own: no registers, no
// barrier.  Tensors behind the first `used` are left out.
template <typename S, int kT>
struct Ring {
    using IO = typename S::IO;
    using V = Vec<IO, S::VEC>;
    static constexpr int kStage = kT * S::NV * kNormThreads;   // vectors of a stage
    static constexpr int kBytes = S::kStages * kStage * (int)sizeof(V);
    V* first;
    long long at, hop;  // the lane's first channel of the row to be asked for; elements to the next
    int put, got;       // stages' first vectors
    int l, d, used, rest;

    __device__ __forceinline__ Ring(char* smem, int l_, int d_, int used_, long long hop_)
        : first(reinterpret_cast<V*>(smem) + threadIdx.x), hop(hop_), l(l_), d(d_), used(used_) {}
    // asks for the next row of the tensors, if there is one, and commits
    __device__ __forceinline__ void ask(const IO* const (&base)[kT]) {
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            if (t >= used) break;
            V* const to = first + put + t * S::NV * kNormThreads;
            if constexpr (S::kWhole) {
#pragma unroll
                for (int k = 0; k < S::NV; ++k)
                    copy_async<16>(smem_u32(to + k * kNormThreads), base[t] + at + k * S::LPG * S::VEC,
                                   rest > 0 && (k * S::LPG + l) * S::VEC < d);
            } else {
                const Raw<S> r = load_row<S>(base[t] + at - l * S::VEC, l, d, rest > 0);
#pragma unroll
                for (int k = 0; k < S::NV; ++k) to[k * kNormThreads] = r.v[k];
            }
        }
        copy_commit();
        at += hop;
        --rest;
        put = put == (S::kStages - 1) * kStage ? 0 : put + kStage;
    }
    // `rows` rows from the ones at element `from` of the tensors on
    __device__ __forceinline__ void open(const IO* const (&base)[kT], size_t from, int rows) {
        copy_wait<0>();
        put = got = 0;
        rest = rows;
        at = (long long)from + l * S::VEC;
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) ask(base);
    }
    // the row asked for longest ago; asks for another (zeros behind the last)
    __device__ __forceinline__ void take(const IO* const (&base)[kT], Raw<S> (&r)[kT]) {
        copy_wait<S::kStages - 2>();
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            if (t >= used) break;
#pragma unroll
            for (int k = 0; k < S::NV; ++k) r[t].v[k] = first[got + (t * S::NV + k) * kNormThreads];
        }
        got = got == (S::kStages - 1) * kStage ? 0 : got + kStage;
        ask(base);
    }
};

template <typename S>
__device__ __forceinline__ Pairs<S> widen(const Raw<S>& r) {
    Pairs<S> f;
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) f.f[k][j] = pair_of(r.v[k], j);
    }
    return f;
}

template <typename S>
__device__ __forceinline__ void store_row(typename S::IO* p, int l, int d, const Pairs<S>& f) {
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = (k * S::LPG + l) * S::VEC;
        Vec<typename S::IO, S::VEC> v;
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) set_pair(v, j, f.f[k][j]);
        if constexpr (S::kWhole) {
            if (c < d) store_raw(p + c, v);
        } else {
#pragma unroll
            for (int j = 0; j < S::VEC; ++j)
                if (c + j < d) p[c + j] = v.x[j];
        }
    }
}

template <typename S>
__device__ __forceinline__ Pairs<S> fill(float x) {
    Pairs<S> f;
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) f.f[k][j] = f2(x);
    }
    return f;
}

// The lane's weights (or biases): ones (zeros) where there are none.
template <typename S>
__device__ __forceinline__ Pairs<S> load_affine(const float* w, float none, int head, int l, int d,
                                                int shared) {
    Pairs<S> f;
    const size_t row = shared ? 0 : (size_t)head * d;
    auto at = [&](int c) { return w && c < d ? __ldg(w + row + c) : none; };
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) {
            const int c = (k * S::LPG + l) * S::VEC + 2 * j;
            f.f[k][j] = f2(at(c), at(c + 1));
        }
    }
    return f;
}

template <typename S>
__device__ __forceinline__ float lane_sum(const Pairs<S>& x) {
    F2 s = x.f[0][0];
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j)
            if (k + j) s = add2(s, x.f[k][j]);
    }
    return s.lo() + s.hi();
}

// x - mean; zeros stay where there are no channels
template <typename S>
__device__ __forceinline__ void centre(Pairs<S>& x, float mean, int l, int d) {
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = (k * S::LPG + l) * S::VEC;
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) {
            const F2 m = S::kWhole ? f2(c < d ? -mean : 0.f)
                                   : f2(c < d ? -mean : 0.f, c + 1 < d ? -mean : 0.f);
            x.f[k][j] = add2(x.f[k][j], m);
        }
    }
}

template <typename S>
__device__ __forceinline__ float lane_squares(const Pairs<S>& x) {
    F2 s = f2(0.f);
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) s = fma2(x.f[k][j], x.f[k][j], s);
    }
    return s.lo() + s.hi();
}

// Calls f with the activation and the gate as compile-time constants: one branch for a row.
template <int kAct_, bool kGate_>
struct Form {
    static constexpr int kAct = kAct_;
    static constexpr bool kGate = kGate_;
};
template <typename F>
__device__ __forceinline__ void with_form(int act, bool gate, F f) {
    if (act == GDR_ACT_SILU) {
        if (gate) f(Form<GDR_ACT_SILU, true>{}); else f(Form<GDR_ACT_SILU, false>{});
    } else if (act == GDR_ACT_SIGMOID) {
        if (gate) f(Form<GDR_ACT_SIGMOID, true>{}); else f(Form<GDR_ACT_SIGMOID, false>{});
    } else {
        if (gate) f(Form<GDR_ACT_NONE, true>{}); else f(Form<GDR_ACT_NONE, false>{});
    }
}

// y from the centred x: n = x rstd, u = n w + b, y = u act(z) or act(u)
template <typename S, typename Fm>
__device__ __forceinline__ Pairs<S> norm_rows(Fm, const Pairs<S>& x, const Pairs<S>& w, const Pairs<S>& b,
                                              const Raw<S>& z, float rstd) {
    Pairs<S> y;
    const F2 r = f2(rstd);
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) {
            const F2 u = fma2(mul2(x.f[k][j], r), w.f[k][j], b.f[k][j]);
            if constexpr (Fm::kGate) y.f[k][j] = mul2(u, act2<Fm::kAct, S::kFine>(pair_of(z.v[k], j)));
            else y.f[k][j] = act2<Fm::kAct, S::kFine>(u);
        }
    }
    return y;
}

// What the backward has of a row (x centred): n, q = du w, dz; du joins the sums for dw and (kBias)
// db if kSums.  Without kBias there is no bias either: sixteen registers less.
template <typename S>
struct Back {
    Pairs<S> n, q, dz;
    float s1, s2;   // the lane's sums of q and q n
};
template <typename S, bool kSums, bool kBias, typename Fm>
__device__ __forceinline__ Back<S> back_rows(Fm, const Pairs<S>& x, const Raw<S>& dy, const Raw<S>& z,
                                             const Pairs<S>& w, const Pairs<S>& b, float rstd,
                                             Pairs<S>& dw, Pairs<S>& db) {
    Back<S> o;
    const F2 r = f2(rstd);
    F2 s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j) {
            const F2 n = mul2(x.f[k][j], r), g = pair_of(dy.v[k], j);
            const F2 u = kBias ? fma2(n, w.f[k][j], b.f[k][j]) : mul2(n, w.f[k][j]);
            F2 a, da, du;
            act2_both<Fm::kAct, S::kFine>(Fm::kGate ? pair_of(z.v[k], j) : u, a, da);
            if constexpr (Fm::kGate) {
                o.dz.f[k][j] = mul2(mul2(g, u), da);
                du = mul2(g, a);
            } else {
                du = mul2(g, da);
            }
            if (kSums) {
                dw.f[k][j] = fma2(du, n, dw.f[k][j]);
                if (kBias) db.f[k][j] = add2(db.f[k][j], du);
            }
            const F2 q = mul2(du, w.f[k][j]);
            s1 = add2(s1, q);
            s2 = fma2(q, n, s2);
            o.n.f[k][j] = n;
            o.q.f[k][j] = q;
        }
    }
    o.s1 = s1.lo() + s1.hi();
    o.s2 = s2.lo() + s2.hi();
    return o;
}

// dx = rstd (q - mean(q) - n mean(q n))
template <typename S>
__device__ __forceinline__ Pairs<S> back_dx(const Back<S>& o, float rstd, float mq, float mqn) {
    Pairs<S> dx;
    const F2 r = f2(rstd), m1 = f2(-mq), m2 = f2(-mqn);
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC / 2; ++j)
            dx.f[k][j] = mul2(fma2(o.n.f[k][j], m2, add2(o.q.f[k][j], m1)), r);
    }
    return dx;
}

// Calls Op::go<Shape>(a, x, st) for the shape that holds d channels; see norm_supported.
template <typename Op, typename IO>
void norm_dispatch_io(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    constexpr int V = 16 / sizeof(IO);
    if (a.d % V == 0) {
        const int n = a.d / V;
        if (n <= 4) Op::template go<Shape<IO, true, 4, 1>>(a, x, st);
        else if (n <= 8) Op::template go<Shape<IO, true, 8, 1>>(a, x, st);
        else if (n <= 16) Op::template go<Shape<IO, true, 16, 1>>(a, x, st);
        else if (n <= 32) Op::template go<Shape<IO, true, 32, 1>>(a, x, st);
        else if (n <= 64) Op::template go<Shape<IO, true, 32, 2>>(a, x, st);
        else if (V == 8 || n <= 128) Op::template go<Shape<IO, true, 32, 4>>(a, x, st);
        else if constexpr (V == 4) Op::template go<Shape<IO, true, 32, 8>>(a, x, st);
    } else if (a.d <= 64) Op::template go<Shape<IO, false, 32, 1>>(a, x, st);
    else if (a.d <= 128) Op::template go<Shape<IO, false, 32, 2>>(a, x, st);
    else Op::template go<Shape<IO, false, 32, 4>>(a, x, st);
}

// Lane groups of a block (Shape::kGroups of the shape the dispatch below takes).
inline int norm_groups(const gdr_norm_args& a) {
    const int v = a.io_dtype == GDR_BF16 ? 8 : 4;
    const int n = a.d % v ? 32 : a.d / v;
    return kNormThreads / (n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32);
}

template <typename Op>
void norm_shape(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    if (a.io_dtype == GDR_BF16) norm_dispatch_io<Op, __nv_bfloat16>(a, x, st);
    else norm_dispatch_io<Op, float>(a, x, st);
}

// Launches with the shared memory of a ring.
template <int kBytes, bool kFollows = false, typename... P, typename... A>
void norm_launch(void (*kernel)(P...), long long blocks, cudaStream_t st, A... args) {
    if (kBytes > 40 << 10)  // (with the kernels' own arrays, above what needs no asking for)
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (kFollows)
        launch_follower(kernel, dim3((unsigned)blocks), dim3(kNormThreads), kBytes, st, args...);
    else
        kernel<<<(unsigned)blocks, kNormThreads, kBytes, st>>>(args...);
}

template <typename Op>
gdr_status norm_dispatch(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    norm_shape<Op>(a, x, st);
    return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

template <typename IO>
NormParams<IO> norm_params(const gdr_norm_args& a, const NormPtrs& x) {
    NormParams<IO> p;
    p.x = static_cast<const IO*>(x.x);
    p.z = static_cast<const IO*>(x.z);
    p.dy = static_cast<const IO*>(x.dy);
    p.w = x.w;
    p.b = x.b;
    p.y = static_cast<IO*>(x.y);
    p.dx = static_cast<IO*>(x.dx);
    p.dz = static_cast<IO*>(x.dz);
    p.stats = x.stats_in;
    p.part = x.ws;
    p.status = a.status;
    p.q = Seqs{x.cu, a.n_seqs, a.T, a.B * a.T};
    p.H = a.H;
    p.d = a.d;
    p.center = a.center;
    p.act = a.activation;
    p.shared = a.shared_weight;
    p.eps = a.eps;
    p.rows = (long long)a.B * a.T * a.H;
    return p;
}

// Sums part[0 .. rows)[2][H][d] over the rows (and the heads of a shared weight) into dw, db.
void launch_norm_reduce(const gdr_norm_args& a, const float* part, int rows, float* dw,
                              float* db, cudaStream_t st);

gdr_status launch_norm_seq_fwd(const gdr_norm_args& a, const NormPtrs& p, cudaStream_t st);
gdr_status launch_norm_seq_bwd(const gdr_norm_args& a, const NormPtrs& p, cudaStream_t st);
size_t norm_seq_fwd_workspace(const gdr_norm_args& a);
size_t norm_seq_bwd_workspace(const gdr_norm_args& a);

}  // namespace gdr
