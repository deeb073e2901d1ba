// layer.cuh -- shared by the operators around the delta rule (scan.cu, conv.cu, norm.cu):
// the sequences of a call, vector access in either dtype, activations.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace gdr {

using tc::ex2;
using tc::smem_u32;

// ---- sequences ------------------------------------------------------------------------------
// The tokens of a call lie on one axis of `total` rows: B rows of T tokens one after the other,
// or packed sequences bounded by cu.  Every offset read from cu is clamped to [0, total], so
// that no access leaves the tensors whatever cu holds; check_cu reports a bad one.
struct Seqs {
    const int32_t* cu;  // [n + 1], or NULL: sequence s is row s
    int n, T;
    int total;
    __device__ __forceinline__ int begin(int s) const {
        return cu ? min(max(cu[s], 0), total) : s * T;
    }
    __device__ __forceinline__ int end(int s) const {
        return cu ? min(max(cu[s + 1], 0), total) : (s + 1) * T;
    }
    // the sequence that holds token t (the last s with begin(s) <= t: an empty sequence shares
    // its offset with the next one and loses the tie)
    __device__ __forceinline__ int of(int t) const {
        if (!cu) return t / T;
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= t) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
};

// One block's threads: records GDR_ERR_DEVICE_CHECK in *status unless cu is 0 .. total and
// never decreases.
__device__ __forceinline__ void check_cu(const Seqs& q, int* status, int tid, int threads) {
    if (!q.cu || !status) return;
    bool bad = false;
#pragma unroll 4
    for (int s = tid; s <= q.n; s += threads) {
        const int x = q.cu[s];
        bad |= (s == 0 && x != 0) || (s == q.n && x != q.total) || (s > 0 && x < q.cu[s - 1]);
    }
    if (bad) atomicCAS(status, (int)GDR_OK, (int)GDR_ERR_DEVICE_CHECK);
}

// ---- vector access -----------------------------------------------------------------------------
template <int kBytes> struct RawOf;
template <> struct RawOf<2> { using T = uint16_t; };
template <> struct RawOf<4> { using T = uint32_t; };
template <> struct RawOf<8> { using T = uint2; };
template <> struct RawOf<16> { using T = uint4; };

// N neighbouring elements as they lie in memory.
template <typename E, int N>
struct alignas(sizeof(E) * N) Vec {
    E x[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E> __device__ __forceinline__ E from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// Two values rounded to bf16 in one word, by one instruction.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

template <typename E, int N>
__device__ __forceinline__ Vec<E, N> load_vec(const E* p) {
    using R = typename RawOf<sizeof(E) * N>::T;
    Vec<E, N> v;
    const R r = __ldg(reinterpret_cast<const R*>(p));
    memcpy(&v, &r, sizeof(R));
    return v;
}

// The same of an array that the kernel may also write (a state updated in place): an ordinary
// load, which keeps its place among the barriers and stores around it.
template <typename E, int N>
__device__ __forceinline__ Vec<E, N> load_in_place(const E* p) {
    using R = typename RawOf<sizeof(E) * N>::T;
    Vec<E, N> v;
    const R r = *reinterpret_cast<const R*>(p);
    memcpy(&v, &r, sizeof(R));
    return v;
}

template <typename E, int N>
__device__ __forceinline__ void store_vec(E* p, const float (&f)[N]) {
    using R = typename RawOf<sizeof(E) * N>::T;
    Vec<E, N> v;
    if constexpr (sizeof(E) == 2 && N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint32_t w = bf16x2(f[i], f[i + 1]);
            memcpy(&v.x[i], &w, 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v.x[i] = from_f<E>(f[i]);
    }
    R r;
    memcpy(&r, &v, sizeof(R));
    *reinterpret_cast<R*>(p) = r;
}

template <typename E, int N>
__device__ __forceinline__ void load_f(const E* p, float (&f)[N]) {
    const Vec<E, N> v = load_vec<E, N>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f(v.x[i]);
}

// ---- asynchronous copies into shared memory ----------------------------------------------------
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

// ---- two channels in one 64-bit register pair ---------------------------------------------------
struct F2 {
    uint64_t v;
    __device__ __forceinline__ float lo() const { return __uint_as_float((uint32_t)v); }
    __device__ __forceinline__ float hi() const { return __uint_as_float((uint32_t)(v >> 32)); }
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 pick2(bool c, F2 a, F2 b) { return F2{c ? a.v : b.v}; }

// max that lets NaN through
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// e^x = 2^(x log2 e).  The product is rounded; what the rounding left out, e, and the low part of
// log2 e multiply the result by 2^e = 1 + e ln 2 to first order (e is below 2^-16 in the range).
// x has to be finite, and below 88.
__device__ __forceinline__ F2 exp_in_range(F2 x) {
    const F2 t = mul2(x, f2(1.44269504f));
    F2 e = fma2(x, f2(-1.44269504f), t);  // -e
    e = fma2(x, f2(-1.92596303e-8f), e);
    const F2 m = f2(ex2(t.lo()), ex2(t.hi()));
    return fma2(mul2(m, e), f2(-0.693147181f), m);
}

// e^g for g <= 0 and above as far as it stays finite.  Below e^-150 the result is zero in either
// case, and the clamp keeps -inf out of the products.
__device__ __forceinline__ F2 exp2ch(F2 g) {
    return exp_in_range(f2(max_nan(g.lo(), -150.f), max_nan(g.hi(), -150.f)));
}

// ---- activations -------------------------------------------------------------------------------
// sigmoid(x) = 1 / (1 + e^-x).
// kFine: exponential and reciprocal are off by one step of fp32 each.  At the lower clamp e^-x is
// above 2^126, whose reciprocal the hardware flushes to zero: so it is for all x below, and
// x sigmoid(x) is -0 (NaN for -inf, as -inf times 0 is).
// Else e^-x is off by another |x| half steps, from the rounded product with log2 e: no more than a
// last-place error of x itself would do, for an x that is a rounded sum or a result that is rounded
// to bf16.  It needs no clamps (infinities go the right way) and half the instructions.
template <bool kFine>
__device__ __forceinline__ F2 sigmoid2(F2 x) {
    if constexpr (!kFine) {
        const F2 t = mul2(x, f2(-1.44269504f));
        const F2 s = add2(f2(ex2(t.lo()), ex2(t.hi())), f2(1.f));
        return f2(rcp_ftz(s.lo()), rcp_ftz(s.hi()));
    }
    const F2 c = f2(min_nan(max_nan(-x.lo(), -88.f), 87.7f), min_nan(max_nan(-x.hi(), -88.f), 87.7f));
    const F2 s = add2(exp_in_range(c), f2(1.f));
    return f2(rcp_ftz(s.lo()), rcp_ftz(s.hi()));
}

template <int kAct, bool kFine>
__device__ __forceinline__ F2 act2(F2 x) {
    if constexpr (kAct == GDR_ACT_NONE) return x;
    const F2 s = sigmoid2<kFine>(x);
    return kAct == GDR_ACT_SILU ? mul2(x, s) : s;
}

// act(x) and act'(x)
template <int kAct, bool kFine>
__device__ __forceinline__ void act2_both(F2 x, F2& a, F2& d) {
    if constexpr (kAct == GDR_ACT_NONE) {
        a = x;
        d = f2(1.f);
    } else {
        const F2 s = sigmoid2<kFine>(x), rest = fma2(s, f2(-1.f), f2(1.f));
        if constexpr (kAct == GDR_ACT_SILU) {
            a = mul2(x, s);
            d = mul2(s, fma2(x, rest, f2(1.f)));
        } else {
            a = s;
            d = mul2(s, rest);
        }
    }
}

// The pair at word i of N neighbouring elements, and the way back.
template <typename E, int N>
__device__ __forceinline__ F2 pair_of(const Vec<E, N>& v, int i) {
    if constexpr (sizeof(E) == 2) {
        uint32_t r;
        memcpy(&r, &v.x[2 * i], 4);
        return f2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    } else {
        return f2(v.x[2 * i], v.x[2 * i + 1]);
    }
}
template <typename E, int N>
__device__ __forceinline__ void set_pair(Vec<E, N>& v, int i, F2 f) {
    if constexpr (sizeof(E) == 2) {
        const uint32_t w = bf16x2(f.lo(), f.hi());
        memcpy(&v.x[2 * i], &w, 4);
    } else {
        v.x[2 * i] = f.lo();
        v.x[2 * i + 1] = f.hi();
    }
}
template <typename E, int N>
__device__ __forceinline__ void store_raw(E* p, const Vec<E, N>& v) {
    using R = typename RawOf<sizeof(E) * N>::T;
    R r;
    memcpy(&r, &v, sizeof(R));
    *reinterpret_cast<R*>(p) = r;
}

// ---- kernels that follow one another --------------------------------------------------------------
// A follower is launched while its predecessor still runs, and waits for its results here, before
// it reads any of them or writes anything.  The predecessor lets it come when it calls let_follow,
// or ends.  What a predecessor writes while a follower runs is not read-only to the follower, which
// takes it through ordinary pointers (not __restrict__, no __ldg): their loads stay behind the wait.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_follow() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_follower(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                            A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// ---- launchers (host) ----------------------------------------------------------------------------
struct ScanPtrs {
    const void *v, *g, *beta, *o_in, *dO;
    const float *h0, *dh_final;
    const int32_t* cu;
    void *o, *dv, *dg, *dbeta;
    float *h_final, *dh0;
};
gdr_status launch_scan_fwd(const gdr_scan_args& a, const ScanPtrs& p, cudaStream_t st);
gdr_status launch_scan_bwd(const gdr_scan_args& a, const ScanPtrs& p, cudaStream_t st);
gdr_status launch_scan_step(const gdr_scan_args& a, const ScanPtrs& p, cudaStream_t st);

struct ConvPtrs {
    const void *x, *state, *dy;
    const float *w, *bias;
    const int32_t* cu;
    void *y, *state_out, *dx, *dstate;
    float *dw, *dbias, *ws;
};
size_t conv_bwd_workspace(const gdr_conv_args& a);
gdr_status launch_conv_fwd(const gdr_conv_args& a, const ConvPtrs& p, cudaStream_t st);
gdr_status launch_conv_bwd(const gdr_conv_args& a, const ConvPtrs& p, cudaStream_t st);
gdr_status launch_conv_step(const gdr_conv_args& a, const ConvPtrs& p, cudaStream_t st);

struct NormPtrs {
    const void *x, *z, *dy;
    const float *w, *b, *stats_in;
    const int32_t* cu;
    void *y, *dx, *dz;
    float *stats, *dw, *db, *ws;
};
bool norm_supported(const gdr_norm_args& a);
size_t norm_fwd_workspace(const gdr_norm_args& a);
size_t norm_bwd_workspace(const gdr_norm_args& a);
gdr_status launch_norm_fwd(const gdr_norm_args& a, const NormPtrs& p, cudaStream_t st);
gdr_status launch_norm_bwd(const gdr_norm_args& a, const NormPtrs& p, cudaStream_t st);

}  // namespace gdr
