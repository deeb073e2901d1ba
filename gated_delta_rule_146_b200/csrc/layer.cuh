// layer.cuh -- shared by the operators around the delta rule (scan.cu, conv.cu, norm.cu):
// the sequences of a call, vector access in either dtype, activations.
#pragma once

#include "common.cuh"

namespace gdr {

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

template <typename E, int N>
__device__ __forceinline__ Vec<E, N> load_vec(const E* p) {
    using R = typename RawOf<sizeof(E) * N>::T;
    Vec<E, N> v;
    const R r = __ldg(reinterpret_cast<const R*>(p));
    memcpy(&v, &r, sizeof(R));
    return v;
}

template <typename E, int N>
__device__ __forceinline__ void store_vec(E* p, const float (&f)[N]) {
    using R = typename RawOf<sizeof(E) * N>::T;
    Vec<E, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.x[i] = from_f<E>(f[i]);
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

// ---- activations -------------------------------------------------------------------------------
// sigmoid from the side that does not overflow: e^-|x| is in (0, 1].
__device__ __forceinline__ float sigmoid_f(float x) {
    const float e = expf(-fabsf(x));
    const float r = 1.f / (1.f + e);
    return x >= 0.f ? r : e * r;
}

__device__ __forceinline__ float act_f(float x, int act) {
    if (act == GDR_ACT_NONE) return x;
    const float s = sigmoid_f(x);
    return act == GDR_ACT_SILU ? x * s : s;
}

// act(x) and act'(x)
__device__ __forceinline__ void act_both(float x, int act, float& a, float& d) {
    if (act == GDR_ACT_NONE) { a = x; d = 1.f; return; }
    const float s = sigmoid_f(x);
    if (act == GDR_ACT_SILU) { a = x * s; d = s * (1.f + x * (1.f - s)); }
    else { a = s; d = s * (1.f - s); }
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
