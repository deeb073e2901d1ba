// norm_impl.cuh -- what the kernels of the group norm share: how a group's channels lie in a
// warp, sums over them, and the formulas of one element.
//
// The d channels of one token's head are spread over LPG lanes, NV vectors of VEC channels
// each (16 bytes where d allows, else one element), so a warp holds 32 / LPG heads and a row of
// a tensor is read in whole lines.
#pragma once

#include "layer.cuh"

namespace gdr {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;

template <typename IO_, int VEC_, int LPG_, int NV_>
struct Shape {
    using IO = IO_;
    static constexpr int VEC = VEC_, LPG = LPG_, NV = NV_;
    static constexpr int kGroups = kNormThreads / LPG;  // heads a block holds at once
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

// One lane's channels of a row; zero where there are none.
template <typename S>
__device__ __forceinline__ void load_row(const typename S::IO* p, int l, int d, bool on,
                                         float (&f)[S::NV][S::VEC]) {
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = (k * S::LPG + l) * S::VEC;
        if (on && c < d) load_f<typename S::IO, S::VEC>(p + c, f[k]);
        else {
#pragma unroll
            for (int j = 0; j < S::VEC; ++j) f[k][j] = 0.f;
        }
    }
}

template <typename S>
__device__ __forceinline__ void store_row(typename S::IO* p, int l, int d,
                                          const float (&f)[S::NV][S::VEC]) {
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = (k * S::LPG + l) * S::VEC;
        if (c < d) store_vec<typename S::IO, S::VEC>(p + c, f[k]);
    }
}

// The lane's weights (or biases): ones (zeros) where there are none.
template <typename S>
__device__ __forceinline__ void load_affine(const float* w, float none, int head, int l,
                                            const int d, int shared, float (&f)[S::NV][S::VEC]) {
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
#pragma unroll
        for (int j = 0; j < S::VEC; ++j) {
            const int c = (k * S::LPG + l) * S::VEC + j;
            f[k][j] = w && c < d ? __ldg(w + (shared ? 0 : (size_t)head * d) + c) : none;
        }
    }
}

// y from the normalised value n (and the gate z)
__device__ __forceinline__ float norm_out(float n, float w, float b, bool gate, float z, int act) {
    const float u = fmaf(n, w, b);
    return gate ? u * act_f(z, act) : act_f(u, act);
}

// du (the gradient of u = n w + b) and dz
__device__ __forceinline__ float norm_du(float n, float w, float b, bool gate, float z, float dy,
                                         int act, float& dz) {
    const float u = fmaf(n, w, b);
    float a, g;
    act_both(gate ? z : u, act, a, g);
    if (!gate) return dy * g;
    dz = dy * u * g;
    return dy * a;
}

// Calls Op::go<Shape>(a, x, st) for the shape that holds d channels; see norm_supported.
template <typename Op, typename IO>
void norm_dispatch_io(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    constexpr int V = 16 / sizeof(IO);
    if (a.d % V == 0) {
        const int n = a.d / V;
        if (n <= 4) Op::template go<Shape<IO, V, 4, 1>>(a, x, st);
        else if (n <= 8) Op::template go<Shape<IO, V, 8, 1>>(a, x, st);
        else if (n <= 16) Op::template go<Shape<IO, V, 16, 1>>(a, x, st);
        else if (n <= 32) Op::template go<Shape<IO, V, 32, 1>>(a, x, st);
        else if (n <= 64) Op::template go<Shape<IO, V, 32, 2>>(a, x, st);
        else if (V == 8 || n <= 128) Op::template go<Shape<IO, V, 32, 4>>(a, x, st);
        else if constexpr (V == 4) Op::template go<Shape<IO, V, 32, 8>>(a, x, st);
    } else if (a.d <= 32) Op::template go<Shape<IO, 1, 32, 1>>(a, x, st);
    else if (a.d <= 64) Op::template go<Shape<IO, 1, 32, 2>>(a, x, st);
    else if (a.d <= 128) Op::template go<Shape<IO, 1, 32, 4>>(a, x, st);
    else Op::template go<Shape<IO, 1, 32, 8>>(a, x, st);
}

// Lane groups of a block (Shape::kGroups of the shape the dispatch below takes).
inline int norm_groups(const gdr_norm_args& a) {
    const int v = a.io_dtype == GDR_BF16 ? 8 : 4;
    const int n = a.d % v ? 32 : a.d / v;
    return kNormThreads / (n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32);
}

template <typename Op>
gdr_status norm_dispatch(const gdr_norm_args& a, const NormPtrs& x, cudaStream_t st) {
    if (a.io_dtype == GDR_BF16) norm_dispatch_io<Op, __nv_bfloat16>(a, x, st);
    else norm_dispatch_io<Op, float>(a, x, st);
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
gdr_status launch_norm_reduce(const gdr_norm_args& a, const float* part, int rows, float* dw,
                              float* db, cudaStream_t st);

gdr_status launch_norm_seq_fwd(const gdr_norm_args& a, const NormPtrs& p, cudaStream_t st);
gdr_status launch_norm_seq_bwd(const gdr_norm_args& a, const NormPtrs& p, cudaStream_t st);
size_t norm_seq_fwd_workspace(const gdr_norm_args& a);
size_t norm_seq_bwd_workspace(const gdr_norm_args& a);

}  // namespace gdr
