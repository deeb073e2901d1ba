// scan.cu -- gated linear recurrence: the forward's dispatch, its kernels for bf16, and one token.
#include "scan_fwd.cuh"

namespace gdr {

namespace {

// ---- one token ------------------------------------------------------------------------------
// Streams the fp32 state once: 14 bytes per channel in bf16 (16 with beta).
template <typename IO, typename GT, int kWrite, int VEC>
__global__ void __launch_bounds__(256)
scan_step_kernel(const IO* __restrict__ v, const GT* __restrict__ g, const GT* __restrict__ beta,
                 const float* h, float* h_out, IO* __restrict__ o, long long n) {
    const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * VEC;
    if (at >= n) return;
    float fh[VEC], fv[VEC], fg[VEC], fb[VEC] = {};
    const Vec<float, VEC> state = load_in_place<float, VEC>(h + at);  // h_out may be h
    load_f<IO, VEC>(v + at, fv);
    load_f<GT, VEC>(g + at, fg);
    if constexpr (kWrite == GDR_WRITE_GATE) load_f<GT, VEC>(beta + at, fb);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const F2 g2 = f2(fg[j]), a = exp2ch(g2);
        float b = fv[j];
        if constexpr (kWrite == GDR_WRITE_GATE) b *= fb[j];
        if constexpr (kWrite == GDR_WRITE_TIED) b *= one_minus(g2, a).lo();
        fh[j] = fmaf(a.lo(), state.x[j], b);
    }
    store_vec<float, VEC>(h_out + at, fh);
    store_vec<IO, VEC>(o + at, fh);
}

struct Step {
    template <typename IO, typename GT, int kWrite>
    static gdr_status go(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
        const long long n = (long long)a.B * a.D;  // the rows join: only the end can be ragged
        const IO* v = static_cast<const IO*>(x.v);
        const GT *g = static_cast<const GT*>(x.g), *b = static_cast<const GT*>(x.beta);
        IO* o = static_cast<IO*>(x.o);
        const int vec = n % 4 ? 1 : 4;
        const long long blocks = (n / vec + 255) / 256;
        if (vec == 4)
            scan_step_kernel<IO, GT, kWrite, 4><<<(unsigned)blocks, 256, 0, st>>>(
                v, g, b, x.h0, x.h_final, o, n);
        else
            scan_step_kernel<IO, GT, kWrite, 1><<<(unsigned)blocks, 256, 0, st>>>(
                v, g, b, x.h0, x.h_final, o, n);
        return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
    }
};

}  // namespace

extern template gdr_status scan_fwd_io<float>(const gdr_scan_args&, const ScanPtrs&, cudaStream_t);
template gdr_status scan_fwd_io<__nv_bfloat16>(const gdr_scan_args&, const ScanPtrs&, cudaStream_t);

gdr_status launch_scan_fwd(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    if (a.B * (long long)a.T == 0) {  // every state stays
        const size_t bytes = sizeof(float) * (size_t)a.n_seqs * a.D;
        if (!x.h_final || x.h_final == x.h0) return GDR_OK;
        const cudaError_t e = x.h0 ? cudaMemcpyAsync(x.h_final, x.h0, bytes,
                                                     cudaMemcpyDeviceToDevice, st)
                                   : cudaMemsetAsync(x.h_final, 0, bytes, st);
        return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
    }
    return a.io_dtype == GDR_BF16 ? scan_fwd_io<__nv_bfloat16>(a, x, st) : scan_fwd_io<float>(a, x, st);
}

gdr_status launch_scan_step(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    return a.io_dtype == GDR_BF16 ? scan_dispatch_gate<Step, __nv_bfloat16>(a, x, st)
                                  : scan_dispatch_gate<Step, float>(a, x, st);
}

}  // namespace gdr
