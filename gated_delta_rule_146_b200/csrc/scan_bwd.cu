// scan_bwd.cu -- gated linear recurrence: the backward's dispatch, its kernels for bf16.
#include "scan_bwd.cuh"

namespace gdr {

extern template gdr_status scan_bwd_io<float>(const gdr_scan_args&, const ScanPtrs&, cudaStream_t);
template gdr_status scan_bwd_io<__nv_bfloat16>(const gdr_scan_args&, const ScanPtrs&, cudaStream_t);

gdr_status launch_scan_bwd(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    if (a.B * (long long)a.T == 0) {
        const size_t bytes = sizeof(float) * (size_t)a.n_seqs * a.D;
        if (!x.dh0 || x.dh0 == x.dh_final) return GDR_OK;
        const cudaError_t e = x.dh_final ? cudaMemcpyAsync(x.dh0, x.dh_final, bytes,
                                                           cudaMemcpyDeviceToDevice, st)
                                         : cudaMemsetAsync(x.dh0, 0, bytes, st);
        return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
    }
    return a.io_dtype == GDR_BF16 ? scan_bwd_io<__nv_bfloat16>(a, x, st) : scan_bwd_io<float>(a, x, st);
}

}  // namespace gdr
