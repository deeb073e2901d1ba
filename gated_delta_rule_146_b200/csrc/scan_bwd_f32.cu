// scan_bwd_f32.cu -- gated linear recurrence: the backward's kernels for fp32.
#include "scan_bwd.cuh"

namespace gdr {
template gdr_status scan_bwd_io<float>(const gdr_scan_args&, const ScanPtrs&, cudaStream_t);
}
