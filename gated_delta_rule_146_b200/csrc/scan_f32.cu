// scan_f32.cu -- gated linear recurrence: the forward's kernels for fp32.
#include "scan_fwd.cuh"

namespace gdr {
template gdr_status scan_fwd_io<float>(const gdr_scan_args&, const ScanPtrs&, cudaStream_t);
}
