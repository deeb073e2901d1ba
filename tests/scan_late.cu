// scan_late.cu -- a cluster's hand-over of runs (scan_impl.cuh) with one block whose publisher falls
// silent: the recurrence x <- a x + b over L tokens of 64 channels, one token a worker and tile.  A
// token with a < 0 starts a sequence.
#include "scan_impl.cuh"

namespace {

using namespace gdr;
constexpr int kWarps = 2, kBlocks = 2;

struct Elements {
    F2 a, b;
    Run before;
};

__global__ void __launch_bounds__(32 * (kWarps + 2))
late_kernel(const float* a, const float* b, float* o, float* state, int* ok_out, int steps, int mute,
            int from) {
    extern __shared__ __align__(128) char smem[];
    auto& sh = *reinterpret_cast<ScanShared<kWarps, true>*>(smem);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, rank = blockIdx.x;
    scan_open(sh);
    if (wid >= kWarps) {
        bool ok = true;
        if (wid > kWarps) {
            const int sends = rank == mute ? from : steps;
            scan_publish<1, true>(sh, sends, kBlocks, rank, lane);
            for (int k = sends; k < steps; ++k) bar_sync(kFormed + (k & 1), blockDim.x);
        } else {
            F2 carry = f2(1.f);
            ok = scan_fold<1, true>(sh, steps, kBlocks, rank, lane, carry);
            if (lane == 0) ok_out[rank] = ok;
            state[rank * 64 + 2 * lane] = carry.lo();
            state[rank * 64 + 2 * lane + 1] = carry.hi();
        }
        scan_close<true>(!ok);
        return;
    }
    auto at = [&](int k) { return ((k * kBlocks + rank) * kWarps + wid) * 64 + 2 * lane; };
    scan_work<1, true, Elements>(
        sh, steps, wid, lane,
        [&](int k, Elements& e) {
            e.a = f2(a[at(k)], a[at(k) + 1]);
            e.b = f2(b[at(k)], b[at(k) + 1]);
            return Run{e.a, e.b};
        },
        [&](int k, const Elements& e, F2 x) {
            const F2 y = run_apply<true>(Run{e.a, e.b}, x);
            o[at(k)] = y.lo();
            o[at(k) + 1] = y.hi();
        });
    scan_close<true>();
}

}  // namespace

// a, b, o: [steps * 4][64]; state: [2][64]; ok_out: [2].  Block `mute` publishes `from` tiles only.
extern "C" int scan_late(const float* a, const float* b, float* o, float* state, int* ok_out,
                         int steps, int mute, int from, void* stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kBlocks);
    cfg.blockDim = dim3(32 * (kWarps + 2));
    cfg.dynamicSmemBytes = sizeof(ScanShared<kWarps, true>);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kBlocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, late_kernel, a, b, o, state, ok_out, steps, mute, from);
}
