// scan.cu -- gated linear recurrence: forward over whole sequences, and one token.
//
//     h_t = alpha_t h_{t-1} + b_t,   alpha = exp(g),   b = v | beta v | (1 - alpha) v,   o = h
//
// Every element is read and written once (6 bytes per token and channel in bf16, 8 with beta),
// for five operations: HBM bounds it.  The split is described in scan_impl.cuh.
#include "scan_impl.cuh"

namespace gdr {

namespace {

constexpr int kStages = 3;

// Tokens of a warp's run: eight in bf16, four where fp32 doubles the bytes of a tile.
template <typename IO, typename GT>
constexpr int seg_of = sizeof(IO) + sizeof(GT) > 4 ? 4 : 8;

template <typename IO, typename GT>
struct FwdParams {
    const IO* v; const GT* g; const GT* beta;
    const float* h0;
    IO* o;
    float* h_final;
    int* status;
    Seqs q;
    int D, L, slabs, reverse;  // L: tokens of a row
};

// alpha and b of one element
template <int kWrite>
__device__ __forceinline__ void decay_write(float g, float v, float beta, float& a, float& b) {
    if constexpr (kWrite == GDR_WRITE_TIED) {
        const float em = expm1f(g);  // 1 - alpha without cancellation
        a = 1.f + em;
        b = -em * v;
    } else {
        a = expf(g);
        b = kWrite == GDR_WRITE_GATE ? beta * v : v;
    }
}

template <typename IO, typename GT, int kWrite>
constexpr int stage_bytes = Rows<IO, seg_of<IO, GT>>::kBytes +
                            (kWrite == GDR_WRITE_GATE ? 2 : 1) * Rows<GT, seg_of<IO, GT>>::kBytes;

// One tile's elements of a lane, from the forming of its run to the output.
template <int kSeg>
struct Elements {
    float a[kSeg][2], b[kSeg][2];
    Run before;  // the block's runs before the warp's
    Marks m;
};

// kSeqs: one row holds all sequences, whose starts reset the state; else a row is a sequence.
template <typename IO, typename GT, int kWrite, Copy kCopy, bool kSeqs>
__global__ void __launch_bounds__(kScanThreads, 2)
scan_fwd_kernel(const FwdParams<IO, GT> p, const int cluster) {
    extern __shared__ __align__(128) char stages[];
    __shared__ ScanShared sh;
    constexpr int kSeg = seg_of<IO, GT>, kTile = kScanWarps * kSeg;
    constexpr int kStage = stage_bytes<IO, GT, kWrite>;
    using RowsIO = Rows<IO, kSeg>;
    using RowsGT = Rows<GT, kSeg>;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = blockIdx.x % cluster;
    const int unit = blockIdx.x / cluster;
    const int slab = unit % p.slabs, row = unit / p.slabs;
    const int left = p.D - slab * kSlab;       // channels of the slab
    const int c = slab * kSlab + 2 * lane, mine = left - 2 * lane;
    const int L = p.L, D = p.D;
    const int origin = p.reverse ? L - 1 : 0, dir = p.reverse ? -1 : 1;

    if (kSeqs && blockIdx.x == 0) check_cu(p.q, p.status, tid, kScanThreads);
    if (kSeqs && rank == 0 && p.h_final) {  // empty sequences keep their state
        for (int s = wid; s < p.q.n; s += kScanWarps) {
            if (p.q.begin(s) != p.q.end(s)) continue;
            float x[2] = {};
            if (p.h0) load_state<kCopy>(p.h0 + (size_t)s * D + c, x, mine);
            store_pair<float, kCopy>(p.h_final + (size_t)s * D + c, x, mine);
        }
    }

    const size_t base = (size_t)row * L * D + slab * kSlab;
    char* const buf = stages + wid * kStages * kStage;
    auto feed = [&](int first, int stage) {
        char* s = buf + stage * kStage;
        feed_rows<IO, kCopy, kSeg>(s, p.v + base, origin, dir, first, L, D, left, lane);
        s += RowsIO::kBytes;
        feed_rows<GT, kCopy, kSeg>(s, p.g + base, origin, dir, first, L, D, left, lane);
        if constexpr (kWrite == GDR_WRITE_GATE)
            feed_rows<GT, kCopy, kSeg>(s + RowsGT::kBytes, p.beta + base, origin, dir, first, L, D, left,
                                 lane);
    };

    const int stride = cluster * kTile;
    const int steps = (int)(((long long)L + stride - 1) / stride);
    const int first0 = rank * kTile + wid * kSeg;
    // places behind L may pass 2^31: a tile that starts there is empty
    auto place = [&](int k) {
        const long long f = first0 + (long long)k * stride;
        return (int)(f < L ? f : L);
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) {
        feed(place(k), k);
        copy_commit();
    }

    Here here{0, 0};
    int stage = 0;  // of the next tile to be formed
    // Forms the run of tile k and hands it to the block.
    auto form = [&](int k, Elements<kSeg>& e) {
        copy_wait<kStages - 2>();
        __syncwarp();
        // the stage of the tile before: every lane has read it
        feed(place(k + kStages - 1), stage == 0 ? kStages - 1 : stage - 1);
        copy_commit();
        const char* s = buf + stage * kStage;
        stage = stage == kStages - 1 ? 0 : stage + 1;
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            float v[2], g[2], w[2] = {};
            RowsIO::read(s, i, lane, v);
            RowsGT::read(s + RowsIO::kBytes, i, lane, g);
            if constexpr (kWrite == GDR_WRITE_GATE)
                RowsGT::read(s + RowsIO::kBytes + RowsGT::kBytes, i, lane, w);
#pragma unroll
            for (int j = 0; j < 2; ++j) decay_write<kWrite>(g[j], v[j], w[j], e.a[i][j], e.b[i][j]);
        }
        if constexpr (kSeqs) {
            const int first = place(k);
            e.m = find_marks(p.q, here, origin, dir, first, min(kSeg, L - first), lane);
            if (e.m.start && p.h0) {  // b at a start takes the initial state in
#pragma unroll
                for (int i = 0; i < kSeg; ++i) {
                    if (!(e.m.start >> i & 1u)) continue;
                    const int q = __shfl_sync(0xffffffffu, e.m.seq, i);
                    float x[2];
                    load_state<kCopy>(p.h0 + (size_t)q * D + c, x, mine);
#pragma unroll
                    for (int j = 0; j < 2; ++j) e.b[i][j] = fmaf(e.a[i][j], x[j], e.b[i][j]);
                }
            }
        }
        Run run;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float A = e.a[0][j], H = e.b[0][j];
#pragma unroll
            for (int i = 1; i < kSeg; ++i) {
                const float y = fmaf(e.a[i][j], H, e.b[i][j]);
                H = kSeqs && (e.m.start >> i & 1u) ? e.b[i][j] : y;
                A *= e.a[i][j];
            }
            run.A[j] = kSeqs && e.m.start ? kReset : A;
            run.H[j] = H;
        }
        sh.warp[k & 1][wid][lane] = run;
    };

    float carry[2] = {};
    if (!kSeqs && p.h0) load_state<kCopy>(p.h0 + (size_t)row * D + c, carry, mine);

    auto cl = cooperative_groups::this_cluster();
    Run whole;   // the block's tile, where the cluster is the block
    // Joins the block's runs of tile k and, in a cluster, hands the result to every block.
    auto publish = [&](int k, Elements<kSeg>& e) {
        join_block<kSeqs>(sh.warp[k & 1], wid, lane, e.before, whole);
        if (cluster > 1) {
            if (wid < cluster) *cl.map_shared_rank(&sh.block[k & 3][rank][lane], wid) = whole;
            cl.barrier_arrive();
        }
    };
    // Finishes tile k: its states from the carry, which becomes the state behind the step.
    auto finish = [&](int k, const Elements<kSeg>& e, const Run& tile) {
        float h[2];
        if (cluster == 1) {
            h[0] = carry[0];
            h[1] = carry[1];
            run_apply<kSeqs>(tile, carry);
        } else {
            for (int r = 0; r < cluster; ++r) {
                if (r == rank) { h[0] = carry[0]; h[1] = carry[1]; }
                run_apply<kSeqs>(sh.block[k & 3][r][lane], carry);
            }
        }
        run_apply<kSeqs>(e.before, h);
        const int first = place(k), n = min(kSeg, L - first);
        IO* out = p.o + base + (long long)(origin + dir * first) * D + 2 * lane;
        const long long next = (long long)dir * D;
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float y = fmaf(e.a[i][j], h[j], e.b[i][j]);
                h[j] = kSeqs && (e.m.start >> i & 1u) ? e.b[i][j] : y;
            }
            if (i < n) store_pair<IO, kCopy>(out, h, mine);
            out += next;
            if (kSeqs && (e.m.end >> i & 1u) && p.h_final) {
                const int q = __shfl_sync(0xffffffffu, e.m.seq, i);
                store_pair<float, kCopy>(p.h_final + (size_t)q * D + c, h, mine);
            }
        }
    };

    // One step of the walk: tile k + 1's run goes out before tile k is finished.  The block
    // barrier between form and publish also keeps the parities apart: a run is written again two
    // tiles later, behind a barrier that every reader of the first has passed.
    auto turn = [&](int k, Elements<kSeg>& now, Elements<kSeg>& next) {
        const Run tile = whole;
        if (k + 1 < steps) {
            form(k + 1, next);
            __syncthreads();
        }
        if (cluster > 1) cl.barrier_wait();
        if (k + 1 < steps) publish(k + 1, next);
        finish(k, now, tile);
    };
    Elements<kSeg> even, odd;
    form(0, even);
    __syncthreads();
    publish(0, even);
    for (int k = 0; k < steps; k += 2) {
        turn(k, even, odd);
        if (k + 1 < steps) turn(k + 1, odd, even);
    }
    copy_wait<0>();
    if (!kSeqs && p.h_final && rank == 0 && wid == 0)
        store_pair<float, kCopy>(p.h_final + (size_t)row * D + c, carry, mine);
}

template <typename IO, typename GT, int kWrite, Copy kCopy>
gdr_status fwd_launch(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    const bool seqs = scan_one_row(a, x.cu);
    FwdParams<IO, GT> p;
    p.v = static_cast<const IO*>(x.v);
    p.g = static_cast<const GT*>(x.g);
    p.beta = static_cast<const GT*>(x.beta);
    p.h0 = x.h0;
    p.o = static_cast<IO*>(x.o);
    p.h_final = x.h_final;
    p.status = a.status;
    p.q = Seqs{x.cu, a.n_seqs, a.T, a.B * a.T};
    p.D = a.D;
    p.L = seqs ? a.B * a.T : a.T;
    p.slabs = (a.D + kSlab - 1) / kSlab;
    p.reverse = a.reverse;
    const long long units = (long long)p.slabs * (seqs ? 1 : a.B);
    const int tile = kScanWarps * seg_of<IO, GT>;
    const size_t smem = (size_t)kScanWarps * kStages * stage_bytes<IO, GT, kWrite>;
    return seqs ? scan_launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, true>, p, units, p.L, tile, smem, st)
                : scan_launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, false>, p, units, p.L, tile, smem, st);
}

struct Fwd {
    template <typename IO, typename GT, int kWrite>
    static gdr_status go(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
        const Copy copy = scan_copy(a);
        if (copy == kCopy16) return fwd_launch<IO, GT, kWrite, kCopy16>(a, x, st);
        if constexpr (sizeof(IO) == sizeof(GT)) {
            if (copy == kCopyPair) return fwd_launch<IO, GT, kWrite, kCopyPair>(a, x, st);
        }
        return fwd_launch<IO, GT, kWrite, kCopyOne>(a, x, st);
    }
};

// ---- one token ------------------------------------------------------------------------------
// Streams the fp32 state once: 14 bytes per channel in bf16 (16 with beta).
template <typename IO, typename GT, int kWrite, int VEC>
__global__ void __launch_bounds__(256)
scan_step_kernel(const IO* __restrict__ v, const GT* __restrict__ g, const GT* __restrict__ beta,
                 const float* h, float* h_out, IO* __restrict__ o, long long n) {
    const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * VEC;
    if (at >= n) return;
    float fh[VEC], fv[VEC], fg[VEC], fb[VEC] = {};
    load_f<float, VEC>(h + at, fh);
    load_f<IO, VEC>(v + at, fv);
    load_f<GT, VEC>(g + at, fg);
    if constexpr (kWrite == GDR_WRITE_GATE) load_f<GT, VEC>(beta + at, fb);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float a, b;
        decay_write<kWrite>(fg[j], fv[j], fb[j], a, b);
        fh[j] = fmaf(a, fh[j], b);
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

int scan_cluster(long long units, long long tiles) {
    int c = 1;
    while (c < kScanMaxCluster && units * c < 2 * 148 && tiles >= 2 * c) c *= 2;
    return c;
}

gdr_status launch_scan_fwd(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    if (a.B * (long long)a.T == 0) {  // every state stays
        const size_t bytes = sizeof(float) * (size_t)a.n_seqs * a.D;
        if (!x.h_final || x.h_final == x.h0) return GDR_OK;
        const cudaError_t e = x.h0 ? cudaMemcpyAsync(x.h_final, x.h0, bytes,
                                                     cudaMemcpyDeviceToDevice, st)
                                   : cudaMemsetAsync(x.h_final, 0, bytes, st);
        return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
    }
    return scan_dispatch<Fwd>(a, x, st);
}

gdr_status launch_scan_step(const gdr_scan_args& a, const ScanPtrs& x, cudaStream_t st) {
    return scan_dispatch<Step>(a, x, st);
}

}  // namespace gdr
