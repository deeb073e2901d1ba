// scan.cu -- gated linear recurrence: forward over whole sequences, and one token.
//
//     h_t = alpha_t h_{t-1} + b_t,   alpha = exp(g),   b = v | beta v | (1 - alpha) v,   o = h
//
// Every element is read and written once (6 bytes per token and channel in bf16, 8 with beta),
// for five operations: HBM bounds it.  The split is described in scan_impl.cuh.
#include "scan_impl.cuh"

namespace gdr {

namespace {

// Two tiles ahead.  More bytes in flight cost: with three tiles ahead the training shape takes 97
// instead of 86 us (beta given), with one 95.
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

template <typename IO, typename GT, int kWrite>
constexpr int stage_bytes = Rows<IO, seg_of<IO, GT>>::kBytes +
                            (kWrite == GDR_WRITE_GATE ? 2 : 1) * Rows<GT, seg_of<IO, GT>>::kBytes;

// A lane's elements of a tile, from the forming of its run to the output.
template <int kSeg>
struct Elements {
    F2 a[kSeg], b[kSeg];
    Marks m;
};

// kSeqs: one row holds all sequences, whose starts reset the state; else a row is a sequence.
template <typename IO, typename GT, int kWrite, Copy kCopy, bool kSeqs, bool kCluster,
          int kWarps>
__global__ void __launch_bounds__(32 * (kWarps + 2 * kCluster), kCluster ? 1 : 2)
scan_fwd_kernel(const FwdParams<IO, GT> p, const int cluster) {
    extern __shared__ __align__(128) char smem[];
    using Shared = ScanShared<kWarps, kCluster>;
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    char* const stages = smem + sizeof(sh) + (kSeqs ? kCuBytes : 0);
    constexpr int kSeg = seg_of<IO, GT>, kTile = kWarps * kSeg;
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

    F2 carry = f2(0.f);  // the folder's; read before any block can write h_final
    if (!kSeqs && (!kCluster || wid == kWarps) && p.h0) carry = load_state<kCopy>(p.h0 + (size_t)row * D + c, mine);
    Seqs seqs = p.q;
    if constexpr (kSeqs) seqs = share_cu(p.q, reinterpret_cast<int32_t*>(smem + sizeof(sh)));
    scan_open<kCluster>(sh.full);
    if (kSeqs && blockIdx.x == 0) check_cu(p.q, p.status, tid, 32 * (kWarps + 2 * kCluster));
    if (kSeqs && rank == 0 && p.h_final) {  // empty sequences keep their state
        for (int s = wid; s < seqs.n; s += kWarps + 2 * kCluster) {
            if (seqs.begin(s) != seqs.end(s)) continue;
            F2 x = f2(0.f);
            if (p.h0) x = load_state<kCopy>(p.h0 + (size_t)s * D + c, mine);
            store_pair<float, kCopy>(p.h_final + (size_t)s * D + c, x, mine);
        }
    }

    const size_t base = (size_t)row * L * D + slab * kSlab;
    const int stride = cluster * kTile, first0 = rank * kTile + wid * kSeg;
    const int steps = (int)(((long long)L + stride - 1) / stride);
    const long long hop = (long long)dir * stride * D;  // elements from a tile to the next
    char* const buf = stages + wid * kStages * kStage;
    Feed<IO, kCopy, kSeg> fv;
    Feed<GT, kCopy, kSeg> fg, fb;
    fv.open(p.v + base, origin, dir, first0, D, left, lane);
    fg.open(p.g + base, origin, dir, first0, D, left, lane);
    if constexpr (kWrite == GDR_WRITE_GATE) fb.open(p.beta + base, origin, dir, first0, D, left, lane);
    // The tiles walk on past L by at most kStages steps: L is bounded so that no place overflows.
    auto feed = [&](int k, int stage) {
        char* s = buf + stage * kStage;
        const int place = k < steps ? first0 + k * stride : L;
        fv.tile(s, place, L, hop);
        fg.tile(s + RowsIO::kBytes, place, L, hop);
        if constexpr (kWrite == GDR_WRITE_GATE)
            fb.tile(s + RowsIO::kBytes + RowsGT::kBytes, place, L, hop);
        copy_commit();
    };
    if constexpr (kCluster) if (wid >= kWarps) {
        if (wid > kWarps) {
            scan_publish<kSeqs>(sh, steps, cluster, rank, lane);
        } else {
            const bool ok = scan_fold<kSeqs>(sh, steps, cluster, rank, lane, carry);
            if (!ok && p.status && lane == 0) atomicCAS(p.status, (int)GDR_OK, (int)GDR_ERR_TIMEOUT);
            if (!kSeqs && p.h_final && rank == 0)
                store_pair<float, kCopy>(p.h_final + (size_t)row * D + c, carry, mine);
        }
        scan_close<kCluster>();
        return;
    }
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) feed(k, k);

    Here here{0, 0};
    int stage = 0;  // of the next tile to be formed
    auto form = [&](int k, Elements<kSeg>& e) -> Run {
        copy_wait<kStages - 2>();
        __syncwarp();
        // into the stage of the tile before: every lane has read it
        feed(k + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        const char* s = buf + stage * kStage;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if constexpr (kSeqs) {
            const int first = first0 + k * stride;
            e.m = find_marks(seqs, here, origin, dir, first, min(kSeg, L - first), lane);
        }
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            const F2 v = RowsIO::read(s, i, lane), g = RowsGT::read(s + RowsIO::kBytes, i, lane);
            e.a[i] = exp2ch(g);
            if constexpr (kWrite == GDR_WRITE_GATE)
                e.b[i] = mul2(RowsGT::read(s + RowsIO::kBytes + RowsGT::kBytes, i, lane), v);
            else if constexpr (kWrite == GDR_WRITE_TIED)
                e.b[i] = mul2(one_minus(g, e.a[i]), v);
            else
                e.b[i] = v;
        }
        if (kSeqs && e.m.start && p.h0) {  // b at a start takes the initial state in
#pragma unroll
            for (int i = 0; i < kSeg; ++i) {
                if (!(e.m.start >> i & 1u)) continue;
                const int q = __shfl_sync(0xffffffffu, e.m.seq, i);
                e.b[i] = fma2(e.a[i], load_state<kCopy>(p.h0 + (size_t)q * D + c, mine), e.b[i]);
            }
        }
        Run run{e.a[0], e.b[0]};
        if (!kSeqs || !e.m.start) {
#pragma unroll
            for (int i = 1; i < kSeg; ++i) {
                run.H = fma2(e.a[i], run.H, e.b[i]);
                run.A = mul2(run.A, e.a[i]);
            }
        } else {
#pragma unroll
            for (int i = 1; i < kSeg; ++i)
                run.H = pick2(e.m.start >> i & 1u, e.b[i], fma2(e.a[i], run.H, e.b[i]));
            run.A = f2(kReset);
        }
        return run;
    };

    const long long next = (long long)dir * D;
    IO* out = p.o + base + (origin + (long long)dir * first0) * D + 2 * lane;
    auto finish = [&](int k, const Elements<kSeg>& e, F2 h) {
        const int n = L - (first0 + k * stride);
        IO* q = out;
        out += hop;
        if (n >= kSeg && !(kSeqs && e.m.any())) {
#pragma unroll
            for (int i = 0; i < kSeg; ++i, q += next) {
                h = fma2(e.a[i], h, e.b[i]);
                store_pair<IO, kCopy>(q, h, mine);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kSeg; ++i, q += next) {
            const F2 y = fma2(e.a[i], h, e.b[i]);
            h = kSeqs ? pick2(e.m.start >> i & 1u, e.b[i], y) : y;
            if (i < n) store_pair<IO, kCopy>(q, h, mine);
            if (kSeqs && (e.m.end >> i & 1u) && p.h_final) {
                const int s = __shfl_sync(0xffffffffu, e.m.seq, i);
                store_pair<float, kCopy>(p.h_final + (size_t)s * D + c, h, mine);
            }
        }
    };
    if constexpr (kCluster) {
        scan_work<Elements<kSeg>>(sh, steps, wid, lane, form, finish);
    } else {
        scan_walk<kSeqs, Elements<kSeg>>(sh, steps, wid, lane, carry, form, finish);
        if (!kSeqs && p.h_final && wid == 0)
            store_pair<float, kCopy>(p.h_final + (size_t)row * D + c, carry, mine);
    }
    copy_wait<0>();
    scan_close<kCluster>();
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
    const int cluster = kCopy == kCopyOne ? 0 : scan_cluster(units);
    constexpr int kWide = 16;
    auto launch = [&](auto kernel, int warps, int threads, size_t shared) {
        const size_t smem = (size_t)warps * kStages * stage_bytes<IO, GT, kWrite> + shared +
                            (seqs ? kCuBytes : 0);
        return scan_launch(kernel, p, units, cluster ? cluster : 1, threads, smem, st);
    };
    if constexpr (kCopy != kCopyOne) {
        if (cluster) {
            constexpr int kThreads = 32 * (kWide + 2);
            constexpr size_t kShared = sizeof(ScanShared<kWide, true>);
            return seqs ? launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, true, true, kWide>, kWide, kThreads, kShared)
                        : launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, false, true, kWide>, kWide, kThreads, kShared);
        }
    }
    return seqs ? launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, true, false, 8>, 8, 256, sizeof(ScanShared<8, false>))
                : launch(scan_fwd_kernel<IO, GT, kWrite, kCopy, false, false, 8>, 8, 256, sizeof(ScanShared<8, false>));
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
        const F2 g2 = f2(fg[j]), a = exp2ch(g2);
        float b = fv[j];
        if constexpr (kWrite == GDR_WRITE_GATE) b *= fb[j];
        if constexpr (kWrite == GDR_WRITE_TIED) b *= one_minus(g2, a).lo();
        fh[j] = fmaf(a.lo(), fh[j], b);
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
