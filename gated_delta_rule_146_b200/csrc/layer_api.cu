// layer_api.cu -- the C ABI of the operators around the delta rule: host-side validation and
// dispatch (scan.cu, scan_bwd.cu, conv.cu, norm.cu, norm_seq.cu).
#include <cmath>
#include <initializer_list>

#include "layer.cuh"

using namespace gdr;

namespace {

bool off16(std::initializer_list<const void*> ptrs) {
    uintptr_t bits = 0;
    for (const void* p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
    return (bits & 15u) != 0;
}

bool off4(std::initializer_list<const void*> ptrs) {
    uintptr_t bits = 0;
    for (const void* p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
    return (bits & 3u) != 0;
}

bool any_null(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (!p) return true;
    return false;
}

// An array of a call, for the comparison of places; an absent one has no bytes.
struct Place {
    uintptr_t at;
    unsigned long long bytes;
    Place(const void* p, unsigned long long n)
        : at(reinterpret_cast<uintptr_t>(p)), bytes(p ? n : 0) {}
    bool meets(const Place& o) const {
        return bytes && o.bytes && at < o.at + o.bytes && o.at < at + bytes;
    }
};

// Whether an output shares bytes with an input or with another output.  Kernels read ahead of what
// they write, so that results would depend on their timing.
bool overlap(std::initializer_list<Place> outs, std::initializer_list<Place> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Place& i : ins)
            if (o->meets(i)) return true;
        for (auto other = outs.begin(); other != o; ++other)
            if (o->meets(*other)) return true;
    }
    return false;
}

// The same of a state that may be updated in place, but not over a part of the old one.
bool overlap_in_place(const Place& out, const Place& in) { return out.at != in.at && out.meets(in); }

bool valid_dtype(gdr_dtype d) { return d == GDR_F32 || d == GDR_BF16; }

// Token and channel counts of every operator: kernels hold token numbers (and one tile more) in
// 32 bits, element offsets in 64.
gdr_status check_sizes(long long B, long long T, long long D, long long n_seqs) {
    if (B < 1 || T < 0 || D < 1 || n_seqs < 1) return GDR_ERR_INVALID_ARG;
    if (B * T > 0x7fff0000LL || n_seqs > 0x7fff0000LL) return GDR_ERR_INVALID_ARG;
    if (D > (1 << 20)) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

unsigned long long size_of(gdr_dtype d) { return d == GDR_BF16 ? 2 : 4; }

// Bytes of a call's arrays: the tokens' (in either type), the states', the bounds.
struct ScanBytes {
    unsigned long long x, g, h, cu;
    explicit ScanBytes(const gdr_scan_args& a) {
        const unsigned long long n = (unsigned long long)a.B * a.T * a.D;
        x = n * size_of(a.io_dtype);
        g = n * size_of(a.gate_dtype);
        h = (unsigned long long)a.n_seqs * a.D * sizeof(float);
        cu = (a.n_seqs + 1ull) * sizeof(int32_t);
    }
};
struct ConvBytes {
    unsigned long long x, state, w, bias, cu;
    explicit ConvBytes(const gdr_conv_args& a) {
        x = (unsigned long long)a.B * a.T * a.D * size_of(a.io_dtype);
        state = (unsigned long long)a.n_seqs * (a.width - 1) * a.D * size_of(a.io_dtype);
        bias = (unsigned long long)a.D * sizeof(float);
        w = bias * a.width;
        cu = (a.n_seqs + 1ull) * sizeof(int32_t);
    }
};
struct NormBytes {
    unsigned long long x, w, stats, cu;
    explicit NormBytes(const gdr_norm_args& a) {
        x = (unsigned long long)a.B * a.T * a.H * a.d * size_of(a.io_dtype);
        w = (a.shared_weight ? 1ull : a.H) * a.d * sizeof(float);
        stats = (unsigned long long)a.n_seqs * a.H * 2 * sizeof(float);
        cu = (a.n_seqs + 1ull) * sizeof(int32_t);
    }
};

template <typename A>
gdr_status check_layout(const A* a, const int32_t* cu) {
    if (cu ? a->B != 1 : a->n_seqs != a->B) return GDR_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->status) & 3u) return GDR_ERR_ALIGNMENT;
    return GDR_OK;
}

gdr_status check_scan(const gdr_scan_args* a) {
    if (!a) return GDR_ERR_INVALID_ARG;
    if (const gdr_status st = check_sizes(a->B, a->T, a->D, a->n_seqs); st != GDR_OK) return st;
    if (!valid_dtype(a->io_dtype) || !valid_dtype(a->gate_dtype)) return GDR_ERR_INVALID_ARG;
    if (a->write != GDR_WRITE_PLAIN && a->write != GDR_WRITE_GATE && a->write != GDR_WRITE_TIED)
        return GDR_ERR_INVALID_ARG;
    if (a->reverse & ~1) return GDR_ERR_INVALID_ARG;
    return GDR_OK;
}

gdr_status check_conv(const gdr_conv_args* a) {
    if (!a) return GDR_ERR_INVALID_ARG;
    if (const gdr_status st = check_sizes(a->B, a->T, a->D, a->n_seqs); st != GDR_OK) return st;
    if (!valid_dtype(a->io_dtype) || a->width < 1 || (a->reverse & ~1)) return GDR_ERR_INVALID_ARG;
    if (a->activation != GDR_ACT_NONE && a->activation != GDR_ACT_SILU)
        return a->activation == GDR_ACT_SIGMOID ? GDR_ERR_UNSUPPORTED : GDR_ERR_INVALID_ARG;
    if (a->width < 2 || a->width > 4) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

gdr_status check_norm(const gdr_norm_args* a) {
    if (!a) return GDR_ERR_INVALID_ARG;
    if (a->H < 1 || a->d < 1) return GDR_ERR_INVALID_ARG;
    if (const gdr_status st = check_sizes(a->B, a->T, (long long)a->H * a->d, a->n_seqs); st != GDR_OK)
        return st;
    if (!valid_dtype(a->io_dtype)) return GDR_ERR_INVALID_ARG;
    if ((a->per_sequence | a->center | a->shared_weight) & ~1) return GDR_ERR_INVALID_ARG;
    if (a->activation != GDR_ACT_NONE && a->activation != GDR_ACT_SILU &&
        a->activation != GDR_ACT_SIGMOID)
        return GDR_ERR_INVALID_ARG;
    if (!(std::isfinite(a->eps) && a->eps >= 0.f)) return GDR_ERR_INVALID_ARG;
    // a grid has at most one block per (token, head) and per (sequence, head)
    if (((long long)a->B * a->T + 1) * a->H > 0x7fffffffLL || (long long)a->n_seqs * a->H > 0x7fffffffLL)
        return GDR_ERR_UNSUPPORTED;
    return norm_supported(*a) ? GDR_OK : GDR_ERR_UNSUPPORTED;
}

// A call of no tokens launches none of the kernels that check the bounds on their way.
__global__ void __launch_bounds__(256) check_cu_kernel(Seqs q, int* status) {
    check_cu(q, status, threadIdx.x, 256);
}

template <typename A>
gdr_status check_empty(const A* a, const int32_t* cu, cudaStream_t st) {
    if (!cu || !a->status) return GDR_OK;
    check_cu_kernel<<<1, 256, 0, st>>>(Seqs{cu, a->n_seqs, 0, 0}, a->status);
    return cudaGetLastError() == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

gdr_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return GDR_OK;
    if (!ws || have < need) return GDR_ERR_WORKSPACE;
    return (reinterpret_cast<uintptr_t>(ws) & 255u) ? GDR_ERR_ALIGNMENT : GDR_OK;
}

}  // namespace

extern "C" {

gdr_status gdr_scan_fwd(const gdr_scan_args* a, const void* v, const void* g, const void* beta,
                        const float* h0, const int32_t* cu, void* o, float* h_final,
                        void* stream) {
    gdr_status st = check_scan(a);
    if (st != GDR_OK || (st = check_layout(a, cu)) != GDR_OK) return st;
    const bool tokens = (long long)a->B * a->T > 0, gate = a->write == GDR_WRITE_GATE;
    if (tokens && (any_null({v, g, o}) || gate != (beta != nullptr))) return GDR_ERR_INVALID_ARG;
    if (off16({v, g, beta, h0, cu, o, h_final})) return GDR_ERR_ALIGNMENT;
    ScanPtrs p{};
    p.v = v; p.g = g; p.beta = beta; p.h0 = h0; p.cu = cu; p.o = o; p.h_final = h_final;
    const ScanBytes n(*a);
    // (h_final may be h0)
    if (overlap({{o, n.x}, {h_final, n.h}}, {{v, n.x}, {g, n.g}, {beta, n.g}, {cu, n.cu}}) ||
        overlap({{o, n.x}}, {{h0, n.h}}) || overlap_in_place({h_final, n.h}, {h0, n.h}))
        return GDR_ERR_INVALID_ARG;
    if (!tokens && (st = check_empty(a, cu, static_cast<cudaStream_t>(stream))) != GDR_OK) return st;
    return launch_scan_fwd(*a, p, static_cast<cudaStream_t>(stream));
}

gdr_status gdr_scan_bwd(const gdr_scan_args* a, const void* v, const void* g, const void* beta,
                        const void* o, const void* dO, const float* h0, const int32_t* cu,
                        const float* dh_final, void* dv, void* dg, void* dbeta, float* dh0,
                        void* stream) {
    gdr_status st = check_scan(a);
    if (st != GDR_OK || (st = check_layout(a, cu)) != GDR_OK) return st;
    const bool tokens = (long long)a->B * a->T > 0, gate = a->write == GDR_WRITE_GATE;
    if (tokens && (any_null({g, o, dO, dv, dg}) || gate != (beta != nullptr) ||
                   gate != (dbeta != nullptr) || (a->write != GDR_WRITE_PLAIN && !v)))
        return GDR_ERR_INVALID_ARG;
    if (off16({v, g, beta, o, dO, h0, cu, dh_final, dv, dg, dbeta, dh0})) return GDR_ERR_ALIGNMENT;
    ScanPtrs p{};
    p.v = v; p.g = g; p.beta = beta; p.o_in = o; p.dO = dO; p.h0 = h0; p.cu = cu;
    p.dh_final = dh_final; p.dv = dv; p.dg = dg; p.dbeta = dbeta; p.dh0 = dh0;
    const ScanBytes n(*a);
    // (dh0 may be dh_final)
    if (overlap({{dv, n.x}, {dg, n.g}, {dbeta, n.g}, {dh0, n.h}},
                {{v, n.x}, {g, n.g}, {beta, n.g}, {o, n.x}, {dO, n.x}, {h0, n.h}, {cu, n.cu}}) ||
        overlap({{dv, n.x}, {dg, n.g}, {dbeta, n.g}}, {{dh_final, n.h}}) ||
        overlap_in_place({dh0, n.h}, {dh_final, n.h}))
        return GDR_ERR_INVALID_ARG;
    if (!tokens && (st = check_empty(a, cu, static_cast<cudaStream_t>(stream))) != GDR_OK) return st;
    return launch_scan_bwd(*a, p, static_cast<cudaStream_t>(stream));
}

gdr_status gdr_scan_step(const gdr_scan_args* a, const void* v, const void* g, const void* beta,
                         const float* h, float* h_out, void* o, void* stream) {
    gdr_status st = check_scan(a);
    if (st != GDR_OK || (st = check_layout(a, nullptr)) != GDR_OK) return st;
    if (a->T != 1 || a->reverse) return GDR_ERR_INVALID_ARG;
    const bool gate = a->write == GDR_WRITE_GATE;
    if (any_null({v, g, h, h_out, o}) || gate != (beta != nullptr)) return GDR_ERR_INVALID_ARG;
    if (off16({v, g, beta, h, h_out, o})) return GDR_ERR_ALIGNMENT;
    ScanPtrs p{};
    p.v = v; p.g = g; p.beta = beta; p.h0 = h; p.h_final = h_out; p.o = o;
    const ScanBytes n(*a);
    if (overlap({{o, n.x}, {h_out, n.h}}, {{v, n.x}, {g, n.g}, {beta, n.g}}) ||
        overlap({{o, n.x}}, {{h, n.h}}) || overlap_in_place({h_out, n.h}, {h, n.h}))
        return GDR_ERR_INVALID_ARG;
    return launch_scan_step(*a, p, static_cast<cudaStream_t>(stream));
}

gdr_status gdr_conv_fwd(const gdr_conv_args* a, const void* x, const float* w, const float* bias,
                        const void* state, const int32_t* cu, void* y, void* state_out,
                        void* stream) {
    gdr_status st = check_conv(a);
    if (st != GDR_OK || (st = check_layout(a, cu)) != GDR_OK) return st;
    if ((long long)a->B * a->T > 0 && any_null({x, y})) return GDR_ERR_INVALID_ARG;
    if (!w) return GDR_ERR_INVALID_ARG;
    if (off16({x, state, cu, y, state_out}) || off4({w, bias})) return GDR_ERR_ALIGNMENT;
    ConvPtrs p{};
    p.x = x; p.w = w; p.bias = bias; p.state = state; p.cu = cu; p.y = y; p.state_out = state_out;
    const ConvBytes n(*a);
    if (overlap({{y, n.x}, {state_out, n.state}},
                {{x, n.x}, {w, n.w}, {bias, n.bias}, {state, n.state}, {cu, n.cu}}))
        return GDR_ERR_INVALID_ARG;
    return launch_conv_fwd(*a, p, static_cast<cudaStream_t>(stream));
}

size_t gdr_conv_bwd_workspace_size(const gdr_conv_args* a) {
    return check_conv(a) == GDR_OK ? conv_bwd_workspace(*a) : 0;
}

gdr_status gdr_conv_bwd(const gdr_conv_args* a, const void* x, const float* w, const float* bias,
                        const void* dy, const void* state, const int32_t* cu, void* dx, float* dw,
                        float* dbias, void* dstate, void* workspace, size_t workspace_bytes,
                        void* stream) {
    gdr_status st = check_conv(a);
    if (st != GDR_OK || (st = check_layout(a, cu)) != GDR_OK) return st;
    if ((long long)a->B * a->T > 0 && any_null({x, dy, dx})) return GDR_ERR_INVALID_ARG;
    if (!w || !dw) return GDR_ERR_INVALID_ARG;
    if (off16({x, dy, state, cu, dx, dstate}) || off4({w, bias, dw, dbias})) return GDR_ERR_ALIGNMENT;
    const size_t need = conv_bwd_workspace(*a);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GDR_OK) return st;
    ConvPtrs p{};
    p.x = x; p.w = w; p.bias = bias; p.dy = dy; p.state = state; p.cu = cu; p.dx = dx; p.dw = dw;
    p.dbias = dbias; p.dstate = dstate; p.ws = static_cast<float*>(workspace);
    const ConvBytes n(*a);
    if (overlap({{dx, n.x}, {dw, n.w}, {dbias, n.bias}, {dstate, n.state}, {workspace, need}},
                {{x, n.x}, {w, n.w}, {bias, n.bias}, {dy, n.x}, {state, n.state}, {cu, n.cu}}))
        return GDR_ERR_INVALID_ARG;
    return launch_conv_bwd(*a, p, static_cast<cudaStream_t>(stream));
}

gdr_status gdr_conv_step(const gdr_conv_args* a, const void* x, const float* w, const float* bias,
                         const void* state, void* state_out, void* y, void* stream) {
    gdr_status st = check_conv(a);
    if (st != GDR_OK || (st = check_layout(a, nullptr)) != GDR_OK) return st;
    if (a->T != 1 || a->reverse) return GDR_ERR_INVALID_ARG;
    if (any_null({x, w, state, state_out, y})) return GDR_ERR_INVALID_ARG;
    if (off16({x, state, state_out, y}) || off4({w, bias})) return GDR_ERR_ALIGNMENT;
    ConvPtrs p{};
    p.x = x; p.w = w; p.bias = bias; p.state = state; p.y = y; p.state_out = state_out;
    const ConvBytes n(*a);
    if (overlap({{y, n.x}, {state_out, n.state}}, {{x, n.x}, {w, n.w}, {bias, n.bias}}) ||
        overlap({{y, n.x}}, {{state, n.state}}) ||
        overlap_in_place({state_out, n.state}, {state, n.state}))
        return GDR_ERR_INVALID_ARG;
    return launch_conv_step(*a, p, static_cast<cudaStream_t>(stream));
}

size_t gdr_norm_fwd_workspace_size(const gdr_norm_args* a) {
    return check_norm(a) == GDR_OK ? norm_fwd_workspace(*a) : 0;
}

gdr_status gdr_norm_fwd(const gdr_norm_args* a, const void* x, const float* w, const float* bias,
                        const void* z, const int32_t* cu, void* y, float* stats, void* workspace,
                        size_t workspace_bytes, void* stream) {
    gdr_status st = check_norm(a);
    if (st != GDR_OK || (st = check_layout(a, cu)) != GDR_OK) return st;
    const bool tokens = (long long)a->B * a->T > 0;
    if (tokens && any_null({x, y})) return GDR_ERR_INVALID_ARG;
    if (stats && !a->per_sequence) return GDR_ERR_INVALID_ARG;
    if (off16({x, z, cu, y, stats}) || off4({w, bias})) return GDR_ERR_ALIGNMENT;
    const size_t need = norm_fwd_workspace(*a);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GDR_OK) return st;
    NormPtrs p{};
    p.x = x; p.w = w; p.b = bias; p.z = z; p.cu = cu; p.y = y; p.stats = stats;
    p.ws = static_cast<float*>(workspace);
    const NormBytes n(*a);
    if (overlap({{y, n.x}, {stats, n.stats}, {workspace, need}},
                {{x, n.x}, {w, n.w}, {bias, n.w}, {z, n.x}, {a->per_sequence ? cu : nullptr, n.cu}}))
        return GDR_ERR_INVALID_ARG;
    if (!tokens && a->per_sequence &&
        (st = check_empty(a, cu, static_cast<cudaStream_t>(stream))) != GDR_OK)
        return st;
    return launch_norm_fwd(*a, p, static_cast<cudaStream_t>(stream));
}

size_t gdr_norm_bwd_workspace_size(const gdr_norm_args* a) {
    return check_norm(a) == GDR_OK ? norm_bwd_workspace(*a) : 0;
}

gdr_status gdr_norm_bwd(const gdr_norm_args* a, const void* x, const float* w, const float* bias,
                        const void* z, const void* dy, const int32_t* cu, const float* stats,
                        void* dx, float* dw, float* dbias, void* dz, void* workspace,
                        size_t workspace_bytes, void* stream) {
    gdr_status st = check_norm(a);
    if (st != GDR_OK || (st = check_layout(a, cu)) != GDR_OK) return st;
    const bool tokens = (long long)a->B * a->T > 0;
    if (tokens && any_null({x, dy, dx})) return GDR_ERR_INVALID_ARG;
    if (tokens && (z != nullptr) != (dz != nullptr)) return GDR_ERR_INVALID_ARG;
    if (a->per_sequence && !stats) return GDR_ERR_INVALID_ARG;
    if (off16({x, z, dy, cu, stats, dx, dz}) || off4({w, bias, dw, dbias})) return GDR_ERR_ALIGNMENT;
    const size_t need = norm_bwd_workspace(*a);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GDR_OK) return st;
    NormPtrs p{};
    p.x = x; p.w = w; p.b = bias; p.z = z; p.dy = dy; p.cu = cu; p.stats_in = stats; p.dx = dx;
    p.dw = dw; p.db = dbias; p.dz = dz; p.ws = static_cast<float*>(workspace);
    const NormBytes n(*a);
    if (overlap({{dx, n.x}, {dw, n.w}, {dbias, n.w}, {dz, n.x}, {workspace, need}},
                {{x, n.x}, {w, n.w}, {bias, n.w}, {z, n.x}, {dy, n.x},
                 {a->per_sequence ? stats : nullptr, n.stats},
                 {a->per_sequence ? cu : nullptr, n.cu}}))
        return GDR_ERR_INVALID_ARG;
    if (!tokens && a->per_sequence &&
        (st = check_empty(a, cu, static_cast<cudaStream_t>(stream))) != GDR_OK)
        return st;
    return launch_norm_bwd(*a, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
