// Linear attention: the launches around its chunk kernel (linear_attn_kernel.h),
// the join of a cut sequence's segments, the sums the backward pass takes over
// workgroups, and the single-token step.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "internal.h"

namespace mamba {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;

// A state's decay over n steps of log decay g, as keep s + change s: a slow one
// by its difference from 1, which rounds only the change, a fast one as a
// factor, whose difference from 1 would round at the state's size. An infinity
// stays one (inf - inf and 0 inf would be NaN) unless the decay is zero.
struct Decay {
    float keep, change;
    bool zero;

    __device__ __forceinline__ Decay(float g, int64_t n) : keep(1.0f), change(0.0f), zero(false) {
        if (g == 0.0f || n == 0) return;
        // the exponent's rounding, put back as a factor 1 + e
        const float steps = static_cast<float>(n);
        const float p = g * steps;
        const float e = fmaf(g, steps, -p) + g * static_cast<float>(n - static_cast<int64_t>(steps));
        if (p > -0.6931472f) {
            change = expm1f(p);
            change = fmaf(e, 1.0f + change, change);
        } else {
            const float x = expf(p);   // 0 for g = -inf, where e is none
            keep = 0.0f;
            change = x > 0.0f ? fmaf(x, e, x) : x;
            zero = p == -__builtin_inff();
        }
    }
    __device__ __forceinline__ float of(float s) const {
        return fabsf(s) == __builtin_inff() && !zero ? s : fmaf(s, change, keep * s);
    }
};

// Join of the segments, in place: on entry seg[(b, h), s] holds what segment
// s adds to the state it is entered with, on exit the state entering it.
// Direction 0 walks the segments up from h0, direction 1 down from dhL. Each
// share is read once and replaced once, 8 loads out together: 16 heads of 128 x
// 128, 16 segments, 10 us of which the 33 MB are 6 at a large copy's rate.
struct JoinArgs {
    int64_t batch, seqlen, seg_len, state_elems;
    int heads, nseg;
    const int32_t* lengths;
    const float* log_decay;
    float* seg[2];
    const float* init[2];
};

__global__ __launch_bounds__(256) void linear_attn_join_kernel(JoinArgs a) {
    const int64_t quads = a.state_elems / 4;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= quads) return;
    const int64_t bh = blockIdx.y;
    const int dir = blockIdx.z;
    const int64_t b = bh / a.heads;
    const float g = a.log_decay[bh - b * a.heads];
    int64_t len = a.seqlen;
    if (a.lengths != nullptr) {
        const int64_t n = a.lengths[b];
        len = n < 0 ? 0 : (n < len ? n : len);
    }
    f32x4* seg = reinterpret_cast<f32x4*>(a.seg[dir] + bh * a.nseg * a.state_elems) + e;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.init[dir] != nullptr)
        s = reinterpret_cast<const f32x4*>(a.init[dir] + bh * a.state_elems)[e];
    const Decay full(g, a.seg_len);
    constexpr int U = 8;   // loads in flight
    for (int k0 = 0; k0 < a.nseg; k0 += U) {
        f32x4 add[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;   // the last of the walk adds to nobody's entry
            add[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (k < a.nseg - 1) add[u] = seg[(dir ? a.nseg - 1 - k : k) * quads];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;
            if (k >= a.nseg) break;
            const int64_t sg = dir ? a.nseg - 1 - k : k;
            seg[sg * quads] = s;
            int64_t n = len - sg * a.seg_len;
            n = n < 0 ? 0 : (n < a.seg_len ? n : a.seg_len);
            const Decay decay = n == a.seg_len ? full : Decay(g, n);
#pragma unroll
            for (int v = 0; v < 4; ++v) s[v] = decay.of(s[v]) + add[u][v];
        }
    }
}

// The decay's gradient: each head's terms in a fixed order, in 64 bits, one
// workgroup of 256 per head.
struct DecaySumArgs {
    int64_t terms;        // of a head
    int heads;
    const double* dg;     // (heads, terms)
    float* out;           // (heads) or nullptr: not wanted
};

__device__ __forceinline__ void decay_sum(const DecaySumArgs& a, int head, double (&red)[4]) {
    const double* p = a.dg + head * a.terms;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < a.terms; i += 256) s += p[i];
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) s += __shfl_xor(s, m);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = s;
    __syncthreads();
    if (threadIdx.x == 0) a.out[head] = static_cast<float>(((red[0] + red[1]) + red[2]) + red[3]);
}

__global__ __launch_bounds__(256) void linear_attn_decay_kernel(DecaySumArgs a) {
    __shared__ double red[4];
    decay_sum(a, static_cast<int>(blockIdx.x), red);
}

// Gradients of keys and values that several heads share: the sum of the
// heads' fp32 gradients (batch, seqlen, heads, dim), rounded once. Added in a
// fixed order, not by atomics. Bound by memory (4 us at 2 x 333 x 6 heads). The
// first workgroups, one per head, sum the decay's gradient, which saves a launch.
struct ShareArgs {
    int64_t rows;           // (batch, seqlen, kv_heads)
    int rep;                // heads per head of keys and values
    int dim[2];
    const float* part[2];
    void* out[2];
    DecaySumArgs decay;
};

template <int IO>
__global__ __launch_bounds__(256) void linear_attn_share_kernel(ShareArgs a) {
    const int which = blockIdx.y;
    const int heads = a.decay.out != nullptr ? a.decay.heads : 0;
    if (static_cast<int>(blockIdx.x) < heads) {
        __shared__ double red[4];
        if (which == 0) decay_sum(a.decay, static_cast<int>(blockIdx.x), red);
        return;
    }
    const int64_t quads = a.dim[which] / 4, count = a.rows * quads;
    const int64_t stride = static_cast<int64_t>(gridDim.x - heads) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x - heads) * 256 + threadIdx.x; i < count; i += stride) {
        const int64_t row = i / quads, q = i - row * quads;
        const f32x4* p = reinterpret_cast<const f32x4*>(a.part[which]) + row * a.rep * quads + q;
        f32x4 s = p[0];
        for (int r = 1; r < a.rep; ++r) s += p[r * quads];
#pragma unroll
        for (int v = 0; v < 4; ++v) store_io<IO>(a.out[which], 4 * i + v, s[v]);
    }
}

// One token: S <- lam S + k^T v in place, o = scale q S. Bound by the state,
// read and written once (256 x 16 heads of 128 x 128: 104 us, 5.2 TB/s where a
// large copy reaches 5.5). A workgroup takes 64 of a head's columns: 16 lanes
// hold 4 columns each of a row, its 16 groups of them rows n = group + 16 u,
// so every lane has all its loads (DK / 16 of 16 bytes) in flight together.
template <int IO, int DK>
__global__ __launch_bounds__(kLinUpdateThreads) void linear_attn_update_kernel(LinUpdateArgs a, int slabs) {
    constexpr int NR = DK / 16;
    __shared__ float qs[DK], ks[DK];
    __shared__ f32x4 red[4][16];
    const int tid = threadIdx.x;
    const int64_t bh = blockIdx.x / slabs;
    const int slab = static_cast<int>(blockIdx.x - bh * slabs);
    const int64_t b = bh / a.heads;
    const int hd = static_cast<int>(bh - b * a.heads);
    const int hk = hd / (a.heads / a.kv_heads);
    const int lane = tid & 15, grp = tid >> 4;
    const int p = 64 * slab + 4 * lane;
    const bool in = p < a.dv;
    float* h = a.h + bh * a.dk * a.dv + p;
    f32x4 s[NR];
#pragma unroll
    for (int u = 0; u < NR; ++u) {
        const int n = grp + 16 * u;
        s[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (in && n < a.dk) s[u] = *reinterpret_cast<const f32x4*>(h + static_cast<int64_t>(n) * a.dv);
    }
    const int64_t kv = b * a.kv_heads + hk;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = raw_to_f32<IO>(load_raw<IO>(a.v, kv * a.dv + p + e));
    }
    for (int n = tid; n < DK; n += kLinUpdateThreads) {
        const bool have = n < a.dk;
        qs[n] = have ? raw_to_f32<IO>(load_raw<IO>(a.q, bh * a.dk + n)) : 0.0f;
        ks[n] = have ? raw_to_f32<IO>(load_raw<IO>(a.k, kv * a.dk + n)) : 0.0f;
    }
    const Decay decay(a.log_decay[hd], 1);
    __syncthreads();
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < NR; ++u) {
        const int n = grp + 16 * u;
        const float kn = ks[n], qn = qs[n];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[u][e] = fmaf(kn, v[e], decay.of(s[u][e]));
            o[e] = fmaf(qn, s[u][e], o[e]);
        }
        if (in && n < a.dk) *reinterpret_cast<f32x4*>(h + static_cast<int64_t>(n) * a.dv) = s[u];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o[e] += __shfl_xor(o[e], 16);
        o[e] += __shfl_xor(o[e], 32);
    }
    if ((tid & 63) < 16) red[tid / kWave][lane] = o;
    __syncthreads();
    if (tid < 16 && in) {
        const f32x4 t = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
#pragma unroll
        for (int e = 0; e < 4; ++e) store_io<IO>(a.o, bh * a.dv + p + e, a.scale * t[e]);
    }
}

template <int IO>
hipError_t launch_update_io(const LinUpdateArgs& a, hipStream_t s) {
    const int slabs = (a.dv + 63) / 64;
    const dim3 grid(static_cast<unsigned>(a.batch * a.heads * slabs)), block(kLinUpdateThreads);
    if (a.dk <= 64) hipLaunchKernelGGL((linear_attn_update_kernel<IO, 64>), grid, block, 0, s, a, slabs);
    else if (a.dk <= 128) hipLaunchKernelGGL((linear_attn_update_kernel<IO, 128>), grid, block, 0, s, a, slabs);
    else hipLaunchKernelGGL((linear_attn_update_kernel<IO, 256>), grid, block, 0, s, a, slabs);
    return hipGetLastError();
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The backward call's scratch, in order: each part 256-byte aligned.
struct BwdScratch {
    size_t seg_s = 0, seg_d = 0, dg = 0, dk = 0, dv = 0, total = 0;
};

BwdScratch bwd_scratch(const LinearAttnCall& c, const LinPlan& p, int nblk) {
    BwdScratch w;
    const size_t bh = static_cast<size_t>(c.batch) * c.heads;
    const size_t seg = p.nseg > 1 ? up256(bh * p.nseg * c.dk * c.dv * 4) : 0;
    w.seg_s = 0;
    w.seg_d = seg;
    w.dg = w.seg_d + seg;
    w.dk = w.dg + up256(bh * p.nseg * nblk * 8);
    const size_t rows = c.heads != c.kv_heads ? static_cast<size_t>(c.batch) * c.seqlen * c.heads : 0;
    w.dv = w.dk + up256(rows * c.dk * 4);
    w.total = w.dv + up256(rows * c.dv * 4);
    return w;
}

int max_dim(const LinearAttnCall& c) { return c.dk > c.dv ? c.dk : c.dv; }

int bwd_blocks(const LinearAttnCall& c) { return lin_blocks(max_dim(c)); }

LinArgs base_args(const LinearAttnCall& c, const LinPlan& p) {
    LinArgs a = {};
    a.batch = c.batch;
    a.seqlen = c.seqlen;
    a.seg_len = p.seg_len;
    a.heads = c.heads;
    a.rep = c.heads / c.kv_heads;
    a.nseg = p.nseg;
    a.npass = 1;
    a.lengths = c.lengths;
    a.log_decay = c.log_decay;
    a.scale = c.scale;
    return a;
}

LinPass forward_pass(const LinearAttnCall& c) {
    LinPass s = {};
    s.q = c.q;
    s.k = c.k;
    s.v = c.v;
    s.out = c.o;
    s.s_in = c.h0;
    s.s_out = c.hL;
    s.sn = c.dv;
    s.sp = 1;
    s.hq = c.heads;
    s.hk = s.hv = c.kv_heads;
    s.dc = c.dk;
    s.dout = c.dv;
    s.out_scale = c.scale;
    s.state_scale = 1.0f;
    return s;
}

template <int MODE>
hipError_t launch_mode(const LinearAttnCall& c, const LinArgs& a, int dc_pad, hipStream_t s) {
    return c.io == kIoF32 ? launch_linear_attn_variant<kIoF32, MODE>(a, dc_pad, s)
                          : launch_linear_attn_variant<kIoBF16, MODE>(a, dc_pad, s);
}

hipError_t launch_join(const LinearAttnCall& c, const LinPlan& p, float* seg_s, float* seg_d,
                       hipStream_t s) {
    JoinArgs j = {};
    j.batch = c.batch;
    j.seqlen = c.seqlen;
    j.seg_len = p.seg_len;
    j.state_elems = static_cast<int64_t>(c.dk) * c.dv;
    j.heads = c.heads;
    j.nseg = p.nseg;
    j.lengths = c.lengths;
    j.log_decay = c.log_decay;
    j.seg[0] = seg_s;
    j.seg[1] = seg_d;
    j.init[0] = c.h0;
    j.init[1] = c.dhL;
    const dim3 grid(static_cast<unsigned>((j.state_elems / 4 + 255) / 256),
                    static_cast<unsigned>(c.batch * c.heads), seg_d != nullptr ? 2 : 1);
    hipLaunchKernelGGL(linear_attn_join_kernel, grid, dim3(256), 0, s, j);
    return hipGetLastError();
}

hipError_t launch_share(const LinearAttnCall& c, const float* part_k, const float* part_v,
                        const DecaySumArgs& decay, hipStream_t s) {
    ShareArgs a = {};
    a.rows = c.batch * c.seqlen * c.kv_heads;
    a.rep = c.heads / c.kv_heads;
    a.dim[0] = c.dk;
    a.dim[1] = c.dv;
    a.part[0] = part_k;
    a.part[1] = part_v;
    a.out[0] = c.d_k;
    a.out[1] = c.d_v;
    a.decay = decay;
    const int64_t sums = decay.out != nullptr ? decay.heads : 0;
    const dim3 grid(static_cast<unsigned>(sums + stride_blocks(a.rows * (max_dim(c) / 4))), 2), block(256);
    if (c.io == kIoF32) hipLaunchKernelGGL((linear_attn_share_kernel<kIoF32>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((linear_attn_share_kernel<kIoBF16>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t linear_attn_workspace_bytes(const LinearAttnCall& c, const LinPlan& p, bool bwd) {
    if (bwd) return bwd_scratch(c, p, bwd_blocks(c)).total;
    return p.nseg > 1 ? static_cast<size_t>(c.batch) * c.heads * p.nseg * c.dk * c.dv * 4 : 0;
}

hipError_t launch_linear_attn_fwd(const LinearAttnCall& c, const LinPlan& p, void* ws, hipStream_t s) {
    LinArgs a = base_args(c, p);
    a.nblk = lin_blocks(c.dv);
    a.pass[0] = forward_pass(c);
    a.pass[0].seg_in = static_cast<float*>(ws);
    a.exact = c.hL != nullptr;
    if (p.nseg > 1) {
        hipError_t e = launch_mode<kLinState>(c, a, lin_padded(c.dk), s);
        if (e != hipSuccess) return e;
        e = launch_join(c, p, static_cast<float*>(ws), nullptr, s);
        if (e != hipSuccess) return e;
    }
    return launch_mode<kLinFwd>(c, a, lin_padded(c.dk), s);
}

hipError_t launch_linear_attn_bwd(const LinearAttnCall& c, const LinPlan& p, void* ws, hipStream_t s) {
    const int dc_pad = lin_padded(max_dim(c));
    const int nblk = p.two ? lin_blocks(c.dk) : bwd_blocks(c);   // of the launch with dq
    const BwdScratch w = bwd_scratch(c, p, bwd_blocks(c));
    char* base = static_cast<char*>(ws);
    float* seg_s = p.nseg > 1 ? reinterpret_cast<float*>(base + w.seg_s) : nullptr;
    float* seg_d = p.nseg > 1 ? reinterpret_cast<float*>(base + w.seg_d) : nullptr;
    const bool shared = c.heads != c.kv_heads;
    float* part_k = reinterpret_cast<float*>(base + w.dk);
    float* part_v = reinterpret_cast<float*>(base + w.dv);
    double* dg = c.dlog_decay != nullptr ? reinterpret_cast<double*>(base + w.dg) : nullptr;
    hipError_t e = hipSuccess;
    if (c.batch > 0) {
        // the states and adjoints, (dk, dv) in memory for every pass
        LinPass states = forward_pass(c);
        states.seg_in = seg_s;
        LinPass adj = {};
        adj.q = c.k;
        adj.k = c.q;
        adj.v = c.d_o;
        adj.out = shared ? part_v : c.d_v;
        adj.s_in = c.dhL;
        adj.s_out = c.dh0;
        adj.seg_in = seg_d;
        adj.sn = c.dv;
        adj.sp = 1;
        adj.hq = c.kv_heads;
        adj.hk = adj.hv = c.heads;
        adj.dc = c.dk;
        adj.dout = c.dv;
        adj.out_scale = 1.0f;
        adj.state_scale = c.scale;
        adj.rev = 1;
        adj.out32 = shared;
        if (p.nseg > 1) {
            LinArgs a = base_args(c, p);
            a.nblk = lin_blocks(c.dv);
            a.npass = 2;
            a.exact = dg != nullptr || c.dh0 != nullptr;
            a.pass[0] = states;
            a.pass[1] = adj;
            e = launch_mode<kLinState>(c, a, lin_padded(c.dk), s);
            if (e != hipSuccess) return e;
            e = launch_join(c, p, seg_s, seg_d, s);
            if (e != hipSuccess) return e;
        }
        LinArgs a = base_args(c, p);
        a.dg = dg;
        a.dhL = c.dhL;
        a.adj_in = seg_d;
        LinPass& q = a.pass[0];   // the pass that forms the decay's gradient is the first
        q = states;
        q.q = c.d_o;
        q.k = c.v;
        q.v = c.k;
        q.x = c.q;
        q.out = c.dq;
        q.s_out = nullptr;
        q.sn = 1;
        q.sp = c.dv;
        q.dc = c.dv;
        q.dout = c.dk;
        LinPass& k = a.pass[1];
        k = adj;
        k.q = c.v;
        k.k = c.d_o;
        k.v = c.q;
        k.out = shared ? static_cast<void*>(part_k) : c.d_k;
        k.s_out = nullptr;
        k.sn = 1;
        k.sp = c.dv;
        k.dc = c.dv;
        k.dout = c.dk;
        a.pass[2] = adj;
        a.npass = p.two ? 2 : 3;
        a.nblk = nblk;
        e = launch_mode<kLinBwd>(c, a, p.two ? lin_padded(c.dv) : dc_pad, s);
        if (e != hipSuccess) return e;
        if (p.two) {
            a.pass[0] = adj;
            a.npass = 1;
            a.nblk = lin_blocks(c.dv);
            a.dg = nullptr;
            e = launch_mode<kLinBwd>(c, a, lin_padded(c.dk), s);
            if (e != hipSuccess) return e;
        }
    }
    // the sums over workgroups and heads
    const DecaySumArgs decay = {c.batch * p.nseg * nblk, c.heads, dg, c.dlog_decay};
    if (shared && c.batch > 0 && c.seqlen > 0) return launch_share(c, part_k, part_v, decay, s);
    if (c.dlog_decay != nullptr) {
        hipLaunchKernelGGL(linear_attn_decay_kernel, dim3(static_cast<unsigned>(c.heads)), dim3(256), 0, s, decay);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_linear_attn_update(const LinUpdateArgs& a, hipStream_t s) {
    return a.io == kIoF32 ? launch_update_io<kIoF32>(a, s) : launch_update_io<kIoBF16>(a, s);
}

}  // namespace mamba
