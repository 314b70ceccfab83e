// Gated linear recurrence: forward, gradients, single token. Per channel, with
// p = sigmoid(decay gate), q = sigmoid(input gate), g = log_decay p:
//     a = exp(g),  b = sqrt(1 - a^2),  w = b q,   h_t = a_t h_{t-1} + w_t x_t
// and backward, with A_t = dy_t + a_{t+1} A_{t+1} the gradient at h_t:
//     dx = A w       d(input gate) = A w x (1 - q)       dh0 = a_0 A_0
//     dg = A a (h_{t-1} - q x a / b)
//     d(decay gate) = dg g (1 - p)       d(log_decay) = sum of dg p
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "internal.h"

namespace mamba {
namespace {

constexpr int kGsChannels = 64;   // channels of a workgroup

// 2^x - 1 = 2^(x/2) 2 sinh(x ln2 / 2), by the odd series of sinh: for x in
// (-1, 0] the terms left out are below 1e-9 of the value, which keeps its
// accuracy however near to 0 it is.
__device__ __forceinline__ float exp2m1_small(float x) {
    const float y = x * (0.5f * kLn2);
    const float t = y * y;
    const float s = fmaf(t, fmaf(t, fmaf(t, 1.0f / 5040.0f, 1.0f / 120.0f), 1.0f / 6.0f), 1.0f);
    return fast_exp2(0.5f * x) * (2.0f * y * s);
}

// A state c carried over tokens whose decays have the base-2 logarithms' sum G
// and that add h: c + (2^G - 1) c + h. Next to 1 the decay is taken by its
// difference from 1: as a factor, its rounding, the same tile after tile where
// gates are constant, would add up over a slow channel's memory. Far from 1 the
// difference would round at the size of the old state, of which little is left.
__device__ __forceinline__ float carried(float c, float G, float h) {
    const float near = c + fmaf(exp2m1_small(G), c, h);
    const float far = fmaf(fast_exp2(G), c, h);
    return G > -1.0f ? near : far;
}

// The gates of one value. s = 1 - a^2 = -2 a sinh(g): for a > 1/2 by the series,
// whose last coefficient takes up the terms left out (1e-8 of s), as 1 - a^2
// would lose what is left of it next to 1.
struct Decay1 {
    float g2, a, s;   // log2(a), a, 1 - a^2

    __device__ __forceinline__ Decay1(float p, float lam2) {
        g2 = lam2 * p;
        a = fast_exp2(g2);
        constexpr float L = kLn2 * kLn2, K = -2.0f * kLn2;
        const float t = g2 * g2;
        const float k = fmaf(t, fmaf(t, fmaf(t, K * L * L * L * (1.0f / 5040.0f + 0.4f / 362880.0f),
                                             K * L * L / 120.0f), K * L / 6.0f), K);
        const float near = (g2 * a) * k;
        s = g2 > -1.0f ? near : fmaf(-a, a, 1.0f);
    }
};

__device__ __forceinline__ float sigmoid(float v) {
    return fast_rcp(1.0f + fast_exp2(-v * kLog2e));
}

// sigmoid(v) and 1 - sigmoid(v), each to its own accuracy.
__device__ __forceinline__ void sigmoid_both(float v, float& p, float& rest) {
    const float e = fast_exp2(fminf(-v * kLog2e, 126.0f));
    p = fast_rcp(1.0f + e);
    rest = e * p;
    if (v != v) p = rest = v;   // the minimum above drops a NaN
}

constexpr int words_of(int io, int v) { return io == kIoF32 ? v : (v + 1) / 2; }

// A lane's V neighbouring channels of T tokens, as loaded.
template <int IO, int V, int T>
struct Raw {
    static constexpr int K = words_of(IO, V);
    uint32_t w[T][K];

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t row_bytes) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int off = static_cast<int>(at + t * row_bytes);
            if constexpr (IO == kIoBF16 && V == 1) {
                w[t][0] = __builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0);
            } else if constexpr (K == 1) {
                w[t][0] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
            } else {
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                static_assert(K == 2, "words of a token");
                const u32x2 r = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
                w[t][0] = r[0];
                w[t][1] = r[1];
            }
        }
    }
    __device__ __forceinline__ float get(int t, int v) const {
        if constexpr (IO == kIoF32) return __uint_as_float(w[t][v]);
        const uint32_t r = w[t][v / 2];
        return __uint_as_float(v % 2 ? r & 0xffff0000u : r << 16);
    }
};

// Stores V neighbouring channels of one token.
template <int IO, int V>
__device__ __forceinline__ void store_channels(__amdgpu_buffer_rsrc_t rs, uint32_t at, const float (&v)[V]) {
    const int off = static_cast<int>(at);
    if constexpr (IO == kIoBF16 && V == 1) {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, static_cast<__bf16>(v[0])), rs, off,
                                              0, 0);
    } else {
        uint32_t w[words_of(IO, V)];
#pragma unroll
        for (int i = 0; i < words_of(IO, V); ++i) {
            if constexpr (IO == kIoF32) {
                w[i] = __float_as_uint(v[i]);
            } else {
                const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[2 * i]));
                const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[2 * i + 1]));
                w[i] = lo | hi << 16;
            }
        }
        if constexpr (words_of(IO, V) == 1) {
            __builtin_amdgcn_raw_buffer_store_b32(w[0], rs, off, 0, 0);
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0], w[1]}, rs, off, 0, 0);
        }
    }
}

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t seqlen) {
    if (lengths == nullptr) return seqlen;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n < seqlen ? n : seqlen);
}

// A workgroup's place: the tile of TILE tokens by 64 channels is cut into S
// segments of T consecutive tokens, V of them side by side in a wave whose 64 / V
// lanes hold V channels each. The buffer resources span a tile's rows, so loads
// behind the row's last token give zeros and stores behind the sequence are
// dropped; a lane without channels has an offset past every resource.
template <int IO, int V, int T, int W>
struct Place {
    static constexpr int S = W * V, TILE = S * T;
    static constexpr int SIZE = IO == kIoF32 ? 4 : 2;
    static constexpr uint32_t kNowhere = 0x80000000u;
    static_assert(TILE % kGatedBlock == 0 && kGatedBlock % T == 0, "blocks of states at segments");
    int wave, sub, cl, seg, ch;   // ch: the lane's first channel; cl: within the workgroup
    bool in;

    __device__ __forceinline__ Place(int64_t dim, int64_t group) {
        const int lane = threadIdx.x % kWave;
        wave = threadIdx.x / kWave;
        sub = lane / (kWave / V);
        cl = lane % (kWave / V) * V;
        seg = wave * V + sub;
        ch = static_cast<int>(group * kGsChannels) + cl;
        in = ch < dim;
    }
    __device__ __forceinline__ uint32_t offset(int64_t stride) const {
        return in ? static_cast<uint32_t>((seg * T * stride + ch) * SIZE) : kNowhere;
    }
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const void* p, int64_t first, int64_t stride,
                                                                  int64_t dim, int64_t count) {
        const int64_t n = count < TILE ? count : TILE;
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(static_cast<const char*>(p) + first * stride * SIZE), 0,
            n > 0 ? static_cast<int>(((n - 1) * stride + dim) * SIZE) : 0, 0x00020000);
    }
};

// What precedes a lane's segment in its wave, and the wave's whole: a state c
// that enters the wave enters the segment as 2^G c + h. BACK goes from the
// last segment to the first.
template <int V, bool BACK>
struct Before {
    float P[V], h[V];

    __device__ __forceinline__ Before(int sub, float (&allP)[V], float (&allh)[V]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.0f;
            h[v] = 0.0f;
        }
#pragma unroll
        for (int m = 1; m < V; m *= 2) {
            const bool later = ((sub & m) != 0) != BACK;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float oP = __shfl_xor(allP[v], m * (kWave / V)), oh = __shfl_xor(allh[v], m * (kWave / V));
                if (later) {
                    h[v] = fmaf(P[v], oh, h[v]);
                    P[v] *= oP;
                    allh[v] = fmaf(allP[v], oh, allh[v]);
                } else {
                    allh[v] = fmaf(oP, allh[v], oh);
                }
                allP[v] *= oP;
            }
        }
    }
};

// The forward pass. A workgroup walks one row's tiles; the state entering a
// tile is known to every lane.
template <int IO, int V, int T, int W, bool GATED>
__global__ __launch_bounds__(W* kWave) void gated_scan_fwd_kernel(GatedScanArgs a, int64_t groups) {
    typedef Place<IO, V, T, W> P;
    typedef Raw<IO, V, T> R;
    __shared__ float2 sums[2][W][kGsChannels];
    const int64_t b = blockIdx.x / groups;
    const P at(a.dim, blockIdx.x - b * groups);
    const int64_t len = row_length(a.lengths, b, a.seqlen);
    const int64_t blocks = (a.seqlen + kGatedBlock - 1) / kGatedBlock;
    float lam2[V], c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        lam2[v] = at.in ? a.log_decay[at.ch + v] * kLog2e : 0.0f;
        c[v] = at.in && a.h0 != nullptr ? a.h0[b * a.dim + at.ch + v] : 0.0f;
    }
    const uint32_t off_x = at.offset(a.x_stride), off_d = at.offset(a.decay_stride),
                   off_i = at.offset(a.input_stride), off_y = at.offset(a.dim);
    const uint32_t step_x = static_cast<uint32_t>(a.x_stride) * P::SIZE,
                   step_d = static_cast<uint32_t>(a.decay_stride) * P::SIZE,
                   step_i = static_cast<uint32_t>(a.input_stride) * P::SIZE,
                   step_y = static_cast<uint32_t>(a.dim) * P::SIZE;
    R x, d, i;
    auto fetch = [&](int64_t t0) {
        const int64_t first = b * a.seqlen + t0;
        d.load(P::rows(a.decay_gate, first, a.decay_stride, a.dim, len - t0), off_d, step_d);
        if constexpr (GATED) i.load(P::rows(a.input_gate, first, a.input_stride, a.dim, len - t0), off_i, step_i);
        x.load(P::rows(a.x, first, a.x_stride, a.dim, len - t0), off_x, step_x);
    };
    int odd = 0;
    if (len > 0) fetch(0);
    for (int64_t t0 = 0; t0 < len; t0 += P::TILE) {
        const int64_t left = len - t0;
        const bool full = left >= P::TILE;
        float ca[T][V], cu[T][V], G[V], hl[V];
#pragma unroll
        for (int v = 0; v < V; ++v) G[v] = hl[v] = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay1 e(sigmoid(d.get(t, v)), lam2[v]);
                float w = __builtin_amdgcn_sqrtf(e.s);
                if constexpr (GATED) w *= sigmoid(i.get(t, v));
                ca[t][v] = e.a;
                cu[t][v] = w * x.get(t, v);
                float g = e.g2;
                if (!full && at.seg * T + t >= left) {   // behind the row's end: the state stays
                    ca[t][v] = 1.0f;
                    cu[t][v] = g = 0.0f;
                }
                G[v] += g;
                hl[v] = fmaf(ca[t][v], hl[v], cu[t][v]);
            }
        if (t0 + P::TILE < len) fetch(t0 + P::TILE);
        float wP[V], wG[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            wP[v] = fast_exp2(G[v]);
            wG[v] = G[v];
#pragma unroll
            for (int m = 1; m < V; m *= 2) wG[v] += __shfl_xor(wG[v], m * (kWave / V));
        }
        const Before<V, false> before(at.sub, wP, hl);
        if (at.sub == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) sums[odd][at.wave][at.cl + v] = make_float2(wG[v], hl[v]);
        }
        __syncthreads();
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float Gz = 0.0f, hz = 0.0f, Gw = 0.0f, hw = 0.0f;   // of the waves so far; before this wave
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 e = sums[odd][w][at.cl + v];
                if (w == at.wave) {
                    Gw = Gz;
                    hw = hz;
                }
                hz = fmaf(fast_exp2(e.x), hz, e.y);
                Gz += e.x;
            }
            h[v] = fmaf(before.P[v], carried(c[v], Gw, hw), before.h[v]);
            c[v] = carried(c[v], Gz, hz);
        }
        odd ^= 1;
        const int64_t tseg = t0 + at.seg * T;
        if (a.states != nullptr && at.seg * T % kGatedBlock == 0 && tseg < len && at.in) {
            float* s = a.states + (b * blocks + tseg / kGatedBlock) * a.dim + at.ch;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = h[v];
        }
        const __amdgpu_buffer_rsrc_t out = P::rows(a.y, b * a.seqlen + t0, a.dim, a.dim, a.seqlen - t0);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[v] = fmaf(ca[t][v], h[v], cu[t][v]);
                y[v] = !full && at.seg * T + t >= left ? 0.0f : h[v];
            }
            store_channels<IO, V>(out, off_y + t * step_y, y);
        }
    }
    if (a.hL != nullptr && at.in && at.seg == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.hL[b * a.dim + at.ch + v] = c[v];
    }
    for (int64_t t0 = (len + P::TILE - 1) / P::TILE * P::TILE; t0 < a.seqlen; t0 += P::TILE) {
        const __amdgpu_buffer_rsrc_t out = P::rows(a.y, b * a.seqlen + t0, a.dim, a.dim, a.seqlen - t0);
        const float none[V] = {};
#pragma unroll
        for (int t = 0; t < T; ++t) store_channels<IO, V>(out, off_y + t * step_y, none);
    }
}

// The backward pass: tiles from the last to the first. The state entering a
// tile comes from the forward pass, the adjoint entering it from behind is known
// to every lane.
template <int IO, int V, int T, int W, bool GATED>
__global__ __launch_bounds__(W* kWave) void gated_scan_bwd_kernel(GatedScanArgs a, int64_t groups,
                                                                  double* partial) {
    typedef Place<IO, V, T, W> P;
    typedef Raw<IO, V, T> R;
    __shared__ float4 sums[2][W][kGsChannels];   // G, what the tokens add to the state, to the adjoint
    const int64_t b = blockIdx.x / groups;
    const P at(a.dim, blockIdx.x - b * groups);
    const int64_t len = row_length(a.lengths, b, a.seqlen);
    const int64_t blocks = (a.seqlen + kGatedBlock - 1) / kGatedBlock;
    float lam2[V], D[V];
    double dl[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        lam2[v] = at.in ? a.log_decay[at.ch + v] * kLog2e : 0.0f;
        D[v] = at.in && a.dhL != nullptr ? a.dhL[b * a.dim + at.ch + v] : 0.0f;
        dl[v] = 0.0;
    }
    const uint32_t off_x = at.offset(a.x_stride), off_d = at.offset(a.decay_stride),
                   off_i = at.offset(a.input_stride), off_y = at.offset(a.dim);
    const uint32_t step_x = static_cast<uint32_t>(a.x_stride) * P::SIZE,
                   step_d = static_cast<uint32_t>(a.decay_stride) * P::SIZE,
                   step_i = static_cast<uint32_t>(a.input_stride) * P::SIZE,
                   step_y = static_cast<uint32_t>(a.dim) * P::SIZE;
    int odd = 0;
    const int64_t tiles = (len + P::TILE - 1) / P::TILE;
    for (int64_t t0 = (tiles - 1) * P::TILE; t0 >= 0; t0 -= P::TILE) {
        const int64_t left = len - t0, first = b * a.seqlen + t0;
        const bool full = left >= P::TILE;
        R x, d, i, dy;
        d.load(P::rows(a.decay_gate, first, a.decay_stride, a.dim, left), off_d, step_d);
        dy.load(P::rows(a.dy, first, a.dim, a.dim, left), off_y, step_y);
        if constexpr (GATED) i.load(P::rows(a.input_gate, first, a.input_stride, a.dim, left), off_i, step_i);
        x.load(P::rows(a.x, first, a.x_stride, a.dim, left), off_x, step_x);
        float c[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            c[v] = at.in ? a.states[(b * blocks + t0 / kGatedBlock) * a.dim + at.ch + v] : 0.0f;
        float ca[T][V], cw[T][V], cp[T][V], cgr[T][V], cir[T][V], ck[T][V], G[V], hl[V], El[V];
#pragma unroll
        for (int v = 0; v < V; ++v) G[v] = hl[v] = El[v] = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p, rest;
                sigmoid_both(d.get(t, v), p, rest);
                const Decay1 e(p, lam2[v]);
                const float rb = e.s > 1.1754944e-38f ? __builtin_amdgcn_rsqf(e.s) : (e.s == e.s ? 0.0f : e.s);
                const float xv = x.get(t, v);
                float w = e.s * rb, qx = xv;
                if constexpr (GATED) {
                    float q, qrest;
                    sigmoid_both(i.get(t, v), q, qrest);
                    w *= q;
                    qx *= q;
                    cir[t][v] = w * xv * qrest;
                }
                ca[t][v] = e.a;
                cw[t][v] = w;
                cp[t][v] = p;
                cgr[t][v] = e.g2 * kLn2 * rest;
                ck[t][v] = qx * (e.a * rb);
                float g = e.g2, u = w * xv;
                if (!full && at.seg * T + t >= left) {
                    ca[t][v] = 1.0f;
                    u = g = 0.0f;
                }
                G[v] += g;
                hl[v] = fmaf(ca[t][v], hl[v], u);
            }
#pragma unroll
        for (int t = T - 1; t >= 0; --t)
#pragma unroll
            for (int v = 0; v < V; ++v) El[v] = ca[t][v] * (dy.get(t, v) + El[v]);
        float wP[V], wPb[V], wG[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            wP[v] = wPb[v] = fast_exp2(G[v]);
            wG[v] = G[v];
#pragma unroll
            for (int m = 1; m < V; m *= 2) wG[v] += __shfl_xor(wG[v], m * (kWave / V));
        }
        const Before<V, false> before(at.sub, wP, hl);
        const Before<V, true> behind(at.sub, wPb, El);
        if (at.sub == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) sums[odd][at.wave][at.cl + v] = make_float4(wG[v], hl[v], El[v], 0.0f);
        }
        __syncthreads();
        float h[V], A[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float Gz = 0.0f, hz = 0.0f, Gw = 0.0f, hw = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float4 e = sums[odd][w][at.cl + v];
                if (w == at.wave) {
                    Gw = Gz;
                    hw = hz;
                }
                hz = fmaf(fast_exp2(e.x), hz, e.y);
                Gz += e.x;
            }
            h[v] = fmaf(before.P[v], carried(c[v], Gw, hw), before.h[v]);
            float Ez = 0.0f, Ew = 0.0f;
            Gz = 0.0f;
#pragma unroll
            for (int w = W - 1; w >= 0; --w) {
                const float4 e = sums[odd][w][at.cl + v];
                if (w == at.wave) {
                    Gw = Gz;
                    Ew = Ez;
                }
                Ez = fmaf(fast_exp2(e.x), Ez, e.z);
                Gz += e.x;
            }
            A[v] = fmaf(behind.P[v], carried(D[v], Gw, Ew), behind.h[v]);
            D[v] = carried(D[v], Gz, Ez);
        }
        odd ^= 1;
        float sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = 0.0f;
        // ck becomes h_{t-1} - q x a / b
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ck[t][v] = h[v] - ck[t][v];
                h[v] = fmaf(ca[t][v], h[v], cw[t][v] * x.get(t, v));
            }
        const __amdgpu_buffer_rsrc_t ox = P::rows(a.dx, first, a.dim, a.dim, a.seqlen - t0),
                                     od = P::rows(a.ddecay, first, a.dim, a.dim, a.seqlen - t0),
                                     oi = P::rows(a.dinput, first, a.dim, a.dim, GATED ? a.seqlen - t0 : 0);
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            float vx[V], vd[V], vi[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const bool gone = !full && at.seg * T + t >= left;
                const float At = dy.get(t, v) + A[v];
                A[v] = ca[t][v] * At;
                const float dg = gone ? 0.0f : A[v] * ck[t][v];
                vx[v] = gone ? 0.0f : At * cw[t][v];
                vd[v] = gone ? 0.0f : dg * cgr[t][v];
                if constexpr (GATED) vi[v] = gone ? 0.0f : At * cir[t][v];
                sum[v] = fmaf(dg, cp[t][v], sum[v]);
            }
            store_channels<IO, V>(ox, off_y + t * step_y, vx);
            store_channels<IO, V>(od, off_y + t * step_y, vd);
            if constexpr (GATED) store_channels<IO, V>(oi, off_y + t * step_y, vi);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) dl[v] += static_cast<double>(sum[v]);
    }
    if (a.dh0 != nullptr && at.in && at.seg == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[b * a.dim + at.ch + v] = D[v];
    }
    if (partial != nullptr) {
        __shared__ double all[P::S][kGsChannels];
#pragma unroll
        for (int v = 0; v < V; ++v) all[at.seg][at.cl + v] = dl[v];
        __syncthreads();
        if (at.seg == 0 && at.in) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                double s = 0.0;
#pragma unroll
                for (int k = 0; k < P::S; ++k) s += all[k][at.cl + v];
                partial[b * a.dim + at.ch + v] = s;
            }
        }
    }
    for (int64_t t0 = tiles * P::TILE; t0 < a.seqlen; t0 += P::TILE) {
        const int64_t first = b * a.seqlen + t0;
        const __amdgpu_buffer_rsrc_t ox = P::rows(a.dx, first, a.dim, a.dim, a.seqlen - t0),
                                     od = P::rows(a.ddecay, first, a.dim, a.dim, a.seqlen - t0),
                                     oi = P::rows(a.dinput, first, a.dim, a.dim, GATED ? a.seqlen - t0 : 0);
        const float none[V] = {};
#pragma unroll
        for (int t = 0; t < T; ++t) {
            store_channels<IO, V>(ox, off_y + t * step_y, none);
            store_channels<IO, V>(od, off_y + t * step_y, none);
            if constexpr (GATED) store_channels<IO, V>(oi, off_y + t * step_y, none);
        }
    }
}

// The rows' sums of d(log_decay), in order.
__global__ __launch_bounds__(256) void gated_scan_sum_kernel(int64_t rows, int64_t dim, const double* partial,
                                                             float* out) {
    const int64_t ch = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (ch >= dim) return;
    double s = 0.0;
    for (int64_t r = 0; r < rows; ++r) s += partial[r * dim + ch];
    out[ch] = static_cast<float>(s);
}

// Without tokens: dh0 = dhL, no gradient of the decay.
__global__ __launch_bounds__(256) void gated_scan_empty_kernel(int64_t state, int64_t dim, const float* from,
                                                               float* to, float* zero) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < state || i < dim; i += stride) {
        if (to != nullptr && i < state) to[i] = from != nullptr ? from[i] : 0.0f;
        if (zero != nullptr && i < dim) zero[i] = 0.0f;
    }
}

// One token: V channels to a lane.
template <int IO, int V>
__global__ __launch_bounds__(256) void gated_scan_update_kernel(GatedScanArgs a) {
    constexpr int SIZE = IO == kIoF32 ? 4 : 2;
    const int64_t lanes = a.dim / V, all = a.batch * lanes;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; j < all; j += stride) {
        const int64_t b = j / lanes, ch = (j - b * lanes) * V;
        struct alignas(V * SIZE) Vec { uint8_t bytes[V * SIZE]; };
        struct alignas(V * 4 < 16 ? V * 4 : 16) Wide { float f[V]; };
        auto read = [&](const void* p, int64_t stride_p, float (&o)[V]) {
            const Vec r = *reinterpret_cast<const Vec*>(static_cast<const char*>(p) + (b * stride_p + ch) * SIZE);
            uint32_t w[words_of(IO, V)];
            if constexpr (V * SIZE < 4) w[0] = *reinterpret_cast<const uint16_t*>(r.bytes);
            else __builtin_memcpy(w, r.bytes, sizeof w);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (IO == kIoF32) o[v] = __uint_as_float(w[v]);
                else o[v] = __uint_as_float(v % 2 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
            }
        };
        float x[V], d[V], i[V];
        Wide* hp = reinterpret_cast<Wide*>(a.h + b * a.dim + ch);
        Wide h = *hp;
        const Wide lam = *reinterpret_cast<const Wide*>(a.log_decay + ch);
        read(a.x, a.x_stride, x);
        read(a.decay_gate, a.decay_stride, d);
        if (a.input_gate != nullptr) read(a.input_gate, a.input_stride, i);
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Decay1 e(sigmoid(d[v]), lam.f[v] * kLog2e);
            float w = __builtin_amdgcn_sqrtf(e.s);
            if (a.input_gate != nullptr) w *= sigmoid(i[v]);
            o[v] = h.f[v] = carried(h.f[v], e.g2, w * x[v]);
        }
        *hp = h;
        if constexpr (IO == kIoF32) {
            Wide r;
#pragma unroll
            for (int v = 0; v < V; ++v) r.f[v] = o[v];
            *reinterpret_cast<Wide*>(static_cast<float*>(a.y) + b * a.dim + ch) = r;
        } else {
            Vec r;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint16_t u = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[v]));
                __builtin_memcpy(r.bytes + 2 * v, &u, 2);
            }
            *reinterpret_cast<Vec*>(static_cast<char*>(a.y) + (b * a.dim + ch) * SIZE) = r;
        }
    }
}

bool divides(const GatedScanArgs& a, int64_t v) {
    return a.dim % v == 0 && a.x_stride % v == 0 && a.decay_stride % v == 0 &&
           (a.input_gate == nullptr || a.input_stride % v == 0);
}

int64_t groups_of(const GatedScanArgs& a) { return (a.dim + kGsChannels - 1) / kGsChannels; }

template <int IO, int V, int T, int W>
hipError_t launch_fwd(const GatedScanArgs& a, hipStream_t s) {
    const int64_t groups = groups_of(a);
    const dim3 grid(static_cast<unsigned>(a.batch * groups)), block(W * kWave);
    if (a.input_gate != nullptr)
        hipLaunchKernelGGL((gated_scan_fwd_kernel<IO, V, T, W, true>), grid, block, 0, s, a, groups);
    else
        hipLaunchKernelGGL((gated_scan_fwd_kernel<IO, V, T, W, false>), grid, block, 0, s, a, groups);
    return hipGetLastError();
}

template <int IO, int V, int T, int W>
hipError_t launch_bwd(const GatedScanArgs& a, double* partial, hipStream_t s) {
    const int64_t groups = groups_of(a);
    const dim3 grid(static_cast<unsigned>(a.batch * groups)), block(W * kWave);
    if (a.input_gate != nullptr)
        hipLaunchKernelGGL((gated_scan_bwd_kernel<IO, V, T, W, true>), grid, block, 0, s, a, groups, partial);
    else
        hipLaunchKernelGGL((gated_scan_bwd_kernel<IO, V, T, W, false>), grid, block, 0, s, a, groups, partial);
    return hipGetLastError();
}

template <int IO, int V>
hipError_t launch_update(const GatedScanArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((gated_scan_update_kernel<IO, V>),
                       dim3(static_cast<unsigned>(stride_blocks(a.batch * (a.dim / V)))), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t gated_scan_fwd_workspace_bytes(const GatedScanArgs&) { return 0; }

size_t gated_scan_bwd_workspace_bytes(const GatedScanArgs& a) {
    return static_cast<size_t>(a.batch) * a.dim * sizeof(double);
}

hipError_t launch_gated_scan_fwd(const GatedScanArgs& a, void*, hipStream_t s) {
    if (a.io == kIoF32) return launch_fwd<kIoF32, 1, 16, 8>(a, s);
    return divides(a, 2) ? launch_fwd<kIoBF16, 2, 16, 4>(a, s) : launch_fwd<kIoBF16, 1, 16, 8>(a, s);
}

hipError_t launch_gated_scan_bwd(const GatedScanArgs& a, void* ws, hipStream_t s) {
    if (a.batch == 0 || a.seqlen == 0) {
        const int64_t state = a.batch * a.dim;
        hipLaunchKernelGGL(gated_scan_empty_kernel,
                           dim3(static_cast<unsigned>(stride_blocks(state > a.dim ? state : a.dim))), dim3(256), 0, s,
                           state, a.dim, a.dhL, a.dh0, a.dlog_decay);
        return hipGetLastError();
    }
    double* partial = a.dlog_decay != nullptr ? static_cast<double*>(ws) : nullptr;
    const hipError_t e = a.io == kIoF32 ? launch_bwd<kIoF32, 1, 8, 8>(a, partial, s)
                         : divides(a, 2) ? launch_bwd<kIoBF16, 2, 8, 4>(a, partial, s)
                                         : launch_bwd<kIoBF16, 1, 8, 8>(a, partial, s);
    if (e != hipSuccess || partial == nullptr) return e;
    hipLaunchKernelGGL(gated_scan_sum_kernel, dim3(static_cast<unsigned>((a.dim + 255) / 256)), dim3(256), 0, s,
                       a.batch, a.dim, partial, a.dlog_decay);
    return hipGetLastError();
}

hipError_t launch_gated_scan_update(const GatedScanArgs& a, hipStream_t s) {
    if (a.io == kIoF32) return divides(a, 4) ? launch_update<kIoF32, 4>(a, s) : launch_update<kIoF32, 1>(a, s);
    return divides(a, 4) ? launch_update<kIoBF16, 4>(a, s) : launch_update<kIoBF16, 1>(a, s);
}

}  // namespace mamba
