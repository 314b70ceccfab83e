// The norms around a block and their gradients.
//   gated:     v = x silu(z) or x,  n = v rstd,  y = n w, times silu(z) where the gate is behind
//              u = dy w (silu(z)),  dv = rstd (u - n mean(u n)),  dw = sum over rows of dy n (silu(z))
//   residual:  total = residual + scale x,  n = total rstd,  y = n w
//              d = dtotal + rstd (dy w - n mean(dy w n)),  dresidual = d,  dx = scale d,
//              dscale = sum of d x,  dw = sum of dy n
//
// All are bound by memory: every tensor is read or written once. A lane holds 8
// consecutive values of a part (16 above 8192 of them), so that a part of n values
// takes as many lanes as it has eights - 16 or 64 of a wave, or as many waves as
// they fill - and few registers; weights and the sums over rows stay in registers
// while a workgroup walks rows, with the next row's loads out.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace mamba {
namespace {

constexpr int kNormMaxWaves = 16;
constexpr int kNormThreads = 256;   // of a workgroup whose teams are waves or parts of one

template <int IO>
constexpr int size_of() { return IO == kIoF32 ? 4 : 2; }

// 16 bytes at any address of a value, for parts whose rows do not start on 16
// bytes: the memory takes such an access, at its cost in lines.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A lane's CH runs of 8 values of a part of n: run u starts at value
// (lane + team u) 8. ALIGNED: runs are whole and start on 16 bytes; else the last
// one may be short, and is taken value by value.
template <int IO, int CH, bool ALIGNED>
struct Cells {
    static constexpr int K = IO == kIoF32 ? 2 : 1;
    u32x4 q[CH * K];

    __device__ __forceinline__ void load(const void* p, int64_t at, int n, int lane, int team) {
        const char* base = static_cast<const char*>(p) + at * size_of<IO>();
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            const int i = (lane + team * u) * 8;
            const char* s = base + static_cast<int64_t>(i) * size_of<IO>();
#pragma unroll
            for (int k = 0; k < K; ++k) q[u * K + k] = u32x4{0, 0, 0, 0};
            if (ALIGNED ? i < n : i + 8 <= n) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if constexpr (ALIGNED) q[u * K + k] = reinterpret_cast<const u32x4*>(s)[k];
                    else q[u * K + k] = *reinterpret_cast<const u32x4_any*>(s + 16 * k);
                }
            } else if (!ALIGNED && i < n) {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (i + e < n) {
                        const uint32_t r = load_raw<IO>(s, e);
                        if constexpr (IO == kIoF32) q[u * K + e / 4][e % 4] = r;
                        else q[u][e / 2] |= e % 2 ? r << 16 : r;
                    }
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        const int u = i / 8, e = i % 8;
        if constexpr (IO == kIoF32) return __uint_as_float(q[u * 2 + e / 4][e % 4]);
        const uint32_t r = q[u][e / 2];
        return __uint_as_float(e % 2 ? r & 0xffff0000u : r << 16);
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, int n, int lane, int team,
                                                 const float (&v)[CH * 8]) {
        char* base = static_cast<char*>(p) + at * size_of<IO>();
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            const int i = (lane + team * u) * 8;
            char* d = base + static_cast<int64_t>(i) * size_of<IO>();
            if (ALIGNED ? i < n : i + 8 <= n) {
                u32x4 o[K];
#pragma unroll
                for (int e = 0; e < 8; e += IO == kIoF32 ? 1 : 2) {
                    if constexpr (IO == kIoF32) {
                        o[e / 4][e % 4] = __float_as_uint(v[8 * u + e]);
                    } else {
                        const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[8 * u + e]));
                        const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[8 * u + e + 1]));
                        o[0][e / 2] = lo | hi << 16;
                    }
                }
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if constexpr (ALIGNED) reinterpret_cast<u32x4*>(d)[k] = o[k];
                    else *reinterpret_cast<u32x4_any*>(d + 16 * k) = o[k];
                }
            } else if (!ALIGNED && i < n) {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (i + e < n) store_io<IO>(d, e, v[8 * u + e]);
            }
        }
    }
};

// The parameters of a lane's values.
template <int CH, bool ALIGNED>
__device__ __forceinline__ void load_params(const float* p, int64_t at, int n, int lane, int team,
                                            float (&v)[CH * 8]) {
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) v[i] = 1.0f;
    if (p == nullptr) return;
    Cells<kIoF32, CH, ALIGNED> t;
    t.load(p, at, n, lane, team);
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) v[i] = t.get(i);
}

// A workgroup's teams: TEAM lanes each, or (TEAM == 0) one of all its waves.
// `red` holds a sum for each wave, twice, so that one barrier a row is enough: a
// wave writes one half while others may still read the other. Waves that a
// workgroup has not count as zeros.
template <int TEAM>
struct Teams {
    int lane, team, size, count;
    int odd = 0;
    float (*red)[kNormMaxWaves];

    __device__ __forceinline__ explicit Teams(float (*slots)[kNormMaxWaves]) : red(slots) {
        size = TEAM == 0 ? blockDim.x : TEAM;
        count = TEAM == 0 ? 1 : kNormThreads / (TEAM == 0 ? 1 : TEAM);
        lane = TEAM == 0 ? threadIdx.x : threadIdx.x % (TEAM == 0 ? 1 : TEAM);
        team = TEAM == 0 ? 0 : threadIdx.x / (TEAM == 0 ? 1 : TEAM);
        if constexpr (TEAM == 0) {
            if (threadIdx.x < 2 * kNormMaxWaves) red[threadIdx.x / kNormMaxWaves][threadIdx.x % kNormMaxWaves] = 0.0f;
            __syncthreads();
        }
    }
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int m = 1; m < (TEAM == 0 ? kWave : TEAM); m *= 2) v += __shfl_xor(v, m);
        if constexpr (TEAM == 0) {
            if (threadIdx.x % kWave == 0) red[odd][threadIdx.x / kWave] = v;
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int w = 0; w < kNormMaxWaves; ++w) v += red[odd][w];
            odd ^= 1;
        }
        return v;
    }
};

// Which rows a workgroup takes: it stays with one group of columns and walks
// rows slot, slot + slots, ... times its teams. Every team takes the same number
// of turns; one without a row works on zeros and writes nothing.
struct Walk {
    int64_t grp, slot, step;

    __device__ __forceinline__ Walk(int64_t groups, int slots, int teams)
        : grp(blockIdx.x % groups), slot(blockIdx.x / groups), step(static_cast<int64_t>(slots) * teams) {}
};

__device__ __forceinline__ float silu_of(float z, float sg) { return z * sg; }

__device__ __forceinline__ float sigmoid(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

template <int IO, int TEAM, int CH, bool AL, int GATE>
__global__ __launch_bounds__(TEAM == 0 ? 1024 : kNormThreads) void gated_norm_fwd_kernel(GatedNormArgs a, int slots) {
    __shared__ float red[2][kNormMaxWaves];
    Teams<TEAM> tm(red);
    typedef Cells<IO, CH, AL> C;
    constexpr int N = CH * 8;
    const int n = static_cast<int>(a.dim / a.groups);
    const Walk walk(a.groups, slots, tm.count);
    const float inv = 1.0f / static_cast<float>(n);
    float w[N];
    load_params<CH, AL>(a.weight, walk.grp * n, n, tm.lane, tm.size, w);
    C x, z;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.rows;
        x.load(a.x, in ? row * a.x_stride + walk.grp * n : 0, in ? n : 0, tm.lane, tm.size);
        if constexpr (GATE != kGateNone)
            z.load(a.z, in ? row * a.z_stride + walk.grp * n : 0, in ? n : 0, tm.lane, tm.size);
    };
    fetch(walk.slot * tm.count + tm.team);
    for (int64_t r0 = walk.slot * tm.count; r0 < a.rows; r0 += walk.step) {
        const int64_t row = r0 + tm.team;
        float v[N], g[N], sq = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = x.get(i);
            if constexpr (GATE != kGateNone) g[i] = z.get(i) * sigmoid(z.get(i));
            if constexpr (GATE == kGateFirst) v[i] *= g[i];
            sq = fmaf(v[i], v[i], sq);
        }
        fetch(row + walk.step);
        const float rstd = 1.0f / sqrtf(fmaf(tm.sum(sq), inv, a.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = v[i] * rstd * w[i];
            if constexpr (GATE == kGateBehind) v[i] *= g[i];
        }
        const bool in = row < a.rows;
        C::store(a.y, in ? row * a.dim + walk.grp * n : 0, in ? n : 0, tm.lane, tm.size, v);
        if (in && tm.lane == 0 && a.rstd != nullptr) a.rstd[row * a.groups + walk.grp] = rstd;
    }
}

// The column sums of a workgroup's teams, in order, to out[i] of the part.
template <int TEAM, int CH>
__device__ __forceinline__ void put_columns(const Teams<TEAM>& tm, float* cols, float* out, int n,
                                            const float (&d)[CH * 8]) {
    if constexpr (TEAM == 0) {
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) {
            const int at = (tm.lane + tm.size * (i / 8)) * 8 + i % 8;
            if (at < n) out[at] = d[i];
        }
    } else {
        static_assert(CH == 1, "runs of a narrow part");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) cols[(tm.team * 8 + i) * TEAM + tm.lane] = d[i];
        __syncthreads();
        for (int j = threadIdx.x; j < TEAM * 8; j += kNormThreads) {
            float t = 0.0f;
            for (int k = 0; k < tm.count; ++k) t += cols[k * 8 * TEAM + j];
            const int at = j % TEAM * 8 + j / TEAM;
            if (at < n) out[at] = t;
        }
    }
}

template <int IO, int TEAM, int CH, bool AL, int GATE>
__global__ __launch_bounds__(TEAM == 0 ? 1024 : kNormThreads) void gated_norm_bwd_kernel(GatedNormArgs a, int slots,
                                                                                        float* partial) {
    __shared__ float red[2][kNormMaxWaves];
    __shared__ float cols[TEAM == 0 ? 1 : 8 * kNormThreads];
    Teams<TEAM> tm(red);
    typedef Cells<IO, CH, AL> C;
    constexpr int N = CH * 8;
    const int n = static_cast<int>(a.dim / a.groups);
    const Walk walk(a.groups, slots, tm.count);
    const float inv = 1.0f / static_cast<float>(n);
    float w[N], dw[N];
    load_params<CH, AL>(a.weight, walk.grp * n, n, tm.lane, tm.size, w);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = 0.0f;
    C x, z, dy;
    float rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.rows;
        const int m = in ? n : 0;
        x.load(a.x, in ? row * a.x_stride + walk.grp * n : 0, m, tm.lane, tm.size);
        if constexpr (GATE != kGateNone)
            z.load(a.z, in ? row * a.z_stride + walk.grp * n : 0, m, tm.lane, tm.size);
        dy.load(a.dy, in ? row * a.dim + walk.grp * n : 0, m, tm.lane, tm.size);
        rstd = in ? a.rstd[row * a.groups + walk.grp] : 0.0f;
    };
    fetch(walk.slot * tm.count + tm.team);
    for (int64_t r0 = walk.slot * tm.count; r0 < a.rows; r0 += walk.step) {
        const int64_t row = r0 + tm.team;
        // nm: the normed values, u: dy w (and the gate), gx and gz: what dx and dz
        // take of dv (of dy where the gate is behind)
        float nm[N], u[N], gx[N], gz[N], s = 0.0f;
        const float rs = rstd;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float xi = x.get(i);
            float up = dy.get(i), v = xi;
            gx[i] = 1.0f;
            gz[i] = 0.0f;
            if constexpr (GATE != kGateNone) {
                const float zi = z.get(i);
                // sigmoid and 1 - sigmoid, each to its own accuracy
                const float e = fast_exp2(fminf(-zi * kLog2e, 126.0f));
                const float sg = fast_rcp(1.0f + e), rest = zi == zi ? e * sg : zi;
                const float sl = zi * sg, dsl = sg * fmaf(zi, rest, 1.0f);
                if constexpr (GATE == kGateFirst) {
                    v = xi * sl;
                    gx[i] = sl;
                    gz[i] = xi * dsl;
                } else {
                    gz[i] = up * dsl * w[i];
                    up *= sl;
                }
            }
            nm[i] = v * rs;
            if constexpr (GATE == kGateBehind) gz[i] *= nm[i];
            dw[i] = fmaf(up, nm[i], dw[i]);
            u[i] = up * w[i];
            s = fmaf(u[i], nm[i], s);
        }
        fetch(row + walk.step);
        const float c = tm.sum(s) * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float dv = rs * fmaf(-nm[i], c, u[i]);
            u[i] = dv * gx[i];
            if constexpr (GATE == kGateFirst) gz[i] *= dv;
        }
        const bool in = row < a.rows;
        const int64_t at = in ? row * a.dim + walk.grp * n : 0;
        C::store(a.dx, at, in ? n : 0, tm.lane, tm.size, u);
        if constexpr (GATE != kGateNone) C::store(a.dz, at, in ? n : 0, tm.lane, tm.size, gz);
    }
    if (a.dweight == nullptr) return;
    float* out = (slots == 1 ? a.dweight : partial + walk.slot * a.dim) + walk.grp * n;
    put_columns<TEAM, CH>(tm, cols, out, n, dw);
}

template <int IO, int RIO, int TEAM, int CH, bool AL>
__global__ __launch_bounds__(TEAM == 0 ? 1024 : kNormThreads) void residual_norm_fwd_kernel(ResidualNormArgs a,
                                                                                           int slots) {
    __shared__ float red[2][kNormMaxWaves];
    Teams<TEAM> tm(red);
    typedef Cells<IO, CH, AL> C;
    typedef Cells<RIO, CH, AL> R;
    constexpr int N = CH * 8;
    const int n = static_cast<int>(a.dim);
    const Walk walk(1, slots, tm.count);
    const float inv = 1.0f / static_cast<float>(n);
    float w[N], sc[N];
    load_params<CH, AL>(a.weight, 0, n, tm.lane, tm.size, w);
    load_params<CH, AL>(a.scale, 0, n, tm.lane, tm.size, sc);
    C x;
    R res;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.rows;
        x.load(a.x, in ? row * n : 0, in ? n : 0, tm.lane, tm.size);
        res.load(a.residual, in ? row * n : 0, in ? n : 0, tm.lane, tm.size);
    };
    fetch(walk.slot * tm.count + tm.team);
    for (int64_t r0 = walk.slot * tm.count; r0 < a.rows; r0 += walk.step) {
        const int64_t row = r0 + tm.team;
        float v[N], sq = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = fmaf(sc[i], x.get(i), res.get(i));
            sq = fmaf(v[i], v[i], sq);
        }
        fetch(row + walk.step);
        const bool in = row < a.rows;
        const int64_t at = in ? row * n : 0;
        R::store(a.total, at, in ? n : 0, tm.lane, tm.size, v);
        const float rstd = 1.0f / sqrtf(fmaf(tm.sum(sq), inv, a.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] * rstd * w[i];
        C::store(a.y, at, in ? n : 0, tm.lane, tm.size, v);
        if (in && tm.lane == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    }
}

// SCALE: x is read and dscale formed.
template <int IO, int RIO, int TEAM, int CH, bool AL, bool SCALE>
__global__ __launch_bounds__(TEAM == 0 ? 1024 : kNormThreads) void residual_norm_bwd_kernel(ResidualNormArgs a,
                                                                                           int slots, float* partial) {
    __shared__ float red[2][kNormMaxWaves];
    __shared__ float cols[TEAM == 0 ? 1 : 8 * kNormThreads];
    Teams<TEAM> tm(red);
    typedef Cells<IO, CH, AL> C;
    typedef Cells<RIO, CH, AL> R;
    constexpr int N = CH * 8;
    const int n = static_cast<int>(a.dim);
    const Walk walk(1, slots, tm.count);
    const float inv = 1.0f / static_cast<float>(n);
    float w[N], sc[N], dw[N], ds[N];
    load_params<CH, AL>(a.weight, 0, n, tm.lane, tm.size, w);
    load_params<CH, AL>(a.scale, 0, n, tm.lane, tm.size, sc);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = ds[i] = 0.0f;
    R total, dt;
    C x, dy;
    float rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.rows;
        const int64_t at = in ? row * n : 0;
        const int m = in ? n : 0;
        total.load(a.total, at, m, tm.lane, tm.size);
        dy.load(a.dy, at, m, tm.lane, tm.size);
        dt.load(a.dtotal, at, a.dtotal != nullptr ? m : 0, tm.lane, tm.size);
        if constexpr (SCALE) x.load(a.x, at, m, tm.lane, tm.size);
        rstd = in ? a.rstd[row] : 0.0f;
    };
    fetch(walk.slot * tm.count + tm.team);
    for (int64_t r0 = walk.slot * tm.count; r0 < a.rows; r0 += walk.step) {
        const int64_t row = r0 + tm.team;
        float nm[N], u[N], s = 0.0f;
        const float rs = rstd;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            nm[i] = total.get(i) * rs;
            const float d = dy.get(i);
            dw[i] = fmaf(d, nm[i], dw[i]);
            u[i] = d * w[i];
            s = fmaf(u[i], nm[i], s);
        }
        const R dnow = dt;
        const C xnow = x;
        fetch(row + walk.step);
        const float c = tm.sum(s) * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float d = fmaf(rs, fmaf(-nm[i], c, u[i]), dnow.get(i));
            nm[i] = d;
            u[i] = d * sc[i];
            if constexpr (SCALE) ds[i] = fmaf(d, xnow.get(i), ds[i]);
        }
        const bool in = row < a.rows;
        const int64_t at = in ? row * n : 0;
        R::store(a.dresidual, at, in ? n : 0, tm.lane, tm.size, nm);
        C::store(a.dx, at, in && a.dx != nullptr ? n : 0, tm.lane, tm.size, u);
    }
    float* out = partial + walk.slot * a.dim;
    if (a.dweight != nullptr) put_columns<TEAM, CH>(tm, cols, slots == 1 ? a.dweight : out, n, dw);
    if constexpr (SCALE)
        put_columns<TEAM, CH>(tm, cols, slots == 1 ? a.dscale : out + static_cast<int64_t>(slots) * a.dim, n, ds);
}

// Column sums over the slots, in 64 bits and a fixed order: 64 columns per
// workgroup, its 16 waves a sixteenth of the slots each, 4 loads in flight. Plane
// y of `partial` goes to out[y].
constexpr int kColumnWaves = 16;

__global__ __launch_bounds__(kColumnWaves * kWave) void norm_columns_kernel(int64_t dim, int slots,
                                                                            const float* partial, float* out0,
                                                                            float* out1) {
    __shared__ double red[kColumnWaves][kWave];
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kWave + lane;
    float* out = blockIdx.y ? out1 : out0;
    if (out == nullptr) return;
    const float* p = partial + static_cast<int64_t>(blockIdx.y) * slots * dim;
    double s = 0.0;
    if (col < dim) {
        constexpr int U = 4;
        for (int k0 = w; k0 < slots; k0 += U * kColumnWaves) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * kColumnWaves;
                x[u] = k < slots ? p[static_cast<int64_t>(k) * dim + col] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) s += static_cast<double>(x[u]);
        }
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && col < dim) {
        double t = 0.0;
#pragma unroll
        for (int k = 0; k < kColumnWaves; ++k) t += red[k][lane];
        out[col] = static_cast<float>(t);
    }
}

__global__ __launch_bounds__(256) void norm_zero_kernel(int64_t dim, float* out0, float* out1) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= dim) return;
    if (out0 != nullptr) out0[i] = 0.0f;
    if (out1 != nullptr) out1[i] = 0.0f;
}

// Lanes of a team (0: all waves of its workgroup), runs of 8 values to a lane and
// threads of a workgroup for parts of n values.
struct Shape {
    int team, runs, threads;
};

constexpr Shape shape_for(int64_t n) {
    if (n <= 128) return {16, 1, kNormThreads};
    if (n <= 512) return {64, 1, kNormThreads};
    const int runs = n <= 8 * kWave * kNormMaxWaves ? 1 : 2;
    const int64_t waves = (n + 8 * kWave * runs - 1) / (8 * kWave * runs);
    return {0, runs, static_cast<int>(waves * kWave)};
}

static_assert(shape_for(kGatedNormMaxDim).threads <= kNormMaxWaves * kWave, "the widest part has a workgroup");

// Workgroups for each group of columns. Forward: several rounds of what the chip
// holds; backward: about `waves` waves to a compute unit, as every workgroup
// leaves its columns' sums.
int slots_for(int64_t rows, int64_t groups, const Shape& sh, int cu, int waves) {
    const int64_t teams = sh.team == 0 ? 1 : sh.threads / sh.team;
    const int64_t most = (rows + teams - 1) / teams;
    int64_t slots = static_cast<int64_t>(cu) * waves * kWave / sh.threads / groups;
    if (slots > most) slots = most;
    return static_cast<int>(slots < 1 ? 1 : slots);
}

constexpr int kFwdWaves = 80, kBwdWaves = 20;

template <typename F>
hipError_t with_shape(const Shape& sh, F f) {
    if (sh.team == 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (sh.team == 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    if (sh.runs == 1) return f(std::integral_constant<int, 0>(), std::integral_constant<int, 1>());
    return f(std::integral_constant<int, 0>(), std::integral_constant<int, 2>());
}

template <int IO, bool AL, int GATE>
hipError_t launch_gated(const GatedNormArgs& a, const Shape& sh, bool bwd, int slots, float* partial, hipStream_t s) {
    return with_shape(sh, [&](auto team, auto runs) {
        constexpr int TEAM = decltype(team)::value, CH = decltype(runs)::value;
        const dim3 grid(static_cast<unsigned>(slots * a.groups)), block(sh.threads);
        if (bwd)
            hipLaunchKernelGGL((gated_norm_bwd_kernel<IO, TEAM, CH, AL, GATE>), grid, block, 0, s, a, slots, partial);
        else
            hipLaunchKernelGGL((gated_norm_fwd_kernel<IO, TEAM, CH, AL, GATE>), grid, block, 0, s, a, slots);
        return hipGetLastError();
    });
}

template <int IO>
hipError_t launch_gated_io(const GatedNormArgs& a, const Shape& sh, bool bwd, int slots, float* partial,
                           hipStream_t s) {
    const bool al = a.dim / a.groups % 8 == 0 && a.x_stride % 8 == 0 && (a.gate == kGateNone || a.z_stride % 8 == 0);
    switch (a.gate * 2 + (al ? 1 : 0)) {
        case 0: return launch_gated<IO, false, kGateNone>(a, sh, bwd, slots, partial, s);
        case 1: return launch_gated<IO, true, kGateNone>(a, sh, bwd, slots, partial, s);
        case 2: return launch_gated<IO, false, kGateFirst>(a, sh, bwd, slots, partial, s);
        case 3: return launch_gated<IO, true, kGateFirst>(a, sh, bwd, slots, partial, s);
        case 4: return launch_gated<IO, false, kGateBehind>(a, sh, bwd, slots, partial, s);
        default: return launch_gated<IO, true, kGateBehind>(a, sh, bwd, slots, partial, s);
    }
}

hipError_t launch_gated_any(const GatedNormArgs& a, const Shape& sh, bool bwd, int slots, float* partial,
                            hipStream_t s) {
    return a.io == kIoF32 ? launch_gated_io<kIoF32>(a, sh, bwd, slots, partial, s)
                          : launch_gated_io<kIoBF16>(a, sh, bwd, slots, partial, s);
}

template <int IO, int RIO, bool AL>
hipError_t launch_residual(const ResidualNormArgs& a, const Shape& sh, bool bwd, int slots, float* partial,
                           hipStream_t s) {
    return with_shape(sh, [&](auto team, auto runs) {
        constexpr int TEAM = decltype(team)::value, CH = decltype(runs)::value;
        const dim3 grid(static_cast<unsigned>(slots)), block(sh.threads);
        if (!bwd)
            hipLaunchKernelGGL((residual_norm_fwd_kernel<IO, RIO, TEAM, CH, AL>), grid, block, 0, s, a, slots);
        else if (a.dscale != nullptr)
            hipLaunchKernelGGL((residual_norm_bwd_kernel<IO, RIO, TEAM, CH, AL, true>), grid, block, 0, s, a, slots,
                               partial);
        else
            hipLaunchKernelGGL((residual_norm_bwd_kernel<IO, RIO, TEAM, CH, AL, false>), grid, block, 0, s, a, slots,
                               partial);
        return hipGetLastError();
    });
}

hipError_t launch_residual_any(const ResidualNormArgs& a, const Shape& sh, bool bwd, int slots, float* partial,
                               hipStream_t s) {
    const bool al = a.dim % 8 == 0;
    if (a.io == kIoF32)
        return al ? launch_residual<kIoF32, kIoF32, true>(a, sh, bwd, slots, partial, s)
                  : launch_residual<kIoF32, kIoF32, false>(a, sh, bwd, slots, partial, s);
    if (a.total_io == kIoF32)
        return al ? launch_residual<kIoBF16, kIoF32, true>(a, sh, bwd, slots, partial, s)
                  : launch_residual<kIoBF16, kIoF32, false>(a, sh, bwd, slots, partial, s);
    return al ? launch_residual<kIoBF16, kIoBF16, true>(a, sh, bwd, slots, partial, s)
              : launch_residual<kIoBF16, kIoBF16, false>(a, sh, bwd, slots, partial, s);
}

hipError_t launch_columns(int64_t dim, int slots, const float* partial, float* out0, float* out1, hipStream_t s) {
    hipLaunchKernelGGL(norm_columns_kernel,
                       dim3(static_cast<unsigned>((dim + kWave - 1) / kWave), out1 != nullptr ? 2 : 1),
                       dim3(kColumnWaves * kWave), 0, s, dim, slots, partial, out0, out1);
    return hipGetLastError();
}

hipError_t launch_zero(int64_t dim, float* out0, float* out1, hipStream_t s) {
    hipLaunchKernelGGL(norm_zero_kernel, dim3(static_cast<unsigned>((dim + 255) / 256)), dim3(256), 0, s, dim, out0,
                       out1);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, int cu, hipStream_t s) {
    const Shape sh = shape_for(a.dim / a.groups);
    return launch_gated_any(a, sh, false, slots_for(a.rows, a.groups, sh, cu, kFwdWaves), nullptr, s);
}

size_t gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t groups, int cu) {
    const int slots = slots_for(rows, groups, shape_for(dim / groups), cu, kBwdWaves);
    return slots > 1 ? static_cast<size_t>(slots) * dim * sizeof(float) : 0;
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, int cu, void* ws, hipStream_t s) {
    if (a.rows == 0) return launch_zero(a.dim, a.dweight, nullptr, s);
    const Shape sh = shape_for(a.dim / a.groups);
    const int slots = slots_for(a.rows, a.groups, sh, cu, kBwdWaves);
    float* partial = static_cast<float*>(ws);
    const hipError_t e = launch_gated_any(a, sh, true, slots, partial, s);
    if (e != hipSuccess || slots == 1 || a.dweight == nullptr) return e;
    return launch_columns(a.dim, slots, partial, a.dweight, nullptr, s);
}

hipError_t launch_residual_norm_fwd(const ResidualNormArgs& a, int cu, hipStream_t s) {
    const Shape sh = shape_for(a.dim);
    return launch_residual_any(a, sh, false, slots_for(a.rows, 1, sh, cu, kFwdWaves), nullptr, s);
}

size_t residual_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int cu) {
    const int slots = slots_for(rows, 1, shape_for(dim), cu, kBwdWaves);
    return slots > 1 ? static_cast<size_t>(slots) * dim * 2 * sizeof(float) : 0;
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a, int cu, void* ws, hipStream_t s) {
    if (a.rows == 0) return launch_zero(a.dim, a.dweight, a.dscale, s);
    const Shape sh = shape_for(a.dim);
    const int slots = slots_for(a.rows, 1, sh, cu, kBwdWaves);
    float* partial = static_cast<float*>(ws);
    const hipError_t e = launch_residual_any(a, sh, true, slots, partial, s);
    if (e != hipSuccess || slots == 1 || (a.dweight == nullptr && a.dscale == nullptr)) return e;
    return launch_columns(a.dim, slots, partial, a.dweight, a.dscale, s);
}

}  // namespace mamba
