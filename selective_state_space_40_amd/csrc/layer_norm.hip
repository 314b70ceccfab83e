// Layer norm over each of the `groups` equal parts of a row, and its
// gradients:
//     xh = (x - mean) rstd,  y = xh w + b
//     dx = rstd (w dy - mean(w dy) - xh mean(w dy xh))
//     dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both are bound by memory: one read of x (and dy), one write of y (dx). A
// part of n = dim / groups values is held by a team of 16 to 1024 lanes, 8 to 32
// values per lane in registers, so the mean, the centred sum of squares and the
// output take one pass over memory; the variance is the mean square of the
// centred values, not a difference of sums. 16384 x 5120 in
// bf16: 66 us forward (5.1 TB/s), 109 us backward (4.6 TB/s with the sums of the
// parameters' gradients, 105 for its main kernel and 4 for the columns'), where a
// large copy reaches 5.5 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "internal.h"

namespace mamba {
namespace {

// Sum over the lanes of a team; `slot` is LDS for one value per wave and
// value, and the team spans whole waves when it is wider than one.
template <int TEAM, int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float* slot) {
    constexpr int LANES = TEAM < kWave ? TEAM : kWave;
#pragma unroll
    for (int m = 1; m < LANES; m *= 2)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], m);
    if constexpr (TEAM > kWave) {
        constexpr int W = TEAM / kWave;
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) slot[wave * NV + i] = v[i];
        }
        __syncthreads();
        const float* t = slot + wave / W * W * NV;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int u = 0; u < W; ++u) s += t[u * NV + i];
            v[i] = s;
        }
    }
}

// A lane's CH x 8 values of a part of n. With VEC a lane holds runs of 8
// consecutive values (the part is then a multiple of 8 values and starts on
// 16 bytes); otherwise single values TEAM apart, for odd widths, which an access
// of 2 or 4 bytes a lane holds to a fraction of the memory's rate (gradients in
// bf16: 2665 x 15734 203 us, 46 by its bytes; in fp32: 2000 x 5001 34 us, 22 by
// them).
template <int IO, int TEAM, int CH, bool VEC>
struct Part {
    static constexpr int kWords = VEC ? (IO == kIoF32 ? 2 : 1) : 0;
    uint4 q[VEC ? CH * kWords : 1];
    uint32_t r[VEC ? 1 : CH * 8];

    static __device__ __forceinline__ int index(int lane, int u, int e) {
        return VEC ? (lane + TEAM * u) * 8 + e : lane + TEAM * (8 * u + e);
    }
    __device__ __forceinline__ void load(const void* p, int64_t at, int n, int lane) {
        if constexpr (VEC) {
            const char* base = static_cast<const char*>(p) + at * (IO == kIoF32 ? 4 : 2);
#pragma unroll
            for (int u = 0; u < CH; ++u) {
                const bool in = (lane + TEAM * u) * 8 < n;
#pragma unroll
                for (int k = 0; k < kWords; ++k)
                    q[u * kWords + k] = in ? reinterpret_cast<const uint4*>(base)[(lane + TEAM * u) * kWords + k]
                                           : make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int u = 0; u < CH; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = index(lane, u, e);
                    r[u * 8 + e] = i < n ? load_raw<IO>(p, at + i) : 0u;
                }
        }
    }
    __device__ __forceinline__ float get(int u, int e) const {
        if constexpr (VEC && IO == kIoF32) {
            const uint4& t = q[u * 2 + e / 4];
            return __uint_as_float(e % 4 == 0 ? t.x : e % 4 == 1 ? t.y : e % 4 == 2 ? t.z : t.w);
        } else if constexpr (VEC) {
            const uint4& t = q[u];
            const uint32_t x = e / 2 == 0 ? t.x : e / 2 == 1 ? t.y : e / 2 == 2 ? t.z : t.w;
            return __uint_as_float(e % 2 ? x & 0xffff0000u : x << 16);
        } else {
            return raw_to_f32<IO>(r[u * 8 + e]);
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, int n, int lane,
                                                 const float (&v)[CH * 8]) {
        if constexpr (VEC) {
            char* base = static_cast<char*>(p) + at * (IO == kIoF32 ? 4 : 2);
#pragma unroll
            for (int u = 0; u < CH; ++u) {
                if ((lane + TEAM * u) * 8 >= n) continue;
                const float* s = v + 8 * u;
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (IO == kIoF32) {
                        o[e] = __float_as_uint(s[e]);
                    } else {
                        const uint32_t h = __builtin_bit_cast(uint16_t, static_cast<__bf16>(s[e]));
                        if (e % 2) o[e / 2] |= h << 16;
                        else o[e / 2] = h;
                    }
                }
                uint4* d = reinterpret_cast<uint4*>(base) + (lane + TEAM * u) * kWords;
                d[0] = make_uint4(o[0], o[1], o[2], o[3]);
                if constexpr (IO == kIoF32) d[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < CH; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = index(lane, u, e);
                    if (i < n) store_io<IO>(p, at + i, v[u * 8 + e]);
                }
        }
    }
};

// The parameters of a lane's values.
template <int TEAM, int CH, bool VEC>
__device__ __forceinline__ void load_params(const float* p, int64_t at, int n, int lane, float none,
                                            float (&v)[CH * 8]) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) v[i] = none;
        return;
    }
    Part<kIoF32, TEAM, CH, VEC> t;
    t.load(p, at, n, lane);
#pragma unroll
    for (int u = 0; u < CH; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u * 8 + e] = t.get(u, e);
}

// The forward pass. A workgroup stays with one group of columns, keeps its
// weights in registers and walks rows slot, slot + slots, ... (times its teams),
// the next row's loads out while one is normed: read per row, the weights'
// fp32 values were twice a bf16 row's bytes from the L2 (16384 x 5120: 78 us
// against 66).
template <int IO, int TEAM, int CH, bool VEC>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void layer_norm_fwd_kernel(NormArgs a, int slots) {
    constexpr int THREADS = TEAM > 256 ? TEAM : 256;
    constexpr int TEAMS = THREADS / TEAM;
    __shared__ float slot_sums[2][THREADS / kWave];
    typedef Part<IO, TEAM, CH, VEC> P;
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const int n = static_cast<int>(a.dim / a.groups);
    const int64_t grp = blockIdx.x % a.groups;
    const int64_t slot = blockIdx.x / a.groups;
    const float inv = 1.0f / static_cast<float>(n);
    float wt[CH * 8], bs[CH * 8];
    load_params<TEAM, CH, VEC>(a.weight, grp * n, n, lane, 1.0f, wt);
    load_params<TEAM, CH, VEC>(a.bias, grp * n, n, lane, 0.0f, bs);
    const int64_t step = static_cast<int64_t>(slots) * TEAMS;
    P x;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.rows;
        x.load(a.x, in ? (row * a.groups + grp) * n : 0, in ? n : 0, lane);
    };
    fetch(slot * TEAMS + team);
    // every team of the workgroup takes the same number of turns
    for (int64_t r0 = slot * TEAMS; r0 < a.rows; r0 += step) {
        const int64_t row = r0 + team;
        float v[CH * 8];
        float sum[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < CH; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[u * 8 + e] = x.get(u, e);
                sum[0] += v[u * 8 + e];
            }
        fetch(row + step);
        team_sum<TEAM>(sum, slot_sums[0]);
        const float mean = sum[0] * inv;
        float sq[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < CH; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float& t = v[u * 8 + e];
                t = P::index(lane, u, e) < n ? t - mean : 0.0f;
                sq[0] = fmaf(t, t, sq[0]);
            }
        team_sum<TEAM>(sq, slot_sums[1]);
        const float rstd = 1.0f / sqrtf(sq[0] * inv + a.eps);
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) v[i] = fmaf(v[i] * rstd, wt[i], bs[i]);
        const int64_t part = row * a.groups + grp;
        const bool in = row < a.rows;
        P::store(a.y, in ? part * n : 0, in ? n : 0, lane, v);
        if (in && lane == 0) {
            if (a.mean != nullptr) a.mean[part] = mean;
            if (a.rstd != nullptr) a.rstd[part] = rstd;
        }
    }
}

// The backward pass. A workgroup stays with one group of columns and walks
// rows blockrow, blockrow + slots, ...: its lanes keep their columns' sums of
// dw and db in registers, its teams' sums meet in LDS at the end, and one
// (slot, column) pair per workgroup goes to `partial` (2, slots, dim), from
// which layer_norm_columns_kernel adds the slots in order.
// The widest parts take teams of 1024 lanes, whose 128 registers hold neither the
// next row's loads nor a row's products: those are formed again after the sums,
// and of the columns' sums 20 to 24 values are spilled all the same (bf16, 2665 x 15734: 203 us, 523 with 512 lanes of 32 values, spilled; of
// 12288 values that 512 lanes hold as 24 each: 48 us against 69).
constexpr int kNormBwdThreads = 512;

template <int IO, int TEAM, int CH, bool VEC>
__global__ __launch_bounds__(TEAM > kNormBwdThreads ? TEAM : kNormBwdThreads) void layer_norm_bwd_kernel(
    NormArgs a, int slots, float* partial) {
    constexpr bool kLean = TEAM > kNormBwdThreads;
    __shared__ float red[2][2 * (kLean ? TEAM : kNormBwdThreads) / kWave];
    __shared__ float cols[TEAM > 256 ? 1 : CH * 8 * kNormBwdThreads];
    typedef Part<IO, TEAM, CH, VEC> P;
    const int lane = threadIdx.x % TEAM;
    const int team = threadIdx.x / TEAM, teams = blockDim.x / TEAM;
    const int n = static_cast<int>(a.dim / a.groups);
    const int64_t grp = blockIdx.x % a.groups;
    const int64_t slot = blockIdx.x / a.groups;
    const float inv = 1.0f / static_cast<float>(n);
    float wt[CH * 8], dw[CH * 8], db[CH * 8];
    load_params<TEAM, CH, VEC>(a.weight, grp * n, n, lane, 1.0f, wt);
#pragma unroll
    for (int i = 0; i < CH * 8; ++i) dw[i] = db[i] = 0.0f;
    const int64_t step = static_cast<int64_t>(slots) * teams;
    P x, dy;
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool in = row < a.rows;
        const int64_t part = in ? row * a.groups + grp : 0;
        x.load(a.x, part * n, in ? n : 0, lane);
        dy.load(a.dy, part * n, in ? n : 0, lane);
        mean = in ? a.mean[part] : 0.0f;
        rstd = in ? a.rstd[part] : 0.0f;
    };
    int odd = 0;
    if constexpr (!kLean) fetch(slot * teams + team);
    // every team of the workgroup takes the same number of turns
    for (int64_t r0 = slot * teams; r0 < a.rows; r0 += step) {
        const int64_t row = r0 + team;
        if constexpr (kLean) fetch(row);
        float xh[CH * 8], wdy[CH * 8];
        float s[2] = {0.0f, 0.0f};
        const float mu = mean, rs = rstd;
#pragma unroll
        for (int u = 0; u < CH; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = u * 8 + e;
                xh[i] = P::index(lane, u, e) < n ? (x.get(u, e) - mu) * rs : 0.0f;
                const float d = dy.get(u, e);
                wdy[i] = d * wt[i];
                dw[i] = fmaf(d, xh[i], dw[i]);
                db[i] += d;
                s[0] += wdy[i];
                s[1] = fmaf(wdy[i], xh[i], s[1]);
            }
        if constexpr (!kLean) fetch(row + step);
        team_sum<TEAM>(s, red[odd]);
        odd ^= 1;   // the other buffer: a wave may still read this one
        const float c1 = s[0] * inv, c2 = s[1] * inv;
        if constexpr (kLean) {
            // values that the compiler cannot tell from new ones, lest it keep
            // the row's products
            float mu_again = mu;
            asm volatile("" : "+v"(mu_again));
#pragma unroll
            for (int u = 0; u < CH; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = u * 8 + e;
                    const float again = (x.get(u, e) - mu_again) * rs;
                    wdy[i] = rs * (fmaf(dy.get(u, e), wt[i], -c1) - again * c2);
                }
        } else {
#pragma unroll
            for (int i = 0; i < CH * 8; ++i) wdy[i] = rs * (wdy[i] - c1 - xh[i] * c2);
        }
        P::store(a.dx, (row < a.rows ? row * a.groups + grp : 0) * n, row < a.rows ? n : 0, lane, wdy);
    }
    if (a.dweight == nullptr && a.dbias == nullptr) return;
    float* pw = partial + slot * a.dim + grp * n;
    float* pb = pw + static_cast<int64_t>(slots) * a.dim;
    if (slots == 1) {
        pw = a.dweight + grp * n;
        pb = a.dbias + grp * n;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float (&d)[CH * 8] = which ? db : dw;
        const bool wanted = (which ? a.dbias : a.dweight) != nullptr;
        float* out = which ? pb : pw;
        if constexpr (TEAM <= 256) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < CH * 8; ++i) cols[(team * CH * 8 + i) * TEAM + lane] = d[i];
            __syncthreads();
            for (int j = threadIdx.x; j < TEAM * CH * 8; j += blockDim.x) {
                float t = 0.0f;
                for (int k = 0; k < teams; ++k) t += cols[k * CH * 8 * TEAM + j];
                const int i = P::index(j % TEAM, j / TEAM / 8, j / TEAM % 8);
                if (wanted && i < n) out[i] = t;
            }
        } else {
#pragma unroll
            for (int u = 0; u < CH; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = P::index(lane, u, e);
                    if (wanted && i < n) out[i] = d[u * 8 + e];
                }
        }
    }
}

// Column sums over the slots: 64 columns per workgroup, its 16 waves a
// sixteenth of the slots each, 4 loads in flight.
constexpr int kColumnWaves = 16;

__global__ __launch_bounds__(kColumnWaves * kWave) void layer_norm_columns_kernel(int64_t dim, int slots,
                                                                                  const float* partial,
                                                                                  float* dweight, float* dbias) {
    __shared__ float red[kColumnWaves][kWave];
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kWave + lane;
    float* out = blockIdx.y ? dbias : dweight;
    if (out == nullptr) return;
    const float* p = partial + static_cast<int64_t>(blockIdx.y) * slots * dim;
    float s = 0.0f;
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
            for (int u = 0; u < U; ++u) s += x[u];
        }
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && col < dim) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < kColumnWaves; ++k) t += red[k][lane];
        out[col] = t;
    }
}

__global__ __launch_bounds__(256) void layer_norm_zero_kernel(int64_t dim, float* dweight, float* dbias) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= dim) return;
    if (dweight != nullptr) dweight[i] = 0.0f;
    if (dbias != nullptr) dbias[i] = 0.0f;
}

// Lanes and 8-value runs per lane for parts of n values. Between 1024 and 1536
// values a wave with 24 values a lane moves most, but four waves end sooner where
// fewer parts than the chip has units leave it idle: up to one part for each where
// lanes load 16 bytes, up to four where they load value by value, 24 loads to a
// lane. In bf16, four waves against one, forward and gradients:
//     200 x 1280   3.3 us against 3.6,   8.0 against 8.3
//     400 x 1280   3.5 against 3.7,      9.3 against 8.5
//     1000 x 1280  4.3 against 3.9,      10.7 against 9.5
//     400 x 1300   4.4 against 6.1,      10.0 against 11.6
//     1000 x 1300  5.4 against 6.3,      12.0 against 12.5
//     2000 x 1300  7.9 against 7.0,      14.8 against 14.3
// (1032 to 1536 and 1030 to 1531 alike, fp32 within 0.5 us of that). A wave with
// 16 values a lane or fewer is never behind by more than 0.3 us (1000 x 760: 3.4
// us against 4.1, gradients 7.9 against 10.0).
constexpr int64_t kFewParts = 256, kFewOddParts = 4 * kFewParts;

struct Team {
    int lanes, runs;
};

// The backward pass, which holds more per value, takes more lanes for the widest
// parts, sooner for those that are loaded value by value (fp32, 2000 x 5001: 34
// us with 512 lanes, 47 with 256).
constexpr Team team_for(int64_t n, int64_t parts, bool bwd) {
    const int64_t wave = parts < (n % 8 == 0 ? kFewParts : kFewOddParts) ? 1024 : 1536;
    int lanes = n <= 384 ? 16 : (n <= wave ? 64 : (n <= 6144 ? 256 : 512));
    if (bwd && n > 4096 && n % 8 != 0) lanes = 512;
    if (bwd && n > (n % 8 == 0 ? 12288 : 8192)) lanes = 1024;
    return {lanes, static_cast<int>((n + 8 * lanes - 1) / (8 * lanes))};
}

// Which teams' kernels are built: those that team_for gives for some part.
constexpr bool norm_built(int lanes, int runs, bool vec, bool bwd) {
    if (lanes == 16 || lanes == 64) return runs <= 3;
    if (!bwd) return lanes == 256 ? runs <= 3 : lanes == 512 && runs >= 2 && runs <= 4;
    if (lanes == 1024) return runs == 2;
    return (lanes == 256 || lanes == 512) && (runs <= 2 || (vec && runs == 3));
}

// Parts of 8 k and of 8 k - 1 values stand for all: every bound in team_for is a
// multiple of 8.
constexpr bool teams_are_built() {
    for (int64_t n = 8; n <= kNormMaxDim; n += 8)
        for (int few = 0; few < 2; ++few)
            for (int bwd = 0; bwd < 2; ++bwd) {
                const int64_t parts = few ? 1 : int64_t(1) << 30;
                const Team v = team_for(n, parts, bwd), o = team_for(n - 1, parts, bwd);
                if (!norm_built(v.lanes, v.runs, true, bwd) || !norm_built(o.lanes, o.runs, false, bwd)) return false;
            }
    return true;
}
static_assert(teams_are_built(), "a kernel for every part");

// Workgroups of the forward pass, when there are rows for them: several rounds
// of what the chip holds, so that the last one's idle part is small.
constexpr int kFwdWorkgroups = 4096;

// Threads per workgroup of the backward pass and slots (workgroups per group
// of columns): one workgroup of 512 per compute unit when there are rows enough.
// More, smaller ones leave more partial sums than they save time (2000 x 1024 in
// bf16: 9.9 us, with workgroups of 256, two to a unit, 13.4; 500 x 5120: 19 against
// 28), but for teams of 16, of which few parts fill few workgroups (500 x 384: 7.3
// us against 7.9; 2000 x 384 7.9 against 8.2, 4000 x 128 7.1 against 6.6), unless one
// of 512 holds all rows and writes the sums itself (32 x 16 parts of 128: 4.1 us
// against 5.6).
struct BwdGrid {
    int threads, slots;
};

BwdGrid bwd_grid(int64_t rows, int64_t groups, int lanes, int cu) {
    int threads = kNormBwdThreads;
    const bool one_holds_all = rows > 256 / 16 && rows <= kNormBwdThreads / 16;   // and a smaller one does not
    if (lanes == 16 && !one_holds_all && rows * groups < 2048) threads = 256;
    if (threads < lanes) threads = lanes;
    const int64_t teams = threads / lanes;
    const int64_t most = (rows + teams - 1) / teams;
    const int64_t per_cu = threads < kNormBwdThreads ? kNormBwdThreads / threads : 1;
    int64_t slots = (per_cu * cu + groups - 1) / groups;
    if (slots > most) slots = most;
    return {threads, static_cast<int>(slots < 1 ? 1 : slots)};
}

template <int IO, int TEAM, int CH, bool VEC>
hipError_t launch_norm(const NormArgs& a, bool bwd, int threads, int slots, float* partial, hipStream_t s) {
    if (!norm_built(TEAM, CH, VEC, bwd)) return hipErrorInvalidValue;
    if (!bwd) {
        if constexpr (norm_built(TEAM, CH, VEC, false)) {
            constexpr int TEAMS = (TEAM > 256 ? TEAM : 256) / TEAM;
            const int64_t most = (a.rows + TEAMS - 1) / TEAMS;
            const int turns = kFwdWorkgroups / static_cast<int>(a.groups < kFwdWorkgroups ? a.groups : kFwdWorkgroups);
            const int row_slots = static_cast<int>(most < turns ? most : turns);
            hipLaunchKernelGGL((layer_norm_fwd_kernel<IO, TEAM, CH, VEC>),
                               dim3(static_cast<unsigned>(row_slots * a.groups)), dim3(TEAM > 256 ? TEAM : 256), 0,
                               s, a, row_slots);
        }
    } else if constexpr (norm_built(TEAM, CH, VEC, true)) {
        hipLaunchKernelGGL((layer_norm_bwd_kernel<IO, TEAM, CH, VEC>),
                           dim3(static_cast<unsigned>(slots * a.groups)), dim3(threads), 0, s, a, slots, partial);
    }
    return hipGetLastError();
}

template <int IO, bool VEC>
hipError_t launch_norm_team(const NormArgs& a, Team t, bool bwd, int threads, int slots, float* partial,
                            hipStream_t s) {
    switch (t.lanes * 8 + t.runs) {
        case 16 * 8 + 1: return launch_norm<IO, 16, 1, VEC>(a, bwd, threads, slots, partial, s);
        case 16 * 8 + 2: return launch_norm<IO, 16, 2, VEC>(a, bwd, threads, slots, partial, s);
        case 16 * 8 + 3: return launch_norm<IO, 16, 3, VEC>(a, bwd, threads, slots, partial, s);
        case 64 * 8 + 1: return launch_norm<IO, 64, 1, VEC>(a, bwd, threads, slots, partial, s);
        case 64 * 8 + 2: return launch_norm<IO, 64, 2, VEC>(a, bwd, threads, slots, partial, s);
        case 64 * 8 + 3: return launch_norm<IO, 64, 3, VEC>(a, bwd, threads, slots, partial, s);
        case 256 * 8 + 1: return launch_norm<IO, 256, 1, VEC>(a, bwd, threads, slots, partial, s);
        case 256 * 8 + 2: return launch_norm<IO, 256, 2, VEC>(a, bwd, threads, slots, partial, s);
        case 256 * 8 + 3: return launch_norm<IO, 256, 3, VEC>(a, bwd, threads, slots, partial, s);
        case 512 * 8 + 2: return launch_norm<IO, 512, 2, VEC>(a, bwd, threads, slots, partial, s);
        case 512 * 8 + 3: return launch_norm<IO, 512, 3, VEC>(a, bwd, threads, slots, partial, s);
        case 512 * 8 + 4: return launch_norm<IO, 512, 4, VEC>(a, bwd, threads, slots, partial, s);
        case 1024 * 8 + 2: return launch_norm<IO, 1024, 2, VEC>(a, bwd, threads, slots, partial, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_norm_any(const NormArgs& a, bool bwd, int threads, int slots, float* partial, hipStream_t s) {
    const int64_t n = a.dim / a.groups;
    const Team t = team_for(n, a.rows * a.groups, bwd);
    const bool vec = n % 8 == 0;
    if (a.io == kIoF32)
        return vec ? launch_norm_team<kIoF32, true>(a, t, bwd, threads, slots, partial, s)
                   : launch_norm_team<kIoF32, false>(a, t, bwd, threads, slots, partial, s);
    return vec ? launch_norm_team<kIoBF16, true>(a, t, bwd, threads, slots, partial, s)
               : launch_norm_team<kIoBF16, false>(a, t, bwd, threads, slots, partial, s);
}

}  // namespace

hipError_t launch_layer_norm_fwd(const NormArgs& a, hipStream_t s) {
    return launch_norm_any(a, false, 0, 0, nullptr, s);
}

size_t layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t groups, int cu) {
    if (rows == 0 || dim == 0) return 0;
    const BwdGrid g = bwd_grid(rows, groups, team_for(dim / groups, rows * groups, true).lanes, cu);
    return g.slots > 1 ? static_cast<size_t>(g.slots) * dim * 2 * sizeof(float) : 0;
}

hipError_t launch_layer_norm_bwd(const NormArgs& a, int cu, void* ws, hipStream_t s) {
    if (a.rows == 0) {
        hipLaunchKernelGGL(layer_norm_zero_kernel, dim3(static_cast<unsigned>((a.dim + 255) / 256)), dim3(256),
                           0, s, a.dim, a.dweight, a.dbias);
        return hipGetLastError();
    }
    const BwdGrid g = bwd_grid(a.rows, a.groups, team_for(a.dim / a.groups, a.rows * a.groups, true).lanes, cu);
    float* partial = static_cast<float*>(ws);
    const hipError_t e = launch_norm_any(a, true, g.threads, g.slots, partial, s);
    if (e != hipSuccess || g.slots == 1 || (a.dweight == nullptr && a.dbias == nullptr)) return e;
    hipLaunchKernelGGL(layer_norm_columns_kernel, dim3(static_cast<unsigned>((a.dim + kWave - 1) / kWave), 2),
                       dim3(kColumnWaves * kWave), 0, s, a.dim, g.slots, partial, a.dweight, a.dbias);
    return hipGetLastError();
}

}  // namespace mamba
