// The norms around a block and their gradients.
//   gated:     v = x silu(z) or x,  n = v rstd,  y = n w, times silu(z) where the gate is behind
//              u = dy w (silu(z)),  dv = rstd (u - n mean(u n)),  dw = sum over rows of dy n (silu(z))
//   residual:  total = residual + scale x,  n = total rstd,  y = n w
//              d = dtotal + rstd (dy w - n mean(dy w n)),  dresidual = d,  dx = scale d,
//              dscale = sum of d x,  dw = sum of dy n
//
// All are bound by memory: every tensor is read or written once. A lane holds 8
// consecutive values of a part (16 above 8192 of them), so that a part of n values
// takes as many lanes as it has eights - some of a wave's, or several waves' - and few
// registers; weights and the sums over rows stay in registers while a workgroup walks
// rows, with the next row's loads out. In bf16 on MI355X, 16384 x 5120: gated forward
// 90 us (5.6 TB/s), gradients 155 to 164 (5.1 to 5.4), with the residual sum in fp32
// 178 (5.6), its gradients 192 (5.2); a large copy reaches 4.9 to 5.6 by machine.
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

// A lane's CH runs of 8 values of a part of n: run u is the (lane + team u)-th.
// ALIGNED: n is a multiple of 8 and runs start on 16 bytes. Else the last run is
// the part's last 8 values, of which the first `skip` are the run's before it as
// well: both form and write the same, sums take them once. A run that the part has
// not is its last one again, with all skipped, and is not written. SHORT: a part
// may be of fewer than 8 values, which are taken one by one.
template <int CH, bool ALIGNED, bool SHORT>
struct Span {
    uint32_t at[CH];
    int skip[CH], n;

    __device__ __forceinline__ Span(int n_, int lane, int team) : n(n_) {
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            const int i = (lane + team * u) * 8, last = SHORT && n < 8 ? 0 : n - 8;
            at[u] = i < last ? i : last;
            skip[u] = i < n ? i - at[u] : 8;
        }
    }
    __device__ __forceinline__ bool mine(int u) const { return skip[u] < 8; }
    __device__ __forceinline__ bool counts(int i) const { return i % 8 >= skip[i / 8] && (!SHORT || i < n); }
    // What a value adds to a sum of the lane's.
    __device__ __forceinline__ float counted(int i, float v) const {
        if constexpr (ALIGNED) return CH == 1 || mine(i / 8) ? v : 0.0f;
        return i % 8 >= skip[i / 8] ? v : 0.0f;
    }
    // What of a sum of counted values is the lane's.
    __device__ __forceinline__ float lane_sum(float v) const { return !ALIGNED || CH > 1 || mine(0) ? v : 0.0f; }
};

// The values of a row's Span; `row` is the part's first.
template <int IO, int CH, bool ALIGNED, bool SHORT>
struct Cells {
    static constexpr int K = IO == kIoF32 ? 2 : 1;
    typedef Span<CH, ALIGNED, SHORT> S;
    u32x4 q[CH * K];

    __device__ __forceinline__ void load(const char* row, const S& span) {
#pragma unroll
        for (int u = 0; u < CH; ++u) load_run(u, row, span);
    }
    __device__ __forceinline__ void load_run(int u, const char* row, const S& span) {
        if (SHORT && span.n < 8) {
#pragma unroll
            for (int k = 0; k < K; ++k) q[u * K + k] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < span.n) {
                    const uint32_t r = load_raw<IO>(row, e);
                    if constexpr (IO == kIoF32) q[u * K + e / 4][e % 4] = r;
                    else q[u][e / 2] |= e % 2 ? r << 16 : r;
                }
            return;
        }
        const char* s = row + span.at[u] * static_cast<uint32_t>(size_of<IO>());
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (ALIGNED) q[u * K + k] = reinterpret_cast<const u32x4*>(s)[k];
            else q[u * K + k] = *reinterpret_cast<const u32x4_any*>(s + 16 * k);
        }
    }
    // The same values, which what follows does not know to be the same.
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int k = 0; k < CH * K; ++k) asm volatile("" : "+v"(q[k]));
    }
    __device__ __forceinline__ float get(int i) const {
        const int u = i / 8, e = i % 8;
        if constexpr (IO == kIoF32) return __uint_as_float(q[u * 2 + e / 4][e % 4]);
        const uint32_t r = q[u][e / 2];
        return __uint_as_float(e % 2 ? r & 0xffff0000u : r << 16);
    }
    static __device__ __forceinline__ void store_run(int u, char* row, const S& span, const float (&v)[8]) {
        if (!span.mine(u)) return;
        char* d = row + span.at[u] * static_cast<uint32_t>(size_of<IO>());
        if (SHORT && span.n < 8) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < span.n) store_io<IO>(d, e, v[e]);
            return;
        }
        u32x4 o[K];
#pragma unroll
        for (int e = 0; e < 8; e += IO == kIoF32 ? 1 : 2) {
            if constexpr (IO == kIoF32) {
                o[e / 4][e % 4] = __float_as_uint(v[e]);
            } else {
                const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[e]));
                const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[e + 1]));
                o[0][e / 2] = lo | hi << 16;
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (ALIGNED) reinterpret_cast<u32x4*>(d)[k] = o[k];
            else *reinterpret_cast<u32x4_any*>(d + 16 * k) = o[k];
        }
    }
};

// The first value of a row's part.
template <int IO>
__device__ __forceinline__ const char* part(const void* p, int64_t row, int64_t stride, int64_t first) {
    return static_cast<const char*>(p) + (row * stride + first) * size_of<IO>();
}
template <int IO>
__device__ __forceinline__ char* part(void* p, int64_t row, int64_t stride, int64_t first) {
    return static_cast<char*>(p) + (row * stride + first) * size_of<IO>();
}

// The parameters of a lane's values, ones where there are none. They stay in
// registers, but for lanes of two runs, which read them for every row (KEEP false), as
// a kernel of 1024 threads has 128 registers to a lane: the gradients take 88 to 128
// without them, the forward kernels 48 to 72.
template <int CH, bool AL, bool SHORT>
struct Params {
    static constexpr bool KEEP = CH == 1;
    Cells<kIoF32, CH, AL, SHORT> v;
    const char* p;

    __device__ __forceinline__ void read(int u, const Span<CH, AL, SHORT>& span) {
        v.q[2 * u] = v.q[2 * u + 1] = u32x4{0x3f800000, 0x3f800000, 0x3f800000, 0x3f800000};
        if (p != nullptr) v.load_run(u, p, span);
    }
    __device__ __forceinline__ Params(const float* all, int64_t first, const Span<CH, AL, SHORT>& span)
        : p(all == nullptr ? nullptr : part<kIoF32>(static_cast<const void*>(all), 0, 0, first)) {
        if constexpr (KEEP)
#pragma unroll
            for (int u = 0; u < CH; ++u) read(u, span);
    }
    // For a row's run u.
    __device__ __forceinline__ void get(int u, const Span<CH, AL, SHORT>& span) {
        if constexpr (!KEEP) {
            asm volatile("" : "+s"(p));   // not once for all rows
            read(u, span);
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return v.get(i); }
};

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}
// The sum over 8 lanes, in all of them, without a trip to LDS: with lanes 1 apart, 2
// apart, and the other four of eight; <0x140> adds the other eight of 16.
__device__ __forceinline__ float sum8(float v) {
    return dpp_add<0x141>(dpp_add<0x4e>(dpp_add<0xb1>(v)));
}
__device__ __forceinline__ float readlane(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// A workgroup's teams, each of which takes a row at a time: TEAM lanes each, or
// (kWhole) one of all its waves, or (kPacked) several of a multiple of 16 lanes up to
// 256, which a wave's bounds may cut. `red` holds a sum for each wave (packed: for
// each 16 lanes), twice, so that one barrier a row is enough: one half is written while
// others may still read the other. Waves that a workgroup has not count as zeros.
constexpr int kWhole = 0, kPacked = 1, kNormSums = kNormMaxWaves * kWave / 16;

// How many lanes a team has, how many teams stand side by side on groups of a row,
// and how many workgroups share a group's rows.
struct Layout {
    int lanes, across, slots;
};

// Most threads of a workgroup.
template <int TEAM>
constexpr int kThreads = TEAM == kWhole || TEAM == kPacked ? kNormMaxWaves * kWave : kNormThreads;

template <int TEAM>
struct Teams {
    static constexpr bool BARRIER = TEAM == kWhole || TEAM == kPacked;   // all teams take their sums together
    int lane, team, size, across, down;   // across * down teams: on groups, on rows
    int odd = 0;
    float (*red)[kNormSums];

    __device__ __forceinline__ Teams(float (*slots)[kNormSums], const Layout& lay) : red(slots) {
        size = TEAM == kWhole ? blockDim.x : TEAM == kPacked ? lay.lanes : TEAM;
        across = TEAM == kWhole ? 1 : lay.across;
        down = TEAM == kWhole ? 1 : blockDim.x / (size * across);
        team = TEAM == kWhole ? 0 : threadIdx.x / size;
        lane = threadIdx.x - team * size;
        if constexpr (TEAM == kWhole) {
            if (threadIdx.x < 2 * kNormMaxWaves) red[threadIdx.x / kNormMaxWaves][threadIdx.x % kNormMaxWaves] = 0.0f;
            __syncthreads();
        }
    }
    __device__ __forceinline__ float sum(float v) {
        v = sum8(v);
        if constexpr (TEAM == 8) return v;
        v = dpp_add<0x140>(v);
        if constexpr (TEAM == 32) v += __shfl_xor(v, 16);
        if constexpr (TEAM == 64 || TEAM == kWhole) {
            float s = readlane(v, 0);
#pragma unroll
            for (int r = 16; r < kWave; r += 16) s += readlane(v, r);
            v = s;
        }
        if constexpr (BARRIER) {
            constexpr int EACH = TEAM == kWhole ? kWave : 16;
            const int at = threadIdx.x % 16, sums = TEAM == kWhole ? kNormMaxWaves : size / 16;
            if (threadIdx.x % EACH == 0) red[odd][threadIdx.x / EACH] = v;
            __syncthreads();
            v = at < sums ? red[odd][team * sums + at] : 0.0f;
            v = dpp_add<0x140>(sum8(v));
            odd ^= 1;
        }
        return v;
    }
};

// Which rows a team takes: it stays with one group of columns and walks rows slot,
// slot + slots, ... times its workgroup's rows. Teams that take their sums together
// take the same number of turns; one without a row does nothing in its last.
template <int TEAM>
struct Walk {
    int64_t grp, row, step, rows, ends, slot;
    int at;   // the group's place in the workgroup

    __device__ __forceinline__ Walk(int64_t rows_, int64_t groups, const Layout& lay, const Teams<TEAM>& tm)
        : rows(rows_) {
        const int64_t blocks = groups / tm.across;
        const int down = tm.team / tm.across;
        at = tm.team - down * tm.across;
        slot = blockIdx.x / blocks;
        grp = (blockIdx.x - slot * blocks) * tm.across + at;
        row = slot * tm.down + down;
        step = static_cast<int64_t>(lay.slots) * tm.down;
        ends = TEAM == kPacked ? rows + down : rows;   // the workgroup's first row is one until then
    }
    __device__ __forceinline__ bool turn() const { return row < ends; }
    __device__ __forceinline__ bool has() const { return TEAM != kPacked || row < rows; }
    __device__ __forceinline__ bool more() const { return row + step < rows; }
};

// Sums over rows of a lane's columns: in registers, or for lanes of two runs in LDS
// (in registers 20 to 90 others would spill; with an fp32 stream, or with a scale in
// fp32, the residual gradients spill 4 to 17 all the same).
template <int CH>
struct Columns {
    float v[8];
    float4* lds;
    int size;

    template <typename T>
    __device__ __forceinline__ Columns(const T& tm, float4* all) : lds(all + threadIdx.x), size(tm.size) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        if constexpr (CH > 1)
            for (int u = 0; u < CH; ++u) close(u);
    }
    __device__ __forceinline__ void open(int u) {
        if constexpr (CH > 1) {
            const float4 a = lds[2 * u * size], b = lds[(2 * u + 1) * size];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
    }
    __device__ __forceinline__ void close(int u) {
        if constexpr (CH > 1) {
            lds[2 * u * size] = make_float4(v[0], v[1], v[2], v[3]);
            lds[(2 * u + 1) * size] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
    __device__ __forceinline__ float& operator[](int i) { return v[i % 8]; }
};

__device__ __forceinline__ float sigmoid(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

// Lanes of two runs load a row when they come to it, and take their runs one after the
// other. In the gradients a row ahead was slower (gated, 4000 x 16384 in bf16 167 us
// against 159); forward, where its registers would find room, it has not been tried.
template <int CH>
constexpr bool kAhead = CH == 1;

template <int CH>
__device__ __forceinline__ void end_run() {
    if constexpr (CH > 1) __builtin_amdgcn_sched_barrier(0);
}
#define MAMBA_NORM_TYPES                                        \
    constexpr int N = CH * 8;                                   \
    constexpr bool SHORT = TEAM == 8 && !AL;                    \
    typedef Span<CH, AL, SHORT> S;                              \
    typedef Cells<IO, CH, AL, SHORT> C;                         \
    typedef Params<CH, AL, SHORT> P

// One sum a row, of the squares: 16384 x 5120 in bf16 90 us, 80 parts of 64 a row 88.
template <int IO, int TEAM, int CH, bool AL, int GATE>
__global__ __launch_bounds__(kThreads<TEAM>) void gated_norm_fwd_kernel(GatedNormArgs a, Layout lay) {
    MAMBA_NORM_TYPES;
    __shared__ float red[2][kNormSums];
    Teams<TEAM> tm(red, lay);
    const int n = static_cast<int>(a.dim / a.groups);
    Walk<TEAM> walk(a.rows, a.groups, lay, tm);
    const S span(n, tm.lane, tm.size);
    const int64_t first = walk.grp * n;
    const float inv = 1.0f / static_cast<float>(n);
    P w(a.weight, first, span);
    C x, z;
    auto fetch = [&](int64_t row) {
        x.load(part<IO>(a.x, row, a.x_stride, first), span);
        if constexpr (GATE != kGateNone) z.load(part<IO>(a.z, row, a.z_stride, first), span);
    };
    if (kAhead<CH> && walk.row < a.rows) fetch(walk.row);
    for (; walk.turn(); walk.row += walk.step) {
        const int64_t row = walk.row;
        const bool has = walk.has();
        if (!kAhead<CH>) fetch(row);
        float v[N], g[N], sq = 0.0f;
        if (has)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = x.get(i);
            if constexpr (GATE != kGateNone) g[i] = z.get(i) * sigmoid(z.get(i));
            if constexpr (GATE == kGateFirst) v[i] *= g[i];
            sq = fmaf(span.counted(i, v[i]), v[i], sq);
        }
        if (kAhead<CH> && walk.more()) fetch(row + walk.step);
        const float rstd = 1.0f / sqrtf(fmaf(tm.sum(span.lane_sum(sq)), inv, a.eps));
        if (!has) continue;
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            w.get(u, span);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 8 * u + e;
                y[e] = v[i] * rstd * w[i];
                if constexpr (GATE == kGateBehind) y[e] *= g[i];
            }
            C::store_run(u, part<IO>(a.y, row, a.dim, first), span, y);
            end_run<CH>();
        }
        if (tm.lane == 0 && a.rstd != nullptr) a.rstd[row * a.groups + walk.grp] = rstd;
    }
}

// The column sums of a workgroup's teams, rows in order; out[i] is column i's.
template <int TEAM, int CH, typename S>
__device__ __forceinline__ void put_columns(const Teams<TEAM>& tm, const Walk<TEAM>& walk, const S& span, float* cols,
                                            float* out, Columns<CH>& d) {
    out += (walk.grp - walk.at) * span.n;
    if constexpr (TEAM == kWhole) {
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            d.open(u);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (span.counts(8 * u + e)) out[span.at[u] + e] = d[e];
        }
    } else {
        static_assert(CH == 1, "runs of a narrow part");
        const int all = tm.across * span.n;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (span.counts(i)) cols[tm.team / tm.across * all + walk.at * span.n + span.at[0] + i] = d[i];
        __syncthreads();
        for (int j = threadIdx.x; j < all; j += blockDim.x) {
            float t = 0.0f;
            for (int k = 0; k < tm.down; ++k) t += cols[k * all + j];
            out[j] = t;
        }
    }
}

// What the gradients of a value are made of: nm the normed value, up dy (and the
// gate), u up w, gx and gz what dx and dz take of dv (gz all of dz where the gate is
// behind).
template <int GATE>
struct GatedTerms {
    float nm, up, u, gx = 1.0f, gz = 0.0f;

    GatedTerms() = default;
    // Keeps what follows from forming them behind the sum, from more values.
    __device__ __forceinline__ void formed() {
        if constexpr (GATE != kGateNone) asm volatile("" : "+v"(nm), "+v"(u));
        if constexpr (GATE == kGateFirst) asm volatile("" : "+v"(gx));
        if constexpr (GATE != kGateNone) asm volatile("" : "+v"(gz));
    }
    __device__ __forceinline__ GatedTerms(float x, float z, float dy, float rs, float w) {
        float v = x;
        up = dy;
        if constexpr (GATE != kGateNone) {
            // sigmoid and 1 - sigmoid, each to its own accuracy. Far down the sigmoid is 0,
            // as forward: a z of the type's lowest value is what masks close a gate with,
            // and times 2^-126 it would still be -4.
            const float t = -z * kLog2e, e = fast_exp2(t);
            const float sg = fast_rcp(1.0f + e), rest = t > 126.0f ? 1.0f : e * sg;
            const float sl = z * sg, dsl = sg * fmaf(z, rest, 1.0f);
            if constexpr (GATE == kGateFirst) {
                v = x * sl;
                gx = sl;
                gz = x * dsl;
            } else {
                gz = up * dsl * w;
                up *= sl;
            }
        }
        nm = v * rs;
        if constexpr (GATE == kGateBehind) gz *= nm;
        u = up * w;
    }
};

// One sum a row, of u n; rstd comes from the forward pass. The terms behind the sum
// are formed before it and kept (asm statements hold them in place: left alone, the
// compiler moves their forming behind the sum, where it takes more registers and half
// the workgroups find room). 16384 x 5120 in bf16: gate behind 155 us, gate first in 8
// groups 164; 4000 x 16384 159 (with its column sums in registers, spilling, 709).
template <int IO, int TEAM, int CH, bool AL, int GATE>
__global__ __launch_bounds__(kThreads<TEAM>) void gated_norm_bwd_kernel(GatedNormArgs a, Layout lay,
                                                                             float* partial) {
    MAMBA_NORM_TYPES;
    __shared__ float red[2][kNormSums];
    __shared__ float cols[TEAM == kWhole ? 1 : 8 * kThreads<TEAM>];
    extern __shared__ float4 sums[];
    Teams<TEAM> tm(red, lay);
    const int n = static_cast<int>(a.dim / a.groups);
    Walk<TEAM> walk(a.rows, a.groups, lay, tm);
    const S span(n, tm.lane, tm.size);
    const int64_t first = walk.grp * n;
    const float inv = 1.0f / static_cast<float>(n);
    P w(a.weight, first, span);
    Columns<CH> dw(tm, sums);
    C x, z, dy;
    float rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        x.load(part<IO>(a.x, row, a.x_stride, first), span);
        if constexpr (GATE != kGateNone) z.load(part<IO>(a.z, row, a.z_stride, first), span);
        dy.load(part<IO>(a.dy, row, a.dim, first), span);
        rstd = a.rstd[row * a.groups + walk.grp];
    };
    if (kAhead<CH> && walk.row < a.rows) fetch(walk.row);
    for (; walk.turn(); walk.row += walk.step) {
        const int64_t row = walk.row;
        const bool has = walk.has();
        if (!kAhead<CH>) fetch(row);
        GatedTerms<GATE> k[N];
        const float rs = rstd;
        auto form = [&](int i) {
            k[i] = GatedTerms<GATE>(x.get(i), GATE != kGateNone ? z.get(i) : 0.0f, dy.get(i), rs, w[i]);
        };
        float s = 0.0f;
        if (has)
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            w.get(u, span);
            dw.open(u);
#pragma unroll
            for (int i = 8 * u; i < 8 * u + 8; ++i) {
                form(i);
                dw[i] = fmaf(k[i].up, k[i].nm, dw[i]);
                s = fmaf(span.counted(i, k[i].u), k[i].nm, s);
                if constexpr (kAhead<CH>) k[i].formed();
            }
            dw.close(u);
            end_run<CH>();
        }
        if (kAhead<CH> && walk.more()) fetch(row + walk.step);
        const float c = tm.sum(span.lane_sum(s)) * inv;
        if (!has) continue;
        if constexpr (!kAhead<CH>) {   // the terms are formed again
            x.again();
            z.again();
            dy.again();
        }
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            w.get(u, span);
            float ox[8], oz[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 8 * u + e;
                if constexpr (!kAhead<CH>) form(i);
                const float dv = rs * fmaf(-k[i].nm, c, k[i].u);
                ox[e] = dv * k[i].gx;
                oz[e] = GATE == kGateFirst ? k[i].gz * dv : k[i].gz;
            }
            C::store_run(u, part<IO>(a.dx, row, a.dim, first), span, ox);
            if constexpr (GATE != kGateNone) C::store_run(u, part<IO>(a.dz, row, a.dim, first), span, oz);
            end_run<CH>();
        }
    }
    if (a.dweight == nullptr) return;
    float* out = lay.slots == 1 ? a.dweight : partial + walk.slot * a.dim;
    put_columns<TEAM, CH>(tm, walk, span, cols, out, dw);
}

// As the gated norm, of the sum before its rounding: 16384 x 5120 in bf16 with an fp32
// stream 178 us.
template <int IO, int RIO, int TEAM, int CH, bool AL>
__global__ __launch_bounds__(kThreads<TEAM>) void residual_norm_fwd_kernel(ResidualNormArgs a, Layout lay) {
    MAMBA_NORM_TYPES;
    typedef Cells<RIO, CH, AL, SHORT> R;
    __shared__ float red[2][kNormSums];
    Teams<TEAM> tm(red, lay);
    const int n = static_cast<int>(a.dim);
    Walk<TEAM> walk(a.rows, 1, lay, tm);
    const S span(n, tm.lane, tm.size);
    const float inv = 1.0f / static_cast<float>(n);
    P w(a.weight, 0, span), sc(a.scale, 0, span);
    C x;
    R res;
    auto fetch = [&](int64_t row) {
        x.load(part<IO>(a.x, row, a.dim, 0), span);
        res.load(part<RIO>(a.residual, row, a.dim, 0), span);
    };
    if (kAhead<CH> && walk.row < a.rows) fetch(walk.row);
    for (; walk.turn(); walk.row += walk.step) {
        const int64_t row = walk.row;
        const bool has = walk.has();
        if (!kAhead<CH>) fetch(row);
        float v[N], sq = 0.0f;
        if (has)
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            sc.get(u, span);
#pragma unroll
            for (int i = 8 * u; i < 8 * u + 8; ++i) {
                v[i] = fmaf(sc[i], x.get(i), res.get(i));
                sq = fmaf(span.counted(i, v[i]), v[i], sq);
            }
            end_run<CH>();
        }
        if (kAhead<CH> && walk.more()) fetch(row + walk.step);
        // Stores come behind the sum, which waits for every lane's loads: total may be
        // the residual, and a run's second holder reads what the first one writes.
        const float rstd = 1.0f / sqrtf(fmaf(tm.sum(span.lane_sum(sq)), inv, a.eps));
        if (!has) continue;
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            w.get(u, span);
            float t[8], y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[e] = v[8 * u + e];
                y[e] = t[e] * rstd * w[8 * u + e];
            }
            R::store_run(u, part<RIO>(a.total, row, a.dim, 0), span, t);
            C::store_run(u, part<IO>(a.y, row, a.dim, 0), span, y);
            end_run<CH>();
        }
        if (tm.lane == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    }
}

// SCALE: x is read and dscale formed. What is read behind the sum is loaded behind the
// row before, which leaves no second copy of it in registers: 16384 x 5120 in bf16 192
// us, with an fp32 stream 279; 4000 x 16384 186 and 285, in fp32 2000 x 16384 185 (4.2
// TB/s); 1000 x 1531 in fp32 18.
template <int IO, int RIO, int TEAM, int CH, bool AL, bool SCALE>
__global__ __launch_bounds__(kThreads<TEAM>) void residual_norm_bwd_kernel(ResidualNormArgs a, Layout lay,
                                                                                float* partial) {
    MAMBA_NORM_TYPES;
    typedef Cells<RIO, CH, AL, SHORT> R;
    __shared__ float red[2][kNormSums];
    __shared__ float cols[TEAM == kWhole ? 1 : 8 * kThreads<TEAM>];
    extern __shared__ float4 sums[];
    Teams<TEAM> tm(red, lay);
    const int n = static_cast<int>(a.dim);
    Walk<TEAM> walk(a.rows, 1, lay, tm);
    const S span(n, tm.lane, tm.size);
    const float inv = 1.0f / static_cast<float>(n);
    P w(a.weight, 0, span), sc(a.scale, 0, span);
    Columns<CH> dw(tm, sums), ds(tm, sums + (SCALE ? 2 * CH * tm.size : 0));
    R total, dt;
    C x, dy;
    float rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        total.load(part<RIO>(a.total, row, a.dim, 0), span);
        dy.load(part<IO>(a.dy, row, a.dim, 0), span);
        rstd = a.rstd[row];
    };
    auto fetch_rest = [&](int64_t row) {   // what is read behind the sum
        if (a.dtotal != nullptr) dt.load(part<RIO>(a.dtotal, row, a.dim, 0), span);
        if constexpr (SCALE) x.load(part<IO>(a.x, row, a.dim, 0), span);
    };
    if (a.dtotal == nullptr)
#pragma unroll
        for (int k = 0; k < R::K * CH; ++k) dt.q[k] = u32x4{0, 0, 0, 0};
    if (kAhead<CH> && walk.row < a.rows) {
        fetch(walk.row);
        fetch_rest(walk.row);
    }
    for (; walk.turn(); walk.row += walk.step) {
        const int64_t row = walk.row;
        const bool has = walk.has();
        if (!kAhead<CH>) fetch(row);
        float nm[N], g[N], s = 0.0f;
        const float rs = rstd;
        auto form = [&](int i) {
            nm[i] = total.get(i) * rs;
            g[i] = dy.get(i) * w[i];
        };
        if (has)
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            w.get(u, span);
            dw.open(u);
#pragma unroll
            for (int i = 8 * u; i < 8 * u + 8; ++i) {
                form(i);
                dw[i] = fmaf(dy.get(i), nm[i], dw[i]);
                s = fmaf(span.counted(i, g[i]), nm[i], s);
            }
            dw.close(u);
            end_run<CH>();
        }
        const bool more = walk.more();
        if (!kAhead<CH>) fetch_rest(row);
        else if (more) fetch(row + walk.step);
        const float c = tm.sum(span.lane_sum(s)) * inv;
        if (!has) continue;
        if constexpr (!kAhead<CH>) {   // the terms are formed again
            total.again();
            dy.again();
        }
#pragma unroll
        for (int u = 0; u < CH; ++u) {
            if constexpr (!kAhead<CH>) w.get(u, span);
            sc.get(u, span);
            if constexpr (SCALE) ds.open(u);
            float od[8], ox[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 8 * u + e;
                if constexpr (!kAhead<CH>) form(i);
                od[e] = fmaf(rs, fmaf(-nm[i], c, g[i]), dt.get(i));
                ox[e] = od[e] * sc[i];
                if constexpr (SCALE) ds[i] = fmaf(od[e], x.get(i), ds[i]);
            }
            if constexpr (SCALE) ds.close(u);
            R::store_run(u, part<RIO>(a.dresidual, row, a.dim, 0), span, od);
            if (a.dx != nullptr) C::store_run(u, part<IO>(a.dx, row, a.dim, 0), span, ox);
            end_run<CH>();
        }
        if (kAhead<CH> && more) fetch_rest(row + walk.step);
    }
    float* out = partial + walk.slot * a.dim;
    const bool one = lay.slots == 1;
    if (a.dweight != nullptr) put_columns<TEAM, CH>(tm, walk, span, cols, one ? a.dweight : out, dw);
    if constexpr (SCALE)
        put_columns<TEAM, CH>(tm, walk, span, cols, one ? a.dscale : out + lay.slots * a.dim, ds);
}

#undef MAMBA_NORM_TYPES

// Column sums over the slots, in 64 bits and a fixed order: 16 columns per
// workgroup, whose 64 rows of 16 lanes take every 64th slot, 8 loads in flight.
// (64 columns by 16: a quarter of the workgroups, and 4 times the turns.) Plane y
// of `partial` goes to out[y].
constexpr int kColumns = 16, kColumnThreads = 1024;

__global__ __launch_bounds__(kColumnThreads) void column_sums_kernel(int64_t dim, int64_t slots, const float* partial,
                                                                      float* out0, float* out1) {
    constexpr int ROWS = kColumnThreads / kColumns, WAVES = kColumnThreads / kWave, U = 8;
    __shared__ double red[WAVES][kColumns];
    const int c = threadIdx.x % kColumns, r = threadIdx.x / kColumns;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kColumns + c;
    float* out = blockIdx.y ? out1 : out0;
    if (out == nullptr) return;
    const float* p = partial + blockIdx.y * slots * dim;
    double s = 0.0;
    if (col < dim) {
        for (int64_t k0 = r; k0 < slots; k0 += U * ROWS) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t k = k0 + u * ROWS;
                x[u] = k < slots ? p[k * dim + col] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) s += static_cast<double>(x[u]);
        }
    }
    s += __shfl_xor(s, kColumns);
    s += __shfl_xor(s, 2 * kColumns);
    if (threadIdx.x % kWave < kColumns) red[threadIdx.x / kWave][c] = s;
    __syncthreads();
    if (r == 0 && col < dim) {
        double t = 0.0;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) t += red[k][c];
        out[col] = static_cast<float>(t);
    }
}

__global__ __launch_bounds__(256) void norm_zero_kernel(int64_t dim, float* out0, float* out1) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= dim) return;
    if (out0 != nullptr) out0[i] = 0.0f;
    if (out1 != nullptr) out1[i] = 0.0f;
}

// How teams are held for parts of n values, their lanes, runs of 8 values to a lane
// and threads of a workgroup. Parts of 513 to 2048 values whose lanes do not fill their
// waves are packed, forward up to 1024 of them (16384 x 4 parts: of 640 gradients
// 85 us against 109 as whole waves, forward 46 against 51; of 1152 144 against 172,
// forward 85 against 82).
struct Shape {
    int team, lanes, runs, threads;
};

constexpr Shape shape_for(int64_t n, bool bwd) {
    if (n <= 512) {
        const int lanes = n <= 64 ? 8 : n <= 128 ? 16 : n <= 256 ? 32 : 64;
        return {lanes, lanes, 1, kNormThreads};
    }
    if (n <= (bwd ? 2048 : 1024)) {
        const int lanes = static_cast<int>((n + 127) / 128) * 16;
        if (lanes % kWave) return {kPacked, lanes, 1, lanes * (lanes % 32 ? 4 : 2)};   // whole waves
    }
    const int runs = n <= 8 * kWave * kNormMaxWaves ? 1 : 2;
    const int threads = static_cast<int>((n + 8 * kWave * runs - 1) / (8 * kWave * runs)) * kWave;
    return {kWhole, threads, runs, threads};
}

static_assert(shape_for(kGatedNormMaxDim, true).threads <= kNormMaxWaves * kWave, "the widest part has a workgroup");

constexpr int kFwdWaves = 320, kBwdWaves = 8;   // to a compute unit, at least
constexpr int64_t kSumRows = 1024;              // rows of a sum in fp32, at most

// Teams stand on so many groups side by side as divide both. Workgroups for a group:
// forward about 320 waves to a compute unit (16384 rows of 5120: 91 us, of 80 waves 99;
// 2048 x 80 parts of 64 118 and 126); backward 8 (16384 x 2048 71 us, of 16 75, of 4
// 85; 16384 x 5120 155 and of 16 167), as fewer rows at once are read in longer
// stretches and every workgroup leaves its columns' sums; no more than a quarter of
// the rows have one (1000 x 1531 in fp32 18 us, a workgroup each 23; 3000 x 1024 22 and
// 25), unless compute units would have none (243 x 12400 37 us, a quarter 40; 8 x 14966
// in fp32 27 and 43). A team adds up its rows in fp32, no more than 1024 of them: their
// roundings come to 2^-14 of the terms at worst, and what is above, over workgroups, is
// summed in 64 bits (262144 rows of 521 groups of 8 were 8192 each, off by 1.2e-4 where
// rows are alike, and took 17.1 ms, now 1.6e-5 and 12.4). Fewer would have more
// workgroups at once than the memory likes: 524288 x 2048 2.2 ms, 256 rows each 2.5.
Layout layout_for(int64_t rows, int64_t groups, const Shape& sh, int cu, bool bwd) {
    const int teams = sh.threads / sh.lanes;
    int across = 1;
    while (across * 2 <= teams && teams % (across * 2) == 0 && groups % (across * 2) == 0) across *= 2;
    const int64_t down = teams / across, most = (rows + down - 1) / down;
    const int64_t each = ((bwd ? kBwdWaves : kFwdWaves) * kWave + sh.threads - 1) / sh.threads;
    const int64_t blocks = groups / across, few = (cu + blocks - 1) / blocks;
    int64_t slots = each * cu / blocks;
    if (bwd && slots > most / 4) slots = most / 4 > few ? most / 4 : few;
    if (slots > most) slots = most;
    const int64_t least = (most + kSumRows - 1) / kSumRows;
    if (bwd && slots < least) slots = least;
    return {sh.lanes, across, static_cast<int>(slots < 1 ? 1 : slots)};
}

// LDS for the column sums of lanes of two runs: at most 2 * 64 KB, of which a
// workgroup of 16 waves can have all.
unsigned columns_bytes(const Shape& sh, int sums) {
    return sh.runs > 1 ? static_cast<unsigned>(sums * sh.runs * 8 * sh.threads * sizeof(float)) : 0;
}

template <typename F>
hipError_t with_shape(const Shape& sh, F f) {
    if (sh.team == 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    if (sh.team == 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (sh.team == 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
    if (sh.team == 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    if (sh.team == kPacked) return f(std::integral_constant<int, kPacked>(), std::integral_constant<int, 1>());
    if (sh.runs == 1) return f(std::integral_constant<int, kWhole>(), std::integral_constant<int, 1>());
    return f(std::integral_constant<int, kWhole>(), std::integral_constant<int, 2>());
}

template <int IO, bool AL, int GATE>
hipError_t launch_gated(const GatedNormArgs& a, const Shape& sh, bool bwd, const Layout& lay, float* partial,
                        hipStream_t s) {
    return with_shape(sh, [&](auto team, auto runs) {
        constexpr int TEAM = decltype(team)::value, CH = decltype(runs)::value;
        const dim3 grid(static_cast<unsigned>(lay.slots * (a.groups / lay.across))), block(sh.threads);
        if (bwd)
            hipLaunchKernelGGL((gated_norm_bwd_kernel<IO, TEAM, CH, AL, GATE>), grid, block, columns_bytes(sh, 1), s, a,
                               lay, partial);
        else
            hipLaunchKernelGGL((gated_norm_fwd_kernel<IO, TEAM, CH, AL, GATE>), grid, block, 0, s, a, lay);
        return hipGetLastError();
    });
}

template <int IO>
hipError_t launch_gated_io(const GatedNormArgs& a, const Shape& sh, bool bwd, const Layout& lay, float* partial,
                           hipStream_t s) {
    const bool al = a.dim / a.groups % 8 == 0 && a.x_stride % 8 == 0 && (a.gate == kGateNone || a.z_stride % 8 == 0);
    switch (a.gate * 2 + (al ? 1 : 0)) {
        case 0: return launch_gated<IO, false, kGateNone>(a, sh, bwd, lay, partial, s);
        case 1: return launch_gated<IO, true, kGateNone>(a, sh, bwd, lay, partial, s);
        case 2: return launch_gated<IO, false, kGateFirst>(a, sh, bwd, lay, partial, s);
        case 3: return launch_gated<IO, true, kGateFirst>(a, sh, bwd, lay, partial, s);
        case 4: return launch_gated<IO, false, kGateBehind>(a, sh, bwd, lay, partial, s);
        default: return launch_gated<IO, true, kGateBehind>(a, sh, bwd, lay, partial, s);
    }
}

hipError_t launch_gated_any(const GatedNormArgs& a, const Shape& sh, bool bwd, const Layout& lay, float* partial,
                            hipStream_t s) {
    return a.io == kIoF32 ? launch_gated_io<kIoF32>(a, sh, bwd, lay, partial, s)
                          : launch_gated_io<kIoBF16>(a, sh, bwd, lay, partial, s);
}

template <int IO, int RIO, bool AL>
hipError_t launch_residual(const ResidualNormArgs& a, const Shape& sh, bool bwd, const Layout& lay, float* partial,
                           hipStream_t s) {
    return with_shape(sh, [&](auto team, auto runs) {
        constexpr int TEAM = decltype(team)::value, CH = decltype(runs)::value;
        const dim3 grid(static_cast<unsigned>(lay.slots)), block(sh.threads);
        if (!bwd)
            hipLaunchKernelGGL((residual_norm_fwd_kernel<IO, RIO, TEAM, CH, AL>), grid, block, 0, s, a, lay);
        else if (a.dscale != nullptr)
            hipLaunchKernelGGL((residual_norm_bwd_kernel<IO, RIO, TEAM, CH, AL, true>), grid, block,
                               columns_bytes(sh, 2), s, a, lay, partial);
        else
            hipLaunchKernelGGL((residual_norm_bwd_kernel<IO, RIO, TEAM, CH, AL, false>), grid, block,
                               columns_bytes(sh, 1), s, a, lay, partial);
        return hipGetLastError();
    });
}

hipError_t launch_residual_any(const ResidualNormArgs& a, const Shape& sh, bool bwd, const Layout& lay, float* partial,
                               hipStream_t s) {
    const bool al = a.dim % 8 == 0;
    if (a.io == kIoF32)
        return al ? launch_residual<kIoF32, kIoF32, true>(a, sh, bwd, lay, partial, s)
                  : launch_residual<kIoF32, kIoF32, false>(a, sh, bwd, lay, partial, s);
    if (a.total_io == kIoF32)
        return al ? launch_residual<kIoBF16, kIoF32, true>(a, sh, bwd, lay, partial, s)
                  : launch_residual<kIoBF16, kIoF32, false>(a, sh, bwd, lay, partial, s);
    return al ? launch_residual<kIoBF16, kIoBF16, true>(a, sh, bwd, lay, partial, s)
              : launch_residual<kIoBF16, kIoBF16, false>(a, sh, bwd, lay, partial, s);
}

hipError_t launch_zero(int64_t dim, float* out0, float* out1, hipStream_t s) {
    hipLaunchKernelGGL(norm_zero_kernel, dim3(static_cast<unsigned>((dim + 255) / 256)), dim3(256), 0, s, dim, out0,
                       out1);
    return hipGetLastError();
}

}  // namespace

// (2^26 columns, more than a launch's threads count, have one slot in all tensors that
// fit the memory.)
hipError_t launch_column_sums(int64_t dim, int64_t slots, const float* partial, float* out0, float* out1,
                              hipStream_t s) {
    hipLaunchKernelGGL(column_sums_kernel,
                       dim3(static_cast<unsigned>((dim + kColumns - 1) / kColumns), out1 != nullptr ? 2 : 1),
                       dim3(kColumnThreads), 0, s, dim, slots, partial, out0, out1);
    return hipGetLastError();
}

hipError_t launch_gated_norm_fwd(const GatedNormArgs& a, int cu, hipStream_t s) {
    const Shape sh = shape_for(a.dim / a.groups, false);
    return launch_gated_any(a, sh, false, layout_for(a.rows, a.groups, sh, cu, false), nullptr, s);
}

size_t gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t groups, int cu) {
    const int slots = layout_for(rows, groups, shape_for(dim / groups, true), cu, true).slots;
    return slots > 1 ? static_cast<size_t>(slots) * dim * sizeof(float) : 0;
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, int cu, void* ws, hipStream_t s) {
    if (a.rows == 0) return launch_zero(a.dim, a.dweight, nullptr, s);
    const Shape sh = shape_for(a.dim / a.groups, true);
    const Layout lay = layout_for(a.rows, a.groups, sh, cu, true);
    float* partial = static_cast<float*>(ws);
    const hipError_t e = launch_gated_any(a, sh, true, lay, partial, s);
    if (e != hipSuccess || lay.slots == 1 || a.dweight == nullptr) return e;
    return launch_column_sums(a.dim, lay.slots, partial, a.dweight, nullptr, s);
}

hipError_t launch_residual_norm_fwd(const ResidualNormArgs& a, int cu, hipStream_t s) {
    const Shape sh = shape_for(a.dim, false);
    return launch_residual_any(a, sh, false, layout_for(a.rows, 1, sh, cu, false), nullptr, s);
}

size_t residual_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int cu) {
    const int slots = layout_for(rows, 1, shape_for(dim, true), cu, true).slots;
    return slots > 1 ? static_cast<size_t>(slots) * dim * 2 * sizeof(float) : 0;
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a, int cu, void* ws, hipStream_t s) {
    if (a.rows == 0) return launch_zero(a.dim, a.dweight, a.dscale, s);
    const Shape sh = shape_for(a.dim, true);
    const Layout lay = layout_for(a.rows, 1, sh, cu, true);
    float* partial = static_cast<float*>(ws);
    const hipError_t e = launch_residual_any(a, sh, true, lay, partial, s);
    if (e != hipSuccess || lay.slots == 1 || (a.dweight == nullptr && a.dscale == nullptr)) return e;
    return launch_column_sums(a.dim, lay.slots, partial, a.dweight, a.dscale, s);
}

}  // namespace mamba
