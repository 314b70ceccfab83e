// Linear attention with a decay for each head, chunk by chunk on the matrix
// cores. One kernel serves the forward pass and the three products of the
// backward pass: each is a pass (q, k, v) -> out over a sequence,
//     out_i = sum_{j <= i} lam^(i-j) (q_i . k_j) v_j  +  decayed state,
// with an fp32 state S (sum of k_j^T v_j, decayed) carried from chunk to
// chunk. For a chunk of C tokens entered with state S, local tokens i, j:
//     P[i,j]  = scale lam^(i-j) (q_i . k_j)  for j <= i, else 0     (C x C)
//     out_i   = sum_j P[i,j] v_j + out_scale lam^(i+1-r) q_i S
//     S      <- lam^cnt S + sum_j state_scale lam^(cnt-1-j+r) k_j^T v_j
// r is 0 for the forward direction. The backward products of k and v run
// through time from the end (token order reversed as rows are loaded) and
// carry the adjoint of the state, which token i reads before its own decay
// and not after it: r is 1 there.
//     forward    (q, k, v) -> o,   state S
//     gradients  (do, v, k) -> dq, state S^T
//                (k, q, do) -> dv, adjoint dS, reversed
//                (v, do, q) -> dk, adjoint dS^T, reversed
//
// Work mapping. A workgroup walks the chunks of one (row, head, segment) for
// 64 output columns, 16 to a wave. The state's columns belong to the same wave,
// so its S (all DC rows, 16 columns) stays in the accumulators for the whole
// walk, and the accumulator of two 16 x 16 blocks is, up to a fixed order of
// the rows, the operand of the product q S: the state passes through neither
// LDS nor another wave. Of heads wider than 128 two waves share 16 columns, each
// with half of S's rows; they form q S for all of a chunk's tokens and exchange
// halves, so that each goes on with half of the tokens. The chunk's q, k and v
// rows are staged in LDS; the next chunk's are loaded into registers meanwhile.
// The C x C matrix P is split over the waves by 16 x 16 blocks and exchanged
// through LDS.
//
// bf16 operands. q, k and v enter the products exactly. P is rounded to bf16
// (its effect on a bf16 output is that of the output's own rounding). What
// reaches fp32 results goes in as a sum of bf16 terms, each the rounding of
// what the ones before leave: three (2^-25 of a term at most) for a state that
// leaves in fp32 and for the gradient of the decay, two (2^-17) for a state
// that only bf16 outputs see, and one for the product q S that they see
// directly. fp32 I/O uses the fp32 matrix instruction and no rounding.
//
// The gradient of the log decay is formed in the pass of dq, with the state's
// derivative T = dS/d(log lam) as a second state:
//     T_i = lam^(i+1) (T + (i+1) S) + sum_{j <= i} (i-j) lam^(i-j) k_j^T v_j
//     dlog_decay = sum_i scale do_i . (q_i T_i) + <adjoint at the end, T_end>
// where the sum over j <= i of one chunk is taken pair by pair, from P. Every
// pair of tokens enters once, with its own number of steps, so nothing
// cancels; a second way, sums of token places against q . dq and k . dk,
// needs no T but cancels down from a window's length to a memory's, and was 6
// to 10 times less exact with windows of 1024 tokens. T starts at zero in every
// segment, whose end's adjoint carries its steps on.
//
// What bounds it. A prompt of 8 x 2048 x 16 heads of 128 in bf16 takes 75 us
// against 50 for its bytes at the rate of a large copy. It is a workgroup per
// compute unit: each SIMD has one wave, whose steps (staging, q k^T and q S, P,
// the state, P v) wait for each other at two barriers a chunk, with the matrix
// cores 25% busy, the vector units 26% and LDS 31%. Cutting it into segments
// for a second workgroup costs the states' pass more than the waiting (103 us).
// The gradients (255 us, 87 by their bytes) hold two workgroups on a unit:
// matrix cores 33%, vector units 41% busy, much of it the terms' splitting.
// fp32 takes the exact fp32 instruction (137 TFLOP/s in a large product, bf16
// 1196) and forms P for every 64 columns and every pass anew: 2 x 2048 x 8 heads of
// 200 x 168 in 131 us forward and 466 with gradients, 32 and 80 by their operations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "internal.h"

namespace mamba {
namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8;
typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4;
typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;
typedef short s16x4 __attribute__((ext_vector_type(4)));

struct F32x8 {
    float v[8];
};

// A fragment holds, in lane (c, g) = (lane % 16, lane / 16), the values 8 g + e
// (e < 8) of the 32 that one row or column c of an operand contributes to a
// product. The fp32 instruction contracts 4 values at a time, value e of the
// four lane groups in step e.
template <int IO>
struct LinOps;

template <>
struct LinOps<kIoBF16> {
    typedef __bf16 T;
    typedef bf16x8 Frag;
    static constexpr bool kSplit = true;    // fp32 values enter as bf16 terms
    static constexpr int kChunk = kLinChunkBF16;
    // LDS row padding (elements). Cycles of a CU per wave's read, measured:
    // whole fragments of 16 rows (nat) 4 with 32 bytes, 8 with 16 or 64, 32
    // without; the transpose read 4 with any, 8 with columns 8 apart and 32
    // bytes, 4 with those and 64. P's rows, written 8 bytes a lane and read
    // whole, take 8 and 8 with 16 bytes, 16 and 4 with 32.
    static constexpr int kPad = 16, kPadK = 32, kPadP = 8;

    static __device__ __forceinline__ Frag nat(const T* row, int g) {
        return *reinterpret_cast<const bf16x8*>(row + 8 * g);
    }
    // 8 rows r0 + 8 g + e of column c0 + c of a row-major tile: the LDS
    // transpose read (ds_read_b64_tr_b16). Within each group of 16 lanes,
    // lane r receives as element e the element (r mod 4) of the 8 bytes that
    // lane 4 e + r / 4 of its group addresses, so lane s of the group
    // addresses row s / 4, columns 4 (s mod 4) .. + 3 of a 4 x 16 block; with
    // STEP 8 the four groups of 4 columns are 8 apart.
    template <int RS, int STEP>
    static __device__ __forceinline__ Frag tr(const T* tile, int r0, int c0, int c, int g) {
        const T* p = tile + (r0 + 8 * g + (c >> 2)) * RS + c0 + STEP * (c & 3);
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(const_cast<T*>(p)));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(const_cast<T*>(p + 4 * RS)));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 acc) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
    }
    static __device__ __forceinline__ float get(const Frag& f, int e) {
        return static_cast<float>(f[e]);
    }
    // The next term of fp32 values: x rounded, and x becomes what is left.
    static __device__ __forceinline__ Frag term(float (&x)[8]) {
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            // one conversion for both, and its halves taken as fp32 again
            const bf16x2 p = {static_cast<__bf16>(x[e]), static_cast<__bf16>(x[e + 1])};
            f[e / 2] = __builtin_bit_cast(uint32_t, p);
            x[e] -= __uint_as_float(f[e / 2] << 16);
            x[e + 1] -= __uint_as_float(f[e / 2] & 0xffff0000u);
        }
        return __builtin_bit_cast(Frag, f);
    }
    // four consecutive elements as fp32
    static __device__ __forceinline__ f32x4 ld4(const T* p) {
        const bf16x4 a = *reinterpret_cast<const bf16x4*>(p);
        return f32x4{static_cast<float>(a[0]), static_cast<float>(a[1]), static_cast<float>(a[2]),
                     static_cast<float>(a[3])};
    }
    static __device__ __forceinline__ void st4(T* p, f32x4 v) {
        bf16x4 a;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = static_cast<__bf16>(v[e]);
        *reinterpret_cast<bf16x4*>(p) = a;
    }
};

template <>
struct LinOps<kIoF32> {
    typedef float T;
    typedef F32x8 Frag;
    static constexpr bool kSplit = false;
    static constexpr int kChunk = kLinChunkF32;
    static constexpr int kPad = 4, kPadK = 4, kPadP = 4;

    static __device__ __forceinline__ Frag pair(const float* a, const float* b) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(a), y = *reinterpret_cast<const f32x4*>(b);
        return F32x8{{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
    }
    static __device__ __forceinline__ Frag nat(const T* row, int g) {
        return pair(row + 8 * g, row + 8 * g + 4);
    }
    template <int RS, int STEP>
    static __device__ __forceinline__ Frag tr(const T* tile, int r0, int c0, int c, int g) {
        Frag f;
        const T* p = tile + (r0 + 8 * g) * RS + c0 + STEP * (c >> 2) + (c & 3);
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = p[e * RS];
        return f;
    }
    static __device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 acc) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], acc, 0, 0, 0);
        return acc;
    }
    static __device__ __forceinline__ float get(const Frag& f, int e) { return f.v[e]; }
    static __device__ __forceinline__ Frag term(float (&x)[8]) {
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = x[e];
        return f;
    }
    static __device__ __forceinline__ f32x4 ld4(const T* p) {
        return *reinterpret_cast<const f32x4*>(p);
    }
    static __device__ __forceinline__ void st4(T* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
};

// Buffer resource over `bytes` bytes from p (raw addressing, gfx9 word 3):
// loads at or past the end return zeros and stores there are dropped, so
// neither ragged chunks nor narrow heads need a branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lin_rsrc(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
// The most bytes of a chunk's rows, and an offset past the end of every resource
// that stays past it a chunk's rows on or, walked backwards, back, inside an int.
constexpr int kChunkBytes = kLinChunkBF16 * kLinMaxHeads * kLinMaxDim * 4;
constexpr int kPastEnd = 1 << 30;
static_assert(kPastEnd - kChunkBytes >= kChunkBytes && kPastEnd + kChunkBytes > kPastEnd, "past the end both ways");

// One head's rows of a (batch, seqlen, heads, dim) tensor from a segment's
// first token on. A chunk's resource ends with its last valid token, so rows
// past it (and, walked backwards, rows before the chunk's first, whose
// offsets are negative) need no test.
struct HeadRows {
    const char* base;
    int stride;   // bytes from token to token
    int width;    // bytes of a row

    __device__ __forceinline__ HeadRows(const void* p, int64_t row0, int heads, int head, int dim, int size)
        : base(static_cast<const char*>(p) + (row0 * heads + head) * dim * size),
          stride(heads * dim * size), width(dim * size) {}
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk(int64_t first, int cnt) const {
        return lin_rsrc(base + first * stride, cnt > 0 ? (cnt - 1) * stride + width : 0);
    }
};

// One tile's share of a thread: COUNT vectors of 16 bytes in the same column,
// ROWS rows apart.
template <int IO, int THREADS, int COLS, int PAD>
struct Tile {
    typedef typename LinOps<IO>::T T;
    static constexpr int kC = LinOps<IO>::kChunk;
    static constexpr int kRow = COLS + PAD;   // LDS row pitch
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int VPR = COLS / kVec;
    static constexpr int ROWS = THREADS / VPR;
    static constexpr int COUNT = kC / ROWS;
    static_assert(THREADS % VPR == 0 && kC % ROWS == 0, "whole vectors per thread");

    uint4 r[COUNT];

    // This thread's offset from a chunk's first token (walked backwards: from
    // its last), columns col0 on.
    static __device__ __forceinline__ int offset(const HeadRows& h, int tid, int col0, bool rev) {
        const int i = tid / VPR, col = (col0 + tid % VPR * kVec) * static_cast<int>(sizeof(T));
        return col < h.width ? (rev ? -i : i) * h.stride + col : kPastEnd;
    }
    __device__ __forceinline__ void load(const HeadRows& h, int off, int64_t first, int cnt, bool rev) {
        const __amdgpu_buffer_rsrc_t rs = h.chunk(first, cnt);
        const int start = rev ? (cnt - 1) * h.stride : 0, step = (rev ? -ROWS : ROWS) * h.stride;
#pragma unroll
        for (int u = 0; u < COUNT; ++u)
            r[u] = __builtin_bit_cast(
                uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, off + (start + u * step), 0, 0));
    }
    __device__ __forceinline__ void stage(T* lds, int tid) const {
        T* p = lds + tid / VPR * kRow + tid % VPR * kVec;
#pragma unroll
        for (int u = 0; u < COUNT; ++u) *reinterpret_cast<uint4*>(p + u * ROWS * kRow) = r[u];
    }
};

template <int IO, int DC, int MODE>
struct LinLds {
    static constexpr int WAVES = lin_waves(DC);
    typedef typename LinOps<IO>::T T;
    static constexpr int kC = LinOps<IO>::kChunk;
    static constexpr int kRowP = kC + LinOps<IO>::kPadP;
    static constexpr int kThreads = WAVES * kWave, kCols = kLinBlock;
    static constexpr int kSplit = lin_split(DC);
    typedef Tile<IO, kThreads, DC, LinOps<IO>::kPadK> TileK;
    typedef Tile<IO, kThreads, kCols, LinOps<IO>::kPad> TileV;
    typedef Tile<IO, kThreads, DC, LinOps<IO>::kPad> TileQ;
    typedef Tile<IO, kThreads, kCols, LinOps<IO>::kPad> TileX;
    alignas(16) T K[kC * TileK::kRow];
    alignas(16) T V[kC * TileV::kRow];
    alignas(16) T Q[MODE == kLinState ? 8 : kC * TileQ::kRow];
    alignas(16) T X[MODE == kLinBwd ? kC * TileX::kRow : 8];
    alignas(16) T P[MODE == kLinState ? 8 : kC * kRowP];
    // half of q S, 16 x 16 blocks as the accumulators hold them
    alignas(16) f32x4 half[kSplit > 1 && MODE != kLinState ? WAVES * (kC / 32) * kWave : 1];
    alignas(16) float W[kC];      // weight of token j in the state update
    float pow[kC + 1];            // lam^n
    float fac[MODE == kLinBwd ? 2 * kC : 1];   // P's factor n tokens apart at n + C: zero for n < 0
    double red[WAVES];
};

// lam^n = exp(g n), the product's rounding error put back.
__device__ __forceinline__ float decay_power(float g, int n) {
    if (n == 0) return 1.0f;   // also for g = -inf, a head that forgets at once
    const float p = g * static_cast<float>(n);
    const float e = fmaf(g, static_cast<float>(n), -p);
    const float x = expf(p);
    return (x > 0.0f && x < __builtin_inff()) ? fmaf(x, e, x) : x;
}

// A value that all lanes hold, moved to a scalar register.
__device__ __forceinline__ float uniform(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// The first of the 4 state rows that lane group g holds in block nt.
__device__ __forceinline__ int state_row(int nt, int g) { return 32 * (nt >> 1) + 8 * g + 4 * (nt & 1); }

// xcd_contiguous_block in 32 bits.
__device__ __forceinline__ uint32_t xcd_order(uint32_t bid, uint32_t nblocks) {
    constexpr uint32_t X = kXcds;
    const uint32_t q = nblocks / X, r = nblocks % X, xcd = bid % X, k = bid / X;
    return xcd * q + (xcd < r ? xcd : r) + k;
}

// One workgroup's walk: column block blk of pass ip over segment seg of (row,
// head) bh. ALT: bf16: the state enters with three terms; fp32: blocks of 32
// state rows past the head's width are left out. DG: the pass also forms the
// decay's gradient. FAST: half of a state or less survives a chunk.
template <int IO, int DC, int MODE, bool ALT, bool DG, bool FAST>
__device__ __forceinline__ void linear_attn_walk(const LinArgs& a, LinLds<IO, DC, MODE>& lds, const int ip,
                                                 const int blk, int seg, const int64_t bh, const int64_t b,
                                                 const int hd) {
    typedef LinOps<IO> O;
    typedef typename O::T T;
    typedef typename O::Frag Frag;
    constexpr int C = O::kChunk;
    constexpr int NT = C / 16;            // blocks of 16 tokens
    constexpr int NS = C / 32;            // product steps over tokens
    constexpr int WAVES = lin_waves(DC);
    constexpr int SPLIT = lin_split(DC);
    constexpr int NN = DC / SPLIT / 16;   // a wave's blocks of 16 state rows
    constexpr int OT = NT / SPLIT;        // and of 16 tokens of the output
    constexpr int DOB = kLinBlock;   // columns per workgroup
    constexpr int THREADS = WAVES * kWave;
    constexpr bool kState = MODE == kLinState, kBwd = MODE == kLinBwd;
    constexpr bool EXACT = O::kSplit && ALT, SKIP = !O::kSplit && ALT;
    typedef LinLds<IO, DC, MODE> Lds;
    constexpr int RK = Lds::TileK::kRow, RV = Lds::TileV::kRow, RQ = Lds::TileQ::kRow, RX = Lds::TileX::kRow;
    // each form's own thread index: derived from one, a thread's places would be
    // worked out in front of the branch between the forms and held from there
    // (gradients of 4 x 4096 x 24 heads of 32 x 64 in fp32: 388 us against 422; of
    // 8 x 2048 x 32 heads of 64 in bf16: 200 against 208)
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid) : "n"(FAST));
    const int lane = tid & (kWave - 1);
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int c = lane & 15, g = lane >> 4;
    // this wave's columns of the block, and its part of the state's rows
    const int wc = SPLIT > 1 ? w % (WAVES / SPLIT) : w, part = SPLIT > 1 ? w / (WAVES / SPLIT) : 0;
    const int n0w = part * (DC / SPLIT);

    const LinPass& ps = a.pass[ip];
    const bool rev = ps.rev != 0;
    if (kState && rev) seg += 1;   // the reversed walk's last segment is the first
    // where the state goes at the end: to the join of the segments (kLinState)
    // or to the caller
    float* sout = nullptr;
    if (kState) sout = ps.seg_in;
    else if (seg == (rev ? 0 : a.nseg - 1)) sout = ps.s_out;
    const int p0 = blk * DOB;
    const int dc = ps.dc, dout = ps.dout;
    double* const dg_out =
        DG ? a.dg + ((static_cast<int64_t>(hd) * a.batch + b) * a.nseg + seg) * a.nblk + blk : nullptr;
    if (p0 >= dout) {   // fewer blocks than another pass of the launch
        if (DG && tid == 0) *dg_out = 0.0;
        return;
    }

    // whether the 32 rows from n on are to be formed
    auto used = [&](int n) { return !SKIP || n < dc; };

    const int64_t L = a.seqlen;
    int64_t len = L;
    if (a.lengths != nullptr) {
        const int64_t n = a.lengths[b];
        len = n < 0 ? 0 : (n < L ? n : L);
    }
    const int64_t seg0 = static_cast<int64_t>(seg) * a.seg_len;
    const int64_t seg1 = seg == a.nseg - 1 ? L : seg0 + a.seg_len;
    const int64_t end = len < seg1 ? len : seg1;         // valid tokens: seg0 .. end
    const int64_t ntok = end > seg0 ? end - seg0 : 0;

    const float g1 = a.log_decay[hd];
    const int r = rev ? 1 : 0;

    // the inputs' rows and this thread's place in them; the first chunk's
    // loads go out before anything else
    const int shared = hd / a.rep;   // the head of keys and values
    const int64_t row0 = b * L + seg0;
    const HeadRows rk(ps.k, row0, ps.hk, ps.hk == a.heads ? hd : shared, dc, sizeof(T));
    const HeadRows rv(ps.v, row0, ps.hv, ps.hv == a.heads ? hd : shared, dout, sizeof(T));
    const HeadRows rq(ps.q, row0, ps.hq, ps.hq == a.heads ? hd : shared, dc, sizeof(T));
    const HeadRows rx(ps.x, row0, a.heads, hd, dout, sizeof(T));
    const int ok = Lds::TileK::offset(rk, tid, 0, rev), ov = Lds::TileV::offset(rv, tid, p0, rev);
    const int oq = Lds::TileQ::offset(rq, tid, 0, rev), ox = Lds::TileX::offset(rx, tid, p0, rev);
    const int64_t nchunks = (ntok + C - 1) / C;
    // chunk ch of the walk: its first token in the segment and count (0 past
    // the end); both directions cut at the same tokens
    auto chunk_at = [&](int64_t ch, int64_t& first, int& cnt) {
        first = (rev ? nchunks - 1 - ch : ch) * C;
        const int64_t left = ch < nchunks ? ntok - first : 0;
        cnt = left >= C ? C : static_cast<int>(left);
    };
    typename Lds::TileK tk;
    typename Lds::TileV tv;
    typename Lds::TileQ tq;
    typename Lds::TileX tx;
    auto fetch_kq = [&](int64_t first, int cnt) {
        tk.load(rk, ok, first, cnt, rev);
        if constexpr (!kState) tq.load(rq, oq, first, cnt, rev);
    };
    auto fetch_vx = [&](int64_t first, int cnt) {
        tv.load(rv, ov, first, cnt, rev);
        if constexpr (DG) tx.load(rx, ox, first, cnt, rev);
    };
    {
        int64_t first;
        int cnt;
        chunk_at(0, first, cnt);
        fetch_kq(first, cnt);
        fetch_vx(first, cnt);
    }

    // S: block nt holds rows state_row(nt, g) + v of column p0 + 16 w + c, so
    // that blocks 2 k and 2 k + 1 of a lane are the rows 32 k + 8 g + 0..7 of a
    // fragment
    const int pc = p0 + kLinCols * wc + c;
    const int64_t state_elems = static_cast<int64_t>(dc) * dout;
    const int state_bytes = dc * dout * 4;
    // a state in memory, read or written by buffer offsets: rows and columns
    // past dc x dout fall outside
    typedef __attribute__((__vector_size__(16))) uint32_t u32x4;
    typedef __attribute__((__vector_size__(8))) uint32_t u32x2;
    const int sn = ps.sn, sp = ps.sp;
    const bool runs = kBwd && sn == 1;   // a block's 4 rows lie together (transposed state)
    // dc is a multiple of 4: a block's 4 rows are all in or all out
    auto state_offset = [&](int nt) {
        const int n = n0w + state_row(nt, g);
        const int off = (n * sn + pc * sp) * 4;
        return ((n < dc) & (pc < dout)) ? off : kPastEnd;
    };
    // f(nt, block) over a state in memory, zeros outside it
    auto load_state = [&](const float* from, auto f) {
        const __amdgpu_buffer_rsrc_t rs = lin_rsrc(from, from != nullptr ? state_bytes : 0);
        if (runs) {
#pragma unroll
            for (int nt = 0; nt < NN; ++nt)
                f(nt, __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, state_offset(nt), 0, 0)));
        } else {
#pragma unroll
            for (int nt = 0; nt < NN; ++nt) {
                f32x4 x;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    x[v] = __uint_as_float(
                        __builtin_amdgcn_raw_buffer_load_b32(rs, state_offset(nt) + v * sn * 4, 0, 0));
                f(nt, x);
            }
        }
    };
    const float* sin = ps.s_in != nullptr ? ps.s_in + bh * state_elems : nullptr;
    if (a.nseg > 1) sin = ps.seg_in + (bh * a.nseg + seg) * state_elems;
    if (kState) sin = nullptr;
    f32x4 S[NN];
    load_state(sin, [&](int nt, f32x4 x) { S[nt] = x; });

    if (tid <= C) lds.pow[tid] = decay_power(g1, tid);
    __syncthreads();

    // P's 16 x 16 blocks: this wave forms those of the columns (tokens j) of
    // block jt, for the rows it = grp + GR u; blocks above the diagonal come out
    // as zeros, which the product P v reads beside those on it. The blocks'
    // factors and those of q S for token 16 it + c are the same for every chunk.
    constexpr int GR = WAVES / NT, OWN = NT > GR ? NT / GR : 1;
    const int jt = w % NT, grp = w / NT;
    const bool forms = grp < NT;
    const int it0 = SPLIT > 1 ? part * OT : 0;   // the first of this wave's blocks of the output
    float eo[NT], fac[DG ? 1 : OWN][4];
    if constexpr (DG) {
        for (int n = tid; n < 2 * C; n += THREADS) lds.fac[n] = n < C ? 0.0f : a.scale * lds.pow[n - C];
    } else if constexpr (!kState) {
#pragma unroll
        for (int u = 0; u < OWN; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int n = 16 * (grp + GR * u - jt) + c - 4 * g - v;
                fac[u][v] = n >= 0 && n < C ? a.scale * lds.pow[n] : 0.0f;
            }
    }
    if constexpr (!kState) {
#pragma unroll
        for (int it = 0; it < NT; ++it) eo[it] = ps.out_scale * lds.pow[16 * it + c + 1 - r];
    }
    // what a chunk makes of the state it is entered with: lam^cnt S (FAST), whose
    // factor is off by its own rounding, gone with the state after few chunks; or
    // S + (lam^cnt - 1) S, which rounds only the change (a factor next to 1 applied
    // chunk after chunk would drift, and a change next to -1 rounds at the old
    // state's size where a far smaller one is to be left)
    auto change = [&](int cnt) {
        if (FAST) return uniform(lds.pow[cnt]);
        return uniform(g1 == 0.0f || cnt == 0 ? 0.0f : expm1f(g1 * static_cast<float>(cnt)));
    };
    const float change_full = change(C), change_short = change(static_cast<int>(ntok % C));
    // where this lane's outputs go: token 16 it + c, columns 4 g .. + 3 of the
    // wave's
    const bool wide = IO == kIoF32 || (kBwd && ps.out32);
    const int osize = wide ? 4 : 2;
    const HeadRows ro(ps.out, row0, a.heads, hd, dout, osize);
    const int po = p0 + kLinCols * wc + 4 * g;
    const int oo = po < dout ? (rev ? -c : c) * ro.stride + po * osize : kPastEnd;
    double dg = 0.0;   // this thread's part of the decay's gradient
    f32x4 D[DG ? NN : 1];   // the state's derivative
#pragma unroll
    for (int nt = 0; nt < (DG ? NN : 1); ++nt) D[nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto store_state = [&](float* to) {
        const __amdgpu_buffer_rsrc_t rs = lin_rsrc(to, state_bytes);
        if (runs) {
#pragma unroll
            for (int nt = 0; nt < NN; ++nt)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[nt]), rs, state_offset(nt), 0, 0);
        } else {
#pragma unroll
            for (int nt = 0; nt < NN; ++nt)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[nt][v]), rs,
                                                          state_offset(nt) + v * sn * 4, 0, 0);
        }
    };

    // the weights of a chunk's tokens in the state update; they change with
    // the one chunk that may be short only
    auto weigh = [&](int cnt) {
        if (tid < C) lds.W[tid] = tid < cnt ? ps.state_scale * lds.pow[cnt - 1 - tid + r] : 0.0f;
    };
    int wcnt;
    {
        int64_t first;
        chunk_at(0, first, wcnt);
        weigh(wcnt);
    }
    // the state is waited for here, not at its uses in the loop
#pragma unroll
    for (int nt = 0; nt < NN; ++nt) asm volatile("" : "+v"(S[nt]));
    if constexpr (!kState) {
        // as many stores before the first chunk as a chunk issues (dropped, past
        // the end of an empty range): the waits for a chunk's loads then
        // count the stores behind them and need not wait for those
        const __amdgpu_buffer_rsrc_t none = lin_rsrc(ps.out, 0);
#pragma unroll
        for (int u = 0; u < OT; ++u) {
            if (wide) __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, none, 16 * u, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b64(u32x2{0, 0}, none, 16 * u, 0, 0);
        }
    }
    for (int64_t ch = 0; ch < nchunks; ++ch) {
        int64_t first;
        int cnt;
        chunk_at(ch, first, cnt);
        // (1) stage. The tiles' last readers passed the barrier before P V.
        tk.stage(lds.K, tid);
        if constexpr (!kState) tq.stage(lds.Q, tid);
        tv.stage(lds.V, tid);
        if constexpr (DG) tx.stage(lds.X, tid);
        if (cnt != wcnt) {
            wcnt = cnt;
            weigh(cnt);
        }
        __syncthreads();
        // the next chunk's loads go out in two groups, as the units that
        // address them take as long as a chunk's products; with a second state
        // the registers for them are free behind its product with q only
        int64_t next;
        int next_cnt;
        chunk_at(ch + 1, next, next_cnt);
        if constexpr (!DG) fetch_kq(next, next_cnt);

        f32x4 Y[NT];
        if constexpr (!kState) {
            // (2) q k^T and q S (from the accumulators), which share q's fragments
            f32x4 G[OWN];
#pragma unroll
            for (int u = 0; u < OWN; ++u) G[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int it = 0; it < NT; ++it) Y[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // the second and third terms of x onto a product
            auto rest_terms = [](float (&x)[8], const Frag (&q)[NT], auto& y) {
                const Frag x1 = O::term(x), x2 = O::term(x);
#pragma unroll
                for (int it = 0; it < NT; ++it) y[it] = O::mma(x1, q[it], y[it]);
#pragma unroll
                for (int it = 0; it < NT; ++it) y[it] = O::mma(x2, q[it], y[it]);
            };
#pragma unroll
            for (int k = 0; k < NN / 2; ++k) {
                if (!used(n0w + 32 * k)) continue;
                Frag q[NT];
#pragma unroll
                for (int it = 0; it < NT; ++it) q[it] = O::nat(lds.Q + (16 * it + c) * RQ + n0w + 32 * k, g);
                if constexpr (GR == 1) {
                    const Frag kf = O::nat(lds.K + (16 * jt + c) * RK + 32 * k, g);
#pragma unroll
                    for (int u = 0; u < OWN; ++u) G[u] = O::mma(kf, q[u], G[u]);
                }
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = S[2 * k][e];
                    x[e + 4] = S[2 * k + 1][e];
                }
                const Frag s0 = O::term(x);
#pragma unroll
                for (int it = 0; it < NT; ++it) Y[it] = O::mma(s0, q[it], Y[it]);
                if constexpr (DG && O::kSplit) rest_terms(x, q, Y);
            }
            float dgi = 0.0f;
            const float* const pf = lds.fac + (C + 16 * (grp - jt) + c - 4 * g);
            if (GR == 1 || forms) {
                if constexpr (GR > 1) {
#pragma unroll
                    for (int k = 0; k < DC; k += 32) {
                        if (!used(k)) continue;
                        const Frag kf = O::nat(lds.K + (16 * jt + c) * RK + k, g);
#pragma unroll
                        for (int u = 0; u < OWN; ++u)
                            G[u] = O::mma(kf, O::nat(lds.Q + (16 * (grp + GR * u) + c) * RQ + k, g), G[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < OWN; ++u) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) G[u][v] *= DG ? pf[16 * GR * u - v] : fac[DG ? 0 : u][v];
                    O::st4(lds.P + (16 * (grp + GR * u) + c) * Lds::kRowP + 16 * jt + 4 * g, G[u]);
                }
                if constexpr (DG) {
                    // this column block's share of x_i . v_j, against P's
                    // value and the steps between i and j
                    f32x4 A[OWN];
#pragma unroll
                    for (int u = 0; u < OWN; ++u) A[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < DOB; k += 32) {
                        const Frag vk = O::nat(lds.V + (16 * jt + c) * RV + k, g);
#pragma unroll
                        for (int u = 0; u < OWN; ++u)
                            A[u] = O::mma(vk, O::nat(lds.X + (16 * (grp + GR * u) + c) * RX + k, g), A[u]);
                    }
                    const float apart = static_cast<float>(c - 4 * g + 16 * (grp - jt));
#pragma unroll
                    for (int u = 0; u < OWN; ++u)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            dgi = fmaf((apart + static_cast<float>(16 * GR * u - v)) * G[u][v], A[u][v], dgi);
                }
            }
#pragma unroll
            for (int it = 0; it < NT; ++it) Y[it] *= DG ? ps.out_scale * lds.pow[16 * it + c + 1] : eo[it];
            if constexpr (DG) {
                // the decay's gradient through the entering state; a second
                // walk over q's fragments, as the registers hold no more at once
                f32x4 YD[NT];
#pragma unroll
                for (int it = 0; it < NT; ++it) YD[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < NN / 2; ++k) {
                    if (!used(n0w + 32 * k)) continue;
                    Frag q[NT];
#pragma unroll
                    for (int it = 0; it < NT; ++it) q[it] = O::nat(lds.Q + (16 * it + c) * RQ + n0w + 32 * k, g);
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = D[2 * k][e];
                        x[e + 4] = D[2 * k + 1][e];
                    }
                    const Frag d0 = O::term(x);
#pragma unroll
                    for (int it = 0; it < NT; ++it) YD[it] = O::mma(d0, q[it], YD[it]);
                    if constexpr (O::kSplit) rest_terms(x, q, YD);
                }
#pragma unroll
                for (int it = 0; it < NT; ++it) {
                    const f32x4 x = O::ld4(lds.X + (16 * it + c) * RX + kLinCols * wc + 4 * g);
                    const float steps = static_cast<float>(16 * it + c + 1);
#pragma unroll
                    for (int v = 0; v < 4; ++v) dgi = fmaf(x[v], fmaf(steps, Y[it][v], YD[it][v] * (ps.out_scale * lds.pow[16 * it + c + 1])), dgi);
                }
                dg += static_cast<double>(dgi);
            }
            if constexpr (SPLIT > 1) {
                // this wave goes on with the tokens of its part; the others'
                // half of q S is left for the wave that has them
                f32x4* to = lds.half + ((1 - part) * (WAVES / SPLIT) + wc) * OT * kWave + lane;
#pragma unroll
                for (int u = 0; u < OT; ++u) {
                    to[u * kWave] = part == 0 ? Y[OT + u] : Y[u];
                    Y[u] = part == 0 ? Y[u] : Y[OT + u];
                }
            }
        }

        if constexpr (DG) fetch_kq(next, next_cnt);
        fetch_vx(next, next_cnt);
        // v as the products over tokens read it
        Frag vf[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) vf[s] = O::template tr<RV, 4>(lds.V, 32 * s, kLinCols * wc, c, g);

        // (4) the state: what is left of it, then the chunk's tokens
        const float kept = cnt == C ? change_full : change_short;
        if constexpr (DG) {
            // the derivative, with the steps that the state takes here
            const float f = uniform(FAST ? static_cast<float>(cnt) : static_cast<float>(cnt) * lds.pow[cnt]);
#pragma unroll
            for (int nt = 0; nt < NN; ++nt)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    D[nt][v] = FAST ? fmaf(S[nt][v], f, D[nt][v]) * kept
                                    : fmaf(S[nt][v], f, fmaf(D[nt][v], kept, D[nt][v]));
        }
#pragma unroll
        for (int nt = 0; nt < NN; ++nt)
#pragma unroll
            for (int v = 0; v < 4; ++v) S[nt][v] = FAST ? S[nt][v] * kept : fmaf(S[nt][v], kept, S[nt][v]);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const f32x4 w0 = *reinterpret_cast<const f32x4*>(&lds.W[32 * s + 8 * g]);
            const f32x4 w1 = *reinterpret_cast<const f32x4*>(&lds.W[32 * s + 8 * g + 4]);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = O::get(vf[s], e) * (e < 4 ? w0[e] : w1[e - 4]);
            float y[DG ? 8 : 1];
            if constexpr (DG)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e] * static_cast<float>(cnt - 1 - (32 * s + 8 * g + e));
            Frag v0 = O::term(x), v1, v2, d0, d1, d2;
            if constexpr (O::kSplit) {
                v1 = O::term(x);
                if constexpr (EXACT) v2 = O::term(x);
            }
            if constexpr (DG) {
                d0 = O::term(y);
                if constexpr (O::kSplit) {
                    d1 = O::term(y);
                    d2 = O::term(y);
                }
            }
            if constexpr (!DG) __builtin_amdgcn_sched_barrier(0);
            constexpr int U = SKIP ? 2 : 4;   // independent blocks between the terms of one
#pragma unroll
            for (int n0 = 0; n0 < NN; n0 += U) {
                if (!used(n0w + state_row(n0, 0))) continue;
                Frag kf[U];
#pragma unroll
                for (int u = 0; u < U; ++u) kf[u] = O::template tr<RK, 8>(lds.K, 32 * s, n0w + state_row(n0 + u, 0), c, g);
#pragma unroll
                for (int u = 0; u < U; ++u) S[n0 + u] = O::mma(kf[u], v0, S[n0 + u]);
                if constexpr (O::kSplit)
#pragma unroll
                    for (int u = 0; u < U; ++u) S[n0 + u] = O::mma(kf[u], v1, S[n0 + u]);
                if constexpr (O::kSplit && EXACT && !DG) __builtin_amdgcn_sched_barrier(0);
                if constexpr (O::kSplit && EXACT)
#pragma unroll
                    for (int u = 0; u < U; ++u) S[n0 + u] = O::mma(kf[u], v2, S[n0 + u]);
                if constexpr (DG) {
#pragma unroll
                    for (int u = 0; u < U; ++u) D[n0 + u] = O::mma(kf[u], d0, D[n0 + u]);
                    if constexpr (O::kSplit) {
#pragma unroll
                        for (int u = 0; u < U; ++u) D[n0 + u] = O::mma(kf[u], d1, D[n0 + u]);
#pragma unroll
                        for (int u = 0; u < U; ++u) D[n0 + u] = O::mma(kf[u], d2, D[n0 + u]);
                    }
                }
            }
        }
        __syncthreads();

        // (5) P v onto q S, and out; the next chunk's tiles may be staged by
        // other waves meanwhile
        if constexpr (!kState) {
            if constexpr (SPLIT > 1) {
                const f32x4* from = lds.half + w * OT * kWave + lane;
#pragma unroll
                for (int u = 0; u < OT; ++u) Y[u] += from[u * kWave];
            }
#pragma unroll
            for (int u = 0; u < OT; ++u)
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (32 * s < 16 * (it0 + u + 1)) {
                        const Frag p = O::nat(lds.P + (16 * (it0 + u) + c) * Lds::kRowP + 32 * s, g);
                        Y[u] = O::mma(vf[s], p, Y[u]);
                    }
            const __amdgpu_buffer_rsrc_t rs = ro.chunk(first, cnt);
            const int start = rev ? (cnt - 1) * ro.stride : 0, step = (rev ? -16 : 16) * ro.stride;
            if (wide) {
#pragma unroll
                for (int u = 0; u < OT; ++u)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, Y[u]), rs,
                                                           oo + (start + (it0 + u) * step), 0, 0);
            } else {
#pragma unroll
                for (int u = 0; u < OT; ++u) {
                    bf16x4 o;
#pragma unroll
                    for (int v = 0; v < 4; ++v) o[v] = static_cast<__bf16>(Y[u][v]);
                    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, o), rs,
                                                          oo + (start + (it0 + u) * step), 0, 0);
                }
            }
        }
    }

    if (!DG && sout != nullptr)   // the pass of dq leaves no state
        store_state(sout + (kState ? bh * a.nseg + seg : bh) * state_elems);
    if constexpr (!kState) {
        // rows behind the sequence's end: zeros
        const int64_t z0 = end > seg0 ? end : seg0;
        const int cols = dout - p0 < DOB ? dout - p0 : DOB;
        const int64_t count = (seg1 - z0) * cols;
        for (int64_t e = tid; e < count; e += THREADS) {
            const int64_t at = ((b * L + z0 + e / cols) * a.heads + hd) * dout + p0 + e % cols;
            if (wide) static_cast<float*>(ps.out)[at] = 0.0f;
            else static_cast<__bf16*>(ps.out)[at] = static_cast<__bf16>(0.0f);
        }
    }
    if constexpr (DG) {
        const float* adj = a.nseg > 1 ? a.adj_in + (bh * a.nseg + seg) * state_elems
                                      : (a.dhL != nullptr ? a.dhL + bh * state_elems : nullptr);
        if (adj != nullptr && ntok > 0) {
            float sum = 0.0f;
            load_state(adj, [&](int nt, f32x4 x) {
#pragma unroll
                for (int v = 0; v < 4; ++v) sum = fmaf(D[nt][v], x[v], sum);
            });
            dg += static_cast<double>(sum);
        }
#pragma unroll
        for (int m = 1; m < kWave; m *= 2) dg += __shfl_xor(dg, m);
        if (lane == 0) lds.red[w] = dg;
        __syncthreads();
        if (tid == 0) {
            double sum = 0.0;
            for (int u = 0; u < WAVES; ++u) sum += lds.red[u];
            *dg_out = sum;
        }
    }
}

// The walk in the form that fits the head's decay, the same for all its chunks:
// chosen once, it costs the loop no operation (both forms as keep S + change S,
// one operation more per value of the state: fp32, 2 x 2048 x 8 heads of 200 x
// 168, 135 us against 131, gradients 476 against 466).
template <int IO, int DC, int MODE, bool ALT, bool DG>
__device__ __forceinline__ void linear_attn_walk_any(const LinArgs& a, LinLds<IO, DC, MODE>& lds, const int ip,
                                                     const int blk, int seg, const int64_t bh, const int64_t b,
                                                     const int hd) {
    if (a.log_decay[hd] * static_cast<float>(LinOps<IO>::kChunk) <= -0.6931472f)
        linear_attn_walk<IO, DC, MODE, ALT, DG, true>(a, lds, ip, blk, seg, bh, b, hd);
    else
        linear_attn_walk<IO, DC, MODE, ALT, DG, false>(a, lds, ip, blk, seg, bh, b, hd);
}

// Waves that a SIMD holds at least. fp32 gradients of heads of 64 fit three, which
// the compiler misses by a few registers left to itself (8 x 2048 x 32 heads of
// 64: 437 us against 448).
constexpr int lin_waves_per_simd(int io, int dc, int mode) {
    return io == kIoF32 && dc == 64 && mode == kLinBwd ? 3 : 2;
}

template <int IO, int DC, int MODE>
__global__ __launch_bounds__(lin_waves(DC) * kWave,
                             lin_waves_per_simd(IO, DC, MODE)) void linear_attn_kernel(LinArgs a) {
    __shared__ LinLds<IO, DC, MODE> lds;
    // which (row, head, segment, pass, column block); neighbours in this
    // order read the same rows and share an XCD's L2. The pass that forms the
    // decay's gradient takes longest and goes first; the others run beside it.
    const bool ordered = MODE == kLinBwd && a.dg != nullptr;
    const uint32_t most = ordered ? gridDim.x / a.npass : 0;
    const bool first = blockIdx.x < most;
    uint32_t id = first ? xcd_order(blockIdx.x, most) : xcd_order(blockIdx.x - most, gridDim.x - most);
    uint32_t up = id / a.nblk;
    const int blk = static_cast<int>(id - up * a.nblk);
    id = up;
    int ip = 0;
    if (!first) {
        const uint32_t np = ordered ? a.npass - 1 : a.npass;
        up = id / np;
        ip = static_cast<int>(id - up * np) + (ordered ? 1 : 0);
        id = up;
    }
    const uint32_t nsegs = MODE == kLinState ? a.nseg - 1 : a.nseg;
    up = id / nsegs;
    const int seg = static_cast<int>(id - up * nsegs);
    const uint32_t row = up / a.heads;
    const int hd = static_cast<int>(up - row * a.heads);
    const LinPass& ps = a.pass[ip];
    // Whole blocks of 32 state rows past the head's width. The fp32 kernels, bound
    // by their matrix instruction, leave them out (6 x 3036 x 18 heads of 24 x
    // 72: 153 us against 198); in bf16, and where nothing is unused, the
    // branches cost more than they save (bf16, 1 x 7905 x 48 heads of 224 x 192:
    // 1717 us against 1353).
    const bool unused = ps.dc <= DC - 32;
    if constexpr (MODE == kLinBwd) {
        if (first) {
            if (IO == kIoBF16 || unused)
                linear_attn_walk_any<IO, DC, MODE, true, true>(a, lds, ip, blk, seg, up, row, hd);
            else
                linear_attn_walk_any<IO, DC, MODE, IO == kIoBF16, true>(a, lds, ip, blk, seg, up, row, hd);
            return;
        }
    }
    // a state that the caller gets
    const bool leaves = ps.s_out != nullptr && seg == (ps.rev ? 0 : a.nseg - 1);
    if (IO == kIoBF16 ? (MODE == kLinState ? a.exact != 0 : leaves) : unused)
        linear_attn_walk_any<IO, DC, MODE, true, false>(a, lds, ip, blk, seg, up, row, hd);
    else
        linear_attn_walk_any<IO, DC, MODE, false, false>(a, lds, ip, blk, seg, up, row, hd);
}

}  // namespace
}  // namespace mamba
