// Gated linear recurrence: forward, gradients, single token. Per channel, with
// p = sigmoid(decay gate), q = sigmoid(input gate), g = log_decay p:
//     a = exp(g),  b = sqrt(1 - a^2),  w = b q,   h_t = a_t h_{t-1} + w_t x_t
// and backward, with A_t = dy_t + a_{t+1} A_{t+1} the gradient at h_t:
//     dx = A w       d(input gate) = A w x (1 - q)       dh0 = a_0 A_0
//     dg = A a (h_{t-1} - q x a / b)
//     d(decay gate) = dg g (1 - p)       d(log_decay) = sum of dg p
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "internal.h"

namespace mamba {
namespace {

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

// The base-2 logarithm of a channel's decay, finite for the lowest natural one as
// well: its product with a closed gate's 0 is 0.
__device__ __forceinline__ float log2_of(float log_decay) {
    constexpr float LOWEST = -3.4028235e38f;
    const float v = log_decay * kLog2e;
    return v < LOWEST ? LOWEST : v;   // a NaN stays one
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

// sigmoid(v) and 1 - sigmoid(v), each to its own accuracy. Far down p is 0, as
// forward: what a gate closed by the type's lowest value lets through is nothing,
// behind which a masked x may be as large as the type goes.
__device__ __forceinline__ void sigmoid_both(float v, float& p, float& rest) {
    const float x = -v * kLog2e, e = fast_exp2(x);
    p = fast_rcp(1.0f + e);
    rest = x > 126.0f ? 1.0f : e * p;   // a NaN stays one
}

// A value that is formed here and not later from what it is made of, which is
// more to keep.
__device__ __forceinline__ void formed(float& v) { asm volatile("" : "+v"(v)); }

// An offset that the compiler takes for a new one, lest it keep the offsets of all
// of a tile's tokens in registers from tile to tile.
__device__ __forceinline__ uint32_t fresh(uint32_t at) {
    asm volatile("" : "+v"(at));
    return at;
}

// Keeps the arithmetic of a few tokens together, lest all of a segment's
// intermediate values be alive at once.
__device__ __forceinline__ void token_fence(int t) {
    if (t % 2 == 1) __builtin_amdgcn_sched_barrier(0);
}

template <int IO>
constexpr int size_of() { return IO == kIoF32 ? 4 : 2; }

// V neighbouring channels of one token, in one access of at most 4 bytes: fp32 one,
// bf16 one or two. A single bf16 value is kept as 16 bits until use, where a shift
// takes it: as 32 the compiler would clear the upper half of each loaded value, and
// wait for it, long before.
template <int IO, int V>
using Token = std::conditional_t<size_of<IO>() * V == 4, uint32_t, uint16_t>;

template <int IO, int V>
__device__ __forceinline__ Token<IO, V> load_value(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t row) {
    static_assert(size_of<IO>() * V <= 4, "a token is one access");
    if constexpr (size_of<IO>() * V == 4)
        return __builtin_amdgcn_raw_buffer_load_b32(rs, static_cast<int>(at), static_cast<int>(row), 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b16(rs, static_cast<int>(at), static_cast<int>(row), 0);
}

template <int IO, typename W>
__device__ __forceinline__ float value(W w, int v) {
    return v == 0 ? raw_to_f32<IO>(w) : __uint_as_float(w & 0xffff0000u);
}

template <int IO, int V>
__device__ __forceinline__ void store_value(__amdgpu_buffer_rsrc_t rs, uint32_t at, uint32_t row, const float (&v)[V]) {
    if constexpr (IO == kIoF32) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), rs, static_cast<int>(at), static_cast<int>(row), 0);
    } else if constexpr (V == 1) {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, static_cast<__bf16>(v[0])), rs,
                                              static_cast<int>(at), static_cast<int>(row), 0);
    } else {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 o = __builtin_convertvector((f32x2{v[0], v[V - 1]}), bf16x2);
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, o), rs, static_cast<int>(at),
                                              static_cast<int>(row), 0);
    }
}

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t seqlen) {
    if (lengths == nullptr) return seqlen;
    // a scalar load: nothing writes lengths, and a vector one would wait behind all others
    const int64_t n = ((const __attribute__((address_space(4))) int32_t*)lengths)[b];
    return n < 0 ? 0 : (n < seqlen ? n : seqlen);
}

// A workgroup's place: 64 channels by W V segments of T consecutive tokens. Of a
// wave, 64 / V lanes hold V channels each of one segment, the next lanes the next.
constexpr int kGsChannels = kWave;

template <int V>
struct Place {
    int wave, lane, sub, cl, ch;   // sub: the lane's segment in its wave; cl: its first channel in the workgroup, ch: of all
    bool in;

    __device__ __forceinline__ Place(int64_t dim, int64_t group) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        lane = threadIdx.x % kWave;
        sub = V == 1 ? 0 : lane / (kWave / V);
        cl = V == 1 ? lane : lane % (kWave / V) * V;
        ch = static_cast<int>(group * kGsChannels) + cl;
        in = ch < dim;
    }
    __device__ __forceinline__ int segment() const { return wave * V + sub; }
};

// One tensor's tile as a wave walks its tokens: a buffer resource that spans the
// tile's rows, so that loads behind the row's last token give zeros and stores
// behind the sequence are dropped; a lane without a channel has an offset past every
// resource. FULL: all of the tile's tokens are there, and the token's place goes into
// the scalar offset, which costs no vector instruction; else into the lane's, as the
// bounds check need not look at the scalar one.
template <int IO, int V, int T, int W, bool FULL>
struct Rows {
    static constexpr int TILE = W * V * T;
    __amdgpu_buffer_rsrc_t rs;
    uint32_t at, row, step;

    __device__ __forceinline__ Rows(const Place<V>& place, const void* p, int64_t first, int64_t stride, int64_t dim,
                                    int64_t count) {
        const int n = static_cast<int>(FULL || count > TILE ? TILE : count);
        const int ld = static_cast<int>(stride);
        rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(static_cast<const char*>(p) + first * stride * size_of<IO>()), 0,
            n > 0 ? ((n - 1) * ld + static_cast<int>(dim)) * size_of<IO>() : 0, 0x00020000);
        step = static_cast<uint32_t>(ld) * size_of<IO>();
        uint32_t lane = static_cast<uint32_t>(place.ch) * size_of<IO>();
        if (V > 1) lane += place.sub * T * step;
        const uint32_t tokens = place.wave * V * T * step;
        if (FULL) {
            at = place.in ? lane : 0x80000000u;
            row = tokens;
        } else {
            at = fresh(place.in ? lane + tokens : 0x80000000u);
            row = 0;
        }
    }
    __device__ __forceinline__ Token<IO, V> load() const { return load_value<IO, V>(rs, at, row); }
    __device__ __forceinline__ void store(const float (&v)[V]) const { store_value<IO, V>(rs, at, row, v); }
    __device__ __forceinline__ void go(int tokens) {
        if (FULL) row += tokens * step;
        else at += tokens * step;
    }
};

// How many of a segment's T tokens lie before the row's end, `left` tokens away from
// the tile's start.
template <int T, int TILE>
__device__ __forceinline__ int live_tokens(int segment, int64_t left) {
    return static_cast<int>(left < TILE ? left : TILE) - segment * T;
}

// What precedes a lane's segment in its wave, and the wave's whole: a state c that
// enters the wave enters the segment as P c + h.
template <int V>
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
            const bool later = (sub & m) != 0;
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

// (G, h) of tokens followed by those of a next segment.
__device__ __forceinline__ void append(float& G, float& h, float nextG, float nexth) {
    h = fmaf(fast_exp2(nextG), h, nexth);
    G += nextG;
}

// ---------------------------------------------------------------------------
// How a tile learns the state that enters it. A workgroup that walks a row knows
// it; where rows and channels are too few to fill the chip, tiles go to the
// workgroups one by one (a chain), in the order of tickets taken from a counter:
// all rows' and groups' first tiles, then all second ones; tiles without tokens, which
// nothing waits for, come last. (In between, they would let some workgroups run ahead
// to tiles that wait for ones which others hold for later: 11 rows of up to 30893 x 240
// took 412 us for their gradients, all rows full 336.) A tile's sum over its
// tokens (G, h) is published at once, and what enters it is folded, always in the
// same order, from the sums of the up to 7 tiles before it in its run of 8, of the
// up to 7 runs before that in their stretch of 8 runs, and the state that enters
// the stretch, which the stretch before publishes at its end. One of the workgroup's
// waves does this, a lane for each channel.
//
// Every wait ends: a tile waits for words of tiles of smaller tickets only. A
// ticket is taken by a workgroup that runs, running workgroups keep their place, and
// a workgroup works on its tickets in their order. So the workgroup that holds the
// smallest unfinished ticket of all is at work on it, and what that tile waits for
// has been published by finished ones; it ends, and then the next.
//
// A word is one 64-bit access and carries its own mark, so no order between words
// is needed: its high half is G, or 0 for a state, and all ones before it is
// written, which no G is (a NaN is written as 0x7fc00000).
constexpr int kRun = 8, kStretch = 64;

typedef unsigned long long Word;
constexpr Word kNoWord = ~0ull;

__device__ __forceinline__ Word word_of(float G, float h) {
    const uint32_t hi = G == G ? __float_as_uint(G) : 0x7fc00000u;
    return static_cast<Word>(hi) << 32 | __float_as_uint(h);
}
__device__ __forceinline__ float word_G(Word w) { return __uint_as_float(static_cast<uint32_t>(w >> 32)); }
__device__ __forceinline__ float word_h(Word w) { return __uint_as_float(static_cast<uint32_t>(w)); }

__device__ __forceinline__ void publish(Word* at, Word w) {
    __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Word look(const Word* at) {
    return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Word await(const Word* at, Word w) {
    while (static_cast<uint32_t>(w >> 32) == 0xffffffffu) {
        __builtin_amdgcn_s_sleep(1);
        w = look(at);
    }
    return w;
}

// The chain's scratch: a counter (256 bytes), words for every (row, tile), (row, run)
// and (row, stretch) of all channels, and the order of the (tile, row) pairs where rows
// are of different lengths.
struct Chain {
    uint32_t* ticket;
    Word *tile, *run, *stretch;
    uint32_t* order;
    const int32_t* lengths;
    int64_t seqlen;
    uint32_t groups, batch, tiles, runs, stretches, pairs;
    int tokens;   // of a tile
    bool once;    // a workgroup for every tile
    int64_t width;

    // Of more rows than this, a pair's place takes longer to count than it saves.
    static constexpr uint32_t kOrdered = 512;

    __host__ __device__ Chain(void* ws, int64_t rows, int64_t length, const int32_t* lens, int64_t channel_groups,
                              int tile_tokens)
        : seqlen(length), tokens(tile_tokens), once(false) {
        groups = static_cast<uint32_t>(channel_groups);
        batch = static_cast<uint32_t>(rows);
        tiles = static_cast<uint32_t>((length + tile_tokens - 1) / tile_tokens);
        runs = (tiles + kRun - 1) / kRun;
        stretches = (tiles + kStretch - 1) / kStretch;
        pairs = batch * tiles;
        width = channel_groups * kGsChannels;
        lengths = batch <= kOrdered ? lens : nullptr;
        ticket = static_cast<uint32_t*>(ws);
        tile = reinterpret_cast<Word*>(static_cast<char*>(ws) + 256);
        run = tile + rows * tiles * width;
        stretch = run + rows * runs * width;
        order = reinterpret_cast<uint32_t*>(tile + words());
    }
    __host__ __device__ int64_t words() const {
        return batch * (static_cast<int64_t>(tiles) + runs + stretches) * width;
    }
};

// Clears the words and the counter, two words to a thread, and sets the order: a pair
// with tokens comes behind all such of smaller tiles, and of its own tile and smaller
// rows; one without behind all with.
__global__ __launch_bounds__(256) void gated_scan_clear_kernel(Chain ch) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i == 0) *ch.ticket = 0;
    if (i < ch.words() / 2) reinterpret_cast<ulonglong2*>(ch.tile)[i] = make_ulonglong2(kNoWord, kNoWord);
    if (ch.lengths == nullptr || i >= ch.pairs) return;
    const uint32_t p = static_cast<uint32_t>(i), j = p / ch.batch, b = p - j * ch.batch;
    uint32_t before = 0, all = 0;
    bool live = false;
    for (uint32_t r = 0; r < ch.batch; ++r) {
        const int64_t len = row_length(ch.lengths, r, ch.seqlen);
        const uint32_t n = static_cast<uint32_t>((len + ch.tokens - 1) / ch.tokens);
        all += n;
        before += (n < j ? n : j) + (r < b && n > j ? 1 : 0);
        if (r == b) live = n > j;
    }
    ch.order[live ? before : all + (p - before)] = p;
}

// The next ticket. (Through an address that the compiler takes for a lane's own: for
// one that all lanes share it adds up their requests first and waits for the answer
// at once, behind all loads on their way.)
__device__ __forceinline__ uint32_t take_ticket(uint32_t* counter) {
    uint32_t none = 0;
    asm volatile("" : "+v"(none));
    return __hip_atomic_fetch_add(counter + none, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A ticket's place in the chain.
constexpr uint32_t kNoTicket = 0xffffffffu;

struct Link {
    uint32_t j, b, group;   // position in the row, row, group of channels
    bool any;

    __device__ __forceinline__ Link(const Chain& ch, uint32_t n) {
        uint32_t p = n / ch.groups;
        group = n - p * ch.groups;
        any = n != kNoTicket && p < ch.pairs;
        p = any ? p : 0;
        if (ch.lengths != nullptr) p = ((const __attribute__((address_space(4))) uint32_t*)ch.order)[p];
        j = p / ch.batch;
        b = p - j * ch.batch;
    }
};

// One channel of (rows, dim), or zero.
__device__ __forceinline__ float load_state(const float* p, int64_t row, int64_t dim, int64_t col) {
    return p != nullptr && col < dim ? p[row * dim + col] : 0.0f;
}

// The state that enters a tile, for the lane's channel col; the tile's own sum
// (G, h) is published on the way. `start` enters the row; the first tile alone reads
// it and publishes it as what enters the first stretch, since the last tile may write
// its result to the same memory. `out` leaves the tile.
__device__ __forceinline__ float enter_tile(const Chain& ch, const Link& at, int64_t dim, int64_t col, float G,
                                            float h, const float* start, float& out) {
    const int kt = at.j % kRun, kr = at.j % kStretch / kRun;
    Word* tile = ch.tile + (static_cast<int64_t>(at.b) * ch.tiles + at.j) * ch.width + col;
    Word* run = ch.run + (static_cast<int64_t>(at.b) * ch.runs + at.j / kRun) * ch.width + col;
    Word* stretch = ch.stretch + (static_cast<int64_t>(at.b) * ch.stretches + at.j / kStretch) * ch.width + col;
    publish(tile, word_of(G, h));
    Word wt[kRun - 1], wr[kRun - 1], ws;
    const Word none = word_of(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < kRun - 1; ++u) wt[u] = u < kt ? look(tile - (kt - u) * ch.width) : none;
#pragma unroll
    for (int u = 0; u < kRun - 1; ++u) wr[u] = u < kr ? look(run - (kr - u) * ch.width) : none;
    if (at.j > 0) {
        ws = look(stretch);
    } else {
        ws = word_of(0.0f, load_state(start, at.b, dim, col));
        if (ch.tiles > 1) publish(stretch, ws);
    }
    float Gt = 0.0f, ht = 0.0f;
#pragma unroll
    for (int u = 0; u < kRun - 1; ++u)
        if (u < kt) {
            const Word w = await(tile - (kt - u) * ch.width, wt[u]);
            append(Gt, ht, word_G(w), word_h(w));
        }
    if (kt == kRun - 1) {   // the run's last: its sum, before what enters it is known
        float Ga = Gt, ha = ht;
        append(Ga, ha, G, h);
        publish(run, word_of(Ga, ha));
    }
    float Gr = 0.0f, hr = 0.0f;
#pragma unroll
    for (int u = 0; u < kRun - 1; ++u)
        if (u < kr) {
            const Word w = await(run - (kr - u) * ch.width, wr[u]);
            append(Gr, hr, word_G(w), word_h(w));
        }
    append(Gr, hr, Gt, ht);
    const float c = carried(word_h(await(stretch, ws)), Gr, hr);
    out = carried(c, G, h);
    if (at.j % kStretch == kStretch - 1 && at.j + 1 < ch.tiles) publish(stretch + ch.width, word_of(0.0f, out));
    return c;
}

// A tile of the forward pass.
template <int IO, int V, int T, int W, bool GATED>
struct FwdTile {
    static constexpr int TILE = T * V * W;
    static_assert(TILE % kGatedBlock == 0 && kGatedBlock % T == 0, "blocks of states at segments");
    typedef Rows<IO, V, T, W, false> R;
    typedef Place<V> P;
    Token<IO, V> x[T], d[T], i[T];
    float ca[T][V], cu[T][V];
    float P0[V], h0[V];   // what precedes the lane's segment in its wave
    float Gw[V], hw[V];   // and the wave in its tile

    // Where the inputs of a tile are; `left` <= 0: nowhere.
    struct In {
        R d, i, x;
        __device__ __forceinline__ In(const GatedScanArgs& a, const P& at, int64_t b, int64_t t0, int64_t left)
            : d(at, a.decay_gate, b * a.seqlen + t0, a.decay_stride, a.dim, left),
              i(at, a.input_gate, b * a.seqlen + t0, a.input_stride, a.dim, GATED ? left : 0),
              x(at, a.x, b * a.seqlen + t0, a.x_stride, a.dim, left) {}
    };
    __device__ __forceinline__ void load(int t, In& in) {
        d[t] = in.d.load();
        in.d.go(1);
        if constexpr (GATED) {
            i[t] = in.i.load();
            in.i.go(1);
        }
        x[t] = in.x.load();
        in.x.go(1);
    }
    // In the order of work()'s loads: a wait for one counts those behind it.
    __device__ __forceinline__ void load_all(In in) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            load(t, in);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // Each token's inputs are used up and the next tile's loaded in their place, so
    // that loads are on their way all the time. Tokens behind the row's end have no
    // decay, so a = 1 and w = 0. The wave's sums go to LDS.
    __device__ __forceinline__ void work(const P& at, const float (&lam2)[V], int64_t left, In next,
                                         float2 (&sums)[W][kGsChannels]) {
        const int live = live_tokens<T, TILE>(at.segment(), left);
        float G[V], hl[V], P1[V];
#pragma unroll
        for (int v = 0; v < V; ++v) G[v] = hl[v] = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay1 e(sigmoid(value<IO>(d[t], v)), t < live ? lam2[v] : 0.0f);
                float w = __builtin_amdgcn_sqrtf(e.s);
                if constexpr (GATED) w *= sigmoid(value<IO>(i[t], v));
                ca[t][v] = e.a;
                cu[t][v] = w * value<IO>(x[t], v);
                formed(ca[t][v]);
                formed(cu[t][v]);
                G[v] += e.g2;
                hl[v] = fmaf(ca[t][v], hl[v], cu[t][v]);
            }
            load(t, next);
            token_fence(t);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P1[v] = V > 1 ? fast_exp2(G[v]) : 1.0f;
#pragma unroll
            for (int m = 1; m < V; m *= 2) G[v] += __shfl_xor(G[v], m * (kWave / V));
        }
        const Before<V> before(at.sub, P1, hl);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P0[v] = before.P[v];
            h0[v] = before.h[v];
            if (at.sub == 0) sums[at.wave][at.cl + v] = make_float2(G[v], hl[v]);
        }
    }
    // What needs the other waves' sums, and not yet what enters the tile.
    __device__ __forceinline__ void gather(const P& at, const float2 (&sums)[W][kGsChannels]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Gw[v] = hw[v] = 0.0f;
            for (int w = 0; w < at.wave; ++w) append(Gw[v], hw[v], sums[w][at.cl + v].x, sums[w][at.cl + v].y);
        }
    }
    // The outputs, from the states entering the tile.
    __device__ __forceinline__ void finish(const GatedScanArgs& a, const P& at, int64_t b, int64_t t0, int64_t len,
                                           const float (&enter)[kGsChannels]) {
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(P0[v], carried(enter[at.cl + v], Gw[v], hw[v]), h0[v]);
        const int64_t tseg = t0 + at.segment() * T;
        if (a.states != nullptr && at.segment() * T % kGatedBlock == 0 && tseg < len && at.in) {
            const int64_t blocks = (a.seqlen + kGatedBlock - 1) / kGatedBlock;
            float* to = a.states + (b * blocks + tseg / kGatedBlock) * a.dim + at.ch;
#pragma unroll
            for (int v = 0; v < V; ++v) to[v] = h[v];
        }
        R y(at, a.y, b * a.seqlen + t0, a.dim, a.dim, a.seqlen - t0);
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(ca[t][v], h[v], cu[t][v]);
            y.store(h);
            y.go(1);
        }
        if (len - t0 < TILE) none(a, at, b, t0, live_tokens<T, TILE>(at.segment(), len - t0));
    }
    // Zeros for a tile's tokens behind the row's last one, from the segment's `from`-th
    // on (over what is there, which a lane's own stores are in order with).
    static __device__ __forceinline__ void none(const GatedScanArgs& a, const P& at, int64_t b, int64_t t0, int from) {
        R y(at, a.y, b * a.seqlen + t0, a.dim, a.dim, a.seqlen - t0);
        const float zero[V] = {};
#pragma unroll
        for (int t = 0; t < T; ++t) {
            if (t >= from) y.store(zero);
            y.go(1);
        }
    }
};

// The log decays of a lane's channels, as loaded; zero where there is none.
template <int V>
__device__ __forceinline__ void load_log_decay(const GatedScanArgs& a, const Place<V>& at, uint32_t (&w)[V]) {
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(a.log_decay), 0, static_cast<int>(a.dim) * 4, 0x00020000);
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = __builtin_amdgcn_raw_buffer_load_b32(rs, (at.ch + v) * 4, 0, 0);
}

template <int V>
__device__ __forceinline__ void log2_decay(const uint32_t (&w)[V], float (&lam2)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) lam2[v] = log2_of(__uint_as_float(w[v]));
}

// A tile's whole sum for one of the workgroup's channels.
template <int W>
__device__ __forceinline__ float2 tile_sum(const float2 (&sums)[W][kGsChannels], int cl) {
    float G = 0.0f, h = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) append(G, h, sums[w][cl].x, sums[w][cl].y);
    return make_float2(G, h);
}

// The forward pass, a workgroup walking one row's tiles. The waves take turns in
// carrying the state over a tile, a lane for each channel. About 38 vector
// instructions a value, 7 of them transcendental, keep the vector units busy for 67% of
// the time: 8 x 2048 x 4096 in bf16 118 us (4.5 TB/s). With an input gate a lane takes
// 139 registers, so that 3 waves find room on a SIMD and one workgroup (2 on each) on a
// unit; narrower, what a row takes is the latency of its tiles, about 3.3 us each (8 x
// 2048 x 1536 53 us).
template <int IO, int V, int T, int W, bool GATED>
__global__ __launch_bounds__(W* kWave) void gated_scan_fwd_kernel(GatedScanArgs a, int64_t groups) {
    typedef FwdTile<IO, V, T, W, GATED> Tile;
    typedef typename Tile::In In;
    __shared__ float2 sums[2][W][kGsChannels];   // by turns, so that one barrier a tile is enough
    __shared__ float enter[2][kGsChannels];
    const int64_t b = blockIdx.x / groups, group = blockIdx.x - b * groups;
    const Place<V> at(a.dim, group);
    const int64_t len = row_length(a.lengths, b, a.seqlen), col = group * kGsChannels + at.lane;
    float lam2[V];
    uint32_t decays[V];
    load_log_decay(a, at, decays);
    log2_decay(decays, lam2);
    if (at.wave == 0) enter[0][at.lane] = load_state(a.h0, b, a.dim, col);
    Tile tile;
    tile.load_all(In(a, at, b, 0, len));
    int k = 0;
    int64_t t0 = 0;
    for (; t0 < len; t0 += Tile::TILE, ++k) {
        const int odd = k & 1;
        tile.work(at, lam2, len - t0, In(a, at, b, t0 + Tile::TILE, len - t0 - Tile::TILE), sums[odd]);
        __syncthreads();
        if (at.wave == k % W) {
            const float2 all = tile_sum<W>(sums[odd], at.lane);
            enter[odd ^ 1][at.lane] = carried(enter[odd][at.lane], all.x, all.y);
        }
        tile.gather(at, sums[odd]);
        tile.finish(a, at, b, t0, len, enter[odd]);
    }
    __syncthreads();
    if (a.hL != nullptr && at.wave == 0 && col < a.dim) a.hL[b * a.dim + col] = enter[k & 1][at.lane];
    for (; t0 < a.seqlen; t0 += Tile::TILE) Tile::none(a, at, b, t0, 0);
}

// The forward pass as a chain. A workgroup takes tickets until none is left, one
// ahead of the tile whose inputs are being loaded. 1 x 262144 x 2048 in bf16 960 us
// (4.5 TB/s), of which the look for what enters a tile, a trip to memory in each, costs
// 150: a wave that does nothing but look, and looking while the next tile is worked
// through, were no faster (981 and 1491 us).
template <int IO, int V, int T, int W, bool GATED>
__global__ __launch_bounds__(W* kWave) void gated_scan_fwd_chain_kernel(GatedScanArgs a, Chain ch) {
    typedef FwdTile<IO, V, T, W, GATED> Tile;
    typedef typename Tile::In In;
    __shared__ float2 sums[2][W][kGsChannels];   // by turns: read behind a tile's second barrier
    __shared__ float enter[kGsChannels];
    __shared__ uint32_t taken[2];
    if (threadIdx.x == 0) {
        taken[0] = take_ticket(ch.ticket);
        taken[1] = ch.once ? kNoTicket : take_ticket(ch.ticket);
    }
    __syncthreads();
    Link at(ch, __builtin_amdgcn_readfirstlane(taken[0])), next(ch, __builtin_amdgcn_readfirstlane(taken[1]));
    __syncthreads();
    Tile tile;
    auto left_of = [&](const Link& l) {
        return l.any ? row_length(a.lengths, l.b, a.seqlen) - static_cast<int64_t>(l.j) * Tile::TILE : int64_t(0);
    };
    auto in_of = [&](const Link& l, int64_t left) {
        return In(a, Place<V>(a.dim, l.group), l.b, static_cast<int64_t>(l.j) * Tile::TILE, left);
    };
    int64_t left = left_of(at);
    uint32_t decays[V], next_decays[V];   // loaded ahead of the inputs: a wait for them would else be for all of those
    load_log_decay(a, Place<V>(a.dim, at.group), decays);
    tile.load_all(in_of(at, left));
    for (int k = 0; at.any; ++k) {
        const Place<V> place(a.dim, at.group);
        load_log_decay(a, Place<V>(a.dim, next.group), next_decays);
        const int64_t b = at.b, t0 = static_cast<int64_t>(at.j) * Tile::TILE, len = t0 + left,
                      next_left = left_of(next), col = static_cast<int64_t>(at.group) * kGsChannels + place.lane;
        uint32_t mine = kNoTicket;
        if (threadIdx.x == 0 && !ch.once) mine = take_ticket(ch.ticket);
        if (left > 0) {
            float lam2[V];
            log2_decay(decays, lam2);
            const bool looks = place.wave == k % W;
            tile.work(place, lam2, left, in_of(next, next_left), sums[k & 1]);
            __syncthreads();
            if (looks) {
                const float2 all = tile_sum<W>(sums[k & 1], place.lane);
                float out;
                enter[place.lane] = enter_tile(ch, at, a.dim, col, all.x, all.y, a.h0, out);
                if (a.hL != nullptr && left <= Tile::TILE && col < a.dim) a.hL[b * a.dim + col] = out;
            }
            if (threadIdx.x == 0) taken[0] = mine;
            if (!looks) tile.gather(place, sums[k & 1]);   // while the other looks
            __syncthreads();
            if (looks) tile.gather(place, sums[k & 1]);
            tile.finish(a, place, b, t0, len, enter);
        } else {
            tile.load_all(in_of(next, next_left));
            Tile::none(a, place, b, t0, 0);
            if (at.j == 0 && a.hL != nullptr && place.wave == 0 && col < a.dim)   // a row without tokens
                a.hL[b * a.dim + col] = load_state(a.h0, b, a.dim, col);
            __syncthreads();   // the ticket before this one has been read
            if (threadIdx.x == 0) taken[0] = mine;
            __syncthreads();
        }
        at = next;
        left = next_left;
#pragma unroll
        for (int v = 0; v < V; ++v) decays[v] = next_decays[v];
        next = Link(ch, __builtin_amdgcn_readfirstlane(taken[0]));
    }
}

// A tile of the backward pass.
template <int IO, int T, int W, bool GATED>
struct BwdTile {
    static constexpr int TILE = T * W;
    static_assert(TILE % kGatedBlock == 0, "tiles start at kept states");
    Token<IO, 1> x[T], d[T], i[T], dy[T];
    float state;   // entering the tile
    float Gw, hw;  // what the later waves of the tile add to the adjoint
    float ca[T], cw[T], cu[T], cp[T], cgr[T], cir[T], ck[T];

    template <bool FULL>
    struct In {
        typedef Rows<IO, 1, T, W, FULL> R;
        R d, i, x, dy;
        const float* state;
        __device__ __forceinline__ In(const GatedScanArgs& a, const Place<1>& at, int64_t b, int64_t t0, int64_t left)
            : d(at, a.decay_gate, b * a.seqlen + t0, a.decay_stride, a.dim, left),
              i(at, a.input_gate, b * a.seqlen + t0, a.input_stride, a.dim, left),
              x(at, a.x, b * a.seqlen + t0, a.x_stride, a.dim, left),
              dy(at, a.dy, b * a.seqlen + t0, a.dim, a.dim, left),
              state(left > 0 && at.in
                        ? a.states + (b * ((a.seqlen + kGatedBlock - 1) / kGatedBlock) + t0 / kGatedBlock) * a.dim + at.ch
                        : nullptr) {}
    };
    template <bool FULL>
    __device__ __forceinline__ void load(int t, In<FULL>& in) {
        d[t] = in.d.load();
        in.d.go(1);
        if constexpr (GATED) {
            i[t] = in.i.load();
            in.i.go(1);
        }
        x[t] = in.x.load();
        in.x.go(1);
    }
    // In the order of the loads of work() and finish(): a wait for one counts those
    // behind it.
    __device__ __forceinline__ void load_all(In<false> in) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            load(t, in);
            __builtin_amdgcn_sched_barrier(0);
        }
        state = in.state != nullptr ? *in.state : 0.0f;
        in.dy.go(T - 1);
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            dy[t] = in.dy.load();
            in.dy.go(-1);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // As forward; the next tile's dy is loaded by finish(), which needs this one's.
    template <bool FULL>
    __device__ __forceinline__ void work(const Place<1>& at, float lam2, int64_t left, In<FULL>& next,
                                         float2 (&sums)[W][kGsChannels], float2 (&backs)[W][kGsChannels]) {
        const int live = FULL ? T : live_tokens<T, TILE>(at.wave, left);
        float G = 0.0f, hl = 0.0f, El = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float p, rest;
            sigmoid_both(raw_to_f32<IO>(d[t]), p, rest);
            const Decay1 e(p, t < live ? lam2 : 0.0f);
            const float r = __builtin_amdgcn_rsqf(e.s);
            const float rb = e.s < 1.1754944e-38f ? 0.0f : r;   // nothing enters: no derivative
            const float xv = raw_to_f32<IO>(x[t]);
            float w = e.s * rb, qx = xv;
            if constexpr (GATED) {
                float q, qrest;
                sigmoid_both(raw_to_f32<IO>(i[t]), q, qrest);
                w *= q;
                qx *= q;
                cir[t] = w * xv * qrest;
                formed(cir[t]);
            }
            ca[t] = e.a;
            cw[t] = w;
            cu[t] = w * xv;
            cp[t] = t < live ? p : 0.0f;
            cgr[t] = e.g2 * kLn2 * rest;
            ck[t] = qx * (e.a * rb);
            formed(ca[t]);
            formed(cw[t]);
            formed(cu[t]);
            formed(cp[t]);
            formed(cgr[t]);
            formed(ck[t]);
            G += e.g2;
            hl = fmaf(ca[t], hl, cu[t]);
            load(t, next);
            token_fence(t);
        }
#pragma unroll
        for (int t = T - 1; t >= 0; --t) El = ca[t] * (raw_to_f32<IO>(dy[t]) + El);
        sums[at.wave][at.lane] = make_float2(G, hl);
        backs[W - 1 - at.wave][at.lane] = make_float2(G, El);   // in the order of the walk back
    }
    // What needs the other waves' sums, and not yet what enters the tile from behind.
    __device__ __forceinline__ void gather(const Place<1>& at, const float2 (&sums)[W][kGsChannels],
                                           const float2 (&backs)[W][kGsChannels]) {
        float G = 0.0f, s = 0.0f;
        for (int w = 0; w < at.wave; ++w) append(G, s, sums[w][at.lane].x, sums[w][at.lane].y);
        float h = carried(state, G, s);
        Gw = hw = 0.0f;
        for (int w = 0; w < W - 1 - at.wave; ++w) append(Gw, hw, backs[w][at.lane].x, backs[w][at.lane].y);
        // ck becomes h_{t-1} - q x a / b
#pragma unroll
        for (int t = 0; t < T; ++t) {
            ck[t] = h - ck[t];
            h = fmaf(ca[t], h, cu[t]);
        }
    }
    // The gradients, from the adjoints entering the tile from behind. Returns the
    // wave's share of the decay's gradient.
    template <bool FULL>
    __device__ __forceinline__ float finish(const GatedScanArgs& a, const Place<1>& at, int64_t b, int64_t t0,
                                            int64_t left, In<FULL>& next, const float (&enter)[kGsChannels]) {
        typedef Rows<IO, 1, T, W, FULL> R;
        const int64_t first = b * a.seqlen + t0;
        float A = carried(enter[at.lane], Gw, hw), sum = 0.0f;
        state = next.state != nullptr ? *next.state : 0.0f;
        R ox(at, a.dx, first, a.dim, a.dim, a.seqlen - t0), od(at, a.ddecay, first, a.dim, a.dim, a.seqlen - t0),
            oi(at, a.dinput, first, a.dim, a.dim, a.seqlen - t0);
        ox.go(T - 1);
        next.dy.go(T - 1);
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            const float At = raw_to_f32<IO>(dy[t]) + A;
            A = ca[t] * At;
            const float dg = A * ck[t];
            sum = fmaf(dg, cp[t], sum);
            dy[t] = next.dy.load();
            next.dy.go(-1);
            ox.store({At * cw[t]});
            store_value<IO, 1>(od.rs, ox.at, ox.row, {dg * cgr[t]});
            if constexpr (GATED) store_value<IO, 1>(oi.rs, ox.at, ox.row, {At * cir[t]});
            ox.go(-1);
            token_fence(t);
        }
        if (!FULL && left < TILE) none(a, at, b, t0, live_tokens<T, TILE>(at.wave, left));
        return sum;
    }
    static __device__ __forceinline__ void none(const GatedScanArgs& a, const Place<1>& at, int64_t b, int64_t t0,
                                                int from) {
        typedef Rows<IO, 1, T, W, false> R;
        const int64_t first = b * a.seqlen + t0;
        R ox(at, a.dx, first, a.dim, a.dim, a.seqlen - t0), od(at, a.ddecay, first, a.dim, a.dim, a.seqlen - t0),
            oi(at, a.dinput, first, a.dim, a.dim, a.seqlen - t0);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            if (t >= from) {
                ox.store({0.0f});
                store_value<IO, 1>(od.rs, ox.at, ox.row, {0.0f});
                if constexpr (GATED) store_value<IO, 1>(oi.rs, ox.at, ox.row, {0.0f});
            }
            ox.go(1);
        }
    }
};

// The backward pass, a workgroup walking one row's tiles from the last to the
// first. The state entering a tile comes from the forward pass, a block's start at a
// time, so that nothing is walked twice. About 70 vector instructions a value keep the
// vector units busy for 59% of the time at 4 waves a SIMD: 8 x 2048 x 5120 in bf16 308
// us (3.8 TB/s), 8 x 2048 x 4096, where all columns run at once, 233 (4.1).
template <int IO, int T, int W, bool GATED>
__global__ __launch_bounds__(W* kWave) void gated_scan_bwd_kernel(GatedScanArgs a, int64_t groups,
                                                               float* partial) {
    typedef BwdTile<IO, T, W, GATED> Tile;
    __shared__ float2 sums[2][W][kGsChannels], backs[2][W][kGsChannels];
    __shared__ float enter[2][kGsChannels];
    const int64_t b = blockIdx.x / groups;
    const Place<1> at(a.dim, blockIdx.x - b * groups);
    const int64_t len = row_length(a.lengths, b, a.seqlen), live = (len + Tile::TILE - 1) / Tile::TILE;
    float lam2[1];
    uint32_t decays[1];
    load_log_decay(a, at, decays);
    log2_decay(decays, lam2);
    double dl = 0.0;
    if (at.wave == 0) enter[0][at.lane] = load_state(a.dhL, b, a.dim, at.ch);
    Tile tile;
    int64_t t0 = (live - 1) * Tile::TILE;
    if (live > 0) tile.load_all(typename Tile::template In<false>(a, at, b, t0, len - t0));
    int k = 0;
    auto step = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        const int odd = k & 1;
        typename Tile::template In<FULL> next(a, at, b, t0 - Tile::TILE, t0 > 0 ? Tile::TILE : 0);
        tile.template work<FULL>(at, lam2[0], len - t0, next, sums[odd], backs[odd]);
        __syncthreads();
        if (at.wave == k % W) {
            const float2 all = tile_sum<W>(backs[odd], at.lane);
            enter[odd ^ 1][at.lane] = carried(enter[odd][at.lane], all.x, all.y);
        }
        tile.gather(at, sums[odd], backs[odd]);
        dl += static_cast<double>(tile.template finish<FULL>(a, at, b, t0, len - t0, next, enter[odd]));
        t0 -= Tile::TILE;
        ++k;
    };
    if (t0 >= 0) step(std::false_type());
    while (t0 > 0) step(std::true_type());
    if (t0 == 0) step(std::false_type());
    __syncthreads();
    if (a.dh0 != nullptr && at.wave == 0 && at.in) a.dh0[b * a.dim + at.ch] = enter[k & 1][at.lane];
    if (partial != nullptr) {
        __shared__ double all[W][kGsChannels];
        all[at.wave][at.lane] = dl;
        __syncthreads();
        if (at.wave == 0 && at.in) {
            double s = 0.0;
#pragma unroll
            for (int q = 0; q < W; ++q) s += all[q][at.lane];
            partial[b * a.dim + at.ch] = static_cast<float>(s);
        }
    }
    for (t0 = live * Tile::TILE; t0 < a.seqlen; t0 += Tile::TILE) Tile::none(a, at, b, t0, 0);
}

// The backward pass as a chain (1 x 65536 x 1536 in bf16 415 us, of which the looks
// cost 60): position j of a row is its j-th tile from the last one with tokens.
// `partial` holds the decay's gradient of every (row, tile),
// zeros for tiles without tokens.
template <int IO, int T, int W, bool GATED>
__global__ __launch_bounds__(W* kWave) void gated_scan_bwd_chain_kernel(GatedScanArgs a, Chain ch,
                                                                     float* partial) {
    typedef BwdTile<IO, T, W, GATED> Tile;
    typedef typename Tile::template In<false> AnyIn;
    __shared__ float2 sums[2][W][kGsChannels], backs[2][W][kGsChannels];   // by turns, as forward
    __shared__ float enter[kGsChannels], shares[W][kGsChannels];
    __shared__ uint32_t taken[2];
    if (threadIdx.x == 0) {
        taken[0] = take_ticket(ch.ticket);
        taken[1] = ch.once ? kNoTicket : take_ticket(ch.ticket);
    }
    __syncthreads();
    Link at(ch, __builtin_amdgcn_readfirstlane(taken[0])), next(ch, __builtin_amdgcn_readfirstlane(taken[1]));
    __syncthreads();
    Tile tile;
    // a link's first token, -1 for one without tokens
    auto first_of = [&](const Link& l) {
        const int64_t len = row_length(a.lengths, l.b, a.seqlen);
        const int64_t t0 = ((len + Tile::TILE - 1) / Tile::TILE - 1 - static_cast<int64_t>(l.j)) * Tile::TILE;
        return l.any && t0 >= 0 ? t0 : int64_t(-1);
    };
    // The waves' shares of the decay's gradient are added up behind the next barrier.
    float* due = nullptr;
    auto put_share = [&](const Place<1>& place, int k) {
        if (due != nullptr && place.wave == k % W) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < W; ++q) s += shares[q][place.lane];
            *due = s;
        }
        due = nullptr;
    };
    auto left_of = [&](const Link& l, int64_t t0) {
        return t0 < 0 ? int64_t(0) : row_length(a.lengths, l.b, a.seqlen) - t0;
    };
    int64_t t0 = first_of(at);
    uint32_t decays[1], next_decays[1];   // as forward
    load_log_decay(a, Place<1>(a.dim, at.group), decays);
    tile.load_all(AnyIn(a, Place<1>(a.dim, at.group), at.b, t0, left_of(at, t0)));
    int k = 0;
    for (; at.any; ++k) {
        const Place<1> place(a.dim, at.group), next_place(a.dim, next.group);
        load_log_decay(a, next_place, next_decays);
        const int64_t b = at.b, left = left_of(at, t0), next_t0 = first_of(next), next_left = left_of(next, next_t0);
        uint32_t mine = kNoTicket;
        if (threadIdx.x == 0 && !ch.once) mine = take_ticket(ch.ticket);
        float* share = partial == nullptr || !place.in ? nullptr : partial + (b * ch.tiles + at.j) * a.dim + place.ch;
        if (left > 0) {
            AnyIn in(a, next_place, next.b, next_t0, next_left);
            float lam2[1];
            log2_decay(decays, lam2);
            tile.template work<false>(place, lam2[0], left, in, sums[k & 1], backs[k & 1]);
            __syncthreads();
            put_share(place, k + 1);   // a wave that has not to look for what enters the tile
            const bool looks = place.wave == k % W;
            if (looks) {
                const float2 all = tile_sum<W>(backs[k & 1], place.lane);
                float out;
                enter[place.lane] = enter_tile(ch, at, a.dim, place.ch, all.x, all.y, a.dhL, out);
                if (a.dh0 != nullptr && t0 == 0 && place.in) a.dh0[b * a.dim + place.ch] = out;
            }
            if (threadIdx.x == 0) taken[0] = mine;
            if (!looks) tile.gather(place, sums[k & 1], backs[k & 1]);   // while the other looks
            __syncthreads();
            if (looks) tile.gather(place, sums[k & 1], backs[k & 1]);
            shares[place.wave][place.lane] = tile.template finish<false>(a, place, b, t0, left, in, enter);
            due = share;
        } else {
            tile.load_all(AnyIn(a, next_place, next.b, next_t0, next_left));
            Tile::none(a, place, b, static_cast<int64_t>(at.j) * Tile::TILE, 0);
            if (at.j == 0 && a.dh0 != nullptr && place.wave == 0 && place.in)   // a row without tokens
                a.dh0[b * a.dim + place.ch] = load_state(a.dhL, b, a.dim, place.ch);
            if (share != nullptr && place.wave == 0) *share = 0.0f;
            __syncthreads();   // the ticket before this one has been read
            put_share(place, k + 1);
            if (threadIdx.x == 0) taken[0] = mine;
            __syncthreads();
        }
        at = next;
        t0 = next_t0;
        decays[0] = next_decays[0];
        next = Link(ch, __builtin_amdgcn_readfirstlane(taken[0]));
    }
    __syncthreads();
    put_share(Place<1>(a.dim, 0), 0);
}

// Without tokens: hL = h0, dh0 = dhL, no gradient of the decay. No other input is
// looked at, as none need be there.
__global__ __launch_bounds__(256) void gated_scan_empty_kernel(int64_t state, int64_t dim, const float* from,
                                                               float* to, float* zero) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < state || i < dim; i += stride) {
        if (to != nullptr && i < state) to[i] = from != nullptr ? from[i] : 0.0f;
        if (zero != nullptr && i < dim) zero[i] = 0.0f;
    }
}

constexpr int words_of(int io, int v) { return io == kIoF32 ? v : (v + 1) / 2; }

// One token: V channels to a lane, all loads out at once. 256 x 5120 in bf16 takes 5.9
// us, of the call's 9.1.
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
            const Decay1 e(sigmoid(d[v]), log2_of(lam.f[v]));
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

// The kernels' shapes: V channels to a lane, T tokens to a segment, W waves. A
// forward tile holds 2 values a token in registers, a backward tile 7, so segments
// are of 16 and 8 tokens where a workgroup walks a row: 8 x 2048 x 4096 in bf16 118
// us, of 8 (4 waves of 16) 126 (128); gradients 233, of 16 the same, 8 x 2048 x 5120
// 308 against 328. A chain's tile has a fixed cost, the look for what enters it, and
// waits are shorter the fewer tiles of a column are on their way, so its tiles are
// longer: 256 tokens where two channels fit a lane (1 x 262144 x 2048 960 us; of
// 128 tokens by 128 channels 1351, by 64 channels 1490), 128 for the gradients (1 x
// 65536 x 1536 415 us, of 64 540 to 615).
template <int IO_, int V_, int T_, int W_>
struct Shape {
    static constexpr int IO = IO_, V = V_, T = T_, W = W_, TILE = W * V * T;
};

template <int IO> using FwdWalk = Shape<IO, 1, 16, 8>;
template <int IO, int V> using FwdChain = Shape<IO, V, 16, 8>;
template <int IO> using BwdWalk = Shape<IO, 1, 8, 8>;
template <int IO> using BwdChain = Shape<IO, 1, 16, 8>;

// Channels to a lane of the forward chain.
int fwd_chain_channels(const GatedScanArgs& a) { return a.io == kIoBF16 && divides(a, 2) ? 2 : 1; }

constexpr int kFwdShortest = FwdChain<kIoF32, 1>::TILE;   // tokens of the shortest tile of a forward chain

int chain_tile(const GatedScanArgs& a, bool bwd) {
    return bwd ? BwdChain<kIoF32>::TILE : fwd_chain_channels(a) * kFwdShortest;
}

// Whether a call runs as a chain: by the times that either takes on MI355X, in
// microseconds. A walk's grows with the length of the sequences and, in bf16, where
// it is bound by issue, with the rounds of one column (a row's 64 channels) to a
// compute unit; in fp32, where it is bound by memory, with the columns. A chain's
// grows with the tokens of all columns, from what clearing its words costs. Of
// 2048 tokens in bf16, walk against chain: 32 columns 50 us against 17, 192 54
// against 58, 256 61 against 72, 384 107 against 101, 512 118 against 128, 640 165
// against 156; gradients 104 against 31, 116 against 114, 120 against 149, 198 against
// 215, 233 against 276, 308 against 344. In fp32 32 columns 47 against 22, 128 74
// against 60, 256 116 against 115, 512 217 against 202; gradients 99 against 36, 143
// against 112, 211 against 200, 412 against 357. Rows of different lengths are taken
// to hold three quarters of the longest, which a walk gains nothing from while all
// columns run at once (12 rows up to 3000 x 640 in bf16 74 us against 45, gradients 155
// against 81; all full 74 and 55, 156 and 111). Sequences of fewer than 4 tiles of
// 128 are walked (512 tokens of 192 columns: 16 us against 25), and so would be 2^26
// tiles, for which clearing the words would count 2^32 threads.
bool chained(const GatedScanArgs& a, bool bwd, bool ragged, int cu) {
    const double columns = static_cast<double>(a.batch * groups_of(a)), len = static_cast<double>(a.seqlen);
    if (a.seqlen < 512 || columns * (len / kFwdShortest + 1.0) >= 67108864.0) return false;
    const double part = ragged ? 0.75 : 1.0;
    const double each = columns * 256.0 / cu * part;   // as of 256 compute units
    double walk, chain;
    if (a.io == kIoBF16) {
        const double rounds = bwd ? fmax(1.0, columns / cu) : ceil(columns / cu);
        walk = (bwd ? 6.0 : 2.0) + len * (bwd ? 0.053 : 0.0255) * (1.0 + (rounds - 1.0) * part);
        chain = bwd ? 14.0 + len * each * 2.6e-4 : 14.0 + len * each * 1.1e-4;
    } else {
        walk = bwd ? 8.0 + len * fmax(0.04 + 1.9e-4 * each, 3.9e-4 * each)
                   : 3.0 + len * fmax(0.021 + 1.1e-4 * each, 2.1e-4 * each);
        chain = bwd ? 18.0 + len * each * 3.4e-4 : 12.0 + len * each * 1.9e-4;
    }
    return chain < walk;
}

bool chained(const GatedScanArgs& a, bool bwd, int cu) { return chained(a, bwd, a.lengths != nullptr, cu); }

// Whether any call of these sizes does.
bool may_chain(const GatedScanArgs& a, bool bwd, int cu) {
    return chained(a, bwd, false, cu) || chained(a, bwd, true, cu);
}

Chain chain_of(const GatedScanArgs& a, void* ws, bool bwd) {
    return Chain(ws, a.batch, a.seqlen, a.lengths, groups_of(a), chain_tile(a, bwd));
}

size_t chain_bytes(const Chain& ch) {
    return 256 + static_cast<size_t>(ch.words()) * sizeof(Word) + (static_cast<size_t>(ch.pairs) * 4 + 15) / 16 * 16;
}

// Of the backward pass, with a share of the decay's gradient for each row, or tile.
size_t bwd_bytes(const GatedScanArgs& a, bool chain, bool shares) {
    const size_t row = shares ? static_cast<size_t>(a.batch) * a.dim * sizeof(float) : 0;
    if (!chain) return row;
    const Chain ch = chain_of(a, nullptr, true);
    return chain_bytes(ch) + ch.tiles * row;
}

// Clears the chain's words; sets its grid: a workgroup for every tile up to two
// rounds of them (of 8 waves, one to a compute unit), else one for each unit.
hipError_t begin_chain(Chain& ch, int cu, unsigned* grid, hipStream_t s) {
    const int64_t total = static_cast<int64_t>(ch.pairs) * ch.groups;
    ch.once = total <= 2 * static_cast<int64_t>(cu);
    *grid = static_cast<unsigned>(ch.once ? total : cu);
    hipLaunchKernelGGL(gated_scan_clear_kernel, dim3(static_cast<unsigned>((ch.words() / 2 + 255) / 256)), dim3(256), 0,
                       s, ch);
    return hipGetLastError();
}

template <typename S, bool GATED>
hipError_t launch_fwd_chain(const GatedScanArgs& a, int cu, void* ws, hipStream_t s) {
    Chain ch = chain_of(a, ws, false);
    unsigned grid = 0;
    const hipError_t e = begin_chain(ch, cu, &grid, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gated_scan_fwd_chain_kernel<S::IO, S::V, S::T, S::W, GATED>), dim3(grid), dim3(S::W * kWave),
                       0, s, a, ch);
    return hipGetLastError();
}

template <int IO, bool GATED>
hipError_t launch_fwd(const GatedScanArgs& a, int cu, void* ws, hipStream_t s) {
    if (chained(a, false, cu)) {
        if constexpr (IO == kIoBF16)
            if (fwd_chain_channels(a) == 2) return launch_fwd_chain<FwdChain<IO, 2>, GATED>(a, cu, ws, s);
        return launch_fwd_chain<FwdChain<IO, 1>, GATED>(a, cu, ws, s);
    }
    typedef FwdWalk<IO> S;
    const int64_t groups = groups_of(a);
    hipLaunchKernelGGL((gated_scan_fwd_kernel<S::IO, S::V, S::T, S::W, GATED>),
                       dim3(static_cast<unsigned>(a.batch * groups)), dim3(S::W * kWave), 0, s, a, groups);
    return hipGetLastError();
}

template <int IO, bool GATED>
hipError_t launch_bwd(const GatedScanArgs& a, int cu, void* ws, hipStream_t s) {
    hipError_t e;
    if (chained(a, true, cu)) {
        typedef BwdChain<IO> S;
        Chain ch = chain_of(a, ws, true);
        unsigned grid = 0;
        float* partial = a.dlog_decay == nullptr
                             ? nullptr
                             : reinterpret_cast<float*>(static_cast<char*>(ws) + chain_bytes(ch));
        e = begin_chain(ch, cu, &grid, s);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((gated_scan_bwd_chain_kernel<S::IO, S::T, S::W, GATED>), dim3(grid), dim3(S::W * kWave), 0,
                           s, a, ch, partial);
        e = hipGetLastError();
        if (e != hipSuccess || partial == nullptr) return e;
        return launch_column_sums(a.dim, a.batch * ch.tiles, partial, a.dlog_decay, nullptr, s);
    }
    typedef BwdWalk<IO> S;
    const int64_t groups = groups_of(a);
    float* partial = a.dlog_decay != nullptr ? static_cast<float*>(ws) : nullptr;
    hipLaunchKernelGGL((gated_scan_bwd_kernel<S::IO, S::T, S::W, GATED>),
                       dim3(static_cast<unsigned>(a.batch * groups)), dim3(S::W * kWave), 0, s, a, groups, partial);
    e = hipGetLastError();
    if (e != hipSuccess || partial == nullptr) return e;
    return launch_column_sums(a.dim, a.batch, partial, a.dlog_decay, nullptr, s);
}

template <int IO, int V>
hipError_t launch_update(const GatedScanArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((gated_scan_update_kernel<IO, V>),
                       dim3(static_cast<unsigned>(stride_blocks(a.batch * (a.dim / V)))), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_empty(int64_t state, int64_t dim, const float* from, float* to, float* zero, hipStream_t s) {
    hipLaunchKernelGGL(gated_scan_empty_kernel, dim3(static_cast<unsigned>(stride_blocks(state > dim ? state : dim))),
                       dim3(256), 0, s, state, dim, from, to, zero);
    return hipGetLastError();
}

}  // namespace

// Without regard to the strides and to whether rows differ in length, which are not
// known when the scratch is asked for: that of the shortest tiles a chain may take.
size_t gated_scan_fwd_workspace_bytes(const GatedScanArgs& a, int cu) {
    if (!may_chain(a, false, cu)) return 0;
    return chain_bytes(Chain(nullptr, a.batch, a.seqlen, nullptr, groups_of(a), kFwdShortest));
}

size_t gated_scan_bwd_workspace_bytes(const GatedScanArgs& a, int cu) {
    return bwd_bytes(a, may_chain(a, true, cu), true);
}

// What a call uses of it.
size_t gated_scan_bwd_needed_bytes(const GatedScanArgs& a, int cu) {
    return bwd_bytes(a, chained(a, true, cu), a.dlog_decay != nullptr);
}

hipError_t launch_gated_scan_fwd(const GatedScanArgs& a, int cu, void* ws, hipStream_t s) {
    if (a.seqlen == 0) return launch_empty(a.batch * a.dim, a.dim, a.h0, a.hL, nullptr, s);
    if (a.io == kIoF32)
        return a.input_gate != nullptr ? launch_fwd<kIoF32, true>(a, cu, ws, s) : launch_fwd<kIoF32, false>(a, cu, ws, s);
    return a.input_gate != nullptr ? launch_fwd<kIoBF16, true>(a, cu, ws, s) : launch_fwd<kIoBF16, false>(a, cu, ws, s);
}

hipError_t launch_gated_scan_bwd(const GatedScanArgs& a, int cu, void* ws, hipStream_t s) {
    if (a.batch == 0 || a.seqlen == 0) return launch_empty(a.batch * a.dim, a.dim, a.dhL, a.dh0, a.dlog_decay, s);
    if (a.io == kIoF32)
        return a.input_gate != nullptr ? launch_bwd<kIoF32, true>(a, cu, ws, s) : launch_bwd<kIoF32, false>(a, cu, ws, s);
    return a.input_gate != nullptr ? launch_bwd<kIoBF16, true>(a, cu, ws, s) : launch_bwd<kIoBF16, false>(a, cu, ws, s);
}

hipError_t launch_gated_scan_update(const GatedScanArgs& a, hipStream_t s) {
    if (a.io == kIoF32) return divides(a, 4) ? launch_update<kIoF32, 4>(a, s) : launch_update<kIoF32, 1>(a, s);
    return divides(a, 4) ? launch_update<kIoBF16, 4>(a, s) : launch_update<kIoBF16, 1>(a, s);
}

}  // namespace mamba
