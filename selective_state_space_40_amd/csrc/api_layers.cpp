// C ABI of linear attention and layer norm (mamba_layers.h): argument checks,
// the automatic plans and error mapping around linear_attn.hip,
// linear_attn_variant.hip and layer_norm.hip. Every check runs on the host
// before any launch; the compute-unit query of the automatic plans is the
// only HIP call made before the arguments are known to be good.
#include <hip/hip_runtime_api.h>

#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "mamba_layers.h"

namespace {

using mamba::LinearAttnCall;
using mamba::LinPlan;

static_assert(mamba::kLinMaxDim == MAMBA_LINATTN_MAX_DIM && mamba::kLinMaxHeads == MAMBA_LINATTN_MAX_HEADS,
              "limits of heads");
static_assert(mamba::kNormMaxDim == MAMBA_NORM_MAX_DIM, "widest part of a norm");

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool known_dtype(int dtype) { return dtype == MAMBA_DTYPE_F32 || dtype == MAMBA_DTYPE_BF16; }

int io_of(int dtype) { return dtype == MAMBA_DTYPE_F32 ? mamba::kIoF32 : mamba::kIoBF16; }

template <int N>
int check_aligned(const void* const (&ptrs)[N]) {
    for (const void* p : ptrs)
        if (p != nullptr && !aligned16(p)) return MAMBA_ERR_MISALIGNED;
    return MAMBA_OK;
}

// Tokens per chunk of the widest-chunked kernel: segments are whole chunks of it.
constexpr int64_t kSegUnit = 64;
// Threads that a launch counts (32 bits), elements of a tensor, rows times
// groups and channels of a norm.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
constexpr int64_t kMaxParts = int64_t(1) << 30;
constexpr int64_t kMaxChannels = int64_t(1) << 27;
constexpr int64_t kMaxElems = int64_t(1) << 48;

int check_attn(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads, int64_t dk, int64_t dv,
               int dtype, int64_t segment_len) {
    if (batch < 0 || seqlen < 0 || heads < 0 || kv_heads < 0 || dk < 1 || dv < 1 || segment_len < 0)
        return MAMBA_ERR_INVALID_ARG;
    if (!known_dtype(dtype) || segment_len % kSegUnit != 0) return MAMBA_ERR_INVALID_ARG;
    if (heads > 0 ? (kv_heads == 0 || heads % kv_heads != 0) : kv_heads != 0) return MAMBA_ERR_INVALID_ARG;
    if (dk > MAMBA_LINATTN_MAX_DIM || dv > MAMBA_LINATTN_MAX_DIM || dk % MAMBA_LINATTN_DIM_UNIT != 0 ||
        dv % MAMBA_LINATTN_DIM_UNIT != 0 || heads > MAMBA_LINATTN_MAX_HEADS)
        return MAMBA_ERR_UNSUPPORTED;
    if (batch > (int64_t(1) << 24) || seqlen > kMaxElems / (MAMBA_LINATTN_MAX_HEADS * MAMBA_LINATTN_MAX_DIM))
        return MAMBA_ERR_UNSUPPORTED;
    if (batch > 0 && seqlen > 0 &&
        seqlen > kMaxElems / (int64_t(MAMBA_LINATTN_MAX_HEADS) * MAMBA_LINATTN_MAX_DIM) / batch)
        return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The automatic division. Segments add a pass over keys and values and a
// join, so a sequence is cut only where its chunks, walked one after the other,
// would leave the chip idle. The time of a plan with n segments is taken as
//     (chunks / n * chunk + entry) * load * (n > 1 ? 1 + summary : 1) + (n > 1 ? join : 0)
// with `chunk` the time of 64 tokens alone on a compute unit, `entry` a
// workgroup's beginning and end, `summary` the states' pass, `join` its launches
// and `load` what sharing the chip costs: a second workgroup on a unit makes a
// round 1.57 times as long, a third waits for the next; of the wide kernels a
// unit holds one. The backward's pass of dq, where the decay's gradient is
// formed, takes `longest` for 64 tokens and goes first, the other two passes
// run beside and behind it (whether that gradient is wanted is not known here).
// Microseconds measured on MI355X with one workgroup per unit; examples, cut
// by this rule against not cut: one sequence of 65536, 16 heads of 128: 365 us
// with 16 segments against 1.79 ms; 8 x 2048 x 16 heads of 128: 73 us whole
// against 103 with 2, gradients 255 whole against 314 with 2; 4 x 1024 x 16
// heads of 64: 27 us whole against 31 with 2, gradients 53 with 4 against 66;
// gradients in fp32 of 2 x 333 x 6 heads: 36 us with 6 against 71; 2 x 2048 x
// 8 heads of 200 x 168: 53 us with 5 against 98, gradients 171 as cut, 156 with 2,
// 222 whole.
struct PlanCost {
    double chunk[2][3];   // [fp32, bf16][head width 64, 128, 256]
    double entry[3];
    double summary;
};
constexpr PlanCost kFwdCost = {{{4.4, 8.0, 10.8}, {1.45, 2.3, 2.75}}, {2.0, 3.0, 9.0}, 0.5};
constexpr PlanCost kBwdCost = {{{4.3, 6.7, 11.0}, {1.95, 2.6, 3.0}}, {2.0, 3.0, 5.0}, 0.35};
constexpr double kBwdLongest[2][3] = {{7.5, 13.0, 19.5}, {3.6, 5.3, 6.6}};
constexpr double kJoinCost = 14.0, kLaunchCost = 4.0, kSharedUnit = 1.57;
constexpr int64_t kMinSegment = 64;

int width_class(int d) { return mamba::lin_padded(d) == 64 ? 0 : (mamba::lin_padded(d) == 128 ? 1 : 2); }

// Microseconds of a pass cut into n segments, without those of the cut: `each`
// runs of 64 tokens per workgroup, of which `walk` is the longest.
double fwd_time(const LinearAttnCall& c, int64_t n, double each, int cu) {
    const int type = c.io == mamba::kIoF32 ? 0 : 1, w = width_class(c.dk);
    const int64_t all = c.batch * c.heads * mamba::lin_blocks(c.dv) * n;
    const int64_t round = w == 2 ? cu : 2 * int64_t(cu), rest = all % round;
    const double load = static_cast<double>(all / round) * (w == 2 ? 1.0 : kSharedUnit) +
                        (rest == 0 ? 0.0 : (rest <= cu ? 1.0 : kSharedUnit));
    return (each * kFwdCost.chunk[type][w] + kFwdCost.entry[w]) * load;
}

// One launch of gradients at width class w: `dq` and `others` workgroups per
// segment of the pass of dq and of the other passes.
double bwd_launch_time(int type, int w, int64_t dq, int64_t others, int64_t n, double each, int cu) {
    const double chunk = kBwdCost.chunk[type][w], longest = dq > 0 ? kBwdLongest[type][w] : chunk;
    const double work = (longest * static_cast<double>(dq) + chunk * static_cast<double>(others)) *
                        static_cast<double>(n) / cu;
    const double alone = w == 2 || (dq + others) * n <= cu ? 1.0 : 1.3;   // beside shorter ones
    double load = work / longest * (w == 2 ? 1.0 : kSharedUnit / 2);
    if (load < alone) load = alone;
    return (each * longest + kBwdCost.entry[w]) * load;
}

// The gradients in one launch, at the wider head's width, or in two: dq and dk
// contract over dv, dv over dk. Two launches save what a narrow head wastes at
// a wide one's width, one lets all passes run beside each other: fp32, 9 x 202 x
// 12 heads of 232 x 16, 126 us in two against 287; 2 x 333 x 6 heads of 64 x 96,
// 39 us in one.
double bwd_time(const LinearAttnCall& c, int64_t n, double each, int cu, bool* two) {
    const int type = c.io == mamba::kIoF32 ? 0 : 1, wk = width_class(c.dk), wv = width_class(c.dv);
    const int64_t bh = c.batch * c.heads, over_k = bh * mamba::lin_blocks(c.dk), over_v = bh * mamba::lin_blocks(c.dv);
    const double one = bwd_launch_time(type, wk > wv ? wk : wv, over_k, over_k + over_v, n, each, cu);
    const double both = bwd_launch_time(type, wv, over_k, over_k, n, each, cu) +
                        bwd_launch_time(type, wk, 0, over_v, n, each, cu) + kLaunchCost;
    *two = wk != wv && both < one;
    return *two ? both : one;
}

double runs_of_64(int64_t seqlen, int64_t n) {
    const double each = static_cast<double>(ceil_div(ceil_div(seqlen, n), kSegUnit));
    const double whole = static_cast<double>(seqlen) / 64.0;
    return each < whole ? each : whole;
}

int64_t choose_segments(const LinearAttnCall& c, bool bwd, int cu) {
    const int64_t bh = c.batch * c.heads;
    const int64_t all = bwd ? bh * (2 * mamba::lin_blocks(c.dk) + mamba::lin_blocks(c.dv))
                            : bh * mamba::lin_blocks(c.dv);
    int64_t best = 1;
    double least = 0.0;
    for (int64_t n = 1; n <= ceil_div(c.seqlen, kMinSegment) && (n == 1 || all * n <= 8 * int64_t(cu)); ++n) {
        const double each = runs_of_64(c.seqlen, n);
        bool two;
        double t = bwd ? bwd_time(c, n, each, cu, &two) : fwd_time(c, n, each, cu);
        if (n > 1) t = t * (1.0 + (bwd ? kBwdCost : kFwdCost).summary) + kJoinCost;
        if (n == 1 || t < least) {
            least = t;
            best = n;
        }
    }
    return best;
}

// How a call is divided. `passes` workgroups run per (row, head, segment,
// column block): one forward, three backward, whose wider head decides.
int make_attn_plan(const LinearAttnCall& c, int passes, int64_t segment_len, LinPlan* p) {
    const int wide = passes == 1 ? c.dv : (c.dk > c.dv ? c.dk : c.dv);
    const int dc_pad = mamba::lin_padded(passes == 1 ? c.dk : wide);
    const int64_t blocks = mamba::lin_blocks(wide);
    p->seg_len = c.seqlen > 0 ? c.seqlen : 1;
    p->nseg = 1;
    if (c.batch == 0 || c.heads == 0) return MAMBA_OK;
    int64_t seg = segment_len;
    if (seg == 0 && c.seqlen > 0) {
        int cu = 0;
        const int st = mamba::current_cu_count(&cu);
        if (st != MAMBA_OK) return st;
        const int64_t n = choose_segments(c, passes > 1, cu);
        seg = n > 1 ? ceil_div(ceil_div(c.seqlen, n), kSegUnit) * kSegUnit : c.seqlen;
    }
    if (seg < c.seqlen) {
        const int64_t n = ceil_div(c.seqlen, seg);
        if (n > (int64_t(1) << 16)) return MAMBA_ERR_UNSUPPORTED;
        p->seg_len = seg;
        p->nseg = static_cast<int>(n);
    }
    const int64_t threads = passes * blocks * mamba::lin_waves(dc_pad) * mamba::kWave;
    if (c.batch * c.heads * p->nseg > kMaxThreads / threads) return MAMBA_ERR_UNSUPPORTED;
    // the join's launch holds (row, head) in a 16-bit grid dimension; the automatic
    // division cuts calls of a few per compute unit only
    if (p->nseg > 1 && c.batch * c.heads > 65535) return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

LinearAttnCall attn_call(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads, int64_t dk,
                         int64_t dv, int dtype) {
    LinearAttnCall c = {};
    c.batch = batch;
    c.seqlen = seqlen;
    c.heads = static_cast<int>(heads);
    c.kv_heads = static_cast<int>(kv_heads);
    c.dk = static_cast<int>(dk);
    c.dv = static_cast<int>(dv);
    c.io = io_of(dtype);
    return c;
}

int attn_workspace(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads, int64_t dk, int64_t dv,
                   int dtype, int64_t segment_len, int passes, size_t* bytes) {
    if (bytes == nullptr) return MAMBA_ERR_INVALID_ARG;
    int st = check_attn(batch, seqlen, heads, kv_heads, dk, dv, dtype, segment_len);
    if (st != MAMBA_OK) return st;
    const LinearAttnCall c = attn_call(batch, seqlen, heads, kv_heads, dk, dv, dtype);
    LinPlan p;
    st = make_attn_plan(c, passes, segment_len, &p);
    if (st != MAMBA_OK) return st;
    *bytes = mamba::linear_attn_workspace_bytes(c, p, passes > 1);
    return MAMBA_OK;
}

int check_norm(int64_t rows, int64_t dim, int64_t groups, int dtype) {
    if (rows < 0 || dim < 0 || groups < 1 || !known_dtype(dtype) || dim % groups != 0)
        return MAMBA_ERR_INVALID_ARG;
    if (dim / groups > MAMBA_NORM_MAX_DIM) return MAMBA_ERR_UNSUPPORTED;
    if (dim > kMaxChannels || groups > kMaxChannels / 32 || (dim > 0 && rows > kMaxElems / dim) ||
        rows > kMaxParts / groups)
        return MAMBA_ERR_UNSUPPORTED;
    return MAMBA_OK;
}

}  // namespace

extern "C" {

int linear_attn_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                                   int64_t dk, int64_t dv, int dtype, int64_t segment_len,
                                   size_t* bytes) {
    return attn_workspace(batch, seqlen, heads, kv_heads, dk, dv, dtype, segment_len, 1, bytes);
}

int linear_attn_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                                   int64_t dk, int64_t dv, int dtype, int64_t segment_len,
                                   size_t* bytes) {
    return attn_workspace(batch, seqlen, heads, kv_heads, dk, dv, dtype, segment_len, 3, bytes);
}

int linear_attn_fwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads, int64_t dk,
                    int64_t dv, int dtype, const void* q, const void* k, const void* v,
                    const float* log_decay, const int32_t* lengths, const float* h0, float scale,
                    void* o, float* hL, int64_t segment_len, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
    int st = check_attn(batch, seqlen, heads, kv_heads, dk, dv, dtype, segment_len);
    if (st != MAMBA_OK) return st;
    if (batch == 0 || heads == 0) return MAMBA_OK;
    if (log_decay == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (seqlen > 0 && (q == nullptr || k == nullptr || v == nullptr || o == nullptr))
        return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {q, k, v, log_decay, lengths, h0, o, hL, workspace};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    if (seqlen == 0 && hL == nullptr) return MAMBA_OK;
    LinearAttnCall c = attn_call(batch, seqlen, heads, kv_heads, dk, dv, dtype);
    LinPlan p;
    st = make_attn_plan(c, 1, segment_len, &p);
    if (st != MAMBA_OK) return st;
    const size_t need = mamba::linear_attn_workspace_bytes(c, p, false);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    c.scale = scale;
    c.q = q;
    c.k = k;
    c.v = v;
    c.log_decay = log_decay;
    c.lengths = lengths;
    c.h0 = h0;
    c.o = o;
    c.hL = hL;
    return mamba::launch_linear_attn_fwd(c, p, workspace, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int linear_attn_bwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads, int64_t dk,
                    int64_t dv, int dtype, const void* q, const void* k, const void* v,
                    const float* log_decay, const int32_t* lengths, const float* h0, float scale,
                    const void* d_o, const float* dhL, void* dq, void* d_k, void* d_v,
                    float* dlog_decay, float* dh0, int64_t segment_len, void* workspace,
                    size_t workspace_bytes, hipStream_t stream) {
    int st = check_attn(batch, seqlen, heads, kv_heads, dk, dv, dtype, segment_len);
    if (st != MAMBA_OK) return st;
    if (heads == 0) return MAMBA_OK;
    if (log_decay == nullptr) return MAMBA_ERR_INVALID_ARG;
    if (batch > 0 && seqlen > 0 &&
        (q == nullptr || k == nullptr || v == nullptr || d_o == nullptr || dq == nullptr || d_k == nullptr ||
         d_v == nullptr))
        return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {q, k, v, log_decay, lengths, h0, d_o, dhL, dq, d_k, d_v, dlog_decay, dh0,
                                workspace};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    LinearAttnCall c = attn_call(batch, seqlen, heads, kv_heads, dk, dv, dtype);
    LinPlan p;
    st = make_attn_plan(c, 3, segment_len, &p);
    if (st != MAMBA_OK) return st;
    const size_t need = mamba::linear_attn_workspace_bytes(c, p, true);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    c.scale = scale;
    c.q = q;
    c.k = k;
    c.v = v;
    c.log_decay = log_decay;
    c.lengths = lengths;
    c.h0 = h0;
    c.d_o = d_o;
    c.dhL = dhL;
    c.dq = dq;
    c.d_k = d_k;
    c.d_v = d_v;
    c.dlog_decay = dlog_decay;
    c.dh0 = dh0;
    if (batch > 0 && seqlen > 0 && mamba::lin_padded(c.dk) != mamba::lin_padded(c.dv)) {
        int cu = 0;
        st = mamba::current_cu_count(&cu);
        if (st != MAMBA_OK) return st;
        bwd_time(c, p.nseg, runs_of_64(seqlen, p.nseg), cu, &p.two);
    }
    return mamba::launch_linear_attn_bwd(c, p, workspace, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int linear_attn_update(int64_t batch, int64_t heads, int64_t kv_heads, int64_t dk, int64_t dv,
                       int dtype, float* h, const void* q, const void* k, const void* v,
                       const float* log_decay, float scale, void* o, hipStream_t stream) {
    int st = check_attn(batch, 1, heads, kv_heads, dk, dv, dtype, 0);
    if (st != MAMBA_OK) return st;
    if (batch == 0 || heads == 0) return MAMBA_OK;
    if (h == nullptr || q == nullptr || k == nullptr || v == nullptr || log_decay == nullptr || o == nullptr)
        return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {h, q, k, v, log_decay, o};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    if (batch * heads > kMaxThreads / (mamba::lin_blocks(static_cast<int>(dv)) * mamba::kLinUpdateThreads))
        return MAMBA_ERR_UNSUPPORTED;
    mamba::LinUpdateArgs a = {};
    a.batch = batch;
    a.heads = static_cast<int>(heads);
    a.kv_heads = static_cast<int>(kv_heads);
    a.dk = static_cast<int>(dk);
    a.dv = static_cast<int>(dv);
    a.io = io_of(dtype);
    a.scale = scale;
    a.h = h;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.o = o;
    return mamba::launch_linear_attn_update(a, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int layer_norm_fwd(int64_t rows, int64_t dim, int64_t groups, int dtype, const void* x,
                   const float* weight, const float* bias, float eps, void* y, float* mean,
                   float* rstd, hipStream_t stream) {
    int st = check_norm(rows, dim, groups, dtype);
    if (st != MAMBA_OK) return st;
    if (!(eps >= 0.0f) || !isfinite(eps)) return MAMBA_ERR_INVALID_ARG;
    if (rows == 0 || dim == 0) return MAMBA_OK;
    if (x == nullptr || y == nullptr) return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {x, weight, bias, y, mean, rstd};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    mamba::NormArgs a = {};
    a.rows = rows;
    a.dim = dim;
    a.groups = groups;
    a.io = io_of(dtype);
    a.eps = eps;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    return mamba::launch_layer_norm_fwd(a, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int layer_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups, int dtype,
                                  size_t* bytes) {
    if (bytes == nullptr) return MAMBA_ERR_INVALID_ARG;
    int st = check_norm(rows, dim, groups, dtype);
    if (st != MAMBA_OK) return st;
    *bytes = 0;
    if (rows == 0 || dim == 0) return MAMBA_OK;
    int cu = 0;
    st = mamba::current_cu_count(&cu);
    if (st != MAMBA_OK) return st;
    *bytes = mamba::layer_norm_bwd_workspace_bytes(rows, dim, groups, cu);
    return MAMBA_OK;
}

int layer_norm_bwd(int64_t rows, int64_t dim, int64_t groups, int dtype, const void* x,
                   const float* weight, const float* mean, const float* rstd, const void* dy,
                   void* dx, float* dweight, float* dbias, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
    int st = check_norm(rows, dim, groups, dtype);
    if (st != MAMBA_OK) return st;
    if (dim == 0) return MAMBA_OK;
    if (rows > 0 && (x == nullptr || mean == nullptr || rstd == nullptr || dy == nullptr || dx == nullptr))
        return MAMBA_ERR_INVALID_ARG;
    const void* const ptrs[] = {x, weight, mean, rstd, dy, dx, dweight, dbias, workspace};
    st = check_aligned(ptrs);
    if (st != MAMBA_OK) return st;
    int cu = 1;
    if (rows > 0) {
        st = mamba::current_cu_count(&cu);
        if (st != MAMBA_OK) return st;
        const size_t need = mamba::layer_norm_bwd_workspace_bytes(rows, dim, groups, cu);
        if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    } else if (dweight == nullptr && dbias == nullptr) {
        return MAMBA_OK;
    }
    mamba::NormArgs a = {};
    a.rows = rows;
    a.dim = dim;
    a.groups = groups;
    a.io = io_of(dtype);
    a.x = x;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    return mamba::launch_layer_norm_bwd(a, cu, workspace, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
