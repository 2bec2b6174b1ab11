// C ABI of the operators on tokens (include/mdcn.h): argument validation and
// dispatch. No exception leaves this file; every entry point returns an
// mdcn_status.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mdcn.h"
#include "mdcn_api.h"
#include "mdcn_attention.h"
#include "mdcn_plan.h"
#include "mdcn_rotary.h"

namespace {

constexpr int64_t kI31 = (int64_t(1) << 31) - 1;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(mdcn_dtype t) { return t == MDCN_F32 || t == MDCN_F16 || t == MDCN_BF16; }
int64_t size_of(mdcn_dtype t) { return t == MDCN_F32 ? 4 : 2; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Strides of an index that has more than one value: positive and below 2^31.
mdcn_status strides_ok(const mdcn_strides& s, int64_t tokens, int64_t heads) {
    if ((tokens > 1 && s.token < 1) || (heads > 1 && s.head < 1)) return MDCN_ERR_SHAPE;
    if ((tokens > 1 && s.token > kI31) || (heads > 1 && s.head > kI31)) return MDCN_ERR_UNSUPPORTED;
    return MDCN_OK;
}

// A stride as the kernels use it: that of an index of extent 1 is never used.
int64_t used(int64_t stride, int64_t extent) { return extent > 1 ? stride : 0; }

bool on16(const mdcn_strides& s, int64_t tokens, int64_t heads, int64_t size) {
    return used(s.token, tokens) * size % 16 == 0 && used(s.head, heads) * size % 16 == 0;
}

// ---------------------------------------------------------------- rotary
// Heads of q and k together at most: the kernels count a token's heads in 32
// bits, and round them up to whole shares of whole warps (32 rows for each of
// the 16 warps to an SM that may share a token) with some rows more ahead.
constexpr int64_t kRotaryHeads = kI31 + 1 - (int64_t(1) << 17);

mdcn_status rotary_check(const mdcn_rotary_attrs* at, const mdcn_rotary_dims* d, mdcn_dtype dtype, bool backward) {
    if (!at || !d) return MDCN_ERR_NULL;
    if (at->layout < 0 || at->layout > 2 || at->norm < 0 || at->norm > 1 || !(at->eps >= 0.0f) || !std::isfinite(at->eps))
        return MDCN_ERR_ATTR;
    if (!dtype_ok(dtype)) return MDCN_ERR_DTYPE;
    if (d->tokens < 0 || d->q_heads < 1 || d->k_heads < 0 || d->head_dim < 1 || d->axes < 1 || d->axes > 4)
        return MDCN_ERR_SHAPE;
    if (d->tokens > kI31 || d->q_heads > kRotaryHeads || d->k_heads > kRotaryHeads ||
        d->q_heads + d->k_heads > kRotaryHeads || d->head_dim > 256 || d->head_dim % 8 != 0)
        return MDCN_ERR_UNSUPPORTED;
    int64_t pairs = 0;
    for (int a = 0; a < 4; ++a) {
        if (d->sections[a] < 0 || d->sections[a] > d->head_dim || (a >= d->axes && d->sections[a] != 0))
            return MDCN_ERR_SHAPE;
        pairs += d->sections[a];
    }
    if (2 * pairs > d->head_dim) return MDCN_ERR_SHAPE;
    const mdcn_strides* qs[] = {&d->q, &d->q_out, &d->q_grad};
    const mdcn_strides* ks[] = {&d->k, &d->k_out, &d->k_grad};
    for (int i = 0; i < (backward ? 3 : 2); ++i) {
        if (i == 0 && backward && !at->norm) continue;  // x is not read
        mdcn_status s = strides_ok(*qs[i], d->tokens, d->q_heads);
        if (s == MDCN_OK && d->k_heads > 0) s = strides_ok(*ks[i], d->tokens, d->k_heads);
        if (s != MDCN_OK) return s;
    }
    return MDCN_OK;
}

mdcn::RotaryTensor tensor(const void* p, const mdcn_strides& s, int64_t tokens, int64_t heads) {
    return {const_cast<void*>(p), used(s.token, tokens), used(s.head, heads)};
}

mdcn::RotaryArgs rotary_args(const mdcn_rotary_attrs& at, const mdcn_rotary_dims& d) {
    mdcn::RotaryArgs a{};
    a.tokens = static_cast<int32_t>(d.tokens);
    a.hq = static_cast<int32_t>(d.q_heads);
    a.rows = static_cast<int32_t>(d.q_heads + d.k_heads);
    a.D = static_cast<int32_t>(d.head_dim);
    a.axes = static_cast<int32_t>(d.axes);
    for (int i = 0; i < 4; ++i) {
        a.pairs += static_cast<int32_t>(d.sections[i]);
        a.sec_end[i] = a.pairs;
    }
    a.layout = at.layout;
    a.norm = at.norm;
    a.eps = at.eps;
    return a;
}

// Whether every row starts on 16 bytes; MDCN_ERR_ALIGN where one is off its type.
mdcn_status rotary_align(const mdcn_rotary_dims& d, mdcn_dtype dtype, const void* const* p, const mdcn_strides* const* s,
                         const int64_t* heads, int n, int32_t* vec) {
    const int64_t size = size_of(dtype);
    *vec = 1;
    for (int i = 0; i < n; ++i) {
        if (!p[i]) continue;
        if (reinterpret_cast<uintptr_t>(p[i]) % static_cast<uintptr_t>(size) != 0) return MDCN_ERR_ALIGN;
        if (!aligned16(p[i]) || !on16(*s[i], d.tokens, heads[i], size)) *vec = 0;
    }
    return MDCN_OK;
}

size_t rotary_ws(const mdcn_rotary_dims& d) {
    return static_cast<size_t>(mdcn::kRotaryMaxBlocks) * 2 * static_cast<size_t>(d.head_dim) * sizeof(float);
}

// ---------------------------------------------------------------- attention
mdcn_status attn_check(const mdcn_attention_attrs* at, const mdcn_attention_dims* d, mdcn_dtype dtype, bool backward) {
    if (!at || !d) return MDCN_ERR_NULL;
    if (at->causal < 0 || at->causal > 1 || !std::isfinite(at->scale)) return MDCN_ERR_ATTR;
    if (!dtype_ok(dtype)) return MDCN_ERR_DTYPE;
    if (d->batch < 0 || d->q_tokens < 0 || d->k_tokens < 0 || d->q_heads < 1 || d->k_heads < 1 || d->head_dim < 1 ||
        d->q_heads % d->k_heads != 0)
        return MDCN_ERR_SHAPE;
    if (d->batch == 0 && (d->q_tokens > 0 || d->k_tokens > 0)) return MDCN_ERR_SHAPE;
    if (d->batch >= kI31 || d->q_tokens > kI31 - 256 || d->k_tokens > kI31 - 256 || d->head_dim > 128 ||
        d->head_dim % 8 != 0 || d->q_heads / d->k_heads > mdcn::kAttnSimtRows || d->k_heads > 65535 ||
        d->q_tokens > (int64_t(1) << 34) / d->q_heads)
        return MDCN_ERR_UNSUPPORTED;
    const mdcn_strides* qs[] = {&d->q, &d->out, &d->grad_out, &d->grad_q};
    const mdcn_strides* ks[] = {&d->k, &d->v, &d->grad_k, &d->grad_v};
    const int nq = backward ? 4 : 2, nk = backward ? 4 : 2;
    for (int i = 0; i < nq; ++i) {
        const mdcn_status s = strides_ok(*qs[i], d->q_tokens, d->q_heads);
        if (s != MDCN_OK) return s;
    }
    for (int i = 0; i < nk; ++i) {
        const mdcn_status s = strides_ok(*ks[i], d->k_tokens, d->k_heads);
        if (s != MDCN_OK) return s;
    }
    for (int i = 0; i < nq; ++i)
        if (!on16(*qs[i], d->q_tokens, d->q_heads, size_of(dtype))) return MDCN_ERR_ALIGN;
    for (int i = 0; i < nk; ++i)
        if (!on16(*ks[i], d->k_tokens, d->k_heads, size_of(dtype))) return MDCN_ERR_ALIGN;
    return MDCN_OK;
}

// The forward's plan: row tiles, and between how many blocks a tile's keys are
// shared out. Estimated in steps (one key tile of a row tile): an item of n
// steps costs n + 2, or n + 4 where the steps wait for memory. Sequences that
// fill their rows: as many waves of items as the SMs need, each as long as an
// item. Sequences of any length up to their rows (k_lengths): half the steps on
// average, taken as they come, and one item's length at the end. In float32 a
// step is some four times as long, several blocks share an SM and most calls
// have few: the SMs' work, and one item's length at the end. The join of the
// shares costs a launch and the partial results' way to memory and back.
// SMs and measured steps are those of the GB300 (152), not asked of the device: the
// plan decides the workspace's size, which is asked without one.
// (Measured: 4 maps of 80 x 80, 2 heads of 64: 114 us with one share, 102 with
// two, 97 with three, 110 with four; 16 new tokens against up to 8192 keys: 90
// with one, 77 to 81 with two to eight; a prompt of 1024 tokens, 32 heads: 28
// with one, 40 with two; float32, 6 maps of up to 32 x 32, 8 heads of 40: 118
// with one, 88 with four, 91 with six.)
struct AttnPlan {
    int64_t tiles, splits;
    size_t off_out, off_lse, bytes;
};

AttnPlan attn_plan(const mdcn_attention_attrs& at, const mdcn_attention_dims& d, mdcn_dtype dtype, bool lengths) {
    constexpr int64_t kSms = 152, kMaxSplits = 32;
    constexpr double kItemSteps = 2.0, kWaitingItemSteps = 4.0, kJoinSteps = 2.5, kStepBytes = 8.0e6;
    constexpr double kF32ItemSteps = 0.3, kF32Step = 0.25;
    AttnPlan p{};
    const int64_t group = d.q_heads / d.k_heads;
    const bool tc = dtype != MDCN_F32;
    const int64_t tokens = tc ? 2 * (mdcn::kAttnTcBlockRows / group) : mdcn::kAttnSimtRows / group;
    const int64_t keys = tc ? 128 : 64;
    p.tiles = mdcn::attn_tiles(d.q_tokens, d.batch, tokens);
    p.splits = 1;
    // the tiles that there are at least: p.tiles has room for one more in each sequence
    int64_t least = (d.q_tokens + tokens - 1) / tokens;
    const int64_t sequences = d.batch < d.q_tokens ? d.batch : d.q_tokens;
    if (least < sequences) least = sequences;
    const int64_t blocks = least * d.k_heads;
    if (blocks > 0 && blocks <= 4 * kSms) {  // beyond, the last wave is a small part of the whole
        const double mean = static_cast<double>(d.k_tokens) / static_cast<double>(d.batch);
        const double own = at.causal ? static_cast<double>(d.q_tokens) / static_cast<double>(d.batch) / 2 : 0.0;
        const double seen = mean > own ? mean - own : mean / 2;
        const int64_t steps = static_cast<int64_t>(seen / static_cast<double>(keys)) + 1;
        const double rows = static_cast<double>(d.q_tokens) * static_cast<double>(d.q_heads) *
                            static_cast<double>(d.head_dim) * 8.0;
        double best = 0.0;
        for (int64_t s = 1; s <= kMaxSplits && s <= steps; ++s) {
            const double item = static_cast<double>((steps + s - 1) / s);
            const double mean_steps = lengths ? static_cast<double>(steps) / 2 : static_cast<double>(steps);
            double cost;
            if (!tc)
                cost = static_cast<double>(blocks) * (mean_steps + kF32ItemSteps * s) / static_cast<double>(kSms) + item;
            else if (lengths)
                cost = static_cast<double>(blocks) * (mean_steps + kWaitingItemSteps * s) / static_cast<double>(kSms) + item;
            else
                cost = static_cast<double>((blocks * s + kSms - 1) / kSms) * (item + kItemSteps);
            if (s > 1) cost += (kJoinSteps + rows * static_cast<double>(s) / kStepBytes) * (tc ? 1.0 : kF32Step);
            if (s == 1 || cost < best) {
                best = cost;
                p.splits = s;
            }
        }
    }
    size_t off = mdcn::kAttnHeaderBytes;
    if (p.splits > 1) {
        const size_t rows = static_cast<size_t>(p.splits) * static_cast<size_t>(d.q_tokens) * static_cast<size_t>(d.q_heads);
        p.off_out = off;
        off = align256(off + rows * static_cast<size_t>(d.head_dim) * 4);
        p.off_lse = off;
        off = align256(off + rows * 4);
    }
    p.bytes = off;
    return p;
}

// The backward's plan: where delta lies, in float16 the sizes that scale dS, and
// in float32 between how many blocks
// the rows that see a key tile, and the keys that a row tile sees, are shared
// out: as many as make three blocks of the first kind to an SM and six of the
// second, each with two tiles at least. (Ragged sequences of up to 700, 6 heads
// of 72 over 2: 374 us with neither shared, 146 with rows, 99 with both; 2
// causal sequences of 2048, heads of 64: 972, 706 and 626.)
struct AttnBwdPlan {
    int64_t tiles, kv_splits, q_splits;
    size_t off_g_size, off_v_size, off_sizes, off_kv, off_q, bytes;
};

AttnBwdPlan attn_bwd_plan(const mdcn_attention_dims& d, mdcn_dtype dtype) {
    constexpr int64_t kSms = 152, kMaxSplits = 16;
    AttnBwdPlan p{};
    const int64_t tokens = mdcn::kAttnSimtRows / (d.q_heads / d.k_heads);
    p.tiles = mdcn::attn_tiles(d.q_tokens, d.batch, tokens);
    p.kv_splits = p.q_splits = 1;
    size_t off = align256(mdcn::kAttnHeaderBytes + static_cast<size_t>(d.q_tokens) * static_cast<size_t>(d.q_heads) * 4);
    if (dtype == MDCN_F16) {
        p.off_g_size = off;
        off = align256(off + static_cast<size_t>(d.q_tokens) * static_cast<size_t>(d.q_heads));
        p.off_v_size = off;
        off = align256(off + static_cast<size_t>(d.k_tokens) * static_cast<size_t>(d.k_heads));
        p.off_sizes = off;
        off = align256(off + static_cast<size_t>(d.batch) * static_cast<size_t>(d.k_heads) * 8);
    }
    if (dtype == MDCN_F32 && d.batch > 0) {
        auto shares = [](int64_t blocks, int64_t wanted, int64_t steps) {
            int64_t s = blocks > 0 ? wanted * kSms / blocks : 1;
            if (s > steps / 2) s = steps / 2;
            return s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s;
        };
        const int64_t row_tiles = (d.q_tokens / d.batch + tokens - 1) / tokens, key_tiles = (d.k_tokens / d.batch + 63) / 64;
        p.kv_splits = shares(mdcn::attn_tiles(d.k_tokens, d.batch, 64) * d.k_heads, 3, row_tiles);
        p.q_splits = shares(p.tiles * d.k_heads, 6, key_tiles);
        if (p.kv_splits > 1) {
            p.off_kv = off;
            off = align256(off + static_cast<size_t>(p.kv_splits) * 2 * static_cast<size_t>(d.k_tokens) *
                                     static_cast<size_t>(d.k_heads) * static_cast<size_t>(d.head_dim) * 4);
        }
        if (p.q_splits > 1) {
            p.off_q = off;
            off = align256(off + static_cast<size_t>(p.q_splits) * static_cast<size_t>(d.q_tokens) *
                                     static_cast<size_t>(d.q_heads) * static_cast<size_t>(d.head_dim) * 4);
        }
    }
    p.bytes = off;
    return p;
}

mdcn::AttnTensor atensor(const void* p, const mdcn_strides& s, int64_t tokens, int64_t heads) {
    return {const_cast<void*>(p), used(s.token, tokens), used(s.head, heads)};
}

mdcn::AttnArgs attn_args(const mdcn_attention_attrs& at, const mdcn_attention_dims& d, const void* q, const void* k,
                         const void* v, const void* out, const void* lse, const void* qs, const void* ks,
                         const void* kl) {
    mdcn::AttnArgs a{};
    a.q = atensor(q, d.q, d.q_tokens, d.q_heads);
    a.k = atensor(k, d.k, d.k_tokens, d.k_heads);
    a.v = atensor(v, d.v, d.k_tokens, d.k_heads);
    a.out = atensor(out, d.out, d.q_tokens, d.q_heads);
    a.lse = static_cast<float*>(const_cast<void*>(lse));
    a.q_starts = static_cast<const int32_t*>(qs);
    a.k_starts = static_cast<const int32_t*>(ks);
    a.k_lengths = static_cast<const int32_t*>(kl);
    a.batch = static_cast<int32_t>(d.batch);
    a.tq = static_cast<int32_t>(d.q_tokens);
    a.tk = static_cast<int32_t>(d.k_tokens);
    a.hq = static_cast<int32_t>(d.q_heads);
    a.hk = static_cast<int32_t>(d.k_heads);
    a.group = static_cast<int32_t>(d.q_heads / d.k_heads);
    a.D = static_cast<int32_t>(d.head_dim);
    a.causal = at.causal;
    a.scale = at.scale;
    a.splits = 1;
    return a;
}

// NULL only where the tensor has no elements.
bool given(const void* p, int64_t elements) { return p != nullptr || elements == 0; }

}  // namespace

extern "C" {

mdcn_status mdcn_rotary_forward(const mdcn_rotary_attrs* attrs, const mdcn_rotary_dims* dims, mdcn_dtype dtype,
                                const void* q, const void* k_or_null, const void* positions, const void* inv_freq,
                                const void* q_weight_or_null, const void* k_weight_or_null, void* q_out,
                                void* k_out_or_null, void* stream) {
    mdcn_status s = rotary_check(attrs, dims, dtype, false);
    if (s != MDCN_OK) return s;
    mdcn::RotaryArgs a = rotary_args(*attrs, *dims);
    const int64_t tk = dims->k_heads > 0 ? dims->tokens : 0;
    if (!given(q, dims->tokens) || !given(q_out, dims->tokens) || !given(k_or_null, tk) || !given(k_out_or_null, tk) ||
        !given(positions, dims->tokens) || !given(inv_freq, a.pairs))
        return MDCN_ERR_NULL;
    if (!attrs->norm && (q_weight_or_null || k_weight_or_null)) return MDCN_ERR_ATTR;
    if (!aligned16(positions) || !aligned16(inv_freq) || !aligned16(q_weight_or_null) || !aligned16(k_weight_or_null))
        return MDCN_ERR_ALIGN;
    if (dims->k_heads == 0) k_or_null = k_out_or_null = nullptr;
    const void* p[] = {q, q_out, k_or_null, k_out_or_null};
    const mdcn_strides* st[] = {&dims->q, &dims->q_out, &dims->k, &dims->k_out};
    const int64_t heads[] = {dims->q_heads, dims->q_heads, dims->k_heads, dims->k_heads};
    s = rotary_align(*dims, dtype, p, st, heads, 4, &a.vec);
    if (s != MDCN_OK) return s;
    int sms = 0;
    s = mdcn::api_check_device(&sms);
    if (s != MDCN_OK) return s;
    if (dims->tokens == 0) return MDCN_OK;
    a.x[0] = tensor(q, dims->q, dims->tokens, dims->q_heads);
    a.x[1] = tensor(k_or_null, dims->k, dims->tokens, dims->k_heads);
    a.y[0] = tensor(q_out, dims->q_out, dims->tokens, dims->q_heads);
    a.y[1] = tensor(k_out_or_null, dims->k_out, dims->tokens, dims->k_heads);
    a.w[0] = q_weight_or_null;
    a.w[1] = k_weight_or_null;
    a.pos = static_cast<const int32_t*>(positions);
    a.freq = static_cast<const float*>(inv_freq);
    const cudaError_t e = mdcn::launch_rotary_forward(dtype, a, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MDCN_OK : mdcn::api_cuda_fail(e);
}

mdcn_status mdcn_rotary_backward_workspace_size(const mdcn_rotary_attrs* attrs, const mdcn_rotary_dims* dims,
                                                mdcn_dtype dtype, size_t* bytes) {
    if (!bytes) return MDCN_ERR_NULL;
    const mdcn_status s = rotary_check(attrs, dims, dtype, true);
    if (s != MDCN_OK) return s;
    *bytes = attrs->norm ? rotary_ws(*dims) : 0;
    return MDCN_OK;
}

mdcn_status mdcn_rotary_backward(const mdcn_rotary_attrs* attrs, const mdcn_rotary_dims* dims, mdcn_dtype dtype,
                                 const void* grad_q_out, const void* grad_k_out_or_null, const void* q_or_null,
                                 const void* k_or_null, const void* positions, const void* inv_freq,
                                 const void* q_weight_or_null, const void* k_weight_or_null, void* grad_q,
                                 void* grad_k_or_null, void* grad_q_weight_or_null, void* grad_k_weight_or_null,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    mdcn_status s = rotary_check(attrs, dims, dtype, true);
    if (s != MDCN_OK) return s;
    mdcn::RotaryArgs a = rotary_args(*attrs, *dims);
    const int64_t tk = dims->k_heads > 0 ? dims->tokens : 0;
    if (!given(grad_q_out, dims->tokens) || !given(grad_q, dims->tokens) || !given(grad_k_out_or_null, tk) ||
        !given(grad_k_or_null, tk) || !given(positions, dims->tokens) || !given(inv_freq, a.pairs))
        return MDCN_ERR_NULL;
    if (attrs->norm && (!given(q_or_null, dims->tokens) || !given(k_or_null, tk))) return MDCN_ERR_NULL;
    if (!attrs->norm && (q_weight_or_null || k_weight_or_null || grad_q_weight_or_null || grad_k_weight_or_null))
        return MDCN_ERR_ATTR;
    if ((q_weight_or_null == nullptr) != (grad_q_weight_or_null == nullptr) ||
        (k_weight_or_null == nullptr) != (grad_k_weight_or_null == nullptr))
        return MDCN_ERR_NULL;
    if (dims->k_heads == 0) grad_k_out_or_null = k_or_null = grad_k_or_null = nullptr;
    if (!attrs->norm) q_or_null = k_or_null = nullptr;
    const bool weights = grad_q_weight_or_null || grad_k_weight_or_null;
    if (weights && !workspace) return MDCN_ERR_NULL;
    const void* al[] = {positions, inv_freq, q_weight_or_null, k_weight_or_null, grad_q_weight_or_null,
                        grad_k_weight_or_null, workspace};
    for (const void* p : al)
        if (!aligned16(p)) return MDCN_ERR_ALIGN;
    const void* p[] = {grad_q_out, grad_q, q_or_null, grad_k_out_or_null, grad_k_or_null, k_or_null};
    const mdcn_strides* st[] = {&dims->q_out, &dims->q_grad, &dims->q, &dims->k_out, &dims->k_grad, &dims->k};
    const int64_t heads[] = {dims->q_heads, dims->q_heads, dims->q_heads, dims->k_heads, dims->k_heads, dims->k_heads};
    s = rotary_align(*dims, dtype, p, st, heads, 6, &a.vec);
    if (s != MDCN_OK) return s;
    if (weights && workspace_bytes < rotary_ws(*dims)) return MDCN_ERR_WORKSPACE;
    int sms = 0;
    s = mdcn::api_check_device(&sms);
    if (s != MDCN_OK) return s;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    // no tokens, or no heads of k: the weights' gradients are empty sums
    const size_t bytes = static_cast<size_t>(dims->head_dim) * static_cast<size_t>(size_of(dtype));
    if (dims->tokens == 0 && grad_q_weight_or_null) e = cudaMemsetAsync(grad_q_weight_or_null, 0, bytes, cs);
    if (e == cudaSuccess && tk == 0 && grad_k_weight_or_null) {
        e = cudaMemsetAsync(grad_k_weight_or_null, 0, bytes, cs);
        grad_k_weight_or_null = nullptr;
    }
    if (e != cudaSuccess) return mdcn::api_cuda_fail(e);
    if (dims->tokens == 0) return MDCN_OK;
    a.y[0] = tensor(grad_q_out, dims->q_out, dims->tokens, dims->q_heads);
    a.y[1] = tensor(grad_k_out_or_null, dims->k_out, dims->tokens, dims->k_heads);
    a.x[0] = tensor(q_or_null, dims->q, dims->tokens, dims->q_heads);
    a.x[1] = tensor(k_or_null, dims->k, dims->tokens, dims->k_heads);
    a.g[0] = tensor(grad_q, dims->q_grad, dims->tokens, dims->q_heads);
    a.g[1] = tensor(grad_k_or_null, dims->k_grad, dims->tokens, dims->k_heads);
    a.w[0] = q_weight_or_null;
    a.w[1] = k_weight_or_null;
    a.pos = static_cast<const int32_t*>(positions);
    a.freq = static_cast<const float*>(inv_freq);
    a.part = grad_q_weight_or_null || grad_k_weight_or_null ? static_cast<float*>(workspace) : nullptr;
    e = mdcn::launch_rotary_backward(dtype, a, grad_q_weight_or_null, grad_k_weight_or_null, sms, cs);
    return e == cudaSuccess ? MDCN_OK : mdcn::api_cuda_fail(e);
}

mdcn_status mdcn_attention_workspace_size(const mdcn_attention_attrs* attrs, const mdcn_attention_dims* dims,
                                          mdcn_dtype dtype, size_t* bytes) {
    if (!bytes) return MDCN_ERR_NULL;
    const mdcn_status s = attn_check(attrs, dims, dtype, false);
    if (s != MDCN_OK) return s;
    // whether the call has k_lengths is not known here: room for either plan
    const size_t with = attn_plan(*attrs, *dims, dtype, true).bytes, without = attn_plan(*attrs, *dims, dtype, false).bytes;
    *bytes = with > without ? with : without;
    return MDCN_OK;
}

mdcn_status mdcn_attention_forward(const mdcn_attention_attrs* attrs, const mdcn_attention_dims* dims,
                                   mdcn_dtype dtype, const void* q, const void* k, const void* v,
                                   const void* q_starts, const void* k_starts, const void* k_lengths_or_null,
                                   void* out, void* lse, void* workspace, size_t workspace_bytes, void* stream) {
    mdcn_status s = attn_check(attrs, dims, dtype, false);
    if (s != MDCN_OK) return s;
    if (!given(q, dims->q_tokens) || !given(k, dims->k_tokens) || !given(v, dims->k_tokens) ||
        !given(out, dims->q_tokens) || !given(lse, dims->q_tokens) || !q_starts || !k_starts || !workspace)
        return MDCN_ERR_NULL;
    const void* al[] = {q, k, v, q_starts, k_starts, k_lengths_or_null, out, lse, workspace};
    for (const void* p : al)
        if (!aligned16(p)) return MDCN_ERR_ALIGN;
    const AttnPlan p = attn_plan(*attrs, *dims, dtype, k_lengths_or_null != nullptr);
    if (p.tiles > kI31 / p.splits / dims->k_heads) return MDCN_ERR_UNSUPPORTED;
    if (workspace_bytes < p.bytes) return MDCN_ERR_WORKSPACE;
    s = mdcn::api_check_device(nullptr);
    if (s != MDCN_OK) return s;
    mdcn::AttnArgs a = attn_args(*attrs, *dims, q, k, v, out, lse, q_starts, k_starts, k_lengths_or_null);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.status = reinterpret_cast<uint32_t*>(ws);
    a.tiles = static_cast<int32_t>(p.tiles);
    a.splits = static_cast<int32_t>(p.splits);
    if (p.splits > 1) {
        a.part_out = reinterpret_cast<float*>(ws + p.off_out);
        a.part_lse = reinterpret_cast<float*>(ws + p.off_lse);
    }
    cudaError_t e;
    if (p.tiles == 0) {
        e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), st);
    } else {
        e = dtype == MDCN_F32 ? mdcn::launch_attention_simt_forward(a, st)
                              : mdcn::launch_attention_tc_forward(dtype, a, st);
        if (e == cudaSuccess && p.splits > 1) e = mdcn::launch_attention_join(dtype, a, st);
    }
    return e == cudaSuccess ? MDCN_OK : mdcn::api_cuda_fail(e);
}

mdcn_status mdcn_attention_backward_workspace_size(const mdcn_attention_attrs* attrs, const mdcn_attention_dims* dims,
                                                   mdcn_dtype dtype, size_t* bytes) {
    if (!bytes) return MDCN_ERR_NULL;
    const mdcn_status s = attn_check(attrs, dims, dtype, true);
    if (s != MDCN_OK) return s;
    *bytes = attn_bwd_plan(*dims, dtype).bytes;
    return MDCN_OK;
}

mdcn_status mdcn_attention_backward(const mdcn_attention_attrs* attrs, const mdcn_attention_dims* dims,
                                    mdcn_dtype dtype, const void* grad_out, const void* q, const void* k,
                                    const void* v, const void* out, const void* lse, const void* q_starts,
                                    const void* k_starts, const void* k_lengths_or_null, void* grad_q, void* grad_k,
                                    void* grad_v, void* workspace, size_t workspace_bytes, void* stream) {
    mdcn_status s = attn_check(attrs, dims, dtype, true);
    if (s != MDCN_OK) return s;
    const void* of_q[] = {grad_out, q, out, lse, grad_q};
    const void* of_k[] = {k, v, grad_k, grad_v};
    for (const void* p : of_q)
        if (!given(p, dims->q_tokens)) return MDCN_ERR_NULL;
    for (const void* p : of_k)
        if (!given(p, dims->k_tokens)) return MDCN_ERR_NULL;
    if (!q_starts || !k_starts || !workspace) return MDCN_ERR_NULL;
    const void* al[] = {grad_out, q, k, v, out, lse, q_starts, k_starts, k_lengths_or_null, grad_q, grad_k, grad_v,
                        workspace};
    for (const void* p : al)
        if (!aligned16(p)) return MDCN_ERR_ALIGN;
    const AttnBwdPlan p = attn_bwd_plan(*dims, dtype);
    if (p.tiles > kI31 / dims->k_heads ||
        mdcn::attn_tiles(dims->k_tokens, dims->batch, 64) * p.kv_splits + p.tiles * p.q_splits > kI31 / dims->k_heads)
        return MDCN_ERR_UNSUPPORTED;
    if (workspace_bytes < p.bytes) return MDCN_ERR_WORKSPACE;
    s = mdcn::api_check_device(nullptr);
    if (s != MDCN_OK) return s;
    mdcn::AttnArgs a = attn_args(*attrs, *dims, q, k, v, out, lse, q_starts, k_starts, k_lengths_or_null);
    a.g = atensor(grad_out, dims->grad_out, dims->q_tokens, dims->q_heads);
    a.gq = atensor(grad_q, dims->grad_q, dims->q_tokens, dims->q_heads);
    a.gk = atensor(grad_k, dims->grad_k, dims->k_tokens, dims->k_heads);
    a.gv = atensor(grad_v, dims->grad_v, dims->k_tokens, dims->k_heads);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.status = reinterpret_cast<uint32_t*>(ws);
    a.delta = reinterpret_cast<float*>(ws + mdcn::kAttnHeaderBytes);
    a.tiles = static_cast<int32_t>(p.tiles);
    a.kv_splits = static_cast<int32_t>(p.kv_splits);
    a.q_splits = static_cast<int32_t>(p.q_splits);
    if (dtype == MDCN_F16) {
        a.g_size = ws + p.off_g_size;
        a.v_size = ws + p.off_v_size;
        a.sizes = reinterpret_cast<int32_t*>(ws + p.off_sizes);
    }
    if (p.kv_splits > 1) a.part_kv = reinterpret_cast<float*>(ws + p.off_kv);
    if (p.q_splits > 1) a.part_q = reinterpret_cast<float*>(ws + p.off_q);
    cudaError_t e = mdcn::launch_attention_delta(dtype, a, st);
    if (e == cudaSuccess)
        e = dtype == MDCN_F32 ? mdcn::launch_attention_simt_backward(a, st)
                              : mdcn::launch_attention_tc_backward(dtype, a, st);
    return e == cudaSuccess ? MDCN_OK : mdcn::api_cuda_fail(e);
}

}  // extern "C"
