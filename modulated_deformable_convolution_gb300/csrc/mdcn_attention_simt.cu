// Attention over packed sequences on the CUDA cores (fp32 products), and the
// small kernels that both forms of the attention use.
//
// Forward, per row: running maximum m and sum l of exp(scale q.k - m) over
// 64-key tiles, accumulator rescaled by exp(m_old - m) when m grows; out =
// acc / l, lse = m + log l. Backward from lse: p = exp(scale q.k - lse), ds =
// p (g.v - delta) scale; one kernel sums ds k over the keys of 64 rows, the
// other p^T g and ds^T q over the rows that see 64 keys.
//
// Bound by fp32 multiply-adds. 256 threads hold a 64 x 64 score tile as 4 x 4
// each and a 64 x D accumulator as 4 rows x 4-element pieces; operands come
// from shared memory as 16-byte vectors (rows padded by 4 words, so that the
// 16 rows a warp reads at once fall into different banks), 64 multiply-adds
// for 8 vectors.
#include <cfloat>
#include <cstdint>

#include "mdcn_attention.cuh"
#include "mdcn_plan.h"

namespace mdcn {

namespace {

constexpr int kR = kAttnSimtRows;  // rows of a tile
constexpr int kC = 64;             // keys of a tile
constexpr int kT = 256;
constexpr int kPP = kC + 4;        // padded row of the probability tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kAcc = 2;            // 4-element pieces of a row per thread: 64 * kAcc >= D

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    c = fmaf(a.x, b.x, c);
    c = fmaf(a.y, b.y, c);
    c = fmaf(a.z, b.z, c);
    return fmaf(a.w, b.w, c);
}

// Rows of a packed row tile into shared memory: row r = (token r / group, head
// r % group) of key head kh, zero past the sequence's end.
template <typename T>
__device__ __forceinline__ void load_rows(float* dst, int pitch, const AttnTensor& t, const AttnArgs& a,
                                          const AttnSeq& s, int32_t tok0, int32_t ntok, int kh) {
    const int v4 = a.D / 4, rows = ntok * a.group;
    for (int i = threadIdx.x; i < kR * v4; i += kT) {
        const int r = i / v4, c = (i - r * v4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const int tk = r / a.group, h = kh * a.group + (r - tk * a.group);
            x = attn_load4(static_cast<const T*>(t.p) + static_cast<int64_t>(s.q0 + tok0 + tk) * t.st +
                           static_cast<int64_t>(h) * t.sh + c);
        }
        *reinterpret_cast<float4*>(dst + r * pitch + c) = x;
    }
}

// Keys (or values) [j0, j0 + 64) of the sequence, zero past its last key.
template <typename T>
__device__ __forceinline__ void load_keys(float* dst, int pitch, const AttnTensor& t, const AttnArgs& a,
                                          const AttnSeq& s, int32_t j0, int kh) {
    const int v4 = a.D / 4;
    for (int i = threadIdx.x; i < kC * v4; i += kT) {
        const int r = i / v4, c = (i - r * v4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + r < s.lk)
            x = attn_load4(static_cast<const T*>(t.p) + static_cast<int64_t>(s.k0 + j0 + r) * t.st +
                           static_cast<int64_t>(kh) * t.sh + c);
        *reinterpret_cast<float4*>(dst + r * pitch + c) = x;
    }
}

// acc[i][j] = row (ty + 16 i) of x . row (tx + 16 j) of y
__device__ __forceinline__ void products(float (&acc)[4][4], const float* x, const float* y, int pitch, int D, int tx,
                                         int ty) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    for (int d = 0; d < D; d += 4) {
        float4 u[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4*>(x + (ty + 16 * i) * pitch + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const float4*>(y + (tx + 16 * j) * pitch + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = dot4(u[i], w[j], acc[i][j]);
    }
}

// o[i] (row ty + 16 i, elements tx * 4 + 64 c) += sum over the 64 columns j of p[row][j] * y[j]
__device__ __forceinline__ void accumulate(float4 (&o)[4][kAcc], const float* p, const float* y, int pitch, int D,
                                           int tx, int ty) {
    for (int j = 0; j < kC; j += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + (ty + 16 * i) * kPP + j);
#pragma unroll
        for (int c = 0; c < kAcc; ++c) {
            const int d = tx * 4 + 64 * c;
            if (d >= D) continue;
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const float4 v = *reinterpret_cast<const float4*>(y + (j + jj) * pitch + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
                    o[i][c].x = fmaf(f, v.x, o[i][c].x);
                    o[i][c].y = fmaf(f, v.y, o[i][c].y);
                    o[i][c].z = fmaf(f, v.z, o[i][c].z);
                    o[i][c].w = fmaf(f, v.w, o[i][c].w);
                }
            }
        }
    }
}

__device__ __forceinline__ float max16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Grid: (tiles * splits, key heads). Block x takes tile x / splits and the
// (x % splits)-th share of the key tiles that the tile's rows see.
template <typename T>
__global__ void __launch_bounds__(kT) attn_forward_simt_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ float sm[];
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
    const int tpt = kR / a.group;
    const AttnSeq s = attn_find(a, false, tpt, blockIdx.x / a.splits);
    if (s.tile < 0) return;
    const int kh = blockIdx.y, split = blockIdx.x % a.splits;
    const int pitch = a.D + 4;
    float* qs = sm;
    float* ks = qs + kR * pitch;  // keys, then values
    float* ps = ks + kC * pitch;
    const int32_t tok0 = s.tile * tpt, ntok = min(tpt, s.lq - tok0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_rows<T>(qs, pitch, a.q, a, s, tok0, ntok, kh);

    int32_t seen[4];
    float m[4], l[4];
    float4 o[4][kAcc];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        seen[i] = r < ntok * a.group ? attn_seen(a, s, tok0 + r / a.group) : 0;
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < kAcc; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int32_t most = attn_seen(a, s, tok0 + ntok - 1);
    const int32_t ktiles = (most + kC - 1) / kC, per = (ktiles + a.splits - 1) / a.splits;
    const int32_t t0 = min(split * per, ktiles), t1 = min(t0 + per, ktiles);
    const float to_log2 = a.scale * kLog2e;
    for (int32_t t = t0; t < t1; ++t) {
        __syncthreads();
        load_keys<T>(ks, pitch, a.k, a, s, t * kC, kh);
        __syncthreads();
        float x[4][4];
        products(x, qs, ks, pitch, a.D, tx, ty);
        float corr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float best = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = t * kC + tx + 16 * j < seen[i] ? x[i][j] * to_log2 : -INFINITY;
                best = fmaxf(best, x[i][j]);
            }
            best = fmaxf(max16(best), m[i]);
            const float base = best == -INFINITY ? 0.0f : best;  // no key seen so far: every term is exp2(-inf) = 0
            corr[i] = exp2f(m[i] - base);
            m[i] = best;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(x[i][j] - base);
                sum += p;
                ps[(ty + 16 * i) * kPP + tx + 16 * j] = p;
            }
            l[i] = fmaf(l[i], corr[i], sum16(sum));
#pragma unroll
            for (int c = 0; c < kAcc; ++c) {
                o[i][c].x *= corr[i];
                o[i][c].y *= corr[i];
                o[i][c].z *= corr[i];
                o[i][c].w *= corr[i];
            }
        }
        __syncthreads();
        load_keys<T>(ks, pitch, a.v, a, s, t * kC, kh);
        __syncthreads();
        accumulate(o, ps, ks, pitch, a.D, tx, ty);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r >= ntok * a.group) continue;
        const int64_t tok = s.q0 + tok0 + r / a.group;
        const int h = kh * a.group + r % a.group;
        const float inv = l[i] > 0.0f ? 1.0f / l[i] : (l[i] == 0.0f ? 0.0f : l[i]);
        const float lse = l[i] == 0.0f ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
#pragma unroll
        for (int c = 0; c < kAcc; ++c) {
            const int d = tx * 4 + 64 * c;
            if (d >= a.D) continue;
            const float4 v = make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv);
            if (a.splits > 1)
                *reinterpret_cast<float4*>(a.part_out + ((static_cast<int64_t>(split) * a.tq + tok) * a.hq + h) * a.D + d) = v;
            else
                attn_store4(static_cast<T*>(a.out.p) + tok * a.out.st + h * a.out.sh + d, v);
        }
        if (tx == 0) {
            if (a.splits > 1)
                a.part_lse[(static_cast<int64_t>(split) * a.hq + h) * a.tq + tok] = lse;
            else
                a.lse[static_cast<int64_t>(h) * a.tq + tok] = lse;
        }
    }
}

// grad_q of one row tile. Grid: (tiles, key heads).
template <typename T>
__global__ void __launch_bounds__(kT) attn_grad_q_simt_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ float sm[];
    const int tpt = kR / a.group;
    const AttnSeq s = attn_find(a, false, tpt, blockIdx.x);
    if (s.tile < 0) return;
    const int kh = blockIdx.y, pitch = a.D + 4;
    float* qs = sm;
    float* gs = qs + kR * pitch;
    float* ks = gs + kR * pitch;
    float* vs = ks + kC * pitch;
    float* ps = vs + kC * pitch;
    const int32_t tok0 = s.tile * tpt, ntok = min(tpt, s.lq - tok0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_rows<T>(qs, pitch, a.q, a, s, tok0, ntok, kh);
    load_rows<T>(gs, pitch, a.g, a, s, tok0, ntok, kh);
    int32_t seen[4];
    float lse[4], delta[4];
    float4 o[4][kAcc];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        const bool live = r < ntok * a.group;
        const int64_t at = live ? static_cast<int64_t>(kh * a.group + r % a.group) * a.tq + s.q0 + tok0 + r / a.group : 0;
        seen[i] = live ? attn_seen(a, s, tok0 + r / a.group) : 0;
        lse[i] = live ? a.lse[at] : 0.0f;
        delta[i] = live ? a.delta[at] : 0.0f;
#pragma unroll
        for (int c = 0; c < kAcc; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int32_t ktiles = (attn_seen(a, s, tok0 + ntok - 1) + kC - 1) / kC;
    for (int32_t t = 0; t < ktiles; ++t) {
        __syncthreads();
        load_keys<T>(ks, pitch, a.k, a, s, t * kC, kh);
        load_keys<T>(vs, pitch, a.v, a, s, t * kC, kh);
        __syncthreads();
        float x[4][4], dp[4][4];
        products(x, qs, ks, pitch, a.D, tx, ty);
        products(dp, gs, vs, pitch, a.D, tx, ty);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool on = t * kC + tx + 16 * j < seen[i];
                const float p = on ? exp2f(fmaf(x[i][j], a.scale, -lse[i]) * kLog2e) : 0.0f;
                ps[(ty + 16 * i) * kPP + tx + 16 * j] = on ? p * (dp[i][j] - delta[i]) : 0.0f;
            }
        __syncthreads();
        accumulate(o, ps, ks, pitch, a.D, tx, ty);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (r >= ntok * a.group) continue;
        const int64_t tok = s.q0 + tok0 + r / a.group;
        const int h = kh * a.group + r % a.group;
#pragma unroll
        for (int c = 0; c < kAcc; ++c) {
            const int d = tx * 4 + 64 * c;
            if (d < a.D)
                attn_store4(static_cast<T*>(a.gq.p) + tok * a.gq.st + h * a.gq.sh + d,
                            make_float4(o[i][c].x * a.scale, o[i][c].y * a.scale, o[i][c].z * a.scale, o[i][c].w * a.scale));
        }
    }
}

// o[i] (row 4 ty + i) += sum over the 64 rows r of p[r][row] * y[r]
__device__ __forceinline__ void accumulate_t(float4 (&o)[4][kAcc], const float* p, const float* y, int pitch, int D,
                                             int tx, int ty) {
#pragma unroll 2
    for (int r = 0; r < kR; ++r) {
        const float4 w = *reinterpret_cast<const float4*>(p + r * kPP + ty * 4);
        const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < kAcc; ++c) {
            const int d = tx * 4 + 64 * c;
            if (d >= D) continue;
            const float4 v = *reinterpret_cast<const float4*>(y + r * pitch + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i][c].x = fmaf(f[i], v.x, o[i][c].x);
                o[i][c].y = fmaf(f[i], v.y, o[i][c].y);
                o[i][c].z = fmaf(f[i], v.z, o[i][c].z);
                o[i][c].w = fmaf(f[i], v.w, o[i][c].w);
            }
        }
    }
}

// grad_k and grad_v of 64 keys of one key head. Grid: (key tiles, key heads).
template <typename T>
__global__ void __launch_bounds__(kT) attn_grad_kv_simt_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ float sm[];
    const AttnSeq s = attn_find(a, true, kC, blockIdx.x);
    if (s.tile < 0) return;
    const int kh = blockIdx.y, pitch = a.D + 4, tpt = kR / a.group;
    float* qs = sm;
    float* gs = qs + kR * pitch;
    float* ks = gs + kR * pitch;
    float* vs = ks + kC * pitch;
    float* ps = vs + kC * pitch;
    float* ds = ps + kR * kPP;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t j0 = s.tile * kC;
    load_keys<T>(ks, pitch, a.k, a, s, j0, kh);
    load_keys<T>(vs, pitch, a.v, a, s, j0, kh);
    float4 ok[4][kAcc], ov[4][kAcc];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < kAcc; ++c) ok[i][c] = ov[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    // the first query that sees key j0
    const int32_t first = j0 >= s.lk ? s.lq : (a.causal ? max(0, j0 + s.lq - s.lk) : 0);
    for (int32_t tok0 = first / tpt * tpt; tok0 < s.lq; tok0 += tpt) {
        const int32_t ntok = min(tpt, s.lq - tok0);
        __syncthreads();
        load_rows<T>(qs, pitch, a.q, a, s, tok0, ntok, kh);
        load_rows<T>(gs, pitch, a.g, a, s, tok0, ntok, kh);
        __syncthreads();
        float x[4][4], dp[4][4];
        products(x, qs, ks, pitch, a.D, tx, ty);
        products(dp, gs, vs, pitch, a.D, tx, ty);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            const bool live = r < ntok * a.group;
            const int64_t at =
                live ? static_cast<int64_t>(kh * a.group + r % a.group) * a.tq + s.q0 + tok0 + r / a.group : 0;
            const int32_t seen = live ? attn_seen(a, s, tok0 + r / a.group) : 0;
            const float lse = live ? a.lse[at] : 0.0f, delta = live ? a.delta[at] : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool on = j0 + tx + 16 * j < seen;
                const float p = on ? exp2f(fmaf(x[i][j], a.scale, -lse) * kLog2e) : 0.0f;  // one rounding before the small difference is scaled
                ps[r * kPP + tx + 16 * j] = p;
                ds[r * kPP + tx + 16 * j] = on ? p * (dp[i][j] - delta) : 0.0f;
            }
        }
        __syncthreads();
        accumulate_t(ov, ps, gs, pitch, a.D, tx, ty);
        accumulate_t(ok, ds, qs, pitch, a.D, tx, ty);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t j = j0 + ty * 4 + i;
        if (j >= s.room) continue;
        const int64_t row = s.k0 + j;
#pragma unroll
        for (int c = 0; c < kAcc; ++c) {
            const int d = tx * 4 + 64 * c;
            if (d >= a.D) continue;
            attn_store4(static_cast<T*>(a.gv.p) + row * a.gv.st + kh * a.gv.sh + d, ov[i][c]);
            attn_store4(static_cast<T*>(a.gk.p) + row * a.gk.st + kh * a.gk.sh + d,
                        make_float4(ok[i][c].x * a.scale, ok[i][c].y * a.scale, ok[i][c].z * a.scale, ok[i][c].w * a.scale));
        }
    }
}

// One warp per (token, head): out = sum over the splits of exp(lse_i - lse) out_i.
template <typename T>
__global__ void __launch_bounds__(kT) attn_join_kernel(const __grid_constant__ AttnArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kT / 32) + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(a.tq) * a.hq) return;
    const int64_t tok = row / a.hq;
    const int h = static_cast<int>(row - tok * a.hq);
    // rows of no sequence have no partial results and are not written
    bool mine = false;
    for (int b = lane; b < a.batch; b += 32) {
        int32_t first, len;
        attn_range(a.q_starts, b, a.tq, first, len);
        mine = mine || (tok >= first && tok < first + len);
    }
    if (!__any_sync(0xffffffffu, mine)) return;
    float best = -INFINITY;
    for (int i = lane; i < a.splits; i += 32) best = fmaxf(best, a.part_lse[(static_cast<int64_t>(i) * a.hq + h) * a.tq + tok]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    const float base = best == -INFINITY ? 0.0f : best;
    float total = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < a.splits; ++i) {
        const float w = expf(a.part_lse[(static_cast<int64_t>(i) * a.hq + h) * a.tq + tok] - base);
        total += w;
        if (lane * 4 < a.D && w != 0.0f) {
            const float4 v = *reinterpret_cast<const float4*>(a.part_out + ((static_cast<int64_t>(i) * a.tq + tok) * a.hq + h) * a.D + lane * 4);
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
    }
    const float inv = total > 0.0f ? 1.0f / total : total;
    if (lane * 4 < a.D)
        attn_store4(static_cast<T*>(a.out.p) + tok * a.out.st + h * a.out.sh + lane * 4,
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (lane == 0) a.lse[static_cast<int64_t>(h) * a.tq + tok] = total == 0.0f ? -INFINITY : base + logf(total);
}

template <typename T>
__global__ void __launch_bounds__(kT) attn_delta_kernel(const __grid_constant__ AttnArgs a) {
    if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    // 16 lanes to a row, up to 8 elements each
    const int sub = threadIdx.x & 15;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kT / 16) + (threadIdx.x >> 4);
    const bool live = row < static_cast<int64_t>(a.tq) * a.hq;
    const int64_t tok = live ? row / a.hq : 0;
    const int h = live ? static_cast<int>(row - tok * a.hq) : 0;
    float sum = 0.0f;
    if (live && sub * 8 < a.D) {
        const T* g = static_cast<const T*>(a.g.p) + tok * a.g.st + h * a.g.sh + sub * 8;
        const T* o = static_cast<const T*>(a.out.p) + tok * a.out.st + h * a.out.sh + sub * 8;
        sum = dot4(attn_load4(g), attn_load4(o), dot4(attn_load4(g + 4), attn_load4(o + 4), 0.0f));
    }
    sum = sum16(sum);
    if (live && sub == 0) a.delta[static_cast<int64_t>(h) * a.tq + tok] = sum;
}

template <typename F>
cudaError_t with_smem(F kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T>
cudaError_t forward_t(const AttnArgs& a, cudaStream_t st) {
    const int smem = (2 * kR * (a.D + 4) + kR * kPP) * 4;
    cudaError_t e = with_smem(attn_forward_simt_kernel<T>, smem);
    if (e != cudaSuccess) return e;
    attn_forward_simt_kernel<T>
        <<<dim3(static_cast<unsigned>(a.tiles) * a.splits, static_cast<unsigned>(a.hk)), kT, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_t(const AttnArgs& a, cudaStream_t st) {
    cudaError_t e;
    if (a.tq > 0) {
        const int smem = (4 * kR * (a.D + 4) + kR * kPP) * 4;
        if ((e = with_smem(attn_grad_q_simt_kernel<T>, smem)) != cudaSuccess) return e;
        attn_grad_q_simt_kernel<T><<<dim3(static_cast<unsigned>(a.tiles), static_cast<unsigned>(a.hk)), kT, smem, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.tk > 0) {
        const int smem = (4 * kR * (a.D + 4) + 2 * kR * kPP) * 4;
        if ((e = with_smem(attn_grad_kv_simt_kernel<T>, smem)) != cudaSuccess) return e;
        const unsigned kt = static_cast<unsigned>(attn_tiles(a.tk, a.batch, kC));
        attn_grad_kv_simt_kernel<T><<<dim3(kt, static_cast<unsigned>(a.hk)), kT, smem, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_attention_simt_forward(const AttnArgs& a, cudaStream_t st) { return forward_t<float>(a, st); }

cudaError_t launch_attention_simt_backward(const AttnArgs& a, cudaStream_t st) { return backward_t<float>(a, st); }

template <typename F>
static cudaError_t launch_after(F kernel, int64_t grid, const AttnArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kT);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_attention_join(int dtype, const AttnArgs& a, cudaStream_t st) {
    const int64_t grid = (static_cast<int64_t>(a.tq) * a.hq + kT / 32 - 1) / (kT / 32);
    if (dtype == kF32) return launch_after(attn_join_kernel<float>, grid, a, st);
    if (dtype == kF16) return launch_after(attn_join_kernel<__half>, grid, a, st);
    return launch_after(attn_join_kernel<__nv_bfloat16>, grid, a, st);
}

cudaError_t launch_attention_delta(int dtype, const AttnArgs& a, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.tq) * a.hq + kT / 16 - 1) / (kT / 16));
    if (grid == 0) return a.status ? cudaMemsetAsync(a.status, 0, sizeof(uint32_t), st) : cudaSuccess;
    if (dtype == kF32)
        attn_delta_kernel<float><<<grid, kT, 0, st>>>(a);
    else if (dtype == kF16)
        attn_delta_kernel<__half><<<grid, kT, 0, st>>>(a);
    else
        attn_delta_kernel<__nv_bfloat16><<<grid, kT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace mdcn
