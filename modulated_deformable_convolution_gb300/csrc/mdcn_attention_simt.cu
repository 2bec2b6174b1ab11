// Attention over packed sequences in float32, on the CUDA cores, and the small
// kernels that both forms of the attention use.
//
// Forward, per row: running maximum m and sum l of exp(scale q.k - m) over
// 64-key tiles, accumulator rescaled by exp(m_old - m) when m grows; out =
// acc / l, lse = m + log l. Backward from lse: p = exp(scale q.k - lse), ds =
// p (g.v - delta) scale; some blocks sum ds k over the keys of 64 rows, the
// others p^T g and ds^T q over the rows that see 64 keys, in one launch.
//
// Bound by fp32 multiply-adds. 256 threads hold a 64 x 64 score tile as 4 x 4
// each and a 64 x D accumulator as 4 rows x 4-element pieces; operands come
// from shared memory as 16-byte vectors (rows padded by 4 words, so that the
// 16 rows a warp reads at once fall into different banks), 64 multiply-adds
// for 8 vectors. Tiles are copied to shared memory asynchronously, each as
// soon as the one before it has been used, and two blocks share an SM where
// their tiles fit, so that one computes while the other waits. Tensor cores
// would need three products of reduced precision for one of fp32 (or six
// with 16-bit parts), each with its own copy of the operands.
#include <cfloat>
#include <cstdint>

#include "mdcn_attention.cuh"
#include "mdcn_pdl.h"
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

// 16 bytes to shared memory, asynchronously; zeros where `there` is false.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the latest n groups of this thread's copies have arrived.
template <int n>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// Rows of a packed row tile into shared memory: row r = (token r / group, head
// r % group) of key head kh, zero past the sequence's end. One group of copies.
__device__ __forceinline__ void load_rows(float* dst, int pitch, const AttnTensor& t, const AttnArgs& a,
                                          const AttnSeq& s, int32_t tok0, int32_t ntok, int kh) {
    const int v4 = a.D / 4, rows = ntok * a.group;
    for (int i = threadIdx.x; i < kR * v4; i += kT) {
        const int r = i / v4, c = (i - r * v4) * 4;
        const bool there = r < rows;
        const int tk = there ? r / a.group : 0, h = kh * a.group + (there ? r - tk * a.group : 0);
        copy16(dst + r * pitch + c,
               static_cast<const float*>(t.p) + static_cast<int64_t>(s.q0 + tok0 + tk) * t.st +
                   static_cast<int64_t>(h) * t.sh + c,
               there);
    }
    copies_end();
}

// Keys (or values) [j0, j0 + 64) of the sequence, zero past its last key. One
// group of copies.
__device__ __forceinline__ void load_keys(float* dst, int pitch, const AttnTensor& t, const AttnArgs& a,
                                          const AttnSeq& s, int32_t j0, int kh) {
    const int v4 = a.D / 4;
    for (int i = threadIdx.x; i < kC * v4; i += kT) {
        const int r = i / v4, c = (i - r * v4) * 4;
        const bool there = j0 + r < s.lk;
        copy16(dst + r * pitch + c,
               static_cast<const float*>(t.p) + static_cast<int64_t>(there ? s.k0 + j0 + r : 0) * t.st +
                   static_cast<int64_t>(kh) * t.sh + c,
               there);
    }
    copies_end();
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
__global__ void __launch_bounds__(kT, 2) attn_forward_simt_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ float sm[];
    dependency_wait();
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
    const int tpt = kR / a.group;
    const AttnSeq s = attn_find(a, false, tpt, blockIdx.x / a.splits);
    if (s.tile < 0) return;
    const int kh = blockIdx.y, split = blockIdx.x % a.splits;
    const int pitch = a.D + 4;
    float* qs = sm;
    float* ks = qs + kR * pitch;
    float* vs = ks + kC * pitch;
    float* ps = vs + kC * pitch;
    const int32_t tok0 = s.tile * tpt, ntok = min(tpt, s.lq - tok0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t most = attn_seen(a, s, tok0 + ntok - 1);
    const int32_t ktiles = (most + kC - 1) / kC, per = (ktiles + a.splits - 1) / a.splits;
    const int32_t t0 = min(split * per, ktiles), t1 = min(t0 + per, ktiles);
    load_rows(qs, pitch, a.q, a, s, tok0, ntok, kh);
    if (t0 < t1) load_keys(ks, pitch, a.k, a, s, t0 * kC, kh);

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
    const float to_log2 = a.scale * kLog2e;
    for (int32_t t = t0; t < t1; ++t) {
        load_keys(vs, pitch, a.v, a, s, t * kC, kh);
        copies_wait<1>();  // the keys
        __syncthreads();
        float x[4][4];
        products(x, qs, ks, pitch, a.D, tx, ty);
        __syncthreads();
        if (t + 1 < t1)
            load_keys(ks, pitch, a.k, a, s, (t + 1) * kC, kh);
        else
            copies_end();
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
        copies_wait<1>();  // the values
        __syncthreads();
        accumulate(o, ps, vs, pitch, a.D, tx, ty);
        __syncthreads();
    }
    copies_wait<0>();
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
                *reinterpret_cast<float4*>(static_cast<float*>(a.out.p) + tok * a.out.st + h * a.out.sh + d) = v;
        }
        if (tx == 0) {
            if (a.splits > 1)
                a.part_lse[(static_cast<int64_t>(split) * a.hq + h) * a.tq + tok] = lse;
            else
                a.lse[static_cast<int64_t>(h) * a.tq + tok] = lse;
        }
    }
}

// grad_q of one row tile.
__device__ __forceinline__ void grad_q_block(const AttnArgs& a, float* sm, int32_t index, int kh) {
    const int tpt = kR / a.group;
    const AttnSeq s = attn_find(a, false, tpt, index);
    if (s.tile < 0) return;
    const int pitch = a.D + 4;
    float* qs = sm;
    float* gs = qs + kR * pitch;
    float* ks = gs + kR * pitch;
    float* vs = ks + kC * pitch;
    float* ps = vs + kC * pitch;
    const int32_t tok0 = s.tile * tpt, ntok = min(tpt, s.lq - tok0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t ktiles = (attn_seen(a, s, tok0 + ntok - 1) + kC - 1) / kC;
    load_rows(qs, pitch, a.q, a, s, tok0, ntok, kh);
    load_rows(gs, pitch, a.g, a, s, tok0, ntok, kh);
    if (ktiles > 0) {
        load_keys(ks, pitch, a.k, a, s, 0, kh);
        load_keys(vs, pitch, a.v, a, s, 0, kh);
    }
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
    for (int32_t t = 0; t < ktiles; ++t) {
        copies_wait<1>();  // the keys
        __syncthreads();
        float x[4][4], dp[4][4];
        products(x, qs, ks, pitch, a.D, tx, ty);
        copies_wait<0>();  // the values
        __syncthreads();
        products(dp, gs, vs, pitch, a.D, tx, ty);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool on = t * kC + tx + 16 * j < seen[i];
                // s - lse is rounded once, before the small difference is scaled
                const float p = on ? exp2f(fmaf(x[i][j], a.scale, -lse[i]) * kLog2e) : 0.0f;
                ps[(ty + 16 * i) * kPP + tx + 16 * j] = on ? p * (dp[i][j] - delta[i]) : 0.0f;
            }
        __syncthreads();
        accumulate(o, ps, ks, pitch, a.D, tx, ty);
        __syncthreads();
        if (t + 1 < ktiles) {
            load_keys(ks, pitch, a.k, a, s, (t + 1) * kC, kh);
            load_keys(vs, pitch, a.v, a, s, (t + 1) * kC, kh);
        }
    }
    copies_wait<0>();
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
                *reinterpret_cast<float4*>(static_cast<float*>(a.gq.p) + tok * a.gq.st + h * a.gq.sh + d) =
                    make_float4(o[i][c].x * a.scale, o[i][c].y * a.scale, o[i][c].z * a.scale, o[i][c].w * a.scale);
        }
    }
}

// o[i] (row 4 ty + i) += sum over the 64 rows r of p[r][row] * y[r]
__device__ __forceinline__ void accumulate_t(float4 (&o)[4][kAcc], const float* p, const float* y, int pitch, int D,
                                             int tx, int ty) {
#pragma unroll 4
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

// grad_k and grad_v of 64 keys of one key head, or (a.kv_splits > 1) the sums
// over a share of the row tiles that see them. P, then dS, in one buffer.
__device__ __forceinline__ void grad_kv_block(const AttnArgs& a, float* sm, int32_t index, int32_t split, int kh) {
    const AttnSeq s = attn_find(a, true, kC, index);
    if (s.tile < 0) return;
    const int pitch = a.D + 4, tpt = kR / a.group;
    float* qs = sm;
    float* gs = qs + kR * pitch;
    float* ks = gs + kR * pitch;
    float* vs = ks + kC * pitch;
    float* ps = vs + kC * pitch;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int32_t j0 = s.tile * kC;
    float4 ok[4][kAcc], ov[4][kAcc];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < kAcc; ++c) ok[i][c] = ov[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    // row tiles from the first that sees key j0
    const int32_t first = a.causal ? max(0, j0 + s.lq - s.lk) / tpt : 0;
    const int32_t tiles = j0 < s.lk ? max(0, (s.lq + tpt - 1) / tpt - first) : 0;
    const int32_t per = (tiles + a.kv_splits - 1) / a.kv_splits;
    const int32_t b0 = first + min(split * per, tiles), b1 = first + min(split * per + per, tiles);
    if (b0 < b1) {
        load_keys(ks, pitch, a.k, a, s, j0, kh);
        load_keys(vs, pitch, a.v, a, s, j0, kh);
        load_rows(qs, pitch, a.q, a, s, b0 * tpt, min(tpt, s.lq - b0 * tpt), kh);
        load_rows(gs, pitch, a.g, a, s, b0 * tpt, min(tpt, s.lq - b0 * tpt), kh);
    }
    for (int32_t b = b0; b < b1; ++b) {
        const int32_t tok0 = b * tpt, ntok = min(tpt, s.lq - tok0);
        float lse[4], delta[4];
        int32_t seen[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            const bool live = r < ntok * a.group;
            const int64_t at =
                live ? static_cast<int64_t>(kh * a.group + r % a.group) * a.tq + s.q0 + tok0 + r / a.group : 0;
            seen[i] = live ? attn_seen(a, s, tok0 + r / a.group) : 0;
            lse[i] = live ? a.lse[at] : 0.0f;
            delta[i] = live ? a.delta[at] : 0.0f;
        }
        copies_wait<1>();  // the queries
        __syncthreads();
        float x[4][4], dp[4][4];
        products(x, qs, ks, pitch, a.D, tx, ty);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool on = j0 + tx + 16 * j < seen[i];
                x[i][j] = on ? exp2f(fmaf(x[i][j], a.scale, -lse[i]) * kLog2e) : 0.0f;
                ps[(ty + 16 * i) * kPP + tx + 16 * j] = x[i][j];
            }
        copies_wait<0>();  // the gradients
        __syncthreads();
        products(dp, gs, vs, pitch, a.D, tx, ty);
        accumulate_t(ov, ps, gs, pitch, a.D, tx, ty);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool on = j0 + tx + 16 * j < seen[i];
                ps[(ty + 16 * i) * kPP + tx + 16 * j] = on ? x[i][j] * (dp[i][j] - delta[i]) : 0.0f;
            }
        __syncthreads();
        accumulate_t(ok, ps, qs, pitch, a.D, tx, ty);
        __syncthreads();
        if (b + 1 < b1) {
            load_rows(qs, pitch, a.q, a, s, tok0 + tpt, min(tpt, s.lq - tok0 - tpt), kh);
            load_rows(gs, pitch, a.g, a, s, tok0 + tpt, min(tpt, s.lq - tok0 - tpt), kh);
        }
    }
    copies_wait<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t j = j0 + ty * 4 + i;
        if (j >= s.room) continue;
        const int64_t row = s.k0 + j;
#pragma unroll
        for (int c = 0; c < kAcc; ++c) {
            const int d = tx * 4 + 64 * c;
            if (d >= a.D) continue;
            const float4 k = make_float4(ok[i][c].x * a.scale, ok[i][c].y * a.scale, ok[i][c].z * a.scale, ok[i][c].w * a.scale);
            if (a.kv_splits > 1) {
                float* at = a.part_kv + ((static_cast<int64_t>(split) * 2 * a.tk + row) * a.hk + kh) * a.D + d;
                *reinterpret_cast<float4*>(at) = k;
                *reinterpret_cast<float4*>(at + static_cast<int64_t>(a.tk) * a.hk * a.D) = ov[i][c];
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(a.gk.p) + row * a.gk.st + kh * a.gk.sh + d) = k;
                *reinterpret_cast<float4*>(static_cast<float*>(a.gv.p) + row * a.gv.st + kh * a.gv.sh + d) = ov[i][c];
            }
        }
    }
}

// Grid: (key tiles * kv_splits + row tiles, key heads): the longer blocks first.
__global__ void __launch_bounds__(kT) attn_backward_simt_kernel(const __grid_constant__ AttnArgs a, int32_t kv_blocks) {
    extern __shared__ float sm[];
    dependency_wait();
    const int32_t b = blockIdx.x;
    if (b < kv_blocks)
        grad_kv_block(a, sm, b / a.kv_splits, b % a.kv_splits, blockIdx.y);
    else
        grad_q_block(a, sm, b - kv_blocks, blockIdx.y);
}

// grad_k (y 0) or grad_v (y 1): the shares' sums added in order, for the keys of a sequence.
__global__ void __launch_bounds__(kT) attn_kv_sum_kernel(const __grid_constant__ AttnArgs a) {
    dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kT / 32) + (threadIdx.x >> 5);  // (key, head)
    if (row >= static_cast<int64_t>(a.tk) * a.hk) return;
    const int64_t key = row / a.hk;
    const int kh = static_cast<int>(row - key * a.hk);
    bool mine = false;  // keys of no sequence are not written
    for (int b = lane; b < a.batch; b += 32) {
        int32_t first, len;
        attn_range(a.k_starts, b, a.tk, first, len);
        mine = mine || (key >= first && key < first + len);
    }
    if (!__any_sync(0xffffffffu, mine) || lane * 4 >= a.D) return;
    const int64_t one = static_cast<int64_t>(a.tk) * a.hk * a.D;
    const float* p = a.part_kv + blockIdx.y * one + row * a.D + lane * 4;
    float4 sum = *reinterpret_cast<const float4*>(p);
    for (int i = 1; i < a.kv_splits; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(p + 2 * i * one);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    const AttnTensor& t = blockIdx.y ? a.gv : a.gk;
    *reinterpret_cast<float4*>(static_cast<float*>(t.p) + key * t.st + kh * t.sh + lane * 4) = sum;
}

// out = sum over the shares of exp(lse_i - lse) out_i; 16 lanes per (token,
// head), up to 8 elements each.
template <typename T>
__global__ void __launch_bounds__(kT) attn_join_kernel(const __grid_constant__ AttnArgs a) {
    dependency_wait();
    const int sub = threadIdx.x & 15;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kT / 16) + (threadIdx.x >> 4);
    const bool real = row < static_cast<int64_t>(a.tq) * a.hq;
    const int64_t tok = real ? row / a.hq : 0;
    const int h = real ? static_cast<int>(row - tok * a.hq) : 0;
    // rows of no sequence have no partial results and are not written
    float mine = 0.0f;
    for (int b = sub; b < a.batch; b += 16) {
        int32_t first, len;
        attn_range(a.q_starts, b, a.tq, first, len);
        if (real && tok >= first && tok < first + len) mine = 1.0f;
    }
    const bool live = max16(mine) > 0.0f;
    float best = -INFINITY;
    for (int i = sub; live && i < a.splits; i += 16)
        best = fmaxf(best, a.part_lse[(static_cast<int64_t>(i) * a.hq + h) * a.tq + tok]);
    best = max16(best);
    if (!live) return;
    const float base = best == -INFINITY ? 0.0f : best;
    const bool on = sub * 8 < a.D;
    float total = 0.0f;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll 4
    for (int i = 0; i < a.splits; ++i) {
        const float w = expf(a.part_lse[(static_cast<int64_t>(i) * a.hq + h) * a.tq + tok] - base);
        total += w;
        if (on) {
            const float* p = a.part_out + ((static_cast<int64_t>(i) * a.tq + tok) * a.hq + h) * a.D + sub * 8;
            const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
            // a share without a key holds zeros
            u.x = fmaf(w, x.x, u.x);
            u.y = fmaf(w, x.y, u.y);
            u.z = fmaf(w, x.z, u.z);
            u.w = fmaf(w, x.w, u.w);
            v.x = fmaf(w, y.x, v.x);
            v.y = fmaf(w, y.y, v.y);
            v.z = fmaf(w, y.z, v.z);
            v.w = fmaf(w, y.w, v.w);
        }
    }
    const float inv = total > 0.0f ? 1.0f / total : total;
    if (on) {
        T* o = static_cast<T*>(a.out.p) + tok * a.out.st + h * a.out.sh + sub * 8;
        attn_store4(o, make_float4(u.x * inv, u.y * inv, u.z * inv, u.w * inv));
        attn_store4(o + 4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    }
    if (sub == 0) a.lse[static_cast<int64_t>(h) * a.tq + tok] = total == 0.0f ? -INFINITY : base + logf(total);
}

template <typename T>
__global__ void __launch_bounds__(kT) attn_delta_kernel(const __grid_constant__ AttnArgs a) {
    dependency_wait();
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

}  // namespace

cudaError_t launch_attention_simt_forward(const AttnArgs& a, cudaStream_t st) {
    const int smem = (3 * kR * (a.D + 4) + kR * kPP) * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = attn_allow_smem(attn_forward_simt_kernel, (3 * kR * 132 + kR * kPP) * 4, done);  // head_dim 128
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_forward_simt_kernel, dim3(static_cast<unsigned>(a.tiles) * a.splits, static_cast<unsigned>(a.hk)),
                            kT, smem, st, a);
}

cudaError_t launch_attention_simt_backward(const AttnArgs& a, cudaStream_t st) {
    const int smem = (4 * kR * (a.D + 4) + kR * kPP) * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = attn_allow_smem(attn_backward_simt_kernel, (4 * kR * 132 + kR * kPP) * 4, done);  // head_dim 128
    if (e != cudaSuccess) return e;
    const int32_t kv = static_cast<int32_t>(attn_tiles(a.tk, a.batch, kC)) * a.kv_splits;
    const int32_t blocks = kv + (a.tq > 0 ? a.tiles : 0);
    if (blocks == 0) return cudaSuccess;
    e = launch_dependent(attn_backward_simt_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.hk)), kT, smem,
                         st, a, kv);
    if (e != cudaSuccess || a.kv_splits == 1) return e;
    const int64_t rows = static_cast<int64_t>(a.tk) * a.hk;
    return launch_dependent(attn_kv_sum_kernel, dim3(static_cast<unsigned>((rows + kT / 32 - 1) / (kT / 32)), 2), kT, 0, st, a);
}

cudaError_t launch_attention_join(int dtype, const AttnArgs& a, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.tq) * a.hq + kT / 16 - 1) / (kT / 16)));
    if (dtype == kF32) return launch_dependent(attn_join_kernel<float>, grid, kT, 0, st, a);
    if (dtype == kF16) return launch_dependent(attn_join_kernel<__half>, grid, kT, 0, st, a);
    return launch_dependent(attn_join_kernel<__nv_bfloat16>, grid, kT, 0, st, a);
}

cudaError_t launch_attention_delta(int dtype, const AttnArgs& a, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.tq) * a.hq + kT / 16 - 1) / (kT / 16));
    if (grid == 0) return a.status ? cudaMemsetAsync(a.status, 0, sizeof(uint32_t), st) : cudaSuccess;
    if (dtype == kF32) return launch_dependent(attn_delta_kernel<float>, grid, kT, 0, st, a);
    if (dtype == kF16) return launch_dependent(attn_delta_kernel<__half>, grid, kT, 0, st, a);
    return launch_dependent(attn_delta_kernel<__nv_bfloat16>, grid, kT, 0, st, a);
}

}  // namespace mdcn
