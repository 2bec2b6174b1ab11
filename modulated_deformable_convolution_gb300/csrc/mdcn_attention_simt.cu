// Attention over packed sequences in float32, on the CUDA cores, and the small
// kernels that both forms of the attention use.
//
// Forward, per row: running maximum m and sum l of exp(scale q.k - m) over
// 64-key tiles, accumulator rescaled by exp(m_old - m) when m grows; out =
// acc / l, lse = m + log l. Backward from lse: p = exp(scale q.k - lse), ds =
// p (g.v - delta) scale; some blocks sum ds k over the keys of 64 rows, the
// others p^T g and ds^T q over the rows that see 64 keys, in one launch.
//
// Bound by fp32 multiply-adds and, as near, by the reads of their operands from
// shared memory. 128 threads hold a 64 x 64 score tile as 4 rows x 8 keys each
// (12 16-byte reads for 128 multiply-adds; 4 x 4 has 16) and a 64 x D
// accumulator as 4 rows x D / 8 elements; two multiply-adds go to an
// instruction, on pairs of elements. Loops over a head have constant bounds, by
// sixteens of D. Tiles are copied to shared memory asynchronously, each as soon
// as the one before it has been used, and two or three blocks share an SM where
// their tiles fit, so that one computes while another waits. Tensor cores would
// need three products of TF32 parts for one of fp32, each with its own copy of
// the operands, and leave products some 2^-22 off where fp32 rounds to 2^-24.
// Measured: forward, 2 sequences of 2048, 8 heads of 64 over 4: 470 us, 36
// TFLOP/s of the 70 that a large float32 matrix product reaches; 6 maps of up to
// 32 x 32, 8 heads of 40 over 4: 77 us. Backward, 4 ragged sequences of up to 700,
// 6 heads of 72 over 2: 94 us; 2 causal sequences of 2048, 6 heads of 64 over 2: 615
// us, 37 TFLOP/s of seven products (without the mask 1180 us, 38).
#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "mdcn_attention.cuh"
#include "mdcn_pdl.h"
#include "mdcn_plan.h"

namespace mdcn {

namespace {

constexpr int kR = kAttnSimtRows;  // rows of a tile
constexpr int kC = 64;             // keys of a tile
constexpr int kT = 256;            // threads of the small kernels
constexpr int kTT = 128;           // threads to a tile
constexpr int kPP = kC + 8;        // padded row of the probability tile

// Of a head of 16 kN elements at most: words of a padded row in shared memory.
// A multiple of 4 and, in units of 4, odd: 8 rows that are read at once lie in
// different banks.
__host__ __device__ constexpr int pitch_of(int kN) { return 16 * kN + 4; }

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

// The part that a thread copies: every second 4-element piece of one row of 64.
struct Copier {
    int row, half;
    int tk, head;  // of a row tile's row: its token and head within the tile

    __device__ __forceinline__ explicit Copier(int group) {
        row = threadIdx.x >> 1;
        half = threadIdx.x & 1;
        tk = row / group;
        head = row - tk * group;
    }
    // One group of copies: the row, with zeros past the head's elements, or all zeros.
    template <int kN>
    __device__ __forceinline__ void copy(float* dst, const float* src, bool there, int D) const {
        float* to = dst + row * pitch_of(kN) + half * 4;
        src += half * 4;
#pragma unroll
        for (int c = 0; c < 2 * kN; ++c) {
            const bool in = there && 8 * c + 4 * half < D;
            copy16(to + 8 * c, in ? src + 8 * c : src, in);
        }
        copies_end();
    }
    // Rows of a packed row tile: row r = (token r / group, head r % group) of
    // key head kh, zero past the sequence's end.
    template <int kN>
    __device__ __forceinline__ void rows(float* dst, const AttnTensor& t, const AttnArgs& a, const AttnSeq& s,
                                         int32_t tok0, int32_t ntok, int kh) const {
        const bool there = tk < ntok;
        copy<kN>(dst,
                 static_cast<const float*>(t.p) +
                     (there ? static_cast<int64_t>(s.q0 + tok0 + tk) * t.st + static_cast<int64_t>(kh * a.group + head) * t.sh
                            : 0),
                 there, a.D);
    }
    // Keys (or values) [j0, j0 + 64) of the sequence, zero past its last key.
    template <int kN>
    __device__ __forceinline__ void keys(float* dst, const AttnTensor& t, const AttnArgs& a, const AttnSeq& s,
                                         int32_t j0, int kh) const {
        const bool there = j0 + row < s.lk;
        copy<kN>(dst,
                 static_cast<const float*>(t.p) +
                     (there ? static_cast<int64_t>(s.k0 + j0 + row) * t.st + static_cast<int64_t>(kh) * t.sh : 0),
                 there, a.D);
    }
};

// The 4 rows of a thread (ty + 16 i): their tokens, heads and whether they are of the tile.
struct Rows {
    int tk[4], head[4];

    __device__ __forceinline__ Rows(int ty, int group) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            tk[i] = (ty + 16 * i) / group;
            head[i] = ty + 16 * i - tk[i] * group;
        }
    }
};

// acc[i][j] = row (ty + 16 i) of x . row (tx + 8 j) of y: even and odd elements
// summed apart, two multiply-adds to an instruction.
template <int kN>
__device__ __forceinline__ void products(float (&acc)[4][8], const float* x, const float* y, int tx, int ty) {
    constexpr int kPitch = pitch_of(kN);
    uint64_t s[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = 0;
    const float* xr = x + ty * kPitch;
    const float* yr = y + tx * kPitch;
#pragma unroll 2
    for (int d = 0; d < 16 * kN; d += 4) {
        ulonglong2 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const ulonglong2*>(xr + 16 * i * kPitch + d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(yr + 8 * j * kPitch + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i][j] = fma2(u[i].y, w.y, fma2(u[i].x, w.x, s[i][j]));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float lo, hi;
            unpack2(s[i][j], lo, hi);
            acc[i][j] = lo + hi;
        }
}

// A thread's elements of a row of 16 kN: pairs, two in each 4-element piece
// 4 tx + 32 c, and one at 2 tx of the last 16 where kN is odd.
template <int kN>
__device__ __forceinline__ int element(int pair, int tx) {
    return pair < 2 * (kN / 2) ? 4 * tx + 32 * (pair / 2) + 2 * (pair & 1) : 32 * (kN / 2) + 2 * tx;
}

template <int kN>
using Sums = uint64_t[4][kN];

// o[i] += f[i] * row y, for the thread's elements.
template <int kN>
__device__ __forceinline__ void add_row(Sums<kN>& o, const float (&f)[4], const float* y, int tx) {
    uint64_t f2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2[i] = pack2(f[i], f[i]);
#pragma unroll
    for (int c = 0; c < kN / 2; ++c) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(y + 4 * tx + 32 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i][2 * c] = fma2(f2[i], v.x, o[i][2 * c]);
            o[i][2 * c + 1] = fma2(f2[i], v.y, o[i][2 * c + 1]);
        }
    }
    if constexpr (kN & 1) {
        const uint64_t v = *reinterpret_cast<const uint64_t*>(y + 32 * (kN / 2) + 2 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i][kN - 1] = fma2(f2[i], v, o[i][kN - 1]);
    }
}

// o[i] (row ty + 16 i) += sum over the 64 columns j of p[row][j] * y[j]
template <int kN>
__device__ __forceinline__ void accumulate(Sums<kN>& o, const float* p, const float* y, int tx, int ty) {
    constexpr int kPitch = pitch_of(kN);
#pragma unroll 1
    for (int j = 0; j < kC; j += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + (ty + 16 * i) * kPP + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
            add_row<kN>(o, f, y + (j + jj) * kPitch, tx);
        }
    }
}

// o[i] (row 4 ty + i) += sum over the 64 rows r of p[r][row] * y[r]
template <int kN>
__device__ __forceinline__ void accumulate_t(Sums<kN>& o, const float* p, const float* y, int tx, int ty) {
#pragma unroll 4
    for (int r = 0; r < kR; ++r) {
        const float4 w = *reinterpret_cast<const float4*>(p + r * kPP + ty * 4);
        const float f[4] = {w.x, w.y, w.z, w.w};
        add_row<kN>(o, f, y + r * pitch_of(kN), tx);
    }
}

template <int kN>
__device__ __forceinline__ void clear(Sums<kN>& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < kN; ++c) o[i][c] = 0;
}

// The thread's elements of a row times f to `to`.
template <int kN>
__device__ __forceinline__ void store_row(float* to, const uint64_t (&o)[kN], float f, int D, int tx) {
#pragma unroll
    for (int c = 0; c < kN; ++c) {
        const int d = element<kN>(c, tx);
        float lo, hi;
        unpack2(o[c], lo, hi);
        if (d < D) *reinterpret_cast<float2*>(to + d) = make_float2(lo * f, hi * f);
    }
}

// Over the 8 lanes (tx) that share rows.
__device__ __forceinline__ float max8(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float max16(float v) { return max8(fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8))); }
__device__ __forceinline__ float sum16(float v) { return sum8(v + __shfl_xor_sync(0xffffffffu, v, 8)); }

// Grid: tiles * splits * key heads, the heads of one share of one tile side by
// side, so that blocks of one length are spread evenly over the SMs. A block
// takes the split-th share of the key tiles that its tile's rows see.
template <int kN>
__global__ void __launch_bounds__(kTT, kN <= 4 ? 3 : 2) attn_forward_simt_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ float sm[];
    dependency_wait();
    if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    const int tpt = kR / a.group;
    const int item = blockIdx.x / a.hk, kh = blockIdx.x - item * a.hk, split = item % a.splits;
    const AttnSeq s = attn_find(a, false, tpt, item / a.splits);
    if (s.tile < 0) return;
    constexpr int kPitch = pitch_of(kN);
    float* qs = sm;
    float* ks = qs + kR * kPitch;
    float* vs = ks + kC * kPitch;
    float* ps = vs + kC * kPitch;
    const int32_t tok0 = s.tile * tpt, ntok = min(tpt, s.lq - tok0);
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int32_t most = attn_seen(a, s, tok0 + ntok - 1);
    const int32_t ktiles = (most + kC - 1) / kC, per = (ktiles + a.splits - 1) / a.splits;
    const int32_t t0 = min(split * per, ktiles), t1 = min(t0 + per, ktiles);
    const Copier mine(a.group);
    mine.rows<kN>(qs, a.q, a, s, tok0, ntok, kh);
    if (t0 < t1) mine.keys<kN>(ks, a.k, a, s, t0 * kC, kh);

    const Rows rows(ty, a.group);
    int32_t seen[4];
    float m[4], l[4];
    Sums<kN> o;
    clear<kN>(o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        seen[i] = rows.tk[i] < ntok ? attn_seen(a, s, tok0 + rows.tk[i]) : 0;
        m[i] = -INFINITY;
        l[i] = 0.0f;
    }
    const float to_log2 = a.scale * kLog2e;
#pragma unroll 1
    for (int32_t t = t0; t < t1; ++t) {
        mine.keys<kN>(vs, a.v, a, s, t * kC, kh);
        copies_wait<1>();  // the keys
        __syncthreads();
        float x[4][8];
        products<kN>(x, qs, ks, tx, ty);
        __syncthreads();
        if (t + 1 < t1)
            mine.keys<kN>(ks, a.k, a, s, (t + 1) * kC, kh);
        else
            copies_end();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float best = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = t * kC + tx + 8 * j < seen[i] ? x[i][j] * to_log2 : -INFINITY;
                best = fmaxf(best, x[i][j]);
            }
            best = fmaxf(max8(best), m[i]);
            const float base = best == -INFINITY ? 0.0f : best;  // no key seen so far: every term is exp2(-inf) = 0
            const float corr = exp2f(m[i] - base);
            m[i] = best;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = exp2f(x[i][j] - base);
                sum += p;
                ps[(ty + 16 * i) * kPP + tx + 8 * j] = p;
            }
            l[i] = fmaf(l[i], corr, sum8(sum));
            const uint64_t corr2 = pack2(corr, corr);
#pragma unroll
            for (int c = 0; c < kN; ++c) o[i][c] = mul2(o[i][c], corr2);
        }
        copies_wait<1>();  // the values
        __syncthreads();
        accumulate<kN>(o, ps, vs, tx, ty);
        __syncthreads();
    }
    copies_wait<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (rows.tk[i] >= ntok) continue;
        const int64_t tok = s.q0 + tok0 + rows.tk[i];
        const int h = kh * a.group + rows.head[i];
        const float inv = l[i] > 0.0f ? 1.0f / l[i] : (l[i] == 0.0f ? 0.0f : l[i]);
        const float lse = l[i] == 0.0f ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
        float* to = a.splits > 1 ? a.part_out + ((static_cast<int64_t>(split) * a.tq + tok) * a.hq + h) * a.D
                                 : static_cast<float*>(a.out.p) + tok * a.out.st + h * a.out.sh;
        store_row<kN>(to, o[i], inv, a.D, tx);
        if (tx == 0) {
            if (a.splits > 1)
                a.part_lse[(static_cast<int64_t>(split) * a.hq + h) * a.tq + tok] = lse;
            else
                a.lse[static_cast<int64_t>(h) * a.tq + tok] = lse;
        }
    }
}

// grad_q of one row tile, or (a.q_splits > 1) the sum over a share of the key
// tiles that it sees.
template <int kN>
__device__ __forceinline__ void grad_q_block(const AttnArgs& a, float* sm, int32_t index, int32_t split, int kh) {
    const int tpt = kR / a.group;
    const AttnSeq s = attn_find(a, false, tpt, index);
    if (s.tile < 0) return;
    constexpr int kPitch = pitch_of(kN);
    float* qs = sm;
    float* gs = qs + kR * kPitch;
    float* ks = gs + kR * kPitch;
    float* vs = ks + kC * kPitch;
    float* ps = vs + kC * kPitch;
    const int32_t tok0 = s.tile * tpt, ntok = min(tpt, s.lq - tok0);
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int32_t ktiles = (attn_seen(a, s, tok0 + ntok - 1) + kC - 1) / kC, per = (ktiles + a.q_splits - 1) / a.q_splits;
    const int32_t t0 = min(split * per, ktiles), t1 = min(t0 + per, ktiles);
    const Copier mine(a.group);
    if (t0 < t1) {
        mine.rows<kN>(qs, a.q, a, s, tok0, ntok, kh);
        mine.rows<kN>(gs, a.g, a, s, tok0, ntok, kh);
        mine.keys<kN>(ks, a.k, a, s, t0 * kC, kh);
        mine.keys<kN>(vs, a.v, a, s, t0 * kC, kh);
    }
    const Rows rows(ty, a.group);
    int32_t seen[4];
    float lse[4], delta[4];
    Sums<kN> o;
    clear<kN>(o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool live = rows.tk[i] < ntok;
        const int64_t at =
            live ? static_cast<int64_t>(kh * a.group + rows.head[i]) * a.tq + s.q0 + tok0 + rows.tk[i] : 0;
        seen[i] = live ? attn_seen(a, s, tok0 + rows.tk[i]) : 0;
        lse[i] = live ? a.lse[at] : 0.0f;
        delta[i] = live ? a.delta[at] : 0.0f;
    }
#pragma unroll 1
    for (int32_t t = t0; t < t1; ++t) {
        copies_wait<1>();  // the keys
        __syncthreads();
        float x[4][8], dp[4][8];
        products<kN>(x, qs, ks, tx, ty);
        copies_wait<0>();  // the values
        __syncthreads();
        products<kN>(dp, gs, vs, tx, ty);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool on = t * kC + tx + 8 * j < seen[i];
                // s - lse is rounded once, before the small difference is scaled
                const float p = on ? exp2f(fmaf(x[i][j], a.scale, -lse[i]) * kLog2e) : 0.0f;
                ps[(ty + 16 * i) * kPP + tx + 8 * j] = on ? p * (dp[i][j] - delta[i]) : 0.0f;
            }
        __syncthreads();
        accumulate<kN>(o, ps, ks, tx, ty);
        __syncthreads();
        if (t + 1 < t1) {
            mine.keys<kN>(ks, a.k, a, s, (t + 1) * kC, kh);
            mine.keys<kN>(vs, a.v, a, s, (t + 1) * kC, kh);
        }
    }
    copies_wait<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (rows.tk[i] >= ntok) continue;
        const int64_t tok = s.q0 + tok0 + rows.tk[i];
        const int h = kh * a.group + rows.head[i];
        float* to = a.q_splits > 1 ? a.part_q + ((static_cast<int64_t>(split) * a.tq + tok) * a.hq + h) * a.D
                                   : static_cast<float*>(a.gq.p) + tok * a.gq.st + h * a.gq.sh;
        store_row<kN>(to, o[i], a.scale, a.D, tx);
    }
}

// grad_k and grad_v of 64 keys of one key head, or (a.kv_splits > 1) the sums
// over a share of the row tiles that see them. P, then dS, in one buffer.
template <int kN>
__device__ __forceinline__ void grad_kv_block(const AttnArgs& a, float* sm, int32_t index, int32_t split, int kh) {
    const AttnSeq s = attn_find(a, true, kC, index);
    if (s.tile < 0) return;
    constexpr int kPitch = pitch_of(kN);
    const int tpt = kR / a.group;
    float* qs = sm;
    float* gs = qs + kR * kPitch;
    float* ks = gs + kR * kPitch;
    float* vs = ks + kC * kPitch;
    float* ps = vs + kC * kPitch;
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int32_t j0 = s.tile * kC;
    Sums<kN> ok, ov;
    clear<kN>(ok);
    clear<kN>(ov);
    // row tiles from the first that sees key j0
    const int32_t first = a.causal ? max(0, j0 + s.lq - s.lk) / tpt : 0;
    const int32_t tiles = j0 < s.lk ? max(0, (s.lq + tpt - 1) / tpt - first) : 0;
    const int32_t per = (tiles + a.kv_splits - 1) / a.kv_splits;
    const int32_t b0 = first + min(split * per, tiles), b1 = first + min(split * per + per, tiles);
    const Copier mine(a.group);
    if (b0 < b1) {
        mine.keys<kN>(ks, a.k, a, s, j0, kh);
        mine.keys<kN>(vs, a.v, a, s, j0, kh);
        mine.rows<kN>(qs, a.q, a, s, b0 * tpt, min(tpt, s.lq - b0 * tpt), kh);
        mine.rows<kN>(gs, a.g, a, s, b0 * tpt, min(tpt, s.lq - b0 * tpt), kh);
    }
    const Rows rows(ty, a.group);
#pragma unroll 1
    for (int32_t b = b0; b < b1; ++b) {
        const int32_t tok0 = b * tpt, ntok = min(tpt, s.lq - tok0);
        float lse[4], delta[4];
        int32_t seen[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool live = rows.tk[i] < ntok;
            const int64_t at =
                live ? static_cast<int64_t>(kh * a.group + rows.head[i]) * a.tq + s.q0 + tok0 + rows.tk[i] : 0;
            seen[i] = live ? attn_seen(a, s, tok0 + rows.tk[i]) : 0;
            lse[i] = live ? a.lse[at] : 0.0f;
            delta[i] = live ? a.delta[at] : 0.0f;
        }
        copies_wait<1>();  // the queries
        __syncthreads();
        float x[4][8];
        products<kN>(x, qs, ks, tx, ty);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool on = j0 + tx + 8 * j < seen[i];
                ps[(ty + 16 * i) * kPP + tx + 8 * j] =
                    on ? exp2f(fmaf(x[i][j], a.scale, -lse[i]) * kLog2e) : 0.0f;
            }
        copies_wait<0>();  // the gradients
        __syncthreads();
        accumulate_t<kN>(ov, ps, gs, tx, ty);
        products<kN>(x, gs, vs, tx, ty);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float* p = ps + (ty + 16 * i) * kPP + tx + 8 * j;
                *p = j0 + tx + 8 * j < seen[i] ? *p * (x[i][j] - delta[i]) : 0.0f;
            }
        __syncthreads();
        accumulate_t<kN>(ok, ps, qs, tx, ty);
        __syncthreads();
        if (b + 1 < b1) {
            mine.rows<kN>(qs, a.q, a, s, tok0 + tpt, min(tpt, s.lq - tok0 - tpt), kh);
            mine.rows<kN>(gs, a.g, a, s, tok0 + tpt, min(tpt, s.lq - tok0 - tpt), kh);
        }
    }
    copies_wait<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t j = j0 + ty * 4 + i;
        if (j >= s.room) continue;
        const int64_t row = s.k0 + j;
        float* to_k = static_cast<float*>(a.gk.p) + row * a.gk.st + kh * a.gk.sh;
        float* to_v = static_cast<float*>(a.gv.p) + row * a.gv.st + kh * a.gv.sh;
        if (a.kv_splits > 1) {
            to_k = a.part_kv + ((static_cast<int64_t>(split) * 2 * a.tk + row) * a.hk + kh) * a.D;
            to_v = to_k + static_cast<int64_t>(a.tk) * a.hk * a.D;
        }
        store_row<kN>(to_k, ok[i], a.scale, a.D, tx);
        store_row<kN>(to_v, ov[i], 1.0f, a.D, tx);
    }
}

// Grid: (key tiles * kv_splits + row tiles * q_splits) * key heads.
template <int kN>
__global__ void __launch_bounds__(kTT, 2)
    attn_backward_simt_kernel(const __grid_constant__ AttnArgs a, int32_t kv_blocks) {
    extern __shared__ float sm[];
    dependency_wait();
    const int32_t b = blockIdx.x / a.hk, kh = blockIdx.x - b * a.hk;
    if (b < kv_blocks)
        grad_kv_block<kN>(a, sm, b / a.kv_splits, b % a.kv_splits, kh);
    else
        grad_q_block<kN>(a, sm, (b - kv_blocks) / a.q_splits, (b - kv_blocks) % a.q_splits, kh);
}

// The small kernels below take a row (a head of a token) with 8 or 16 lanes, 8
// elements each: as few as cover head_dim. Bound by the memory that they read
// once, mostly from L2; measured cold: the join of 2 shares of 51200 rows of 64
// 12 us (19 with 16 lanes to a row and its sequence looked for), of 4 shares of
// 512 rows of 128 5 us; delta of 521000 rows of 128, bfloat16, 45 us, 5.9 TB/s; of
// 131000 rows of 64 8.5 us, in float16 with the sizes and as many values 15, and 4
// each sequence's largest (looked for by the kernels that use it instead, item by
// item: 2 us less here, 30 more on prompts of 6400).
__device__ __forceinline__ void token_head(int64_t row, int heads, int64_t& token, int& head) {
    if (row >> 31 == 0)
        token = static_cast<uint32_t>(row) / static_cast<uint32_t>(heads);
    else
        token = row / heads;
    head = static_cast<int>(row - token * heads);
}

// Whether a sequence has the row: they lie side by side from the first's start to the last's end.
__device__ __forceinline__ bool of_a_sequence(const int32_t* starts, int32_t batch, int64_t token) {
    return token >= starts[0] && token < starts[batch];
}

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
    return kLanes == 8 ? sum8(v) : sum16(v);
}

// The shares' sums added in order: of kv_rows (key, head) grad_k, as many
// grad_v, then of q_rows (token, head) grad_q. Rows of no sequence are not
// written.
template <int kLanes>
__global__ void __launch_bounds__(kT)
    attn_grad_sum_kernel(const __grid_constant__ AttnArgs a, int64_t kv_rows, int64_t q_rows) {
    dependency_wait();
    const int d = threadIdx.x % kLanes * 8;
    const int64_t index = static_cast<int64_t>(blockIdx.x) * (kT / kLanes) + threadIdx.x / kLanes;
    if (index >= 2 * kv_rows + q_rows || d >= a.D) return;
    const int which = index < kv_rows ? 0 : index < 2 * kv_rows ? 1 : 2;  // grad_k, grad_v, grad_q
    const bool of_q = which == 2;
    const int64_t row = index - which * kv_rows;
    const int heads = of_q ? a.hq : a.hk, shares = of_q ? a.q_splits : a.kv_splits;
    int64_t token;
    int head;
    token_head(row, heads, token, head);
    if (!of_a_sequence(of_q ? a.q_starts : a.k_starts, a.batch, token)) return;
    const int64_t one = static_cast<int64_t>(of_q ? a.tq : a.tk) * heads * a.D, step = of_q ? one : 2 * one;
    const float* p = (of_q ? a.part_q : a.part_kv + which * one) + row * a.D + d;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll 4
    for (int i = 0; i < shares; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(p + i * step);
        const float4 y = *reinterpret_cast<const float4*>(p + i * step + 4);
        u.x += x.x;
        u.y += x.y;
        u.z += x.z;
        u.w += x.w;
        v.x += y.x;
        v.y += y.y;
        v.z += y.z;
        v.w += y.w;
    }
    const AttnTensor& t = of_q ? a.gq : which ? a.gv : a.gk;
    float* to = static_cast<float*>(t.p) + token * t.st + head * t.sh + d;
    *reinterpret_cast<float4*>(to) = u;
    *reinterpret_cast<float4*>(to + 4) = v;
}

// out = sum over the shares of exp(lse_i - lse) out_i.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kT) attn_join_kernel(const __grid_constant__ AttnArgs a) {
    dependency_wait();
    const int sub = threadIdx.x % kLanes, d = sub * 8;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kT / kLanes) + threadIdx.x / kLanes;
    int64_t tok = 0;
    int h = 0;
    bool live = row < static_cast<int64_t>(a.tq) * a.hq;
    if (live) token_head(row, a.hq, tok, h);
    // rows of no sequence have no partial results and are not written
    live = live && of_a_sequence(a.q_starts, a.batch, tok);
    const float* lse = a.part_lse + static_cast<int64_t>(h) * a.tq + tok;
    const int64_t step = static_cast<int64_t>(a.hq) * a.tq;
    float best = -INFINITY;
    for (int i = sub; live && i < a.splits; i += kLanes) best = fmaxf(best, lse[i * step]);
    best = kLanes == 8 ? max8(best) : max16(best);
    if (!live) return;
    const float base = best == -INFINITY ? 0.0f : best;
    const bool on = d < a.D;
    const float* p = a.part_out + (tok * a.hq + h) * a.D + (on ? d : 0);
    float total = 0.0f;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll 4
    for (int i = 0; i < a.splits; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(p + i * step * a.D);
        const float4 y = *reinterpret_cast<const float4*>(p + i * step * a.D + 4);
        const float w = expf(lse[i * step] - base);
        total += w;
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
    const float inv = total > 0.0f ? 1.0f / total : total;
    if (on) {
        T* o = static_cast<T*>(a.out.p) + tok * a.out.st + h * a.out.sh + d;
        attn_store4(o, make_float4(u.x * inv, u.y * inv, u.z * inv, u.w * inv));
        attn_store4(o + 4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    }
    if (sub == 0) a.lse[static_cast<int64_t>(h) * a.tq + tok] = total == 0.0f ? -INFINITY : base + logf(total);
}

__device__ __forceinline__ float dot8(const float4 (&x)[2], const float4 (&y)[2]) {
    return dot4(x[0], y[0], dot4(x[1], y[1], 0.0f));
}

// Sum of the squares of 8 float16 elements, in fp32.
__device__ __forceinline__ float squares8(uint4 u) {
    const __half2* e = reinterpret_cast<const __half2*>(&u);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(e[i]);
        sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
    }
    return sum;
}

// delta = sum(grad_out * out) of each row. In float16 the sizes of the rows of
// grad_out too, and in blocks from `row_blocks` on those of the values, of which a
// thread has several under way.
constexpr int kValueRows = 2;
template <typename T, int kLanes>
__global__ void __launch_bounds__(kT, 8) attn_delta_kernel(const __grid_constant__ AttnArgs a, uint32_t row_blocks) {
    constexpr bool kSizes = std::is_same_v<T, __half>;
    constexpr int kPer = kT / kLanes;
    dependency_wait();
    if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    const int sub = threadIdx.x % kLanes, d = sub * 8;
    if constexpr (kSizes) {
        if (blockIdx.x >= row_blocks) {
            const uint32_t block = blockIdx.x - row_blocks;
            const int64_t all = static_cast<int64_t>(a.batch) * a.hk * 2;
            for (int64_t i = static_cast<int64_t>(block) * kT + threadIdx.x; i < all;
                 i += static_cast<int64_t>(gridDim.x - row_blocks) * kT)
                a.sizes[i] = 0;
            const int64_t row0 = static_cast<int64_t>(block) * (kPer * kValueRows) + threadIdx.x / kLanes;
            const int64_t rows = static_cast<int64_t>(a.tk) * a.hk;
            int64_t key;
            int kh;
            uint4 v[kValueRows];
#pragma unroll
            for (int i = 0; i < kValueRows; ++i) {
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (row0 + i * kPer < rows && d < a.D) {
                    token_head(row0 + i * kPer, a.hk, key, kh);
                    v[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v.p) + key * a.v.st + kh * a.v.sh + d);
                }
            }
#pragma unroll
            for (int i = 0; i < kValueRows; ++i) {
                const float sum = lanes_sum<kLanes>(squares8(v[i]));
                if (sub == 0 && row0 + i * kPer < rows) {
                    token_head(row0 + i * kPer, a.hk, key, kh);
                    a.v_size[static_cast<int64_t>(kh) * a.tk + key] = norm_size(sum);
                }
            }
            return;
        }
    }
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / kLanes;
    const bool live = row < static_cast<int64_t>(a.tq) * a.hq;
    int64_t tok = 0;
    int h = 0;
    if (live) token_head(row, a.hq, tok, h);
    float sum = 0.0f, squares = 0.0f;
    if (live && d < a.D) {
        float4 g[2], o[2];
        attn_load8(static_cast<const T*>(a.g.p) + tok * a.g.st + h * a.g.sh + d, g);
        attn_load8(static_cast<const T*>(a.out.p) + tok * a.out.st + h * a.out.sh + d, o);
        sum = dot8(g, o);
        if constexpr (kSizes) squares = dot8(g, g);
    }
    sum = lanes_sum<kLanes>(sum);
    if constexpr (kSizes) squares = lanes_sum<kLanes>(squares);
    if (live && sub == 0) {
        const int64_t at = static_cast<int64_t>(h) * a.tq + tok;
        a.delta[at] = sum;
        if constexpr (kSizes) a.g_size[at] = norm_size(squares);
    }
}

// The largest of the n sizes from `at` on in each of `heads` rows `pitch` apart:
// a thread's part, of the `step` threads that share them, in bytes. 16 bytes at
// a time: the array starts on 16 bytes and has room up to a multiple of 16.
__device__ __forceinline__ uint32_t top_sizes(const uint8_t* at, uint32_t heads, int64_t pitch, uint32_t n,
                                              uint32_t thread, uint32_t step) {
    const uint32_t words = (n + 30u) / 16u;  // that a head's sizes can touch; heads * words < 2^31
    uint32_t top = 0;
#pragma unroll 4
    for (uint32_t i = thread; i < heads * words; i += step) {
        const uint32_t head = i / words;
        const uintptr_t first = reinterpret_cast<uintptr_t>(at + head * pitch), end = first + n;
        const uintptr_t w = (first & ~static_cast<uintptr_t>(15)) + 16u * (i - head * words);
        if (w >= end) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(w);
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
        if (w < first || w + 16 > end) {  // bytes before the first and past the last count as 0
            const int lo = w < first ? static_cast<int>(first - w) : 0, hi = w + 16 > end ? static_cast<int>(end - w) : 16;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int from = min(max(lo - 4 * k, 0), 4), to = min(max(hi - 4 * k, 0), 4);
                x[k] &= static_cast<uint32_t>((uint64_t(1) << (8 * to)) - (uint64_t(1) << (8 * min(from, to))));
            }
        }
        top = __vmaxu4(__vmaxu4(top, x[0]), __vmaxu4(x[1], __vmaxu4(x[2], x[3])));
    }
    return top;
}

// Each sequence's largest size of a grad_out row, and of a value in use, for
// each key head. Grid: (sequences * key heads or fewer, blocks that share one's
// rows). The largest is the same in any order.
__global__ void __launch_bounds__(kT) attn_sizes_kernel(const __grid_constant__ AttnArgs a) {
    dependency_wait();
    const int64_t all = static_cast<int64_t>(a.batch) * a.hk;
    const uint32_t thread = blockIdx.y * kT + threadIdx.x, step = gridDim.y * kT;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const int b = static_cast<int>(i / a.hk), kh = static_cast<int>(i - static_cast<int64_t>(b) * a.hk);
        int32_t q0, lq, k0, lk;
        attn_range(a.q_starts, b, a.tq, q0, lq);
        attn_range(a.k_starts, b, a.tk, k0, lk);
        if (a.k_lengths) lk = min(max(a.k_lengths[b], 0), lk);
        const uint32_t top[2] = {top_sizes(a.g_size + static_cast<int64_t>(kh) * a.group * a.tq + q0,
                                           static_cast<uint32_t>(a.group), a.tq, static_cast<uint32_t>(lq), thread, step),
                                 top_sizes(a.v_size + static_cast<int64_t>(kh) * a.tk + k0, 1, 0,
                                           static_cast<uint32_t>(lk), thread, step)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t t = top[k];
            const uint32_t most = max(max(t & 255u, t >> 8 & 255u), max(t >> 16 & 255u, t >> 24));
            const int32_t one = static_cast<int32_t>(__reduce_max_sync(0xffffffffu, most));
            if ((threadIdx.x & 31) == 0 && one > 0) atomicMax(a.sizes + 2 * i + k, one);
        }
    }
}

}  // namespace

namespace {

// Blocks for `rows` rows of so many lanes.
unsigned groups(int64_t rows, int lanes) { return static_cast<unsigned>((rows + kT / lanes - 1) / (kT / lanes)); }

template <int kN>
cudaError_t launch_forward(const AttnArgs& a, cudaStream_t st) {
    constexpr int smem = (3 * kR * pitch_of(kN) + kR * kPP) * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = attn_allow_smem(attn_forward_simt_kernel<kN>, smem, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_forward_simt_kernel<kN>,
                            static_cast<unsigned>(a.tiles) * static_cast<unsigned>(a.splits) * static_cast<unsigned>(a.hk),
                            kTT, smem, st, a);
}

template <int kN>
cudaError_t launch_backward(const AttnArgs& a, int32_t kv, int32_t blocks, cudaStream_t st) {
    constexpr int smem = (4 * kR * pitch_of(kN) + kR * kPP) * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = attn_allow_smem(attn_backward_simt_kernel<kN>, smem, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_backward_simt_kernel<kN>, static_cast<unsigned>(blocks) * static_cast<unsigned>(a.hk), kTT, smem,
                            st, a, kv);
}

}  // namespace

// By sixteens of head_dim: the loops over a head's elements then have constant
// bounds and shared memory holds no more than the head (at 40 and 72 elements
// a power of two would compute on 1.6 and 1.8 times as many).
cudaError_t launch_attention_simt_forward(const AttnArgs& a, cudaStream_t st) {
    switch ((a.D + 15) / 16) {
        case 1: return launch_forward<1>(a, st);
        case 2: return launch_forward<2>(a, st);
        case 3: return launch_forward<3>(a, st);
        case 4: return launch_forward<4>(a, st);
        case 5: return launch_forward<5>(a, st);
        case 6: return launch_forward<6>(a, st);
        case 7: return launch_forward<7>(a, st);
        default: return launch_forward<8>(a, st);
    }
}

cudaError_t launch_attention_simt_backward(const AttnArgs& a, cudaStream_t st) {
    const int32_t kv = static_cast<int32_t>(attn_tiles(a.tk, a.batch, kC)) * a.kv_splits;
    const int32_t blocks = kv + (a.tq > 0 ? a.tiles * a.q_splits : 0);
    if (blocks == 0) return cudaSuccess;
    cudaError_t e;
    switch ((a.D + 15) / 16) {
        case 1: e = launch_backward<1>(a, kv, blocks, st); break;
        case 2: e = launch_backward<2>(a, kv, blocks, st); break;
        case 3: e = launch_backward<3>(a, kv, blocks, st); break;
        case 4: e = launch_backward<4>(a, kv, blocks, st); break;
        case 5: e = launch_backward<5>(a, kv, blocks, st); break;
        case 6: e = launch_backward<6>(a, kv, blocks, st); break;
        case 7: e = launch_backward<7>(a, kv, blocks, st); break;
        default: e = launch_backward<8>(a, kv, blocks, st); break;
    }
    const int64_t kv_rows = a.kv_splits > 1 ? static_cast<int64_t>(a.tk) * a.hk : 0;
    const int64_t q_rows = a.q_splits > 1 ? static_cast<int64_t>(a.tq) * a.hq : 0;
    if (e != cudaSuccess || 2 * kv_rows + q_rows == 0) return e;
    if (a.D <= 64)
        return launch_dependent(attn_grad_sum_kernel<8>, groups(2 * kv_rows + q_rows, 8), kT, 0, st, a, kv_rows, q_rows);
    return launch_dependent(attn_grad_sum_kernel<16>, groups(2 * kv_rows + q_rows, 16), kT, 0, st, a, kv_rows, q_rows);
}

namespace {

template <typename T>
cudaError_t join(const AttnArgs& a, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.tq) * a.hq;
    if (a.D <= 64) return launch_dependent(attn_join_kernel<T, 8>, groups(rows, 8), kT, 0, st, a);
    return launch_dependent(attn_join_kernel<T, 16>, groups(rows, 16), kT, 0, st, a);
}

template <typename T>
cudaError_t delta(const AttnArgs& a, cudaStream_t st) {
    const int lanes = a.D <= 64 ? 8 : 16;
    const uint32_t rows = groups(static_cast<int64_t>(a.tq) * a.hq, lanes);
    const uint32_t values =
        a.sizes ? groups((static_cast<int64_t>(a.tk) * a.hk + kValueRows - 1) / kValueRows, lanes) + 1 : 0;
    const cudaError_t e = lanes == 8 ? launch_dependent(attn_delta_kernel<T, 8>, rows + values, kT, 0, st, a, rows)
                                     : launch_dependent(attn_delta_kernel<T, 16>, rows + values, kT, 0, st, a, rows);
    if (e != cudaSuccess || !a.sizes) return e;
    // blocks that share a sequence's rows of a key head: two to each of 152 SMs in all, 16 sizes to a thread
    const int64_t pairs = static_cast<int64_t>(a.batch) * a.hk;
    const int64_t words = (static_cast<int64_t>(a.tq) * a.group + a.tk) / a.batch / (16 * kT) + 1;
    const int64_t shares = std::min(std::max<int64_t>(2 * 152 / pairs, 1), words);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(pairs, 1 << 16)), static_cast<unsigned>(shares));
    return launch_dependent(attn_sizes_kernel, grid, kT, 0, st, a);
}

}  // namespace

cudaError_t launch_attention_join(int dtype, const AttnArgs& a, cudaStream_t st) {
    if (dtype == kF32) return join<float>(a, st);
    if (dtype == kF16) return join<__half>(a, st);
    return join<__nv_bfloat16>(a, st);
}

cudaError_t launch_attention_delta(int dtype, const AttnArgs& a, cudaStream_t st) {
    if (a.tq == 0) return a.status ? cudaMemsetAsync(a.status, 0, sizeof(uint32_t), st) : cudaSuccess;
    if (dtype == kF32) return delta<float>(a, st);
    if (dtype == kF16) return delta<__half>(a, st);
    return delta<__nv_bfloat16>(a, st);
}

}  // namespace mdcn
