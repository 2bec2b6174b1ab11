// Device code shared by the attention kernels: which sequence a tile belongs
// to, packed fp32 arithmetic, element conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "mdcn_attention.h"

namespace mdcn {

constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 values in one register pair: (lo, hi).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float attn_to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float attn_to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T attn_from_f(float v);
template <>
__device__ __forceinline__ __half attn_from_f<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 attn_from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// 8 consecutive elements as fp32, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void attn_load8(const T* p, float4 (&v)[2]) {
    if constexpr (sizeof(T) == 4) {
        v[0] = reinterpret_cast<const float4*>(p)[0];
        v[1] = reinterpret_cast<const float4*>(p)[1];
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const T* e = reinterpret_cast<const T*>(&u);
        v[0] = make_float4(attn_to_f(e[0]), attn_to_f(e[1]), attn_to_f(e[2]), attn_to_f(e[3]));
        v[1] = make_float4(attn_to_f(e[4]), attn_to_f(e[5]), attn_to_f(e[6]), attn_to_f(e[7]));
    }
}
// 4 elements (16-byte aligned fp32, 8-byte aligned 16-bit).
template <typename T>
__device__ __forceinline__ void attn_store4(T* p, float4 v) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        uint2 u;
        T* e = reinterpret_cast<T*>(&u);
        e[0] = attn_from_f<T>(v.x);
        e[1] = attn_from_f<T>(v.y);
        e[2] = attn_from_f<T>(v.z);
        e[3] = attn_from_f<T>(v.w);
        *reinterpret_cast<uint2*>(p) = u;
    }
}

// Size of a row with the sum of squares s, in one byte: 64 + E with norm <= 2^E
// <= 2 norm; 0 for a row of zeros. (float16: E from -23 to 20.)
__device__ __forceinline__ uint8_t norm_size(float s) {
    if (s == 0.0f) return 0;
    const int e = static_cast<int>(__float_as_uint(s) >> 23 & 255u) - 127;  // s < 2^(e + 1)
    return static_cast<uint8_t>(64 + ((e + 2) >> 1));
}

struct AttnSeq {
    int32_t tile;    // tile of the sequence; -1: there is none
    int32_t q0, lq;  // first query row, queries
    int32_t k0, lk;  // first key row, keys in use
    int32_t room;    // keys the sequence has rows for
    int32_t b;       // the sequence
};

// Rows [start, end) of sequence b, clamped to the tensor. Plain loads, here and
// wherever a kernel reads after dependency_wait(): the compiler keeps them
// behind it, which it need not do with read-only ones (__ldg).
__device__ __forceinline__ void attn_range(const int32_t* starts, int b, int32_t total, int32_t& first, int32_t& len) {
    const int32_t s = min(max(starts[b], 0), total);
    const int32_t e = min(max(starts[b + 1], s), total);
    first = s;
    len = e - s;
}

// The sequence and tile of tile `index`, sequences in order and each cut into
// tiles of `tokens` rows. Under a causal mask the last queries see the most
// keys and the first keys are seen by the most queries, so that tiles of
// queries come from a sequence's last to its first, tiles of keys from its
// first. All 32 lanes of a warp call it; every lane gets the answer.
__device__ __forceinline__ AttnSeq attn_find(const AttnArgs& a, bool by_keys, int32_t tokens, int32_t index) {
    const int lane = threadIdx.x & 31;
    const int32_t* starts = by_keys ? a.k_starts : a.q_starts;
    const int32_t total = by_keys ? a.tk : a.tq;
    AttnSeq s{-1, 0, 0, 0, 0, 0, 0};
    int32_t left = index;
    for (int32_t b0 = 0; b0 < a.batch; b0 += 32) {
        int32_t first = 0, len = 0, n = 0;
        if (b0 + lane < a.batch) {
            attn_range(starts, b0 + lane, total, first, len);
            n = (len + tokens - 1) / tokens;
        }
        int32_t sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, sum > left);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int32_t before = __shfl_sync(0xffffffffu, sum - n, src);
            const int32_t tiles = __shfl_sync(0xffffffffu, n, src);
            const int b = b0 + src;
            s.b = b;
            s.tile = by_keys ? left - before : tiles - 1 - (left - before);
            attn_range(a.q_starts, b, a.tq, s.q0, s.lq);
            attn_range(a.k_starts, b, a.tk, s.k0, s.room);
            s.lk = a.k_lengths ? min(max(a.k_lengths[b], 0), s.room) : s.room;
            return s;
        }
        left -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return s;
}

// Keys that query i of the sequence sees: the first so many.
__device__ __forceinline__ int32_t attn_seen(const AttnArgs& a, const AttnSeq& s, int32_t i) {
    return a.causal ? min(max(i + 1 + s.lk - s.lq, 0), s.lk) : s.lk;
}

}  // namespace mdcn
