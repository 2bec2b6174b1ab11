// Device code shared by the tensor-core attention kernels: tensor maps of
// packed row tiles and of key tiles, packed fp32 arithmetic, conversions.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "mdcn_attention.cuh"
#include "mdcn_ptx.cuh"

namespace mdcn {

constexpr int kAttnTcRows = kAttnTcBlockRows;       // rows of a tile: the MMA's M
constexpr uint32_t kAtomBytes = 128 * 128;          // 64 elements of 128 rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Host: tensor maps with 64-element, 128-byte swizzled boxes; elements past
// head_dim and rows past the tensor read as zero.
// Row tiles [head_dim][group][k_heads][tokens], box of `tokens` x group rows.
bool attn_encode_rows(CUtensorMap* m, const AttnArgs& a, const AttnTensor& t, int dtype, int tokens);
// Key tiles [head_dim][k_heads][tokens], box of `rows` rows.
bool attn_encode_keys(CUtensorMap* m, const AttnArgs& a, const AttnTensor& t, int dtype, int rows);

__device__ __forceinline__ float attn_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

// (lo, hi) rounded to two 16-bit elements, lo in the low half.
template <bool kBf>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
    uint32_t r;
    if constexpr (kBf)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Zeroes rows [first, 128) of a tile of `atoms` 64-element atoms; one warp.
// The tensor cores multiply these rows by probabilities of 0, and 0 times
// another sequence's NaN or infinity would not be 0.
__device__ __forceinline__ void zero_rows(uint32_t tile, int atoms, uint32_t atom_bytes, int first, int rows) {
    const int lane = threadIdx.x & 31;
    for (int at = 0; at < atoms; ++at)
        for (int i = first * 8 + lane; i < rows * 8; i += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + at * atom_bytes + i * 16u), "r"(0u)
                         : "memory");
    fence_proxy_async_smem();
    __syncwarp();
}

// 16 fp32 values, rounded, to 16 consecutive elements; `wide`: 32-byte aligned
// (one 32-byte store, a whole sector), else 16-byte aligned. n: elements that
// exist (a multiple of 8).
template <bool kBf>
__device__ __forceinline__ void store16(void* p, const float (&v)[16], int n, bool wide) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = round2<kBf>(v[2 * i], v[2 * i + 1]);
    if (wide && n >= 16) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
        return;
    }
    if (n >= 8) st_global_v4(p, make_uint4(r[0], r[1], r[2], r[3]));
    if (n >= 16) st_global_v4(static_cast<uint8_t*>(p) + 16, make_uint4(r[4], r[5], r[6], r[7]));
}

}  // namespace mdcn
