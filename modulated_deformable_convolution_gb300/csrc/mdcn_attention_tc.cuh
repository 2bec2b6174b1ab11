// Device code shared by the tensor-core attention kernels: tensor maps of
// packed row tiles and of key tiles, conversions.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "mdcn_attention.cuh"
#include "mdcn_ptx.cuh"

namespace mdcn {

constexpr int kAttnTcRows = kAttnTcBlockRows;       // rows of a tile: the MMA's M
constexpr uint32_t kAtomBytes = 128 * 128;          // 64 elements of 128 rows
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

// 8 fp32 values; `wide`: to a 32-byte aligned address (one store, a whole
// sector), else to a 16-byte aligned one.
__device__ __forceinline__ void store8(float* p, const float* v, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
                     "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
        return;
    }
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// ---------------------------------------------------------------- work items
// A block works through items (a row or key tile of one key head) one after
// the other: its own index first, then indices of blocks that have not started
// yet, which it asks for ahead of time. So the set-up of a block (barriers,
// tensor memory) is paid once per SM, the next item's loads run during this
// one's last steps, and long and short items even out. One warp asks, finds the
// item's sequence and publishes the item in shared memory; two slots.
struct alignas(16) AttnItem {
    int32_t go;          // 0: no more items
    int32_t kh, split;   // key head; share of the keys (float16 gradients: see score_shift)
    int32_t q0, k0;      // the sequence's first query and key row
    int32_t lq, lk, room;
    int32_t first;       // first token (row tiles) or key (key tiles)
    int32_t n0, n1;      // steps of the item (two row tiles: of each)
    int32_t j0;          // first step's key tile or row block
    int32_t pad[4];
};
static_assert(sizeof(AttnItem) == 64, "four vectors");

// Shared memory of the item queue, at 16-byte aligned `base`. `limit`: a role
// that has nothing to do in an item waits for the others to finish it.
struct ItemQueue {
    static constexpr uint32_t kBytes = 2 * 64 + 16 + 5 * 8 + 8;
    uint32_t base;
    uint64_t limit;
    __device__ __forceinline__ uint32_t slot(uint32_t i) const { return base + 64u * i; }
    __device__ __forceinline__ uint32_t answer() const { return base + 128u; }
    __device__ __forceinline__ uint32_t full(uint32_t i) const { return base + 144u + 8u * i; }
    __device__ __forceinline__ uint32_t empty(uint32_t i) const { return base + 160u + 8u * i; }
    __device__ __forceinline__ uint32_t asked() const { return base + 176u; }
    __device__ __forceinline__ void init(uint32_t readers) const {
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), readers);
        }
        mbar_init(asked(), 1);
    }
};

__device__ __forceinline__ void st_shared_v4(uint32_t addr, int32_t a, int32_t b, int32_t c, int32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ AttnItem read_item(uint32_t slot) {
    const uint4 a = ld_shared_v4(slot), b = ld_shared_v4(slot + 16u), c = ld_shared_v4(slot + 32u);
    AttnItem it;
    it.go = static_cast<int32_t>(a.x);
    it.kh = static_cast<int32_t>(a.y);
    it.split = static_cast<int32_t>(a.z);
    it.q0 = static_cast<int32_t>(a.w);
    it.k0 = static_cast<int32_t>(b.x);
    it.lq = static_cast<int32_t>(b.y);
    it.lk = static_cast<int32_t>(b.z);
    it.room = static_cast<int32_t>(b.w);
    it.first = static_cast<int32_t>(c.x);
    it.n0 = static_cast<int32_t>(c.y);
    it.n1 = static_cast<int32_t>(c.z);
    it.j0 = static_cast<int32_t>(c.w);
    return it;
}

// A warp's turn through the items: each item to `body` (which returns false to
// stop). The reader frees the slot as soon as it has copied the item.
template <typename F>
__device__ __forceinline__ void for_items(const ItemQueue& q, volatile int* abort_flag, uint32_t* status, F body) {
    for (uint32_t i = 0;; ++i) {
        const uint32_t s = i & 1u;
        if (!warp_wait2(q.full(s), 0u, (i >> 1) & 1u, abort_flag, status, kSiteEpilogue, q.limit)) return;
        const AttnItem it = read_item(q.slot(s));
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(q.empty(s));
        if (!it.go || !body(it)) return;
    }
}

// The same for a role that one thread plays.
template <typename F>
__device__ __forceinline__ void for_items_one(const ItemQueue& q, volatile int* abort_flag, uint32_t* status, F body) {
    for (uint32_t i = 0;; ++i) {
        const uint32_t s = i & 1u;
        if (!mbar_wait_bounded(q.full(s), (i >> 1) & 1u, abort_flag, status, kSiteEpilogue, q.limit)) return;
        const AttnItem it = read_item(q.slot(s));
        mbar_arrive(q.empty(s));
        if (!it.go || !body(it)) return;
    }
}

// The asking warp: `find` turns an index into an item (false: there is none
// under this index).
template <typename F>
__device__ __forceinline__ void serve_items(const ItemQueue& q, volatile int* abort_flag, uint32_t* status, F find) {
    const int lane = threadIdx.x & 31;
    int32_t index = static_cast<int32_t>(blockIdx.x);
    uint32_t out = 0;
    for (uint32_t i = 0;; ++i) {
        if (lane == 0 && index >= 0) {
            mbar_arrive_expect_tx(q.asked(), 16u);
            steal_block(q.answer(), q.asked());
        }
        __syncwarp();
        AttnItem it{};
        const bool there = index >= 0 && find(index, it);
        it.go = there ? 1 : 0;
        if (there || index < 0) {
            const uint32_t s = out & 1u;
            if (!warp_wait2(q.empty(s), 0u, ((out >> 1) & 1u) ^ 1u, abort_flag, status, kSiteTmaEmpty, q.limit)) {
                if (index >= 0) {  // the answer asked for lands before the block exits
                    volatile int never = 0;
                    warp_wait_bounded(q.asked(), i & 1u, &never, status, kSiteDrain, 200000000ull);
                }
                return;
            }
            if (lane == 0) {
                st_shared_v4(q.slot(s), it.go, it.kh, it.split, it.q0);
                st_shared_v4(q.slot(s) + 16u, it.k0, it.lq, it.lk, it.room);
                st_shared_v4(q.slot(s) + 32u, it.first, it.n0, it.n1, it.j0);
                mbar_arrive(q.full(s));
            }
            __syncwarp();
            ++out;
        }
        if (index < 0) return;
        if (!warp_wait2(q.asked(), 0u, i & 1u, abort_flag, status, kSiteTmaEmpty)) {
            volatile int never = 0;
            warp_wait_bounded(q.asked(), i & 1u, &never, status, kSiteDrain, 200000000ull);
            return;
        }
        index = stolen_block(q.answer());
        __syncwarp();
        fence_proxy_async_smem();  // the answer has been read before the next one is written
    }
}

}  // namespace mdcn
