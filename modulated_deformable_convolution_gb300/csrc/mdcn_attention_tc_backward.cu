// Attention over packed sequences on the tensor cores (float16, bfloat16):
// the gradients.
//
// From the forward's lse and delta = sum(grad_out * out), for each (query row,
// key): p = exp2(scale' S - lse'), ds = p (dP - delta), with S = Q K^T and dP =
// G V^T. Two kernels, so that every output is summed by one block in a fixed
// order (no atomic additions, no second pass over fp32 sums), at the price of
// S and dP computed twice (seven products instead of five):
//   grad_q:  128 query rows to a block, over the key tiles that they see:
//            dQ += dS K;
//   grad_kv: 128 keys to a block, over the blocks of 128 query rows (all heads
//            of the key head) that see them: S^T = K Q^T, dP^T = V G^T,
//            dV += P^T G, dK += dS^T Q.
// In both the fp32 products stay in tensor memory and P and dS, rounded to the
// tensors' type, go back there as the next product's left operand. Two
// warpgroups take 64 of a product's 128 columns each, a thread one row. P is
// kept times 2^8 (exact): probabilities down to 2^-22 then stay normal float16
// numbers. dS, whose size is the gradients', is kept in float16 times a power of
// two, undone when the sums are read: |ds| <= 2 |grad_out row| |value|, so that the
// norms bound it that two small launches leave behind: a grad_q row's own with
// the sequence's largest value's, in grad_kv the sequence's largest of both. The
// bound goes to 2^15: nothing passes float16's largest number, and what is 2^-29 of
// it is still a normal one (unscaled, gradients of 1e-4 over 6400 keys were off by
// 8%). bfloat16 has fp32's range and needs none.
//
// Bound by the tensor cores: 3 (grad_q) and 4 (grad_kv) products of 128 x 128 x
// D per tile, about 512 cycles each at D = 128. While the elementwise step of
// one tile runs, the next tile's S and dP, or this tile's sums, are computed.
//
// Measured with delta (bfloat16, 32 heads of 128 over 8): 9 packed causal prompts
// of up to 6400 tokens 1525 us, 912 TFLOP/s of five products, 1277 of the seven;
// 2 x 8192 without a mask 4.7 to 4.9 ms, 1120 to 1170 and 1570 to 1640. 16 maps of
// 32 x 32, 8 heads of 64, float16: 152 us, 566 TFLOP/s of five products, 10 us of
// them for the sizes: at D = 64 the products of a tile take half as long and its
// elementwise step as long as before (a grad_kv block about 2130 cycles,
// exponentials 710, dS 510, loads and stores of tensor memory and waits the rest;
// 16 elementwise warps instead of 8 changed nothing).
#include <cuda.h>

#include <cstdint>

#include "mdcn_attention_tc.cuh"
#include "mdcn_pdl.h"
#include "mdcn_plan.h"

namespace mdcn {

namespace {

constexpr int kTcThreads = 384;
constexpr int kWarpLoad = 8, kWarpIssue = 9, kWarpServe = 10, kWarpAid = 11;
constexpr int kRegsRow = 216, kRegsCtl = 72;  // of 168 a thread at launch
static_assert(2 * kRegsRow + kRegsCtl <= 3 * 168, "register split must fit the launch's");
constexpr int kKeys = 128;
constexpr float kShift = 8.0f, kUnshift = 0.00390625f;  // P is kept times 2^8

__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of the factor that dS is kept times, from the sizes of a row of
// grad_out and of a value (norm_size): 2 |g| |v| 2^shift <= 2^15.
__device__ __forceinline__ int score_shift(int sizes) { return min(max(14 - (sizes - 128), -60), 60); }

// ds = p 2^8 * (dp - delta) 2^-8 for 64 columns of a row; p in, packed ds out.
// un: 2^-8 (float16: times dS's factor) twice; minus_delta: -delta * un for column pairs.
template <bool kBf, typename F>
__device__ __forceinline__ void score_grads(const uint32_t (&p)[2][32], const uint32_t (&dp)[2][32], uint64_t un,
                                            F minus_delta, uint32_t (&out)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int c = i >> 4, o = 2 * (i & 15);
        const uint64_t d =
            fma2(pack2(__uint_as_float(dp[c][o]), __uint_as_float(dp[c][o + 1])), un, minus_delta(2 * i));
        float u, w;
        unpack2(mul2(pack2(__uint_as_float(p[c][o]), __uint_as_float(p[c][o + 1])), d), u, w);
        out[i] = round2<kBf>(u, w);
    }
}

__device__ __forceinline__ void load_half(uint32_t col, uint32_t (&x)[2][32]) {
    tmem_ld32_async(col, x[0]);
    tmem_ld32_async(col + 32u, x[1]);
    tmem_wait_ld();
    tmem_landed(x[0]);
    tmem_landed(x[1]);
}

// Columns [c0, c1) of an fp32 accumulator row times f, rounded, to global
// memory; `any` false: zeros.
template <bool kBf>
__device__ __forceinline__ void store_row(uint32_t col, uint8_t* p, int c0, int c1, float f, bool any, bool live) {
    const bool wide = (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
#pragma unroll 1
    for (int c = c0; c < c1; c += 16) {
        float v[16];
        __syncwarp();  // the stores part the lanes; the load needs the whole warp
        if (any) tmem_ld16(col + static_cast<uint32_t>(c), v);
        if (live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = any ? v[i] * f : 0.0f;
            store16<kBf>(p + 2 * c, v, c1 - c, wide);
        }
    }
    __syncwarp();
}

// d (+)= rows of x times rows of y over the head, both K-major; one thread.
template <int kAtoms>
__device__ __forceinline__ void head_product(uint32_t d, uint64_t x, uint64_t y, uint32_t idesc, int ksteps) {
#pragma unroll
    for (int kk = 0; kk < 4 * kAtoms; ++kk) {
        const uint32_t off = (static_cast<uint32_t>(kk >> 2) * kAtomBytes + 32u * (kk & 3)) >> 4;
        if (kk < ksteps) mma_f16(d, x + off, y + off, idesc, kk > 0);
    }
}

__host__ __device__ constexpr int stages_of(int atoms) { return atoms == 2 ? 5 : 8; }
__host__ __device__ constexpr int smem_q(int atoms) {
    return 1024 + (2 + stages_of(atoms)) * atoms * static_cast<int>(kAtomBytes) + 512;
}

// ---------------------------------------------------------------- grad_q
// Tensor memory: S [0, 128), dP [128, 256), dS [256, 320), dQ [320, 320 + D).
template <int kAtoms, bool kBf>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_grad_q_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                          const __grid_constant__ AttnArgs a) {
    constexpr uint32_t S = stages_of(kAtoms);
    constexpr uint32_t kTile = kAtoms * kAtomBytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t q_s = base, g_s = base + kTile, ring = base + 2 * kTile;
    const ItemQueue queue{ring + S * kTile, a.item_limit};
    const uint32_t bars = queue.base + ItemQueue::kBytes;
    auto full = [&](uint32_t s) { return bars + 8u * s; };
    auto empty = [&](uint32_t s) { return bars + 8u * (S + s); };
    const uint32_t rest = bars + 16u * S;
    const uint32_t q_full = rest, q_empty = rest + 8, s_full = rest + 16, dp_full = rest + 24, s_read = rest + 32,
                   dp_read = rest + 40, ds_full = rest + 48, dq_done = rest + 56, dq_read = rest + 64,
                   drain = rest + 72, cleared = rest + 80, to_clear = rest + 88;
    const uint32_t slot_off = rest + 96 - raw;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + slot_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + slot_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kWarpLoad && lane == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        const uint32_t ones[] = {q_full, q_empty, s_full, dp_full, dq_done, drain, cleared, to_clear};
        for (uint32_t b : ones) mbar_init(b, 1);
        const uint32_t eights[] = {s_read, dp_read, ds_full, dq_read};
        for (uint32_t b : eights) mbar_init(b, 8);
        queue.init(11);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mg);
        tma_prefetch_desc(&mk);
        tma_prefetch_desc(&mv);
    }
    if (warp == kWarpIssue) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    dependency_wait();
    const uint32_t c_s = tmem, c_dp = tmem + 128u, c_ds = tmem + 256u, c_dq = tmem + 320u;
    const int tpt = kAttnTcRows / a.group;

    if (warp >= 8) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == kWarpServe) {
            // ------------------------------------------------------------ items
            serve_items(queue, abort_flag, a.status, [&](int32_t index, AttnItem& it) {
                it.kh = index % a.hk;
                const AttnSeq s = attn_find(a, false, tpt, index / a.hk);
                if (s.tile < 0) return false;
                it.q0 = s.q0;
                it.k0 = s.k0;
                it.lq = s.lq;
                it.lk = s.lk;
                it.first = s.tile * tpt;
                it.n0 = (attn_seen(a, s, it.first + min(tpt, s.lq - it.first) - 1) + kKeys - 1) / kKeys;
                if constexpr (!kBf) it.split = a.sizes[(static_cast<int64_t>(s.b) * a.hk + it.kh) * 2 + 1];
                return true;
            });
        } else if (warp == kWarpLoad) {
            // ------------------------------------------------------------ loads
            uint32_t issued = 0, rows = 0;
            for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
                if (it.n0 == 0) return true;
                if (!warp_wait_bounded(q_empty, (rows & 1u) ^ 1u, abort_flag, a.status, kSiteTmaEmpty)) return false;
                mbar_arrive_expect_tx_elect(q_full, 2u * kAtoms * static_cast<uint32_t>(tpt * a.group) * 128u);
                for (int at = 0; at < kAtoms; ++at) {
                    tma_load_4d_elect(q_s + at * kAtomBytes, &mq, 64 * at, 0, it.kh, it.q0 + it.first, q_full);
                    tma_load_4d_elect(g_s + at * kAtomBytes, &mg, 64 * at, 0, it.kh, it.q0 + it.first, q_full);
                }
                ++rows;
                for (int32_t j = 0; j < it.n0; ++j) {
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t st = issued % S;
                        if (!warp_wait_bounded(empty(st), ((issued / S) & 1u) ^ 1u, abort_flag, a.status, kSiteTmaEmpty))
                            return false;
                        mbar_arrive_expect_tx_elect(full(st), kTile);
                        for (int at = 0; at < kAtoms; ++at)
                            tma_load_3d_elect(ring + st * kTile + at * kAtomBytes, kv ? &mv : &mk, 64 * at, it.kh,
                                              it.k0 + j * kKeys, full(st));
                        ++issued;
                    }
                }
                return true;
            });
            if (*abort_flag) {  // the copies already issued land before the CTA exits
                volatile int never = 0;
                if (rows) warp_wait_bounded(q_full, (rows - 1) & 1u, &never, a.status, kSiteDrain, 200000000ull);
                for (uint32_t i = issued > S ? issued - S : 0; i < issued; ++i)
                    warp_wait_bounded(full(i % S), (i / S) & 1, &never, a.status, kSiteDrain, 200000000ull);
            }
        } else if (warp == kWarpAid) {
            // ------------------------------------------------------------ keys past the last one
            uint32_t e = 0, turn = 0;
            for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
                if (it.n0 == 0) return true;
                const int32_t valid = it.lk - (it.n0 - 1) * kKeys;
                const uint32_t st = (e + 2u * it.n0 - 2u) % S;
                e += 2u * it.n0;
                if (valid >= kKeys) return true;
                // the issuing thread has seen the tile arrive
                if (!warp_wait2(to_clear, 0u, turn, abort_flag, a.status, kSiteTmaEmpty, a.item_limit)) return false;
                turn ^= 1u;
                zero_rows(ring + st * kTile, kAtoms, kAtomBytes, valid, kKeys);
                if (lane == 0) mbar_arrive(cleared);
                return true;
            });
        } else {
            // ------------------------------------------------------------ MMAs, one thread
            if (elect_lane()) {
                const uint32_t fmt = kBf ? 1u : 0u;
                const uint32_t nd = static_cast<uint32_t>((a.D + 15) & ~15);
                const uint32_t id_s = make_idesc(fmt, 128u, kKeys), id_q = make_idesc(fmt, 128u, nd) | (1u << 16);
                const int ksteps = (a.D + 15) / 16;
                const uint64_t dq0 = desc_sw128(q_s, 16u, 1024u), dg0 = desc_sw128(g_s, 16u, 1024u);
                const uint64_t dk0 = desc_sw128(ring, 16u, 1024u), dm0 = desc_sw128(ring, kAtomBytes, 1024u);
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    return mbar_wait_bounded(bar, parity, abort_flag, a.status, kSiteMmaFull);
                };
                uint32_t st = 0, ph = 0;        // stage and phase of the next tile to arrive
                uint32_t ks = 0;                // stage of the next K to be summed
                uint32_t read_s = 1, read_dp = 1, ds = 0;  // parities: S and dP read, dS written
                uint32_t items = 0, clear = 0;  // parities
                auto next = [&](uint32_t& s) {
                    const bool wrap = ++s == S;
                    if (wrap) s = 0;
                    return wrap;
                };
                for_items_one(queue, abort_flag, a.status, [&](const AttnItem& it) {
                    const int32_t n = it.n0;
                    if (n == 0) return true;
                    const bool partial = it.lk - (n - 1) * kKeys < kKeys;
                    // S, then dP, of the next key tile, into the buffer whose previous values have been read
                    auto scores = [&](bool last) {
                        if (!wait(full(st), ph) || !wait(s_read, read_s)) return false;
                        if (last && partial) mbar_arrive(to_clear);
                        tc_fence_after();
                        head_product<kAtoms>(c_s, dq0, dk0 + st * (kTile >> 4), id_s, ksteps);
                        mma_commit(s_full);
                        if (next(st)) ph ^= 1u;
                        read_s ^= 1u;
                        return true;
                    };
                    auto grads = [&](bool last) {
                        if (!wait(full(st), ph) || !wait(dp_read, read_dp)) return false;
                        tc_fence_after();
                        head_product<kAtoms>(c_dp, dg0, dk0 + st * (kTile >> 4), id_s, ksteps);
                        mma_commit(dp_full);
                        mma_commit(empty(st));
                        if (last) mma_commit(q_empty);
                        if (next(st)) ph ^= 1u;
                        read_dp ^= 1u;
                        return true;
                    };
                    if (!wait(q_full, items) || !scores(n == 1) || !grads(n == 1)) return false;
                    for (int32_t j = 0; j < n; ++j) {
                        const bool more = j + 1 < n, last = j + 2 == n;
                        if (more && !scores(last)) return false;
                        // The ring of five 128-element tiles has no room for the next V before this K is
                        // summed and freed; that of eight 64-element tiles does
                        if (more && kAtoms == 1 && !grads(last)) return false;
                        if (j == 0 && !wait(dq_read, items ^ 1u)) return false;
                        // dQ += dS K multiplies the rows past the last key by 0
                        if (!more && partial) {
                            if (!wait(cleared, clear)) return false;
                            clear ^= 1u;
                        }
                        const uint64_t dm = dm0 + ks * (kTile >> 4);
                        if (!wait(ds_full, ds)) return false;
                        ds ^= 1u;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            mma_f16_ts(c_dq, c_ds + 8u * kk, dm + 128u * kk, id_q, j > 0 || kk > 0);
                        mma_commit(dq_done);
                        mma_commit(empty(ks));
                        next(ks);
                        next(ks);
                        if (more && kAtoms == 2 && !grads(last)) return false;
                    }
                    items ^= 1u;
                    return true;
                });
                mma_commit(drain);
                volatile int never = 0;
                mbar_wait_bounded(drain, 0, &never, a.status, kSiteDrain, 200000000ull);
            }
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<kRegsRow>();
        const int half = warp >> 2;  // columns [64 half, 64 half + 64) of each tile
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int tk = r / a.group, sub = r - tk * a.group;
        const float sc = a.scale * kLog2e;
        const uint64_t sc2 = pack2(sc, sc);
        uint32_t g = 0;  // steps so far
        for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
            const int32_t n = it.n0;
            const bool live = r < min(tpt, it.lq - it.first) * a.group;
            const int h = it.kh * a.group + sub;
            const int64_t tok = it.q0 + it.first + tk;
            int32_t seen = it.lk;
            if (a.causal) seen = min(max(it.first + tk + 1 + it.lk - it.lq, 0), it.lk);
            if (!live) seen = 0;
            const int32_t seen_all = __reduce_min_sync(0xffffffffu, live ? seen : 0x7fffffff);
            const float lse = live ? a.lse[static_cast<int64_t>(h) * a.tq + tok] * kLog2e : 0.0f;
            float un = kUnshift, factor = a.scale;
            if constexpr (!kBf) {
                const int shift =
                    score_shift(live ? a.g_size[static_cast<int64_t>(h) * a.tq + tok] + it.split : 128);
                un = power2(shift - 8);
                factor *= power2(-shift);
            }
            const float delta = live ? a.delta[static_cast<int64_t>(h) * a.tq + tok] * un : 0.0f;
            const uint64_t l2 = pack2(kShift - lse, kShift - lse), d2 = pack2(-delta, -delta), un2 = pack2(un, un);
            for (int32_t j = 0; j < n; ++j, ++g) {
                if (!warp_wait2(s_full, 0u, g & 1u, abort_flag, a.status, kSiteGatherEmpty)) return false;
                tc_fence_after();
                uint32_t x[2][32];
                load_half(c_s + lanes + 64u * half, x);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
                const int32_t first = j * kKeys + 64 * half;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float u, w;
                        unpack2(fma2(pack2(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1])), sc2, l2), u, w);
                        x[c][i] = __float_as_uint(attn_exp2(u));
                        x[c][i + 1] = __float_as_uint(attn_exp2(w));
                    }
                if (!warp_wait2(dp_full, 0u, g & 1u, abort_flag, a.status, kSiteGatherEmpty)) return false;
                tc_fence_after();
                uint32_t dp[2][32], ds[32];
                load_half(c_dp + lanes + 64u * half, dp);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dp_read);
                if (seen_all < first + 64) {
                    const int32_t left = seen - first;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i >= left) x[c][i] = dp[c][i] = 0u;
                    __syncwarp();  // lanes differ in what they mask; the store below needs the whole warp
                }
                score_grads<kBf>(x, dp, un2, [&](int) { return d2; }, ds);
                // the sum before this step has read dS
                if (j > 0 && !warp_wait2(dq_done, 0u, (g - 1u) & 1u, abort_flag, a.status, kSiteGatherEmpty))
                    return false;
                tc_fence_after();
                tmem_st32(c_ds + lanes + 32u * half, ds);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full);
            }
            const bool any = n > 0;
            if (any && !warp_wait2(dq_done, 0u, (g - 1u) & 1u, abort_flag, a.status, kSiteEpilogue)) return false;
            tc_fence_after();
            uint8_t* p = static_cast<uint8_t*>(a.gq.p) + 2 * (tok * a.gq.st + h * a.gq.sh);
            const int mid = min(32 * kAtoms, a.D);
            store_row<kBf>(c_dq + lanes, p, half ? mid : 0, half ? a.D : mid, factor, any, live);
            if (any) {  // the next item's first sum may overwrite dQ
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dq_read);
            }
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpIssue) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- grad_k, grad_v
// Tensor memory: S^T with P^T over it, dP^T with dS^T over it (128 columns
// each), dV, dK. Each half of the columns keeps its rounded values in its own
// half (at 0 and 64), so neither warpgroup overwrites what the other still
// reads. Heads of at most 64 elements leave room for a second S^T, so that a
// block's S is there when the elementwise step of the one before ends.
// Shared memory: K, V, rings of Q (whose tiles are held longest, from S to dK)
// and of G, and the rows' lse and delta. At D = 128 it is used to the last
// kilobyte: a third Q tile is worth more than any slack.
__host__ __device__ constexpr uint32_t kv_q_stages(int atoms) { return atoms == 2 ? 3 : 5; }
__host__ __device__ constexpr uint32_t kv_g_stages(int atoms) { return atoms == 2 ? 2 : 4; }
constexpr uint32_t kStatStages = 2;
__host__ __device__ constexpr int smem_kv(int atoms) {
    return static_cast<int>((2 + kv_q_stages(atoms) + kv_g_stages(atoms)) * atoms * kAtomBytes + kStatStages * 1024u) + 1024;
}

template <int kAtoms, bool kBf>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_grad_kv_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                           const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                           const __grid_constant__ AttnArgs a) {
    constexpr uint32_t SQ = kv_q_stages(kAtoms), SG = kv_g_stages(kAtoms), ST = kStatStages;
    constexpr uint32_t NS = kAtoms == 2 ? 1 : 2;  // S^T buffers
    constexpr uint32_t kTile = kAtoms * kAtomBytes;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    if (raw & 1023u) {  // the tiles' swizzle needs the alignment asked for above
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTimeout | kSiteSelftest);
        return;
    }
    const uint32_t k_s = raw, v_s = raw + kTile, q_ring = raw + 2 * kTile, g_ring = q_ring + SQ * kTile;
    const uint32_t stats = g_ring + SG * kTile;  // per stage: 128 x (8 - lse'), 128 x (-delta 2^-8, scaled as dS)
    const ItemQueue queue{stats + ST * 1024u, a.item_limit};
    const uint32_t bars = queue.base + ItemQueue::kBytes;
    auto q_full = [&](uint32_t s) { return bars + 8u * s; };
    auto q_empty = [&](uint32_t s) { return bars + 8u * (SQ + s); };
    const uint32_t bars_g = bars + 16u * SQ, bars_t = bars_g + 16u * SG, rest = bars_t + 16u * ST;
    auto g_full = [&](uint32_t s) { return bars_g + 8u * s; };
    auto g_empty = [&](uint32_t s) { return bars_g + 8u * (SG + s); };
    auto t_full = [&](uint32_t s) { return bars_t + 8u * s; };
    auto t_empty = [&](uint32_t s) { return bars_t + 8u * (ST + s); };
    // a block's S and P signal by its buffer: either side may be one block ahead of the other
    auto s_full = [&](uint32_t b) { return rest + 8u * b; };
    auto p_ready = [&](uint32_t b) { return rest + 16u + 8u * b; };
    const uint32_t kv_full = rest + 32, kv_empty = rest + 40, dp_full = rest + 48, ds_ready = rest + 56,
                   done = rest + 64, acc_read = rest + 72, drain = rest + 80, cleared = rest + 88, to_clear = rest + 96;
    const uint32_t slot_off = rest + 104 - raw;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + slot_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + slot_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tpt = kAttnTcRows / a.group, most = tpt * a.group;  // rows of a full block
    if (warp == kWarpLoad && lane == 0) {
        for (uint32_t i = 0; i < 2 * SQ; ++i) mbar_init(bars + 8u * i, 1);
        for (uint32_t i = 0; i < 2 * SG; ++i) mbar_init(bars_g + 8u * i, 1);
        for (uint32_t i = 0; i < ST; ++i) {
            mbar_init(t_full(i), 1);
            mbar_init(t_empty(i), 8);
        }
        const uint32_t ones[] = {s_full(0), s_full(1), kv_full, kv_empty, dp_full, done, drain, cleared, to_clear};
        for (uint32_t b : ones) mbar_init(b, 1);
        const uint32_t eights[] = {p_ready(0), p_ready(1), ds_ready, acc_read};
        for (uint32_t b : eights) mbar_init(b, 8);
        queue.init(11);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mg);
        tma_prefetch_desc(&mk);
        tma_prefetch_desc(&mv);
    }
    if (warp == kWarpIssue) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
        tmem_relinquish();
    }
    if (warp == kWarpAid && most < kAttnTcRows) {
        // rows that no copy ever writes (a group that does not divide the tile): zero for good, since
        // the sums multiply them by 0
        for (uint32_t i = 0; i < SQ + SG; ++i) zero_rows(q_ring + i * kTile, kAtoms, kAtomBytes, most, kAttnTcRows);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    dependency_wait();
    const uint32_t c_dp = tmem + 128u * NS, c_dv = c_dp + 128u, c_dk = c_dv + 64u * kAtoms;
    auto c_s = [&](uint32_t b) { return tmem + 128u * b; };

    if (warp >= 8) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == kWarpServe) {
            // ------------------------------------------------------------ items
            serve_items(queue, abort_flag, a.status, [&](int32_t index, AttnItem& it) {
                it.kh = index % a.hk;
                const AttnSeq s = attn_find(a, true, kKeys, index / a.hk);
                if (s.tile < 0) return false;
                it.q0 = s.q0;
                it.k0 = s.k0;
                it.lq = s.lq;
                it.lk = s.lk;
                it.room = s.room;
                it.first = s.tile * kKeys;
                // the blocks of query rows that see the tile's first key, or later ones
                it.j0 = a.causal ? max(0, it.first + s.lq - s.lk) / tpt : 0;
                it.n0 = it.first < s.lk ? max(0, (s.lq + tpt - 1) / tpt - it.j0) : 0;
                if constexpr (!kBf) {
                    const int32_t* sizes = a.sizes + (static_cast<int64_t>(s.b) * a.hk + it.kh) * 2;
                    it.split = sizes[0] + sizes[1];
                }
                return true;
            });
        } else if (warp == kWarpLoad) {
            // ------------------------------------------------------------ loads
            const uint32_t bytes = static_cast<uint32_t>(kAtoms * most) * 128u;
            uint32_t qi = 0, gi = 0, tiles = 0;
            for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
                if (it.n0 == 0) return true;
                if (!warp_wait_bounded(kv_empty, (tiles & 1u) ^ 1u, abort_flag, a.status, kSiteTmaEmpty)) return false;
                mbar_arrive_expect_tx_elect(kv_full, 2u * kTile);
                for (int at = 0; at < kAtoms; ++at) {
                    tma_load_3d_elect(k_s + at * kAtomBytes, &mk, 64 * at, it.kh, it.k0 + it.first, kv_full);
                    tma_load_3d_elect(v_s + at * kAtomBytes, &mv, 64 * at, it.kh, it.k0 + it.first, kv_full);
                }
                ++tiles;
                for (int32_t i = 0; i < it.n0; ++i) {
                    const int32_t row = it.q0 + (it.j0 + i) * tpt;
                    const uint32_t sq = qi % SQ, sg = gi % SG;
                    if (!warp_wait_bounded(q_empty(sq), ((qi / SQ) & 1u) ^ 1u, abort_flag, a.status, kSiteTmaEmpty))
                        return false;
                    mbar_arrive_expect_tx_elect(q_full(sq), bytes);
                    for (int at = 0; at < kAtoms; ++at)
                        tma_load_4d_elect(q_ring + sq * kTile + at * kAtomBytes, &mq, 64 * at, 0, it.kh, row, q_full(sq));
                    ++qi;
                    if (!warp_wait_bounded(g_empty(sg), ((gi / SG) & 1u) ^ 1u, abort_flag, a.status, kSiteTmaEmpty))
                        return false;
                    mbar_arrive_expect_tx_elect(g_full(sg), bytes);
                    for (int at = 0; at < kAtoms; ++at)
                        tma_load_4d_elect(g_ring + sg * kTile + at * kAtomBytes, &mg, 64 * at, 0, it.kh, row, g_full(sg));
                    ++gi;
                }
                return true;
            });
            if (*abort_flag) {  // the copies already issued land before the CTA exits
                volatile int never = 0;
                if (tiles) warp_wait_bounded(kv_full, (tiles - 1) & 1u, &never, a.status, kSiteDrain, 200000000ull);
                for (uint32_t i = qi > SQ ? qi - SQ : 0; i < qi; ++i)
                    warp_wait_bounded(q_full(i % SQ), (i / SQ) & 1, &never, a.status, kSiteDrain, 200000000ull);
                for (uint32_t i = gi > SG ? gi - SG : 0; i < gi; ++i)
                    warp_wait_bounded(g_full(i % SG), (i / SG) & 1, &never, a.status, kSiteDrain, 200000000ull);
            }
        } else if (warp == kWarpAid) {
            // ------------------------------------------------------------ lse and delta of a block's rows
            // A lane's four rows of a block are the same in every block: their places are taken apart
            // once, and the next block's values are on their way while this one's are handed over.
            uint32_t b = 0, turn = 0;  // blocks so far
            int64_t place[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = lane + 32 * k;
                place[k] = static_cast<int64_t>(r % a.group) * a.tq + r / a.group;
            }
            for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
                const int64_t head = static_cast<int64_t>(it.kh) * a.group * a.tq + it.q0;
                const float un = kBf ? kUnshift : power2(score_shift(it.split) - 8);
                float nl[4], nd[4];
                auto fetch = [&](int32_t i) {
                    const int32_t tok0 = (it.j0 + i) * tpt, rows = i < it.n0 ? min(tpt, it.lq - tok0) * a.group : 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        nl[k] = nd[k] = 0.0f;
                        if (lane + 32 * k < rows) {
                            nl[k] = a.lse[head + tok0 + place[k]];
                            nd[k] = a.delta[head + tok0 + place[k]];
                        }
                    }
                };
                fetch(0);
                for (int32_t i = 0; i < it.n0; ++i, ++b) {
                    const uint32_t st = b % ST, ph = (b / ST) & 1u;
                    const int32_t rows = min(tpt, it.lq - (it.j0 + i) * tpt) * a.group;
                    float l[4], d[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        l[k] = nl[k];
                        d[k] = nd[k];
                    }
                    fetch(i + 1);
                    if (!warp_wait_bounded(t_empty(st), ph ^ 1u, abort_flag, a.status, kSiteTmaEmpty)) return false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        st_shared_f32(stats + st * 1024u + 4u * (lane + 32 * k), fmaf(-kLog2e, l[k], kShift));
                        st_shared_f32(stats + st * 1024u + 512u + 4u * (lane + 32 * k), -d[k] * un);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(t_full(st));
                    if (i + 1 == it.n0 && rows < most) {
                        // the sequence's last block: another's rows behind its own, multiplied by 0 (the
                        // issuing thread has seen both tiles arrive)
                        if (!warp_wait2(to_clear, 0u, turn, abort_flag, a.status, kSiteTmaEmpty)) return false;
                        turn ^= 1u;
                        zero_rows(q_ring + (b % SQ) * kTile, kAtoms, kAtomBytes, rows, kAttnTcRows);
                        zero_rows(g_ring + (b % SG) * kTile, kAtoms, kAtomBytes, rows, kAttnTcRows);
                        if (lane == 0) mbar_arrive(cleared);
                    }
                }
                return true;
            });
        } else {
            // ------------------------------------------------------------ MMAs, one thread
            if (elect_lane()) {
                const uint32_t fmt = kBf ? 1u : 0u;
                const uint32_t nd = static_cast<uint32_t>((a.D + 15) & ~15);
                const uint32_t id_s = make_idesc(fmt, 128u, 128u), id_o = make_idesc(fmt, 128u, nd) | (1u << 16);
                const int ksteps = (a.D + 15) / 16;
                const uint64_t dk0 = desc_sw128(k_s, 16u, 1024u), dv0 = desc_sw128(v_s, 16u, 1024u);
                const uint64_t dq0 = desc_sw128(q_ring, 16u, 1024u), dg0 = desc_sw128(g_ring, 16u, 1024u);
                const uint64_t mq0 = desc_sw128(q_ring, kAtomBytes, 1024u), mg0 = desc_sw128(g_ring, kAtomBytes, 1024u);
                auto wait = [&](uint32_t b, uint32_t parity) {
                    return mbar_wait_bounded(b, parity, abort_flag, a.status, kSiteMmaFull);
                };
                // d (+)= the rounded values at x times the rows at y, over the block's 128 rows
                auto sums = [&](uint32_t d, uint32_t x, uint64_t y, bool more) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_f16_ts(d, x + 8u * kk + (kk >= 4 ? 32u : 0u), y + 128u * kk, id_o, more || kk > 0);
                };
                uint32_t sq = 0, pq = 0, sg = 0, pg = 0;  // stage and phase of the next Q and G to arrive
                uint32_t tq = 0, tg = 0;                  // stages of the next sums
                uint32_t bs = 0;                          // blocks whose S has been issued
                uint32_t b = 0;                           // blocks summed
                uint32_t items = 0, clear = 0;            // parities
                auto next = [](uint32_t& s, uint32_t n) {
                    const bool wrap = ++s == n;
                    if (wrap) s = 0;
                    return wrap;
                };
                for_items_one(queue, abort_flag, a.status, [&](const AttnItem& it) {
                    const int32_t n = it.n0;
                    if (n == 0) return true;
                    const bool partial = (it.lq - (it.j0 + n - 1) * tpt) * a.group < most;
                    auto scores = [&]() {
                        if (!wait(q_full(sq), pq)) return false;
                        tc_fence_after();
                        head_product<kAtoms>(c_s(bs % NS), dk0, dq0 + sq * (kTile >> 4), id_s, ksteps);
                        mma_commit(s_full(bs % NS));
                        ++bs;
                        if (next(sq, SQ)) pq ^= 1u;
                        return true;
                    };
                    auto grads = [&](bool last) {
                        if (!wait(g_full(sg), pg)) return false;
                        if (last && partial) mbar_arrive(to_clear);  // this block's Q came before
                        tc_fence_after();
                        head_product<kAtoms>(c_dp, dv0, dg0 + sg * (kTile >> 4), id_s, ksteps);
                        mma_commit(dp_full);
                        if (last) mma_commit(kv_empty);
                        if (next(sg, SG)) pg ^= 1u;
                        return true;
                    };
                    if (!wait(kv_full, items) || !scores() || !grads(n == 1)) return false;
                    for (int32_t i = 0; i < n; ++i, ++b) {
                        const uint64_t yq = mq0 + tq * (kTile >> 4), yg = mg0 + tg * (kTile >> 4);
                        // a second S^T: the next block's goes ahead of this one's sums
                        if (NS == 2 && i + 1 < n && !scores()) return false;
                        if (i == 0 && !wait(acc_read, items ^ 1u)) return false;
                        if (i + 1 == n && partial) {
                            if (!wait(cleared, clear)) return false;
                            clear ^= 1u;
                        }
                        if (!wait(p_ready(b % NS), (b / NS) & 1u)) return false;
                        tc_fence_after();
                        sums(c_dv, c_s(b % NS), yg, i > 0);
                        mma_commit(g_empty(tg));
                        if (NS == 1 && i + 1 < n && !scores()) return false;
                        if (!wait(ds_ready, b & 1u)) return false;
                        tc_fence_after();
                        sums(c_dk, c_dp, yq, i > 0);
                        mma_commit(q_empty(tq));
                        if (i + 1 < n && !grads(i + 2 == n)) return false;
                        next(tq, SQ);
                        next(tg, SG);
                    }
                    mma_commit(done);
                    items ^= 1u;
                    return true;
                });
                mma_commit(drain);
                volatile int never = 0;
                mbar_wait_bounded(drain, 0, &never, a.status, kSiteDrain, 200000000ull);
            }
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<kRegsRow>();
        // ---------------------------------------------------------------- a key per thread
        const int half = warp >> 2;  // columns (query rows) [64 half, 64 half + 64) of each block
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float sc = a.scale * kLog2e;
        const uint64_t sc2 = pack2(sc, sc);
        uint32_t b = 0, items = 0;  // blocks, and items with any, so far
        for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
            const int32_t key = it.first + r, shift = it.lk - it.lq, n = it.n0;
            const int scaled = kBf ? 0 : score_shift(it.split);  // of dS: its factor's exponent
            const uint64_t un2 = pack2(power2(scaled - 8), power2(scaled - 8));
            for (int32_t i = 0; i < n; ++i, ++b) {
                const uint32_t st = b % ST, ph = (b / ST) & 1u, scol = c_s(b % NS) + lanes + 64u * half;
                const int32_t tok0 = (it.j0 + i) * tpt, rows = min(tpt, it.lq - tok0) * a.group;
                // this key is seen by the block's rows from `from` on
                const int32_t from = a.causal ? min(max(0, key - shift - tok0), tpt) * a.group : 0;
                const bool masked = __any_sync(0xffffffffu, from > 64 * half) || rows < 64 * half + 64;
                const uint32_t lse_s = stats + st * 1024u + 256u * half, delta_s = lse_s + 512u;
                if (!warp_wait2(t_full(st), 0u, ph, abort_flag, a.status, kSiteGatherEmpty)) return false;
                if (!warp_wait2(s_full(b % NS), 0u, (b / NS) & 1u, abort_flag, a.status, kSiteGatherEmpty)) return false;
                tc_fence_after();
                uint32_t x[2][32], out[32];
                load_half(scol, x);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const uint4 l = ld_shared_v4(lse_s + 4u * (32 * c + k));
                        float u, w;
                        unpack2(fma2(pack2(__uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1])), sc2,
                                     pack2(__uint_as_float(l.x), __uint_as_float(l.y))),
                                u, w);
                        x[c][k] = __float_as_uint(attn_exp2(u));
                        x[c][k + 1] = __float_as_uint(attn_exp2(w));
                        unpack2(fma2(pack2(__uint_as_float(x[c][k + 2]), __uint_as_float(x[c][k + 3])), sc2,
                                     pack2(__uint_as_float(l.z), __uint_as_float(l.w))),
                                u, w);
                        x[c][k + 2] = __float_as_uint(attn_exp2(u));
                        x[c][k + 3] = __float_as_uint(attn_exp2(w));
                    }
                if (masked) {
                    const int32_t lo = from - 64 * half, hi = rows - 64 * half;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k < lo || 32 * c + k >= hi) x[c][k] = 0u;
                    __syncwarp();
                }
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    out[k] =
                        round2<kBf>(__uint_as_float(x[k >> 4][2 * (k & 15)]), __uint_as_float(x[k >> 4][2 * (k & 15) + 1]));
                tmem_st32(scol, out);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready(b % NS));

                if (!warp_wait2(dp_full, 0u, b & 1u, abort_flag, a.status, kSiteGatherEmpty)) return false;
                tc_fence_after();
                uint32_t dp[2][32];
                load_half(c_dp + lanes + 64u * half, dp);
                if (masked) {
                    const int32_t lo = from - 64 * half, hi = rows - 64 * half;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k < lo || 32 * c + k >= hi) dp[c][k] = 0u;
                    __syncwarp();
                }
                uint64_t d2[2];
                score_grads<kBf>(
                    x, dp, un2,
                    [&](int k) {
                        if ((k & 2) == 0) {
                            const uint4 d = ld_shared_v4(delta_s + 4u * k);
                            d2[0] = pack2(__uint_as_float(d.x), __uint_as_float(d.y));
                            d2[1] = pack2(__uint_as_float(d.z), __uint_as_float(d.w));
                        }
                        return d2[(k >> 1) & 1];
                    },
                    out);
                tmem_st32(c_dp + lanes + 64u * half, out);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(ds_ready);
                    mbar_arrive(t_empty(st));
                }
            }
            const bool any = n > 0;
            if (any) {
                if (!warp_wait2(done, 0u, items & 1u, abort_flag, a.status, kSiteEpilogue)) return false;
                ++items;
                tc_fence_after();
            }
            const AttnTensor& t = half ? a.gk : a.gv;
            uint8_t* p = static_cast<uint8_t*>(t.p) + 2 * (static_cast<int64_t>(it.k0 + key) * t.st + it.kh * t.sh);
            // keys past the last in use see nothing: their rows hold zeros
            const bool used = any && key < it.lk;
            const float f = used ? (half ? a.scale * power2(-scaled) : kUnshift) : 0.0f;
            const bool live = key < it.room;
            const bool wide = (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
#pragma unroll 1
            for (int c = 0; c < a.D; c += 16) {
                float v[16];
                __syncwarp();
                if (any) tmem_ld16((half ? c_dk : c_dv) + lanes + static_cast<uint32_t>(c), v);
                if (live) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = used ? v[i] * f : 0.0f;
                    store16<kBf>(p + 2 * c, v, a.D - c, wide);
                }
            }
            __syncwarp();
            if (any) {  // the next item's first sums may overwrite dV and dK
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_read);
            }
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpIssue) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int kAtoms, bool kBf>
cudaError_t launch_backward(int dtype, const AttnArgs& a, cudaStream_t st) {
    CUtensorMap mq, mg, mk, mv;
    const int tpt = kAttnTcRows / a.group;
    if (!attn_encode_rows(&mq, a, a.q, dtype, tpt) || !attn_encode_rows(&mg, a, a.g, dtype, tpt) ||
        !attn_encode_keys(&mk, a, a.k, dtype, kKeys) || !attn_encode_keys(&mv, a, a.v, dtype, kKeys))
        return cudaErrorInvalidValue;
    cudaError_t e;
    const unsigned hk = static_cast<unsigned>(a.hk);
    if (a.tq > 0) {
        auto kern = attn_grad_q_tc_kernel<kAtoms, kBf>;
        constexpr int smem = smem_q(kAtoms);
        static_assert(smem <= 227 * 1024, "shared memory");
        static std::atomic<uint64_t> done{0};
        if ((e = attn_allow_smem(kern, smem, done)) != cudaSuccess) return e;
        const unsigned tiles = static_cast<unsigned>(attn_tiles(a.tq, a.batch, tpt));
        if ((e = launch_dependent(kern, dim3(tiles * hk), kTcThreads, smem, st, mq, mg, mk, mv, a)) != cudaSuccess) return e;
    }
    if (a.tk > 0) {
        auto kern = attn_grad_kv_tc_kernel<kAtoms, kBf>;
        constexpr int smem = smem_kv(kAtoms);
        static_assert(smem <= 227 * 1024, "shared memory");
        static std::atomic<uint64_t> done{0};
        if ((e = attn_allow_smem(kern, smem, done)) != cudaSuccess) return e;
        const unsigned tiles = static_cast<unsigned>(attn_tiles(a.tk, a.batch, kKeys));
        if ((e = launch_dependent(kern, dim3(tiles * hk), kTcThreads, smem, st, mq, mg, mk, mv, a)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_attention_tc_backward(int dtype, const AttnArgs& args, cudaStream_t st) {
    AttnArgs a = args;
    const int64_t row_steps = a.tq / (kAttnTcRows / a.group) + 1, key_steps = a.tk / kKeys + 1;
    a.item_limit = attn_item_limit(kWaitLimitCycles, row_steps > key_steps ? row_steps : key_steps);
    if (a.D <= 64)
        return dtype == kBF16 ? launch_backward<1, true>(dtype, a, st) : launch_backward<1, false>(dtype, a, st);
    return dtype == kBF16 ? launch_backward<2, true>(dtype, a, st) : launch_backward<2, false>(dtype, a, st);
}

}  // namespace mdcn
