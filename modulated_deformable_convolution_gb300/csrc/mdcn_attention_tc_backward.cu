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
// numbers; dS is kept unscaled, since a gradient's size is not bounded.
//
// Bound by the tensor cores: 3 (grad_q) and 4 (grad_kv) products of 128 x 128 x
// D per tile, about 512 cycles each at D = 128. While the elementwise step of
// one tile runs, the next tile's S and dP, or this tile's sums, are computed.
#include <cuda.h>

#include <cstdint>

#include "mdcn_attention_tc.cuh"
#include "mdcn_plan.h"

namespace mdcn {

namespace {

constexpr int kTcThreads = 384;
constexpr int kWarpLoad = 8, kWarpIssue = 9, kWarpStats = 10;
constexpr int kRegsRow = 216, kRegsCtl = 72;  // of 168 a thread at launch
static_assert(2 * kRegsRow + kRegsCtl <= 3 * 168, "register split must fit the launch's");
constexpr int kKeys = 128;
constexpr float kShift = 8.0f, kUnshift = 0.00390625f;  // P is kept times 2^8

// ds = p 2^8 * (dp - delta) 2^-8 for 64 columns of a row; p in, packed ds out.
// d2: -delta * 2^-8 for column pairs.
template <bool kBf, typename F>
__device__ __forceinline__ void score_grads(const uint32_t (&p)[2][32], const uint32_t (&dp)[2][32], F minus_delta,
                                            uint32_t (&out)[32]) {
    const uint64_t un = pack2(kUnshift, kUnshift);
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
        if (any) tmem_ld16(col + static_cast<uint32_t>(c), v);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = any ? v[i] * f : 0.0f;
        store16<kBf>(p + 2 * c, v, c1 - c, wide);
    }
}

__host__ __device__ constexpr int stages_of(int atoms) { return atoms == 2 ? 5 : 8; }
__host__ __device__ constexpr int smem_q(int atoms) {
    return 1024 + (2 + stages_of(atoms)) * atoms * static_cast<int>(kAtomBytes) + 256;
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
    const uint32_t q_s = base, g_s = base + kTile, ring = base + 2 * kTile, bars = ring + S * kTile;
    auto full = [&](uint32_t s) { return bars + 8u * s; };
    auto empty = [&](uint32_t s) { return bars + 8u * (S + s); };
    const uint32_t rest = bars + 16u * S;
    const uint32_t q_full = rest, drain = rest + 8, s_full = rest + 16, p_full = rest + 24, s_read = rest + 32,
                   dp_read = rest + 40, ds_full = rest + 48, dq_done = rest + 56;
    const uint32_t slot_off = rest + 64 - raw;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + slot_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + slot_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tpt = kAttnTcRows / a.group;
    const AttnSeq s = attn_find(a, false, tpt, blockIdx.x);
    if (s.tile < 0) return;
    const int kh = blockIdx.y;
    const int32_t tok0 = s.tile * tpt, ntok = min(tpt, s.lq - tok0);
    const int32_t n = (attn_seen(a, s, tok0 + ntok - 1) + kKeys - 1) / kKeys;

    if (warp == kWarpLoad && lane == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(drain, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 1);
        mbar_init(s_read, 8);
        mbar_init(dp_read, 8);
        mbar_init(ds_full, 8);
        mbar_init(dq_done, 1);
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
    const uint32_t c_s = tmem, c_dp = tmem + 128u, c_ds = tmem + 256u, c_dq = tmem + 320u;

    if (warp >= 8) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == kWarpLoad && n > 0) {
            mbar_arrive_expect_tx_elect(q_full, 2u * kAtoms * static_cast<uint32_t>(tpt * a.group) * 128u);
            for (int at = 0; at < kAtoms; ++at) {
                tma_load_4d_elect(q_s + at * kAtomBytes, &mq, 64 * at, 0, kh, s.q0 + tok0, q_full);
                tma_load_4d_elect(g_s + at * kAtomBytes, &mg, 64 * at, 0, kh, s.q0 + tok0, q_full);
            }
            bool ok = true;
            uint32_t st = 0, ph = 0, issued = 0;
            for (int32_t j = 0; j < n && ok; ++j) {
                for (int kv = 0; kv < 2; ++kv) {
                    if (!warp_wait_bounded(empty(st), ph ^ 1u, abort_flag, a.status, kSiteTmaEmpty)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx_elect(full(st), kTile);
                    for (int at = 0; at < kAtoms; ++at)
                        tma_load_3d_elect(ring + st * kTile + at * kAtomBytes, kv ? &mv : &mk, 64 * at, kh,
                                          s.k0 + j * kKeys, full(st));
                    ++issued;
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {  // the copies already issued land before the CTA exits
                volatile int never = 0;
                warp_wait_bounded(q_full, 0, &never, a.status, kSiteDrain, 200000000ull);
                const uint32_t first = issued > S ? issued - S : 0;
                for (uint32_t i = first; i < issued; ++i)
                    warp_wait_bounded(full(i % S), (i / S) & 1, &never, a.status, kSiteDrain, 200000000ull);
            }
        } else if (warp == kWarpIssue && n > 0) {
            const uint32_t fmt = kBf ? 1u : 0u;
            const uint32_t nd = static_cast<uint32_t>((a.D + 15) & ~15);
            const uint32_t id_s = make_idesc(fmt, 128u, kKeys), id_q = make_idesc(fmt, 128u, nd) | (1u << 16);
            const int ksteps = (a.D + 15) / 16;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return warp_wait2(bar, 0u, parity, abort_flag, a.status, kSiteMmaFull);
            };
            auto product = [&](uint32_t d, uint32_t x, uint32_t y) {
                for (int kk = 0; kk < ksteps; ++kk) {
                    const uint32_t off = static_cast<uint32_t>(kk >> 2) * kAtomBytes + 32u * (kk & 3);
                    mma_f16_elect(d, desc_sw128(x + off, 16u, 1024u), desc_sw128(y + off, 16u, 1024u), id_s, kk > 0);
                }
            };
            // S and dP of key tile j, into the buffers whose previous values have been read
            auto scores = [&](int32_t j) {
                const uint32_t e = 2u * j, sk = e % S, sv = (e + 1) % S;
                if (!wait(full(sk), (e / S) & 1)) return false;
                // dQ += dS K multiplies the rows past the last key by 0
                const int32_t valid = s.lk - j * kKeys;
                if (valid < kKeys) zero_rows(ring + sk * kTile, kAtoms, kAtomBytes, valid, kKeys);
                if (j > 0 && !wait(s_read, (j - 1) & 1)) return false;
                tc_fence_after();
                product(c_s, q_s, ring + sk * kTile);
                mma_commit_elect(s_full);
                if (!wait(full(sv), ((e + 1) / S) & 1)) return false;
                if (j > 0 && !wait(dp_read, (j - 1) & 1)) return false;
                tc_fence_after();
                product(c_dp, g_s, ring + sv * kTile);
                mma_commit_elect(p_full);
                mma_commit_elect(empty(sv));
                return true;
            };
            bool ok = wait(q_full, 0) && scores(0);
            for (int32_t j = 0; j < n && ok; ++j) {
                if (j + 1 < n && !(ok = scores(j + 1))) break;
                if (!(ok = wait(ds_full, j & 1))) break;
                tc_fence_after();
                const uint32_t sk = (2u * j) % S;
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    mma_f16_ts_elect(c_dq, c_ds + 8u * kk, desc_sw128(ring + sk * kTile + 2048u * kk, kAtomBytes, 1024u),
                                     id_q, j > 0 || kk > 0);
                mma_commit_elect(empty(sk));
                mma_commit_elect(dq_done);
            }
            mma_commit_elect(drain);
            volatile int never = 0;
            warp_wait2(drain, 0u, 0, &never, a.status, kSiteDrain, 200000000ull);
        }
    } else {
        setmaxnreg_inc<kRegsRow>();
        const int half = warp >> 2;  // columns [64 half, 64 half + 64) of each tile
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const bool live = r < ntok * a.group;
        const int tk = r / a.group, h = kh * a.group + (r - tk * a.group);
        const int64_t tok = s.q0 + tok0 + tk;
        const int32_t seen = live ? attn_seen(a, s, tok0 + tk) : 0;
        const int32_t seen_all = __reduce_min_sync(0xffffffffu, live ? seen : 0x7fffffff);
        const float sc = a.scale * kLog2e;
        const float lse = live ? a.lse[static_cast<int64_t>(h) * a.tq + tok] * kLog2e : 0.0f;
        const float delta = live ? a.delta[static_cast<int64_t>(h) * a.tq + tok] * kUnshift : 0.0f;
        const uint64_t sc2 = pack2(sc, sc), l2 = pack2(kShift - lse, kShift - lse), d2 = pack2(-delta, -delta);
        bool ok = true;
        for (int32_t j = 0; j < n; ++j) {
            if (!(ok = warp_wait2(s_full, 0u, j & 1, abort_flag, a.status, kSiteGatherEmpty))) break;
            tc_fence_after();
            uint32_t x[2][32];
            load_half(c_s + lanes + 64u * half, x);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_read);
            const int32_t first = j * kKeys + 64 * half;
            const bool masked = seen_all < first + 64;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float u, w;
                    unpack2(fma2(pack2(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1])), sc2, l2), u, w);
                    x[c][i] = __float_as_uint(attn_exp2(u));
                    x[c][i + 1] = __float_as_uint(attn_exp2(w));
                }
            if (!(ok = warp_wait2(p_full, 0u, j & 1, abort_flag, a.status, kSiteGatherEmpty))) break;
            tc_fence_after();
            uint32_t dp[2][32], ds[32];
            load_half(c_dp + lanes + 64u * half, dp);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dp_read);
            if (masked) {
                const int32_t left = seen - first;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * c + i >= left) x[c][i] = dp[c][i] = 0u;
            }
            score_grads<kBf>(x, dp, [&](int) { return d2; }, ds);
            if (j > 0 && !(ok = warp_wait2(dq_done, 0u, (j - 1) & 1, abort_flag, a.status, kSiteGatherEmpty))) break;
            tc_fence_after();
            tmem_st32(c_ds + lanes + 32u * half, ds);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        const bool any = n > 0;
        if (any && ok) ok = warp_wait2(dq_done, 0u, (n - 1) & 1, abort_flag, a.status, kSiteEpilogue);
        if (ok && *abort_flag == 0) {
            tc_fence_after();
            uint8_t* p = static_cast<uint8_t*>(a.gq.p) + 2 * (tok * a.gq.st + h * a.gq.sh);
            const int mid = min(32 * kAtoms, a.D);
            store_row<kBf>(c_dq + lanes, p, half ? mid : 0, half ? a.D : mid, a.scale, any, live);
        }
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
// Tensor memory: S^T [0, 128) with P^T over it, dP^T [128, 256) with dS^T over
// it, dV [256, 256 + D), dK [384, 384 + D). Each half of the columns keeps its
// rounded values in its own half (at 0 and 64), so neither warpgroup overwrites
// what the other still reads.
__host__ __device__ constexpr uint32_t kv_stages(int atoms) { return atoms == 2 ? 2 : 4; }
__host__ __device__ constexpr int smem_kv(int atoms) {
    return 1024 + static_cast<int>((2 + 2 * kv_stages(atoms)) * atoms * kAtomBytes + kv_stages(atoms) * 1024u) + 512;
}

template <int kAtoms, bool kBf>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_grad_kv_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                           const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                           const __grid_constant__ AttnArgs a) {
    constexpr uint32_t S = kv_stages(kAtoms);
    constexpr uint32_t kTile = kAtoms * kAtomBytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t k_s = base, v_s = base + kTile, q_ring = base + 2 * kTile, g_ring = q_ring + S * kTile;
    const uint32_t stats = g_ring + S * kTile;  // per stage: 128 x (8 - lse'), 128 x (-delta 2^-8)
    const uint32_t bars = stats + S * 1024u;
    auto bar = [&](uint32_t kind, uint32_t s) { return bars + 8u * (kind * S + s); };
    auto q_full = [&](uint32_t s) { return bar(0, s); };
    auto q_empty = [&](uint32_t s) { return bar(1, s); };
    auto g_full = [&](uint32_t s) { return bar(2, s); };
    auto g_empty = [&](uint32_t s) { return bar(3, s); };
    auto t_full = [&](uint32_t s) { return bar(4, s); };
    auto t_empty = [&](uint32_t s) { return bar(5, s); };
    const uint32_t rest = bars + 48u * S;
    const uint32_t kv_full = rest, drain = rest + 8, s_full = rest + 16, dp_full = rest + 24, p_ready = rest + 32,
                   ds_ready = rest + 40, done = rest + 48;
    const uint32_t slot_off = rest + 56 - raw;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + slot_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + slot_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tpt = kAttnTcRows / a.group;
    const AttnSeq s = attn_find(a, true, kKeys, blockIdx.x);
    if (s.tile < 0) return;
    const int kh = blockIdx.y;
    const int32_t j0 = s.tile * kKeys;
    // the blocks of query rows that see key j0 and later ones
    const int32_t shift = s.lk - s.lq;
    int32_t b0 = a.causal ? max(0, j0 - shift) / tpt : 0;
    const int32_t b1 = j0 < s.lk ? (s.lq + tpt - 1) / tpt : 0;
    const int32_t n = max(0, b1 - b0);

    if (warp == kWarpLoad && lane == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), 1);
            mbar_init(g_full(i), 1);
            mbar_init(g_empty(i), 1);
            mbar_init(t_full(i), 1);
            mbar_init(t_empty(i), 8);
        }
        mbar_init(kv_full, 1);
        mbar_init(drain, 1);
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_ready, 8);
        mbar_init(ds_ready, 8);
        mbar_init(done, 1);
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
    const uint32_t c_s = tmem, c_dp = tmem + 128u, c_dv = tmem + 256u, c_dk = tmem + 384u;

    if (warp >= 8) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == kWarpLoad && n > 0) {
            // ------------------------------------------------------------ loads
            mbar_arrive_expect_tx_elect(kv_full, 2u * kTile);
            for (int at = 0; at < kAtoms; ++at) {
                tma_load_3d_elect(k_s + at * kAtomBytes, &mk, 64 * at, kh, s.k0 + j0, kv_full);
                tma_load_3d_elect(v_s + at * kAtomBytes, &mv, 64 * at, kh, s.k0 + j0, kv_full);
            }
            const uint32_t bytes = static_cast<uint32_t>(kAtoms * tpt * a.group) * 128u;
            bool ok = true;
            uint32_t qi = 0, gi = 0;
            for (int32_t i = 0; i < n && ok; ++i) {
                const uint32_t st = static_cast<uint32_t>(i) % S, ph = (static_cast<uint32_t>(i) / S) & 1u;
                const int32_t row = s.q0 + (b0 + i) * tpt;
                if (!(ok = warp_wait_bounded(q_empty(st), ph ^ 1u, abort_flag, a.status, kSiteTmaEmpty))) break;
                mbar_arrive_expect_tx_elect(q_full(st), bytes);
                for (int at = 0; at < kAtoms; ++at)
                    tma_load_4d_elect(q_ring + st * kTile + at * kAtomBytes, &mq, 64 * at, 0, kh, row, q_full(st));
                ++qi;
                if (!(ok = warp_wait_bounded(g_empty(st), ph ^ 1u, abort_flag, a.status, kSiteTmaEmpty))) break;
                mbar_arrive_expect_tx_elect(g_full(st), bytes);
                for (int at = 0; at < kAtoms; ++at)
                    tma_load_4d_elect(g_ring + st * kTile + at * kAtomBytes, &mg, 64 * at, 0, kh, row, g_full(st));
                ++gi;
            }
            if (!ok) {  // the copies already issued land before the CTA exits
                volatile int never = 0;
                warp_wait_bounded(kv_full, 0, &never, a.status, kSiteDrain, 200000000ull);
                for (uint32_t i = qi > S ? qi - S : 0; i < qi; ++i)
                    warp_wait_bounded(q_full(i % S), (i / S) & 1, &never, a.status, kSiteDrain, 200000000ull);
                for (uint32_t i = gi > S ? gi - S : 0; i < gi; ++i)
                    warp_wait_bounded(g_full(i % S), (i / S) & 1, &never, a.status, kSiteDrain, 200000000ull);
            }
        } else if (warp == kWarpStats && n > 0) {
            // ------------------------------------------------------------ lse and delta of a block's rows
            for (int32_t i = 0; i < n; ++i) {
                const uint32_t st = static_cast<uint32_t>(i) % S, ph = (static_cast<uint32_t>(i) / S) & 1u;
                const int32_t tok0 = (b0 + i) * tpt, rows = min(tpt, s.lq - tok0) * a.group;
                float l[4], d[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = lane + 32 * k;
                    l[k] = d[k] = 0.0f;
                    if (r < rows) {
                        const int64_t at = static_cast<int64_t>(kh * a.group + r % a.group) * a.tq + s.q0 + tok0 + r / a.group;
                        l[k] = a.lse[at];
                        d[k] = a.delta[at];
                    }
                }
                if (!warp_wait_bounded(t_empty(st), ph ^ 1u, abort_flag, a.status, kSiteTmaEmpty)) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    st_shared_f32(stats + st * 1024u + 4u * (lane + 32 * k), fmaf(-kLog2e, l[k], kShift));
                    st_shared_f32(stats + st * 1024u + 512u + 4u * (lane + 32 * k), -d[k] * kUnshift);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(t_full(st));
            }
        } else if (warp == kWarpIssue && n > 0) {
            // ------------------------------------------------------------ MMAs
            const uint32_t fmt = kBf ? 1u : 0u;
            const uint32_t nd = static_cast<uint32_t>((a.D + 15) & ~15);
            const uint32_t id_s = make_idesc(fmt, 128u, 128u), id_o = make_idesc(fmt, 128u, nd) | (1u << 16);
            const int ksteps = (a.D + 15) / 16;
            auto wait = [&](uint32_t b, uint32_t parity) {
                return warp_wait2(b, 0u, parity, abort_flag, a.status, kSiteMmaFull);
            };
            auto product = [&](uint32_t d, uint32_t x, uint32_t y) {
                for (int kk = 0; kk < ksteps; ++kk) {
                    const uint32_t off = static_cast<uint32_t>(kk >> 2) * kAtomBytes + 32u * (kk & 3);
                    mma_f16_elect(d, desc_sw128(x + off, 16u, 1024u), desc_sw128(y + off, 16u, 1024u), id_s, kk > 0);
                }
            };
            auto sums = [&](uint32_t d, uint32_t x, uint32_t y, bool more) {
                for (int kk = 0; kk < 8; ++kk)
                    mma_f16_ts_elect(d, x + 8u * kk + (kk >= 4 ? 32u : 0u), desc_sw128(y + 2048u * kk, kAtomBytes, 1024u),
                                     id_o, more || kk > 0);
            };
            // a block's rows past its last (another sequence's, or none) are multiplied by 0
            auto arrived = [&](uint32_t b, uint32_t tile, int32_t i) {
                if (!wait(b, (static_cast<uint32_t>(i) / S) & 1u)) return false;
                const int32_t rows = min(tpt, s.lq - (b0 + i) * tpt) * a.group;
                if (rows < kAttnTcRows) zero_rows(tile, kAtoms, kAtomBytes, rows, kAttnTcRows);
                tc_fence_after();
                return true;
            };
            auto scores = [&](int32_t i) {
                const uint32_t st = static_cast<uint32_t>(i) % S;
                if (!arrived(q_full(st), q_ring + st * kTile, i)) return false;
                product(c_s, k_s, q_ring + st * kTile);
                mma_commit_elect(s_full);
                return true;
            };
            auto grads = [&](int32_t i) {
                const uint32_t st = static_cast<uint32_t>(i) % S;
                if (!arrived(g_full(st), g_ring + st * kTile, i)) return false;
                product(c_dp, v_s, g_ring + st * kTile);
                mma_commit_elect(dp_full);
                return true;
            };
            bool ok = wait(kv_full, 0) && scores(0) && grads(0);
            for (int32_t i = 0; i < n && ok; ++i) {
                const uint32_t st = static_cast<uint32_t>(i) % S;
                if (!(ok = wait(p_ready, i & 1))) break;
                tc_fence_after();
                sums(c_dv, c_s, g_ring + st * kTile, i > 0);
                mma_commit_elect(g_empty(st));
                if (i + 1 < n && !(ok = scores(i + 1))) break;
                if (!(ok = wait(ds_ready, i & 1))) break;
                tc_fence_after();
                sums(c_dk, c_dp, q_ring + st * kTile, i > 0);
                mma_commit_elect(q_empty(st));
                if (i + 1 < n && !(ok = grads(i + 1))) break;
            }
            mma_commit_elect(done);
            mma_commit_elect(drain);
            volatile int never = 0;
            warp_wait2(drain, 0u, 0, &never, a.status, kSiteDrain, 200000000ull);
        }
    } else {
        setmaxnreg_inc<kRegsRow>();
        // ---------------------------------------------------------------- a key per thread
        const int half = warp >> 2;  // columns (query rows) [64 half, 64 half + 64) of each block
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int32_t key = j0 + r;
        const float sc = a.scale * kLog2e;
        const uint64_t sc2 = pack2(sc, sc);
        bool ok = true;
        for (int32_t i = 0; i < n; ++i) {
            const uint32_t st = static_cast<uint32_t>(i) % S, ph = (static_cast<uint32_t>(i) / S) & 1u;
            const int32_t tok0 = (b0 + i) * tpt, rows = min(tpt, s.lq - tok0) * a.group;
            // this key is seen by the block's rows from `from` on
            const int32_t from = a.causal ? min(max(0, key - shift - tok0), tpt) * a.group : 0;
            const bool masked = __any_sync(0xffffffffu, from > 64 * half) || rows < 64 * half + 64;
            const uint32_t lse_s = stats + st * 1024u + 256u * half, delta_s = lse_s + 512u;
            if (!(ok = warp_wait2(t_full(st), 0u, ph, abort_flag, a.status, kSiteGatherEmpty))) break;
            if (!(ok = warp_wait2(s_full, 0u, i & 1, abort_flag, a.status, kSiteGatherEmpty))) break;
            tc_fence_after();
            uint32_t x[2][32], out[32];
            load_half(c_s + lanes + 64u * half, x);
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
            }
#pragma unroll
            for (int k = 0; k < 32; ++k)
                out[k] = round2<kBf>(__uint_as_float(x[k >> 4][2 * (k & 15)]), __uint_as_float(x[k >> 4][2 * (k & 15) + 1]));
            tmem_st32(c_s + lanes + 64u * half, out);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_ready);

            if (!(ok = warp_wait2(dp_full, 0u, i & 1, abort_flag, a.status, kSiteGatherEmpty))) break;
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
            }
            uint64_t d2[2];
            score_grads<kBf>(
                x, dp,
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
        if (any && ok) ok = warp_wait2(done, 0u, 0, abort_flag, a.status, kSiteEpilogue);
        if (ok && *abort_flag == 0) {
            tc_fence_after();
            const AttnTensor& t = half ? a.gk : a.gv;
            uint8_t* p = static_cast<uint8_t*>(t.p) + 2 * (static_cast<int64_t>(s.k0 + key) * t.st + kh * t.sh);
            // keys past the last in use see nothing: their rows hold zeros
            const bool used = any && key < s.lk;
            const float f = used ? (half ? a.scale : kUnshift) : 0.0f;
            const bool live = key < s.room;
            const bool wide = (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
#pragma unroll 1
            for (int c = 0; c < a.D; c += 16) {
                float v[16];
                if (any) tmem_ld16((half ? c_dk : c_dv) + lanes + static_cast<uint32_t>(c), v);
                if (!live) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = used ? v[i] * f : 0.0f;
                store16<kBf>(p + 2 * c, v, a.D - c, wide);
            }
        }
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
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        const unsigned tiles = static_cast<unsigned>(attn_tiles(a.tq, a.batch, tpt));
        kern<<<dim3(tiles, hk), kTcThreads, smem, st>>>(mq, mg, mk, mv, a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.tk > 0) {
        auto kern = attn_grad_kv_tc_kernel<kAtoms, kBf>;
        constexpr int smem = smem_kv(kAtoms);
        static_assert(smem <= 227 * 1024, "shared memory");
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        const unsigned tiles = static_cast<unsigned>(attn_tiles(a.tk, a.batch, kKeys));
        kern<<<dim3(tiles, hk), kTcThreads, smem, st>>>(mq, mg, mk, mv, a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_attention_tc_backward(int dtype, const AttnArgs& a, cudaStream_t st) {
    if (a.D <= 64)
        return dtype == kBF16 ? launch_backward<1, true>(dtype, a, st) : launch_backward<1, false>(dtype, a, st);
    return dtype == kBF16 ? launch_backward<2, true>(dtype, a, st) : launch_backward<2, false>(dtype, a, st);
}

}  // namespace mdcn
