// Attention over packed sequences on the tensor cores (float16, bfloat16):
// the forward.
//
// A work item is two row tiles of 128 rows (row = token and query head of one
// key head) over the key tiles of 128 keys that they see:
//   S = Q K^T (fp32, tensor memory), P = exp2(scale' S - m) rounded to the
//   type of v, written over S in tensor memory, O += P V (fp32, tensor memory).
// Warps 0-3 and 4-7 hold one row per thread of the first and second tile (a
// tensor-memory lane each, so row maxima and sums need no exchange), warp 8
// loads tiles by TMA into a ring, warp 9 issues the MMAs, warp 10 gets items.
// The steps of the two row tiles alternate, and the products of one run while
// the other's probabilities are computed. Heads of at most 64 elements leave
// room for three S in tensor memory, so that a row tile's next S is ready when
// its probabilities are done; with two, S follows the step's O += P V.
// O is rescaled only when a row's maximum has grown by more than 2^8 since it
// was last taken (P then stays below 2^8, exact in the sums: the result does
// not depend on which maximum is used beyond rounding), by the row's own warp.
//
// Bound by the tensor cores for long rows: per key tile and row tile two
// 128 x 128 x D products, 4 * 128 * 128 * D operations; at D = 64 by a row
// tile's chain of score, probabilities, sum.
// Shared memory: Q once, K and V in a ring of 128-row tiles, 227 KB in all.
//
// Measured (32 heads of 128 over 8, bfloat16): 12 packed causal prompts of up to
// 8192 tokens 1176 us, 1425 TFLOP/s of the pairs that are seen; 4 x 8192 without a mask
// 2590 us, 1700 TFLOP/s. A step of both row tiles takes about 2600 cycles, of
// which the tensor pipe works 2048: with P over S, the next S waits for it. At
// D = 64 (4 maps of 80 x 80, 2 heads, float16) 92 us, 912 TFLOP/s: some 2000
// cycles a step; the exponentials of a warp's 64 pairs of columns alone take
// 740 cycles, of two warps to a scheduler 630 each, the tensor pipe 1024. One
// new token against 16 caches of up to 8192 keys: 63 us, 4.6 TB/s of keys and
// values.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <type_traits>

#include "mdcn_attention_tc.cuh"
#include "mdcn_pdl.h"
#include "mdcn_plan.h"

namespace mdcn {

namespace {

constexpr int kTcThreads = 384;
constexpr int kWarpLoad = 8, kWarpIssue = 9, kWarpServe = 10, kWarpClear = 11;
constexpr int kRegsRow = 216, kRegsCtl = 72;  // of 168 a thread at launch
static_assert(2 * kRegsRow + kRegsCtl <= 3 * 168, "register split must fit the launch's");
constexpr int kKeys = 128;
constexpr float kRescaleLog2 = 8.0f;
using Zero = std::integral_constant<int, 0>;
using One = std::integral_constant<int, 1>;

// Stages of the ring: as many 128-row tiles as fit beside Q.
__host__ __device__ constexpr int stages_of(int atoms) { return atoms == 2 ? 5 : 8; }
__host__ __device__ constexpr int smem_of(int atoms) {
    return (2 + stages_of(atoms)) * atoms * static_cast<int>(kAtomBytes) + 768;
}

// S buffers in tensor memory, which the steps of both row tiles use in turn.
__host__ __device__ constexpr int scores_of(int atoms) { return atoms == 2 ? 2 : 3; }

// Which S buffer row tile t's key tile j goes to, in an item with n0 and n1 key
// tiles: with three, the next in turn (j by j, tile 0 first; `before`: S of
// earlier items); with two, one for each row tile, or both in turn where only
// one row tile has keys.
template <int kAtoms>
__device__ __forceinline__ uint32_t score_buffer(int t, int32_t j, int32_t n0, int32_t n1, uint32_t before) {
    if constexpr (scores_of(kAtoms) == 3) {
        const int32_t i = t ? min(j + 1, n0) + j : j + min(j, n1);
        return (before + static_cast<uint32_t>(i)) % 3u;
    } else {
        return n0 == 0 || n1 == 0 ? static_cast<uint32_t>(j & 1) : static_cast<uint32_t>(t);
    }
}

// kAtoms: 64-element atoms of a head (head_dim <= 64: 1, else 2).
template <int kAtoms, bool kBf>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_forward_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnArgs a) {
    constexpr uint32_t S = stages_of(kAtoms);
    constexpr uint32_t kTile = kAtoms * kAtomBytes;
    constexpr uint32_t NB = scores_of(kAtoms);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    if (raw & 1023u) {  // the tiles' swizzle needs the alignment asked for above
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTimeout | kSiteSelftest);
        return;
    }
    const uint32_t q_s = raw, ring = raw + 2 * kTile;
    const ItemQueue queue{ring + S * kTile, a.item_limit};
    const uint32_t bars = queue.base + ItemQueue::kBytes;
    auto full = [&](uint32_t s) { return bars + 8u * s; };
    auto empty = [&](uint32_t s) { return bars + 8u * (S + s); };
    const uint32_t rest = bars + 16u * S;
    // A row tile's i-th S signals barrier i % NB of that tile, its i-th P likewise: a barrier's next
    // use waits for what follows step i, so none gets two phases ahead of who waits for it, however
    // far either side lags (up to NB steps of a tile are under way)
    const uint32_t s_full0 = rest, p_full0 = rest + 48u, o_done0 = rest + 96u;
    auto s_full = [&](int t, uint32_t i) { return s_full0 + 24u * t + 8u * (i % NB); };
    auto p_full = [&](int t, uint32_t i) { return p_full0 + 24u * t + 8u * (i % NB); };
    auto o_done = [&](int t, uint32_t i) { return o_done0 + 24u * t + 8u * (i % NB); };  // O += P V of a step
    auto o_read = [&](int t) { return rest + 144u + 8u * t; };                           // an item's O
    auto q_full = [&](int t) { return rest + 160u + 8u * t; };
    auto q_empty = [&](int t) { return rest + 176u + 8u * t; };
    const uint32_t drain = rest + 192u, cleared = rest + 200u, to_clear = rest + 208u;
    const uint32_t slot_off = rest + 216u - raw;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + slot_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + slot_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kWarpLoad && lane == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            for (uint32_t i = 0; i < NB; ++i) {
                mbar_init(s_full(t, i), 1);
                mbar_init(p_full(t, i), 4);
                mbar_init(o_done(t, i), 1);
            }
            mbar_init(o_read(t), 4);
            mbar_init(q_full(t), 1);
            mbar_init(q_empty(t), 1);
        }
        mbar_init(drain, 1);
        queue.init(11);
        mbar_init(cleared, 1);
        mbar_init(to_clear, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&mq);
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
    if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    // tensor memory: the S buffers (128 columns each, P over the first 64), O of row tile 0 and 1
    auto s_col = [&](uint32_t b) { return tmem + 128u * b; };
    auto o_col = [&](int t) { return tmem + 128u * NB + 64u * kAtoms * t; };
    const int tpt = kAttnTcRows / a.group;

    if (warp >= 8) {
        setmaxnreg_dec<kRegsCtl>();
        if (warp == kWarpServe) {
            // ------------------------------------------------------------ items
            serve_items(queue, abort_flag, a.status, [&](int32_t index, AttnItem& it) {
                // key heads fastest, then the shares of a row tile's keys
                it.kh = index % a.hk;
                const int32_t rest_index = index / a.hk;
                it.split = rest_index % a.splits;
                const AttnSeq s = attn_find(a, false, 2 * tpt, rest_index / a.splits);
                if (s.tile < 0) return false;
                it.q0 = s.q0;
                it.k0 = s.k0;
                it.lq = s.lq;
                it.lk = s.lk;
                it.first = s.tile * 2 * tpt;
                const int32_t left = s.lq - it.first;
                const int32_t all0 = (attn_seen(a, s, it.first + min(tpt, left) - 1) + kKeys - 1) / kKeys;
                const int32_t all1 =
                    left > tpt ? (attn_seen(a, s, it.first + min(2 * tpt, left) - 1) + kKeys - 1) / kKeys : 0;
                const int32_t per = (max(all0, all1) + a.splits - 1) / a.splits;
                it.j0 = it.split * per;
                it.n0 = max(0, min(per, all0 - it.j0));
                it.n1 = max(0, min(per, all1 - it.j0));
                return true;
            });
        } else if (warp == kWarpLoad) {
            // ------------------------------------------------------------ loads
            const uint32_t qbytes = static_cast<uint32_t>(tpt * a.group) * 128u * kAtoms;
            uint32_t issued = 0, qn[2] = {0, 0};
            bool ok = true;
            for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
                auto rows = [&](int t) {
                    if ((t ? it.n1 : it.n0) == 0) return true;
                    if (!warp_wait_bounded(q_empty(t), (qn[t] & 1u) ^ 1u, abort_flag, a.status, kSiteTmaEmpty))
                        return false;
                    mbar_arrive_expect_tx_elect(q_full(t), qbytes);
                    for (int at = 0; at < kAtoms; ++at)
                        tma_load_4d_elect(q_s + t * kTile + at * kAtomBytes, &mq, 64 * at, 0, it.kh,
                                          it.q0 + it.first + t * tpt, q_full(t));
                    ++qn[t];
                    return true;
                };
                const int32_t n = max(it.n0, it.n1);
                for (int32_t j = 0; j < n; ++j) {
                    const int32_t row = it.k0 + (it.j0 + j) * kKeys;
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t st = issued % S;
                        if (j == 0 && kv == 0 && !(ok = rows(0) && rows(1))) return false;
                        if (!(ok = warp_wait_bounded(empty(st), ((issued / S) & 1u) ^ 1u, abort_flag, a.status,
                                                     kSiteTmaEmpty)))
                            return false;
                        mbar_arrive_expect_tx_elect(full(st), kTile);
                        for (int at = 0; at < kAtoms; ++at)
                            tma_load_3d_elect(ring + st * kTile + at * kAtomBytes, kv ? &mv : &mk, 64 * at, it.kh, row,
                                              full(st));
                        ++issued;
                    }
                }
                return true;
            });
            if (!ok || *abort_flag) {  // the copies already issued land before the CTA exits
                volatile int never = 0;
                for (int t = 0; t < 2; ++t)
                    if (qn[t]) warp_wait_bounded(q_full(t), (qn[t] - 1) & 1u, &never, a.status, kSiteDrain, 200000000ull);
                for (uint32_t i = issued > S ? issued - S : 0; i < issued; ++i)
                    warp_wait_bounded(full(i % S), (i / S) & 1, &never, a.status, kSiteDrain, 200000000ull);
            }
        } else if (warp == kWarpIssue) {
            // ------------------------------------------------------------ MMAs
            // One thread. The tensor pipe holds a few products; what this thread does between two
            // groups of them has to be shorter than those take, so stages, phases, buffers and
            // descriptors advance by additions, and no other lane is waited for.
            if (elect_lane()) {
                const uint32_t fmt = kBf ? 1u : 0u;
                const uint32_t nd = static_cast<uint32_t>((a.D + 15) & ~15);
                const uint32_t id_s = make_idesc(fmt, 128u, kKeys), id_o = make_idesc(fmt, 128u, nd) | (1u << 16);
                const int ksteps = (a.D + 15) / 16;
                const uint64_t dq0 = desc_sw128(q_s, 16u, 1024u), dk0 = desc_sw128(ring, 16u, 1024u);
                const uint64_t dv0 = desc_sw128(ring, kAtomBytes, 1024u);
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    return mbar_wait_bounded(bar, parity, abort_flag, a.status, kSiteMmaFull);
                };
                uint32_t ks = 0, kp = 0, vs = 1, vp = 0;     // stage and phase of the next K and V
                auto next2 = [&](uint32_t& st, uint32_t& ph) {
                    st += 2;
                    if (st >= S) {
                        st -= S;
                        ph ^= 1u;
                    }
                };
                uint32_t sb = 0, pb = 0;                     // buffer of the next S and of the next P
                uint32_t si0 = 0, si1 = 0;                   // barrier of a row tile's next S
                uint32_t pi0 = 0, pi1 = 0, pp0 = 0, pp1 = 0; // barrier and phase of its next P
                uint32_t it0 = 0, it1 = 0, zeroed = 0;       // parities: items of a row tile, cleared tiles
                for_items_one(queue, abort_flag, a.status, [&](const AttnItem& it) {
                    const int32_t n0 = it.n0, n1 = it.n1, nmax = max(n0, n1);
                    if (nmax == 0) return true;
                    const bool solo = NB == 2 && (n0 == 0 || n1 == 0);
                    if (NB == 2) sb = pb = 0;
                    const bool partial = it.lk - (it.j0 + nmax - 1) * kKeys < kKeys;
                    // S of row tile T from the K in stage ks
                    auto scores = [&](auto T, bool last) {
                        constexpr int t = decltype(T)::value;
                        uint32_t& si = t ? si1 : si0;
                        const uint32_t d = s_col(NB == 3 || solo ? sb : t);
                        const uint64_t dq = dq0 + t * (kTile >> 4), dk = dk0 + ks * (kTile >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4 * kAtoms; ++kk) {
                            const uint32_t off = (static_cast<uint32_t>(kk >> 2) * kAtomBytes + 32u * (kk & 3)) >> 4;
                            if (kk < ksteps) mma_f16(d, dq + off, dk + off, id_s, kk > 0);
                        }
                        mma_commit(s_full0 + 24u * t + 8u * si);
                        if (last) mma_commit(q_empty(t));
                        si = si + 1 == NB ? 0 : si + 1;
                        sb = sb + 1 == NB ? 0 : sb + 1;
                    };
                    bool have = false;      // the K in stage ks has been waited for
                    bool clearing = false;  // V's rows past the last key are being cleared
                    auto key = [&] {
                        if (!have && !wait(full(ks), kp)) return false;
                        have = true;
                        tc_fence_after();
                        return true;
                    };
                    auto begin = [&](auto T) {
                        constexpr int t = decltype(T)::value;
                        const int32_t n = t ? n1 : n0;
                        if (n == 0) return true;
                        if (!key() || !wait(q_full(t), t ? it1 : it0)) return false;
                        tc_fence_after();
                        scores(T, n == 1);
                        return true;
                    };
                    // step j of row tile T: O += P V, and the next S
                    auto step = [&](auto T, int32_t j) {
                        constexpr int t = decltype(T)::value;
                        const int32_t n = t ? n1 : n0;
                        if (j >= n) return true;
                        const bool more = j + 1 < n;
                        // a free S buffer: the next S goes ahead of this step's sum
                        if (more && (NB == 3 || solo)) {
                            if (!key()) return false;
                            scores(T, j + 2 == n);
                        }
                        uint32_t& pi = t ? pi1 : pi0;
                        uint32_t& pp = t ? pp1 : pp0;
                        const uint32_t p = s_col(NB == 3 || solo ? pb : t);
                        const uint64_t dv = dv0 + vs * (kTile >> 4);
                        if (j == 0 && !wait(o_read(t), (t ? it1 : it0) ^ 1u)) return false;
                        if (clearing) {
                            if (!wait(cleared, zeroed)) return false;
                            zeroed ^= 1u;
                            clearing = false;
                        }
                        if (!wait(p_full0 + 24u * t + 8u * pi, pp)) return false;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            mma_f16_ts(o_col(t), p + 8u * kk, dv + 128u * kk, id_o, j > 0 || kk > 0);
                        mma_commit(o_done0 + 24u * t + 8u * pi);
                        if (++pi == NB) {
                            pi = 0;
                            pp ^= 1u;
                        }
                        pb = pb + 1 == NB ? 0 : pb + 1;
                        if (more && NB == 2 && !solo) {
                            if (!key()) return false;
                            scores(T, j + 2 == n);
                        }
                        return true;
                    };
                    if (!begin(Zero{}) || !begin(One{})) return false;
                    mma_commit(empty(ks));
                    next2(ks, kp);
                    for (int32_t j = 0; j < nmax; ++j) {
                        have = false;
                        if (!wait(full(vs), vp)) return false;
                        if (partial && j + 1 == nmax) {
                            mbar_arrive(to_clear);
                            clearing = true;
                        }
                        if (!step(Zero{}, j) || !step(One{}, j)) return false;
                        mma_commit(empty(vs));
                        next2(vs, vp);
                        if (j + 1 < nmax) {
                            mma_commit(empty(ks));
                            next2(ks, kp);
                        }
                    }
                    it0 ^= n0 > 0 ? 1u : 0u;
                    it1 ^= n1 > 0 ? 1u : 0u;
                    return true;
                });
                // every MMA issued has completed before tensor memory is released
                mma_commit(drain);
                volatile int never = 0;
                mbar_wait_bounded(drain, 0, &never, a.status, kSiteDrain, 200000000ull);
            }
            __syncwarp();
        } else if (warp == kWarpClear) {
            // ------------------------------------------------------------ values past the last key
            uint32_t e = 0, turn = 0;  // ring entries of earlier items; tiles cleared
            for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
                const int32_t nmax = max(it.n0, it.n1);
                if (nmax == 0) return true;
                const int32_t valid = it.lk - (it.j0 + nmax - 1) * kKeys;
                const uint32_t st = (e + 2u * nmax - 1u) % S;
                e += 2u * nmax;
                if (valid >= kKeys) return true;
                // the issuing thread has seen the tile arrive
                if (!warp_wait2(to_clear, 0u, turn, abort_flag, a.status, kSiteTmaEmpty, a.item_limit)) return false;
                turn ^= 1u;
                zero_rows(ring + st * kTile, kAtoms, kAtomBytes, valid, kKeys);
                if (lane == 0) mbar_arrive(cleared);
                return true;
            });
        }
    } else {
        setmaxnreg_inc<kRegsRow>();
        // ---------------------------------------------------------------- rows
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int tk = r / a.group, sub = r - tk * a.group;
        const float sc = fmaxf(fabsf(a.scale), 1e-30f) * kLog2e;
        const bool neg = a.scale < 0.0f;
        const uint32_t ocol = o_col(t) + lanes;
        uint32_t g = 0, done = 0;  // steps of earlier items; steps of this row tile so far
        for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
            const int32_t tokt = it.first + t * tpt;
            const int rows = max(0, min(tpt, it.lq - tokt)) * a.group;
            const bool live = r < rows;
            // keys seen from the share's first on; rows past the tile compute what is never stored
            int32_t seen = it.lk;
            if (a.causal) seen = min(max(tokt + tk + 1 + it.lk - it.lq, 0), it.lk);
            seen = (live ? seen : 0) - it.j0 * kKeys;
            const int32_t seen_all = __reduce_min_sync(0xffffffffu, live ? seen : 0x7fffffff);
            float m = -INFINITY, l = 0.0f;
            const int nt = t ? it.n1 : it.n0;
            for (int32_t j = 0; j < nt; ++j) {
                // an item of the other row tile alone may come before this one's first S
                if (!warp_wait2(s_full(t, done), 0u, (done / NB) & 1u, abort_flag, a.status, kSiteGatherEmpty,
                                a.item_limit))
                    return false;
                tc_fence_after();
                const uint32_t scol = s_col(score_buffer<kAtoms>(t, j, it.n0, it.n1, g)) + lanes;
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_async(scol + 32u * c, x[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_landed(x[c]);
                if (neg) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[c][i] ^= 0x80000000u;
                }
                if (seen_all < (j + 1) * kKeys) {
                    const int32_t left = seen - j * kKeys, left_all = seen_all - j * kKeys;  // of this tile's keys
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (left_all >= 32 * (c + 1)) continue;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i >= left) x[c][i] = 0xff800000u;  // -infinity
                    }
                }
                float best[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    best[c] = __uint_as_float(x[c][0]);
#pragma unroll
                    for (int i = 1; i < 31; i += 2)
                        best[c] = fmaxf(fmaxf(best[c], __uint_as_float(x[c][i])), __uint_as_float(x[c][i + 1]));
                    best[c] = fmaxf(best[c], __uint_as_float(x[c][31]));
                }
                const float top = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
                const bool grow = (top - m) * sc > kRescaleLog2;
                if (__any_sync(0xffffffffu, grow)) {
                    const float corr = grow ? attn_exp2((m - top) * sc) : 1.0f;
                    if (grow) m = top;
                    l *= corr;
                    if (j > 0) {
                        // the sum before this step has been added
                        if (!warp_wait2(o_done(t, done - 1u), 0u, ((done - 1u) / NB) & 1u, abort_flag, a.status,
                                        kSiteGatherEmpty))
                            return false;
                        tc_fence_after();
                        const uint64_t c2 = pack2(corr, corr);
#pragma unroll 1
                        for (int c = 0; c < 4 * kAtoms; ++c) {
                            float o[16];
                            uint32_t s[16];
                            tmem_ld16(ocol + 16u * c, o);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float u, w;
                                unpack2(mul2(pack2(o[i], o[i + 1]), c2), u, w);
                                s[i] = __float_as_uint(u);
                                s[i + 1] = __float_as_uint(w);
                            }
                            tmem_st16(ocol + 16u * c, s);
                        }
                    }
                }
                const float mm = m == -INFINITY ? 0.0f : m * sc;
                const uint64_t sc2 = pack2(sc, sc), m2 = pack2(-mm, -mm);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float u, w;
                        unpack2(fma2(pack2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), sc2, m2), u, w);
                        u = attn_exp2(u);
                        w = attn_exp2(w);
                        sum[i & 3] = add2(sum[i & 3], pack2(u, w));
                        p[i] = round2<kBf>(u, w);
                    }
                    tmem_st16(scol + 16u * c, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t, done));
                ++done;
                float u, w;
                unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), u, w);
                l += u + w;
            }
            // ------------------------------------------------------------ results
            const int64_t tok = it.q0 + tokt + tk;
            const int h = it.kh * a.group + sub;
            const bool any = nt > 0;
            if (any) {
                if (!warp_wait2(o_done(t, done - 1u), 0u, ((done - 1u) / NB) & 1u, abort_flag, a.status, kSiteEpilogue))
                    return false;
                tc_fence_after();
            }
            const bool some = any && l != 0.0f;  // the row saw a key
            const float inv = some ? 1.0f / l : 0.0f;
            const float lse = some ? fmaf(m, sc, log2f(l)) * kLn2 : -INFINITY;
            if (a.splits > 1) {
                float* po = a.part_out + ((static_cast<int64_t>(it.split) * a.tq + tok) * a.hq + h) * a.D;
                // rows lie a multiple of 32 bytes apart, so that all have the workspace's alignment: 16 at least
                const bool wide = (reinterpret_cast<uintptr_t>(a.part_out) & 31u) == 0;
#pragma unroll 1
                for (int c = 0; c < a.D; c += 16) {
                    float v[16];
                    __syncwarp();  // the stores part the lanes; the load needs the whole warp
                    if (any) tmem_ld16(ocol + static_cast<uint32_t>(c), v);
                    if (live) {
                        // whole sectors where they can be (head_dim is a multiple of 8)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = some ? v[i] * inv : 0.0f;
                        store8(po + c, v, wide);
                        if (c + 8 < a.D) store8(po + c + 8, v + 8, wide);
                    }
                }
                __syncwarp();
                if (live) a.part_lse[(static_cast<int64_t>(it.split) * a.hq + h) * a.tq + tok] = lse;
            } else {
                uint8_t* po = static_cast<uint8_t*>(a.out.p) + 2 * (tok * a.out.st + h * a.out.sh);
                const bool wide = (reinterpret_cast<uintptr_t>(po) & 31u) == 0;
#pragma unroll 1
                for (int c = 0; c < a.D; c += 16) {
                    float v[16];
                    __syncwarp();
                    if (any) tmem_ld16(ocol + static_cast<uint32_t>(c), v);
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = some ? v[i] * inv : 0.0f;
                        store16<kBf>(po + 2 * c, v, a.D - c, wide);
                    }
                }
                __syncwarp();
                if (live) a.lse[static_cast<int64_t>(h) * a.tq + tok] = lse;
            }
            if (any) {  // the next item's first product may overwrite O
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_read(t));
            }
            g += static_cast<uint32_t>(it.n0 + it.n1);
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

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    }();
    return fn;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, int dtype) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint32_t es[5] = {1u, 1u, 1u, 1u, 1u};
    const CUtensorMapDataType t = dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return enc(m, t, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Byte stride of an index as a tensor map takes it (that of an index of
// extent 1 is never used, but has to be a valid number).
cuuint64_t map_stride(int64_t elements) { return elements > 0 ? static_cast<cuuint64_t>(elements) * 2u : 16u; }

template <int kAtoms, bool kBf>
cudaError_t launch_forward(int dtype, const AttnArgs& a, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    if (!attn_encode_rows(&mq, a, a.q, dtype, kAttnTcRows / a.group) || !attn_encode_keys(&mk, a, a.k, dtype, kKeys) ||
        !attn_encode_keys(&mv, a, a.v, dtype, kKeys))
        return cudaErrorInvalidValue;
    auto kern = attn_forward_tc_kernel<kAtoms, kBf>;
    constexpr int smem = smem_of(kAtoms);
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = attn_allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(static_cast<unsigned>(a.tiles) * static_cast<unsigned>(a.splits) * static_cast<unsigned>(a.hk)),
                            kTcThreads, smem, st, mq, mk, mv, a);
}

}  // namespace

// Of a tensor without tokens nothing is loaded, but a map needs an address and
// an extent: those of the offsets, which are always there.
bool attn_encode_rows(CUtensorMap* m, const AttnArgs& a, const AttnTensor& t, int dtype, int tokens) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.group),
                                static_cast<cuuint64_t>(a.hk), static_cast<cuuint64_t>(a.tq > 0 ? a.tq : 1)};
    const void* base = a.tq > 0 ? t.p : a.q_starts;
    const cuuint64_t strides[3] = {map_stride(t.sh), map_stride(t.sh * a.group), map_stride(t.st)};
    const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(a.group), 1u, static_cast<cuuint32_t>(tokens)};
    return encode(m, base, 4, dims, strides, box, dtype);
}

bool attn_encode_keys(CUtensorMap* m, const AttnArgs& a, const AttnTensor& t, int dtype, int rows) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.hk),
                                static_cast<cuuint64_t>(a.tk > 0 ? a.tk : 1)};
    const void* base = a.tk > 0 ? t.p : a.k_starts;
    const cuuint64_t strides[2] = {map_stride(t.sh), map_stride(t.st)};
    const cuuint32_t box[3] = {64u, 1u, static_cast<cuuint32_t>(rows)};
    return encode(m, base, 3, dims, strides, box, dtype);
}

cudaError_t launch_attention_tc_forward(int dtype, const AttnArgs& args, cudaStream_t st) {
    AttnArgs a = args;
    a.item_limit = attn_item_limit(kWaitLimitCycles, a.tk / kKeys + 1);
    if (a.D <= 64)
        return dtype == kBF16 ? launch_forward<1, true>(dtype, a, st) : launch_forward<1, false>(dtype, a, st);
    return dtype == kBF16 ? launch_forward<2, true>(dtype, a, st) : launch_forward<2, false>(dtype, a, st);
}

}  // namespace mdcn
