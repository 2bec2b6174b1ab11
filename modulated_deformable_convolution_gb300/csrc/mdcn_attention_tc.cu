// Attention over packed sequences on the tensor cores (float16, bfloat16):
// the forward.
//
// A CTA takes two row tiles of 128 rows (row = token and query head of one key
// head) and runs over the key tiles of 128 keys that they see:
//   S = Q K^T (fp32, tensor memory), P = exp2(scale' S - m) rounded to the
//   type of v, written over S in tensor memory, O += P V (fp32, tensor memory).
// Warps 0-3 and 4-7 hold one row per thread of the first and second tile (a
// tensor-memory lane each, so row maxima and sums need no exchange), warp 8
// loads tiles by TMA into a ring, warp 9 issues the MMAs: the products of one
// tile run while the other tile's probabilities are computed. O is rescaled
// only when a row's maximum has grown by more than 2^8 since it was last
// taken (P then stays below 2^8, exact in the sums: the result does not
// depend on which maximum is used beyond rounding); by the row's own warp,
// which knows the previous O += P V finished because the S it waits for was
// issued after it.
//
// Bound by the tensor cores for long rows: per key tile and row tile two
// 128 x 128 x D products, 4 * 128 * 128 * D operations; next by the exponentials.
// Shared memory: Q once, K and V in a ring of 128-row tiles, 227 KB in all.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "mdcn_attention_tc.cuh"
#include "mdcn_plan.h"

namespace mdcn {

namespace {

constexpr int kTcThreads = 384;
constexpr int kWarpLoad = 8, kWarpIssue = 9, kWarpServe = 10;
constexpr int kRegsRow = 216, kRegsCtl = 72;  // of 168 a thread at launch
static_assert(2 * kRegsRow + kRegsCtl <= 3 * 168, "register split must fit the launch's");
constexpr int kKeys = 128;
constexpr float kRescaleLog2 = 8.0f;

// Stages of the ring: as many 128-row tiles as fit beside Q.
__host__ __device__ constexpr int stages_of(int atoms) { return atoms == 2 ? 5 : 8; }
__host__ __device__ constexpr int smem_of(int atoms) {
    return 1024 + (2 + stages_of(atoms)) * atoms * static_cast<int>(kAtomBytes) + 512;
}

// kAtoms: 64-element atoms of a head (head_dim <= 64: 1, else 2).
template <int kAtoms, bool kBf>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_forward_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnArgs a) {
    constexpr uint32_t S = stages_of(kAtoms);
    constexpr uint32_t kTile = kAtoms * kAtomBytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t q_s = base, ring = base + 2 * kTile;
    const ItemQueue queue{ring + S * kTile};
    const uint32_t bars = queue.base + ItemQueue::kBytes;
    auto full = [&](uint32_t s) { return bars + 8u * s; };
    auto empty = [&](uint32_t s) { return bars + 8u * (S + s); };
    const uint32_t rest = bars + 16u * S;
    auto s_full = [&](int t) { return rest + 8u * t; };
    auto p_full = [&](int t) { return rest + 16u + 8u * t; };
    auto o_full = [&](int t) { return rest + 32u + 8u * t; };
    auto o_read = [&](int t) { return rest + 48u + 8u * t; };
    auto q_full = [&](int t) { return rest + 64u + 8u * t; };
    auto q_empty = [&](int t) { return rest + 80u + 8u * t; };
    const uint32_t drain = rest + 96u;
    const uint32_t slot_off = rest + 104u - raw;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + slot_off);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + slot_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    if (warp == kWarpLoad && lane == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t), 4);
            mbar_init(o_full(t), 1);
            mbar_init(o_read(t), 4);
            mbar_init(q_full(t), 1);
            mbar_init(q_empty(t), 1);
        }
        mbar_init(drain, 1);
        queue.init(10);
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
    // tensor memory: S of tile 0 and 1 (128 columns each, P over the first 64), O of tile 0 and 1
    auto s_col = [&](int t) { return tmem + 128u * t; };
    auto o_col = [&](int t) { return tmem + 256u + 64u * kAtoms * t; };
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
            const uint32_t fmt = kBf ? 1u : 0u;
            const uint32_t nd = static_cast<uint32_t>((a.D + 15) & ~15);
            const uint32_t id_s = make_idesc(fmt, 128u, kKeys), id_o = make_idesc(fmt, 128u, nd) | (1u << 16);
            const int ksteps = (a.D + 15) / 16;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return warp_wait2(bar, 0u, parity, abort_flag, a.status, kSiteMmaFull);
            };
            uint32_t e = 0;                          // ring entries used up by earlier items
            uint32_t items[2] = {0, 0}, ps[2] = {0, 0};  // items and probability tiles of each row tile so far
            for_items(queue, abort_flag, a.status, [&](const AttnItem& it) {
                const int32_t nmax = max(it.n0, it.n1);
                if (nmax == 0) return true;
                const int32_t n[2] = {it.n0, it.n1};
                // S of row tile t and key tile j
                auto scores = [&](int t, uint32_t k_s, int32_t j) {
                    for (int kk = 0; kk < ksteps; ++kk) {
                        const uint32_t off = static_cast<uint32_t>(kk >> 2) * kAtomBytes + 32u * (kk & 3);
                        mma_f16_elect(s_col(t), desc_sw128(q_s + t * kTile + off, 16u, 1024u),
                                      desc_sw128(k_s + off, 16u, 1024u), id_s, kk > 0);
                    }
                    mma_commit_elect(s_full(t));
                    if (j + 1 == n[t]) mma_commit_elect(q_empty(t));
                };
                if (!wait(full(e % S), (e / S) & 1u)) return false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (n[t] == 0) continue;
                    if (!wait(q_full(t), items[t] & 1u)) return false;
                    tc_fence_after();
                    scores(t, ring + (e % S) * kTile, 0);
                }
                mma_commit_elect(empty(e % S));
                for (int32_t j = 0; j < nmax; ++j) {
                    const uint32_t ev = e + 2 * j + 1, ek = ev + 1;  // V_j, K_{j+1}
                    const uint32_t sv = ev % S, sk = ek % S;
                    const uint32_t v_s = ring + sv * kTile;
                    if (!wait(full(sv), (ev / S) & 1u)) return false;
                    const int32_t valid = it.lk - (it.j0 + j) * kKeys;
                    if (valid < kKeys) zero_rows(v_s, kAtoms, kAtomBytes, valid, kKeys);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j >= n[t]) continue;
                        if (j == 0 && !wait(o_read(t), (items[t] & 1u) ^ 1u)) return false;
                        if (!wait(p_full(t), ps[t] & 1u)) return false;
                        ++ps[t];
                        tc_fence_after();
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            mma_f16_ts_elect(o_col(t), s_col(t) + 8u * kk,
                                             desc_sw128(v_s + 2048u * kk, kAtomBytes, 1024u), id_o, j > 0 || kk > 0);
                        if (j + 1 < n[t]) {
                            if (!wait(full(sk), (ek / S) & 1u)) return false;
                            tc_fence_after();
                            scores(t, ring + sk * kTile, j + 1);
                        } else {
                            mma_commit_elect(o_full(t));
                        }
                    }
                    mma_commit_elect(empty(sv));
                    if (j + 1 < nmax) mma_commit_elect(empty(sk));
                }
                e += 2 * nmax;
#pragma unroll
                for (int t = 0; t < 2; ++t) items[t] += n[t] > 0 ? 1u : 0u;
                return true;
            });
            // every MMA issued has completed before tensor memory is released
            mma_commit_elect(drain);
            volatile int never = 0;
            warp_wait2(drain, 0u, 0, &never, a.status, kSiteDrain, 200000000ull);
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
        const uint32_t scol = s_col(t) + lanes, ocol = o_col(t) + lanes;
        uint32_t ss = 0, items = 0;  // score tiles and items of this row tile so far
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
                if (!warp_wait2(s_full(t), 0u, ss & 1u, abort_flag, a.status, kSiteGatherEmpty)) return false;
                ++ss;
                tc_fence_after();
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
                    const int32_t left = seen - j * kKeys;  // of this tile's keys
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i >= left) x[c][i] = 0xff800000u;  // -infinity
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
                        const uint64_t c2 = pack2(corr, corr);
#pragma unroll 1
                        for (int c = 0; c < 2 * kAtoms; ++c) {
                            uint32_t o[32];
                            tmem_ld32_async(ocol + 32u * c, o);
                            tmem_wait_ld();
                            tmem_landed(o);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                float u, w;
                                unpack2(mul2(pack2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), c2), u, w);
                                o[i] = __float_as_uint(u);
                                o[i + 1] = __float_as_uint(w);
                            }
                            tmem_st32(ocol + 32u * c, o);
                        }
                    }
                }
                const float mm = m == -INFINITY ? 0.0f : m * sc;
                const uint64_t sc2 = pack2(sc, sc), m2 = pack2(-mm, -mm);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int c = 2 * h + i / 16, o = 2 * (i % 16);
                        float u, w;
                        unpack2(fma2(pack2(__uint_as_float(x[c][o]), __uint_as_float(x[c][o + 1])), sc2, m2), u, w);
                        u = attn_exp2(u);
                        w = attn_exp2(w);
                        sum[i & 3] = add2(sum[i & 3], pack2(u, w));
                        p[i] = round2<kBf>(u, w);
                    }
                    tmem_st32(scol + 32u * h, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t));
                float u, w;
                unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), u, w);
                l += u + w;
            }
            // ------------------------------------------------------------ results
            const int64_t tok = it.q0 + tokt + tk;
            const int h = it.kh * a.group + sub;
            const bool any = nt > 0;
            if (any) {
                if (!warp_wait2(o_full(t), 0u, items & 1u, abort_flag, a.status, kSiteEpilogue)) return false;
                ++items;
                tc_fence_after();
            }
            const bool some = any && l != 0.0f;  // the row saw a key
            const float inv = some ? 1.0f / l : 0.0f;
            const float lse = some ? fmaf(m, sc, log2f(l)) * kLn2 : -INFINITY;
            if (a.splits > 1) {
                float* po = a.part_out + ((static_cast<int64_t>(it.split) * a.tq + tok) * a.hq + h) * a.D;
#pragma unroll 1
                for (int c = 0; c < a.D; c += 16) {
                    float v[16];
                    if (any) tmem_ld16(ocol + static_cast<uint32_t>(c), v);
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        if (c + i < a.D)
                            *reinterpret_cast<float4*>(po + c + i) =
                                some ? make_float4(v[i] * inv, v[i + 1] * inv, v[i + 2] * inv, v[i + 3] * inv)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (live) a.part_lse[(static_cast<int64_t>(it.split) * a.hq + h) * a.tq + tok] = lse;
            } else {
                uint8_t* po = static_cast<uint8_t*>(a.out.p) + 2 * (tok * a.out.st + h * a.out.sh);
                const bool wide = (reinterpret_cast<uintptr_t>(po) & 31u) == 0;
#pragma unroll 1
                for (int c = 0; c < a.D; c += 16) {
                    float v[16];
                    if (any) tmem_ld16(ocol + static_cast<uint32_t>(c), v);
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = some ? v[i] * inv : 0.0f;
                    store16<kBf>(po + 2 * c, v, a.D - c, wide);
                }
                if (live) a.lse[static_cast<int64_t>(h) * a.tq + tok] = lse;
            }
            if (any) {  // the next item's first product may overwrite O
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_read(t));
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(a.tiles) * static_cast<unsigned>(a.splits) * static_cast<unsigned>(a.hk), kTcThreads,
           smem, st>>>(mq, mk, mv, a);
    return cudaGetLastError();
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

cudaError_t launch_attention_tc_forward(int dtype, const AttnArgs& a, cudaStream_t st) {
    if (a.D <= 64)
        return dtype == kBF16 ? launch_forward<1, true>(dtype, a, st) : launch_forward<1, false>(dtype, a, st);
    return dtype == kBF16 ? launch_forward<2, true>(dtype, a, st) : launch_forward<2, false>(dtype, a, st);
}

}  // namespace mdcn
