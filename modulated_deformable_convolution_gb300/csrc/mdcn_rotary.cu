// Rotary positions over several axes, with the norms of queries and keys in
// the same pass, and the gradient of both.
//
// Forward, for each head x of each token (D elements):
//   n = x * rsqrt(mean(x^2) + eps) * w,  y[lo] = n[lo] c - n[hi] s,
//   y[hi] = n[hi] c + n[lo] s, with (c, s) = cos, sin of position * frequency.
// Backward, g = the output's gradient rotated by the opposite angle:
//   gw = sum g * n0,  gx = r * (g w - n0 mean(g w n0)),  n0 = x r.
//
// Both move each element once in and once out (the backward reads two) and do
// a few operations on it: bound by device memory. So a row is 16 or 32 bytes
// per lane, D / 8 lanes per row, and several rows are in flight per warp. A
// warp takes all heads of a token (or a share of them, when tokens are few),
// because the cosines and sines depend on the token alone: it computes each
// pair's once, into shared memory, and each lane keeps those of its own 8
// elements in registers for all of the token's heads. The partner of an
// element lies in the same lane for neighbouring pairs; otherwise the row goes
// through the warp's shared memory (any distance, so odd sections cost the
// same as even ones).
//
// Angles: position * frequency is taken in turns as an exact product (two
// fp32 words), its whole turns are dropped, and only then is it rounded, so
// the error stays 2^-24 of a turn at positions where a rounded product would
// be off by more than a 16-bit unit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "mdcn_plan.h"
#include "mdcn_rotary.h"

namespace mdcn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxD = 256;
constexpr int kE = 8;  // elements of a row per lane

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

template <typename T>
struct Pack {
    static constexpr int kV = static_cast<int>(kE * sizeof(T) / 16);
    union {
        uint4 v[kV];
        T e[kE];
    };
    __device__ Pack() {}
    __device__ __forceinline__ void load(const T* p, bool vec) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < kV; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < kE; ++i) e[i] = p[i];
        }
    }
    __device__ __forceinline__ void store(T* p, bool vec) const {
        if (vec) {
#pragma unroll
            for (int i = 0; i < kV; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < kE; ++i) p[i] = e[i];
        }
    }
};

// cos and sin of position * frequency.
__device__ __forceinline__ void pair_turn(int32_t pos, float freq, float& c, float& s) {
    constexpr float kHi = 0.15915494309189535f;                                        // 1 / (2 pi), rounded
    constexpr float kLo = static_cast<float>(0.15915494309189533577 - static_cast<double>(kHi));  // what is left
    const float hi = freq * kHi;
    const float lo = fmaf(freq, kHi, -hi) + freq * kLo;
    // the position in two parts that fp32 holds exactly
    const float pb = static_cast<float>(pos & 4095), pa = static_cast<float>(pos - (pos & 4095));
    float ta = pa * hi, tb = pb * hi;
    float ea = fmaf(pa, hi, -ta), eb = fmaf(pb, hi, -tb);
    ta -= rintf(ta);
    tb -= rintf(tb);
    ea -= rintf(ea);
    const float rest = (pa + pb) * lo;
    float t = (ta + tb) + ((ea + eb) + (rest - rintf(rest)));
    t -= rintf(t);
    sincospif(2.0f * t, &s, &c);
}

// Element e of a head: its pair (or -1 past the rotated part), its partner,
// and the sign of its sine term in the forward.
__device__ __forceinline__ int pair_of(const RotaryArgs& a, int e, int& partner, float& sign) {
    partner = e;
    sign = 0.0f;
    if (e >= 2 * a.pairs) return -1;
    int p, d;
    bool low;
    if (a.layout == 1) {
        p = e >> 1;
        d = 1;
        low = (e & 1) == 0;
    } else if (a.layout == 0) {
        d = a.pairs;
        low = e < d;
        p = low ? e : e - d;
    } else {
        int first = 0, ax = 0;
        while (ax < 3 && e >= 2 * a.sec_end[ax]) first = a.sec_end[ax++];
        d = a.sec_end[ax] - first;
        const int r = e - 2 * first;
        low = r < d;
        p = first + (low ? r : r - d);
    }
    partner = low ? e + d : e - d;
    sign = low ? -1.0f : 1.0f;
    return p;
}

// Sum over the lanes that share a row.
__device__ __forceinline__ float row_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp's shared memory: a token's (cos, sin) and one row per lane group.
struct alignas(16) WarpSmem {
    float cs[kMaxD];         // (cos, sin) of each pair
    float row[32 * kE];
};

// What a lane keeps for its 8 elements: where each partner's value lies in
// the warp's row buffer (4 x 16 bits would do; kept as shorts).
struct LaneMap {
    int16_t pair[kE];
    int16_t partner[kE];
    float sign[kE];
};

template <bool kNeighbour>
__device__ __forceinline__ void rotate(float (&n)[kE], const float (&c)[kE], const float (&s)[kE], const LaneMap& m,
                                       float* row, int lane) {
    if constexpr (kNeighbour) {
#pragma unroll
        for (int i = 0; i < kE; i += 2) {
            const float a = n[i], b = n[i + 1];
            n[i] = fmaf(a, c[i], b * s[i]);
            n[i + 1] = fmaf(b, c[i + 1], a * s[i + 1]);
        }
    } else {
        __syncwarp();
        float4* mine = reinterpret_cast<float4*>(row + lane * kE);
        mine[0] = make_float4(n[0], n[1], n[2], n[3]);
        mine[1] = make_float4(n[4], n[5], n[6], n[7]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kE; ++i) n[i] = fmaf(n[i], c[i], row[m.partner[i]] * s[i]);
    }
}

// Lane set-up shared by both directions.
struct LaneSetup {
    int lane, sub, row_in_warp, rows_per_warp, e0;
    bool on;
    LaneMap m;
    __device__ __forceinline__ LaneSetup(const RotaryArgs& a) {
        lane = threadIdx.x & 31;
        sub = lane & (a.lanes - 1);
        rows_per_warp = 32 / a.lanes;
        row_in_warp = lane / a.lanes;
        e0 = sub * kE;
        on = e0 < a.D;
        const int base = row_in_warp * a.lanes * kE;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            int partner = e0 + i;
            float sg = 0.0f;
            m.pair[i] = static_cast<int16_t>(on ? pair_of(a, e0 + i, partner, sg) : -1);
            m.partner[i] = static_cast<int16_t>(base + partner);
            m.sign[i] = sg;
        }
    }
    // The token's cosines and signed sines of this lane's elements.
    __device__ __forceinline__ void turns(const RotaryArgs& a, int token, WarpSmem& w, float direction, float (&c)[kE],
                                          float (&s)[kE]) const {
        __syncwarp();
        for (int p = lane; p < a.pairs; p += 32) {
            int ax = 0;
            while (ax < 3 && p >= a.sec_end[ax]) ++ax;
            float cp, sp;
            pair_turn(__ldg(a.pos + static_cast<int64_t>(token) * a.axes + ax), __ldg(a.freq + p), cp, sp);
            *reinterpret_cast<float2*>(&w.cs[2 * p]) = make_float2(cp, sp);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            c[i] = 1.0f;
            s[i] = 0.0f;
            if (m.pair[i] >= 0) {
                const float2 v = *reinterpret_cast<const float2*>(&w.cs[2 * m.pair[i]]);
                c[i] = v.x;
                s[i] = v.y * m.sign[i] * direction;
            }
        }
    }
};

template <typename T, bool kNeighbour>
__global__ void __launch_bounds__(kThreads) rotary_forward_kernel(const __grid_constant__ RotaryArgs a) {
    __shared__ WarpSmem smem[kWarps];
    WarpSmem& w = smem[threadIdx.x >> 5];
    const LaneSetup L(a);
    const bool vec = a.vec != 0;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    float wt[2][kE];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kE; ++i)
            wt[t][i] = (L.on && a.w[t]) ? to_f(static_cast<const T*>(a.w[t])[L.e0 + i]) : 1.0f;

    const int64_t units = static_cast<int64_t>(a.tokens) * a.parts;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
    // rows of a token per unit, whole warps' worth
    const int share = ((a.rows + a.parts * L.rows_per_warp - 1) / (a.parts * L.rows_per_warp)) * L.rows_per_warp;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units; u += stride) {
        const int token = static_cast<int>(u / a.parts), part = static_cast<int>(u % a.parts);
        const int r0 = part * share, r1 = min(r0 + share, a.rows);
        if (r0 >= r1) continue;
        auto addr = [&](const RotaryTensor* t, int r) {
            const int i = r >= a.hq ? 1 : 0;
            const int h = i ? r - a.hq : r;
            return static_cast<T*>(t[i].p) + static_cast<int64_t>(token) * t[i].st + static_cast<int64_t>(h) * t[i].sh +
                   L.e0;
        };
        // the next rows' loads are in flight while a row is worked on
        constexpr int kAhead = 4;
        Pack<T> buf[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k * L.rows_per_warp + L.row_in_warp;
            if (L.on && r < r1) buf[k].load(addr(a.x, r), vec);
        }
        float c[kE], s[kE];
        L.turns(a, token, w, 1.0f, c, s);
        for (int rb = r0; rb < r1; rb += kAhead * L.rows_per_warp) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int base = rb + k * L.rows_per_warp;
                if (base >= r1) break;
                const int r = base + L.row_in_warp;
                const bool live = L.on && r < r1;
                float n[kE];
#pragma unroll
                for (int i = 0; i < kE; ++i) n[i] = live ? to_f(buf[k].e[i]) : 0.0f;
                const int rn = r + kAhead * L.rows_per_warp;
                if (L.on && rn < r1) buf[k].load(addr(a.x, rn), vec);
                if (a.norm) {
                    float ss = 0.0f;
#pragma unroll
                    for (int i = 0; i < kE; ++i) ss = fmaf(n[i], n[i], ss);
                    ss = row_sum(ss, a.lanes);
                    const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
                    const int t = r >= a.hq ? 1 : 0;
#pragma unroll
                    for (int i = 0; i < kE; ++i) n[i] *= inv * (t ? wt[1][i] : wt[0][i]);
                }
                rotate<kNeighbour>(n, c, s, L.m, w.row, L.lane);
                if (live) {
                    Pack<T> o;
#pragma unroll
                    for (int i = 0; i < kE; ++i) o.e[i] = from_f<T>(n[i]);
                    o.store(addr(a.y, r), vec);
                }
            }
        }
    }
}

template <typename T, bool kNeighbour>
__global__ void __launch_bounds__(kThreads) rotary_backward_kernel(const __grid_constant__ RotaryArgs a) {
    __shared__ WarpSmem smem[kWarps];
    WarpSmem& w = smem[threadIdx.x >> 5];
    const LaneSetup L(a);
    const bool vec = a.vec != 0;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    float wt[2][kE], gw[2][kE];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            wt[t][i] = (L.on && a.w[t]) ? to_f(static_cast<const T*>(a.w[t])[L.e0 + i]) : 1.0f;
            gw[t][i] = 0.0f;
        }

    const int64_t units = static_cast<int64_t>(a.tokens) * a.parts;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
    const int share = ((a.rows + a.parts * L.rows_per_warp - 1) / (a.parts * L.rows_per_warp)) * L.rows_per_warp;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units; u += stride) {
        const int token = static_cast<int>(u / a.parts), part = static_cast<int>(u % a.parts);
        const int r0 = part * share, r1 = min(r0 + share, a.rows);
        if (r0 >= r1) continue;
        auto addr = [&](const RotaryTensor* t, int r) {
            const int i = r >= a.hq ? 1 : 0;
            const int h = i ? r - a.hq : r;
            return static_cast<T*>(t[i].p) + static_cast<int64_t>(token) * t[i].st + static_cast<int64_t>(h) * t[i].sh +
                   L.e0;
        };
        constexpr int kAhead = 2;
        Pack<T> gb[kAhead], xb[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k * L.rows_per_warp + L.row_in_warp;
            if (L.on && r < r1) {
                gb[k].load(addr(a.y, r), vec);
                if (a.norm) xb[k].load(addr(a.x, r), vec);
            }
        }
        float c[kE], s[kE];
        L.turns(a, token, w, -1.0f, c, s);
        for (int rb = r0; rb < r1; rb += kAhead * L.rows_per_warp) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int base = rb + k * L.rows_per_warp;
                if (base >= r1) break;
                const int r = base + L.row_in_warp;
                const bool live = L.on && r < r1;
                float g[kE], x[kE];
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    g[i] = live ? to_f(gb[k].e[i]) : 0.0f;
                    x[i] = (live && a.norm) ? to_f(xb[k].e[i]) : 0.0f;
                }
                const int rn = r + kAhead * L.rows_per_warp;
                if (L.on && rn < r1) {
                    gb[k].load(addr(a.y, rn), vec);
                    if (a.norm) xb[k].load(addr(a.x, rn), vec);
                }
                rotate<kNeighbour>(g, c, s, L.m, w.row, L.lane);
                if (a.norm) {
                    const int t = r >= a.hq ? 1 : 0;
                    float ss = 0.0f, dot = 0.0f;
#pragma unroll
                    for (int i = 0; i < kE; ++i) {
                        ss = fmaf(x[i], x[i], ss);
                        dot = fmaf(g[i] * (t ? wt[1][i] : wt[0][i]), x[i], dot);
                    }
                    ss = row_sum(ss, a.lanes);
                    dot = row_sum(dot, a.lanes);
                    const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
                    const float mean = dot * inv * inv_d;  // mean(g w n)
#pragma unroll
                    for (int i = 0; i < kE; ++i) {
                        const float n = x[i] * inv;
                        gw[0][i] += t ? 0.0f : g[i] * n;
                        gw[1][i] += t ? g[i] * n : 0.0f;
                        g[i] = inv * fmaf(-n, mean, g[i] * (t ? wt[1][i] : wt[0][i]));
                    }
                }
                if (live) {
                    Pack<T> o;
#pragma unroll
                    for (int i = 0; i < kE; ++i) o.e[i] = from_f<T>(g[i]);
                    o.store(addr(a.g, r), vec);
                }
            }
        }
    }
    if (!a.part) return;
    // the block's partial sums, warps and row groups added in order
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kE; ++i) w.row[L.lane * kE + i] = t ? gw[1][i] : gw[0][i];
        __syncthreads();
        for (int e = threadIdx.x; e < a.D; e += kThreads) {
            float sum = 0.0f;
            for (int v = 0; v < kWarps; ++v)
                for (int r = 0; r < L.rows_per_warp; ++r) sum += smem[v].row[r * a.lanes * kE + e];
            a.part[(static_cast<int64_t>(blockIdx.x) * 2 + t) * a.D + e] = sum;
        }
        __syncthreads();
    }
}

// The weights' gradients: the blocks' partial sums added in a fixed order, 32
// lanes to an element. Grid: (head_dim / 8, 2).
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_weight_sum_kernel(const float* part, int blocks, int D, T* gq, T* gk) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    T* g = blockIdx.y ? gk : gq;
    if (!g) return;
    // 8 neighbouring elements x 32 slices of the blocks
    __shared__ float sums[32][9];
    const int e = threadIdx.x & 7, slice = threadIdx.x >> 3;
    float v = 0.0f;
    for (int b = slice; b < blocks; b += 32) v += part[(static_cast<int64_t>(b) * 2 + blockIdx.y) * D + blockIdx.x * 8 + e];
    sums[slice][e] = v;
    __syncthreads();
    if (threadIdx.x < 8) {
        float t = 0.0f;
        for (int k = 0; k < 32; ++k) t += sums[k][threadIdx.x];
        g[blockIdx.x * 8 + threadIdx.x] = from_f<T>(t);
    }
}

// Lanes per row, and how many warps share a token's rows: one where tokens
// alone fill the GPU (the token's cosines are then computed once), more where
// they are few.
void plan_lanes(RotaryArgs* a, int sms) {
    a->lanes = 1;
    while (a->lanes * kE < a->D) a->lanes *= 2;
    const int rpw = 32 / a->lanes;
    const int most = (a->rows + rpw - 1) / rpw;
    const int64_t want = static_cast<int64_t>(sms) * 24;  // warps that keep the loads in flight
    int64_t parts = (want + a->tokens - 1) / a->tokens;
    a->parts = static_cast<int32_t>(parts < most ? parts : most);
}

int64_t blocks_for(const RotaryArgs& a) {
    return (static_cast<int64_t>(a.tokens) * a.parts + kWarps - 1) / kWarps;
}

template <typename T>
cudaError_t forward_t(const RotaryArgs& a, int64_t grid, cudaStream_t st) {
    if (a.layout == 1)
        rotary_forward_kernel<T, true><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
    else
        rotary_forward_kernel<T, false><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_t(const RotaryArgs& a, int64_t grid, void* gqw, void* gkw, cudaStream_t st) {
    if (a.layout == 1)
        rotary_backward_kernel<T, true><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
    else
        rotary_backward_kernel<T, false><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.D / 8), 2);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, rotary_weight_sum_kernel<T>, static_cast<const float*>(a.part),
                           static_cast<int>(grid), static_cast<int>(a.D), static_cast<T*>(gqw), static_cast<T*>(gkw));
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_rotary_forward(int dtype, RotaryArgs a, int sms, cudaStream_t st) {
    plan_lanes(&a, sms);
    int64_t grid = blocks_for(a);
    if (grid > static_cast<int64_t>(sms) * 16) grid = static_cast<int64_t>(sms) * 16;
    if (dtype == kF32) return forward_t<float>(a, grid, st);
    if (dtype == kF16) return forward_t<__half>(a, grid, st);
    return forward_t<__nv_bfloat16>(a, grid, st);
}

cudaError_t launch_rotary_backward(int dtype, RotaryArgs a, void* gqw, void* gkw, int sms, cudaStream_t st) {
    plan_lanes(&a, sms);
    int64_t grid = blocks_for(a);
    if (grid > kRotaryMaxBlocks) grid = kRotaryMaxBlocks;
    if (dtype == kF32) return backward_t<float>(a, grid, gqw, gkw, st);
    if (dtype == kF16) return backward_t<__half>(a, grid, gqw, gkw, st);
    return backward_t<__nv_bfloat16>(a, grid, gqw, gkw, st);
}

}  // namespace mdcn
