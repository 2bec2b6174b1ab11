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
// per lane, D / 8 lanes per row, several rows in flight per warp, and the
// arithmetic is kept short: two values per instruction, weights folded into
// the cosines and sines, the norm's factor applied last. A warp takes all heads
// of a token (or a share of them, when tokens are few), because the cosines
// and sines depend on the token alone: it computes each pair's once, into
// shared memory, and each lane keeps those of its own 8 elements in registers
// for all of the token's heads. The partner of an element lies in the same lane
// for neighbouring pairs; otherwise the lane loads the partners' values too, of
// the row that the warp is loading anyway (first-level cache): as a vector where
// they are 8 neighbours on a multiple of 8, else one by one.
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

// Two fp32 values in one register pair: one instruction works on both.
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t swap2(uint64_t v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(hi, lo);
}
__device__ __forceinline__ float sum2(uint64_t v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return lo + hi;
}

// 8 elements of a row.
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
    __device__ __forceinline__ void widen(uint64_t (&x)[kE / 2]) const {
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) x[i] = pack2(to_f(e[2 * i]), to_f(e[2 * i + 1]));
    }
    __device__ __forceinline__ void round(const uint64_t (&x)[kE / 2]) {
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
            float lo, hi;
            unpack2(x[i], lo, hi);
            e[2 * i] = from_f<T>(lo);
            e[2 * i + 1] = from_f<T>(hi);
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

// One warp's shared memory: a token's (cos, sin) of each pair.
struct alignas(16) WarpSmem {
    float cs[kMaxD];
};

// A lane's place in its row: 8 elements from e0 on, and where their partners
// lie.
struct LaneSetup {
    int lane, rows_per_warp, row_in_warp, e0;
    bool on;               // the lane has elements
    bool run;              // its 8 partners are 8 neighbouring elements that start on a multiple of 8
    uint32_t code[kE / 2]; // two elements each: partner, 8 bits; pair, 7 bits; rotated, 1 bit
    __device__ __forceinline__ LaneSetup(const RotaryArgs& a) {
        lane = threadIdx.x & 31;
        const int sub = lane & (a.lanes - 1);
        rows_per_warp = 32 / a.lanes;
        row_in_warp = lane / a.lanes;
        e0 = sub * kE;
        on = e0 < a.D;
        run = true;
        int first = 0;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            int to = e0 + i;
            float sg = 0.0f;
            const int p = on ? pair_of(a, e0 + i, to, sg) : -1;
            if (i == 0) first = to;
            run = run && to == first + i;
            const uint32_t v = static_cast<uint32_t>(to) | (p >= 0 ? (static_cast<uint32_t>(p) << 8 | 0x8000u) : 0u);
            code[i / 2] = i & 1 ? code[i / 2] | v << 16 : v;
        }
        run = run && (first & 7) == 0;
        // one path for the warp: narrow partner loads wherever one lane needs them
        run = __all_sync(0xffffffffu, run || !on) != 0;
    }
    __device__ __forceinline__ uint32_t entry(int i) const { return code[i / 2] >> (16 * (i & 1)); }
    __device__ __forceinline__ int partner(int i) const { return static_cast<int>(entry(i) & 0xffu); }
    // The partners of the lane's elements, from the row that starts at `row`.
    template <typename T>
    __device__ __forceinline__ void load_partners(Pack<T>& p, const T* row, bool vec) const {
        if (run) {
            p.load(row + partner(0), vec);
        } else {
#pragma unroll
            for (int i = 0; i < kE; ++i) p.e[i] = row[partner(i)];
        }
    }
    // The cosine of each of the token's pairs, and its sine, into the warp's shared memory.
    __device__ __forceinline__ void turn_pairs(const RotaryArgs& a, int token, WarpSmem& w) const {
        __syncwarp();
        for (int p = lane; p < a.pairs; p += 32) {
            int ax = 0;
            while (ax < 3 && p >= a.sec_end[ax]) ++ax;
            float cp, sp;
            pair_turn(__ldg(a.pos + static_cast<int64_t>(token) * a.axes + ax), __ldg(a.freq + p), cp, sp);
            *reinterpret_cast<float2*>(&w.cs[2 * p]) = make_float2(cp, sp);
        }
        __syncwarp();
    }
    // Of this lane's element i: the cosine, and the sine with the sign that it
    // has in the forward (first of its pair: minus) times `direction`.
    __device__ __forceinline__ void turn_of(const WarpSmem& w, int i, float direction, float& c, float& s) const {
        const uint32_t v = entry(i);
        c = 1.0f;
        s = 0.0f;
        if (v & 0x8000u) {
            const float2 t = *reinterpret_cast<const float2*>(&w.cs[2 * ((v >> 8) & 0x7fu)]);
            c = t.x;
            s = static_cast<int>(v & 0xffu) > e0 + i ? -direction * t.y : direction * t.y;
        }
    }
};

// The rows of q (t 0) or k (t 1) in rows [r0, r1) of a token.
__device__ __forceinline__ void part_rows(const RotaryArgs& a, int t, int r0, int r1, int& h0, int& h1) {
    h0 = t ? max(r0 - a.hq, 0) : r0;
    h1 = t ? r1 - a.hq : min(r1, a.hq);
}

template <typename T, bool kNeighbour>
__global__ void __launch_bounds__(kThreads, 3) rotary_forward_kernel(const __grid_constant__ RotaryArgs a) {
    __shared__ WarpSmem smem[kWarps];
    WarpSmem& w = smem[threadIdx.x >> 5];
    const LaneSetup L(a);
    const bool vec = a.vec != 0;
    const float inv_d = 1.0f / static_cast<float>(a.D);

    const int64_t units = static_cast<int64_t>(a.tokens) * a.parts;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
    // rows of a token per unit, whole warps' worth
    const int share = ((a.rows + a.parts * L.rows_per_warp - 1) / (a.parts * L.rows_per_warp)) * L.rows_per_warp;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units; u += stride) {
        const int token = static_cast<int>(u / a.parts), part = static_cast<int>(u % a.parts);
        const int r0 = part * share, r1 = min(r0 + share, a.rows);
        if (r0 >= r1) continue;
        bool turned = false;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            int h0, h1;
            part_rows(a, t, r0, r1, h0, h1);
            if (h0 >= h1) continue;
            const T* in = static_cast<const T*>(a.x[t].p) + static_cast<int64_t>(token) * a.x[t].st;
            T* out = static_cast<T*>(a.y[t].p) + static_cast<int64_t>(token) * a.y[t].st + L.e0;
            const int64_t in_h = a.x[t].sh, out_h = a.y[t].sh;
            // the next rows' loads are in flight while a row is worked on
            constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;
            Pack<T> own[kAhead];
            auto fetch = [&](int k, int h) {
                if (L.on && h < h1) own[k].load(in + h * in_h + L.e0, vec);
            };
#pragma unroll
            for (int k = 0; k < kAhead; ++k) fetch(k, h0 + k * L.rows_per_warp + L.row_in_warp);
            if (!turned) L.turn_pairs(a, token, w);
            turned = true;
            // y = r (x w c + x' w' s), x' the partner and w' its weight: the norm's factor r comes last
            uint64_t wc[kE / 2], ws[kE / 2];
            const T* wt = static_cast<const T*>(a.w[t]);
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) {
                float c[2], s[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    L.turn_of(w, 2 * i + j, 1.0f, c[j], s[j]);
                    if (wt && L.on) {
                        c[j] *= to_f(wt[L.e0 + 2 * i + j]);
                        s[j] *= to_f(wt[L.partner(2 * i + j)]);
                    }
                }
                wc[i] = pack2(c[0], c[1]);
                ws[i] = pack2(s[0], s[1]);
            }
            for (int hb = h0; hb < h1; hb += kAhead * L.rows_per_warp) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int first = hb + k * L.rows_per_warp;
                    if (first >= h1) break;
                    const int h = first + L.row_in_warp;
                    const bool live = L.on && h < h1;
                    uint64_t x[kE / 2], y[kE / 2];
                    own[k].widen(x);
                    if constexpr (kNeighbour) {
#pragma unroll
                        for (int i = 0; i < kE / 2; ++i) y[i] = swap2(x[i]);
                    } else {
                        Pack<T> far;
                        if (live) L.load_partners(far, in + h * in_h, vec);
                        far.widen(y);
                    }
                    fetch(k, h + kAhead * L.rows_per_warp);
#pragma unroll
                    for (int i = 0; i < kE / 2; ++i) y[i] = fma2(x[i], wc[i], mul2(y[i], ws[i]));
                    if (a.norm) {
                        uint64_t q = mul2(x[0], x[0]);
#pragma unroll
                        for (int i = 1; i < kE / 2; ++i) q = fma2(x[i], x[i], q);
                        const float ss = row_sum(live ? sum2(q) : 0.0f, a.lanes);
                        const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
                        const uint64_t r2 = pack2(r, r);
#pragma unroll
                        for (int i = 0; i < kE / 2; ++i) y[i] = mul2(y[i], r2);
                    }
                    __syncwarp();  // y may be x: every lane has loaded its partners
                    if (live) {
                        Pack<T> o;
                        o.round(y);
                        o.store(out + h * out_h, vec);
                    }
                }
            }
        }
    }
}

template <typename T, bool kNeighbour>
__global__ void __launch_bounds__(kThreads, 2) rotary_backward_kernel(const __grid_constant__ RotaryArgs a) {
    __shared__ WarpSmem smem[kWarps];
    __shared__ alignas(16) float sums[kWarps][32 * kE];
    WarpSmem& w = smem[threadIdx.x >> 5];
    const LaneSetup L(a);
    const bool vec = a.vec != 0;
    const float inv_d = 1.0f / static_cast<float>(a.D);
    uint64_t gw[2][kE / 2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) gw[t][i] = 0;

    const int64_t units = static_cast<int64_t>(a.tokens) * a.parts;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
    const int share = ((a.rows + a.parts * L.rows_per_warp - 1) / (a.parts * L.rows_per_warp)) * L.rows_per_warp;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units; u += stride) {
        const int token = static_cast<int>(u / a.parts), part = static_cast<int>(u % a.parts);
        const int r0 = part * share, r1 = min(r0 + share, a.rows);
        if (r0 >= r1) continue;
        uint64_t c[kE / 2], s[kE / 2];
        bool turned = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            int h0, h1;
            part_rows(a, t, r0, r1, h0, h1);
            if (h0 >= h1) continue;
            const T* gin = static_cast<const T*>(a.y[t].p) + static_cast<int64_t>(token) * a.y[t].st;
            const T* xin = static_cast<const T*>(a.x[t].p) + static_cast<int64_t>(token) * a.x[t].st + L.e0;
            T* out = static_cast<T*>(a.g[t].p) + static_cast<int64_t>(token) * a.g[t].st + L.e0;
            const int64_t g_h = a.y[t].sh, x_h = a.x[t].sh, out_h = a.g[t].sh;
            constexpr int kAhead = 2;
            Pack<T> own[kAhead], val[kAhead];
            auto fetch = [&](int k, int h) {
                if (L.on && h < h1) {
                    own[k].load(gin + h * g_h + L.e0, vec);
                    if (a.norm) val[k].load(xin + h * x_h, vec);
                }
            };
#pragma unroll
            for (int k = 0; k < kAhead; ++k) fetch(k, h0 + k * L.rows_per_warp + L.row_in_warp);
            if (!turned) {
                L.turn_pairs(a, token, w);
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) {
                    float cf[2], sf[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) L.turn_of(w, 2 * i + j, -1.0f, cf[j], sf[j]);
                    c[i] = pack2(cf[0], cf[1]);
                    s[i] = pack2(sf[0], sf[1]);
                }
            }
            turned = true;
            uint64_t wt[kE / 2];
            const T* wp = static_cast<const T*>(a.w[t]);
#pragma unroll
            for (int i = 0; i < kE / 2; ++i)
                wt[i] = wp && L.on ? pack2(to_f(wp[L.e0 + 2 * i]), to_f(wp[L.e0 + 2 * i + 1])) : pack2(1.0f, 1.0f);
            for (int hb = h0; hb < h1; hb += kAhead * L.rows_per_warp) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int first = hb + k * L.rows_per_warp;
                    if (first >= h1) break;
                    const int h = first + L.row_in_warp;
                    const bool live = L.on && h < h1;
                    uint64_t g[kE / 2], x[kE / 2], o[kE / 2];
                    own[k].widen(o);
                    if constexpr (kNeighbour) {
#pragma unroll
                        for (int i = 0; i < kE / 2; ++i) g[i] = swap2(o[i]);
                    } else {
                        Pack<T> far;
                        if (live) L.load_partners(far, gin + h * g_h, vec);
                        far.widen(g);
                    }
                    val[k].widen(x);
                    fetch(k, h + kAhead * L.rows_per_warp);
#pragma unroll
                    for (int i = 0; i < kE / 2; ++i) o[i] = fma2(o[i], c[i], mul2(g[i], s[i]));
                    if (a.norm) {
                        // o = g rotated back; x the head
                        uint64_t q = mul2(x[0], x[0]), d = 0;
#pragma unroll
                        for (int i = 1; i < kE / 2; ++i) q = fma2(x[i], x[i], q);
#pragma unroll
                        for (int i = 0; i < kE / 2; ++i) {
                            g[i] = mul2(o[i], wt[i]);
                            d = fma2(g[i], x[i], d);
                        }
                        const float ss = row_sum(live ? sum2(q) : 0.0f, a.lanes);
                        const float dot = row_sum(live ? sum2(d) : 0.0f, a.lanes);
                        const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
                        const float mean = dot * r * inv_d;  // mean(g w n)
                        const uint64_t r2 = pack2(r, r), m2 = pack2(-mean, -mean);
#pragma unroll
                        for (int i = 0; i < kE / 2; ++i) {
                            const uint64_t n = mul2(x[i], r2);
                            if (live) gw[t][i] = fma2(o[i], n, gw[t][i]);
                            o[i] = mul2(r2, fma2(n, m2, g[i]));
                        }
                    }
                    __syncwarp();  // the output may be the gradient read: every lane has loaded its partners
                    if (live) {
                        Pack<T> y;
                        y.round(o);
                        y.store(out + h * out_h, vec);
                    }
                }
            }
        }
    }
    if (!a.part) return;
    // the block's partial sums, warps and row groups added in order
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < kE / 2; ++i)
            *reinterpret_cast<uint64_t*>(&sums[threadIdx.x >> 5][L.lane * kE + 2 * i]) = gw[t][i];
        __syncthreads();
        for (int e = threadIdx.x; e < a.D; e += kThreads) {
            float sum = 0.0f;
            for (int v = 0; v < kWarps; ++v)
                for (int r = 0; r < L.rows_per_warp; ++r) sum += sums[v][r * a.lanes * kE + e];
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
