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
// a few operations on it: bound by device memory. So rows are read and written
// in 16-byte pieces, several rows in flight per warp, and the arithmetic is
// kept short: two values per instruction, weights folded into the cosines and
// sines, the norm's factor applied last. A warp takes all heads of a token (or
// a share of them, when tokens are few), because the cosines and sines depend
// on the token alone: it computes each pair's once, into shared memory, and
// each lane keeps those of its own elements in registers for all of the token's
// heads. Where an element's partner is decides what a lane holds: neighbouring
// pairs, or runs of 8 elements whose partners are a run of 8 too, lie in one
// lane (16 elements); at any other distance the row goes through the warp's
// shared memory (8 elements a lane).
//
// Angles: position * frequency is taken in turns as an exact product (two
// fp32 words), its whole turns are dropped, and only then is it rounded, so
// the error stays 2^-24 of a turn at positions where a rounded product would
// be off by more than a 16-bit unit.
//
// Measured (L2 flushed; q 32 heads of 128 and k 8, three axes, bfloat16): forward
// of 32768 tokens 120 us, 5.6 TB/s; backward of 16384 tokens 109 us, 4.6 TB/s.
// Both wait for memory and for the arithmetic's latency in turn, with as many
// warps as their registers allow (16 and 12 to an SM). 4 maps of 80 x 80, 2 + 2 heads of
// 64, float16: 12 us, of which the chain of launch, frequencies and first rows
// is more than half; 16 tokens: 6 us, all of it that chain.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "mdcn_pdl.h"
#include "mdcn_plan.h"
#include "mdcn_rotary.h"

namespace mdcn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBwdWarps = 4;
constexpr int kBwdThreads = 32 * kBwdWarps;
constexpr int kMaxD = 256;
constexpr int kE = 8;  // elements of a chunk
// A warp's rows together have at most 32 lanes' 16 elements, so 256 pairs,
// whether they are of one token or of several.
constexpr int kMaxTurns = 256;

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

// (lo, hi) rounded to two neighbouring 16-bit elements.
__device__ __forceinline__ void round_pair(float lo, float hi, __half* e) {
    *reinterpret_cast<__half2*>(e) = __floats2half2_rn(lo, hi);
}
__device__ __forceinline__ void round_pair(float lo, float hi, __nv_bfloat16* e) {
    *reinterpret_cast<__nv_bfloat162*>(e) = __floats2bfloat162_rn(lo, hi);
}
__device__ __forceinline__ void round_pair(float lo, float hi, float* e) {
    e[0] = lo;
    e[1] = hi;
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
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
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
            round_pair(lo, hi, e + 2 * i);
        }
    }
};

// A pair's frequency in turns per position (two fp32 words) and its axis.
struct PairFreq {
    float hi, lo;
    int32_t axis;
};

__device__ __forceinline__ PairFreq pair_freq(const RotaryArgs& a, int p, float freq) {
    constexpr float kHi = 0.15915494309189535f;                                        // 1 / (2 pi), rounded
    constexpr float kLo = static_cast<float>(0.15915494309189533577 - static_cast<double>(kHi));  // what is left
    PairFreq f;
    f.hi = freq * kHi;
    f.lo = fmaf(freq, kHi, -f.hi) + freq * kLo;
    f.axis = 0;
    while (f.axis < 3 && p >= a.sec_end[f.axis]) ++f.axis;
    return f;
}

// cos and sin of position * frequency. For 16-bit tensors with the hardware's
// functions, some 2^-20 off (the results are rounded to 2^-12 at best) and a
// third of the instructions.
template <typename T>
__device__ __forceinline__ float2 pair_turn(int32_t pos, const PairFreq& f) {
    // the position in two parts that fp32 holds exactly
    const float pb = static_cast<float>(pos & 4095), pa = static_cast<float>(pos - (pos & 4095));
    float ta = pa * f.hi, tb = pb * f.hi;
    float ea = fmaf(pa, f.hi, -ta), eb = fmaf(pb, f.hi, -tb);
    ta -= rintf(ta);
    tb -= rintf(tb);
    ea -= rintf(ea);
    const float rest = (pa + pb) * f.lo;
    float t = (ta + tb) + ((ea + eb) + (rest - rintf(rest)));
    t -= rintf(t);
    float2 cs;
    if constexpr (sizeof(T) == 2)
        __sincosf(6.28318530717958648f * t, &cs.y, &cs.x);
    else
        sincospif(2.0f * t, &cs.y, &cs.x);
    return cs;
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

// Sum over the lanes that share a row (a power of two of them).
__device__ __forceinline__ float row_sum(float v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (lanes > o) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Where an element's partner is.
enum RotaryMode {
    kBeside = 0,   // neighbouring pairs: in the same register pair
    kChunks = 1,   // every run of 8 elements has a run of 8 partners: the lane holds both
    kAnywhere = 2  // any distance, or rows off 16 bytes: through the warp's shared memory
};

template <int kMode>
struct alignas(16) WarpSmem {
    float2 cs[kMaxTurns];                             // (cos, sin) of the pairs of the warp's tokens
    int32_t pos[4 * 32];                              // their positions, axis by axis
    float row[2][kMode == kAnywhere ? 32 * kE : 4];   // kAnywhere: the warp's rows, two in turn
};

// A lane's place in its row: one chunk of 8 elements (kAnywhere) or two, at
// e0[0] and e0[1]; and where to find its pairs' cosines and sines.
template <int kMode>
struct LaneSetup {
    static constexpr int kC = kMode == kAnywhere ? 1 : 2;
    int lane, rows_per_warp, row_in_warp;
    int e0[kC];
    bool on[kC];  // the chunk exists
    int pair0;    // kBeside, kChunks: the lane's first pair; kChunks: past the pairs where it is not rotated
    // kAnywhere, two elements to a word: partner's index in the warp's rows (8 bits) and
    // pair (7 bits), rotated (1 bit)
    uint32_t code[kMode == kAnywhere ? kE / 2 : 1];
    __device__ __forceinline__ LaneSetup(const RotaryArgs& a) {
        lane = threadIdx.x & 31;
        const int sub = lane & (a.lanes - 1);
        rows_per_warp = 32 / a.lanes;
        row_in_warp = lane / a.lanes;
        if constexpr (kMode == kAnywhere) {
            e0[0] = sub * kE;
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                int to = e0[0] + i;
                float sign;
                const int p = e0[0] < a.D ? pair_of(a, e0[0] + i, to, sign) : -1;
                const uint32_t v = static_cast<uint32_t>(row_in_warp * a.lanes * kE + to) |
                                   (p >= 0 ? static_cast<uint32_t>(p) << 8 | 0x8000u : 0u);
                code[i / 2] = i & 1 ? code[i / 2] | v << 16 : v;
            }
        } else if constexpr (kMode == kBeside) {
            e0[0] = sub * 2 * kE;
            e0[1] = e0[0] + kE;
            pair0 = sub * kE;
        } else {
            // the rotated chunks first, each with its partner, then the others two by two
            const int pairs8 = a.pairs / kE;
            pair0 = sub * kE;
            if (sub >= pairs8) {
                e0[0] = (2 * pairs8 + 2 * (sub - pairs8)) * kE;
                e0[1] = e0[0] + kE;
            } else if (a.layout == 0) {
                e0[0] = sub * kE;
                e0[1] = e0[0] + a.pairs;
            } else {
                int first = 0, ax = 0;
                while (ax < 3 && sub * kE >= a.sec_end[ax]) first = a.sec_end[ax++];
                e0[0] = first + sub * kE;  // 2 first + (8 sub - first)
                e0[1] = e0[0] + a.sec_end[ax] - first;
            }
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) on[c] = e0[c] < a.D;
    }
};

// The block's table of pair frequencies (all threads; ends with a barrier).
// `mine` is the thread's, fetched at the kernel's start: of the first loads none
// waits for another. (At most as many pairs as threads.)
__device__ __forceinline__ float fetch_freq(const RotaryArgs& a) {
    return threadIdx.x < a.pairs ? a.freq[threadIdx.x] : 0.0f;
}
__device__ __forceinline__ void fill_freqs(const RotaryArgs& a, PairFreq* table, float mine) {
    if (threadIdx.x < a.pairs) table[threadIdx.x] = pair_freq(a, threadIdx.x, mine);
    __syncthreads();
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The positions of the warp's next tokens (at most 32), on their way while it
// works on others.
struct Positions {
    int32_t v[4];
    __device__ __forceinline__ void load(const RotaryArgs& a, int64_t token, int n, int lane) {
        const int32_t* p = a.pos + token * a.axes;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < n * a.axes) v[k] = p[lane + 32 * k];
    }
    __device__ __forceinline__ void put(int32_t* to, int count, int lane) const {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < count) to[lane + 32 * k] = v[k];
    }
};

// The cosine of each pair, and its sine, of the n tokens whose positions are at
// `pos` into the warp's shared memory.
template <typename T, int kMode>
__device__ __forceinline__ void turn_pairs(const RotaryArgs& a, const int32_t* pos, int n, const PairFreq* table,
                                           WarpSmem<kMode>& w, int lane) {
    __syncwarp();
    for (int p = lane; p < a.pairs; p += 32) {
        const PairFreq f = table[p];
#pragma unroll 2
        for (int i = 0; i < n; ++i) w.cs[i * a.pairs + p] = pair_turn<T>(pos[i * a.axes + f.axis], f);
    }
    __syncwarp();
}

// A token's turns for the lane's 8 pairs (kBeside, kChunks: one cosine and
// sine per pair) or 8 elements (kAnywhere: the sine has the sign of the
// element's place in its pair). direction -1 turns back. Where part of a head
// is not rotated, its elements are left out of the arithmetic rather than
// turned by nothing: an infinity times a sine of 0 would be NaN.
// kWhole: every element of a head is rotated (32768 tokens of 32 + 8 heads of 128:
// 120 us, and 123 with one kernel for both).
template <int kMode, bool kWhole>
struct Turns {
    float c[kE], s[kE];
    int32_t mine;  // kBeside, kChunks: so many of the lane's pairs are rotated, all where it has fewer
    // `cs`: the pairs of the lane's token.
    __device__ __forceinline__ Turns(const RotaryArgs& a, const LaneSetup<kMode>& L, const float2* cs,
                                     float direction) {
        mine = 0;
        if constexpr (kMode != kAnywhere) mine = a.pairs - L.pair0;
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            float2 v = make_float2(1.0f, 0.0f);
            if constexpr (kMode == kAnywhere) {
                const uint32_t e = L.code[i / 2] >> (16 * (i & 1));
                if (e & 0x8000u) v = cs[(e >> 8) & 0x7fu];
                // the first element of a pair lies before its partner
                const bool low = static_cast<int>(e & 0xffu) > L.lane * kE + i;
                s[i] = low ? -direction * v.y : direction * v.y;
            } else {
                if (L.pair0 + i < a.pairs) v = cs[L.pair0 + i];
                s[i] = direction * v.y;
            }
            c[i] = v.x;
        }
    }
    // x turned; kAnywhere: through `buf`, a row buffer of the warp that no lane reads any more.
    template <int kC>
    __device__ __forceinline__ void turn(uint64_t (&x)[kC][kE / 2], const LaneSetup<kMode>& L, float* buf) const {
        if constexpr (kMode == kBeside) {
#pragma unroll
            for (int k = 0; k < kC; ++k)
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) {
                    const int p = k * (kE / 2) + i;
                    float lo, hi;
                    unpack2(x[k][i], lo, hi);
                    const uint64_t turned = pack2(fmaf(lo, c[p], -(hi * s[p])), fmaf(hi, c[p], lo * s[p]));
                    x[k][i] = kWhole || p < mine ? turned : x[k][i];
                }
        } else if constexpr (kMode == kChunks) {
            if (!kWhole && mine <= 0) return;
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) {
                const uint64_t c2 = pack2(c[2 * i], c[2 * i + 1]), s2 = pack2(s[2 * i], s[2 * i + 1]);
                const uint64_t n2 = pack2(-s[2 * i], -s[2 * i + 1]);
                const uint64_t lo = fma2(x[1][i], n2, mul2(x[0][i], c2));
                x[1][i] = fma2(x[0][i], s2, mul2(x[1][i], c2));
                x[0][i] = lo;
            }
        } else {
            ulonglong2* mine = reinterpret_cast<ulonglong2*>(buf + L.lane * kE);
            mine[0] = make_ulonglong2(x[0][0], x[0][1]);
            mine[1] = make_ulonglong2(x[0][2], x[0][3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) {
                float far0 = buf[L.code[i] & 0xffu], far1 = buf[(L.code[i] >> 16) & 0xffu];
                if constexpr (!kWhole) {
                    far0 = L.code[i] & 0x8000u ? far0 : 0.0f;
                    far1 = L.code[i] & 0x80000000u ? far1 : 0.0f;
                }
                const uint64_t far = pack2(far0, far1);
                const uint64_t c2 = pack2(c[2 * i], c[2 * i + 1]), s2 = pack2(s[2 * i], s[2 * i + 1]);
                x[0][i] = fma2(x[0][i], c2, mul2(far, s2));
            }
        }
    }
};

// The weight of the lane's elements (ones where there is none), as it was
// loaded: half the registers of its fp32 form for 16-bit types.
template <typename T, int kMode>
struct Weights {
    static constexpr int kC = LaneSetup<kMode>::kC;
    Pack<T> w[kC];
    __device__ __forceinline__ Weights(const void* p, const LaneSetup<kMode>& L) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int i = 0; i < kE; ++i) w[c].e[i] = from_f<T>(1.0f);
            if (p && L.on[c]) w[c].load(static_cast<const T*>(p) + L.e0[c], true);
        }
    }
};

// One direction's work on one row per lane group. `At` is where a row lies in
// each tensor; `fetch` loads it into buffers, `work` takes it out of them (and
// then starts their next loads, `next`) and writes the result. Buffers start
// as zeros, so that the chunks that a lane lacks add nothing to its row's sums.
template <typename T, int kMode, bool kWhole>
struct Forward {
    using Type = T;
    static constexpr int kC = LaneSetup<kMode>::kC;
    static constexpr int kAhead = sizeof(T) == 4 ? 2 : (kMode == kAnywhere ? 4 : 3);
    static constexpr bool kForward = true;
    static constexpr float kDirection = 1.0f;
    struct Buffers {
        Pack<T> x[kC];
        __device__ Buffers() {
#pragma unroll
            for (int c = 0; c < kC; ++c) x[c].clear();
        }
    };
    struct At {
        const T* in;
        T* out;
    };
    const LaneSetup<kMode>& L;
    uint64_t wt[kC][kE / 2];
    const RotaryTensor x, y;
    float inv_d, eps;
    int lanes, norm;
    bool vec;
    __device__ __forceinline__ Forward(const RotaryArgs& a, int t, const LaneSetup<kMode>& L)
        : L(L), x(a.x[t]), y(a.y[t]) {
        const Weights<T, kMode> w(a.w[t], L);
#pragma unroll
        for (int c = 0; c < kC; ++c) w.w[c].widen(wt[c]);
        inv_d = 1.0f / static_cast<float>(a.D);
        eps = a.eps;
        lanes = a.lanes;
        norm = a.norm;
        vec = kMode != kAnywhere || a.vec != 0;
    }
    __device__ __forceinline__ At at(int64_t token, int64_t head) const {
        return {static_cast<const T*>(x.p) + token * x.st + head * x.sh + L.e0[0],
                static_cast<T*>(y.p) + token * y.st + head * y.sh + L.e0[0]};
    }
    __device__ __forceinline__ void prefetch(const At& p) const {
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (L.on[c]) prefetch_l2(p.in + (L.e0[c] - L.e0[0]));
    }
    __device__ __forceinline__ void advance_in(At& p, int heads) const { p.in += heads * x.sh; }
    __device__ __forceinline__ void advance_out(At& p, int heads) const { p.out += heads * y.sh; }
    __device__ __forceinline__ void fetch(Buffers& b, const At& p, bool live) const {
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (live && L.on[c]) b.x[c].load(p.in + (L.e0[c] - L.e0[0]), vec);
    }
    template <typename F>
    __device__ __forceinline__ void work(Buffers& b, const At& at, bool live, const Turns<kMode, kWhole>& turns, float* row,
                                         F next) {
        uint64_t v[kC][kE / 2];
#pragma unroll
        for (int c = 0; c < kC; ++c) b.x[c].widen(v[c]);
        next();
        float r = 1.0f;
        if (norm) {
            uint64_t q = 0;
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) {
                    q = fma2(v[c][i], v[c][i], q);
                    v[c][i] = mul2(v[c][i], wt[c][i]);
                }
            r = rsqrtf(fmaf(row_sum(sum2(q), lanes), inv_d, eps));
        }
        turns.turn(v, L, row);
        const uint64_t r2 = pack2(r, r);
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (live && L.on[c]) {
                // the norm's factor, common to the row, comes last
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) v[c][i] = mul2(v[c][i], r2);
                Pack<T> o;
                o.round(v[c]);
                o.store(at.out + (L.e0[c] - L.e0[0]), vec);
            }
    }
};

template <typename T, int kMode, bool kWhole>
struct Backward {
    using Type = T;
    static constexpr int kC = LaneSetup<kMode>::kC;
    static constexpr int kAhead = sizeof(T) == 4 ? 1 : 2;
    static constexpr bool kForward = false;
    static constexpr float kDirection = -1.0f;
    struct Buffers {
        Pack<T> g[kC], x[kC];
        __device__ Buffers() {
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                g[c].clear();
                x[c].clear();
            }
        }
    };
    struct At {
        const T *g, *x;
        T* out;
    };
    const LaneSetup<kMode>& L;
    const Weights<T, kMode> wt;
    const RotaryTensor gy, x, gx;
    float inv_d, eps;
    int lanes, norm;
    bool vec;
    uint64_t gw[kC][kE / 2];  // the weight's gradient, this lane's rows so far
    __device__ __forceinline__ Backward(const RotaryArgs& a, int t, const LaneSetup<kMode>& L)
        : L(L), wt(a.w[t], L), gy(a.y[t]), x(a.x[t]), gx(a.g[t]) {
        inv_d = 1.0f / static_cast<float>(a.D);
        eps = a.eps;
        lanes = a.lanes;
        norm = a.norm;
        vec = kMode != kAnywhere || a.vec != 0;
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int i = 0; i < kE / 2; ++i) gw[c][i] = 0;
    }
    __device__ __forceinline__ At at(int64_t token, int64_t head) const {
        return {static_cast<const T*>(gy.p) + token * gy.st + head * gy.sh + L.e0[0],
                static_cast<const T*>(x.p) + token * x.st + head * x.sh + L.e0[0],
                static_cast<T*>(gx.p) + token * gx.st + head * gx.sh + L.e0[0]};
    }
    __device__ __forceinline__ void advance_in(At& p, int heads) const {
        p.g += heads * gy.sh;
        p.x += heads * x.sh;
    }
    __device__ __forceinline__ void advance_out(At& p, int heads) const { p.out += heads * gx.sh; }
    __device__ __forceinline__ void fetch(Buffers& b, const At& p, bool live) const {
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (live && L.on[c]) {
                b.g[c].load(p.g + (L.e0[c] - L.e0[0]), vec);
                if (norm) b.x[c].load(p.x + (L.e0[c] - L.e0[0]), vec);
            }
    }
    template <typename F>
    __device__ __forceinline__ void work(Buffers& b, const At& at, bool live, const Turns<kMode, kWhole>& turns, float* row,
                                         F next) {
        uint64_t g[kC][kE / 2], v[kC][kE / 2], o[kC][kE / 2];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            b.g[c].widen(o[c]);
            if (norm) b.x[c].widen(v[c]);
        }
        next();
        turns.turn(o, L, row);
        if (norm) {
            // o = the gradient rotated back; v the head
            uint64_t q = 0, d = 0;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                wt.w[c].widen(g[c]);
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) {
                    q = fma2(v[c][i], v[c][i], q);
                    g[c][i] = mul2(o[c][i], g[c][i]);
                    d = fma2(g[c][i], v[c][i], d);
                }
            }
            const float ss = row_sum(sum2(q), lanes), dot = row_sum(sum2(d), lanes);
            const float r = rsqrtf(fmaf(ss, inv_d, eps));
            const float mean = dot * r * inv_d;  // mean(g w n)
            const uint64_t r2 = pack2(r, r), m2 = pack2(-mean, -mean);
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) {
                    const uint64_t n = mul2(v[c][i], r2);
                    if (live) gw[c][i] = fma2(o[c][i], n, gw[c][i]);
                    o[c][i] = mul2(r2, fma2(n, m2, g[c][i]));
                }
        }
#pragma unroll
        for (int c = 0; c < kC; ++c)
            if (live && L.on[c]) {
                Pack<T> y;
                y.round(o[c]);
                y.store(at.out + (L.e0[c] - L.e0[0]), vec);
            }
    }
};

// All rows of q (t 0) or k (t 1), by warp `warp` of `warps`. Heads enough for
// the warp's lane groups: a warp takes a token's heads (or a `parts`-th of
// them), so many passes ahead in flight. Fewer: the lane groups take several
// tokens' heads at once, the next blocks of tokens in flight. The first loads
// start before the block's frequencies are laid out.
template <int kMode, bool kWhole, typename Op>
__device__ __forceinline__ void all_rows(const RotaryArgs& a, int heads, const LaneSetup<kMode>& L, Op& op,
                                         float freq, PairFreq* table, WarpSmem<kMode>& w, int64_t warp,
                                         int64_t warps) {
    constexpr int kAhead = Op::kAhead;
    typename Op::Buffers buf[kAhead];
    Positions pos;
    int which = 0;
    const int rpw = L.rows_per_warp;
    if (heads > rpw / 2) {
        const int64_t units = static_cast<int64_t>(a.tokens) * a.parts;
        const int share = ((heads + a.parts * rpw - 1) / (a.parts * rpw)) * rpw;  // whole warps' worth
        if constexpr (Op::kForward) {
            // the first unit's rows and positions on their way to L2 (the backward, with
            // more to a row, gains nothing: 109 us either way)
            if (warp < units && L.on[0]) {
                const int64_t token = warp / a.parts;
                const int h = static_cast<int>(warp % a.parts) * share + L.row_in_warp;
                if (h < heads) op.prefetch(op.at(token, h));
                prefetch_l2(a.pos + token * a.axes);
            }
        }
        fill_freqs(a, table, freq);
        for (int64_t u = warp; u < units; u += warps) {
            const int token = static_cast<int>(u / a.parts), part = static_cast<int>(u % a.parts);
            const int h0 = part * share, h1 = min(h0 + share, heads);
            if (h0 >= h1) continue;
            typename Op::At ahead = op.at(token, h0 + L.row_in_warp), here = ahead;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                op.fetch(buf[k], ahead, h0 + k * rpw + L.row_in_warp < h1);
                op.advance_in(ahead, rpw);
            }
            turn_pairs<typename Op::Type>(a, a.pos + static_cast<int64_t>(token) * a.axes, 1, table, w, L.lane);
            const Turns<kMode, kWhole> turns(a, L, w.cs, Op::kDirection);
            for (int hb = h0; hb < h1; hb += kAhead * rpw) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int first = hb + k * rpw;
                    if (first >= h1) break;
                    const int h = first + L.row_in_warp;
                    op.work(buf[k], here, h < h1, turns, w.row[which], [&] {
                        op.fetch(buf[k], ahead, h + kAhead * rpw < h1);
                        op.advance_in(ahead, rpw);
                    });
                    op.advance_out(here, rpw);
                    which ^= 1;
                }
            }
        }
    } else if (heads > 0) {
        const int n = rpw / heads;  // tokens at once
        const int mine = L.row_in_warp / heads, h = L.row_in_warp - mine * heads;
        const int64_t blocks = (static_cast<int64_t>(a.tokens) + n - 1) / n;
        // this lane's token of block b, and whether there is one
        auto token_of = [&](int64_t b) { return static_cast<int>(b * n) + mine; };
        auto there = [&](int64_t b) { return b < blocks && mine < n && b * n + mine < a.tokens; };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) op.fetch(buf[k], op.at(token_of(warp + k * warps), h), there(warp + k * warps));
        // the tokens of block b that there are
        auto count = [&](int64_t b) {
            return b < blocks ? static_cast<int>(min(static_cast<int64_t>(n), a.tokens - b * n)) : 0;
        };
        pos.load(a, warp * n, count(warp), L.lane);
        fill_freqs(a, table, freq);
        for (int64_t b0 = warp; b0 < blocks; b0 += kAhead * warps) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t b = b0 + k * warps, bn = b + kAhead * warps;
                if (b >= blocks) break;
                __syncwarp();
                pos.put(w.pos, count(b) * a.axes, L.lane);
                turn_pairs<typename Op::Type>(a, w.pos, count(b), table, w, L.lane);
                pos.load(a, (b + warps) * n, count(b + warps), L.lane);
                const Turns<kMode, kWhole> turns(a, L, w.cs + (mine < n ? mine : 0) * a.pairs, Op::kDirection);
                op.work(buf[k], op.at(token_of(b), h), there(b), turns, w.row[which],
                        [&] { op.fetch(buf[k], op.at(token_of(bn), h), there(bn)); });
                which ^= 1;
            }
        }
    }
}

// Grid: (blocks, 2): q and k by blocks of their own.
template <typename T, int kMode, bool kWhole>
__global__ void __launch_bounds__(kThreads, 2) rotary_forward_kernel(const __grid_constant__ RotaryArgs a) {
    __shared__ WarpSmem<kMode> smem[kWarps];
    __shared__ PairFreq table[kMaxD / 2];
    const LaneSetup<kMode> L(a);
    dependency_wait();
    const float freq = fetch_freq(a);
    const int t = blockIdx.y;
    Forward<T, kMode, kWhole> op(a, t, L);
    all_rows<kMode, kWhole>(a, t ? a.rows - a.hq : a.hq, L, op, freq, table, smem[threadIdx.x >> 5],
                    static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5),
                    static_cast<int64_t>(gridDim.x) * kWarps);
}

// 12 warps to an SM with 168 registers each, two rows of gradients and heads
// in flight: with 16 warps the registers spill.
template <typename T, int kMode, bool kWhole>
__global__ void __launch_bounds__(kBwdThreads, 3) rotary_backward_kernel(const __grid_constant__ RotaryArgs a) {
    constexpr int kC = LaneSetup<kMode>::kC;
    __shared__ WarpSmem<kMode> smem[kBwdWarps];
    __shared__ PairFreq table[kMaxD / 2];
    __shared__ float sums[kBwdWarps][kMaxD];
    const LaneSetup<kMode> L(a);
    dependency_wait();
    const float freq = fetch_freq(a);
    const int t = blockIdx.y;
    Backward<T, kMode, kWhole> op(a, t, L);
    all_rows<kMode, kWhole>(a, t ? a.rows - a.hq : a.hq, L, op, freq, table, smem[threadIdx.x >> 5],
                    static_cast<int64_t>(blockIdx.x) * kBwdWarps + (threadIdx.x >> 5),
                    static_cast<int64_t>(gridDim.x) * kBwdWarps);
    if (!a.part) return;
    // the block's partial sums, warps and row groups added in order
    for (int g = 0; g < L.rows_per_warp; ++g) {
        if (L.row_in_warp == g) {
#pragma unroll
            for (int c = 0; c < kC; ++c)
                if (L.on[c]) {
#pragma unroll
                    for (int i = 0; i < kE / 2; ++i) {
                        float lo, hi;
                        unpack2(op.gw[c][i], lo, hi);
                        float* at = &sums[threadIdx.x >> 5][L.e0[c] + 2 * i];
                        at[0] = g ? at[0] + lo : lo;
                        at[1] = g ? at[1] + hi : hi;
                    }
                }
        }
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += kBwdThreads) {
        float sum = 0.0f;
        for (int v = 0; v < kBwdWarps; ++v) sum += sums[v][e];
        a.part[(static_cast<int64_t>(blockIdx.x) * 2 + t) * a.D + e] = sum;
    }
}

// The weights' gradients: the blocks' partial sums added in a fixed order, 32
// lanes to an element. Grid: (head_dim / 8, 2).
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_weight_sum_kernel(const float* part, int blocks, int D, T* gq, T* gk) {
    dependency_wait();
    T* g = blockIdx.y ? gk : gq;
    if (!g) return;
    // 8 neighbouring elements x 32 slices of the blocks
    __shared__ float sums[32][9];
    const int e = threadIdx.x & 7, slice = threadIdx.x >> 3;
    float v = 0.0f;
#pragma unroll 8
    for (int b = slice; b < blocks; b += 32) v += part[(static_cast<int64_t>(b) * 2 + blockIdx.y) * D + blockIdx.x * 8 + e];
    sums[slice][e] = v;
    __syncthreads();
    if (threadIdx.x < 8) {
        float t = 0.0f;
        for (int k = 0; k < 32; ++k) t += sums[k][threadIdx.x];
        g[blockIdx.x * 8 + threadIdx.x] = from_f<T>(t);
    }
}

// Where the partners are; lanes per row; and how many warps share a token's
// rows: one where tokens alone fill the GPU (the token's cosines are then
// computed once), more where they are few.
RotaryMode plan_lanes(RotaryArgs* a, int sms) {
    bool runs = a->layout == 0 ? a->pairs % kE == 0 : true;
    for (int i = 0; a->layout == 2 && i < 4; ++i) runs = runs && a->sec_end[i] % kE == 0;
    const RotaryMode mode = !a->vec ? kAnywhere : a->layout == 1 ? kBeside : runs ? kChunks : kAnywhere;
    const int per_lane = mode == kAnywhere ? kE : 2 * kE;
    a->lanes = 1;
    while (a->lanes * per_lane < a->D) a->lanes *= 2;
    const int rpw = 32 / a->lanes;
    const int most = (a->rows + rpw - 1) / rpw;
    const int64_t want = static_cast<int64_t>(sms) * 16;  // warps that keep the loads in flight
    int64_t parts = (want + a->tokens - 1) / a->tokens;
    a->parts = static_cast<int32_t>(parts < most ? parts : most);
    return mode;
}

int64_t blocks_for(const RotaryArgs& a, int warps) {
    return (static_cast<int64_t>(a.tokens) * a.parts + warps - 1) / warps;
}

template <typename T, bool kWhole>
cudaError_t forward_of(const RotaryArgs& a, RotaryMode mode, dim3 g, cudaStream_t st) {
    if (mode == kBeside) return launch_dependent(rotary_forward_kernel<T, kBeside, kWhole>, g, kThreads, 0, st, a);
    if (mode == kChunks) return launch_dependent(rotary_forward_kernel<T, kChunks, kWhole>, g, kThreads, 0, st, a);
    return launch_dependent(rotary_forward_kernel<T, kAnywhere, kWhole>, g, kThreads, 0, st, a);
}

template <typename T>
cudaError_t forward_t(const RotaryArgs& a, RotaryMode mode, int64_t grid, cudaStream_t st) {
    const dim3 g(static_cast<unsigned>(grid), a.rows > a.hq ? 2u : 1u);
    return 2 * a.pairs == a.D ? forward_of<T, true>(a, mode, g, st) : forward_of<T, false>(a, mode, g, st);
}

template <typename T, bool kWhole>
cudaError_t backward_of(const RotaryArgs& a, RotaryMode mode, dim3 g, cudaStream_t st) {
    if (mode == kBeside) return launch_dependent(rotary_backward_kernel<T, kBeside, kWhole>, g, kBwdThreads, 0, st, a);
    if (mode == kChunks) return launch_dependent(rotary_backward_kernel<T, kChunks, kWhole>, g, kBwdThreads, 0, st, a);
    return launch_dependent(rotary_backward_kernel<T, kAnywhere, kWhole>, g, kBwdThreads, 0, st, a);
}

template <typename T>
cudaError_t backward_t(const RotaryArgs& a, RotaryMode mode, int64_t grid, void* gqw, void* gkw, cudaStream_t st) {
    const dim3 g(static_cast<unsigned>(grid), a.rows > a.hq ? 2u : 1u);
    const cudaError_t e =
        2 * a.pairs == a.D ? backward_of<T, true>(a, mode, g, st) : backward_of<T, false>(a, mode, g, st);
    if (e != cudaSuccess || !a.part) return e;
    return launch_dependent(rotary_weight_sum_kernel<T>, dim3(static_cast<unsigned>(a.D / 8), 2), kThreads, 0, st,
                            static_cast<const float*>(a.part), static_cast<int>(grid), static_cast<int>(a.D),
                            static_cast<T*>(gqw), static_cast<T*>(gkw));
}

}  // namespace

cudaError_t launch_rotary_forward(int dtype, RotaryArgs a, int sms, cudaStream_t st) {
    const RotaryMode mode = plan_lanes(&a, sms);
    int64_t grid = blocks_for(a, kWarps);
    if (grid > static_cast<int64_t>(sms) * 2) grid = static_cast<int64_t>(sms) * 2;  // one wave each for q and k
    if (dtype == kF32) return forward_t<float>(a, mode, grid, st);
    if (dtype == kF16) return forward_t<__half>(a, mode, grid, st);
    return forward_t<__nv_bfloat16>(a, mode, grid, st);
}

cudaError_t launch_rotary_backward(int dtype, RotaryArgs a, void* gqw, void* gkw, int sms, cudaStream_t st) {
    const RotaryMode mode = plan_lanes(&a, sms);
    int64_t grid = blocks_for(a, kBwdWarps);
    if (grid > static_cast<int64_t>(sms) * 3) grid = static_cast<int64_t>(sms) * 3;  // one wave each for q and k
    if (grid > kRotaryMaxBlocks) grid = kRotaryMaxBlocks;
    if (dtype == kF32) return backward_t<float>(a, mode, grid, gqw, gkw, st);
    if (dtype == kF16) return backward_t<__half>(a, mode, grid, gqw, gkw, st);
    return backward_t<__nv_bfloat16>(a, mode, grid, gqw, gkw, st);
}

}  // namespace mdcn
