// Problem description of one rotary call (internal; the public interface is
// include/mdcn.h).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace mdcn {

struct RotaryTensor {
    void* p;
    int64_t st, sh;  // token and head strides, elements
};

struct RotaryArgs {
    // x: q and k (read); y: q_out and k_out, in the backward their gradients (read);
    // g: grad_q and grad_k (written by the backward)
    RotaryTensor x[2], y[2], g[2];
    const void* w[2];    // weights or null
    const int32_t* pos;  // [tokens][axes]
    const float* freq;   // [pairs]
    float* part;         // backward: [blocks][2][head_dim] partial sums of the weights' gradients
    int32_t tokens, hq, rows;  // rows = q_heads + k_heads
    int32_t D, axes, pairs;
    int32_t sec_end[4];  // running sums of the sections
    int32_t layout, norm;
    float eps;
    int32_t vec;         // every row of x, y and g starts on 16 bytes
    int32_t lanes;       // lanes per row: power of two >= D / 16, or D / 8 through shared memory
    int32_t parts;       // warps that share one token's rows
};

cudaError_t launch_rotary_forward(int dtype, RotaryArgs a, int sms, cudaStream_t st);
// blocks of the backward's main kernel at most, so rows of its partial sums
constexpr int kRotaryMaxBlocks = 608;
cudaError_t launch_rotary_backward(int dtype, RotaryArgs a, void* gqw, void* gkw, int sms, cudaStream_t st);

}  // namespace mdcn
