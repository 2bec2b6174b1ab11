// Problem description and launchers of the attention over packed sequences
// (internal; the public interface is include/mdcn.h).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

namespace mdcn {

struct AttnTensor {
    void* p;
    int64_t st, sh;  // token and head strides, elements
};

struct AttnArgs {
    AttnTensor q, k, v, out;          // out: written by the forward, read by the backward
    AttnTensor g, gq, gk, gv;         // backward: grad_out (read), gradients (written)
    float* lse;                       // [hq][tq]
    const int32_t* q_starts;          // [batch + 1]
    const int32_t* k_starts;          // [batch + 1]
    const int32_t* k_lengths;         // [batch] or null
    uint32_t* status;                 // first word of the workspace
    float* part_out;                  // forward, keys shared out: [splits][tq][hq][D]
    float* part_lse;                  // [splits][hq][tq]
    float* delta;                     // backward: [hq][tq]
    uint8_t* g_size;                  // float16 backward: [hq][tq], sizes of the rows of grad_out (norm_size)
    uint8_t* v_size;                  // float16 backward: [hk][tk], sizes of the values
    int32_t* sizes;                   // float16 backward: [batch][hk][2], a sequence's largest of both
    float* part_kv;                   // float32 backward, row tiles shared out: [kv_splits][grad_k, grad_v][tk][hk][D]
    float* part_q;                    // float32 backward, key tiles shared out: [q_splits][tq][hq][D]
    int32_t batch, tq, tk, hq, hk, group, D;
    int32_t causal;
    float scale;
    int32_t splits;                   // blocks that share a row tile's keys
    int32_t kv_splits;                // float32 backward: blocks that share a key tile's rows
    int32_t q_splits;                 // float32 backward: blocks that share a row tile's keys
    int32_t tiles;                    // row tiles of one key head at most (see attn_tiles)
    uint64_t item_limit;              // tensor-core kernels: cycles to wait for an item's end at most
};

// Row tiles hold the query heads of one key head together: row r of a tile is
// token r / group, head r % group, so that each key and value is read once for
// all heads that share it. A tile of `rows` rows takes rows / group tokens.
// The number of tiles of `tokens` tokens each that `batch` sequences of `total`
// tokens in all can need at most.
inline int64_t attn_tiles(int64_t total, int64_t batch, int64_t tokens) {
    const int64_t least = total < batch ? total : batch;  // sequences that are not empty
    return (total - least) / tokens + least;
}

constexpr size_t kAttnHeaderBytes = 256;  // the workspace's status word

// Lets a kernel use `bytes` of dynamic shared memory: asked of the runtime the
// first time on each device (`done`, one per kernel, holds a bit for each).
template <typename F>
cudaError_t attn_allow_smem(F kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// CUDA-core kernels (float32; 64 rows x 64 keys).
constexpr int kAttnSimtRows = 64;
cudaError_t launch_attention_simt_forward(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attention_simt_backward(const AttnArgs& a, cudaStream_t st);

// Tensor-core kernels (float16, bfloat16; 128 rows x 128 keys, two row tiles to
// a block).
constexpr int kAttnTcBlockRows = 128;
// Cycles that a role may wait for another to finish an item of `steps` tiles
// (or two of them): the limit of a pipeline's step, and for each tile some 40
// times what one was measured to take.
constexpr uint64_t kAttnStepLimitCycles = 100000;
constexpr uint64_t attn_item_limit(uint64_t step_limit, int64_t steps) {
    return step_limit + static_cast<uint64_t>(steps) * kAttnStepLimitCycles;
}
cudaError_t launch_attention_tc_forward(int dtype, const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attention_tc_backward(int dtype, const AttnArgs& a, cudaStream_t st);

// Joins the partial results of rows whose keys were shared out.
cudaError_t launch_attention_join(int dtype, const AttnArgs& a, cudaStream_t st);
// delta[h][t] = sum over the head of grad_out * out; clears the status word.
// float16: the sizes of grad_out's rows and of the values too, then each
// sequence's largest of both (they scale dS).
cudaError_t launch_attention_delta(int dtype, const AttnArgs& a, cudaStream_t st);

}  // namespace mdcn
