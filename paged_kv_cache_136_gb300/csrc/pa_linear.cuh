// pa_linear.cuh -- parameters of the linear-attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {
namespace lin {

struct LinearParams {
    void *out;                      // [T, H, D]
    const void *q, *k, *v;          // rows of H, Hkv, Hkv heads at their token strides
    const float *log_decay;
    float *states;                  // [num_states, Hkv, D, D]
    const int32_t *src_states, *dst_states;
    const int32_t *query_start_loc; // [num_seqs + 1]; not read by the decode step
    unsigned int *err;
    int64_t decay_stride, q_stride, k_stride, v_stride; // elements
    // prompts of several segments: the lines of the grid (a segment each, at most),
    // tokens of a segment, and each line's state [lines, Hkv, D, D] and decay
    float *parts, *part_decay;
    int lines, segment, num_seqs;
    int num_tokens, max_query_len, num_heads, num_kv_heads, num_states;
    float scale;
};

} // namespace lin
} // namespace pa
