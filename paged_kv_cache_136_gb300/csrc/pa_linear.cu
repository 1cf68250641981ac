// pa_linear.cu -- linear attention with a decay for each head: the recurrent
// kernel (single tokens, short prompts) and the host side of both entry points.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pa.h"
#include "pa_block.cuh"
#include "pa_internal.h"
#include "pa_linear.cuh"
#include "pa_linear_tc.cuh"

namespace pa {
namespace lin {

constexpr int kStepThreads = 128, kCols = 64; // of a CTA of the recurrent kernel
constexpr int kHeadsAtOnce = 8; // query heads whose products share the state in registers

// One CTA walks one sequence's tokens for 64 value channels of one kv head with that
// part of the state in registers: a thread has 4 value channels (16 bytes of a state's
// row) of every 8th key channel, so the state is read and written once, in pieces of 256
// bytes, with all of a CTA's loads in flight, and a token's products cost one pass over
// registers and a sum over the 8 row groups in shared memory.  Bound by HBM.  Five small
// CTAs an SM keep reads and writes going side by side, and the states, which the next
// step wants, go past the caches: 64 x 32 states of 128 x 128 take 41 us, 6.5 TB/s, 256 x
// 8 with four query heads each 43 (with cached loads and stores 43 and 46, with whole
// states by 256 threads 51 and 56, with four heads in one pass over the state 45 and 47,
// with the stores before the products 45 and 48).
template <typename T, int D, bool kPrompt>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(const LinearParams p)
{
    constexpr int kLanes = kCols / 4, kGroups = kStepThreads / kLanes, kRows = D / kGroups;
    __shared__ float sk[D], sq[kHeadsAtOnce][D];
    __shared__ float part[kGroups][kHeadsAtOnce][kCols];
    griddep_wait();
    const int tid = threadIdx.x, head = blockIdx.x / (D / kCols), s = blockIdx.y;
    const int col0 = blockIdx.x % (D / kCols) * kCols; // this CTA's value channels
    const int col = tid % kLanes * 4, group = tid / kLanes;
    const int dst = p.dst_states[s], src = p.src_states[s];
    int t0 = s, t1 = s + 1;
    if constexpr (kPrompt) {
        t0 = p.query_start_loc[s], t1 = p.query_start_loc[s + 1];
        if (t0 < 0 || t1 > p.num_tokens || t1 < t0 || t1 - t0 > p.max_query_len) {
            if (tid == 0 && blockIdx.x == 0)
                atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
            return;
        }
    }
    if (dst < 0)
        return;
    if (tid == 0 && blockIdx.x == 0 && (src >= p.num_states || dst >= p.num_states))
        atomicOr(p.err, PA_DEVERR_STATE_);
    const int64_t at = (int64_t)group * D + col0 + col, one = (int64_t)D * D;
    float4 S[kRows];
    if (src >= 0 && src < p.num_states) {
        const float *const from = p.states + ((int64_t)src * p.num_kv_heads + head) * one + at;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            S[i] = __ldcs(reinterpret_cast<const float4 *>(from + (int64_t)i * kGroups * D));
    } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int per = p.num_heads / p.num_kv_heads;
    for (int t = t0; t < t1; ++t) {
        // The decay less one: a decay near one, rounded to 24 bits, would be off by
        // the same 2^-25 in every step, and 256 steps of memory by 2^-17.
        const float a = expm1f(p.log_decay[t * p.decay_stride + head]);
        const T *const k = static_cast<const T *>(p.k) + t * p.k_stride + head * D;
        const T *const v = static_cast<const T *>(p.v) + t * p.v_stride + head * D + col0;
        const T *const q = static_cast<const T *>(p.q) + t * p.q_stride + (int64_t)head * per * D;
        T *const out = static_cast<T *>(p.out) + ((int64_t)t * p.num_heads + head * per) * D + col0;
        const float2 v01 = block::float2_of<T>(*reinterpret_cast<const uint32_t *>(v + col));
        const float2 v23 = block::float2_of<T>(*reinterpret_cast<const uint32_t *>(v + col + 2));
        for (int g0 = 0; g0 < per; g0 += kHeadsAtOnce) {
            const int n = min(kHeadsAtOnce, per - g0);
            if (g0 == 0)
                for (int i = tid; i < D; i += kStepThreads)
                    sk[i] = (float)k[i];
            for (int i = tid; i < n * D; i += kStepThreads)
                sq[i / D][i % D] = (float)q[g0 * D + i] * p.scale;
            __syncthreads();
            if (g0 == 0) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const float kk = sk[group + i * kGroups];
                    S[i].x = fmaf(kk, v01.x, fmaf(a, S[i].x, S[i].x));
                    S[i].y = fmaf(kk, v01.y, fmaf(a, S[i].y, S[i].y));
                    S[i].z = fmaf(kk, v23.x, fmaf(a, S[i].z, S[i].z));
                    S[i].w = fmaf(kk, v23.y, fmaf(a, S[i].w, S[i].w));
                }
            }
            for (int g = 0; g < n; ++g) {
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const float qq = sq[g][group + i * kGroups];
                    o.x = fmaf(qq, S[i].x, o.x);
                    o.y = fmaf(qq, S[i].y, o.y);
                    o.z = fmaf(qq, S[i].z, o.z);
                    o.w = fmaf(qq, S[i].w, o.w);
                }
                *reinterpret_cast<float4 *>(&part[group][g][col]) = o;
            }
            __syncthreads();
            for (int i = tid; i < n * kCols; i += kStepThreads) {
                float o = 0.f;
#pragma unroll
                for (int j = 0; j < kGroups; ++j)
                    o += part[j][i / kCols][i % kCols];
                out[(g0 + i / kCols) * D + i % kCols] = (T)o;
            }
            __syncthreads();
        }
    }
    if (dst < p.num_states) {
        float *const to = p.states + ((int64_t)dst * p.num_kv_heads + head) * one + at;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            __stcs(reinterpret_cast<float4 *>(to + (int64_t)i * kGroups * D), S[i]);
    }
}

static bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Checks that both entry points share, and the parameters.
static pa_status read_args(LinearParams *p, void *out, const void *q, const void *k, const void *v,
                           const float *log_decay, int64_t decay_stride, float *states,
                           const int32_t *src_states, const int32_t *dst_states, int num_seqs,
                           int num_tokens, int num_heads, int num_kv_heads, int head_size,
                           int num_states, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           float scale, pa_dtype dtype)
{
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 ||
        num_states <= 0 || num_heads % num_kv_heads || !isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if ((head_size != 64 && head_size != 128) || (dtype != PA_FP16 && dtype != PA_BF16) ||
        num_seqs > 65535 || num_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    const int64_t kv = (int64_t)num_kv_heads * head_size;
    if (q_stride < (int64_t)num_heads * head_size || k_stride < kv || v_stride < kv ||
        q_stride % 8 || k_stride % 8 || v_stride % 8 ||
        (decay_stride != 0 && decay_stride < num_kv_heads))
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!states || !src_states || !dst_states))
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && num_tokens > 0 && (!out || !q || !k || !v || !log_decay))
        return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(states, 16) || !aligned(log_decay, 4) || !aligned(src_states, 4) ||
        !aligned(dst_states, 4))
        return PA_ERR_INVALID_ARG;
    *p = {};
    p->out = out;
    p->q = q;
    p->k = k;
    p->v = v;
    p->log_decay = log_decay;
    p->decay_stride = decay_stride;
    p->states = states;
    p->src_states = src_states;
    p->dst_states = dst_states;
    p->num_tokens = num_tokens;
    p->num_heads = num_heads;
    p->num_kv_heads = num_kv_heads;
    p->num_states = num_states;
    p->q_stride = q_stride;
    p->k_stride = k_stride;
    p->v_stride = v_stride;
    p->scale = scale;
    return PA_OK;
}

template <bool kPrompt>
static cudaError_t launch_step(const LinearParams &p, int num_seqs, int head_size, pa_dtype dtype,
                               cudaStream_t s)
{
    const dim3 grid(p.num_kv_heads * (head_size / kCols), num_seqs), threads(kStepThreads);
    if (head_size == 128)
        return dtype == PA_BF16
                   ? launch_after_previous(linear_step_kernel<__nv_bfloat16, 128, kPrompt>, grid, threads, 0, s, p)
                   : launch_after_previous(linear_step_kernel<__half, 128, kPrompt>, grid, threads, 0, s, p);
    return dtype == PA_BF16
               ? launch_after_previous(linear_step_kernel<__nv_bfloat16, 64, kPrompt>, grid, threads, 0, s, p)
               : launch_after_previous(linear_step_kernel<__half, 64, kPrompt>, grid, threads, 0, s, p);
}

// ---------------------------------------------------------------------------
// Prompts on the tensor cores
// ---------------------------------------------------------------------------
constexpr int kSms = 152;
// The longest prompt, in tokens, that the recurrent kernel takes.
constexpr int kShort = 16;

// How prompts are cut.  A sequence and kv head is a chain of chunks that one CTA
// walks.  Where the longest chain takes more than twice an SM's share of all work,
// sequences are cut into segments (four for each SM, no shorter than four chunks)
// whose states a first pass forms, at the price of reading K and V twice.
struct Cut {
    int segment, lines;
};

static Cut cut_of(int num_seqs, int num_tokens, int max_query_len, int num_kv_heads)
{
    const int64_t share = (int64_t)num_tokens * num_kv_heads / kSms;
    if (max_query_len <= std::max<int64_t>(2 * share, 8 * kChunk))
        return {INT32_MAX, num_seqs};
    const int64_t segment = std::max<int64_t>(4, (share / 4 + kChunk - 1) / kChunk) * kChunk;
    const int64_t lines = num_tokens / segment + num_seqs + 1;
    return lines <= 65535 ? Cut{(int)segment, (int)lines} : Cut{INT32_MAX, num_seqs};
}

static bool rows_map(CUtensorMap *map, const void *x, pa_dtype dtype, int num_tokens, int heads,
                     int head_size, int64_t stride)
{
    cudaError_t err;
    const auto fn = encode_fn(&err);
    if (!fn)
        return false;
    // {head_size, heads, tokens}; a box is 64 elements of one head of 128 tokens
    cuuint64_t dims[3] = {(cuuint64_t)head_size, (cuuint64_t)heads, (cuuint64_t)num_tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head_size * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, kChunk}, step[3] = {1, 1, 1};
    return fn(map, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              3, const_cast<void *>(x), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap q, k, v, out;
};

template <typename T, int D, bool kParts>
static cudaError_t launch_pass(const Maps &maps, const LinearParams &p, cudaStream_t s)
{
    const auto kern = linear_chunk_kernel<T, D, kParts>;
    constexpr int kSmem = tc_smem_bytes<T, D>();
    static unsigned long long done_mask = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess)
            return e;
        // the registers that the warpgroups trade have to be there at the launch
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, kern);
        if (e != cudaSuccess)
            return e;
        if (a.numRegs < kRegsLaunched)
            return cudaErrorInvalidConfiguration;
        __atomic_fetch_or(&done_mask, bit, __ATOMIC_ACQ_REL);
    }
    return launch_after_previous(kern, dim3(p.num_kv_heads, p.lines), dim3(kTcThreads), kSmem, s, maps.q,
                                 maps.k, maps.v, maps.out, p);
}

template <typename T, int D>
static cudaError_t launch_chunks(const Maps &maps, const LinearParams &p, cudaStream_t s)
{
    if (p.segment != INT32_MAX) {
        cudaError_t e = launch_pass<T, D, true>(maps, p, s);
        if (e == cudaSuccess)
            e = launch_after_previous(linear_join_kernel<D>, dim3(D * D / 1024, p.num_kv_heads, p.num_seqs),
                                      dim3(256), 0, s, p);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pass<T, D, false>(maps, p, s);
}

} // namespace lin
} // namespace pa

using namespace pa;
using namespace pa::lin;

extern "C" {

pa_status pa_linear_decode(void *out, const void *q, const void *k, const void *v,
                           const float *log_decay, int64_t decay_stride, float *states,
                           const int32_t *src_states, const int32_t *dst_states, int num_seqs,
                           int num_heads, int num_kv_heads, int head_size, int num_states,
                           int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                           pa_dtype dtype, void *stream)
{
    LinearParams p;
    const pa_status st = read_args(&p, out, q, k, v, log_decay, decay_stride, states, src_states,
                                   dst_states, num_seqs, num_seqs, num_heads, num_kv_heads,
                                   head_size, num_states, q_stride, k_stride, v_stride, scale, dtype);
    if (st != PA_OK)
        return st;
    if (num_seqs == 0)
        return PA_OK;
    cudaError_t e;
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    e = launch_step<false>(p, num_seqs, head_size, dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_linear_prefill_workspace_size(int num_seqs, int num_tokens, int max_query_len,
                                        int num_kv_heads, int head_size)
{
    if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || num_kv_heads <= 0 || head_size <= 0)
        return 0;
    const Cut cut = cut_of(num_seqs, num_tokens, max_query_len, num_kv_heads);
    if (cut.segment == INT32_MAX)
        return 256;
    const size_t each = (size_t)num_kv_heads * 4 * ((size_t)head_size * head_size + 1);
    return (each * (size_t)cut.lines + 255) / 256 * 256;
}

pa_status pa_linear_prefill(void *out, const void *q, const void *k, const void *v,
                            const float *log_decay, int64_t decay_stride, float *states,
                            const int32_t *src_states, const int32_t *dst_states,
                            const int32_t *query_start_loc, int num_seqs, int num_tokens,
                            int max_query_len, int num_heads, int num_kv_heads, int head_size,
                            int num_states, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                            float scale, pa_dtype dtype, void *workspace, size_t workspace_bytes,
                            void *stream)
{
    LinearParams p;
    const pa_status st = read_args(&p, out, q, k, v, log_decay, decay_stride, states, src_states,
                                   dst_states, num_seqs, num_tokens, num_heads, num_kv_heads,
                                   head_size, num_states, q_stride, k_stride, v_stride, scale, dtype);
    if (st != PA_OK)
        return st;
    if (max_query_len < 0 || (num_seqs > 0 && !query_start_loc) || !aligned(query_start_loc, 4))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0)
        return PA_OK;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < pa_linear_prefill_workspace_size(num_seqs, num_tokens, max_query_len,
                                                           num_kv_heads, head_size))
        return PA_ERR_WORKSPACE;
    cudaError_t e;
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    p.query_start_loc = query_start_loc;
    p.max_query_len = max_query_len;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (num_tokens == 0 || max_query_len <= kShort) {
        e = launch_step<true>(p, num_seqs, head_size, dtype, s);
        return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    }
    const Cut cut = cut_of(num_seqs, num_tokens, max_query_len, num_kv_heads);
    p.num_seqs = num_seqs;
    p.segment = cut.segment;
    p.lines = cut.lines;
    p.parts = static_cast<float *>(workspace);
    p.part_decay = p.parts + (int64_t)cut.lines * num_kv_heads * head_size * head_size;
    Maps maps;
    if (!rows_map(&maps.out, out, dtype, num_tokens, num_heads, head_size,
                  (int64_t)num_heads * head_size) ||
        !rows_map(&maps.q, q, dtype, num_tokens, num_heads, head_size, q_stride) ||
        !rows_map(&maps.k, k, dtype, num_tokens, num_kv_heads, head_size, k_stride) ||
        !rows_map(&maps.v, v, dtype, num_tokens, num_kv_heads, head_size, v_stride))
        return PA_ERR_CUDA;
    if (head_size == 128)
        e = dtype == PA_BF16 ? launch_chunks<__nv_bfloat16, 128>(maps, p, s)
                             : launch_chunks<__half, 128>(maps, p, s);
    else
        e = dtype == PA_BF16 ? launch_chunks<__nv_bfloat16, 64>(maps, p, s)
                             : launch_chunks<__half, 64>(maps, p, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

} // extern "C"
