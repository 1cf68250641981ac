// pa_linear.cu -- linear attention with a decay for each head: the recurrent
// kernel (single tokens, short prompts) and the host side of both entry points.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "pa.h"
#include "pa_block.cuh"
#include "pa_internal.h"
#include "pa_linear.cuh"
#include "pa_linear_tc.cuh"

namespace pa {
namespace lin {

constexpr int kStepThreads = 128, kCols = 64; // of a CTA of the recurrent kernel
constexpr int kHeadsAtOnce = 8; // query heads whose products share the state in registers

// S = e^g S + k v^T and out = scale q S, token by token.  One CTA walks one sequence's
// tokens for 64 value channels of one kv head with that part of the state in registers: a
// thread has 4 value channels (16 bytes of a state's row) of an eighth of the key
// channels, so the state is read and written once, in pieces of 256 bytes, with all of a
// CTA's loads in flight, and a token's products cost one pass over registers and a sum
// over the 8 row groups in shared memory.
//
// One token is bound by HBM.  Five small CTAs an SM keep reads and writes going side by
// side, and the states, which the next step wants, go past the caches: 64 x 32 states of
// 128 x 128 take 40.6 us, 6.6 TB/s, 256 x 8 with four query heads each 41.5 (43 where the
// states' order is random), with eight 43.3 (with rows one by one, not in fours, from
// shared memory 41.3, 43.1 and 47; that form with cached loads and stores 43 and 46 for
// the first two, with whole states by 256 threads 51 and 56, with four heads in one pass
// over the state 45 and 47).  More tokens are bound by their chain of sums and barriers:
// 0.6 us a token alone on the card, 256 x 8 with four heads 10 (13.5 without the next
// token's loads under way).
template <typename T, int D, bool kPrompt>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(const LinearParams p)
{
    constexpr int kLanes = kCols / 4, kGroups = kStepThreads / kLanes, kQuads = D / kGroups / 4;
    constexpr int kPairs = kHeadsAtOnce * D / 2 / kStepThreads; // of a thread, of the queries
    __shared__ __align__(16) float sk[D], sq[kHeadsAtOnce][D];
    __shared__ __align__(16) float part[kGroups][kHeadsAtOnce][kCols];
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
    // rows 4 group to 4 group + 3 of every 4 kGroups
    const int64_t at = (int64_t)group * 4 * D + col0 + col, one = (int64_t)D * D;
    float4 S[kQuads][4];
    if (src >= 0 && src < p.num_states) {
        const float *const from = p.states + ((int64_t)src * p.num_kv_heads + head) * one + at;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[i][r] = __ldcs(reinterpret_cast<const float4 *>(from + (int64_t)(4 * kGroups * i + r) * D));
    } else {
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[i][r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int per = p.num_heads / p.num_kv_heads;

    // A token's inputs, or those of its next kHeadsAtOnce heads, are loaded while the
    // ones before are worked on.
    uint32_t k2 = 0, q2[kPairs];
    uint2 v4 = {};
    float decay = 0.f;
    auto load = [&](int t, int g0) {
        if (g0 == 0) {
            decay = p.log_decay[t * p.decay_stride + head];
            const T *const k = static_cast<const T *>(p.k) + t * p.k_stride + (int64_t)head * D;
            const T *const v = static_cast<const T *>(p.v) + t * p.v_stride + (int64_t)head * D + col0;
            if (tid < D / 2)
                k2 = reinterpret_cast<const uint32_t *>(k)[tid];
            v4 = *reinterpret_cast<const uint2 *>(v + col);
        }
        const T *const q = static_cast<const T *>(p.q) + t * p.q_stride + ((int64_t)head * per + g0) * D;
        const int pairs = min(kHeadsAtOnce, per - g0) * (D / 2);
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            if (tid + i * kStepThreads < pairs)
                q2[i] = reinterpret_cast<const uint32_t *>(q)[tid + i * kStepThreads];
    };
    auto stage = [&](int g0) {
        if (g0 == 0 && tid < D / 2)
            reinterpret_cast<float2 *>(sk)[tid] = block::float2_of<T>(k2);
        const int pairs = min(kHeadsAtOnce, per - g0) * (D / 2);
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            if (tid + i * kStepThreads < pairs) {
                const float2 x = block::float2_of<T>(q2[i]);
                reinterpret_cast<float2 *>(sq)[tid + i * kStepThreads] = make_float2(x.x * p.scale, x.y * p.scale);
            }
    };
    if (t0 < t1) {
        load(t0, 0);
        stage(0);
        __syncthreads();
    }
    for (int t = t0; t < t1; ++t) {
        T *const out = static_cast<T *>(p.out) + ((int64_t)t * p.num_heads + (int64_t)head * per) * D + col0;
        // S e^g, by e^g less one where that is at least a half: a decay near one, rounded
        // to 24 bits, would be off by the same 2^-25 in every step, and 256 steps of memory
        // by 2^-17.  A smaller one is formed as it is: S + (e^g - 1) S is off by 2^-25 of
        // the old state, which is 2^-25 e^(-g) of the new one.  Either way a step's states
        // are within 2^-22 of their size.
        const bool strong = decay < -0.6931472f;
        const float a = strong ? expf(decay) : expm1f(decay);
        const float2 v01 = block::float2_of<T>(v4.x), v23 = block::float2_of<T>(v4.y);
        for (int g0 = 0; g0 < per; g0 += kHeadsAtOnce) {
            const int n = min(kHeadsAtOnce, per - g0);
            const bool last = g0 + kHeadsAtOnce >= per, more = !last || t + 1 < t1;
            const int next = last ? 0 : g0 + kHeadsAtOnce;
            if (more)
                load(last ? t + 1 : t, next);
            if (g0 == 0) {
                auto step = [&](auto is_strong) {
#pragma unroll
                    for (int i = 0; i < kQuads; ++i) {
                        const float4 kk = *reinterpret_cast<const float4 *>(&sk[4 * (kGroups * i + group)]);
                        const float k4[4] = {kk.x, kk.y, kk.z, kk.w};
                        auto decayed = [&](float x) { return is_strong ? a * x : fmaf(a, x, x); };
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            S[i][r].x = fmaf(k4[r], v01.x, decayed(S[i][r].x));
                            S[i][r].y = fmaf(k4[r], v01.y, decayed(S[i][r].y));
                            S[i][r].z = fmaf(k4[r], v23.x, decayed(S[i][r].z));
                            S[i][r].w = fmaf(k4[r], v23.y, decayed(S[i][r].w));
                        }
                    }
                };
                if (strong)
                    step(std::true_type());
                else
                    step(std::false_type());
            }
            for (int g = 0; g < n; ++g) {
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kQuads; ++i) {
                    const float4 qq = *reinterpret_cast<const float4 *>(&sq[g][4 * (kGroups * i + group)]);
                    const float qr[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        o.x = fmaf(qr[r], S[i][r].x, o.x);
                        o.y = fmaf(qr[r], S[i][r].y, o.y);
                        o.z = fmaf(qr[r], S[i][r].z, o.z);
                        o.w = fmaf(qr[r], S[i][r].w, o.w);
                    }
                }
                *reinterpret_cast<float4 *>(&part[group][g][col]) = o;
            }
            __syncthreads();
            if (more)
                stage(next);
            for (int i = tid; i < n * kCols; i += kStepThreads) {
                float o = 0.f;
#pragma unroll
                for (int j = 0; j < kGroups; ++j)
                    o += part[j][i / kCols][i % kCols];
                out[(g0 + i / kCols) * D + i % kCols] = (T)o;
            }
            if (more)
                __syncthreads();
        }
    }
    if (dst < p.num_states) {
        float *const to = p.states + ((int64_t)dst * p.num_kv_heads + head) * one + at;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                __stcs(reinterpret_cast<float4 *>(to + (int64_t)(4 * kGroups * i + r) * D), S[i][r]);
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
// The longest prompt, in tokens, that the recurrent kernel takes.  A chunk costs the same
// however few its tokens.  1, 4, 8, 16 and 32 tokens in us, and chunks: 1 sequence of 32
// heads 8, 10, 14, 22, 37, chunks 15; 32 of 32 heads 28, 39, 55, 86, 158, chunks 78; 256 of
// 32 heads and 8 kv heads 49, 76, 117, 207, 391, chunks 229; with head_size 64 256 of 8
// heads 18, 25, 37, 57, 104, chunks 106.  One number for all sizes: it is that of many
// grouped sequences; for 32 sequences of 32 heads 13 would be right, for a single one 8,
// with head_size 64 32.
constexpr int kShort = 16;

// How prompts are cut.  A sequence and kv head is a chain of chunks that one CTA
// walks, an SM at a time.  Chains can be cut into segments whose states a first pass
// forms, at the price of reading K and V twice.  Taken is the best of at most eight
// cuts, the ones whose segments fill the SMs once, twice, ..., if it is a ninth
// better than none, by these times in us (head_size 128; 64 is a tenth to a fifth
// less on both sides): a chunk 2.3 for each query head and 2.4, or 3.9 with one query
// head, in the first pass 2.5; a chain 8, a segment 12 in both passes; launches 4 and
// 10.  Measured, without a cut and with one: one prompt of 1024, 4096 and 16384 tokens, 32
// heads, 8 kv heads 102 and 36, 379 and 54, 1488 and 131; 32 kv heads 43 and 39, 137 and
// 79, 512 and 239; one of 8192 among 32 of 1024, 8 kv heads, 762 and 347, among 511 of 64
// 1236 and 909.  Left alone are, with 32 kv heads, 4 prompts of 4096 tokens (141, cut 259)
// and, less rightly, one of 8192 among 16 of 512 (270 and 244); with 8, 16 of 4096 (395 and
// 487) and one of 65536 among 4095 of 64 (9800 and 19300).
struct Cut {
    int segment, lines;
};

constexpr float kPassChunk = 2.5f, kChain = 8.f, kSegment = 12.f, kOnePass = 4.f, kTwoPasses = 10.f,
                kWorth = 0.89f, kReturn = 2.5f, kLook = 0.55f;

struct Work {
    float chunks, longest; // in chunks
    int seqs, kv_heads;
    // us without a cut, at `chunk` us a chunk; `fixed` 0 leaves out all that does not grow
    // with that
    float uncut(float chunk, float fixed) const
    {
        const float rounds = ceilf((float)seqs * kv_heads / kSms);
        const float one = longest * chunk + kChain * fixed,
                    all = rounds * (chunks / seqs * chunk + kChain * fixed);
        // Up to 32 sequences the longest starts first.  Of more it starts anywhere in the
        // others' time; this is the mean, of terms linear in `chunk`, so convex in it.
        const float us = seqs <= 32 ? std::max(one, all)
                         : one < all ? all + 0.5f * one * one / all
                                     : one + 0.5f * all;
        return us + kOnePass * fixed;
    }
    // chunks of a segment that fills the SMs `rounds` times; 0 if it does not cut
    int segment(int rounds) const
    {
        const int each = kSms * rounds / kv_heads; // segments of a kv head
        const int n = each ? (int)ceilf(chunks / each) : 0;
        return n < longest ? n : 0;
    }
    // us of whole rounds of such segments: a bound that even lengths come near to
    float rounds_of(int rounds, int n, float chunk, float fixed) const
    {
        return rounds * ((chunk + kPassChunk * fixed) * n + kSegment * fixed) + kTwoPasses * fixed;
    }
    // us of an SM's share and half of a segment, since what is left of uneven lengths ends
    // unevenly; if the others are shorter than a segment at the mean, the longest alone is
    // taken to be cut
    float uneven(int n, float chunk) const
    {
        const bool one = seqs == 1 || (chunks - longest) / (seqs - 1) <= n;
        const float passed = one ? std::min(longest, chunks) : chunks;
        const float chains = one ? ceilf(longest / n) * kSegment + (seqs - 1) * kChain
                                 : (chunks / n + 0.5f * seqs) * kSegment;
        return (chunks * chunk + passed * kPassChunk + chains) * kv_heads / kSms +
               0.5f * (1.f - 1.f / seqs) * (n * (chunk + kPassChunk) + kSegment) + kTwoPasses;
    }
    // us of what grows with the sequences besides: CTAs of the first pass that have nothing
    // to do, and every CTA's search, in both passes, past half of the sequences at the mean
    float search(int64_t lines) const
    {
        const float looks = 0.5f * (float)((seqs - 1) / 32);
        return (seqs * kReturn + lines * 2 * looks * kLook) * kv_heads / kSms;
    }
};
constexpr int kRounds = 8;

static Work work_of(int num_seqs, int num_tokens, int max_query_len, int num_kv_heads)
{
    return {(float)num_tokens / kChunk, ceilf((float)std::min(num_tokens, max_query_len) / kChunk),
            std::max(1, num_seqs), num_kv_heads};
}

static int64_t lines_of(int segment_chunks, int num_seqs, int num_tokens)
{
    return num_tokens / ((int64_t)segment_chunks * kChunk) + num_seqs + 1;
}

static float chunk_us(int heads_each) { return heads_each == 1 ? 3.9f : 2.3f * heads_each + 2.4f; }

static Cut cut_of(int num_seqs, int num_tokens, int max_query_len, int num_heads, int num_kv_heads)
{
    const Work w = work_of(num_seqs, num_tokens, max_query_len, num_kv_heads);
    const float chunk = chunk_us(num_heads / num_kv_heads);
    float best = kWorth * w.uncut(chunk, 1.f);
    Cut cut = {INT32_MAX, num_seqs};
    for (int r = 1; r <= kRounds; ++r) {
        const int n = w.segment(r);
        if (!n || lines_of(n, num_seqs, num_tokens) > 65535)
            continue;
        const float us = std::max(w.rounds_of(r, n, chunk, 1.f), w.uneven(n, chunk)) +
                         w.search(lines_of(n, num_seqs, num_tokens));
        if (us < best) {
            best = us;
            cut = {n * kChunk, (int)lines_of(n, num_seqs, num_tokens)};
        }
    }
    return cut;
}

// The most lines that cut_of can ask for with any number of query heads: a cut takes
// rounds_of at least, which is linear in a chunk's time, and the uncut time is convex, so
// a cut that is no better with one query head or with very many is none in between.
static int64_t most_lines(int num_seqs, int num_tokens, int max_query_len, int num_kv_heads)
{
    const Work w = work_of(num_seqs, num_tokens, max_query_len, num_kv_heads);
    int64_t most = 0;
    for (int r = 1; r <= kRounds; ++r) {
        const int n = w.segment(r);
        if (!n || lines_of(n, num_seqs, num_tokens) > 65535)
            continue;
        if (w.rounds_of(r, n, chunk_us(1), 1.f) < kWorth * w.uncut(chunk_us(1), 1.f) ||
            w.rounds_of(r, n, 1.f, 0.f) < kWorth * w.uncut(1.f, 0.f) * 1.0001f)
            most = std::max(most, lines_of(n, num_seqs, num_tokens));
    }
    return most;
}

// Bytes for the states and decays of `lines` segments.
static size_t workspace_of(int64_t lines, int num_kv_heads, int head_size)
{
    const size_t each = (size_t)num_kv_heads * 4 * ((size_t)head_size * head_size + 1);
    return lines ? (each * (size_t)lines + 255) / 256 * 256 : 256;
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
    return workspace_of(most_lines(num_seqs, num_tokens, max_query_len, num_kv_heads), num_kv_heads,
                        head_size);
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
    Cut cut = cut_of(num_seqs, num_tokens, max_query_len, num_heads, num_kv_heads);
    // the size asked for covers every cut; were the last bit of a float to say otherwise, none
    if (cut.segment != INT32_MAX && workspace_bytes < workspace_of(cut.lines, num_kv_heads, head_size))
        cut = {INT32_MAX, num_seqs};
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
