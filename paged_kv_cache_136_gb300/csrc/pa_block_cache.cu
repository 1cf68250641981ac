// pa_block_cache.cu -- the cache-side operators that work block by block: the
// write of new tokens into an e4m3 pool with one scale for each (plane, block,
// kv head), and the bounds of each block's keys.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include "pa.h"
#include "pa_block.cuh"
#include "pa_internal.h"

namespace pa {
namespace block {

struct WriteParams {
    const void *key, *value;     // [T, Hkv, D] rows, strides in elements
    uint8_t *pool;               // [2, NB, bs, Hkv, D] e4m3
    float *scales;               // [2, NB, Hkv]
    const int32_t *tables;       // [R, table_stride]
    const int32_t *seq_lens;     // [R]
    const int32_t *query_start_loc; // [R + 1]
    unsigned int *err;
    int64_t table_stride, key_stride, value_stride;
    int num_tokens, max_query_len, num_kv_heads, num_blocks, len_cap, units;
};

constexpr int kWriteWarps = 8;

// One warp quantises one (request's block, plane, kv head): it reads the new
// tokens' values once, keeps them in registers while it forms their largest
// magnitude, and writes the codes; the block's older codes are touched only
// when the scale grows.  Grid: x = chunks of kWriteWarps (plane, head) units
// of one block, y = block of the request, z = request.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(32 * kWriteWarps) write_block_kernel(const WriteParams p)
{
    constexpr int kLanesPerRow = D / 8;           // 16-byte loads of 8 values
    constexpr int kRowsAtOnce = 32 / kLanesPerRow;
    constexpr int kLoads = BS / kRowsAtOnce;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
    if (unit >= p.units)
        return;
    const int r = blockIdx.z;
    Request q;
    if (!read_request(q, r, p.seq_lens, p.query_start_loc, p.num_tokens, p.max_query_len,
                      p.len_cap, unit == 0 && blockIdx.y == 0 && lane == 0, p.err))
        return;
    const int first = q.len - q.fresh;            // position of the first new token
    const int j = first / BS + blockIdx.y;
    if (j * BS >= q.len)
        return;
    const int blk = p.tables[r * p.table_stride + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (unit == 0 && lane == 0)
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
        return;
    }
    const int plane = unit >= p.num_kv_heads, head = unit - plane * p.num_kv_heads;
    const int lo = max(0, first - j * BS), hi = min(BS, q.len - j * BS); // rows written
    const T *src = static_cast<const T *>(plane ? p.value : p.key);
    const int64_t stride = plane ? p.value_stride : p.key_stride;
    const int sub = lane / kLanesPerRow, col = lane % kLanesPerRow * 8;
    src += (q.row + (int64_t)j * BS - first) * stride + head * D + col;

    uint4 x[kLoads];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = i * kRowsAtOnce + sub;
        x[i] = row >= lo && row < hi ? load16(src + row * stride) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = float2_of<T>((&x[i].x)[k]);
            amax = fmaxf(amax, isfinite(f.x) ? fabsf(f.x) : 0.f);
            amax = fmaxf(amax, isfinite(f.y) ? fabsf(f.y) : 0.f);
        }
    amax = warp_max(amax);
    float scale = pow2_scale<448>(amax);
    const int64_t pool_row = ((int64_t)plane * p.num_blocks + blk) * BS;
    float *const where = p.scales + ((int64_t)plane * p.num_blocks + blk) * p.num_kv_heads + head;
    uint8_t *dst = p.pool + (pool_row * p.num_kv_heads + head) * D + col;
    const int64_t step = (int64_t)p.num_kv_heads * D;
    if (lo > 0) {
        const float before = *where;
        scale = fmaxf(scale, before);
        if (scale > before) { // older codes move to the larger scale
            const float ratio = before / scale;
            for (int row = sub; row < lo; row += kRowsAtOnce) {
                uint2 c = *reinterpret_cast<uint2 *>(dst + row * step);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t &w = k ? c.y : c.x;
                    const float2 a = float2_of<__half>(half2_of_e4m3x2(w));
                    const float2 b = float2_of<__half>(half2_of_e4m3x2_hi(w));
                    w = e4m3x2(a.x * ratio, a.y * ratio) | e4m3x2(b.x * ratio, b.y * ratio) << 16;
                }
                *reinterpret_cast<uint2 *>(dst + row * step) = c;
            }
        }
    }
    __syncwarp();
    if (lane == 0)
        *where = scale;
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = i * kRowsAtOnce + sub;
        if (row < lo || row >= hi)
            continue;
        uint2 c;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 a = float2_of<T>((&x[i].x)[2 * k]);
            const float2 b = float2_of<T>((&x[i].x)[2 * k + 1]);
            (k ? c.y : c.x) = e4m3x2(a.x * inv, a.y * inv) | e4m3x2(b.x * inv, b.y * inv) << 16;
        }
        *reinterpret_cast<uint2 *>(dst + row * step) = c;
    }
}

struct BoundsParams {
    int8_t *bounds;              // [NB, Hkv, 2, D]
    float *bounds_scale;         // [NB, Hkv]
    const void *pool;            // the pool's key plane
    const float *scales;         // its scales [NB, Hkv], or NULL (16-bit pool)
    const int32_t *tables, *seq_lens, *query_start_loc;
    unsigned int *err;
    int64_t table_stride;
    int max_query_len, num_kv_heads, num_blocks, len_cap;
};

constexpr int kBoundsWarps = 8;

// One warp forms the bounds of one (request's block, kv head): a lane holds
// D / 32 channels and walks the block's rows that are in the cache.  The
// kernel reads those keys once and writes 2 D + 4 bytes.  KIND: 0 fp16, 1
// bf16, 2 e4m3 with scales.  Grid as the write's, without the planes.
template <int KIND, int D, int BS>
__global__ void __launch_bounds__(32 * kBoundsWarps) block_bounds_kernel(const BoundsParams p)
{
    constexpr int kPer = D / 32;                  // channels of a lane: 2 or 4
    constexpr int kBytes = kPer * (KIND == 2 ? 1 : 2);
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int head = blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
    if (head >= p.num_kv_heads)
        return;
    const int r = blockIdx.z;
    Request q;
    if (!read_request(q, r, p.seq_lens, p.query_start_loc, INT32_MAX, p.max_query_len, p.len_cap,
                      head == 0 && blockIdx.y == 0 && lane == 0, p.err))
        return;
    const int j = (q.len - q.fresh) / BS + blockIdx.y;
    if (j * BS >= q.len)
        return;
    const int blk = p.tables[r * p.table_stride + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (head == 0 && lane == 0)
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
        return;
    }
    const int rows = min(BS, q.len - j * BS);
    const int64_t step = (int64_t)p.num_kv_heads * D * (KIND == 2 ? 1 : 2);
    const char *src = static_cast<const char *>(p.pool) + (int64_t)blk * BS * step +
                      (head * 32 + lane) * kBytes;
    uint2 raw[BS];
#pragma unroll
    for (int i = 0; i < BS; ++i) {
        raw[i] = make_uint2(0, 0);
        const int row = min(i, rows - 1); // a repeated row changes no bound
        if constexpr (kBytes == 8)
            raw[i] = *reinterpret_cast<const uint2 *>(src + row * step);
        else if constexpr (kBytes == 4)
            raw[i].x = *reinterpret_cast<const uint32_t *>(src + row * step);
        else
            raw[i].x = *reinterpret_cast<const uint16_t *>(src + row * step);
    }
    float up[kPer], low[kPer];
    bool odd = false; // a key that is not finite
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        up[k] = -INFINITY, low[k] = INFINITY;
#pragma unroll
    for (int i = 0; i < BS; ++i)
#pragma unroll
        for (int k = 0; k < kPer; k += 2) {
            float2 f;
            if constexpr (KIND == 2)
                f = float2_of<__half>(k ? half2_of_e4m3x2_hi(raw[i].x) : half2_of_e4m3x2(raw[i].x));
            else if constexpr (KIND == 1)
                f = float2_of<__nv_bfloat16>(k ? raw[i].y : raw[i].x);
            else
                f = float2_of<__half>(k ? raw[i].y : raw[i].x);
            odd |= !isfinite(f.x) || !isfinite(f.y);
            up[k] = fmaxf(up[k], f.x);
            low[k] = fminf(low[k], f.x);
            up[k + 1] = fmaxf(up[k + 1], f.y);
            low[k + 1] = fminf(low[k + 1], f.y);
        }
    if constexpr (KIND == 2) {
        const float s = p.scales[(int64_t)blk * p.num_kv_heads + head];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            up[k] *= s;
            low[k] *= s;
            odd |= !isfinite(up[k]) || !isfinite(low[k]);
        }
    }
    odd = __any_sync(~0u, odd);
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        amax = fmaxf(amax, fmaxf(fabsf(up[k]), fabsf(low[k])));
    amax = warp_max(amax);
    const float scale = pow2_scale<127>(odd ? 0.f : amax), inv = pow2_inverse(scale);
    uint32_t cu = 0, cl = 0;
    if (!odd) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) { // rounded outwards: still bounds
            const int u = (int)fminf(fmaxf(ceilf(up[k] * inv), -127.f), 127.f);
            const int l = (int)fminf(fmaxf(floorf(low[k] * inv), -127.f), 127.f);
            cu |= (uint32_t)(u & 255) << 8 * k;
            cl |= (uint32_t)(l & 255) << 8 * k;
        }
    }
    const int64_t at = (int64_t)blk * p.num_kv_heads + head;
    int8_t *dst = p.bounds + at * 2 * D + lane * kPer;
    if constexpr (kPer == 4) {
        *reinterpret_cast<uint32_t *>(dst) = cu;
        *reinterpret_cast<uint32_t *>(dst + D) = cl;
    } else {
        *reinterpret_cast<uint16_t *>(dst) = (uint16_t)cu;
        *reinterpret_cast<uint16_t *>(dst + D) = (uint16_t)cl;
    }
    if (lane == 0)
        p.bounds_scale[at] = odd ? INFINITY : scale;
}

static bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// What both calls require of their sizes; PA_OK with nothing to do is left to
// the caller.
static pa_status check_requests(const int32_t *tables, int64_t table_stride,
                                const int32_t *seq_lens, const int32_t *query_start_loc,
                                int num_reqs, int max_query_len, int num_kv_heads, int head_size,
                                int block_size, int num_blocks, int max_blocks_per_seq)
{
    if (num_reqs < 0 || max_query_len < 0 || num_kv_heads <= 0 || head_size <= 0 ||
        block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 ||
        table_stride < max_blocks_per_seq)
        return PA_ERR_INVALID_ARG;
    if (num_reqs > 0 && (!tables || !seq_lens || !query_start_loc))
        return PA_ERR_INVALID_ARG;
    if (!aligned(tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4))
        return PA_ERR_INVALID_ARG;
    if ((head_size != 64 && head_size != 128) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if (num_reqs > 65535 || num_kv_heads > 65535 ||
        (int64_t)num_blocks * block_size >= (int64_t)INT32_MAX ||
        (int64_t)max_blocks_per_seq * block_size >= (int64_t)INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    // blocks that one request's new tokens can reach: the grid's y extent
    if ((max_query_len + (int64_t)block_size - 2) / block_size + 1 > 65535)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

static int reached_blocks(int max_query_len, int block_size)
{
    return (max_query_len + block_size - 2) / block_size + 1;
}

template <typename T>
static cudaError_t launch_write(int head_size, int block_size, const WriteParams &p, dim3 grid,
                                cudaStream_t s)
{
    const dim3 threads(32 * kWriteWarps);
    if (head_size == 128)
        return block_size == 16
                   ? launch_after_previous(write_block_kernel<T, 128, 16>, grid, threads, 0, s, p)
                   : launch_after_previous(write_block_kernel<T, 128, 32>, grid, threads, 0, s, p);
    return block_size == 16
               ? launch_after_previous(write_block_kernel<T, 64, 16>, grid, threads, 0, s, p)
               : launch_after_previous(write_block_kernel<T, 64, 32>, grid, threads, 0, s, p);
}

template <int KIND>
static cudaError_t launch_bounds(int head_size, int block_size, const BoundsParams &p, dim3 grid,
                                 cudaStream_t s)
{
    const dim3 threads(32 * kBoundsWarps);
    if (head_size == 128)
        return block_size == 16
                   ? launch_after_previous(block_bounds_kernel<KIND, 128, 16>, grid, threads, 0, s, p)
                   : launch_after_previous(block_bounds_kernel<KIND, 128, 32>, grid, threads, 0, s, p);
    return block_size == 16
               ? launch_after_previous(block_bounds_kernel<KIND, 64, 16>, grid, threads, 0, s, p)
               : launch_after_previous(block_bounds_kernel<KIND, 64, 32>, grid, threads, 0, s, p);
}

} // namespace block
} // namespace pa

using namespace pa;
using namespace pa::block;

extern "C" {

pa_status pa_reshape_and_cache_fp8_block(const void *key, const void *value, void *kv_cache,
                                         float *kv_scales, const int32_t *block_tables,
                                         int64_t block_table_stride, const int32_t *seq_lens,
                                         const int32_t *query_start_loc, int num_reqs,
                                         int num_tokens, int max_query_len, int num_kv_heads,
                                         int head_size, int block_size, int num_blocks,
                                         int max_blocks_per_seq, int64_t key_stride,
                                         int64_t value_stride, pa_dtype src_dtype, void *stream)
{
    const pa_status st = check_requests(block_tables, block_table_stride, seq_lens,
                                        query_start_loc, num_reqs, max_query_len, num_kv_heads,
                                        head_size, block_size, num_blocks, max_blocks_per_seq);
    if (st != PA_OK)
        return st;
    if (src_dtype != PA_FP16 && src_dtype != PA_BF16)
        return PA_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)num_kv_heads * head_size;
    if (num_tokens < 0 || key_stride < row || value_stride < row || key_stride % 8 ||
        value_stride % 8)
        return PA_ERR_INVALID_ARG;
    if (num_reqs == 0 || num_tokens == 0 || max_query_len == 0)
        return PA_OK;
    if (!key || !value || !kv_cache || !kv_scales || !aligned(key, 16) || !aligned(value, 16) ||
        !aligned(kv_cache, 16) || !aligned(kv_scales, 4))
        return PA_ERR_INVALID_ARG;
    cudaError_t e;
    WriteParams p = {};
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    p.key = key;
    p.value = value;
    p.pool = static_cast<uint8_t *>(kv_cache);
    p.scales = kv_scales;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.query_start_loc = query_start_loc;
    p.table_stride = block_table_stride;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.num_tokens = num_tokens;
    p.max_query_len = max_query_len;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = num_blocks;
    p.len_cap = max_blocks_per_seq * block_size;
    p.units = 2 * num_kv_heads;
    const dim3 grid((p.units + kWriteWarps - 1) / kWriteWarps,
                    reached_blocks(max_query_len, block_size), num_reqs);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = src_dtype == PA_BF16 ? launch_write<__nv_bfloat16>(head_size, block_size, p, grid, s)
                             : launch_write<__half>(head_size, block_size, p, grid, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_update_block_bounds(int8_t *bounds, float *bounds_scale, const void *kv_cache,
                                 const float *kv_scales, const int32_t *block_tables,
                                 int64_t block_table_stride, const int32_t *seq_lens,
                                 const int32_t *query_start_loc, int num_reqs, int max_query_len,
                                 int num_kv_heads, int head_size, int block_size, int num_blocks,
                                 int max_blocks_per_seq, pa_dtype dtype, void *stream)
{
    const pa_status st = check_requests(block_tables, block_table_stride, seq_lens,
                                        query_start_loc, num_reqs, max_query_len, num_kv_heads,
                                        head_size, block_size, num_blocks, max_blocks_per_seq);
    if (st != PA_OK)
        return st;
    if (dtype != PA_FP16 && dtype != PA_BF16)
        return PA_ERR_UNSUPPORTED;
    if (num_reqs == 0 || max_query_len == 0)
        return PA_OK;
    if (!bounds || !bounds_scale || !kv_cache || !aligned(bounds, 16) ||
        !aligned(bounds_scale, 4) || !aligned(kv_cache, 16) || !aligned(kv_scales, 4))
        return PA_ERR_INVALID_ARG;
    cudaError_t e;
    BoundsParams p = {};
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    p.bounds = bounds;
    p.bounds_scale = bounds_scale;
    p.pool = kv_cache;
    p.scales = kv_scales;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.query_start_loc = query_start_loc;
    p.table_stride = block_table_stride;
    p.max_query_len = max_query_len;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = num_blocks;
    p.len_cap = max_blocks_per_seq * block_size;
    const dim3 grid((num_kv_heads + kBoundsWarps - 1) / kBoundsWarps,
                    reached_blocks(max_query_len, block_size), num_reqs);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = kv_scales            ? launch_bounds<2>(head_size, block_size, p, grid, s)
        : dtype == PA_BF16   ? launch_bounds<1>(head_size, block_size, p, grid, s)
                             : launch_bounds<0>(head_size, block_size, p, grid, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

} // extern "C"
