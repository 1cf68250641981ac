// pa_block_cache.cu -- the cache-side operators that work block by block: the
// write of new tokens into an e4m3 pool with one scale for each (plane, block,
// kv head), and the bounds of each block's keys.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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
    int num_tokens, max_query_len, num_kv_heads, num_blocks, len_cap, pieces;
};

constexpr int kWriteWarps = 8;

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) // unsigned 16-bit pairs
{
    return __vmaxu2(a, b);
}

// One warp quantises one block of a request for the kv heads of 32 consecutive
// 16-byte (8-byte for blocks of 32) pieces of a token row: a lane holds the
// same 8 (4) channels of every row of the block, so the new values are read
// once, coalesced, and stay in registers while their largest magnitude is
// formed.  The block's older codes are touched only when the scale grows.
// Bound by HBM: 2 bytes read and 1 written a value; 15540 tokens of 16 prompts
// with 32 kv heads of 128 (382 MB) take 67 us, 5.7 TB/s, and one token of each
// of 256 requests with 8 heads 3.5 us, the latency of three loads in turn.
// (With 80 registers, three CTAs an SM and spills 72 us; with 8-byte loads 70.)
// Grid: x = chunks of kWriteWarps (block of the request, plane, piece of the
// row) units, y = request.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(32 * kWriteWarps) write_block_kernel(const WriteParams p)
{
    constexpr int kWords = BS == 16 ? 4 : 2;      // 32-bit words of a lane and row
    constexpr int kVals = 2 * kWords;             // values of a lane and row
    constexpr int kLanes = D / kVals;             // lanes of a head
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
    const int r = blockIdx.y;
    const int piece = unit % p.pieces, plane = unit / p.pieces % 2, jj = unit / p.pieces / 2;
    Request q;
    if (!read_request(q, r, p.seq_lens, p.query_start_loc, p.num_tokens, p.max_query_len,
                      p.len_cap, unit == 0 && lane == 0, p.err))
        return;
    const int first = q.len - q.fresh;            // position of the first new token
    const int j = first / BS + jj;
    if ((int64_t)j * BS >= q.len)
        return;
    const int blk = p.tables[r * p.table_stride + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (piece == 0 && plane == 0 && lane == 0)
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
        return;
    }
    const int lo = max(0, first - j * BS), hi = min(BS, q.len - j * BS); // rows written
    const int64_t stride = plane ? p.value_stride : p.key_stride, wide = (int64_t)p.num_kv_heads * D;
    const int col = (piece * 32 + lane) * kVals, head = col / D;
    const bool in = col < wide;                   // the row may end inside the piece
    const T *src = static_cast<const T *>(plane ? p.value : p.key) +
                   (q.row + (int64_t)j * BS - first) * stride + col;

    uint32_t x[BS][kWords];
#pragma unroll
    for (int i = 0; i < BS; ++i) {
        const bool read = in && i >= lo && i < hi;
        if constexpr (kWords == 4) {
            const uint4 v = read ? load16(src + i * stride) : make_uint4(0, 0, 0, 0);
            x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        } else {
            const uint2 v = read ? load8(src + i * stride) : make_uint2(0, 0);
            x[i][0] = v.x, x[i][1] = v.y;
        }
    }
    // Magnitudes of 16-bit floats order as their bits do; what is not finite
    // is left out, in a second look that is rarely taken.
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < BS; ++i)
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            top = max_halves(top, x[i][k] & 0x7FFF7FFFu);
    if (__any_sync(~0u, (top & 0xFFFFu) >= kInf || top >> 16 >= kInf)) {
        top = 0;
#pragma unroll
        for (int i = 0; i < BS; ++i)
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                uint32_t m = x[i][k] & 0x7FFF7FFFu;
                if ((m & 0xFFFFu) >= kInf)
                    m &= 0xFFFF0000u;
                if (m >> 16 >= kInf)
                    m &= 0xFFFFu;
                top = max_halves(top, m);
            }
    }
    uint32_t most = max(top & 0xFFFFu, top >> 16);
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1)
        most = max(most, __shfl_xor_sync(~0u, most, o));
    float scale = pow2_scale<448>(float2_of<T>(most).x);

    const int64_t at = (int64_t)plane * p.num_blocks + blk;
    float *const where = p.scales + at * p.num_kv_heads + head;
    uint8_t *dst = p.pool + at * BS * wide + col;
    const unsigned writers = __ballot_sync(~0u, in);
    if (!in)
        return;
    if (lo > 0) {
        const float before = *where;
        scale = fmaxf(scale, before);
        if (scale > before) { // older codes move to the larger scale
            const float ratio = before / scale;
            for (int row = 0; row < lo; ++row) {
#pragma unroll
                for (int k = 0; k < kVals / 4; ++k) {
                    uint32_t *const at4 = reinterpret_cast<uint32_t *>(dst + row * wide) + k;
                    const uint32_t w = *at4;
                    const float2 a = float2_of<__half>(half2_of_e4m3x2(w));
                    const float2 b = float2_of<__half>(half2_of_e4m3x2_hi(w));
                    *at4 = e4m3x2(a.x * ratio, a.y * ratio) | e4m3x2(b.x * ratio, b.y * ratio) << 16;
                }
            }
        }
        // every lane of the head has read the old scale before one writes it
        __syncwarp(writers);
    }
    if (lane % kLanes == 0)
        *where = scale;
    const float inv = pow2_inverse(scale);
#pragma unroll
    for (int i = 0; i < BS; ++i) {
        if (i < lo || i >= hi)
            continue;
        uint32_t c[kVals / 4];
#pragma unroll
        for (int k = 0; k < kVals / 4; ++k) {
            const float2 a = float2_of<T>(x[i][2 * k]), b = float2_of<T>(x[i][2 * k + 1]);
            c[k] = e4m3x2(a.x * inv, a.y * inv) | e4m3x2(b.x * inv, b.y * inv) << 16;
        }
        if constexpr (kWords == 4)
            *reinterpret_cast<uint2 *>(dst + i * wide) = make_uint2(c[0], c[1]);
        else
            *reinterpret_cast<uint32_t *>(dst + i * wide) = c[0];
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
    int max_query_len, num_kv_heads, num_blocks, len_cap, pieces;
};

constexpr int kBoundsWarps = 8;

// Larger and smaller of two pairs; NaN wins.
template <typename T> __device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b);
template <typename T> __device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t pair_max<__half>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t pair_min<__half>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t pair_max<__nv_bfloat16>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t pair_min<__nv_bfloat16>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// One warp forms the bounds of one block of a request for the kv heads of 32
// consecutive 16-byte (8-byte for blocks of 32) pieces of a key row: a lane
// walks the same channels down the block's rows, so each key is read once,
// coalesced, and only the largest magnitude goes across the head's lanes.
// Bound by the latency of three loads in turn (lengths, table, keys) over few
// waves: 72 MB of the same prompts in e4m3 take 15.6 us, 4.6 TB/s, with four
// CTAs an SM (17.4 us with three).  T: type of a 16-bit pool (e4m3 codes become
// halves).  Grid as the write's, without planes.
template <typename T, bool E4M3, int D, int BS>
__global__ void __launch_bounds__(32 * kBoundsWarps, 4) block_bounds_kernel(const BoundsParams p)
{
    constexpr int kWords = BS == 16 ? 4 : 2;      // 32-bit words of a lane and row
    constexpr int kVals = kWords * (E4M3 ? 4 : 2);
    constexpr int kPairs = kVals / 2;
    constexpr int kLanes = D / kVals;             // lanes of a head
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
    const int r = blockIdx.y, piece = unit % p.pieces, jj = unit / p.pieces;
    Request q;
    if (!read_request(q, r, p.seq_lens, p.query_start_loc, INT32_MAX, p.max_query_len, p.len_cap,
                      unit == 0 && lane == 0, p.err))
        return;
    const int j = (q.len - q.fresh) / BS + jj;
    if ((int64_t)j * BS >= q.len)
        return;
    const int blk = p.tables[r * p.table_stride + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (piece == 0 && lane == 0)
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
        return;
    }
    const int rows = min(BS, q.len - j * BS);
    const int wide = p.num_kv_heads * D, head = (piece * 32 + lane) * kVals / D;
    const int col = min((piece * 32 + lane) * kVals, wide - kVals); // past the row: not written
    const bool in = (piece * 32 + lane) * kVals < wide;
    const int64_t step = (int64_t)wide * (E4M3 ? 1 : 2);
    const char *src = static_cast<const char *>(p.pool) + blk * (BS * step) + col * (E4M3 ? 1 : 2);
    uint32_t raw[BS][kWords];
#pragma unroll
    for (int i = 0; i < BS; ++i) {
        const char *const at = src + min(i, rows - 1) * step; // a repeated row changes no bound
        if constexpr (kWords == 4) {
            const uint4 v = load16(at);
            raw[i][0] = v.x, raw[i][1] = v.y, raw[i][2] = v.z, raw[i][3] = v.w;
        } else {
            const uint2 v = load8(at);
            raw[i][0] = v.x, raw[i][1] = v.y;
        }
    }
    float s = 1.f;
    if constexpr (E4M3)
        s = p.scales[(int64_t)blk * p.num_kv_heads + min(head, p.num_kv_heads - 1)];
    uint32_t up[kPairs], low[kPairs];
#pragma unroll
    for (int i = 0; i < BS; ++i)
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            uint32_t v;
            if constexpr (E4M3)
                v = k % 2 ? half2_of_e4m3x2_hi(raw[i][k / 2]) : half2_of_e4m3x2(raw[i][k / 2]);
            else
                v = raw[i][k];
            up[k] = i ? pair_max<T>(up[k], v) : v;
            low[k] = i ? pair_min<T>(low[k], v) : v;
        }
    bool odd = false; // a key that is not finite
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
        const float2 u = float2_of<T>(up[k]), l = float2_of<T>(low[k]);
        const float a = fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(l.x), fabsf(l.y))) * s;
        odd |= !isfinite(a) || u.x != u.x || u.y != u.y;
        amax = fmaxf(amax, a);
    }
    amax = odd ? INFINITY : amax;
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    odd = amax == INFINITY;
    const float scale = pow2_scale<127>(odd ? 0.f : amax), inv = pow2_inverse(scale);
    uint32_t cu[kVals / 4], cl[kVals / 4];
#pragma unroll
    for (int k = 0; k < kVals / 4; ++k)
        cu[k] = cl[k] = 0;
    if (!odd) {
#pragma unroll
        for (int k = 0; k < kVals; ++k) { // rounded outwards: still bounds
            const float2 u = float2_of<T>(up[k / 2]), l = float2_of<T>(low[k / 2]);
            const float a = (k % 2 ? u.y : u.x) * s * inv;
            const float b = (k % 2 ? l.y : l.x) * s * inv;
            const int x = (int)fminf(fmaxf(ceilf(a), -127.f), 127.f);
            const int y = (int)fminf(fmaxf(floorf(b), -127.f), 127.f);
            cu[k / 4] |= (uint32_t)(x & 255) << 8 * (k % 4);
            cl[k / 4] |= (uint32_t)(y & 255) << 8 * (k % 4);
        }
    }
    if (!in)
        return;
    const int64_t at = (int64_t)blk * p.num_kv_heads + head;
    uint32_t *const dst = reinterpret_cast<uint32_t *>(p.bounds + at * 2 * D + col % D);
#pragma unroll
    for (int k = 0; k < kVals / 4; ++k) {
        dst[k] = cu[k];
        dst[k + D / 4] = cl[k];
    }
    if (lane % kLanes == 0)
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
    return PA_OK;
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

template <typename T, bool E4M3>
static cudaError_t launch_bounds(int head_size, int block_size, const BoundsParams &p, dim3 grid,
                                 cudaStream_t s)
{
    const dim3 threads(32 * kBoundsWarps);
    if (head_size == 128)
        return block_size == 16
                   ? launch_after_previous(block_bounds_kernel<T, E4M3, 128, 16>, grid, threads, 0, s, p)
                   : launch_after_previous(block_bounds_kernel<T, E4M3, 128, 32>, grid, threads, 0, s, p);
    return block_size == 16
               ? launch_after_previous(block_bounds_kernel<T, E4M3, 64, 16>, grid, threads, 0, s, p)
               : launch_after_previous(block_bounds_kernel<T, E4M3, 64, 32>, grid, threads, 0, s, p);
}

// Grid x of `warps` warps a CTA: every (block that a request's new tokens can
// reach, 32-lane piece of `bytes` bytes a row) times `planes`.
static int64_t chunks(int max_query_len, int block_size, int64_t pieces, int planes, int warps)
{
    const int64_t reached = (max_query_len + (int64_t)block_size - 2) / block_size + 1;
    return (reached * pieces * planes + warps - 1) / warps;
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
    const int piece = 32 * (block_size == 16 ? 8 : 4); // values of a warp and row
    p.pieces = (int)((row + piece - 1) / piece);
    const int64_t gx = chunks(std::min(max_query_len, p.len_cap), block_size, p.pieces, 2,
                              kWriteWarps);
    if (gx > INT32_MAX / kWriteWarps)
        return PA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)gx, num_reqs);
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
    const int64_t row = (int64_t)num_kv_heads * head_size * (kv_scales ? 1 : 2);
    const int piece = 32 * (block_size == 16 ? 16 : 8); // bytes of a warp and row
    p.pieces = (int)((row + piece - 1) / piece);
    const int64_t gx = chunks(std::min(max_query_len, p.len_cap), block_size, p.pieces, 1,
                              kBoundsWarps);
    if (gx > INT32_MAX / kBoundsWarps)
        return PA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)gx, num_reqs);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    e = kv_scales          ? launch_bounds<__half, true>(head_size, block_size, p, grid, s)
        : dtype == PA_BF16 ? launch_bounds<__nv_bfloat16, false>(head_size, block_size, p, grid, s)
                           : launch_bounds<__half, false>(head_size, block_size, p, grid, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

} // extern "C"
