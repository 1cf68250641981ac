// pa_block_select.cu -- choosing the cache blocks a decode step attends: an
// exact upper-bound score of every block for every (sequence, kv head), and
// the blocks of the highest scores.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pa.h"
#include "pa_block.cuh"
#include "pa_internal.h"

namespace pa {
namespace block {

// Order-preserving keys of scores; a block that is kept whatever its score
// comes before all of them (a score of +inf is 0xFF800000).
constexpr uint32_t kKeyKept = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t key_of(float score)
{
    const uint32_t b = __float_as_uint(score);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

struct SelectParams {
    int32_t *lists;              // [B, Hkv, K]
    int32_t *list_lens;          // [B]
    const void *q;               // [B, H, D]
    const int8_t *bounds;        // [NB, Hkv, 2, D]
    const float *bounds_scale;   // [NB, Hkv]
    const int32_t *tables, *seq_lens;
    uint32_t *keys;              // [B, Hkv, stride]
    unsigned int *err;
    int num_heads, num_kv_heads, group, num_blocks, max_blocks, block_size, len_cap, most, sink,
        recent, stride, heads_log2, chunk; // kv heads and 16-block tiles of a score CTA
};

__device__ __forceinline__ int checked_len(const SelectParams &p, int s, bool report)
{
    const int len = p.seq_lens[s];
    if (len >= 0 && len <= p.len_cap)
        return len;
    if (report)
        atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
    return len < 0 ? 0 : p.len_cap;
}

constexpr int kScoreWarps = 8;

// Scores.  With U and L a block's upper and lower codes and c a query's codes,
//   sum_d c_d (c_d > 0 ? U_d : L_d) = sum_d max(c_d, 0) U_d + min(c_d, 0) L_d,
// one product of length 2 D.  A warp scores 16 consecutive blocks of one
// (sequence, kv head) at a time against the group's (at most 8) queries, the
// bounds loaded straight into the operand's registers: the contraction index
// of a product is any permutation of the channels as long as the queries use
// the same, so a lane takes 16-byte pieces.
//
// The products are m16n8k16 in halves (a byte product of this shape is eight
// times slower here: 65 against 8 cycles an SM quarter), and exact: a code b
// goes in as the half with the bits b + 128, the subnormal (b + 128) 2^-24,
// which takes one exclusive-or and two byte permutations for four codes.  The
// sum of (b + 128) c is a whole number below 255 * 127 * 256 < 2^24 and stays
// exact in the fp32 accumulator; 128 sum c is taken off at the end.  The two
// scales are powers of two.  So a score has one value, whatever the order.
//
// Bound by the read of the bounds, 2 D + 4 bytes a block and head.  A CTA's 8
// warps are 8 kv heads (or fewer, times several tiles), so that the bounds of a
// block, which lie together, are read at one time, and go through p.chunk tiles.
// A tile's bounds are asked for while the tile before it (or the queries) are
// worked on.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kScoreWarps, 2) score_kernel(const SelectParams p)
{
    constexpr int kPieces = 2 * D / 64;           // 16-byte pieces of a lane and row
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warp = threadIdx.x >> 5, groups = p.num_kv_heads >> p.heads_log2;
    const int head = (blockIdx.x % groups << p.heads_log2) + (warp & ((1 << p.heads_log2) - 1));
    const int step = 16 * (kScoreWarps >> p.heads_log2); // blocks the CTA takes at a time
    const int s = blockIdx.y;
    const int len = checked_len(p, s, blockIdx.x == 0 && threadIdx.x == 0);
    const int n = (len + p.block_size - 1) / p.block_size;
    const int first = blockIdx.x / groups * p.chunk * 16;
    const int last = min(n, first + p.chunk * 16);
    int j0 = first + (warp >> p.heads_log2) * 16;
    if (j0 >= last || n <= p.most)
        return;
    const int32_t *const row = p.tables + (int64_t)s * p.max_blocks;
    // Rows g and g + 8 of a tile: blocks, then bounds and scales.
    int ids[2];
    uint4 v[2][kPieces];
    float bs[2];
    auto name = [&](int j) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            ids[r] = j + g + 8 * r < last ? row[j + g + 8 * r] : -1;
    };
    auto read = [&](int j) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool past = j + g + 8 * r >= last;
            const bool in = !past && ids[r] >= 0 && ids[r] < p.num_blocks;
            if (!past && !in && t == 0)
                atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
            const int64_t at = (int64_t)(in ? ids[r] : 0) * p.num_kv_heads + head;
            if (!past)
#pragma unroll
                for (int c = 0; c < kPieces; ++c)
                    v[r][c] = load16(p.bounds + at * 2 * D + c * 64 + t * 16);
            bs[r] = in ? p.bounds_scale[at] : 0.f; // a block outside the pool scores 0
        }
    };
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < kPieces; ++c)
            v[r][c] = make_uint4(0, 0, 0, 0);
    name(j0);
    read(j0);
    name(j0 + step);

    // Query codes: c = rint(q / 2^e), the largest magnitude within 127; NaN
    // counts as zero.  Lane 4g + t holds query g's channels of its pieces, the
    // positive codes for the upper bounds, then the negative for the lower.
    uint32_t bq[kPieces][4][2];
    float qs, off;
    {
        float x[kPieces / 2][16];
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < kPieces / 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const T *src = static_cast<const T *>(p.q) +
                               ((int64_t)s * p.num_heads + head * p.group + min(g, p.group - 1)) * D +
                               c * 64 + t * 16 + h * 8;
                const uint4 v = *reinterpret_cast<const uint4 *>(src);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = float2_of<T>((&v.x)[k]);
                    x[c][h * 8 + 2 * k] = f.x;
                    x[c][h * 8 + 2 * k + 1] = f.y;
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
        amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
        qs = pow2_scale<127>(amax);
        const float inv = pow2_inverse(qs);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < kPieces / 2; ++c)
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
                float r[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float f = x[c][k + i];
                    r[i] = f == f ? fminf(fmaxf(rintf(f * inv), -127.f), 127.f) : 0.f;
                    sum += r[i];
                }
                bq[c][k / 4][k / 2 % 2] = pair_of<__half>(fmaxf(r[0], 0.f), fmaxf(r[1], 0.f));
                bq[kPieces / 2 + c][k / 4][k / 2 % 2] =
                    pair_of<__half>(fminf(r[0], 0.f), fminf(r[1], 0.f));
            }
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        off = 128.f * sum;
    }
    // Columns 2t and 2t + 1 are queries 2t and 2t + 1 of the group.
    const float q0 = __shfl_sync(~0u, qs, 8 * t), q1 = __shfl_sync(~0u, qs, 8 * t + 4);
    const float off0 = __shfl_sync(~0u, off, 8 * t), off1 = __shfl_sync(~0u, off, 8 * t + 4);
    uint32_t *const keys = p.keys + ((int64_t)s * p.num_kv_heads + head) * p.stride;

    for (; j0 < last; j0 += step) {
        uint4 now[2][kPieces];
        float scale[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            scale[r] = bs[r];
#pragma unroll
            for (int c = 0; c < kPieces; ++c)
                now[r][c] = v[r][c];
        }
        if (j0 + step < last) {
            read(j0 + step);
            name(j0 + 2 * step);
        }
        // two chains of products
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, more[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kPieces; ++c)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t a = (&now[0][c].x)[w] ^ 0x80808080u;
                const uint32_t b = (&now[1][c].x)[w] ^ 0x80808080u;
                mma_16816<__half>(w % 2 ? more : acc, __byte_perm(a, 0, 0x4140),
                                  __byte_perm(b, 0, 0x4140), __byte_perm(a, 0, 0x4342),
                                  __byte_perm(b, 0, 0x4342), bq[c][w][0], bq[c][w][1]);
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            acc[k] += more[k]; // exact, as the sums are
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int j = j0 + g + 8 * r;
            float best = -INFINITY;
            if (2 * t < p.group)
                best = (acc[2 * r] * 16777216.f - off0) * q0 * scale[r];
            if (2 * t + 1 < p.group)
                best = fmaxf(best, (acc[2 * r + 1] * 16777216.f - off1) * q1 * scale[r]);
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 1));
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 2));
            if (t == r && j < last)
                keys[j] = j < p.sink || j >= n - p.recent
                              ? kKeyKept
                              : key_of(scale[r] == INFINITY ? INFINITY : best + 0.f);
        }
    }
}

// Exclusive prefix of a count over the block's threads, and the total.
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    uint32_t sum = lane < THREADS / 32 ? warp_sums[lane] : 0, up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, up, o);
        if (lane >= o)
            up += y;
    }
    total = __shfl_sync(~0u, up, 31);
    const uint32_t base = __shfl_sync(~0u, up - sum, warp);
    __syncthreads();
    return base + x - v;
}

constexpr int kDigit = 8;        // bits of a pass
constexpr int kCandidates = 256; // keys that are ranked against each other

// The `most` largest keys of one (sequence, kv head), in ascending order of
// the block's position; among equal keys the lowest positions.  A radix pass
// over the range that the keys take finds the digit in which the smallest
// chosen key lies.  Mostly few keys share it: they are ranked against each
// other by (key, position), which ends the search; else the next 8 bits are
// looked at.  An ordered scan then writes the positions.  A thread holds PER
// consecutive keys in registers; a longer row goes through in several rounds,
// read again (from L2) each time.  Bound by latency: the barriers, and the fetch
// of code that runs once (2048 bins of 11 bits took longer than 256 of 8).
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) pick_kernel(const SelectParams p)
{
    __shared__ uint32_t hist[1 << kDigit], warp_sums[32], seen[3][32], found[3], candidates;
    __shared__ uint2 candidate[kCandidates]; // distance, position
    __shared__ uint2 edge;                   // the smallest chosen one
    griddep_wait();
    griddep_launch_dependents();
    const int head = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    const int len = checked_len(p, s, false);
    const int n = (len + p.block_size - 1) / p.block_size;
    const int count = min(n, p.most);
    int32_t *list = p.lists + ((int64_t)s * p.num_kv_heads + head) * p.most;
    if (head == 0 && tid == 0)
        p.list_lens[s] = count;
    for (int i = count + tid; i < p.most; i += THREADS)
        list[i] = -1;
    if (n <= p.most) {
        for (int i = tid; i < n; i += THREADS)
            list[i] = i;
        return;
    }
    const uint32_t *keys = p.keys + ((int64_t)s * p.num_kv_heads + head) * p.stride;
    const int rounds = (n + THREADS * PER - 1) / (THREADS * PER);
    uint32_t k[PER];
    auto load = [&](int round) { // keys past the end are 0, below every score
        const int i0 = (round * THREADS + tid) * PER;
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i0 + i < n)
                v = *reinterpret_cast<const uint4 *>(keys + i0 + i);
            k[i] = v.x;
            k[i + 1] = i0 + i + 1 < n ? v.y : 0;
            k[i + 2] = i0 + i + 2 < n ? v.z : 0;
            k[i + 3] = i0 + i + 3 < n ? v.w : 0;
        }
    };
    // how many are kept anyway, and the range of the others
    uint32_t lo = ~0u, hi = 0, kept = 0;
    for (int round = 0; round < rounds; ++round) {
        load(round);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool scored = k[i] != 0 && k[i] != kKeyKept;
            lo = scored ? min(lo, k[i]) : lo;
            hi = scored ? max(hi, k[i]) : hi;
            kept += k[i] == kKeyKept;
        }
    }
    lo = __reduce_min_sync(~0u, lo);
    hi = __reduce_max_sync(~0u, hi);
    kept = __reduce_add_sync(~0u, kept);
    if (lane == 0) {
        seen[0][warp] = lo;
        seen[1][warp] = hi;
        seen[2][warp] = kept;
    }
    if (tid < 1 << kDigit)
        hist[tid] = 0;
    if (tid == 0)
        candidates = 0;
    __syncthreads();
    const bool some = lane < THREADS / 32;
    lo = __reduce_min_sync(~0u, some ? seen[0][lane] : ~0u);
    hi = __reduce_max_sync(~0u, some ? seen[1][lane] : 0u);
    const uint32_t all = __reduce_add_sync(~0u, some ? seen[2][lane] : 0u);
    uint32_t need = p.most - all; // of the scored ones
    // Distances d = key - lo from the smallest key; of the smallest chosen one
    // the bits from `top` up are known, and `need` of the `left` keys that
    // share them are to be chosen.
    uint32_t border = 0, left = ~0u;
    int top = 32 - __clz(hi - lo);
    auto shares = [&](uint32_t key) {
        return key != 0 && key != kKeyKept && (top == 32 || ((key - lo) ^ border) >> top == 0);
    };
    while (top > 0 && left > kCandidates && left != need && need > 0) {
        const int shift = max(top - kDigit, 0);
        for (int round = 0; round < rounds; ++round) {
            if (rounds > 1)
                load(round);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (shares(k[i]))
                    atomicAdd(&hist[(k[i] - lo) >> shift & ((1 << kDigit) - 1)], 1u);
        }
        __syncthreads();
        if (warp == 0) { // lane l: the digits 255 - 8 l .. 248 - 8 l
            constexpr int kEach = (1 << kDigit) / 32;
            uint32_t c[kEach], sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                uint32_t &bin = hist[(1 << kDigit) - 1 - lane * kEach - i];
                sum += c[i] = bin;
                bin = 0;
            }
            uint32_t x = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o)
                    x += y;
            }
            uint32_t before = x - sum;
            if (before < need && x >= need) {
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    if (before < need && before + c[i] >= need) {
                        found[0] = (1 << kDigit) - 1 - lane * kEach - i;
                        found[1] = need - before;
                        found[2] = c[i];
                    }
                    before += c[i];
                }
            }
        }
        __syncthreads();
        border |= found[0] << shift;
        need = found[1];
        left = found[2];
        top = shift;
    }
    // Chosen: the kept, those above the edge's key, and those of its key up to
    // its position.
    uint32_t edge_d = border, edge_at = 0x7FFFFFFFu;
    if (need == 0) { // only the kept
        edge_d = ~0u;
    } else if (left == need) { // all that share the border's bits
    } else if (left <= kCandidates) {
        for (int round = 0; round < rounds; ++round) {
            if (rounds > 1)
                load(round);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (shares(k[i]))
                    candidate[atomicAdd(&candidates, 1u)] =
                        make_uint2(k[i] - lo, (round * THREADS + tid) * PER + i);
        }
        __syncthreads();
        if (tid < (int)left) {
            const uint2 mine = candidate[tid];
            uint32_t rank = 0;
            for (uint32_t j = 0; j < left; ++j) {
                const uint2 other = candidate[j];
                rank += other.x > mine.x || (other.x == mine.x && other.y < mine.y);
            }
            if (rank == need - 1)
                edge = mine;
        }
        __syncthreads();
        edge_d = edge.x;
        edge_at = edge.y;
    } else { // many equal keys: the position of the need-th of them
        uint32_t equal = 0;
        for (int round = 0; round < rounds; ++round) {
            if (rounds > 1)
                load(round);
            uint32_t e = 0, total;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                e += shares(k[i]);
            uint32_t at = equal + block_scan<THREADS>(e, warp_sums, total);
            equal += total;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (shares(k[i]) && ++at == need)
                    edge.y = (round * THREADS + tid) * PER + i;
        }
        __syncthreads();
        edge_at = edge.y;
    }
    uint32_t written = 0;
    for (int round = 0; round < rounds; ++round) {
        if (rounds > 1)
            load(round);
        const uint32_t i0 = (round * THREADS + tid) * PER;
        uint32_t chosen = 0, total; // a bit for each key
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t d = k[i] - lo;
            const bool yes = k[i] == kKeyKept ||
                             (k[i] != 0 && (d > edge_d || (d == edge_d && i0 + i <= edge_at)));
            chosen |= (yes ? 1u : 0u) << i;
        }
        uint32_t at = written + block_scan<THREADS>(__popc(chosen), warp_sums, total);
        written += total;
        for (; chosen; chosen &= chosen - 1)
            list[at++] = i0 + __ffs(chosen) - 1;
    }
}

static bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Keys of a row, a multiple of four.
static size_t key_stride(int max_seq_len, int block_size)
{
    return (((size_t)max_seq_len + block_size - 1) / block_size + 3) / 4 * 4;
}

} // namespace block
} // namespace pa

using namespace pa;
using namespace pa::block;

extern "C" {

size_t pa_select_blocks_workspace_size(int num_seqs, int num_kv_heads, int max_seq_len,
                                       int block_size)
{
    if (num_seqs < 0 || num_kv_heads <= 0 || max_seq_len < 0 || block_size <= 0)
        return 0;
    const size_t bytes = (size_t)num_seqs * num_kv_heads * key_stride(max_seq_len, block_size) * 4;
    return (bytes + 256) / 256 * 256;
}

pa_status pa_select_blocks(int32_t *block_lists, int32_t *list_lens, const void *q,
                           const int8_t *bounds, const float *bounds_scale,
                           const int32_t *block_tables, const int32_t *seq_lens, int num_seqs,
                           int num_heads, int num_kv_heads, int head_size, int block_size,
                           int num_blocks, int max_blocks_per_seq, int max_selected,
                           int num_sink_blocks, int num_recent_blocks, pa_dtype dtype,
                           int max_seq_len, void *workspace, size_t workspace_bytes, void *stream)
{
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 ||
        block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_selected <= 0 ||
        num_sink_blocks < 0 || num_recent_blocks < 0 || max_seq_len < 0 ||
        (int64_t)num_sink_blocks + num_recent_blocks > max_selected ||
        num_heads % num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!block_lists || !list_lens || !q || !bounds || !bounds_scale ||
                         !block_tables || !seq_lens))
        return PA_ERR_INVALID_ARG;
    if (!aligned(block_lists, 4) || !aligned(list_lens, 4) || !aligned(q, 16) ||
        !aligned(bounds, 16) || !aligned(bounds_scale, 4) || !aligned(block_tables, 4) ||
        !aligned(seq_lens, 4))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if ((head_size != 64 && head_size != 128) || (block_size != 16 && block_size != 32) ||
        (group != 1 && group != 2 && group != 4 && group != 8) ||
        (dtype != PA_FP16 && dtype != PA_BF16))
        return PA_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || num_kv_heads > 65535 ||
        (int64_t)num_blocks * block_size >= (int64_t)INT32_MAX ||
        (int64_t)max_blocks_per_seq * block_size >= (int64_t)INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    const int64_t len_cap = (int64_t)max_blocks_per_seq * block_size;
    const int64_t cap = max_seq_len < len_cap ? max_seq_len : len_cap;
    const int stride = (int)key_stride((int)cap, block_size);
    const int64_t row_tiles = (stride + 15) / 16;
    if (row_tiles * num_kv_heads > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0)
        return PA_OK;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < pa_select_blocks_workspace_size(num_seqs, num_kv_heads, max_seq_len,
                                                          block_size))
        return PA_ERR_WORKSPACE;
    cudaError_t e;
    SelectParams p = {};
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    p.lists = block_lists;
    p.list_lens = list_lens;
    p.q = q;
    p.bounds = bounds;
    p.bounds_scale = bounds_scale;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.keys = static_cast<uint32_t *>(workspace);
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.len_cap = (int)cap;
    p.most = max_selected;
    p.sink = num_sink_blocks;
    p.recent = num_recent_blocks;
    p.stride = stride;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (stride > max_selected) { // else every block of every sequence is chosen
        // Tiles of a CTA: about two CTAs an SM in all, so that the queries'
        // codes are formed few times, but no more than 16 tiles a warp.
        const int sms = sm_count(&e);
        if (!sms)
            return PA_ERR_CUDA;
        const int64_t all = row_tiles * num_kv_heads * num_seqs, slots = 2ll * sms * kScoreWarps;
        const int64_t each = std::min<int64_t>((all + slots - 1) / slots, 16);
        p.heads_log2 = heads_log2(num_kv_heads);
        p.chunk = (int)each * (kScoreWarps >> p.heads_log2);
        const dim3 grid((unsigned)((row_tiles + p.chunk - 1) / p.chunk *
                                   (num_kv_heads >> p.heads_log2)),
                        num_seqs);
        const dim3 threads(32 * kScoreWarps);
        if (dtype == PA_BF16)
            e = head_size == 128
                    ? launch_after_previous(score_kernel<__nv_bfloat16, 128>, grid, threads, 0, st, p)
                    : launch_after_previous(score_kernel<__nv_bfloat16, 64>, grid, threads, 0, st, p);
        else
            e = head_size == 128
                    ? launch_after_previous(score_kernel<__half, 128>, grid, threads, 0, st, p)
                    : launch_after_previous(score_kernel<__half, 64>, grid, threads, 0, st, p);
        if (e != cudaSuccess)
            return PA_ERR_CUDA;
    }
    // Rows that fit the registers of 512 threads of 8 keys; longer ones, 16384
    // keys at a time.
    const dim3 rows(num_kv_heads, num_seqs);
    e = stride <= 4096 ? launch_after_previous(pick_kernel<512, 8>, rows, dim3(512), 0, st, p)
                       : launch_after_previous(pick_kernel<1024, 16>, rows, dim3(1024), 0, st, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

} // extern "C"
