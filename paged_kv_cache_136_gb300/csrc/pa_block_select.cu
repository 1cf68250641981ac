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
// comes before all of them (a score of +inf is 0xFF800000).  Scores are never
// NaN, whose keys are kKeyKept and 0: a block whose scale is not finite scores
// +inf, and everything else a score is made of is finite.
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
        recent, stride;
    int heads;                   // kv heads that a scoring CTA takes side by side
    int chunk;                   // score_kernel: tiles of a CTA; pick_kernel: keys of shared memory
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
// Bound by the read of the bounds, 2 D + 4 bytes a block and head.  A CTA's
// warps are up to 8 kv heads (times several tiles where that is 8 at most), so
// that the heads of a block, which lie together, are read together.
//
// Scores the blocks j0 .. j0 + 15, then those `step` further, below `last`, of
// a sequence of n blocks, and gives their keys to put(position, key).
template <typename T, int D, typename Put>
__device__ __forceinline__ void score_blocks(const SelectParams &p, int s, int head, int n, int j0,
                                             int step, int last, Put put)
{
    constexpr int kPieces = 2 * D / 64;           // 16-byte pieces of a lane and row
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (j0 >= last)
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
    // Scores are formed 2^-16 times as large: a sum below 2^21 times two scales of
    // up to 2^60 then stays below infinity, and the smallest, whole multiples of
    // 2^-136, are fp32 numbers still (subnormal, kept: no flushing here).
    const float qd = qs * 0x1p-16f;
    const float q0 = __shfl_sync(~0u, qd, 8 * t), q1 = __shfl_sync(~0u, qd, 8 * t + 4);
    const float off0 = __shfl_sync(~0u, off, 8 * t), off1 = __shfl_sync(~0u, off, 8 * t + 4);

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
                put(j, j < p.sink || j >= n - p.recent
                           ? kKeyKept
                           : key_of(isfinite(scale[r]) ? best + 0.f : INFINITY));
        }
    }
}

// The keys of p.chunk tiles of one (sequence, head group) into the workspace.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kScoreWarps, 2) score_kernel(const SelectParams p)
{
    griddep_wait();
    const int warp = threadIdx.x >> 5, groups = p.num_kv_heads / p.heads;
    const int head = blockIdx.x % groups * p.heads + warp % p.heads;
    const int s = blockIdx.y;
    const int len = checked_len(p, s, blockIdx.x == 0 && threadIdx.x == 0);
    const int n = (len + p.block_size - 1) / p.block_size;
    if (n <= p.most)
        return;
    const int first = blockIdx.x / groups * p.chunk * 16;
    uint32_t *const keys = p.keys + ((int64_t)s * p.num_kv_heads + head) * p.stride;
    score_blocks<T, D>(p, s, head, n, first + warp / p.heads * 16,
                       16 * (kScoreWarps / p.heads), min(n, first + p.chunk * 16),
                       [&](int j, uint32_t key) { keys[j] = key; });
    // Not before: the picking CTAs would crowd on the SMs that are free first
    // (27 against 20 us for 8 sequences of 4096 blocks).
    griddep_launch_dependents();
}

constexpr int kDigit = 8;        // bits of a pass
constexpr int kCandidates = 256; // keys that are ranked against each other

// The p.most largest of n > p.most keys of one (sequence, kv head), in
// ascending order of their positions; among equal keys the lowest positions.
// A radix pass over the range that the keys take finds the digit in which the
// smallest chosen key lies.  Mostly few keys share it: they are ranked against
// each other by (key, position), which ends the search; else the next 8 bits
// are looked at.  A warp then counts and writes what is chosen of its own run of
// the keys.  Bound by latency: the barriers, and the fetch of code that runs
// once a launch, so that the loops are rolled but for the four keys of a load: 6
// us for 64 rows of 4096 keys after their scores, 3 us for 32 of 420.
// `keys` is aligned to 16 bytes and may be read up to a multiple of four.
template <int THREADS>
__device__ __forceinline__ void pick_blocks(const SelectParams &p, int n, int32_t *list,
                                            const uint32_t *keys)
{
    constexpr int kWarps = THREADS / 32;
    __shared__ uint32_t hist[1 << kDigit], seen[5][32], found[3], candidates;
    __shared__ uint2 candidate[kCandidates]; // distance, position
    __shared__ uint2 edge;                   // the smallest chosen one
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    struct Quad {
        uint32_t k[4];
    };
    auto read = [&](int i) { // keys i .. i + 3; past the end 0, below every score
        Quad q;
        const uint4 v = *reinterpret_cast<const uint4 *>(keys + i);
        q.k[0] = v.x;
        q.k[1] = i + 1 < n ? v.y : 0;
        q.k[2] = i + 2 < n ? v.z : 0;
        q.k[3] = i + 3 < n ? v.w : 0;
        return q;
    };
    // how many are kept anyway, and the range of the others
    uint32_t lo = ~0u, hi = 0, kept = 0;
#pragma unroll 1
    for (int i = 4 * tid; i < n; i += 4 * THREADS) {
        const Quad q = read(i);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const bool scored = q.k[c] != 0 && q.k[c] != kKeyKept;
            lo = scored ? min(lo, q.k[c]) : lo;
            hi = scored ? max(hi, q.k[c]) : hi;
            kept += q.k[c] == kKeyKept;
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
    const bool some = lane < kWarps;
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
#pragma unroll 1
    while (top > 0 && left > kCandidates && left != need && need > 0) {
        const int shift = max(top - kDigit, 0);
#pragma unroll 1
        for (int i = 4 * tid; i < n; i += 4 * THREADS) {
            const Quad q = read(i);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (shares(q.k[c]))
                    atomicAdd(&hist[(q.k[c] - lo) >> shift & ((1 << kDigit) - 1)], 1u);
        }
        __syncthreads();
        if (warp == 0) { // lane l: the digits 255 - 8 l .. 248 - 8 l
            constexpr int kEach = (1 << kDigit) / 32;
            uint32_t sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                sum += hist[(1 << kDigit) - 1 - lane * kEach - i];
            uint32_t x = sum;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(~0u, x, o);
                x += lane >= o ? y : 0;
            }
            uint32_t before = x - sum;
            if (before < need && x >= need) {
                int digit = (1 << kDigit) - 1 - lane * kEach;
#pragma unroll 1
                for (; before + hist[digit] < need; --digit)
                    before += hist[digit];
                found[0] = digit;
                found[1] = need - before;
                found[2] = hist[digit];
            }
            __syncwarp();
#pragma unroll 1
            for (int i = lane; i < 1 << kDigit; i += 32)
                hist[i] = 0;
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
#pragma unroll 1
        for (int i = 4 * tid; i < n; i += 4 * THREADS) {
            const Quad q = read(i);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (shares(q.k[c]))
                    candidate[atomicAdd(&candidates, 1u)] = make_uint2(q.k[c] - lo, i + c);
        }
        __syncthreads();
        if (tid < (int)left) {
            const uint2 mine = candidate[tid];
            uint32_t rank = 0;
#pragma unroll 4
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
    }
    // A warp's run of the keys, and what is chosen of those before it.  Where
    // many keys are equal to the border, the first `need` of them are.
    const bool equals = need != 0 && left != need && left > kCandidates;
    const int run = ((n + kWarps - 1) / kWarps + 127) / 128 * 128;
    const int first = warp * run + 4 * lane, last = min(n, (warp + 1) * run);
    // of four keys, which are chosen for certain and which are on the border
    auto look = [&](int i, uint32_t &sure, uint32_t &maybe) {
        const Quad q = read(i);
        sure = maybe = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t d = q.k[c] - lo;
            const bool scored = q.k[c] != 0 && q.k[c] != kKeyKept, on = scored && d == edge_d;
            if (q.k[c] == kKeyKept || (scored && d > edge_d) ||
                (on && !equals && (uint32_t)(i + c) <= edge_at))
                sure |= 1u << c;
            else if (on && equals)
                maybe |= 1u << c;
        }
    };
    uint32_t sums[2] = {0, 0};
#pragma unroll 1
    for (int i = first; i < last; i += 128) {
        uint32_t a, b;
        look(i, a, b);
        sums[0] += __popc(a);
        sums[1] += __popc(b);
    }
    sums[0] = __reduce_add_sync(~0u, sums[0]);
    sums[1] = __reduce_add_sync(~0u, sums[1]);
    // Rows of their own: where no digit was looked at and nothing ranked, no
    // barrier lies between here and the other warps' reads of the first three.
    if (lane == 0) {
        seen[3][warp] = sums[0];
        seen[4][warp] = sums[1];
    }
    __syncthreads();
    uint32_t above = __reduce_add_sync(~0u, lane < warp ? seen[3][lane] : 0u);
    uint32_t on = __reduce_add_sync(~0u, lane < warp ? seen[4][lane] : 0u);
    const uint32_t most_on = equals ? need : 0;
#pragma unroll 1
    for (int i = first; i - 4 * lane < last; i += 128) {
        uint32_t a = 0, b = 0;
        if (i < last)
            look(i, a, b);
        const uint32_t counts = __popc(a) | __popc(b) << 16;
        uint32_t x = counts;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(~0u, x, o);
            x += lane >= o ? y : 0;
        }
        const uint32_t total = __shfl_sync(~0u, x, 31);
        x -= counts;
        uint32_t at_a = above + (x & 0xFFFF), at_b = on + (x >> 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const bool sure = a >> c & 1, maybe = b >> c & 1;
            if (sure || (maybe && at_b < most_on))
                list[at_a + min(at_b, most_on)] = i + c;
            at_a += sure;
            at_b += maybe;
        }
        above += total & 0xFFFF;
        on += total >> 16;
    }
}

// The list of a sequence of n <= p.most blocks (all of them), and what lies
// behind every list.
__device__ __forceinline__ void fill_list(const SelectParams &p, int n, int32_t *list)
{
    for (int i = threadIdx.x; i < p.most; i += blockDim.x)
        if (i >= n || n <= p.most)
            list[i] = i < n ? i : -1;
}

// The lists of the keys in the workspace; rows that fit p.chunk keys of shared
// memory are read from there.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) pick_kernel(const SelectParams p)
{
    extern __shared__ __align__(16) uint32_t near_keys[];
    griddep_wait();
    const int head = blockIdx.x, s = blockIdx.y;
    const int n = (checked_len(p, s, false) + p.block_size - 1) / p.block_size;
    const int64_t row = (int64_t)s * p.num_kv_heads + head;
    if (head == 0 && threadIdx.x == 0)
        p.list_lens[s] = min(n, p.most);
    fill_list(p, n, p.lists + row * p.most);
    if (n <= p.most)
        return;
    const uint32_t *keys = p.keys + row * p.stride;
    if (n <= p.chunk) {
        for (int i = threadIdx.x * 4; i < n; i += THREADS * 4)
            *reinterpret_cast<uint4 *>(near_keys + i) = *reinterpret_cast<const uint4 *>(keys + i);
        __syncthreads();
        keys = near_keys;
    }
    pick_blocks<THREADS>(p, n, p.lists + row * p.most, keys);
}

constexpr int kPickSmem = 40 << 10;   // keys of a row in shared memory, without asking for more

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
    const int sms = sm_count(&e);
    if (!sms)
        return PA_ERR_CUDA;
    if (stride > max_selected) { // else every block of every sequence is chosen
        // Tiles of a warp: those that take the fewest steps in waves of two
        // CTAs an SM, with the start of a CTA (its queries' codes) as 3; at most
        // 16, so that sequences shorter than max_seq_len still spread.  Every
        // row is taken for a full one: batches of far shorter ones lose by it (18
        // sequences of 1 to 34559 tokens, 8 heads: 19.7 us, 16.7 with 4 tiles at
        // most), full rows gain (5 of 94762, 32 heads: 41.4, 48.6 with 4).
        p.heads = heads_together(num_kv_heads);
        const int at_once = kScoreWarps / p.heads; // tiles
        const int64_t rows = (int64_t)(num_kv_heads / p.heads) * num_seqs, slots = 2 * sms;
        int64_t best = INT64_MAX;
        for (int each = 1; each <= 16; ++each) {
            const int64_t runs = (row_tiles + each * at_once - 1) / (each * at_once);
            const int64_t steps = (runs * rows + slots - 1) / slots * (3 + each);
            if (steps < best) {
                best = steps;
                p.chunk = each * at_once;
            }
        }
        const dim3 grid((unsigned)((row_tiles + p.chunk - 1) / p.chunk * (num_kv_heads / p.heads)),
                        num_seqs);
        const dim3 threads(32 * p.heads * at_once);
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
    const dim3 rows(num_kv_heads, num_seqs);
    p.chunk = stride * 4 <= kPickSmem ? stride : 0;
    // Long rows get 1024 threads, if there are no more of them than fit at once.
    e = stride <= 1024 || (int64_t)num_kv_heads * num_seqs > 2 * sms
            ? launch_after_previous(pick_kernel<256>, rows, dim3(256), p.chunk * 4, st, p)
            : launch_after_previous(pick_kernel<1024>, rows, dim3(1024), p.chunk * 4, st, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

} // extern "C"
