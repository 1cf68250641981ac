// pa_sequences.cu -- the life of sequences in a block pool: forking and freeing
// rows of the block tables, room for new tokens (blocks taken, shared last
// blocks copied, slots), and moving the live blocks to the front of the pool.
//
// All of it is whole numbers and copied bytes, so every result has one right
// value whatever the order in which CTAs run: a block is taken by its rank among
// the free ones, counts are changed by integer atomics.
#include <cuda_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace seqs {

constexpr int kThreads = 256;      // of the wide kernels
constexpr int kChunk = 1024;       // table entries of a CTA
constexpr int kRankThreads = 1024; // of a CTA of the ranking kernels
constexpr int kCluster = 8;        // CTAs of a ranking kernel
constexpr int kRows = 8;           // table rows of a thread of theirs: 65536 in all
constexpr int kTile = 4 * kRankThreads; // counts that a CTA ranks at once
constexpr int kUnit = 16384;       // bytes of a block that a CTA copies at once
// A sum of at most 65535 rows' needs: blocks, fewer than 2^31 a row, and above
// them the rows that copy a block.
constexpr int kCopyBit = 47;

// ---------------------------------------------------------------------------
// Pools: what a block's bytes are, for the copies of extend and compact
// ---------------------------------------------------------------------------
struct Pool {
    uint8_t *data;       // [planes, num_blocks, block_bytes]
    int64_t block_bytes, plane_bytes;
    int first_unit;      // units of the pools before this one
    int plane_units;     // units of a block of one plane
    int planes;
    int width;           // bytes of a load: 16, 4 or 1
};

struct Pools {
    Pool pool[PA_MAX_POOLS];
    int count, units;    // units of a block, over all pools
};

// One CTA copies `bytes` bytes.  Eight CTAs an SM, four loads of 16 bytes a thread in
// flight: half of a pool of 1.6 GB moves at 6.7 TB/s, read and written.
template <typename W>
__device__ __forceinline__ void copy_bytes(uint8_t *dst, const uint8_t *src, int64_t bytes)
{
    const W *const s = reinterpret_cast<const W *>(src);
    W *const d = reinterpret_cast<W *>(dst);
    const int n = (int)(bytes / (int)sizeof(W));
    // four loads in flight a thread
    for (int i = threadIdx.x; i < n; i += 4 * kThreads) {
        W v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k * kThreads < n)
                v[k] = s[i + k * kThreads];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k * kThreads < n)
                d[i + k * kThreads] = v[k];
    }
}

// One CTA copies unit `u` of block src to block dst.
__device__ __forceinline__ void copy_unit(const Pools &ps, int u, int64_t src, int64_t dst)
{
    int lo = 0, hi = ps.count - 1; // the last pool that begins at or before u
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (ps.pool[mid].first_unit <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Pool &p = ps.pool[lo];
    const int at = u - p.first_unit, plane = at / p.plane_units;
    const int64_t off = (int64_t)(at - plane * p.plane_units) * kUnit;
    const int64_t bytes = min((int64_t)kUnit, p.block_bytes - off);
    uint8_t *const base = p.data + plane * p.plane_bytes + off;
    uint8_t *const d = base + dst * p.block_bytes;
    const uint8_t *const s = base + src * p.block_bytes;
    if (p.width == 16)
        copy_bytes<uint4>(d, s, bytes);
    else if (p.width == 4)
        copy_bytes<uint32_t>(d, s, bytes);
    else
        copy_bytes<uint8_t>(d, s, bytes);
}

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------
struct ForkParams {
    int32_t *tables_out, *lens_out, *refs;
    const int32_t *tables, *lens, *parents;
    unsigned int *err;
    int rows_in, rows_out, num_blocks, max_blocks, block_size, len_cap;
};

__device__ __forceinline__ int blocks_of(int len, int bs) { return len / bs + (len % bs != 0); }

// A row's length, held to what its table can hold.
__device__ __forceinline__ int length_of(const int32_t *lens, int r, int cap, bool tell,
                                         unsigned int *err)
{
    const int n = lens[r];
    if (n >= 0 && n <= cap)
        return n;
    if (tell)
        atomicOr(err, PA_DEVERR_SEQ_LEN_);
    return n < 0 ? 0 : cap;
}

__global__ void __launch_bounds__(kThreads) copy_counts_kernel(int32_t *__restrict__ out,
                                                               const int32_t *__restrict__ in, int n)
{
    griddep_wait();
    const int first = blockIdx.x * (4 * kThreads) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (first + k * kThreads < n)
            out[first + k * kThreads] = in[first + k * kThreads];
}

// CTA (r, c): entries [c kChunk, (c + 1) kChunk) of new row r, and of old row r,
// whose blocks' counts change by its children less one.  Rows with one child, the
// most of a beam search's, touch no count.  Every CTA counts its row's children among
// all parents itself, so that no pass comes before.  Bound by latency: with counts
// copied first 6.4 us for 16 rows in a pool of 127 blocks, 8.1 for 512 rows of 720000
// entries in all in one of 310000 blocks.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkParams p)
{
    griddep_wait();
    const int r = blockIdx.x, base = blockIdx.y * kChunk, tid = threadIdx.x;
    const bool first = blockIdx.y == 0 && tid == 0;
    if (r < p.rows_out) {
        const int parent = p.parents[r];
        int n = 0;
        if (parent >= 0 && parent < p.rows_in)
            n = length_of(p.lens, parent, p.len_cap, first, p.err);
        else if (parent >= p.rows_in && first)
            atomicOr(p.err, PA_DEVERR_PARENT_);
        if (first)
            p.lens_out[r] = n;
        const int end = min(blocks_of(n, p.block_size), base + kChunk);
        const int32_t *const src = p.tables + (int64_t)parent * p.max_blocks;
        int32_t *const dst = p.tables_out + (int64_t)r * p.max_blocks;
        int32_t v[kChunk / kThreads];
#pragma unroll
        for (int k = 0; k < kChunk / kThreads; ++k)
            if (base + tid + k * kThreads < end)
                v[k] = src[base + tid + k * kThreads];
#pragma unroll
        for (int k = 0; k < kChunk / kThreads; ++k)
            if (base + tid + k * kThreads < end) {
                if (v[k] < 0 || v[k] >= p.num_blocks)
                    atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
                dst[base + tid + k * kThreads] = v[k];
            }
    }
    if (r >= p.rows_in)
        return;
    const int n = blocks_of(length_of(p.lens, r, p.len_cap, first, p.err), p.block_size);
    if (base >= n)
        return;
    int children = 0;
    for (int i = 0; i < p.rows_out; i += kThreads)
        children += __syncthreads_count(i + tid < p.rows_out && p.parents[i + tid] == r);
    if (children == 1)
        return;
    const int end = min(n, base + kChunk);
    for (int j = base + tid; j < end; j += kThreads) {
        const int b = p.tables[(int64_t)r * p.max_blocks + j];
        if (b >= 0 && b < p.num_blocks)
            atomicAdd(p.refs + b, children - 1);
        else
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
    }
}

// ---------------------------------------------------------------------------
// Ranks, by one cluster
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What a CTA of the cluster tells the others, in the workspace: at most three sums.
struct Told {
    int64_t v[4];
};

// The first N sums of the CTAs before this one, and of all: each lane reads one CTA's,
// so that the reads take one latency.
template <int N>
__device__ __forceinline__ void hear(const Told *told, int rank, int ctas, int64_t (&before)[N],
                                     int64_t (&all)[N])
{
    const int lane = threadIdx.x & 31;
    int64_t x[N];
#pragma unroll
    for (int n = 0; n < N; ++n)
        x[n] = lane < ctas ? __ldcg(&told[lane].v[n]) : 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        int64_t y = lane < rank ? x[n] : 0;
#pragma unroll
        for (int o = kCluster / 2; o; o /= 2) {
            x[n] += __shfl_xor_sync(~0u, x[n], o);
            y += __shfl_xor_sync(~0u, y, o);
        }
        all[n] = __shfl_sync(~0u, x[n], 0);
        before[n] = __shfl_sync(~0u, y, 0);
    }
}

// Exclusive prefixes of N values over the CTA's threads, and their sums; `sums` has a
// slot for each of the 32 warps.  Two barriers.
template <int N>
__device__ __forceinline__ void prefix(int64_t (&v)[N], int64_t (*sums)[32], int64_t (&total)[N])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x[N];
#pragma unroll
    for (int n = 0; n < N; ++n)
        x[n] = v[n];
#pragma unroll
    for (int o = 1; o < 32; o *= 2)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t y = __shfl_up_sync(~0u, x[n], o);
            if (lane >= o)
                x[n] += y;
        }
    __syncthreads();
    if (lane == 31)
#pragma unroll
        for (int n = 0; n < N; ++n)
            sums[n][warp] = x[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        int64_t w = sums[n][lane];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t y = __shfl_up_sync(~0u, w, o);
            if (lane >= o)
                w += y;
        }
        total[n] = __shfl_sync(~0u, w, 31);
        const int64_t before = __shfl_sync(~0u, w, (warp + 31) & 31);
        v[n] = (warp ? before : 0) + x[n] - v[n];
    }
}

// f(id, count, number of free ids in [begin, id)) for every id of [begin, end), in
// tiles of kTile: a warp has 128 consecutive ids, 32 at a time.
template <typename F>
__device__ __forceinline__ void ranked(const int32_t *refs, int begin, int end, int *sums, F f)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int carry = 0;
    for (int t = begin; t < end; t += kTile) {
        const int at = t + warp * 128 + lane;
        int v[4];
        unsigned m[4];
        int mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = at + 32 * k < end ? refs[at + 32 * k] : 1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m[k] = __ballot_sync(~0u, v[k] == 0);
            mine += __popc(m[k]);
        }
        __syncthreads();
        if (lane == 0)
            sums[warp] = mine;
        __syncthreads();
        const int other = sums[lane];
        int before = __reduce_add_sync(~0u, lane < warp ? other : 0) + carry;
        carry += __reduce_add_sync(~0u, other);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (at + 32 * k < end)
                f(at + 32 * k, v[k], before + __popc(m[k] & ((1u << lane) - 1)));
            before += __popc(m[k]);
        }
    }
}

// This thread's free ids of [begin, end); the CTA's, the same for every thread.
__device__ __forceinline__ int my_free(const int32_t *refs, int begin, int end)
{
    int n = 0;
#pragma unroll 8
    for (int i = begin + threadIdx.x; i < end; i += kRankThreads)
        n += refs[i] == 0;
    return n;
}
__device__ __forceinline__ int sum_of(int n, int *sums)
{
    n = __reduce_add_sync(~0u, n);
    if ((threadIdx.x & 31) == 0)
        sums[threadIdx.x >> 5] = n;
    __syncthreads();
    n = __reduce_add_sync(~0u, sums[threadIdx.x & 31]);
    __syncthreads();
    return n;
}

struct ExtendParams {
    int32_t *tables_out, *lens_out, *refs_out, *info;
    int64_t *slots;
    const int32_t *tables, *lens, *refs, *num_new;
    unsigned int *err;
    // workspace: per block
    int32_t *writers, *latest, *free_ids;
    // per row: old length, new tokens, first rank of its blocks, first token, and
    // its old last block if that is copied, else kKept or kLost; the rows that copy
    int32_t *row_len, *row_new, *row_begin, *row_token, *row_copy, *copy_rows;
    Told *told;          // of each CTA
    int32_t *head;       // tokens, rows that copy
    int rows, num_blocks, max_blocks, block_size, len_cap, num_tokens;
};

constexpr int kKept = -1, kLost = -2;
struct Row {
    int len, fresh, last; // last: the block that new tokens go on in, or kKept
};

__device__ __forceinline__ Row read_row(const ExtendParams &p, int r)
{
    Row x;
    x.fresh = p.num_new[r];
    x.len = length_of(p.lens, r, p.len_cap, true, p.err);
    if (x.fresh < 0 || x.fresh > p.len_cap - x.len) {
        atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
        x.fresh = 0;
    }
    x.last = kKept;
    if (x.fresh > 0 && x.len % p.block_size) {
        const int b = p.tables[(int64_t)r * p.max_blocks + x.len / p.block_size];
        if (b >= 0 && b < p.num_blocks)
            x.last = b;
        else
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
    }
    return x;
}

// One cluster: every row's needs, their prefix sums, and the ids of as many free
// blocks.  A row that goes on in a shared block copies it, but for the last of its
// holders where all of them go on; that is what row after row would come to.
//
// Bound by a chain of latencies: lengths, last entries, counts, two rounds of atomics,
// the counts again; so one cluster, whose barriers cost less than launches, with each
// step's loads side by side.  The whole call takes 16.4 us for 256 rows in a pool of 8200
// blocks, 19.4 with 40000 and 31 for 16 rows with 400000 (one CTA in place of eight: 18.4,
// 31 and 131; with 16 rows in 1000 blocks both take 16).
__global__ void __launch_bounds__(kRankThreads) extend_rank_kernel(const ExtendParams p)
{
    __shared__ int64_t sums[2][32];
    __shared__ int counts[32];
    griddep_wait();
    const int rank = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x;
    const int per = (p.rows + ctas - 1) / ctas;
    const int r0 = min(p.rows, rank * per), r1 = min(p.rows, r0 + per);
    const int part = ((p.num_blocks + ctas - 1) / ctas + 31) / 32 * 32;
    const int b0 = min(p.num_blocks, rank * part), b1 = min(p.num_blocks, b0 + part);

    // A thread's rows stay in registers over the barriers: the last block only where it
    // is shared, and its count.  One that is free may be another row's in a moment: no
    // token goes on there.
    Row row[kRows];
    int held[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int r = r0 + tid + k * kRankThreads;
        row[k] = {0, 0, kKept};
        held[k] = 0;
        if (r >= r1)
            continue;
        row[k] = read_row(p, r);
        if (row[k].last >= 0) {
            held[k] = p.refs[row[k].last];
            if (held[k] > 1)
                p.writers[row[k].last] = 0, p.latest[row[k].last] = -1;
            else
                row[k].last = held[k] == 1 ? kKept : kLost;
            if (row[k].last == kLost)
                atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
        }
    }
    const int free_here = sum_of(my_free(p.refs, b0, b1), counts);
    cluster_sync();
#pragma unroll
    for (int k = 0; k < kRows; ++k)
        if (row[k].last >= 0) {
            atomicAdd(p.writers + row[k].last, 1);
            atomicMax(p.latest + row[k].last, r0 + tid + k * kRankThreads);
        }
    cluster_sync();
    constexpr int64_t low = (1ll << kCopyBit) - 1;
    int64_t needs = 0, tokens = 0, begin[kRows], token[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        if (r0 + k * kRankThreads >= r1) // no thread has a row
            continue;
        Row &x = row[k];
        const int r = r0 + tid + k * kRankThreads;
        if (x.last >= 0 && __ldcg(p.writers + x.last) == held[k] && __ldcg(p.latest + x.last) == r)
            x.last = kKept;
        // need: blocks below kCopyBit, rows that copy above
        int64_t v[2] = {blocks_of(x.len + x.fresh, p.block_size) - blocks_of(x.len, p.block_size), x.fresh};
        if (x.last >= 0)
            v[0] += 1 + (1ll << kCopyBit);
        int64_t all[2];
        prefix(v, sums, all);
        begin[k] = needs + v[0];
        token[k] = tokens + v[1];
        needs += all[0], tokens += all[1];
    }
    if (tid == 0)
        p.told[rank].v[0] = needs, p.told[rank].v[1] = tokens, p.told[rank].v[2] = free_here;
    cluster_sync();
    int64_t before[3], all[3];
    hear(p.told, rank, ctas, before, all);
    const int64_t need_before = before[0], new_before = before[1], free_before = before[2];
    const int64_t need_all = all[0], total = all[1], free = all[2], want = need_all & low;
    const bool ok = want <= free && total <= p.num_tokens;
    if (rank == 0 && tid == 0) {
        if (!ok)
            atomicOr(p.err, PA_DEVERR_POOL_);
        p.info[0] = (int)min(want, (int64_t)INT32_MAX);
        p.info[1] = (int)max(free - want, -(int64_t)INT32_MAX);
        p.head[0] = ok ? (int)total : 0;
        p.head[1] = ok ? (int)(need_all >> kCopyBit) : 0;
    }
    const int take = ok ? (int)want : 0;
    if (take > free_before || p.refs_out != p.refs)
        ranked(p.refs, b0, b1, counts, [&](int id, int refs, int before) {
            const int k = before + (int)free_before;
            const bool taken = refs == 0 && k < take;
            if (taken)
                p.free_ids[k] = id;
            if (taken || p.refs_out != p.refs)
                p.refs_out[id] = taken ? 1 : refs;
        });
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int r = r0 + tid + k * kRankThreads;
        if (r >= r1)
            continue;
        const Row &x = row[k];
        const bool copies = ok && x.last >= 0;
        const int64_t need = need_before + begin[k];
        p.row_len[r] = x.len;
        p.row_new[r] = ok ? x.fresh : 0;
        p.row_copy[r] = copies || x.last < 0 ? x.last : kKept;
        p.row_begin[r] = (int)(need & low);
        p.row_token[r] = ok ? (int)(new_before + token[k]) : 0;
        p.lens_out[r] = x.len + (ok ? x.fresh : 0);
        if (copies)
            p.copy_rows[need >> kCopyBit] = r;
    }
    cluster_sync();
#pragma unroll
    for (int k = 0; k < kRows; ++k)
        if (ok && row[k].last >= 0)
            atomicSub(p.refs_out + row[k].last, 1);
}

// The tables, the slots and the copies of extend: items of one list, CTA after
// CTA.  Bound by the copies' bytes where there are any, else by latency.
__global__ void __launch_bounds__(kThreads) extend_apply_kernel(const ExtendParams p,
                                                                const __grid_constant__ Pools ps)
{
    griddep_wait();
    const int tid = threadIdx.x, tokens = p.head[0], bs = p.block_size;
    const int64_t copies = (int64_t)p.head[1] * ps.units;
    const int chunks = (p.max_blocks + kChunk - 1) / kChunk;
    const int64_t entries = (int64_t)p.rows * chunks;
    const int64_t items = copies + entries + (p.num_tokens + kThreads - 1) / kThreads;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        if (item < copies) {
            const int r = p.copy_rows[item / ps.units];
            copy_unit(ps, (int)(item % ps.units), p.row_copy[r], p.free_ids[p.row_begin[r]]);
            continue;
        }
        if (item < copies + entries) {
            const int r = (int)((item - copies) / chunks);
            const int base = (int)((item - copies) % chunks) * kChunk;
            const int len = p.row_len[r], kept = blocks_of(len, bs) - (p.row_copy[r] >= 0);
            const int end = min(base + kChunk, blocks_of(len + p.row_new[r], bs));
            const int32_t *const got = p.free_ids + p.row_begin[r] - kept;
            const int64_t row = (int64_t)r * p.max_blocks;
            for (int j = base + tid; j < end; j += kThreads)
                if (j >= kept) {
                    p.tables_out[row + j] = got[j];
                } else {
                    const int b = p.tables[row + j];
                    if (b < 0 || b >= p.num_blocks)
                        atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
                    if (p.tables_out != p.tables)
                        p.tables_out[row + j] = b;
                }
            continue;
        }
        const int64_t t64 = (item - copies - entries) * kThreads + tid;
        if (t64 >= p.num_tokens)
            continue;
        const int t = (int)t64;
        int64_t slot = -1;
        if (t < tokens) {
            int lo = 0, hi = p.rows - 1; // the last row whose tokens begin at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (p.row_token[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int len = p.row_len[lo], pos = len + t - p.row_token[lo], j = pos / bs;
            const int kept = blocks_of(len, bs) - (p.row_copy[lo] >= 0);
            const int block = j < kept ? p.tables[(int64_t)lo * p.max_blocks + j]
                                       : p.free_ids[p.row_begin[lo] + j - kept];
            const bool lost = j < kept && p.row_copy[lo] == kLost;
            if (block >= 0 && block < p.num_blocks && !lost)
                slot = (int64_t)block * bs + pos % bs;
        }
        p.slots[t] = slot;
    }
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
struct CompactParams {
    int32_t *tables_out, *refs_out, *new_ids, *info;
    const int32_t *tables, *lens, *refs;
    unsigned int *err;
    int32_t *holes, *movers; // workspace: free ids below the live blocks' number, and what goes there
    Told *told;
    int32_t *head;           // live blocks below their number; blocks that move
    int rows, num_blocks, max_blocks, block_size, len_cap;
};

// One cluster: with n live blocks, the k-th live id at or above n moves to the
// k-th free id below n.  Two passes over the counts, bound by their latency as
// extend_rank_kernel: where nothing moves the call takes 10 us in a pool of 1000 blocks
// and 15 in one of 40000 (with one CTA in place of eight 10 and 33).
__global__ void __launch_bounds__(kRankThreads) compact_rank_kernel(const CompactParams p)
{
    __shared__ int counts[32];
    griddep_wait();
    const int rank = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x;
    const int part = ((p.num_blocks + ctas - 1) / ctas + 31) / 32 * 32;
    const int b0 = min(p.num_blocks, rank * part), b1 = min(p.num_blocks, b0 + part);
    const int mine = sum_of(my_free(p.refs, b0, b1), counts);
    if (tid == 0)
        p.told[rank].v[0] = mine;
    cluster_sync();
    int64_t before[1], all[1];
    hear(p.told, rank, ctas, before, all);
    const int free_before = (int)before[0], free = (int)all[0];
    const int n = p.num_blocks - free;
    ranked(p.refs, b0, b1, counts, [&](int id, int refs, int before) {
        const int f = before + free_before, live = id - f; // free and live ids below this one
        if (id == n)
            p.head[0] = live;
        // what moves is marked with its rank for the second pass
        p.new_ids[id] = refs == 0 ? -1 : id < n ? id : -2 - live;
        if (refs == 0 && id < n)
            p.holes[f] = id;
    });
    cluster_sync();
    const int low = n == p.num_blocks ? n : __ldcg(p.head); // live ids below n
    if (rank == 0 && tid == 0) {
        p.info[0] = n;
        p.info[1] = n - low;
        p.head[1] = n - low;
    }
    for (int id = b0 + tid; id < b1; id += kRankThreads) {
        const int x = p.new_ids[id];
        if (x <= -2) {
            const int k = -2 - x - low, to = __ldcg(p.holes + k);
            const int refs = p.refs[id];
            p.movers[k] = id;
            p.new_ids[id] = to;
            p.refs_out[to] = refs;
            p.refs_out[id] = 0;
        } else if (p.refs_out != p.refs && (x >= 0 || id >= n)) {
            p.refs_out[id] = x >= 0 ? p.refs[id] : 0; // a hole's is written by what goes there
        }
    }
}

// The moves and the tables of compact; as extend_apply_kernel.
__global__ void __launch_bounds__(kThreads) compact_apply_kernel(const CompactParams p,
                                                                 const __grid_constant__ Pools ps)
{
    griddep_wait();
    const int64_t copies = (int64_t)p.head[1] * ps.units;
    const int chunks = (p.max_blocks + kChunk - 1) / kChunk;
    const int64_t items = copies + (int64_t)p.rows * chunks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        if (item < copies) {
            const int k = (int)(item / ps.units);
            copy_unit(ps, (int)(item % ps.units), p.movers[k], p.holes[k]);
            continue;
        }
        const int r = (int)((item - copies) / chunks);
        const int base = (int)((item - copies) % chunks) * kChunk;
        const int len = length_of(p.lens, r, p.len_cap, base == 0 && threadIdx.x == 0, p.err);
        const int end = min(base + kChunk, blocks_of(len, p.block_size));
        const int64_t row = (int64_t)r * p.max_blocks;
        for (int j = base + threadIdx.x; j < end; j += kThreads) {
            const int b = p.tables[row + j];
            int to = -1;
            if (b >= 0 && b < p.num_blocks)
                to = p.new_ids[b];
            if (to < 0)
                atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
            p.tables_out[row + j] = to;
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// An array of a call; of an output, the input that it may be.
struct Span {
    const void *at;
    int64_t bytes;
    const void *self;
};

// Whether an output lies on another output, or on an input that it may not be.
template <int N, int M> static bool overlap(const Span (&out)[N], const Span (&in)[M])
{
    auto meet = [](const Span &a, const Span &b) {
        const char *x = static_cast<const char *>(a.at), *y = static_cast<const char *>(b.at);
        return a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
    };
    for (int i = 0; i < N; ++i) {
        for (int k = 0; k < i; ++k)
            if (meet(out[i], out[k]))
                return true;
        for (const Span &x : in)
            if (!(x.at == out[i].at && x.at == out[i].self) && meet(out[i], x))
                return true;
    }
    return false;
}

// Rows and blocks of the tables and counts.
static pa_status check_sizes(int rows, int num_blocks, int max_blocks, int block_size)
{
    if (rows < 0 || num_blocks <= 0 || max_blocks <= 0 || block_size <= 0)
        return PA_ERR_INVALID_ARG;
    if (rows > 65535 || (int64_t)max_blocks * block_size > INT32_MAX ||
        num_blocks > (1 << 29) || (max_blocks - 1) / kChunk + 1 > 65535)
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Launch on one cluster, after the kernel before.
template <typename P>
static cudaError_t launch_cluster(void (*kern)(const P), cudaStream_t s, const P &p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kRankThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

static pa_status read_pools(Pools *to, const pa_block_pool *from, int count, int num_blocks)
{
    if (count < 0 || (count > 0 && !from))
        return PA_ERR_INVALID_ARG;
    if (count > PA_MAX_POOLS)
        return PA_ERR_UNSUPPORTED;
    int64_t units = 0;
    for (int i = 0; i < count; ++i) {
        const pa_block_pool &f = from[i];
        if (!f.data || f.block_bytes <= 0 || f.planes <= 0)
            return PA_ERR_INVALID_ARG;
        Pool &p = to->pool[i];
        p.data = static_cast<uint8_t *>(f.data);
        p.block_bytes = f.block_bytes;
        p.plane_bytes = f.block_bytes * num_blocks;
        p.planes = f.planes;
        p.first_unit = (int)units;
        const int64_t each = (f.block_bytes + kUnit - 1) / kUnit;
        p.plane_units = (int)each;
        const uintptr_t all = reinterpret_cast<uintptr_t>(f.data) | (uintptr_t)f.block_bytes;
        p.width = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
        units += each * f.planes;
        if (f.block_bytes > ((int64_t)1 << 40) / num_blocks || units > (1 << 30))
            return PA_ERR_UNSUPPORTED;
    }
    to->count = count;
    to->units = (int)units;
    return PA_OK;
}

template <typename P>
static cudaError_t launch_apply(void (*kern)(const P, const Pools), const P &p, const Pools &ps,
                                int64_t items, cudaStream_t s)
{
    cudaError_t e;
    const int sms = sm_count(&e);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(items, (int64_t)sms * 8)));
    return launch_after_previous(kern, grid, dim3(kThreads), 0, s, p, ps);
}

} // namespace seqs
} // namespace pa

using namespace pa;
using namespace pa::seqs;

extern "C" {

pa_status pa_fork_sequences(int32_t *tables_out, int32_t *seq_lens_out, int32_t *ref_counts_out,
                            const int32_t *block_tables, const int32_t *seq_lens,
                            const int32_t *ref_counts, const int32_t *parents, int num_seqs,
                            int num_seqs_out, int num_blocks, int max_blocks_per_seq,
                            int block_size, void *stream)
{
    pa_status st = check_sizes(num_seqs, num_blocks, max_blocks_per_seq, block_size);
    if (st == PA_OK)
        st = check_sizes(num_seqs_out, num_blocks, max_blocks_per_seq, block_size);
    if (st != PA_OK)
        return st;
    if (!ref_counts || !ref_counts_out || !aligned(ref_counts, 4) || !aligned(ref_counts_out, 4) ||
        (num_seqs > 0 && (!block_tables || !seq_lens)) ||
        (num_seqs_out > 0 && (!tables_out || !seq_lens_out || !parents)) ||
        !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(tables_out, 4) ||
        !aligned(seq_lens_out, 4) || !aligned(parents, 4))
        return PA_ERR_INVALID_ARG;
    const int64_t wide = 4ll * max_blocks_per_seq, counts = 4ll * num_blocks;
    // rows trade places, so that they cannot be written where others are read
    const Span out[] = {{tables_out, num_seqs_out * wide, nullptr},
                        {seq_lens_out, num_seqs_out * 4ll, nullptr},
                        {ref_counts_out, counts, ref_counts}};
    const Span in[] = {{block_tables, num_seqs * wide}, {seq_lens, num_seqs * 4ll}, {ref_counts, counts},
                       {parents, num_seqs_out * 4ll}};
    if (overlap(out, in))
        return PA_ERR_INVALID_ARG;
    cudaError_t e;
    ForkParams p = {};
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    p.tables_out = tables_out;
    p.lens_out = seq_lens_out;
    p.refs = ref_counts_out;
    p.tables = block_tables;
    p.lens = seq_lens;
    p.parents = parents;
    p.rows_in = num_seqs;
    p.rows_out = num_seqs_out;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.len_cap = max_blocks_per_seq * block_size;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ref_counts_out != ref_counts) {
        const unsigned n = (unsigned)((num_blocks + 4 * kThreads - 1) / (4 * kThreads));
        if (launch_after_previous(copy_counts_kernel, dim3(n), dim3(kThreads), 0, s, ref_counts_out,
                                  ref_counts, num_blocks) != cudaSuccess)
            return PA_ERR_CUDA;
    }
    const int rows = std::max(num_seqs, num_seqs_out);
    if (rows == 0)
        return PA_OK;
    const dim3 grid(rows, (max_blocks_per_seq + kChunk - 1) / kChunk);
    return launch_after_previous(fork_kernel, grid, dim3(kThreads), 0, s, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

size_t pa_sequences_workspace_size(int num_seqs, int num_blocks)
{
    if (check_sizes(num_seqs, num_blocks, 1, 1) != PA_OK)
        return 0;
    // the CTAs' sums and two numbers, three numbers a block, six a row
    return kCluster * sizeof(Told) + 16 + 4 * (3 * (size_t)num_blocks + 6 * (size_t)num_seqs);
}

pa_status pa_extend_sequences(int32_t *tables_out, int32_t *seq_lens_out, int32_t *ref_counts_out,
                              int64_t *slot_mapping, int32_t *info, const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *ref_counts,
                              const int32_t *num_new, const pa_block_pool *pools, int num_pools,
                              int num_seqs, int num_tokens, int num_blocks, int max_blocks_per_seq,
                              int block_size, void *workspace, size_t workspace_bytes, void *stream)
{
    pa_status st = check_sizes(num_seqs, num_blocks, max_blocks_per_seq, block_size);
    if (st != PA_OK)
        return st;
    if (num_tokens < 0 || !info || !ref_counts || !ref_counts_out || (num_tokens > 0 && !slot_mapping) ||
        (num_seqs > 0 &&
         (!tables_out || !seq_lens_out || !block_tables || !seq_lens || !num_new)) ||
        !aligned(tables_out, 4) || !aligned(seq_lens_out, 4) || !aligned(ref_counts_out, 4) ||
        !aligned(slot_mapping, 8) || !aligned(info, 4) || !aligned(block_tables, 4) ||
        !aligned(seq_lens, 4) || !aligned(ref_counts, 4) || !aligned(num_new, 4))
        return PA_ERR_INVALID_ARG;
    const int64_t wide = 4ll * num_seqs * max_blocks_per_seq, rows = 4ll * num_seqs,
                  counts = 4ll * num_blocks;
    const int64_t needed = (int64_t)pa_sequences_workspace_size(num_seqs, num_blocks);
    const Span out[] = {{tables_out, wide, block_tables}, {seq_lens_out, rows, seq_lens},
                        {ref_counts_out, counts, ref_counts}, {slot_mapping, 8ll * num_tokens, nullptr},
                        {info, 8, nullptr}, {workspace, needed, nullptr}};
    const Span in[] = {{block_tables, wide}, {seq_lens, rows}, {ref_counts, counts}, {num_new, rows}};
    if (overlap(out, in))
        return PA_ERR_INVALID_ARG;
    Pools ps;
    st = read_pools(&ps, pools, num_pools, num_blocks);
    if (st != PA_OK)
        return st;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < (size_t)needed)
        return PA_ERR_WORKSPACE;
    cudaError_t e;
    ExtendParams p = {};
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    p.tables_out = tables_out;
    p.lens_out = seq_lens_out;
    p.refs_out = ref_counts_out;
    p.info = info;
    p.slots = slot_mapping;
    p.tables = block_tables;
    p.lens = seq_lens;
    p.refs = ref_counts;
    p.num_new = num_new;
    p.told = static_cast<Told *>(workspace);
    p.head = reinterpret_cast<int32_t *>(p.told + kCluster);
    p.writers = p.head + 4;
    p.latest = p.writers + num_blocks;
    p.free_ids = p.latest + num_blocks;
    p.row_len = p.free_ids + num_blocks;
    p.row_new = p.row_len + num_seqs;
    p.row_begin = p.row_new + num_seqs;
    p.row_token = p.row_begin + num_seqs;
    p.row_copy = p.row_token + num_seqs;
    p.copy_rows = p.row_copy + num_seqs;
    p.rows = num_seqs;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.len_cap = max_blocks_per_seq * block_size;
    p.num_tokens = num_tokens;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (launch_cluster(extend_rank_kernel, s, p) != cudaSuccess)
        return PA_ERR_CUDA;
    // as many items as there can be: every row may copy its last block
    const int64_t items = (int64_t)num_seqs * ((max_blocks_per_seq + kChunk - 1) / kChunk) +
                          (num_tokens + kThreads - 1) / kThreads + (int64_t)num_seqs * ps.units;
    e = launch_apply(extend_apply_kernel, p, ps, items, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_compact_blocks(int32_t *tables_out, int32_t *ref_counts_out, int32_t *new_ids,
                            int32_t *info, const int32_t *block_tables, const int32_t *seq_lens,
                            const int32_t *ref_counts, const pa_block_pool *pools, int num_pools,
                            int num_seqs, int num_blocks, int max_blocks_per_seq, int block_size,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    pa_status st = check_sizes(num_seqs, num_blocks, max_blocks_per_seq, block_size);
    if (st != PA_OK)
        return st;
    if (!info || !new_ids || !ref_counts || !ref_counts_out ||
        (num_seqs > 0 && (!tables_out || !block_tables || !seq_lens)) || !aligned(tables_out, 4) ||
        !aligned(ref_counts_out, 4) || !aligned(new_ids, 4) || !aligned(info, 4) ||
        !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(ref_counts, 4))
        return PA_ERR_INVALID_ARG;
    const int64_t wide = 4ll * num_seqs * max_blocks_per_seq, counts = 4ll * num_blocks;
    const int64_t needed = (int64_t)pa_sequences_workspace_size(num_seqs, num_blocks);
    const Span out[] = {{tables_out, wide, block_tables}, {ref_counts_out, counts, ref_counts},
                        {new_ids, counts, nullptr}, {info, 8, nullptr}, {workspace, needed, nullptr}};
    const Span in[] = {{block_tables, wide}, {seq_lens, 4ll * num_seqs}, {ref_counts, counts}};
    if (overlap(out, in))
        return PA_ERR_INVALID_ARG;
    Pools ps;
    st = read_pools(&ps, pools, num_pools, num_blocks);
    if (st != PA_OK)
        return st;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < (size_t)needed)
        return PA_ERR_WORKSPACE;
    cudaError_t e;
    CompactParams p = {};
    p.err = device_error_word(&e);
    if (!p.err)
        return PA_ERR_CUDA;
    p.tables_out = tables_out;
    p.refs_out = ref_counts_out;
    p.new_ids = new_ids;
    p.info = info;
    p.tables = block_tables;
    p.lens = seq_lens;
    p.refs = ref_counts;
    p.told = static_cast<Told *>(workspace);
    p.head = reinterpret_cast<int32_t *>(p.told + kCluster);
    p.holes = p.head + 4;
    p.movers = p.holes + num_blocks;
    p.rows = num_seqs;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.len_cap = max_blocks_per_seq * block_size;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (launch_cluster(compact_rank_kernel, s, p) != cudaSuccess)
        return PA_ERR_CUDA;
    const int64_t items = (int64_t)num_seqs * ((max_blocks_per_seq + kChunk - 1) / kChunk) +
                          (int64_t)num_blocks * ps.units;
    e = launch_apply(compact_apply_kernel, p, ps, items, s);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

} // extern "C"
