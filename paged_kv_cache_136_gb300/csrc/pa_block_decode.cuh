// pa_block_decode.cuh -- decode attention over whole or listed blocks of a
// 16-bit pool, or of an e4m3 pool with one scale for each (plane, block, kv
// head).
//
// For a sequence, a kv head and the (at most 8) query heads of its group:
//   out = sum_t softmax_t(scale * q . k_t) v_t
// over the tokens of the sequence, or of its listed blocks.  One pass: a warp
// takes 16 tokens of one kv head at a time, forms S^T = K Q^T (16 x 8) and
// O^T += V^T P (D x 8) with m16n8k16 products, and keeps the running maximum
// and normaliser of the softmax in fp32.
//
// A tile comes by one TMA copy (both planes of 16 rows) into the warp's own
// ring, and from there straight into the registers of the products.  The
// contraction index of a product is any permutation of the channels (S) or of
// the tokens (O) as long as both operands use the same one, and the rows of
// O^T are any permutation of the channels, so every lane takes 16-byte pieces:
//   K  lane 4g + t: rows token(g) and token(g) + 8, bytes 16t + 64c of the row;
//   V  lane 4g + t: rows token(2t), token(2t+1) and those + 8, bytes 16g of
//      each 128.
// With token(k) = k for even k, (k + 4) mod 8 for odd k, the eight lanes that
// read at once meet eight different 16-byte columns of the 128-byte swizzle.
// e4m3 codes become halves (exactly) in registers.
//
// Work.  Inside a CTA the (up to 8) warps are HG kv heads times 1, 2, 4 or 8
// interleaved tiles.  The host splits the work one of two ways, whichever costs
// less.  Cut: the (sequence, group of HG heads, 16-token tile) triples are laid
// out in one line and cut into equal runs, one for each CTA that fits at once,
// so that any mix of lengths balances; HG is the most, up to 8, that divide the
// kv heads.  A (sequence, group) that a cut divides leaves partial states, which
// a second kernel merges.  Whole: a CTA is one (sequence, group), HG any divisor
// of the kv heads, and nothing is merged.
//
// What bounds it.  HBM on long work: 8 sequences of 131072 tokens (64 query, 8
// kv heads, e4m3, 2.15 GB) take 321 to 327 us, 6.6 TB/s; 64 of up to 2048 with 32
// kv heads 90 us, 6.2 TB/s.  The products (m16n8k16: the 8 query rows of a group are
// the narrow side, so no part of a product is idle at 8) keep the tensor pipe
// busy for a quarter of that.  On listed blocks each 128- or 256-byte row of a head is
// read apart from its neighbours', which HBM serves at about 5.8 TB/s.  Tiles of
// 2 KB (e4m3, head_size 64) are bound by a warp's latency for a tile: about 2.4
// times the time of their bytes.  Besides, a launch takes 3.5 us until its first
// tiles are in, and a merge 3 to 5 us.
//
// e4m3 scales: the score takes the key scale; the value scale multiplies the
// probability before it is rounded to 16 bits.  The softmax's reference m is
// the maximum of score + log2(value scale), so that the largest product
// p * scale is 2^lift (2^15 in halves, see lift_of) and halves hold the products
// of every block to the same absolute precision.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "pa_block.cuh"
#include "pa_internal.h"

namespace pa {
namespace block {

constexpr int kWarps = 8;      // warps of a CTA, at most
constexpr int kMaxCtas = 456;  // CTAs of a launch that cuts, at most
constexpr int kTile = 16;      // tokens a warp takes at a time
constexpr int kMinRun = 4;     // tiles a warp takes at least before work is cut
constexpr int kTruncated = 512; // tiles of an e4m3 pool that a warp may sum without rounding

struct DecodeArgs {
    void *out;                 // [B, H, D]
    float *lse;                // [B, H] or NULL
    const void *q;             // [B, H, D]
    const float *scales;       // [2, NB, Hkv] (e4m3 pool)
    const int32_t *tables;     // [B, MB]
    const int32_t *seq_lens;   // [B]
    const int32_t *lists;      // [B, Hkv, K] block positions, or NULL: all blocks
    const int32_t *list_lens;  // [B]
    unsigned int *err;
    int4 *cuts;                // [CTAs] {sequence, head group, CTAs sharing it, -}
    float *ws_o;               // [CTAs, 2, HG * G, D]
    float *ws_ml;              // [CTAs, 2, HG * G, 2]
    int num_seqs, num_heads, num_kv_heads, group, num_groups, num_blocks, max_blocks,
        block_log2, max_listed, len_cap;
    int heads, tiles_at_once;  // warps of a CTA: kv heads times interleaved tiles
    int whole;                 // a CTA is one (sequence, head group): nothing is cut
    float qscale;              // scale * log2 e
};

// Tiles of sequence s, at least one (an empty sequence writes zeros).
__device__ __forceinline__ int tiles_of(const DecodeArgs &p, int s, bool report)
{
    int n;
    if (p.lists) {
        n = p.list_lens[s];
        if (n < 0 || n > p.max_listed) {
            if (report)
                atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
            n = n < 0 ? 0 : p.max_listed;
        }
        n <<= p.block_log2 - 4;
    } else {
        n = p.seq_lens[s];
        n = (min(max(n, 0), p.len_cap) + kTile - 1) / kTile;
    }
    return max(n, 1);
}

__device__ __forceinline__ int length_of(const DecodeArgs &p, int s, bool report)
{
    const int len = p.seq_lens[s];
    if (len >= 0 && len <= p.len_cap)
        return len;
    if (report)
        atomicOr(p.err, PA_DEVERR_SEQ_LEN_);
    return len < 0 ? 0 : p.len_cap;
}

// Where a tile's 16 tokens are: the first pool row, or -1 for a block outside
// the pool (read as zeros); how many of them count.  `listed`: entries of the
// sequence's lists.
__device__ __forceinline__ void locate(const DecodeArgs &p, int s, int head, int tile, int len,
                                       int listed, int &row, int &live)
{
    const int per = p.block_log2 - 4;
    int j = tile >> per;
    const int sub = tile & ((1 << per) - 1);
    const int blocks = (len + (1 << p.block_log2) - 1) >> p.block_log2;
    row = -1;
    live = 0;
    if (p.lists) {
        if (j >= listed)
            return;
        j = p.lists[((int64_t)s * p.num_kv_heads + head) * p.max_listed + j];
        if (j < 0)
            return; // padding
        if (j >= blocks) {
            atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
            return;
        }
    }
    live = j >= blocks ? 0 : max(0, min(kTile, len - (j << p.block_log2) - sub * kTile));
    if (live == 0)
        return;
    const int blk = p.tables[(int64_t)s * p.max_blocks + j];
    if (blk < 0 || blk >= p.num_blocks) {
        atomicOr(p.err, PA_DEVERR_BLOCK_ID_);
        return;
    }
    row = (blk << p.block_log2) + sub * kTile;
}

constexpr float kLn2 = 0.6931471805599453f;

// Probabilities and normalisers are carried times 2^lift.  In halves the
// largest probability is then 2^15, and the smallest that is not lost 2^-39 of
// it; bf16 has fp32's range and needs none.
template <typename M> constexpr float lift_of() { return std::is_same<M, __half>::value ? 15.f : 0.f; }

// Tiles of up to 4 KB: two CTAs of eight warps an SM, 12 KB of tiles in flight a
// warp.  Tiles of 8 KB: one CTA, 24 KB a warp.  (Three CTAs for 2 KB tiles, with
// 80 registers, were slower: 322 against 204 us for 227 sequences of up to 7111
// tokens, 8 kv heads of 64.)
template <bool E4M3, int D> constexpr int tile_bytes() { return 2 * kTile * D * (E4M3 ? 1 : 2); }
template <bool E4M3, int D> constexpr int ctas_per_sm() { return tile_bytes<E4M3, D>() > 4096 ? 1 : 2; }
template <bool E4M3, int D> constexpr int stages_of()
{
    return 24576 / ctas_per_sm<E4M3, D>() / tile_bytes<E4M3, D>();
}

// One tile of a warp's ring: whose it is, and its scales.
struct Meta {
    int live, seq, head, flags; // tokens that count; whose; kLast.. bits
    float k_scale, v_scale;
    uint64_t bar;               // completes when the tile has landed
};
constexpr int kLast = 1;   // the warp's last tile of its part of a (sequence, group)
constexpr int kBegins = 2; // that part begins the (sequence, group)
constexpr int kEnds = 4;   // ... and ends it

// Shared memory of a CTA: the rings (aligned to 1024), their Metas, and half of
// the states that a head's upper warps hand to its lower ones
// (none where every warp has a head of its own).
template <bool E4M3, int D> constexpr int decode_smem(int warps, bool hand_over)
{
    return 1024 + warps * stages_of<E4M3, D>() * (tile_bytes<E4M3, D>() + (int)sizeof(Meta)) +
           (hand_over ? warps / 2 * 4 * (D + 2) * 4 : 0);
}

// Where a warp's walk over its CTA's run stands.
struct Walk {
    int at, seq, tiles, grp, seg; // run position; (sequence, group), its tiles and first one
    int len, listed, next, left, flags; // of the part being walked: tokens, list entries, the
                                        // warp's next tile and how many it has left
};

__device__ __forceinline__ void tma_load_5d_hint(void *dst, const CUtensorMap *map, uint64_t *bar,
                                                 int c0, int c1, int c2, int c3, int c4,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
        "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two additions in one instruction, to nearest.
__device__ __forceinline__ void add2(float &a, float &b, float x, float y)
{
    asm("{ .reg .b64 s, t; mov.b64 s, {%0, %1}; mov.b64 t, {%2, %3}; add.rn.f32x2 s, s, t; "
        "mov.b64 {%0, %1}, s; }"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y));
}

// The running maximum starts here: finite, so that differences of maxima are
// never NaN, and below no score but -inf.
constexpr float kNone = -3.402823466e38f;

// T: type of q and out (and of a 16-bit pool).  E4M3: pool of e4m3 codes.
// NEAREST: a tile's value products begin at zero, and are added to the sums by
// additions that round to nearest; else they begin at the sums, to which the
// matrix unit adds by truncation.  That takes up to 2^-23 of the sum so far off
// it in each of a tile's two products (1.5e-3 measured in a run of 32768 tiles of
// one sign): at most 2^-13 in the kTruncated tiles it is used for, 2^-14 of a sum
// that grows evenly, where half a step of fp16 is 2^-12.  A 16-bit pool always rounds: it costs nothing there (30.6
// against 30.5 us at 8 x 131072 tokens, 128 blocks each).  An e4m3 pool, at 128
// registers, would take 83.5 instead of 79.0 us at 256 sequences of up to 4096
// and 330 instead of 327 at 8 x 131072, runs of up to 216 tiles.
//
// A warp fetches for itself, kStages tiles ahead: the lane that looked a tile
// up issues its copy, so nothing is handed from warp to warp before a part's
// end.
template <typename T, bool E4M3, int D, bool NEAREST>
__global__ void __launch_bounds__(32 * kWarps, ctas_per_sm<E4M3, D>())
    block_decode_kernel(const __grid_constant__ CUtensorMap pool_map, const DecodeArgs p)
{
    using M = typename std::conditional<E4M3, __half, T>::type; // type of the products
    constexpr float kLift = lift_of<M>();
    constexpr int kRow = D * (E4M3 ? 1 : 2);     // bytes of a head's row
    constexpr int kKPieces = kRow / 64;          // 16-byte pieces of a lane and row of K
    constexpr int kVWords = kRow / 32;           // words of a lane and row of V
    constexpr int kSteps = D / 16;               // products along D
    constexpr int kStages = stages_of<E4M3, D>();
    constexpr int kTileBytes = tile_bytes<E4M3, D>();
    extern __shared__ char smem_raw[];
    __shared__ int3 first; // sequence that the run begins in, its first tile, its tiles
    __shared__ int warp_sums[kWarps];
    __shared__ Walk walks[kWarps];

    char *const smem = smem_raw + (-smem_addr(smem_raw) & 1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int heads = p.heads, tws = p.tiles_at_once, warps = heads * tws;
    const int tw = warp / heads, hl = warp - tw * heads;
    char *const ring = smem + warp * kStages * kTileBytes;
    Meta *const meta = reinterpret_cast<Meta *>(smem + warps * kStages * kTileBytes) +
                       warp * kStages;
    float *const handed = reinterpret_cast<float *>(smem + warps * kStages *
                                                    (kTileBytes + (int)sizeof(Meta)));
    if (lane < kStages)
        mbar_init(&meta[lane].bar, 1);
    fence_barrier_init();
    if (tid == 0)
        prefetch_tensormap(&pool_map);
    __syncwarp();
    griddep_wait();

    // ---- this CTA's run: [begin, end) of the line of tiles ----
    int run = 0, begin = 0, end;
    int f_seq, f_tiles, f_grp, f_seg; // sequence and group that it begins in
    if (p.whole) {
        f_seq = blockIdx.x / p.num_groups;
        f_grp = blockIdx.x - f_seq * p.num_groups;
        f_seg = 0;
        end = f_tiles = tiles_of(p, f_seq, warp == 0);
    } else {
        const int slice = (p.num_seqs + 32 * warps - 1) / (32 * warps);
        const int s_lo = min(tid * slice, p.num_seqs), s_hi = min(s_lo + slice, p.num_seqs);
        int mine = 0;
        for (int s = s_lo; s < s_hi; ++s)
            mine += tiles_of(p, s, blockIdx.x == 0);
        mine *= p.num_groups;
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            warp_sums[warp] = x;
        __syncthreads();
        int base = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            base += w < warp ? warp_sums[w] : 0;
            total += w < warps ? warp_sums[w] : 0;
        }
        base += x - mine;
        run = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinRun * tws);
        begin = blockIdx.x * run;
        end = min(begin + run, total);
        if (tid == 0)
            p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
        if (begin >= total)
            return;
        if (begin >= base && begin < base + mine) {
            int s = s_lo, n = slice == 1 ? mine : tiles_of(p, s, false) * p.num_groups;
            while (begin >= base + n) {
                base += n;
                n = tiles_of(p, ++s, false) * p.num_groups;
            }
            first = make_int3(s, base, n);
        }
        __syncthreads();
        f_seq = first.x;
        f_tiles = first.z / p.num_groups;
        f_grp = (begin - first.y) / f_tiles;
        f_seg = first.y + f_grp * f_tiles;
    }

    // ---- the walk that fetches: one part of a (sequence, group) after the
    // other, in batches of 32 tiles whose places the lanes look up at once.
    // Its state is looked at once a batch and waits in shared memory. ----
    Walk &walk = walks[warp];
    if (lane == 0)
        walk = Walk{begin, f_seq, f_tiles, f_grp, f_seg, 0, 0, 0, 0, 0};
    __syncwarp();
    // The batch being fetched, and the one behind it: a lane's tile (first pool
    // row, scales, live | flags << 8 | batch's last tile ends the part << 12 |
    // tiles of the batch << 16) and whose it is (sequence << 16 | head).
    int b_row = 0, b_info = 0, b_whose = 0, b_i = 0, n_row = 0, n_info = 0, n_whose = 0;
    float b_ks = 1.f, b_vs = 1.f, n_ks = 1.f, n_vs = 1.f;

    auto look_up = [&]() { // fills the batch behind
        Walk w = walk;
        n_info = 0;
        if (w.left == 0) {
            if (w.at >= end)
                return;
            const int seg_end = w.seg + w.tiles, stop = min(end, seg_end);
            w.flags = (w.at == w.seg ? kBegins : 0) | (stop == seg_end ? kEnds : 0);
            w.len = length_of(p, w.seq, lane == 0 && warp == 0);
            w.listed = p.lists ? min(p.list_lens[w.seq], p.max_listed) : 0;
            w.next = w.at - w.seg + tw;
            // a warp without a tile takes an empty one: all meet at the part's end
            w.left = max(1, (stop - w.at - tw + tws - 1) / tws);
            if (stop - w.at <= tw)
                w.next = -1;
            if (tid == 0 && w.flags == kBegins)
                p.cuts[blockIdx.x] =
                    make_int4(w.seq, w.grp, (seg_end - 1) / run - (int)blockIdx.x + 1, 0);
            w.at = stop;
        }
        const int head = w.grp * heads + hl, n = min(32, w.left);
        n_whose = w.seq << 16 | head;
        w.left -= n;
        int live = 0;
        n_row = -1;
        if (lane < n && w.next >= 0)
            locate(p, w.seq, head, w.next + lane * tws, w.len, w.listed, n_row, live);
        n_info = live | w.flags << 8 | (w.left == 0 ? 1 << 12 : 0) | n << 16;
        if constexpr (E4M3) {
            n_ks = n_vs = 1.f;
            if (n_row >= 0) {
                const float *sc = p.scales + (int64_t)(n_row >> p.block_log2) * p.num_kv_heads +
                                  head;
                n_ks = *sc;
                n_vs = sc[(int64_t)p.num_blocks * p.num_kv_heads];
            }
        }
        w.next += 32 * tws;
        if (w.left == 0 && w.at == w.seg + w.tiles) {
            w.seg = w.at;
            if (++w.grp == p.num_groups) {
                w.grp = 0;
                if (++w.seq < p.num_seqs)
                    w.tiles = tiles_of(p, w.seq, false);
            }
        }
        __syncwarp();
        if (lane == 0)
            walk = w;
        __syncwarp();
    };

    const uint64_t policy = policy_evict_first();
    bool lost = false;
    auto fetch = [&](int stage) { // the next tile, or the end, into `stage`
        if (b_i == b_info >> 16) {
            b_row = n_row, b_info = n_info, b_whose = n_whose, b_ks = n_ks, b_vs = n_vs;
            b_i = 0;
            if (b_info >> 16)
                look_up();
        }
        Meta &m = meta[stage];
        if (b_i < b_info >> 16) {
            if (lane == b_i) {
                const int live = b_info & 255;
                const bool ends = b_info >> 12 & 1 && b_i + 1 == b_info >> 16;
                *reinterpret_cast<int4 *>(&m) =
                    make_int4(live, b_whose >> 16 & 0xFFFF, b_whose & 0xFFFF,
                              (b_info >> 8 & 15) | (ends ? kLast : 0));
                if (lost) {
                } else if (live) {
                    // a row past the pool reads as zeros
                    const int row = b_row < 0 ? p.num_blocks << p.block_log2 : b_row;
                    mbar_arrive_expect_tx(&m.bar, kTileBytes);
                    if constexpr (kRow == 256)
                        tma_load_5d_hint(ring + stage * kTileBytes, &pool_map, &m.bar, 0, row, 0,
                                         b_whose & 0xFFFF, 0, policy);
                    else if constexpr (kRow == 128)
                        tma_load_4d_hint(ring + stage * kTileBytes, &pool_map, &m.bar, 0, row,
                                         b_whose & 0xFFFF, 0, policy);
                    else // half a line of L2: the other half is another warp's
                        tma_load_4d(ring + stage * kTileBytes, &pool_map, &m.bar, 0, row,
                                    b_whose & 0xFFFF, 0);
                    if constexpr (E4M3)
                        *reinterpret_cast<float2 *>(&m.k_scale) = make_float2(b_ks, b_vs);
                } else {
                    mbar_arrive(&m.bar);
                }
            }
            ++b_i;
        } else if (lane == 0) {
            m.flags = -1;
            if (!lost)
                mbar_arrive(&m.bar);
        }
    };

    look_up();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(i);

    // lane constants: token(g), and where the lane's pieces lie in a tile
    const int token = g & 1 ? (g + 4) & 7 : g;
    const int tok0 = 2 * t, tok1 = (2 * t + 5) & 7;
    const int k_at = kRow == 64 ? token * 64 + ((t ^ (token >> 1 & 3)) << 4)
                                : token * 128 + ((t ^ token) << 4);
    const int v_at0 = kRow == 64
                          ? tok0 * 64 + ((g >> 1 ^ (tok0 >> 1 & 3)) << 4) + (g & 1) * 8
                          : tok0 * 128 + ((g ^ tok0) << 4);
    const int v_at1 = kRow == 64
                          ? tok1 * 64 + ((g >> 1 ^ (tok1 >> 1 & 3)) << 4) + (g & 1) * 8
                          : tok1 * 128 + ((g ^ tok1) << 4);
    constexpr int kEight = 8 * (kRow == 64 ? 64 : 128); // eight rows further
    constexpr int kHalf = 16 * 128;                     // the row's second 128 bytes
    uint32_t qf[kSteps][2];
    float qmul0 = 0.f, qmul1 = 0.f;
    float o[kSteps][4];
    float m0 = kNone, m1 = kNone, l0 = 0.f, l1 = 0.f;
    bool fresh = true;
    int stage = 0, drain = 0;
    uint32_t parity = 0;
    while (true) {
        __syncwarp();
        const int4 info = *reinterpret_cast<const int4 *>(&meta[stage]);
        const int s = info.y, head = info.z, flags = info.w;
        if (flags < 0)
            break;
        if (fresh) { // a part begins: ask for the query rows of the group
            const T *q = static_cast<const T *>(p.q) +
                         ((int64_t)s * p.num_heads + head * p.group + min(g, p.group - 1)) * D;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int d = E4M3 ? (i / 4) * 64 + t * 16 + (i % 4) * 4
                                   : (i / 2) * 32 + t * 8 + (i % 2) * 4;
                const uint2 v = *reinterpret_cast<const uint2 *>(q + d);
                qf[i][0] = v.x, qf[i][1] = v.y;
            }
        }
        // A copy that does not arrive is reported; the warp then starts no
        // more, waits (within the limit) for those in flight, and walks on
        // without data, so that it still meets the others.
        if (!lost || drain > 0) {
            const bool here = __all_sync(~0u, mbar_wait(&meta[stage].bar, parity));
            if (lost) {
                --drain;
            } else if (!here) {
                lost = true;
                drain = kStages - 1;
                if (lane == 0)
                    atomicOr(p.err, PA_DEVERR_TIMEOUT_);
            }
        }
        const int live = lost ? 0 : info.x;

        if (fresh) {
            fresh = false;
            // The queries as the products take them; for e4m3 in halves, bf16
            // ones scaled by a power of two so that the largest is near 2^15
            // (they keep their 8 bits over 29 binades below it).
            qmul0 = qmul1 = p.qscale;
            if (g >= p.group)
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
                    qf[i][0] = qf[i][1] = 0;
            if constexpr (E4M3 && std::is_same<T, __nv_bfloat16>::value) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const float2 a = float2_of<T>(qf[i][0]), b = float2_of<T>(qf[i][1]);
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)),
                                             fmaxf(fabsf(b.x), fabsf(b.y))));
                }
                amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
                const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -120);
                const float down = two_to(-e);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const float2 a = float2_of<T>(qf[i][0]), b = float2_of<T>(qf[i][1]);
                    qf[i][0] = pair_of<__half>(a.x * down, a.y * down);
                    qf[i][1] = pair_of<__half>(b.x * down, b.y * down);
                }
                const float up = two_to(e);
                qmul0 *= __shfl_sync(~0u, up, 8 * t);
                qmul1 *= __shfl_sync(~0u, up, 8 * t + 4);
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[i][k] = 0.f;
            m0 = m1 = kNone;
            l0 = l1 = 0.f;
        }

        if (live) {
            const char *const slot = ring + stage * kTileBytes;
            float ks = 1.f, vs = 1.f;
            if constexpr (E4M3) {
                const float2 sc = *reinterpret_cast<const float2 *>(&meta[stage].k_scale);
                ks = sc.x;
                vs = sc.y;
            }
            // S^T: rows are token(g) and token(g) + 8, columns queries 2t and 2t + 1
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < kKPieces; ++j) {
                const char *const k = slot + (j >> 1) * kHalf + (k_at ^ (j & 1) * 64);
                const uint4 ka = *reinterpret_cast<const uint4 *>(k);
                const uint4 kb = *reinterpret_cast<const uint4 *>(k + kEight);
#pragma unroll
                for (int i = 0; i < (E4M3 ? 4 : 2); ++i) {
                    if constexpr (E4M3) {
                        const uint32_t a = (&ka.x)[i], b = (&kb.x)[i];
                        mma_16816<M>(c, half2_of_e4m3x2(a), half2_of_e4m3x2(b),
                                     half2_of_e4m3x2_hi(a), half2_of_e4m3x2_hi(b),
                                     qf[4 * j + i][0], qf[4 * j + i][1]);
                    } else {
                        mma_16816<M>(c, (&ka.x)[2 * i], (&kb.x)[2 * i], (&ka.x)[2 * i + 1],
                                     (&kb.x)[2 * i + 1], qf[2 * j + i][0], qf[2 * j + i][1]);
                    }
                }
            }
            // every lane has left the stage before this one: refill it, while the
            // products run
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            const float f0 = E4M3 ? qmul0 * ks : qmul0, f1 = E4M3 ? qmul1 * ks : qmul1;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                c[k] *= k & 1 ? f1 : f0;
            if (live < kTile) {
                if (token >= live)
                    c[0] = c[1] = -INFINITY;
                if (token + 8 >= live)
                    c[2] = c[3] = -INFINITY;
            }

            // running maximum of score + log2(value scale), over the 16 tokens
            float n0 = fmaxf(c[0], c[2]), n1 = fmaxf(c[1], c[3]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, off));
                n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, off));
            }
            if constexpr (E4M3) {
                const float lift = lg2(vs);
                n0 += lift;
                n1 += lift;
            }
            n0 = fmaxf(m0, n0);
            n1 = fmaxf(m1, n1);
            if (__any_sync(~0u, n0 != m0 || n1 != m1)) {
                const float a0 = ex2(m0 - n0), a1 = ex2(m1 - n1);
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    o[i][0] *= a0;
                    o[i][1] *= a1;
                    o[i][2] *= a0;
                    o[i][3] *= a1;
                }
                m0 = n0;
                m1 = n1;
            }
            const float r0 = m0 - kLift, r1 = m1 - kLift;
            c[0] = ex2(c[0] - r0);
            c[1] = ex2(c[1] - r1);
            c[2] = ex2(c[2] - r0);
            c[3] = ex2(c[3] - r1);
            l0 += c[0] + c[2];
            l1 += c[1] + c[3];
            if constexpr (E4M3)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    c[k] *= vs;
            // P as a 16-bit part and the rounded remainder: 22 bits in halves, 16 in
            // bf16.  One part alone (11, 8) would show where the values cancel.
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t h = pair_of<M>(c[2 * k], c[2 * k + 1]);
                const float2 back = float2_of<M>(h);
                hi[k] = transpose_8x8(h);
                lo[k] = transpose_8x8(pair_of<M>(c[2 * k] - back.x, c[2 * k + 1] - back.y));
            }

            // O^T: rows are channels 2i and 2i + 1 of each lane's list
            uint32_t vr[4][kVWords];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char *const v =
                    slot + kTileBytes / 2 + (i & 1 ? v_at1 : v_at0) + (i >> 1) * kEight;
                if constexpr (kRow == 64) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(v);
                    vr[i][0] = w.x, vr[i][1] = w.y;
                } else {
#pragma unroll
                    for (int k = 0; k < kVWords; k += 4) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(v + (k >> 2) * kHalf);
                        vr[i][k] = w.x, vr[i][k + 1] = w.y, vr[i][k + 2] = w.z, vr[i][k + 3] = w.w;
                    }
                }
            }
            if (live < kTile) { // what lies behind the last token may be NaN
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((i & 1 ? tok1 : tok0) + (i >> 1) * 8 >= live)
#pragma unroll
                        for (int k = 0; k < kVWords; ++k)
                            vr[i][k] = 0;
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                uint32_t a0, a1, a2, a3;
                if constexpr (E4M3) {
                    const uint32_t sel = i % 2 ? 0x7362 : 0x5140;
                    const uint32_t u = __byte_perm(vr[0][i / 2], vr[1][i / 2], sel);
                    const uint32_t v = __byte_perm(vr[2][i / 2], vr[3][i / 2], sel);
                    a0 = half2_of_e4m3x2(u);
                    a1 = half2_of_e4m3x2_hi(u);
                    a2 = half2_of_e4m3x2(v);
                    a3 = half2_of_e4m3x2_hi(v);
                } else {
                    a0 = __byte_perm(vr[0][i], vr[1][i], 0x5410);
                    a1 = __byte_perm(vr[0][i], vr[1][i], 0x7632);
                    a2 = __byte_perm(vr[2][i], vr[3][i], 0x5410);
                    a3 = __byte_perm(vr[2][i], vr[3][i], 0x7632);
                }
                if constexpr (NEAREST) {
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_16816<M>(part, a0, a1, a2, a3, hi[0], hi[1]);
                    mma_16816<M>(part, a0, a1, a2, a3, lo[0], lo[1]);
                    add2(o[i][0], o[i][1], part[0], part[1]);
                    add2(o[i][2], o[i][3], part[2], part[3]);
                } else {
                    mma_16816<M>(o[i], a0, a1, a2, a3, hi[0], hi[1]);
                    mma_16816<M>(o[i], a0, a1, a2, a3, lo[0], lo[1]);
                }
            }
        }
        else
            fetch(stage == 0 ? kStages - 1 : stage - 1);
        if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
        }

        if (!(flags & kLast))
            continue;
        fresh = true;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(~0u, l0, off);
            l1 += __shfl_xor_sync(~0u, l1, off);
        }

        // Join the warps that shared the head's tiles: half of the warps at a
        // time, and of their queries the even ones, then the odd ones.
        for (int half = tws >> 1; half; half >>= 1) {
            float *const box =
                handed + (((tw & (half - 1)) * heads + hl) * 4 + t) * (D + 2);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float &m = k ? m1 : m0, &l = k ? l1 : l0;
                if (tw >= half && tw < 2 * half) {
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
                        *reinterpret_cast<float2 *>(box + g * (D / 8) + 2 * i) =
                            make_float2(o[i][k], o[i][k + 2]);
                    if (g == 0)
                        *reinterpret_cast<float2 *>(box + D) = make_float2(m, l);
                }
                __syncthreads();
                if (tw < half) {
                    const float2 other = *reinterpret_cast<float2 *>(box + D);
                    const float top = fmaxf(m, other.x);
                    const float a = ex2(m - top), b = ex2(other.x - top);
                    l = l * a + b * other.y;
                    m = top;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        const float2 y = *reinterpret_cast<float2 *>(box + g * (D / 8) + 2 * i);
                        o[i][k] = o[i][k] * a + b * y.x;
                        o[i][k + 2] = o[i][k + 2] * a + b * y.y;
                    }
                }
                __syncthreads();
            }
        }
        if (tw != 0)
            continue;

        // A whole (sequence, group) is finished here; a cut one leaves its
        // state: slot 1 of the CTA that began it, slot 0 of the others.
        const bool whole = (flags & (kBegins | kEnds)) == (kBegins | kEnds);
        const int slot = flags & kBegins ? 1 : 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int col = 2 * t + k;
            if (col >= p.group)
                continue;
            const float l = k ? l1 : l0, m = k ? m1 : m0;
            if (whole) {
                const int64_t row = (int64_t)s * p.num_heads + head * p.group + col;
                const float inv = l != 0.f ? 1.f / l : 0.f;
                T *dst = static_cast<T *>(p.out) + row * D;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int d = E4M3 || D == 64 ? g * (D / 8) + 2 * i
                                                  : (i / 4) * 64 + g * 8 + (i % 4) * 2;
                    *reinterpret_cast<uint32_t *>(dst + d) =
                        pair_of<T>(o[i][k] * inv, o[i][k + 2] * inv);
                }
                if (p.lse && g == 0)
                    p.lse[row] = l != 0.f ? (m - kLift + log2f(l)) * kLn2 : -INFINITY;
            } else {
                const int64_t row =
                    ((int64_t)(2 * blockIdx.x + slot) * heads + hl) * p.group + col;
                float *dst = p.ws_o + row * D;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int d = E4M3 || D == 64 ? g * (D / 8) + 2 * i
                                                  : (i / 4) * 64 + g * 8 + (i % 4) * 2;
                    *reinterpret_cast<float2 *>(dst + d) = make_float2(o[i][k], o[i][k + 2]);
                }
                if (g == 0)
                    *reinterpret_cast<float2 *>(p.ws_ml + row * 2) = make_float2(m, l);
            }
        }
    }
    griddep_launch_dependents();
}

// Merge of the (sequence, group)s that a cut divides: with M = max m_i,
// out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  Every CTA lists the cuts;
// the (cut, query row) pairs then go round the warps, or round 3, 5 or all of a
// CTA's warps, which split the states, where there are many
// states and too few rows to fill the warps.  Bound by latency, so that what a
// row needs is asked for at once: four states' m, l and o at a time.
constexpr int kMergeWarps = 15; // a thread for each cut there can be
static_assert(32 * kMergeWarps >= kMaxCtas, "one look at the cuts");

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(32 * kMergeWarps, 2) block_merge_kernel(const DecodeArgs p, int ctas)
{
    constexpr float kLift = lift_of<typename std::conditional<E4M3, __half, T>::type>();
    constexpr int kCols = D / 32;                // columns of a lane
    constexpr int kAtOnce = 4;
    using Vec = typename std::conditional<kCols == 4, float4, float2>::type;
    __shared__ int4 list[kMaxCtas];              // sequence, head group, states, first CTA
    __shared__ int counts[kMergeWarps], most[kMergeWarps];
    __shared__ float part[kMergeWarps][D + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    int4 seen = make_int4(0, 0, 0, 0);
    if ((int)threadIdx.x < ctas)
        seen = p.cuts[threadIdx.x];
    seen.w = threadIdx.x;
    const unsigned some = __ballot_sync(~0u, seen.z >= 2);
    const int longest = __reduce_max_sync(~0u, seen.z);
    if (lane == 0) {
        counts[warp] = __popc(some);
        most[warp] = longest;
    }
    __syncthreads();
    int at = __popc(some & ((1u << lane) - 1)), found = 0, states = 0;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
        at += w < warp ? counts[w] : 0;
        found += counts[w];
        states = max(states, most[w]);
    }
    if (seen.z >= 2)
        list[at] = seen;
    __syncthreads();
    const int rows = p.group * p.heads, items = found * rows;
    // warps of a row: 1, 3, 5 or all 15, with some kAtOnce states each
    int each = 1;
#pragma unroll
    for (int e = 3; e <= 15; e = e == 3 ? 5 : e + 10)
        if (states > kAtOnce * (e - 1) && items * e <= (int)gridDim.x * kMergeWarps)
            each = e;
    const int at_once = kMergeWarps / each, mine = warp / each, lead = mine * each;
    for (int item0 = blockIdx.x * at_once; item0 < items; item0 += gridDim.x * at_once) {
        const int item = item0 + mine;
        const bool some_row = item < items;
        const int4 cut = some_row ? list[item / rows] : make_int4(0, 0, 0, 0);
        const int r = item % rows;
        float top = kNone, l = 0.f, acc[kCols];
#pragma unroll
        for (int k = 0; k < kCols; ++k)
            acc[k] = 0.f;
        for (int i0 = warp - lead; i0 < cut.z; i0 += kAtOnce * each) {
            float2 ml[kAtOnce];
            Vec v[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int i = i0 + j * each;
                // the state of the CTA that began the pair, or of one that went on
                const int64_t row = (int64_t)(2 * (cut.w + i) + (i == 0)) * rows + r;
                ml[j] = make_float2(kNone, 0.f);
                if (i < cut.z) {
                    ml[j] = *reinterpret_cast<const float2 *>(p.ws_ml + row * 2);
                    v[j] = reinterpret_cast<const Vec *>(p.ws_o + row * D)[lane];
                }
            }
            float now = top;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                now = fmaxf(now, ml[j].x);
            const float old = ex2(top - now);
            top = now;
            l *= old;
#pragma unroll
            for (int k = 0; k < kCols; ++k)
                acc[k] *= old;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (i0 + j * each >= cut.z)
                    continue;
                const float w = ex2(ml[j].x - now);
                l += w * ml[j].y;
                acc[0] += w * v[j].x;
                acc[1] += w * v[j].y;
                if constexpr (kCols == 4) {
                    acc[2] += w * v[j].z;
                    acc[3] += w * v[j].w;
                }
            }
        }
        if (each > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kCols; ++k)
                part[warp][lane * kCols + k] = acc[k];
            if (lane == 0) {
                part[warp][D] = top;
                part[warp][D + 1] = l;
            }
            __syncthreads();
            if (warp != lead)
                continue;
            for (int w = lead + 1; w < lead + min(each, cut.z); ++w) {
                const float now = fmaxf(top, part[w][D]);
                const float a = ex2(top - now), b = ex2(part[w][D] - now);
                top = now;
                l = l * a + b * part[w][D + 1];
#pragma unroll
                for (int k = 0; k < kCols; ++k)
                    acc[k] = acc[k] * a + b * part[w][lane * kCols + k];
            }
        }
        if (!some_row)
            continue;
        const int64_t row = (int64_t)cut.x * p.num_heads + (int64_t)cut.y * rows + r;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + row * D) +
                        lane * (kCols / 2);
#pragma unroll
        for (int k = 0; k < kCols; k += 2)
            dst[k / 2] = pair_of<T>(acc[k] * inv, acc[k + 1] * inv);
        if (p.lse && lane == 0)
            p.lse[row] = l != 0.f ? (top - kLift + log2f(l)) * kLn2 : -INFINITY;
    }
}

} // namespace block
} // namespace pa
