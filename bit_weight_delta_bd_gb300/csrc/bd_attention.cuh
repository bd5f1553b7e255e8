// What the attention kernels share: how the work of a call is cut into items
// and dealt to the blocks, where partial results go, and how they are joined.
//
// Rows.  The query rows that share a kv head are the G = n_q / n_kv heads of
// each new token: row r of sequence s is token q_off[s] + r / G, head
// h * G + r % G.  An item is up to MB consecutive rows of one sequence; its
// keys are 0 .. kv_end - 1 (kv_end = what its last row sees), cut into tiles.
//
// Dealing.  The units (item, kv head, tile), in this order, are dealt to the
// blocks in equal consecutive ranges: block c of N takes units c U / N up to
// (c + 1) U / N.  So every block streams the same number of tiles whatever
// the lengths are, a long sequence is split over many blocks, and a short
// one shares its block with others.  A block that does not see all tiles of
// an (item, head) leaves its unnormalised sum, maximum and denominator in the
// workspace; at most its first and its last are of that kind.  The second
// block of such an (item, head) notes it down, and the join adds its parts in
// block order, so results do not depend on timing.
// (The decode kernel does without a deal where caches are short or few.)
//
// Finding its units.  The decode kernel's blocks work the deal out from the
// lengths by themselves (one load per sequence and a scan: no launch before
// theirs, which is what a small call's time would go into); for chunks, whose
// items differ in length within a sequence, a one-block kernel lists the
// items first.
#pragma once

#include "bd_device.cuh"

namespace bd {

constexpr int kAttnMaxBlocks = 456;       // blocks of a launch at most: three for each of 152 SMs
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnItem {
    int seq;
    int row0;    // first row in the sequence
    int tiles;   // key tiles of one head (at least 1)
    int before;  // tiles of one head of the items before this one
};

// The (item, head) whose parts the join adds at block c: parts of blocks
// c - 1 .. c + parts - 2; parts == 0: none.  With all that the join has to
// know of the sequence, so that it need not look it up.
struct AttnJoin {
    int q0, rows;  // of the sequence: its first token, and its rows
    int row0, h, parts;
};

struct AttnHeader {
    int n_items;
    int tiles;  // of one head, over all items
};

struct AttnParams {
    AttentionArgs a;
    int G;                // query heads of a kv head
    int tile, mb;         // keys per tile, rows per item
    int blocks;           // N
    int rows_above, rows_upto;  // sequences with no more, or more, rows than these are another launch's
    int whole;            // a cluster of so many blocks for each (sequence, head), and no deal (decode kernel); or 0
    AttnHeader* head;
    AttnItem* items;
    int32_t* item_off;    // [n_seq + 1] first item of a sequence
    AttnJoin* joins;      // [N]
    float* part_o;        // [2 N][mb][dim]
    float2* part_ml;      // [2 N][mb] (maximum in log2 units, denominator)
};

// A sequence's lengths, clamped to what is in range.
struct AttnSeq {
    int q0, n_new;  // first token and number of new tokens
    int len;        // keys in the cache
};

__device__ __forceinline__ AttnSeq attn_seq(const AttentionArgs& a, int s, bool report)
{
    AttnSeq r;
    const int64_t T = a.T;
    const int64_t cap = a.max_pages << a.cache.page_shift;
    int64_t q0 = a.q_off[s], q1 = a.q_off[s + 1], len = a.kv_len[s];
    const bool bad = q0 < 0 || q0 > T || q1 < q0 || q1 > T || len < 0 || len > cap;
    if (bad) {
        if (report) raise_error(a.err, kErrBadIndex);
        q0 = q0 < 0 ? 0 : q0 > T ? T : q0;
        q1 = q1 < q0 ? q0 : q1 > T ? T : q1;
        len = len < 0 ? 0 : len > cap ? cap : len;
    }
    r.q0 = static_cast<int>(q0);
    r.n_new = static_cast<int>(q1 - q0);
    r.len = static_cast<int>(len);
    return r;
}

// The same, without new tokens where the sequence is another launch's.
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int s, bool report)
{
    AttnSeq r = attn_seq(p.a, s, report);
    const int64_t rows = static_cast<int64_t>(r.n_new) * p.G;
    if (rows <= p.rows_above || rows > p.rows_upto) r.n_new = 0;
    return r;
}

// Keys that token i of the sequence sees: 0 .. seen - 1.
__device__ __forceinline__ int attn_seen(const AttnSeq& s, int i, int causal)
{
    if (!causal) return s.len;
    const int64_t e = static_cast<int64_t>(s.len) - s.n_new + i + 1;
    return e < 0 ? 0 : e > s.len ? s.len : static_cast<int>(e);
}

// Number of blocks that take part, and the first unit of block c.  (Few units,
// the usual case: 32-bit divisions, which take a fraction of the time of
// 64-bit ones, and a block makes several before it can start.)
__device__ __forceinline__ int attn_active(int64_t units, int blocks)
{
    return units < blocks ? static_cast<int>(units) : blocks;
}
constexpr int64_t kAttnFewUnits = 0xFFFFFFFFll / (kAttnMaxBlocks + 1) - 1;
__device__ __forceinline__ int64_t attn_first(int64_t units, int n, int c)
{
    if (units < kAttnFewUnits)
        return static_cast<uint32_t>(units) * static_cast<uint32_t>(c) / static_cast<uint32_t>(n);
    return units * c / n;
}
// The block that takes unit u: the last c with attn_first(c) <= u.
__device__ __forceinline__ int attn_owner(int64_t units, int n, int64_t u)
{
    if (units < kAttnFewUnits)
        return static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(n) - 1u) /
                                static_cast<uint32_t>(units));
    return static_cast<int>(((u + 1) * n - 1) / units);
}
// rel / tiles for 0 <= rel < tiles * n_kv
__device__ __forceinline__ int attn_div(int64_t rel, int tiles)
{
    return rel <= 0xFFFFFFFFll ? static_cast<int>(static_cast<uint32_t>(rel) / static_cast<uint32_t>(tiles))
                               : static_cast<int>(rel / tiles);
}

// What block c, whose first unit u lies in the (item, head) with units
// [start, start + tiles), notes down for the join.
__device__ __forceinline__ AttnJoin attn_join_of(int64_t units, int n, int c, int64_t u, int64_t start, int tiles,
                                                 const AttnSeq& sq, int G, int row0, int h)
{
    AttnJoin j{sq.q0, sq.n_new * G, row0, h, 0};
    if (start != u && attn_owner(units, n, start) == c - 1) j.parts = attn_owner(units, n, start + tiles - 1) - c + 2;
    return j;
}

// The item that unit u belongs to: the last i with n_kv * before <= u.  All
// 32 lanes of a warp call it together.
__device__ __forceinline__ int attn_find_item(const AttnItem* items, int n_items, int n_kv, int64_t u)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_items;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = i < lo + n && static_cast<int64_t>(n_kv) * items[i].before <= u;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int last = 31 - __clz(m | 1u);
        const int end = lo + n;
        lo += last * step;
        n = step < end - lo ? step : end - lo;
    }
    return lo;
}

// The slot of block c's partial result that starts at the (item, head)'s
// first tile (its last segment) or later (its first segment).
__device__ __forceinline__ int attn_slot(int c, bool from_start) { return 2 * c + (from_start ? 1 : 0); }

// Probabilities are formed as exp2(score - maximum + bias): what is far below
// the maximum stays a normal number when it is rounded to 16 bits, after the
// product with an int8 value's scale too.  Numerator and denominator carry
// the same factor; a stored maximum is the one less the bias.  (Sums overflow
// only for values above 2^80.)
template <bool INT8>
__device__ __forceinline__ constexpr float attn_bias()
{
    return INT8 ? 24.0f : 8.0f;
}

// The factor of a partial sum with maximum m and denominator l when it joins
// others under the maximum of all: 0 where it has seen no key.  (A maximum of
// -infinity with a denominator other than 0 is a row of NaN scores, which
// stays NaN.)
__device__ __forceinline__ float attn_weight(float m, float l, float m_all)
{
    if (m == -INFINITY) return l == 0.0f ? 0.0f : 1.0f;
    return exp2f(m - m_all);
}

// Log-sum-exp of a row; m is in units of log2, l == 0 marks a row that saw no key.
__device__ __forceinline__ float attn_lse(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2; }

// Few rows per sequence (bd_attention.cu): 8 or 16 rows an item, 64 keys a tile.
cudaError_t launch_attention_mma(const AttnParams& p, cudaStream_t stream);
// Chunks (bd_attention_chunk.cu): 256 or 512 rows an item, 128 keys a tile.
cudaError_t launch_attention_chunk(const AttnParams& p, cudaStream_t stream);
constexpr int kChunkTile = 128;
// CTA pairs: 512 rows an item
constexpr int kChunkRows = 256, kPairRows = 512;
constexpr int chunk_max_blocks(int rows) { return 152 * kChunkRows / rows; }  // of the deal: CTAs, or pairs

}  // namespace bd
