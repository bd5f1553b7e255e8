// Attention over the paged KV cache: the plan, the kernel for few query rows
// per sequence (decode steps), and the join of partial results.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp2(c q_r . k_j - m_r),  c = scale log2(e)
//
// in one pass over the keys with a running maximum m_r: where a tile raises
// it, the sums so far are multiplied by exp2(m_old - m_new).
//
// The decode kernel is bound by the cache's bytes.  One warp keeps a ring of
// stages (64 keys: K, V, scales) filled by TMA, one box per page; four
// consumer warps take turns, two of them 32 keys each of every other stage,
// with a running maximum, denominator and sum of their own, so that nothing is
// exchanged between warps until an item ends.  Keys are the 16 rows of
// m16n8k16, the query heads that share a kv head its 8 columns: S^T = K Q^T
// and O^T += V^T P^T, so that 8 heads leave no row of the product empty (heads
// as rows: twice the products, exponentials and registers).  K enters by
// ldmatrix, V by its transposing form, and P by movmatrix, which turns an 8 x 8
// block of the first product's result into the second's operand.
//
// Short or few caches take no deal: a cluster of blocks has a (sequence, head)
// to itself, each a share of its keys, and the blocks send one another the
// parts of the rows that each joins, through distributed shared memory.
//
// Int8.  Both products run in fp16, which holds the codes exactly: with u =
// code + 128 the bits 0x6400 | u are 1024 + u, and one logic operation and
// one packed addition give two codes.  q is scaled per row by the power of two
// that brings its largest element to 2^14 .. 2^15: its bf16 values are then
// exact in fp16 down to 2^-29 of that element.  K's scale multiplies the fp32
// score.  V's scale multiplies the fp32 probability, and the product enters
// fp16 over a power of two that follows the largest scale seen, so that it
// stays below 2^15, with 11 bits where a bf16 cache's probabilities, rounded
// to bf16 like its values, have 8.  A step with a product below 2^-14, where
// fp16 loses bits, runs P V in bf16 instead (a dim in which the likeliest keys'
// codes are 0 takes its value from the others, however small they are).  The
// step's large products then have 8 bits as well, as in a bf16 cache: a step
// has one type, and two products for each step would cost more than the bits
// are worth.  A bf16 step takes a logic operation more for two codes: 92.5 us
// where all steps do, 88.0 where none does (4 sequences of up to 65538 keys,
// 64/8 heads; 86.7 without the test).

#include "bd_attention.cuh"

#include <cuda_fp16.h>

#include <type_traits>

#include "bd_tma.h"

namespace bd {
namespace {

// ------------------------------------------------------------------------------- plan

constexpr int kPlanThreads = 256;

// Exclusive scan over the block; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* red, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int w = lane < kPlanThreads / 32 ? red[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int base = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    return base + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ int red[32];
    const AttentionArgs& a = p.a;
    const int n_seq = static_cast<int>(a.n_seq);
    grid_launch_dependents();
    grid_dependency_wait();

    int items = 0;
    for (int s0 = 0; s0 < n_seq; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        int n = 0;
        if (s < n_seq) {
            const AttnSeq q = attn_seq(p, s, true);
            n = static_cast<int>((static_cast<int64_t>(q.n_new) * p.G + p.mb - 1) / p.mb);
        }
        int total;
        const int off = block_scan(n, red, &total);
        if (s < n_seq) p.item_off[s] = items + off;
        items += total;
    }
    __syncthreads();
    // offsets that run backwards in a bad q_off could make more items than there is room for
    const int64_t room = (a.T * p.G + p.mb - 1) / p.mb + a.n_seq;
    if (items > room) items = static_cast<int>(room);

    int tiles = 0;
    for (int i0 = 0; i0 < items; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        AttnItem it{};
        if (i < items) {
            int lo = 0, hi = n_seq;  // the last s with item_off[s] <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (p.item_off[mid] <= i) lo = mid;
                else hi = mid;
            }
            const AttnSeq q = attn_seq(p, lo, false);
            it.seq = lo;
            it.row0 = (i - p.item_off[lo]) * p.mb;
            int64_t last = static_cast<int64_t>(it.row0) + p.mb - 1;
            const int64_t rows = static_cast<int64_t>(q.n_new) * p.G;
            if (last >= rows) last = rows - 1;
            const int end = attn_seen(q, static_cast<int>(last / p.G), a.causal);
            it.tiles = end > 0 ? (end + p.tile - 1) / p.tile : 1;
        }
        int total;
        it.before = tiles + block_scan(it.tiles, red, &total);
        if (i < items && bd_in(kBkAttnPlan, i, room)) p.items[i] = it;
        tiles += total;
    }
    if (threadIdx.x == 0) *p.head = AttnHeader{items, tiles};
}

// ------------------------------------------------------------------------------- decode kernel

constexpr int kMmaTile = 64;     // keys of a stage
constexpr int kMmaConsumers = 4;
constexpr int kMmaKeys = 32;     // keys of a stage that one warp takes
constexpr int kMmaThreads = 32 * (kMmaConsumers + 1);
constexpr int kMmaMaxStages = 8;
constexpr int kMmaMaxRows = 16;  // rows of an item: 8, or 16

// Blocks that an SM holds: 3 with items of 8 rows, whose threads need 128
// registers or fewer, unless a stage takes 32 KB (three blocks then have room
// for two stages each: 155 us for the batch of 32 caches of 4096 .. 8192 keys
// against 132).
constexpr int mma_blocks_per_sm(int rows, int dim, bool int8) { return rows == 8 && (int8 || dim == 64) ? 3 : 2; }

struct MmaParams {
    CUtensorMap k_map, v_map;  // [n_pages * n_kv][page][dim], box a row (in halves of 128 bytes) x min(page, 64)
    AttnParams p;
    int stages;
};

// NT: groups of 8 rows of an item.
template <int DIM, bool INT8, int NT>
struct MmaShape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kRowBytes = DIM * (INT8 ? 1 : 2);
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one box
    static constexpr int kHalves = kRowBytes / kBoxBytes;
    static constexpr int kTileBytes = kMmaTile * kRowBytes;               // K (or V) of a stage
    static constexpr int kStageBytes = 2 * kTileBytes + (INT8 ? 1024 : 0);  // stages stay 1024-byte aligned
    static constexpr int kBufBytes = 2 * kRows * DIM * 4;              // sums of an item, two warps each
    // what a block of a cluster gets of its rows from the others, for two items in turn
    static constexpr int kRecvBytes = 2 * kRows * (DIM + 4) * 4;
};

struct alignas(16) MmaShared {
    uint64_t full[kMmaMaxStages];
    uint64_t empty[kMmaMaxStages];
    float m[kMmaConsumers][kMmaMaxRows];
    float l[kMmaConsumers][kMmaMaxRows];
    uint64_t joined[2];  // the cluster's blocks have sent their parts of this block's rows, by the item's parity
    volatile int abort;
    int64_t scan[kMmaThreads / 32];
    int seq, row0;      // the block's first item,
    int64_t before;     // and the units before it
};

// Key tiles of one head of the item of sequence q that starts at row0.
__device__ __forceinline__ int mma_tiles(const AttnParams& p, const AttnSeq& q, int row0)
{
    int last = row0 + p.mb - 1;
    const int rows = q.n_new * p.G;
    if (last >= rows) last = rows - 1;
    const int end = attn_seen(q, last / p.G, p.a.causal);
    return end > 0 ? (end + kMmaTile - 1) / kMmaTile : 1;
}

// What a block does next: key tiles [t0, t1) of one (item, kv head).
struct MmaSegment {
    AttnSeq sq;
    int seq, row0, rows, tiles;
    int h, t0, t1;
};

// A block's segments in order.  The lengths of the next sequence are loaded
// while the present one is worked on.
struct MmaWalk {
    const AttnParams& p;
    int64_t u, end, before;  // next unit, last one + 1, units before the present item
    MmaSegment s;
    AttnSeq ahead;

    __device__ __forceinline__ MmaWalk(const AttnParams& pp, int64_t u0, int64_t u1, int seq, int row0, int64_t b)
        : p(pp), u(u0), end(u1), before(b)
    {
        if (u >= end) return;
        s.seq = seq;
        s.row0 = row0;
        s.sq = attn_seq(p, seq, false);
        s.rows = s.sq.n_new * p.G;
        s.tiles = mma_tiles(p, s.sq, row0);
        look_ahead();
    }
    __device__ __forceinline__ void look_ahead()
    {
        if (s.seq + 1 < p.a.n_seq) ahead = attn_seq(p, s.seq + 1, false);
    }
    __device__ __forceinline__ bool next()
    {
        if (u >= end) return false;
        const int n_kv = p.a.cache.n_kv;
        while (u - before >= static_cast<int64_t>(s.tiles) * n_kv) {  // on to the next item
            before += static_cast<int64_t>(s.tiles) * n_kv;
            s.row0 += p.mb;
            while (s.row0 >= s.rows && s.seq + 1 < p.a.n_seq) {
                ++s.seq;
                s.sq = ahead;
                s.rows = s.sq.n_new * p.G;
                s.row0 = 0;
                look_ahead();
            }
            s.tiles = mma_tiles(p, s.sq, s.row0);
        }
        const int64_t rel = u - before;
        s.h = attn_div(rel, s.tiles);
        s.t0 = static_cast<int>(rel - static_cast<int64_t>(s.h) * s.tiles);
        const int64_t left = end - u;
        s.t1 = left < s.tiles - s.t0 ? s.t0 + static_cast<int>(left) : s.tiles;
        u += s.t1 - s.t0;
        return true;
    }
};

// The segments of a block of a cluster that has a (sequence, head) to itself:
// its items in order (one, in a decode step), with this block's share of their
// tiles, which may be none.
struct WholeWalk {
    const AttnParams& p;
    MmaSegment s;
    int rank;  // of the block in its cluster

    __device__ __forceinline__ explicit WholeWalk(const AttnParams& pp) : p(pp)
    {
        const int pair = static_cast<int>(blockIdx.x) / p.whole;
        rank = static_cast<int>(blockIdx.x) - pair * p.whole;
        s.seq = pair / p.a.cache.n_kv;
        s.h = pair - s.seq * p.a.cache.n_kv;
        s.sq = attn_seq(p, s.seq, s.h == 0 && rank == 0);
        s.rows = s.sq.n_new * p.G;
        s.row0 = -p.mb;
    }
    __device__ __forceinline__ bool next()
    {
        s.row0 += p.mb;
        if (s.row0 >= s.rows) return false;
        s.tiles = mma_tiles(p, s.sq, s.row0);
        s.t0 = static_cast<int>(static_cast<int64_t>(s.tiles) * rank / p.whole);
        s.t1 = static_cast<int>(static_cast<int64_t>(s.tiles) * (rank + 1) / p.whole);
        return true;
    }
};

// The whole block: adds up the tiles of all sequences (each thread those of
// consecutive ones), finds the item of the block's first unit and notes down
// what the join needs.  The block's segments.
__device__ __forceinline__ MmaWalk mma_deal(const AttnParams& p, MmaShared& sh)
{
    const AttentionArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_seq = static_cast<int>(a.n_seq);
    const int per = (n_seq + kMmaThreads - 1) / kMmaThreads;
    const int s0 = static_cast<int>(threadIdx.x) * per < n_seq ? threadIdx.x * per : n_seq;
    const int s1 = s0 + per < n_seq ? s0 + per : n_seq;
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        const AttnSeq q = attn_seq(p, s, blockIdx.x == 0);
        for (int row0 = 0; row0 < q.n_new * p.G; row0 += p.mb) mine += mma_tiles(p, q, row0);
    }
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh.scan[warp] = x;
    __syncthreads();
    int64_t total = 0, at = x - mine;
#pragma unroll
    for (int w = 0; w < kMmaThreads / 32; ++w) {
        if (w < warp) at += sh.scan[w];
        total += sh.scan[w];
    }
    const int n_kv = a.cache.n_kv;
    const int64_t units = total * n_kv;
    const int active = attn_active(units, p.blocks);
    if (static_cast<int>(blockIdx.x) < active) {
        const int64_t u = attn_first(units, active, blockIdx.x);
        if (u >= at * n_kv && u < (at + mine) * n_kv) {
            // this thread's sequences hold it
            int64_t before = at * n_kv;
            for (int s = s0; s < s1; ++s) {
                const AttnSeq q = attn_seq(p, s, false);
                for (int row0 = 0; row0 < q.n_new * p.G; row0 += p.mb) {
                    const int64_t n = static_cast<int64_t>(mma_tiles(p, q, row0)) * n_kv;
                    if (u >= before && u < before + n) {
                        sh.seq = s;
                        sh.row0 = row0;
                        sh.before = before;
                    }
                    before += n;
                }
            }
        }
    }
    __syncthreads();
    const int c = blockIdx.x;
    MmaWalk walk(p, c < active ? attn_first(units, active, c) : 0, c < active ? attn_first(units, active, c + 1) : 0,
                 sh.seq, sh.row0, sh.before);
    if (threadIdx.x == 0) {
        AttnJoin j{};
        if (c < active) {
            const int64_t rel = walk.u - walk.before;
            const int h = attn_div(rel, walk.s.tiles);
            j = attn_join_of(units, active, c, walk.u, walk.before + static_cast<int64_t>(h) * walk.s.tiles,
                             walk.s.tiles, walk.s.sq, p.G, walk.s.row0, h);
        }
        p.joins[c] = j;
    }
    return walk;
}

template <bool WHOLE>
__device__ __forceinline__ auto mma_walk(const AttnParams& p, MmaShared& sh)
{
    if constexpr (WHOLE) return WholeWalk(p);
    else return mma_deal(p, sh);
}

__device__ __forceinline__ bool attn_wait(volatile int* abort_flag, uint64_t* bar, uint32_t parity, uint32_t* err)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            raise_error(err, kErrTimeout);
            return false;
        }
    }
    return true;
}

// A wait for the other blocks of the cluster; false once given up.
__device__ __forceinline__ bool mbar_wait_cluster_bounded(uint64_t* bar, uint32_t parity, uint32_t* err)
{
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_cluster(bar, parity))
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            raise_error(err, kErrTimeout);
            return false;
        }
    return true;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The 8 x 8 block of b16 that the warp holds as an accumulator fragment, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}


// Two int8 codes, bytes 0 and 2 of r, as a pair of fp16.
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t r)
{
    const uint32_t x = (r & 0x00FF00FFu) ^ 0x64806480u;  // 1024 + 128 + code
    const uint32_t offset = 0xE480E480u;                 // -1152
    const __half2 d = __hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&offset));
    return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr uint32_t kFp16Normal = 0x38800000u;  // the bits of 2^-14

// Two int8 codes as a pair of bf16, which have no room for 128 + code: with c
// the byte, 0x4300 | (c & 0x7f) is 128 + (c & 0x7f), 0x4300 | (c & 0x80) is 128
// or 256, and the difference is the code.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t r)
{
    const uint32_t hi = (r & 0x007F007Fu) | 0x43004300u, lo = (r & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&hi), *reinterpret_cast<const __nv_bfloat162*>(&lo));
    return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^e with e the exponent of |x| (x normal), kept within 2^-100 .. 2^100
__device__ __forceinline__ float pow2_of(float x)
{
    const float c = fminf(fmaxf(fabsf(x), 7.9e-31f), 1.2e30f);
    return __uint_as_float(__float_as_uint(c) & 0x7F800000u);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void consumers_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kMmaConsumers) : "memory");
}

// Byte offset of 16-byte chunk c of row t in a box of 128- or 64-byte rows
// (TMA's 128- or 64-byte swizzle).
template <int BOX_BYTES>
__device__ __forceinline__ uint32_t swizzled(int t, int c)
{
    if constexpr (BOX_BYTES == 128)
        return static_cast<uint32_t>(t * 128 + ((c ^ (t & 7)) << 4));
    else
        return static_cast<uint32_t>(t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
}

template <int DIM, bool INT8, int NT, bool WHOLE>
__global__ void __launch_bounds__(kMmaThreads, mma_blocks_per_sm(8 * NT, DIM, INT8))
    attn_mma_kernel(const __grid_constant__ MmaParams mp)
{
    using S = MmaShape<DIM, INT8, NT>;
    constexpr int kSteps = DIM / 16;  // MMA steps of q . k, and 16-dim tiles of the output
    // all of it dynamic: the ring starts on a 1024-byte boundary without padding
    extern __shared__ __align__(1024) uint8_t dyn_raw[];
    uint8_t* ring = dyn_raw;
    float* buf = reinterpret_cast<float*>(ring + static_cast<size_t>(mp.stages) * S::kStageBytes);
    MmaShared& sh = *reinterpret_cast<MmaShared*>(reinterpret_cast<uint8_t*>(buf) + S::kBufBytes);
    // A cluster's parts: row k of those that this block joins, from rank w, for the item's parity.  A
    // block sends an item's parts only after it has all of the one before, so two places suffice, and
    // two barriers: one would take a block's arrival for the next item, which a third block's late one
    // for this item does not hold back, for that.  Item i + 2, which shares item i's, is sent only
    // after every block's arrival for i + 1, so after every block has had all of item i.
    constexpr int kRecvStride = DIM + 4;  // the sum, its maximum and denominator
    [[maybe_unused]] float* recv = reinterpret_cast<float*>(&sh + 1);
    [[maybe_unused]] const auto recv_row = [&](uint32_t item, int w, int k) {
        return static_cast<int>(item & 1) * S::kRows + w * (S::kRows / mp.p.whole) + k;
    };

    const AttnParams& p = mp.p;
    const AttentionArgs& a = p.a;
    const KvPages& cache = a.cache;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    grid_launch_dependents();
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mp.k_map)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mp.v_map)) : "memory");
        for (int s = 0; s < mp.stages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], kMmaConsumers);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&sh.joined[i], WHOLE ? p.whole : 1);
        sh.abort = 0;
        fence_mbarrier_init();
    }
    if (WHOLE && p.whole > 1) cluster_sync_all();  // the others' barriers are there before anything is sent
    else __syncthreads();
    grid_dependency_wait();

    const int n_kv = cache.n_kv;
    auto walk = mma_walk<WHOLE>(p, sh);
    const MmaSegment& sg = walk.s;
    int walk_rank = 0;
    if constexpr (WHOLE) walk_rank = walk.rank;
    int stage = 0;
    uint32_t phase = 0;

    if (warp == kMmaConsumers) {
        // ------------------------------------------------------------ producer warp
        const int box_rows = cache.page < kMmaTile ? cache.page : kMmaTile;
        const int pages_per_tile = kMmaTile / box_rows;
        // The page of this lane's box in a tile (lane j looks after the j-th box), looked up one tile
        // ahead, whether the sequence reaches it or not.
        const auto page_of = [&](int t) {
            const int at = (t * kMmaTile + lane * box_rows) >> cache.page_shift;
            return lane < pages_per_tile && at < a.max_pages
                       ? a.table[static_cast<int64_t>(sg.seq) * a.max_pages + at]
                       : 0;
        };
        while (walk.next()) {
            const int h = sg.h;
            const int pages = (sg.sq.len + cache.page - 1) >> cache.page_shift;  // that the sequence has
            int page_next = page_of(sg.t0);
            for (int t = sg.t0; t < sg.t1; ++t) {
                const int key = t * kMmaTile + lane * box_rows;
                const bool mine = lane < pages_per_tile && (key >> cache.page_shift) < pages;
                int page = page_next;
                if (t + 1 < sg.t1) page_next = page_of(t + 1);
                if (mine && (page < 0 || page >= cache.n_pages)) {
                    raise_error(a.err, kErrBadIndex);
                    page = 0;
                }
                const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
                bool ok = true;
                if (lane == 0) {
                    ok = attn_wait(&sh.abort, &sh.empty[stage], phase ^ 1, a.err);
                    if (ok)
                        mbar_arrive_expect_tx(&sh.full[stage],
                                              static_cast<uint32_t>(boxes * box_rows) *
                                                  (2 * S::kRowBytes + (INT8 ? 8 : 0)));
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) {
                    // given up: leave only when the copies in flight have landed (each stage's last
                    // fill has this cycle's parity below `stage` and the one before's from there on)
                    if (lane < mp.stages)
                        mbar_wait_bounded(&sh.full[lane], lane < stage ? phase : phase ^ 1);
                    return;
                }
                if (mine) {
                    uint8_t* st = ring + static_cast<size_t>(stage) * S::kStageBytes;
                    const int row = key & (cache.page - 1);
                    const int outer = page * n_kv + h;
                    uint8_t* dst = st + lane * box_rows * S::kRowBytes;
                    if constexpr (S::kHalves == 2) {
                        tma_load_4d(dst, &mp.k_map, 0, row, 0, outer, &sh.full[stage]);
                        tma_load_4d(dst + S::kTileBytes, &mp.v_map, 0, row, 0, outer, &sh.full[stage]);
                    } else {
                        tma_load_3d(dst, &mp.k_map, 0, row, outer, &sh.full[stage]);
                        tma_load_3d(dst + S::kTileBytes, &mp.v_map, 0, row, outer, &sh.full[stage]);
                    }
                    if constexpr (INT8) {
                        const int64_t vec = (static_cast<int64_t>(outer) << cache.page_shift) + row;
                        uint8_t* sc = st + 2 * S::kTileBytes + lane * box_rows * 4;
                        bulk_g2s(sc, cache.k_scale + vec, box_rows * 4, &sh.full[stage]);
                        bulk_g2s(sc + kMmaTile * 4, cache.v_scale + vec, box_rows * 4, &sh.full[stage]);
                    }
                }
                if (++stage == mp.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumer warps
    const int g = lane >> 2, q4 = lane & 3;
    const float c2 = a.scale * kLog2e;
    [[maybe_unused]] uint32_t item = 0;  // of a cluster, so far
    [[maybe_unused]] bool gave_up = false;
    int turn = 0;  // stages so far: this warp takes those of its parity
    while (walk.next()) {
        const AttnSeq sq = sg.sq;
        const int h = sg.h, t0 = sg.t0, t1 = sg.t1, rows = sg.rows, row0 = sg.row0;

        // Q as B fragments: this thread has dims of query row 8 n + g.  Its scores, sums and maxima are
        // those of rows 8 n + 2 q4 + {0, 1}: keys they see, and the factor of their scores.
        uint32_t qf[NT][kSteps][2];
        int seen[NT][2];
        float cr[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + 8 * n + g;
            const bool live = r < rows;
            const int tok = live ? r / p.G : 0;
            const uint16_t* src = a.q + (static_cast<int64_t>(sq.q0) + tok) * a.q_stride +
                                  static_cast<int64_t>(h * p.G + (live ? r - tok * p.G : 0)) * DIM;
            const int sees = live ? attn_seen(sq, tok, a.causal) : 0;
            float factor = c2;
            if constexpr (INT8) {
                // a code fragment holds dims 4 q4 + {0, 2} and 4 q4 + {1, 3} of a step's 16
                uint2 w[kSteps];
                float big = 0.0f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    w[k] = live ? *reinterpret_cast<const uint2*>(src + 16 * k + 4 * q4) : make_uint2(0, 0);
                    big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[k].x << 16)),
                                           fabsf(__uint_as_float(w[k].x & 0xFFFF0000u))));
                    big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[k].y << 16)),
                                           fabsf(__uint_as_float(w[k].y & 0xFFFF0000u))));
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const float unit = pow2_of(big), f = 16384.0f / unit;
                factor = c2 * (unit / 16384.0f);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    qf[n][k][0] = pack_f16x2(__uint_as_float(w[k].x << 16) * f, __uint_as_float(w[k].y << 16) * f);
                    qf[n][k][1] = pack_f16x2(__uint_as_float(w[k].x & 0xFFFF0000u) * f,
                                             __uint_as_float(w[k].y & 0xFFFF0000u) * f);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int d = 16 * k + 2 * q4;
                    qf[n][k][0] = live ? *reinterpret_cast<const uint32_t*>(src + d) : 0u;
                    qf[n][k][1] = live ? *reinterpret_cast<const uint32_t*>(src + d + 8) : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // from the lanes that loaded these rows
                seen[n][i] = __shfl_sync(0xffffffffu, sees, 4 * (2 * q4 + i));
                cr[n][i] = INT8 ? __shfl_sync(0xffffffffu, factor, 4 * (2 * q4 + i)) : c2;
            }
        }
        // a tile in shared memory: page boxes of box_rows keys, in each the halves of 128 bytes one
        // after the other (rows of 128 bytes or less have one)
        const int box_shift = cache.page < kMmaTile ? cache.page_shift : 6;
        const auto chunk_at = [&](int row, int chunk) {
            if constexpr (S::kHalves == 1) return swizzled<S::kBoxBytes>(row, chunk);
            const int box = row >> box_shift, half = chunk >> 3;
            return ((static_cast<uint32_t>(box) << box_shift) << 8) + ((static_cast<uint32_t>(half) << box_shift) << 7) +
                   swizzled<128>(row & ((1 << box_shift) - 1), chunk & 7);
        };
        // the keys that every live row sees: below, no mask is needed
        const int all_seen = attn_seen(sq, row0 / p.G, a.causal);

        float o[NT][kSteps][4];  // dims of tile k (bf16: g, g + 8; int8: 2 g, 2 g + 1) x rows 8 n + 2 q4 + {0, 1}
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][k][e] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = -INFINITY;
                l[n][i] = 0.0f;
            }
        }
        float v_unit = 0.0f;  // int8: power of two at or above every scale of V so far, times 2^(bias - 15)

        for (int t = t0; t < t1; ++t, ++turn) {
            // every warp waits for every stage and hands it back, the ones that are not its own at once:
            // a warp that did neither could be two phases away from a barrier, which its parity cannot
            // tell from none.  On a timeout (reported) the warps still meet at the barriers below.
            if (!__all_sync(0xffffffffu, attn_wait(&sh.abort, &sh.full[stage], phase, a.err))) {
                turn += t1 - t;
                break;
            }
            if ((turn & 1) != (warp >> 1)) {
                if (lane == 0) mbar_arrive(&sh.empty[stage]);
                if (++stage == mp.stages) {
                    stage = 0;
                    phase ^= 1;
                }
                continue;
            }
            const uint32_t st = smem_u32(ring) + static_cast<uint32_t>(stage) * S::kStageBytes;
            const int slice = kMmaKeys * (warp & 1);  // this warp's keys of the stage
            const int key0 = t * kMmaTile + slice;    // and in the sequence
            const int mi = lane >> 3, mr = lane & 7;

            // ---- scores of 32 keys x 8 NT rows: this thread's keys are 16 b + 8 j + g
            float s[NT][2][4] = {};  // [row group][b][2 j + row]
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int row = slice + 16 * b + (mi & 1) * 8 + mr;
                if constexpr (INT8) {
#pragma unroll
                    for (int k = 0; k < kSteps; k += 2) {
                        uint32_t r[4];
                        ldsm_x4(st + swizzled<S::kBoxBytes>(row, k + (mi >> 1)), r);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t a0 = codes_f16x2(r[2 * x]), a1 = codes_f16x2(r[2 * x + 1]);
                            const uint32_t a2 = codes_f16x2(r[2 * x] >> 8), a3 = codes_f16x2(r[2 * x + 1] >> 8);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16_16816(s[n][b], a0, a1, a2, a3, qf[n][k + x][0], qf[n][k + x][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        uint32_t r[4];
                        const int chunk = 2 * k + (mi >> 1);
                        ldsm_x4(st + chunk_at(row, chunk), r);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_bf16_16816(s[n][b], r[0], r[1], r[2], r[3], qf[n][k][0], qf[n][k][1]);
                    }
                }
            }

            // ---- to units of log2, masked
            float vs[2][2];
            if constexpr (INT8) {
                const float* sc = reinterpret_cast<const float*>(ring + static_cast<size_t>(stage) * S::kStageBytes +
                                                                 2 * S::kTileBytes) +
                                  slice + g;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float ks = sc[16 * b + 8 * j];
                        vs[b][j] = sc[kMmaTile + 16 * b + 8 * j];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) s[n][b][2 * j + i] *= ks * cr[n][i];
                    }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][b][e] *= c2;
            }
            const bool tail = key0 + kMmaKeys > sq.len;
            if (key0 + kMmaKeys > all_seen) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = key0 + 16 * b + 8 * j + g;
                        // what lies past the sequence may be anything, NaN included: zeros instead
                        if (INT8 && key >= sq.len) vs[b][j] = 0.0f;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (key >= seen[n][i]) s[n][b][2 * j + i] = -INFINITY;
                    }
            }

            // ---- running maxima, over this thread's keys and the 8 lanes of its rows
            float mt[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mt[n][i] = fmaxf(fmaxf(s[n][0][i], s[n][0][2 + i]), fmaxf(s[n][1][i], s[n][1][2 + i]));
            float v_new = v_unit, v_max = 0.0f;
            if constexpr (INT8) v_max = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) mt[n][i] = fmaxf(mt[n][i], __shfl_xor_sync(0xffffffffu, mt[n][i], x));
                if constexpr (INT8) v_max = fmaxf(v_max, __shfl_xor_sync(0xffffffffu, v_max, x));
            }
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) grow = grow || mt[n][i] > m[n][i];
            if constexpr (INT8) {
                constexpr float kUnit = static_cast<float>(1u << (static_cast<int>(attn_bias<true>()) - 14));
                if (v_max * (0.5f * kUnit) > 0.5f * v_unit) v_new = pow2_of(v_max) * kUnit;
                grow = grow || v_new != v_unit;
            }
            if (__any_sync(0xffffffffu, grow)) {
                const float fv = INT8 && v_new != v_unit ? v_unit / v_new : 1.0f;
                v_unit = v_new;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float up = fmaxf(m[n][i], mt[n][i]);
                        const float f = up == -INFINITY ? 1.0f : ex2(m[n][i] - up);
                        m[n][i] = up;
                        l[n][i] *= f;
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            o[n][k][i] *= f * fv;
                            o[n][k][2 + i] *= f * fv;
                        }
                    }
            }

            // ---- probabilities, turned into B fragments: keys 16 b + 8 j + 2 q4 + {0, 1} of row 8 n + g
            uint32_t pb[NT][2][2];
            [[maybe_unused]] float pw[NT][2][4];  // int8: what is to be rounded
            [[maybe_unused]] uint32_t least = 0xFFFFFFFFu;  // the least of it that is not 0: its bits less 1
            const float v_inv = INT8 ? (v_unit > 0.0f ? 1.0f / v_unit : 0.0f) : 1.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float mu[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) mu[i] = m[n][i] == -INFINITY ? 0.0f : m[n][i] - attn_bias<INT8>();
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float p0 = ex2(s[n][b][2 * j] - mu[0]), p1 = ex2(s[n][b][2 * j + 1] - mu[1]);
                        l[n][0] += p0;
                        l[n][1] += p1;
                        if constexpr (INT8) {
                            const float w = vs[b][j] * v_inv;
                            pw[n][b][2 * j] = p0 * w, pw[n][b][2 * j + 1] = p1 * w;
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                least = min(least, __float_as_uint(pw[n][b][2 * j + e]) - 1u);
                        } else {
                            pb[n][b][j] = transpose8(pack_bf16x2(p0, p1));
                        }
                    }
            }

            // ---- sums: dim x 8 NT rows += V^T (dim x 32) P^T (32 x 8 NT)
            const uint32_t vt = st + S::kTileBytes;
            // a b16 element is a pair of dims: the transposed fragment holds dims 2 g, 2 g + 1 of two keys;
            // the tile's rows 0..7 take the even dims of a chunk, rows 8..15 the odd ones
            [[maybe_unused]] const auto add_codes = [&](auto as_bf16) {
                constexpr bool kBf16 = decltype(as_bf16)::value;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float x = pw[n][b][2 * j], y = pw[n][b][2 * j + 1];
                            pb[n][b][j] = transpose8(kBf16 ? pack_bf16x2(x, y) : pack_f16x2(x, y));
                        }
                    const int row = slice + 16 * b + (mi & 1) * 8 + mr;
#pragma unroll
                    for (int k = 0; k < kSteps; k += 2) {
                        uint32_t r[4];
                        ldsm_x4_t(vt + swizzled<S::kBoxBytes>(row, k + (mi >> 1)), r);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if constexpr (kBf16) {
                                const uint32_t a0 = codes_bf16x2(r[2 * x]), a1 = codes_bf16x2(r[2 * x] >> 8);
                                const uint32_t a2 = codes_bf16x2(r[2 * x + 1]), a3 = codes_bf16x2(r[2 * x + 1] >> 8);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma_bf16_16816(o[n][k + x], a0, a1, a2, a3, pb[n][b][0], pb[n][b][1]);
                            } else {
                                const uint32_t a0 = codes_f16x2(r[2 * x]), a1 = codes_f16x2(r[2 * x] >> 8);
                                const uint32_t a2 = codes_f16x2(r[2 * x + 1]), a3 = codes_f16x2(r[2 * x + 1] >> 8);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma_f16_16816(o[n][k + x], a0, a1, a2, a3, pb[n][b][0], pb[n][b][1]);
                            }
                        }
                    }
                }
            };
            if constexpr (INT8) {
                // some of it would lose bits in fp16
                if (__any_sync(0xffffffffu, least < kFp16Normal)) add_codes(std::true_type{});
                else add_codes(std::false_type{});
            } else {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t mask0 = 0xFFFFFFFFu, mask1 = 0xFFFFFFFFu;
                    if (tail) {
                        // zeros for what lies past the sequence
                        const int k = key0 + 16 * b + 2 * q4;
                        mask0 = (k < sq.len ? 0xFFFFu : 0u) | (k + 1 < sq.len ? 0xFFFF0000u : 0u);
                        mask1 = (k + 8 < sq.len ? 0xFFFFu : 0u) | (k + 9 < sq.len ? 0xFFFF0000u : 0u);
                    }
                    const int row = slice + 16 * b + (mi >> 1) * 8 + mr;
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        uint32_t r[4];
                        const int chunk = 2 * k + (mi & 1);
                        ldsm_x4_t(vt + chunk_at(row, chunk), r);
                        if (tail) {
                            r[0] &= mask0;
                            r[1] &= mask0;
                            r[2] &= mask1;
                            r[3] &= mask1;
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_bf16_16816(o[n][k], r[0], r[1], r[2], r[3], pb[n][b][0], pb[n][b][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[stage]);
            if (++stage == mp.stages) {
                stage = 0;
                phase ^= 1;
            }
        }

        // ---- join the four warps: (0 + 2) and (1 + 3) in the two buffers
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], x);
                m[n][i] -= attn_bias<INT8>();
                if (g == 0) {
                    sh.m[warp][8 * n + 2 * q4 + i] = m[n][i];
                    sh.l[warp][8 * n + 2 * q4 + i] = l[n][i];
                }
            }
        consumers_sync();
        float f[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * q4 + i;
                float mm = sh.m[0][r];
#pragma unroll
                for (int w = 1; w < kMmaConsumers; ++w) mm = fmaxf(mm, sh.m[w][r]);
                f[n][i] = attn_weight(m[n][i], l[n][i], mm);
                if (INT8 && f[n][i] != 0.0f) f[n][i] *= v_unit;  // the sums are over the scales' unit
            }
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
            if ((warp >> 1) == w) {
                float* mine = buf + (warp & 1) * S::kRows * DIM;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float* line = mine + (8 * n + 2 * q4 + i) * DIM;
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            // (in an order of the row's own: the lanes' banks differ)
                            const float x = f[n][i] == 0.0f ? 0.0f : o[n][k][i] * f[n][i];
                            const float y = f[n][i] == 0.0f ? 0.0f : o[n][k][2 + i] * f[n][i];
                            if constexpr (INT8) {
                                float2* b = reinterpret_cast<float2*>(line + ((16 * k + 2 * g) ^ (q4 << 4)));
                                const float2 old = w ? *b : make_float2(0.0f, 0.0f);
                                *b = make_float2(old.x + x, old.y + y);
                            } else {
                                float* b0 = line + ((16 * k + g) ^ (q4 << 3));
                                float* b1 = line + ((16 * k + 8 + g) ^ (q4 << 3));
                                *b0 = w ? *b0 + x : x;
                                *b1 = w ? *b1 + y : y;
                            }
                        }
                    }
            }
            consumers_sync();
        }

        const auto write_row = [&](int r, int d, float4 v, float mm, float ll) {
            const int row = row0 + r, tok = row / p.G;
            const int64_t at = (static_cast<int64_t>(sq.q0) + tok) * a.n_q + h * p.G + (row - tok * p.G);
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
            if (bd_in(kBkAttn, at, a.T * a.n_q)) {
                *reinterpret_cast<uint2*>(a.out + at * DIM + d) =
                    make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                if (d == 0 && a.lse) a.lse[at] = attn_lse(mm, ll);
            }
        };
        const bool whole = t0 == 0 && t1 == sg.tiles;
        const int slot = attn_slot(blockIdx.x, t0 == 0);
        const int live_rows = rows - row0 < S::kRows ? rows - row0 : S::kRows;
        for (int i = threadIdx.x; i < live_rows * (DIM / 4); i += 32 * kMmaConsumers) {
            const int r = i / (DIM / 4), d = 4 * (i % (DIM / 4));
            float mm = sh.m[0][r];
#pragma unroll
            for (int w = 1; w < kMmaConsumers; ++w) mm = fmaxf(mm, sh.m[w][r]);
            float ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kMmaConsumers; ++w) {
                const float lw = sh.l[w][r];
                ll += lw * attn_weight(sh.m[w][r], lw, mm);
            }
            const int place = r * DIM + (d ^ (((r >> 1) & 3) << (INT8 ? 4 : 3)));
            float4 v = *reinterpret_cast<const float4*>(buf + place);
            const float4 v1 = *reinterpret_cast<const float4*>(buf + S::kRows * DIM + place);
            v = make_float4(v.x + v1.x, v.y + v1.y, v.z + v1.z, v.w + v1.w);
            if (WHOLE && p.whole > 1) {
                // to the block of the cluster that joins this row: rank r mod the cluster's size
                const int place_there = recv_row(item, walk_rank, r / p.whole);
                const uint32_t there = cluster_address(recv + place_there * kRecvStride, r % p.whole);
                st_cluster_v4(there + 4 * d, v);
                if (d == 0) st_cluster_v4(there + 4 * DIM, make_float4(mm, ll, 0.0f, 0.0f));
            } else if (whole) {
                write_row(r, d, v, mm, ll);
            } else {
                const int64_t at = static_cast<int64_t>(slot) * S::kRows + r;
                if (bd_in(kBkAttn, at, 2ll * p.blocks * S::kRows)) {
                    *reinterpret_cast<float4*>(p.part_o + at * DIM + d) = v;
                    if (d == 0) p.part_ml[at] = make_float2(mm, ll);
                }
            }
        }
        consumers_sync();  // the buffers are free for the next item
        if constexpr (WHOLE) {
            if (p.whole > 1) {
                uint64_t* const joined = &sh.joined[item & 1];
                if (static_cast<int>(threadIdx.x) < p.whole) mbar_arrive_remote_release(joined, threadIdx.x);
                // (given up, which is reported: what is there is joined)
                if (!mbar_wait_cluster_bounded(joined, (item >> 1) & 1, a.err)) gave_up = true;
                for (int i = threadIdx.x; i < S::kRows / p.whole * (DIM / 4); i += 32 * kMmaConsumers) {
                    const int k = i / (DIM / 4), d = 4 * (i % (DIM / 4)), r = k * p.whole + walk_rank;
                    if (r >= live_rows) break;
                    float mm = -INFINITY, ll = 0.0f;
                    for (int w = 0; w < p.whole; ++w) mm = fmaxf(mm, recv[recv_row(item, w, k) * kRecvStride + DIM]);
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int w = 0; w < p.whole; ++w) {
                        const float* part = recv + recv_row(item, w, k) * kRecvStride;
                        const float lw = part[DIM + 1], f = attn_weight(part[DIM], lw, mm);
                        if (f == 0.0f) continue;
                        const float4 x = *reinterpret_cast<const float4*>(part + d);
                        ll += lw * f;
                        v = make_float4(v.x + x.x * f, v.y + x.y * f, v.z + x.z * f, v.w + x.w * f);
                    }
                    write_row(r, d, v, mm, ll);
                }
                ++item;
            }
        }
    }
    // a block leaves when it has all that is sent to it, or else with the rest of its cluster: nothing
    // is sent to one that has left (the barrier does not wait for threads that have)
    if constexpr (WHOLE)
        if (gave_up) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// ------------------------------------------------------------------------------- join

constexpr int kJoinThreads = 128;

// Block (c - 1, y) joins what block c of the main kernel noted down: a row per
// warp, and more where sequences have more rows than the host expects.  It
// waits twice, for what was noted down and then for the parts with their
// maxima, the first BATCH parts at once.  (Where it waited four times, for the
// sequence's offsets and for one part after another too, the chunk of 4096 over
// 8192 keys, 64/8 heads, took 27 us for its join instead of 14.)  A chunk's
// items have few parts and many rows, for which more warps at a time are
// better; a decode step's have many parts and few rows.
template <int DIM, int BATCH>
__global__ void __launch_bounds__(kJoinThreads, BATCH <= 4 ? 12 : 4)
    attn_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kPer = DIM / 32;  // values of a lane
    grid_launch_dependents();
    grid_dependency_wait();
    const AttentionArgs& a = p.a;
    const int c = blockIdx.x + 1;
    const AttnJoin it = p.joins[c];
    if (it.parts == 0) return;
    const int lane = threadIdx.x & 31;
    const int parts = it.parts;
    const int live = it.rows - it.row0 < p.mb ? it.rows - it.row0 : p.mb;
    constexpr int kWarps = kJoinThreads / 32;
    for (int r = kWarps * blockIdx.y + (threadIdx.x >> 5); r < live; r += kWarps * gridDim.y) {
        const auto row_of = [&](int i) { return static_cast<int64_t>(attn_slot(c - 1 + i, i == 0)) * p.mb + r; };
        float v[BATCH][kPer];
        const auto load = [&](int i0) {
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const float* src = p.part_o + row_of(i0 + j < parts ? i0 + j : parts - 1) * DIM + kPer * lane;
                if constexpr (kPer == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(src);
                    v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(src);
                    v[j][0] = x.x, v[j][1] = x.y;
                }
            }
        };
        load(0);
        float2 ml = make_float2(-INFINITY, 0.0f);  // of part 32 n + lane
        if (lane < parts) ml = p.part_ml[row_of(lane)];
        float mm = ml.x;
        for (int i = 32 + lane; i < parts; i += 32) mm = fmaxf(mm, p.part_ml[row_of(i)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        float acc[kPer] = {}, ll = 0.0f, w = attn_weight(ml.x, ml.y, mm);
        for (int i0 = 0; i0 < parts; i0 += BATCH) {
            if (i0) load(i0);
            if (i0 && (i0 & 31) == 0) {
                ml = make_float2(-INFINITY, 0.0f);
                if (i0 + lane < parts) ml = p.part_ml[row_of(i0 + lane)];
                w = attn_weight(ml.x, ml.y, mm);
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, (i0 + j) & 31);
                const float lj = __shfl_sync(0xffffffffu, ml.y, (i0 + j) & 31);
                if (i0 + j < parts && wj != 0.0f) {
                    ll += wj * lj;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) acc[e] += wj * v[j][e];
                }
            }
        }
        const int row = it.row0 + r, tok = row / p.G;
        const int64_t at = (static_cast<int64_t>(it.q0) + tok) * a.n_q + it.h * p.G + (row - tok * p.G);
        if (!bd_in(kBkAttnCombine, at, a.T * a.n_q)) continue;
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        uint32_t y[kPer / 2];
#pragma unroll
        for (int e = 0; e < kPer; e += 2) y[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        uint16_t* dst = a.out + at * DIM + kPer * lane;
        if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
        else *reinterpret_cast<uint32_t*>(dst) = y[0];
        if (lane == 0 && a.lse) a.lse[at] = attn_lse(mm, ll);
    }
}

template <int DIM, bool INT8, int NT, bool WHOLE>
cudaError_t launch_mma_shape(const AttnParams& p, cudaStream_t stream)
{
    using S = MmaShape<DIM, INT8, NT>;
    static std::atomic<size_t> smem_set[kHostMaxDevices];
    const KvPages& kv = p.a.cache;
    MmaParams mp{};
    mp.p = p;
    const uint32_t box_rows = kv.page < kMmaTile ? kv.page : kMmaTile;
    const auto type = INT8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto swz = S::kBoxBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const uint64_t outer = static_cast<uint64_t>(kv.n_pages) * kv.n_kv;
    for (int i = 0; i < 2; ++i) {
        CUtensorMap* map = i ? &mp.v_map : &mp.k_map;
        const void* base = i ? kv.v : kv.k;
        if (!(S::kHalves == 2 ? encode_tma_parts(map, type, 2, base, DIM, kv.page, outer, 2, box_rows, swz)
                              : encode_tma_3d(map, type, INT8 ? 1 : 2, base, DIM, kv.page, outer, DIM, box_rows, swz)))
            return cudaErrorInvalidValue;
    }
    // the SM's shared memory shared by the blocks that it holds; all of it
    // where there are no more blocks than SMs
    const size_t rest = S::kBufBytes + sizeof(MmaShared) + (p.whole > 1 ? S::kRecvBytes : 0);
    const size_t budget = p.blocks <= p.a.sm_count ? 227u * 1024u
                                                   : 228u * 1024u / mma_blocks_per_sm(8 * NT, DIM, INT8) - 1024u;
    mp.stages = static_cast<int>((budget - rest) / S::kStageBytes);
    if (mp.stages > kMmaMaxStages) mp.stages = kMmaMaxStages;
    const size_t smem = static_cast<size_t>(mp.stages) * S::kStageBytes + rest;
    const auto kernel = attn_mma_kernel<DIM, INT8, NT, WHOLE>;
    cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem, smem_set);
    launch_dep_clusters(err, kernel, dim3(p.blocks), dim3(kMmaThreads), WHOLE ? p.whole : 1, smem, stream, mp);
    return err;
}

constexpr size_t align_up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct AttnWs {
    size_t head, item_off, items, joins, ml, o, total;
};

// rows: of all sequences, where the items are listed (chunks); else 0
AttnWs attn_layout(int64_t rows, int64_t n_seq, int dim, int mb, int blocks)
{
    AttnWs w{};
    w.head = 256;
    w.item_off = w.head + 256;
    w.items = w.item_off + align_up(static_cast<size_t>(n_seq + 1) * 4);
    const size_t items = rows > 0 ? static_cast<size_t>((rows + mb - 1) / mb + n_seq) : 0;
    w.joins = w.items + align_up(items * sizeof(AttnItem));
    w.ml = w.joins + align_up(static_cast<size_t>(blocks) * sizeof(AttnJoin));
    w.o = w.ml + align_up(static_cast<size_t>(2 * blocks) * mb * 8);
    w.total = w.o + align_up(static_cast<size_t>(2 * blocks) * mb * dim * 4);
    return w;
}

}  // namespace

cudaError_t launch_attention_mma(const AttnParams& p, cudaStream_t stream)
{
    const auto of = [&](auto dim, auto int8) {
        constexpr int kDim = decltype(dim)::value;
        constexpr bool kInt8 = decltype(int8)::value;
        if (p.mb == 8)
            return p.whole ? launch_mma_shape<kDim, kInt8, 1, true>(p, stream)
                           : launch_mma_shape<kDim, kInt8, 1, false>(p, stream);
        return p.whole ? launch_mma_shape<kDim, kInt8, 2, true>(p, stream)
                       : launch_mma_shape<kDim, kInt8, 2, false>(p, stream);
    };
    using Dim64 = std::integral_constant<int, 64>;
    using Dim128 = std::integral_constant<int, 128>;
    using Yes = std::true_type;
    using No = std::false_type;
    if (p.a.cache.dim == 128)
        return p.a.cache.int8 ? of(Dim128{}, Yes{}) : of(Dim128{}, No{});
    return p.a.cache.int8 ? of(Dim64{}, Yes{}) : of(Dim64{}, No{});
}

size_t attention_workspace_size(int64_t T, int64_t n_seq, int n_q, int n_kv, int dim)
{
    // the host may learn how long the chunks are only with the call: room for both kernels
    const int G = n_q / n_kv;
    const size_t few = attn_layout(0, n_seq, dim, kMmaMaxRows, kAttnMaxBlocks).total;
    const size_t chunk = attn_layout(T * G, n_seq, dim, kChunkRows, chunk_max_blocks(kChunkRows)).total;
    return few + chunk;
}

// Takes the workspace's next part (the first 256 bytes of it all are the error word's).
static void attn_take_workspace(AttnParams& p, int64_t rows, int most_blocks, char*& ws)
{
    const AttnWs w = attn_layout(rows, p.a.n_seq, p.a.cache.dim, p.mb, most_blocks);
    p.head = reinterpret_cast<AttnHeader*>(ws + w.head);
    p.item_off = reinterpret_cast<int32_t*>(ws + w.item_off);
    p.items = reinterpret_cast<AttnItem*>(ws + w.items);
    p.joins = reinterpret_cast<AttnJoin*>(ws + w.joins);
    p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    ws += w.total;
}

static void launch_join(cudaError_t& err, const AttnParams& p, int64_t rows, bool chunk, cudaStream_t stream)
{
    constexpr int kWarps = kJoinThreads / 32;
    const int live = rows < p.mb ? static_cast<int>(rows) : p.mb;  // of an item, at most
    const dim3 grid(static_cast<unsigned>(p.blocks > 1 ? p.blocks - 1 : 1), (live + kWarps - 1) / kWarps);
    const auto join = p.a.cache.dim == 128 ? chunk ? attn_join_kernel<128, 4> : attn_join_kernel<128, 16>
                                           : chunk ? attn_join_kernel<64, 4> : attn_join_kernel<64, 16>;
    launch_dep(err, join, grid, dim3(kJoinThreads), 0, stream, p);
}

// Chunks: the items' list, the kernel, the join.
static void launch_chunks(cudaError_t& err, AttnParams p, int64_t rows, char*& ws, cudaStream_t stream)
{
    p.tile = kChunkTile;
    p.mb = p.a.cache.dim == 128 && rows > kChunkRows ? kPairRows : kChunkRows;
    const int most = chunk_max_blocks(p.mb);
    p.blocks = p.a.sm_count * kChunkRows / p.mb;
    if (p.blocks > most) p.blocks = most;
    attn_take_workspace(p, p.a.T * p.G, most, ws);
    launch_dep(err, attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
    if (err == cudaSuccess) err = launch_attention_chunk(p, stream);
    launch_join(err, p, rows, true, stream);
}

// Few rows a sequence.
static void launch_few_rows(cudaError_t& err, AttnParams p, int rows, bool deal, char*& ws, cudaStream_t stream)
{
    const AttentionArgs& a = p.a;
    p.tile = kMmaTile;
    p.mb = rows > 8 ? kMmaMaxRows : 8;
    p.blocks = mma_blocks_per_sm(p.mb, a.cache.dim, a.cache.int8) * a.sm_count;
    if (p.blocks > kAttnMaxBlocks) p.blocks = kAttnMaxBlocks;
    // Short caches, or few: a cluster of up to 8 blocks for each (sequence,
    // head), which needs no deal and no second launch.  (cap is the longest
    // cache as far as the page table's width says; 64/8 heads, bf16, pages of
    // 16, us on the GPU, the deal and its join against clusters:
    //   1 sequence    511 keys 8.7 / 6.7   2047 11.5 / 8.4   4000 13.0 / 10.7
    //   4             511      8.9 / 7.0   2047 15.6 / 10.6  4000 21.7 / 16.6
    //   16                                 1500 26.8 / 20.8  2047 31.7 / 25.5
    // and 27.9 / 22.8 for 16 whose lengths lie below 2047 at random.)  A
    // cluster is doubled while its blocks have more than 128 keys each and an
    // SM to themselves, or more than 256 and half an SM: 16 sequences of 1023
    // int8 keys take 20.0 with one block each and 17.0 with two, of 200 keys 8.0
    // and 8.7.  Blocks of more than 1024 keys are too uneven for what they
    // save; a block alone wins up to 512, or 1024 where there are many.
    const int64_t cap = a.max_pages * a.cache.page, pairs = a.n_seq * a.cache.n_kv;
    if (!deal) {
        int c = 1;
        const auto keys = [&] { return pairs * 2 * c <= a.sm_count ? 128 : 256; };  // a block's, where doubling pays
        while (c < 8 && pairs * 2 * c <= 2 * a.sm_count && cap > keys() * c) c *= 2;
        const int64_t most_keys = c > 1 || pairs >= 64 ? 1024 : 512;
        if (cap <= most_keys * c && pairs * c <= INT32_MAX) p.whole = c;
    }
    if (p.whole) p.blocks = static_cast<int>(pairs) * p.whole;
    attn_take_workspace(p, 0, kAttnMaxBlocks, ws);
    if (err == cudaSuccess) err = launch_attention_mma(p, stream);
    if (!p.whole) launch_join(err, p, p.mb, false, stream);
}

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t stream)
{
    if (a.T == 0 || a.n_seq == 0) return cudaSuccess;
    AttnParams p{};
    p.a = a;
    p.G = a.n_q / a.cache.n_kv;
    p.rows_upto = INT32_MAX;
    char* ws = static_cast<char*>(a.ws);
    cudaError_t err = cudaSuccess;
    // new tokens and rows of a sequence, as far as the host knows
    const int64_t max_new = a.max_new < a.T ? a.max_new : a.T, rows = max_new * p.G;
    if (rows <= kMmaMaxRows) {
        launch_few_rows(err, p, static_cast<int>(rows), false, ws, stream);
        return err;
    }
    // A batch that mixes chunks with decode steps: the sequences of up to 16
    // rows take the kernel for few rows, in a launch of its own, since a tile
    // of the other has 128 rows or more (a chunk of 512 tokens and m single
    // ones over 4000 keys, 64/8 heads, us apart / together: bf16 m = 1 88 / 77,
    // 7 108 / 108, 31 168 / 218; int8 109 / 101, 122 / 143, 157 / 302).  Not
    // where the number of tokens says that all sequences have max_new, nor for
    // few sequences, nor for chunks so small that the launch costs too much.
    const bool split = rows >= 128 && a.n_seq >= 4 && a.T < a.n_seq * max_new;
    if (split) p.rows_above = kMmaMaxRows;
    launch_chunks(err, p, rows, ws, stream);
    if (split) {
        p.rows_above = 0;
        p.rows_upto = kMmaMaxRows;
        launch_few_rows(err, p, p.G <= 8 ? 8 : kMmaMaxRows, true, ws, stream);
    }
    return err;
}

BD_BOUNDS_TAKE(bounds_take_attention)

}  // namespace bd
