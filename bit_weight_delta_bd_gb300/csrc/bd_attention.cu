// Attention over the paged KV cache: the plan, the kernel for few query rows
// per sequence (decode steps), and the join of partial results.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp2(c q_r . k_j - m_r),  c = scale log2(e)
//
// in one pass over the keys with a running maximum m_r: where a tile raises
// it, the sums so far are multiplied by exp2(m_old - m_new).
//
// The decode kernel is bound by the cache's bytes.  One thread of a producer
// warp's tile keeps a ring of stages (64 keys: K, V, scales) filled by TMA,
// one box per page; four consumer warps take turns, two of them 32 keys each
// of every other stage, with a running maximum, denominator and 16 x dim sum
// of their own, so that nothing is exchanged between warps until an item
// ends.  Rows are the 16 rows of m16n8k16 (query heads that share a kv head),
// keys its columns.
//
// Int8.  Both products run in fp16, which holds the codes exactly: with u =
// code + 128 the bits 0x6400 | u are 1024 + u, and one logic operation and
// one packed addition give two codes (bf16, whose 8 bits have no room for u,
// takes twice as many).  q is scaled per row by the power of two that brings
// its largest element to 2^14 .. 2^15: its bf16 values are then exact in fp16
// down to 2^-29 of that element.  K's scale multiplies the fp32 score.  V's
// scale multiplies the fp32 probability, and the product enters fp16 over a
// power of two that follows the largest scale seen, so that it stays below
// 2^15 and what is rounded away lies 2^-40 below the largest.  Probabilities
// so keep 11 bits, where a bf16 cache's, rounded to bf16 like its values, keep 8.

#include "bd_attention.cuh"

#include <cuda_fp16.h>

#include "bd_tma.h"

namespace bd {
namespace {

// ------------------------------------------------------------------------------- plan

constexpr int kPlanThreads = 1024;

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
            const AttnSeq q = attn_seq(a, s, true);
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
            const AttnSeq q = attn_seq(a, lo, false);
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
constexpr int kMmaRows = 16;     // rows of an item
constexpr int kMmaConsumers = 4;
constexpr int kMmaKeys = 32;     // keys of a stage that one warp takes
constexpr int kMmaThreads = 32 * (kMmaConsumers + 1);
constexpr int kMmaMaxStages = 8;

struct MmaParams {
    CUtensorMap k_map, v_map;  // [n_pages * n_kv][page][dim], box (128 bytes or a row) x min(page, 64)
    AttnParams p;
    int stages;
};

template <int DIM, bool INT8>
struct MmaShape {
    static constexpr int kRowBytes = DIM * (INT8 ? 1 : 2);
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one box
    static constexpr int kHalves = kRowBytes / kBoxBytes;
    static constexpr int kHalfBytes = kMmaTile * kBoxBytes;
    static constexpr int kTileBytes = kMmaTile * kRowBytes;               // K (or V) of a stage
    static constexpr int kStageBytes = 2 * kTileBytes + (INT8 ? 1024 : 0);  // stages stay 1024-byte aligned
    static constexpr int kBufBytes = 2 * kMmaRows * DIM * 4;              // sums of an item, two warps each
};

struct MmaShared {
    uint64_t full[kMmaMaxStages];
    uint64_t empty[kMmaMaxStages];
    float m[kMmaConsumers][kMmaRows];
    float l[kMmaConsumers][kMmaRows];
    volatile int abort;
    int64_t scan[kMmaThreads / 32];
    int seq, row0;      // the block's first item,
    int64_t before;     // and the units before it
};

// Key tiles of one head of the item of sequence q that starts at row0.
__device__ __forceinline__ int mma_tiles(const AttnParams& p, const AttnSeq& q, int row0)
{
    int last = row0 + kMmaRows - 1;
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
        s.sq = attn_seq(p.a, seq, false);
        s.rows = s.sq.n_new * p.G;
        s.tiles = mma_tiles(p, s.sq, row0);
        look_ahead();
    }
    __device__ __forceinline__ void look_ahead()
    {
        if (s.seq + 1 < p.a.n_seq) ahead = attn_seq(p.a, s.seq + 1, false);
    }
    __device__ __forceinline__ bool next()
    {
        if (u >= end) return false;
        const int n_kv = p.a.cache.n_kv;
        while (u - before >= static_cast<int64_t>(s.tiles) * n_kv) {  // on to the next item
            before += static_cast<int64_t>(s.tiles) * n_kv;
            s.row0 += kMmaRows;
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

// The whole block: adds up the tiles of all sequences (each thread those of
// consecutive ones) and finds the item of the block's first unit.  Returns
// the units of the call.
__device__ __forceinline__ int64_t mma_deal(const AttnParams& p, MmaShared& sh)
{
    const AttentionArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_seq = static_cast<int>(a.n_seq);
    const int per = (n_seq + kMmaThreads - 1) / kMmaThreads;
    const int s0 = static_cast<int>(threadIdx.x) * per < n_seq ? threadIdx.x * per : n_seq;
    const int s1 = s0 + per < n_seq ? s0 + per : n_seq;
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        const AttnSeq q = attn_seq(a, s, blockIdx.x == 0);
        for (int row0 = 0; row0 < q.n_new * p.G; row0 += kMmaRows) mine += mma_tiles(p, q, row0);
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
                const AttnSeq q = attn_seq(a, s, false);
                for (int row0 = 0; row0 < q.n_new * p.G; row0 += kMmaRows) {
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
    return units;
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

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
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

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kMmaConsumers) : "memory"); }

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

template <int DIM, bool INT8>
__global__ void __launch_bounds__(kMmaThreads, 2) attn_mma_kernel(const __grid_constant__ MmaParams mp)
{
    using S = MmaShape<DIM, INT8>;
    constexpr int kSteps = DIM / 16;  // MMA steps of q . k, and pairs of 8-dim tiles of the output
    // all of it dynamic: the ring starts on a 1024-byte boundary without padding
    extern __shared__ __align__(1024) uint8_t dyn_raw[];
    uint8_t* ring = dyn_raw;
    float* buf = reinterpret_cast<float*>(ring + static_cast<size_t>(mp.stages) * S::kStageBytes);
    MmaShared& sh = *reinterpret_cast<MmaShared*>(reinterpret_cast<uint8_t*>(buf) + S::kBufBytes);

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
        sh.abort = 0;
        fence_mbarrier_init();
    }
    __syncthreads();
    grid_dependency_wait();

    const int n_kv = cache.n_kv;
    const int64_t units = mma_deal(p, sh);
    const int active = attn_active(units, p.blocks);
    const int c = blockIdx.x;
    MmaWalk walk(p, c < active ? attn_first(units, active, c) : 0, c < active ? attn_first(units, active, c + 1) : 0,
                 sh.seq, sh.row0, sh.before);
    if (threadIdx.x == 0) {
        AttnJoin j{0, 0, 0, 0};
        if (c < active) {
            const int64_t rel = walk.u - walk.before;
            const int h = attn_div(rel, walk.s.tiles);
            j = attn_join_of(units, active, c, walk.u, walk.before + static_cast<int64_t>(h) * walk.s.tiles,
                             walk.s.tiles, walk.s.seq, walk.s.row0, h);
        }
        p.joins[c] = j;
    }
    if (c >= active) return;
    const MmaSegment& sg = walk.s;
    int stage = 0;
    uint32_t phase = 0;

    if (warp == kMmaConsumers) {
        // ------------------------------------------------------------ producer warp
        const int box_rows = cache.page < kMmaTile ? cache.page : kMmaTile;
        const int pages_per_tile = kMmaTile / box_rows;
        while (walk.next()) {
            const int h = sg.h;
            const int32_t* table = a.table + static_cast<int64_t>(sg.seq) * a.max_pages;
            const int pages = (sg.sq.len + cache.page - 1) >> cache.page_shift;  // that the sequence has
            for (int t = sg.t0; t < sg.t1; ++t) {
                // lane j looks after the j-th box of the tile
                const int key = t * kMmaTile + lane * box_rows;
                const int at = key >> cache.page_shift;
                const bool mine = lane < pages_per_tile && at < pages;
                int page = 0;
                if (mine) {
                    page = table[at];
                    if (page < 0 || page >= cache.n_pages) {
                        raise_error(a.err, kErrBadIndex);
                        page = 0;
                    }
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
#pragma unroll
                    for (int half = 0; half < S::kHalves; ++half) {
                        uint8_t* dst = st + half * S::kHalfBytes + lane * box_rows * S::kBoxBytes;
                        const int col = half * (S::kBoxBytes / (INT8 ? 1 : 2));
                        tma_load_3d(dst, &mp.k_map, col, row, outer, &sh.full[stage]);
                        tma_load_3d(dst + S::kTileBytes, &mp.v_map, col, row, outer, &sh.full[stage]);
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
    int turn = 0;  // stages so far: this warp takes those of its parity
    while (walk.next()) {
        const AttnSeq sq = sg.sq;
        const int h = sg.h, t0 = sg.t0, t1 = sg.t1, rows = sg.rows, row0 = sg.row0;

        // the two rows of this thread: keys they see, q as A fragments, and the factor of their scores
        int seen[2];
        float cr[2] = {c2, c2};
        uint32_t qf[kSteps][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = row0 + g + 8 * i;
            const bool live = r < rows;
            const int tok = live ? r / p.G : 0;
            seen[i] = live ? attn_seen(sq, tok, a.causal) : 0;
            const uint16_t* src = a.q + (static_cast<int64_t>(sq.q0) + tok) * a.q_stride +
                                  static_cast<int64_t>(h * p.G + (live ? r - tok * p.G : 0)) * DIM;
            if constexpr (INT8) {
                // a code fragment holds dims 4 q4 + {0, 2} and 4 q4 + {1, 3} of a step's 16
                float v[kSteps][4];
                float big = 0.0f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const uint2 w = live ? *reinterpret_cast<const uint2*>(src + 16 * k + 4 * q4) : make_uint2(0, 0);
                    v[k][0] = __uint_as_float(w.x << 16);
                    v[k][1] = __uint_as_float(w.x & 0xFFFF0000u);
                    v[k][2] = __uint_as_float(w.y << 16);
                    v[k][3] = __uint_as_float(w.y & 0xFFFF0000u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(v[k][e]));
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const float unit = pow2_of(big), f = 16384.0f / unit;
                cr[i] = c2 * (unit / 16384.0f);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    qf[k][i] = pack_f16x2(v[k][0] * f, v[k][2] * f);
                    qf[k][i + 2] = pack_f16x2(v[k][1] * f, v[k][3] * f);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int d = 16 * k + 2 * q4;
                    qf[k][i] = live ? *reinterpret_cast<const uint32_t*>(src + d) : 0u;
                    qf[k][i + 2] = live ? *reinterpret_cast<const uint32_t*>(src + d + 8) : 0u;
                }
            }
        }
        // the keys that every live row sees: below, no mask is needed
        const int all_seen = attn_seen(sq, row0 / p.G, a.causal);

        float o[2 * kSteps][4];
#pragma unroll
        for (int i = 0; i < 2 * kSteps; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
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

            // ---- scores of 16 rows x 32 keys: s[n] keys 8 n .. 8 n + 7
            float s[4][4] = {};
            if constexpr (INT8) {
#pragma unroll
                for (int k = 0; k < kSteps; k += 2)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t r[4];
                        ldsm_x4(st + swizzled<S::kBoxBytes>(slice + 16 * b + (mi & 1) * 8 + mr, k + (mi >> 1)), r);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma_f16_16816(s[2 * b + (x & 1)], qf[k + (x >> 1)][0], qf[k + (x >> 1)][1],
                                          qf[k + (x >> 1)][2], qf[k + (x >> 1)][3], codes_f16x2(r[x]),
                                          codes_f16x2(r[x] >> 8));
                    }
            } else {
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t r[4];
                        const int chunk = 2 * k + (mi & 1), row = slice + 16 * b + (mi >> 1) * 8 + mr;
                        ldsm_x4(st + (chunk >> 3) * S::kHalfBytes + swizzled<S::kBoxBytes>(row, chunk & 7), r);
                        mma_bf16_16816(s[2 * b], qf[k][0], qf[k][1], qf[k][2], qf[k][3], r[0], r[1]);
                        mma_bf16_16816(s[2 * b + 1], qf[k][0], qf[k][1], qf[k][2], qf[k][3], r[2], r[3]);
                    }
            }

            // ---- to units of log2, masked; this thread's keys are 8 n + 2 q4 + {0, 1}
            float vs[4][2];
            if constexpr (INT8) {
                const float* sc = reinterpret_cast<const float*>(ring + static_cast<size_t>(stage) * S::kStageBytes +
                                                                 2 * S::kTileBytes) +
                                  slice + 2 * q4;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 ks = *reinterpret_cast<const float2*>(sc + 8 * n);
                    const float2 v = *reinterpret_cast<const float2*>(sc + kMmaTile + 8 * n);
                    vs[n][0] = v.x;
                    vs[n][1] = v.y;
                    s[n][0] *= ks.x * cr[0];
                    s[n][1] *= ks.y * cr[0];
                    s[n][2] *= ks.x * cr[1];
                    s[n][3] *= ks.y * cr[1];
                }
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] *= c2;
            }
            const bool tail = key0 + kMmaKeys > sq.len;
            if (key0 + kMmaKeys > all_seen) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + 8 * n + 2 * q4 + (e & 1);
                        if (key >= seen[e >> 1]) s[n][e] = -INFINITY;
                        // what lies past the sequence may be anything, NaN included: zeros instead
                        if (INT8 && e < 2 && key >= sq.len) vs[n][e] = 0.0f;
                    }
            }

            // ---- running maximum
            float mt[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                v = fmaxf(v, fmaxf(fmaxf(s[2][2 * i], s[2][2 * i + 1]), fmaxf(s[3][2 * i], s[3][2 * i + 1])));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                mt[i] = fmaxf(m[i], v);
            }
            float v_new = v_unit;
            if constexpr (INT8) {
                float v = fmaxf(fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1])),
                                fmaxf(fmaxf(vs[2][0], vs[2][1]), fmaxf(vs[3][0], vs[3][1])));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                constexpr float kUnit = static_cast<float>(1u << (static_cast<int>(attn_bias<true>()) - 14));
                if (v * (0.5f * kUnit) > 0.5f * v_unit) v_new = pow2_of(v) * kUnit;
            }
            if (__any_sync(0xffffffffu, mt[0] > m[0] || mt[1] > m[1] || v_new != v_unit)) {
                const float fv = INT8 && v_new != v_unit ? v_unit / v_new : 1.0f;
                v_unit = v_new;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float f = mt[i] == -INFINITY ? 1.0f : exp2f(m[i] - mt[i]);
                    m[i] = mt[i];
                    l[i] *= f;
#pragma unroll
                    for (int n = 0; n < 2 * kSteps; ++n) {
                        o[n][2 * i] *= f * fv;
                        o[n][2 * i + 1] *= f * fv;
                    }
                }
            }

            // ---- probabilities as A fragments of two steps of 16 keys
            uint32_t pa[2][4];
            const float v_inv = INT8 ? (v_unit > 0.0f ? 1.0f / v_unit : 0.0f) : 1.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mu = m[i] == -INFINITY ? 0.0f : m[i] - attn_bias<INT8>();
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float p0 = ex2(s[2 * b][2 * i] - mu), p1 = ex2(s[2 * b][2 * i + 1] - mu);
                    const float p2 = ex2(s[2 * b + 1][2 * i] - mu), p3 = ex2(s[2 * b + 1][2 * i + 1] - mu);
                    l[i] += (p0 + p1) + (p2 + p3);
                    if constexpr (INT8) {
                        pa[b][i] = pack_f16x2(p0 * (vs[2 * b][0] * v_inv), p1 * (vs[2 * b][1] * v_inv));
                        pa[b][i + 2] = pack_f16x2(p2 * (vs[2 * b + 1][0] * v_inv), p3 * (vs[2 * b + 1][1] * v_inv));
                    } else {
                        pa[b][i] = pack_bf16x2(p0, p1);
                        pa[b][i + 2] = pack_bf16x2(p2, p3);
                    }
                }
            }

            // ---- sums: 16 rows x dim += P (16 x 32) V (32 x dim)
            const uint32_t vt = st + S::kTileBytes;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int row = slice + 16 * b + (mi & 1) * 8 + mr;
                if constexpr (INT8) {
                    // a b16 element is a pair of dims: the transposed fragment holds dims 2n, 2n + 1 of
                    // two keys; tile 2k takes the even dims of a chunk, tile 2k + 1 the odd ones
#pragma unroll
                    for (int k = 0; k < kSteps; k += 2) {
                        uint32_t r[4];
                        ldsm_x4_t(vt + swizzled<S::kBoxBytes>(row, k + (mi >> 1)), r);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            mma_f16_16816(o[2 * (k + x)], pa[b][0], pa[b][1], pa[b][2], pa[b][3],
                                          codes_f16x2(r[2 * x]), codes_f16x2(r[2 * x + 1]));
                            mma_f16_16816(o[2 * (k + x) + 1], pa[b][0], pa[b][1], pa[b][2], pa[b][3],
                                          codes_f16x2(r[2 * x] >> 8), codes_f16x2(r[2 * x + 1] >> 8));
                        }
                    }
                } else {
                    uint32_t mask0 = 0xFFFFFFFFu, mask1 = 0xFFFFFFFFu;
                    if (tail) {
                        // zeros for what lies past the sequence
                        const int k = key0 + 16 * b + 2 * q4;
                        mask0 = (k < sq.len ? 0xFFFFu : 0u) | (k + 1 < sq.len ? 0xFFFF0000u : 0u);
                        mask1 = (k + 8 < sq.len ? 0xFFFFu : 0u) | (k + 9 < sq.len ? 0xFFFF0000u : 0u);
                    }
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        uint32_t r[4];
                        const int chunk = 2 * k + (mi >> 1);
                        ldsm_x4_t(vt + (chunk >> 3) * S::kHalfBytes + swizzled<S::kBoxBytes>(row, chunk & 7), r);
                        if (tail) {
                            r[0] &= mask0;
                            r[1] &= mask1;
                            r[2] &= mask0;
                            r[3] &= mask1;
                        }
                        mma_bf16_16816(o[2 * k], pa[b][0], pa[b][1], pa[b][2], pa[b][3], r[0], r[1]);
                        mma_bf16_16816(o[2 * k + 1], pa[b][0], pa[b][1], pa[b][2], pa[b][3], r[2], r[3]);
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
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (q4 == 0) {
                sh.m[warp][g + 8 * i] = m[i] - attn_bias<INT8>();
                sh.l[warp][g + 8 * i] = l[i];
            }
        }
        consumers_sync();
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mm = sh.m[0][g + 8 * i];
#pragma unroll
            for (int w = 1; w < kMmaConsumers; ++w) mm = fmaxf(mm, sh.m[w][g + 8 * i]);
            f[i] = attn_weight(m[i] - attn_bias<INT8>(), l[i], mm);
            if (INT8 && f[i] != 0.0f) f[i] *= v_unit;  // the sums are over the scales' unit
        }
        for (int w = 0; w < 2; ++w) {
            if ((warp >> 1) == w) {
                float* mine = buf + (warp & 1) * kMmaRows * DIM;
#pragma unroll
                for (int n = 0; n < 2 * kSteps; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // bf16: tile n, columns 2 q4 + {0, 1}; int8: chunk n / 2, dims 4 q4 + {0, 2} of
                        // the even tile and 4 q4 + {1, 3} of the odd one, kept at places 2 (n & 1) + {0, 1}
                        const int d = INT8 ? 16 * (n >> 1) + 4 * q4 + 2 * (n & 1) : 8 * n + 2 * q4;
                        float2* b = reinterpret_cast<float2*>(mine + (g + 8 * i) * DIM + d);
                        float2 v = make_float2(0.0f, 0.0f);
                        if (f[i] != 0.0f) v = make_float2(o[n][2 * i] * f[i], o[n][2 * i + 1] * f[i]);
                        if (w == 1) {
                            const float2 x = *b;
                            v.x += x.x;
                            v.y += x.y;
                        }
                        *b = v;
                    }
            }
            consumers_sync();
        }

        const bool whole = t0 == 0 && t1 == sg.tiles;
        const int slot = attn_slot(c, t0 == 0);
        const int live_rows = rows - row0 < kMmaRows ? rows - row0 : kMmaRows;
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
            float4 v = *reinterpret_cast<const float4*>(buf + r * DIM + d);
            const float4 v1 = *reinterpret_cast<const float4*>(buf + kMmaRows * DIM + r * DIM + d);
            v = make_float4(v.x + v1.x, v.y + v1.y, v.z + v1.z, v.w + v1.w);
            if constexpr (INT8) v = make_float4(v.x, v.z, v.y, v.w);  // from places to dims
            if (whole) {
                const int row = row0 + r, tok = row / p.G;
                const int64_t at = (static_cast<int64_t>(sq.q0) + tok) * a.n_q + h * p.G + (row - tok * p.G);
                const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
                if (bd_in(kBkAttn, at, a.T * a.n_q)) {
                    *reinterpret_cast<uint2*>(a.out + at * DIM + d) =
                        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                    if (d == 0 && a.lse) a.lse[at] = attn_lse(mm, ll);
                }
            } else {
                const int64_t at = static_cast<int64_t>(slot) * kMmaRows + r;
                if (bd_in(kBkAttn, at, 2ll * p.blocks * kMmaRows)) {
                    *reinterpret_cast<float4*>(p.part_o + at * DIM + d) = v;
                    if (d == 0) p.part_ml[at] = make_float2(mm, ll);
                }
            }
        }
        consumers_sync();  // the buffers are free for the next item
    }
}

// ------------------------------------------------------------------------------- join

constexpr int kJoinThreads = 128;

// Block (c, y): joins what block c of the main kernel noted down; a warp takes the rows
// 4 y + w, 4 (y + gridDim.y) + w, ...
template <int DIM>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kPer = DIM / 32;  // values of a lane
    grid_launch_dependents();
    grid_dependency_wait();
    const AttentionArgs& a = p.a;
    const int c = blockIdx.x + 1;
    const AttnJoin it = p.joins[c];
    if (it.parts == 0) return;
    const int lane = threadIdx.x & 31;
    const int h = it.h, parts = it.parts;
    const AttnSeq sq = attn_seq(a, it.seq, false);
    const int rows = sq.n_new * p.G;
    const int live = rows - it.row0 < p.mb ? rows - it.row0 : p.mb;
    for (int r = 4 * blockIdx.y + (threadIdx.x >> 5); r < live; r += 4 * gridDim.y) {
        float mm = -INFINITY;
        for (int i = lane; i < parts; i += 32)
            mm = fmaxf(mm, p.part_ml[static_cast<int64_t>(attn_slot(c - 1 + i, i == 0)) * p.mb + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        float acc[kPer] = {}, ll = 0.0f;
        for (int i0 = 0; i0 < parts; i0 += 32) {
            float w = 0.0f, lw = 0.0f;
            if (i0 + lane < parts) {
                const float2 ml =
                    p.part_ml[static_cast<int64_t>(attn_slot(c - 1 + i0 + lane, i0 + lane == 0)) * p.mb + r];
                w = attn_weight(ml.x, ml.y, mm);
                lw = ml.y;
            }
            const int n = parts - i0 < 32 ? parts - i0 : 32;
            for (int j0 = 0; j0 < n; j0 += 8) {
                float v[8][kPer];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = i0 + (j0 + j < n ? j0 + j : n - 1);
                    const float* src =
                        p.part_o + (static_cast<int64_t>(attn_slot(c - 1 + i, i == 0)) * p.mb + r) * DIM + kPer * lane;
                    if constexpr (kPer == 4) {
                        const float4 x = *reinterpret_cast<const float4*>(src);
                        v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2*>(src);
                        v[j][0] = x.x, v[j][1] = x.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float wi = __shfl_sync(0xffffffffu, w, j0 + j), li = __shfl_sync(0xffffffffu, lw, j0 + j);
                    if (j0 + j < n && wi != 0.0f) {
                        ll += wi * li;
#pragma unroll
                        for (int e = 0; e < kPer; ++e) acc[e] += wi * v[j][e];
                    }
                }
            }
        }
        const int row = it.row0 + r, tok = row / p.G;
        const int64_t at = (static_cast<int64_t>(sq.q0) + tok) * a.n_q + h * p.G + (row - tok * p.G);
        if (!bd_in(kBkAttnCombine, at, a.T * a.n_q)) continue;
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * DIM + kPer * lane);
#pragma unroll
        for (int e = 0; e < kPer; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        if (lane == 0 && a.lse) a.lse[at] = attn_lse(mm, ll);
    }
}

template <int DIM, bool INT8>
cudaError_t launch_mma_shape(const AttnParams& p, cudaStream_t stream)
{
    using S = MmaShape<DIM, INT8>;
    static std::atomic<size_t> smem_set[kHostMaxDevices];
    const KvPages& kv = p.a.cache;
    MmaParams mp{};
    mp.p = p;
    const uint32_t box_rows = kv.page < kMmaTile ? kv.page : kMmaTile;
    const auto type = INT8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto swz = S::kBoxBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const uint64_t outer = static_cast<uint64_t>(kv.n_pages) * kv.n_kv;
    for (int i = 0; i < 2; ++i)
        if (!encode_tma_3d(i ? &mp.v_map : &mp.k_map, type, INT8 ? 1 : 2, i ? kv.v : kv.k, DIM, kv.page, outer,
                           S::kBoxBytes / (INT8 ? 1 : 2), box_rows, swz))
            return cudaErrorInvalidValue;
    // two blocks per SM: 113 KB each
    constexpr size_t kBudget = 113u * 1024u, kRest = S::kBufBytes + sizeof(MmaShared);
    mp.stages = static_cast<int>((kBudget - kRest) / S::kStageBytes);
    if (mp.stages > kMmaMaxStages) mp.stages = kMmaMaxStages;
    const size_t smem = static_cast<size_t>(mp.stages) * S::kStageBytes + kRest;
    cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(attn_mma_kernel<DIM, INT8>), smem, smem_set);
    launch_dep(err, attn_mma_kernel<DIM, INT8>, dim3(p.blocks), dim3(kMmaThreads), smem, stream, mp);
    return err;
}

constexpr size_t align_up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct AttnWs {
    size_t head, item_off, items, joins, ml, o, total;
};

AttnWs attn_layout(int64_t T, int64_t n_seq, int64_t G, int dim, int mb, int blocks)
{
    AttnWs w{};
    w.head = 256;
    w.item_off = w.head + 256;
    w.items = w.item_off + align_up(static_cast<size_t>(n_seq + 1) * 4);
    const size_t items = static_cast<size_t>((T * G + mb - 1) / mb + n_seq);
    w.joins = w.items + align_up(items * sizeof(AttnItem));
    w.ml = w.joins + align_up(static_cast<size_t>(blocks) * sizeof(AttnJoin));
    w.o = w.ml + align_up(static_cast<size_t>(2 * blocks) * mb * 8);
    w.total = w.o + align_up(static_cast<size_t>(2 * blocks) * mb * dim * 4);
    return w;
}

}  // namespace

cudaError_t launch_attention_mma(const AttnParams& p, cudaStream_t stream)
{
    if (p.a.cache.dim == 128)
        return p.a.cache.int8 ? launch_mma_shape<128, true>(p, stream) : launch_mma_shape<128, false>(p, stream);
    return p.a.cache.int8 ? launch_mma_shape<64, true>(p, stream) : launch_mma_shape<64, false>(p, stream);
}

size_t attention_workspace_size(int64_t T, int64_t n_seq, int n_q, int n_kv, int dim)
{
    // the host may learn how long the chunks are only with the call: room for either kernel
    const int G = n_q / n_kv;
    const size_t mma = attn_layout(T, n_seq, G, dim, kMmaRows, kAttnMaxBlocks).total;
    const size_t chunk = attn_layout(T, n_seq, G, dim, kChunkRows, kAttnMaxBlocks / 2).total;
    return mma > chunk ? mma : chunk;
}

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t stream)
{
    if (a.T == 0 || a.n_seq == 0) return cudaSuccess;
    AttnParams p{};
    p.a = a;
    p.G = a.n_q / a.cache.n_kv;
    const bool chunk = a.max_new * p.G > kMmaRows;
    p.tile = chunk ? kChunkTile : kMmaTile;
    p.mb = chunk ? kChunkRows : kMmaRows;
    const int most = chunk ? kAttnMaxBlocks / 2 : kAttnMaxBlocks;
    p.blocks = chunk ? a.sm_count : 2 * a.sm_count;
    if (p.blocks > most) p.blocks = most;
    const AttnWs w = attn_layout(a.T, a.n_seq, p.G, a.cache.dim, p.mb, most);
    char* ws = static_cast<char*>(a.ws);
    p.head = reinterpret_cast<AttnHeader*>(ws + w.head);
    p.item_off = reinterpret_cast<int32_t*>(ws + w.item_off);
    p.items = reinterpret_cast<AttnItem*>(ws + w.items);
    p.joins = reinterpret_cast<AttnJoin*>(ws + w.joins);
    p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    p.part_o = reinterpret_cast<float*>(ws + w.o);
    cudaError_t err = cudaSuccess;
    if (chunk) launch_dep(err, attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
    if (err == cudaSuccess) err = chunk ? launch_attention_chunk(p, stream) : launch_attention_mma(p, stream);
    const dim3 grid(static_cast<unsigned>(p.blocks > 1 ? p.blocks - 1 : 1), chunk ? 16 : 4);
    launch_dep(err, a.cache.dim == 128 ? attn_join_kernel<128> : attn_join_kernel<64>, grid, dim3(kJoinThreads), 0,
               stream, p);
    return err;
}

BD_BOUNDS_TAKE(bounds_take_attention)

}  // namespace bd
