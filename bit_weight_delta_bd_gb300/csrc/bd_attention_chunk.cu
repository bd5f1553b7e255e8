// Attention over the paged KV cache for chunks of new tokens, on the tcgen05
// tensor cores (the formulas and the dealing of the work: bd_attention.cuh).
//
// An item is 256 query rows (two tiles of 128) of one kv head; its keys are
// read in tiles of 128 by TMA.  Per key tile and query tile
//   S = Q K^T       128 x 128, operands in shared memory, fp32 in tensor memory
//   P = exp2(c S - m)   one thread per row: maximum, probabilities, denominator
//   O += P V        P as bf16 in tensor memory (over S), V in shared memory
// Two warpgroups, one per query tile, take turns with the tensor cores: while
// one computes probabilities, the products of the other run.  The running
// maximum that P is formed with lags behind the true one by at most 2^8 (a
// row's sums are rescaled in tensor memory only when its maximum grew by more
// than 8 in units of log2; the fp32 sums have room for that factor), so that
// rescaling is rare after a row's first tiles.  A warp issues the products of
// both tiles in order, which also orders them: the commit that announces S of
// key tile t + 1 stands behind P V of tile t.
//
// Int8 keys and values: TMA brings the codes, a fourth warpgroup turns them
// into bf16 tiles (exactly, as in the decode kernel), once for both query
// tiles; the scales multiply S and P in the softmax's registers.
//
// Warps: 0..3 and 4..7 softmax of query tiles 0 and 1 (and loading Q, and
// writing O); 8 TMA; 9 MMA; 12..15 conversion (int8).
#include <type_traits>

#include "bd_attention.cuh"
#include "bd_tcgen05.cuh"
#include "bd_tma.h"

namespace bd {
namespace {

constexpr int kTile = 128;       // keys of a tile
constexpr int kQRows = 128;      // rows of a query tile
constexpr float kLag = 8.0f;     // how far (log2) a row's maximum may run ahead of the one in use

struct ChunkParams {
    CUtensorMap k_map, v_map;  // [n_pages * n_kv][page][dim]; bf16: box 64 x page rows, 128-byte swizzle; int8: box dim x page rows
    AttnParams p;
};

template <int DIM, bool INT8>
struct ChunkShape {
    static constexpr int kThreads = INT8 ? 512 : 384;
    static constexpr int kBufs = INT8 ? 3 : (DIM == 128 ? 5 : 8);  // bf16 tiles in shared memory
    static constexpr int kRaw = INT8 ? 3 : 0;                      // tiles of codes
    static constexpr int kScaleBufs = INT8 ? 3 : 0;                // scales of a key tile, K and V
    static constexpr int kHalves = DIM / 64;
    static constexpr int kHalfBytes = kTile * 128;                 // 64 dims of 128 keys
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kRawBytes = kTile * DIM;
    static constexpr int kQBytes = kQRows * DIM * 2;
    static constexpr int kOffBufs = 2 * kQBytes;
    static constexpr int kOffRaw = kOffBufs + kBufs * kTileBytes;
    static constexpr int kOffScale = kOffRaw + kRaw * kRawBytes;
    static constexpr int kBytes = kOffScale + kScaleBufs * 2 * kTile * 4;
    // registers of a softmax thread, and of the others: the sum over the
    // warpgroups is what the block was launched with
    static constexpr int kSoftRegs = INT8 ? 184 : 216;
    static constexpr int kOtherRegs = 72;
    static_assert(2 * kSoftRegs + (INT8 ? 2 : 1) * kOtherRegs <= (INT8 ? 4 * 128 : 3 * 168), "register split");
    static_assert(kBytes + 1024 + 1024 <= 227 * 1024, "shared memory");
};

constexpr int kMaxBufs = 8;

struct ChunkShared {
    uint64_t full[kMaxBufs], empty[kMaxBufs];    // bf16 tiles
    uint64_t raw_full[3], raw_empty[3];          // tiles of codes
    uint64_t sc_full[3], sc_empty[3];            // scales
    uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2];  // P in two halves of 64 keys
    uint64_t done;
    uint32_t tmem;
    volatile int abort;
};

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;  // S tiles at 0 and 128, O tiles from 256 on

// A wait of a whole warp; false (for all lanes) once the block has given up.
__device__ __forceinline__ bool warp_wait(volatile int* abort_flag, uint64_t* bar, uint32_t parity, uint32_t* err)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool late = global_timer_ns() - t0 > kWaitLimitNs;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            if (late && !*abort_flag) {
                *abort_flag = 1;
                raise_error(err, kErrTimeout);
            }
            return false;
        }
    }
}

template <int N>
__device__ __forceinline__ void reg_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// 32 columns of this warp's lanes, not waited for
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// Waits for the loads started so far; v is named so that no use of it moves above the wait.
__device__ __forceinline__ void tmem_ld_wait(uint32_t* v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}

__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Shared-memory descriptor of an operand whose rows run along the contracted
// index and whose 64-element (128-byte, swizzled) rows run along N: blocks of
// 64 along N are `block` bytes apart, groups of 8 rows 1024 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t block)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((block >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// One lane of the warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Two fp32 values in one 64-bit register, and their packed arithmetic.
__device__ __forceinline__ uint64_t f32x2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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

// codes (byte picks 0..1 and 2..3 of r) as pairs of bf16: see bd_attention.cu
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t r, uint32_t sel)
{
    const uint32_t x = __byte_perm(r, 0x43434343u, sel);
    const uint32_t hi = x & 0xFF7FFF7Fu, lo = x & 0xFF80FF80u;
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&hi), *reinterpret_cast<const __nv_bfloat162*>(&lo));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// What a block does next: key tiles [t0, t1) of one (item, kv head).
struct Segment {
    AttnItem it;
    AttnSeq sq;
    int h, t0, t1, rows, q_tiles;
};

struct Walk {
    const AttnParams& p;
    int64_t u, end;
    int item;

    __device__ __forceinline__ bool next(Segment& s)
    {
        if (u >= end) return false;
        const int n_kv = p.a.cache.n_kv;
        s.it = p.items[item];
        const int64_t rel = u - static_cast<int64_t>(s.it.before) * n_kv;
        s.h = attn_div(rel, s.it.tiles);
        s.t0 = static_cast<int>(rel - static_cast<int64_t>(s.h) * s.it.tiles);
        const int64_t left = end - u;
        s.t1 = left < s.it.tiles - s.t0 ? s.t0 + static_cast<int>(left) : s.it.tiles;
        s.sq = attn_seq(p.a, s.it.seq, false);
        s.rows = s.sq.n_new * p.G - s.it.row0;
        u += s.t1 - s.t0;
        if (s.t1 == s.it.tiles && s.h == n_kv - 1) ++item;
        // known for uniform
        s.t0 = __shfl_sync(0xffffffffu, s.t0, 0);
        s.t1 = __shfl_sync(0xffffffffu, s.t1, 0);
        s.rows = __shfl_sync(0xffffffffu, s.rows, 0);
        s.sq.len = __shfl_sync(0xffffffffu, s.sq.len, 0);
        s.q_tiles = s.rows > kQRows ? 2 : 1;
        return true;
    }
};

// This thread's row of a segment's query tile i, in shared memory (K-major,
// 128-byte swizzle, halves of 64 dims); rows past the item are zeros.  A
// negative scale is taken into Q's sign.
template <int DIM>
__device__ __forceinline__ void load_q_row(const AttnParams& p, const Segment& s, int i, int r, uint8_t* dst)
{
    const AttentionArgs& a = p.a;
    const int row = i * kQRows + r;
    const bool live = row < s.rows && row < p.mb;
    const int abs_row = s.it.row0 + row, tok = live ? abs_row / p.G : 0;
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + (static_cast<int64_t>(s.sq.q0) + tok) * a.q_stride +
        static_cast<int64_t>(s.h * p.G + (live ? abs_row - tok * p.G : 0)) * DIM);
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int c = 0; c < DIM / 8; ++c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = src[c];
        v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
        *reinterpret_cast<uint4*>(dst + (c >> 3) * (kQRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
    }
}

template <int DIM, bool INT8>
__global__ void __launch_bounds__(ChunkShape<DIM, INT8>::kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ ChunkParams cp)
{
    using S = ChunkShape<DIM, INT8>;
    extern __shared__ uint8_t dyn_raw[];
    __shared__ ChunkShared sh;
    uint8_t* dyn = dyn_raw + ((1024u - (smem_u32(dyn_raw) & 1023u)) & 1023u);
    const AttnParams& p = cp.p;
    const AttentionArgs& a = p.a;
    const KvPages& cache = a.cache;
    // (taken from lane 0, so that the compiler knows it for uniform: the
    // branches below, and the descriptors that the MMA warp forms in them)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&sh.full[i], INT8 ? 4 : 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
            mbar_init(&sh.sc_full[i], 1);
            mbar_init(&sh.sc_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 4);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 4);
            mbar_init(&sh.p_full[i][1], 4);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.done, 1);
        sh.abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 9) tmem_alloc(&sh.tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();

    const uint32_t tmem = sh.tmem;
    const AttnHeader head = *p.head;
    const int n_kv = cache.n_kv;
    const int64_t units = static_cast<int64_t>(head.tiles) * n_kv;
    const int active = attn_active(units, p.blocks);
    const int c = blockIdx.x;
    Walk walk{p, 0, 0, 0};
    if (c < active) {
        walk.u = attn_first(units, active, c);
        walk.end = attn_first(units, active, c + 1);
        walk.item = attn_find_item(p.items, head.n_items, n_kv, walk.u);
    }
    if (threadIdx.x == 0) {
        AttnJoin j{0, 0, 0, 0};
        if (c < active) {
            const AttnItem it = p.items[walk.item];
            const int64_t first = static_cast<int64_t>(it.before) * n_kv;
            const int h = attn_div(walk.u - first, it.tiles);
            j = attn_join_of(units, active, c, walk.u, first + static_cast<int64_t>(h) * it.tiles, it.tiles, it.seq,
                             it.row0, h);
        }
        p.joins[c] = j;
    }
    __syncwarp();
    Segment s;

    if (warp < 8) {
        // -------------------------------------------------------- softmax of query tile i
        reg_inc<S::kSoftRegs>();
        const int i = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + i * 128, to = tmem + lane_base + kTmemO + i * DIM;
        uint8_t* q_smem = dyn + i * S::kQBytes;
        const float c2 = fabsf(a.scale) * kLog2e;
        uint32_t s_phase = 0, o_phase = 0, sc_phase = 0;
        int sc = 0;
        bool have = walk.next(s);
        bool ok = true;
        const auto put_q = [&](const Segment& q) {
            load_q_row<DIM>(p, q, i, r, q_smem);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full[i]);
        };
        if (have && i < s.q_tiles) put_q(s);
        while (have && ok) {
            const Segment cur = s;
            if (i >= cur.q_tiles) {
                // no rows here: only the scales' slots have to be handed on
                if constexpr (INT8) {
                    for (int t = cur.t0; t < cur.t1 && ok; ++t) {
                        ok = warp_wait(&sh.abort, &sh.sc_full[sc], sc_phase, a.err);
                        if (lane == 0) mbar_arrive(&sh.sc_empty[sc]);
                        if (++sc == S::kScaleBufs) sc = 0, sc_phase ^= 1;
                    }
                }
                have = walk.next(s);
                if (have && i < s.q_tiles) put_q(s);
                continue;
            }
            const int row = i * kQRows + r;
            const bool live = row < cur.rows && row < p.mb;
            const int abs_row = cur.it.row0 + row, tok = live ? abs_row / p.G : 0;
            const int seen = live ? attn_seen(cur.sq, tok, a.causal) : 0;
            // what the tile's first row sees (the others see at least as much): below it no mask
            const int all_seen = attn_seen(cur.sq, (cur.it.row0 + i * kQRows) / p.G, a.causal);
            float m = -INFINITY, l = 0.0f;
            for (int t = cur.t0; t < cur.t1; ++t) {
                if (!(ok = warp_wait(&sh.abort, &sh.s_full[i], s_phase, a.err))) break;
                s_phase ^= 1;
                tc_fence_after();
                uint32_t v[128];
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld32_start(ts + 32 * j, v + 32 * j);
                const float *ks = nullptr, *vs = nullptr;
                if constexpr (INT8) {
                    ok = warp_wait(&sh.abort, &sh.sc_full[sc], sc_phase, a.err);
                    ks = reinterpret_cast<const float*>(dyn + S::kOffScale) + sc * 2 * kTile;
                    vs = ks + kTile;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld_wait(v + 32 * j);
                if (!ok) break;
                if constexpr (INT8) {
#pragma unroll
                    for (int j = 0; j < 128; j += 4) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(ks + j);
                        const float2 a0 = unpack2(mul2(f32x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), f.x));
                        const float2 a1 =
                            unpack2(mul2(f32x2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), f.y));
                        v[j] = __float_as_uint(a0.x), v[j + 1] = __float_as_uint(a0.y);
                        v[j + 2] = __float_as_uint(a1.x), v[j + 3] = __float_as_uint(a1.y);
                    }
                }
                const int left = seen - t * kTile;  // keys of the tile that this row sees
                const bool masked = (t + 1) * kTile > all_seen;
                if (masked) {
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j >= left) v[j] = 0xFF800000u;  // -infinity
                }
                __syncwarp();
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
#pragma unroll
                for (int j = 8; j < 128; j += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = max3(mx[k], __uint_as_float(v[j + 2 * k]), __uint_as_float(v[j + 2 * k + 1]));
                const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                if (t == cur.t0) {
                    m = mt;
                } else {
                    const bool grow = mt > m && (m == -INFINITY || (mt - m) * c2 > kLag);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = !grow ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - mt) * c2);
                        if (grow) m = mt;
                        l *= f;
#pragma unroll
                        for (int j = 0; j < DIM; j += 32) {
                            uint32_t o[32];
                            tmem_ld32_start(to + j, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16_start(to + j, o);
                            tmem_st16_start(to + j + 16, o + 16);
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : fmaf(-m, c2, attn_bias<INT8>());
                uint64_t sum[2] = {0, 0};  // pairs of zeros
                const uint64_t c22 = f32x2(c2, c2), nm2 = f32x2(nm, nm);
                const auto probabilities = [&](auto mask) {
                    constexpr bool kMask = decltype(mask)::value;
#pragma unroll
                    for (int j = 0; j < 128; j += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            [[maybe_unused]] ulonglong2 f{};
                            if constexpr (INT8) f = *reinterpret_cast<const ulonglong2*>(vs + j + e);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int at = j + e + 2 * k;
                                float2 pr =
                                    unpack2(fma2(f32x2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), c22, nm2));
                                pr.x = ex2(pr.x);
                                pr.y = ex2(pr.y);
                                if (kMask && at >= left) pr.x = 0.0f;
                                if (kMask && at + 1 >= left) pr.y = 0.0f;
                                const uint64_t pp = f32x2(pr.x, pr.y);
                                sum[k] = add2(sum[k], pp);
                                if constexpr (INT8) {
                                    pr = unpack2(mul2(pp, k ? f.y : f.x));
                                    if (kMask && at >= left) pr.x = 0.0f;
                                    if (kMask && at + 1 >= left) pr.y = 0.0f;
                                }
                                pk[e / 2 + k] = pack_bf16x2(pr.x, pr.y);
                            }
                        }
                        tmem_st16_start(ts + j / 2, pk);
                        if (j == 32 || j == 96) {
                            // P V of this half may start
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh.p_full[i][j == 96]);
                        }
                    }
                };
                if (masked) probabilities(std::true_type{});
                else probabilities(std::false_type{});
                const float2 s2 = unpack2(add2(sum[0], sum[1]));
                l += s2.x + s2.y;
                if constexpr (INT8) {
                    if (lane == 0) mbar_arrive(&sh.sc_empty[sc]);
                    if (++sc == S::kScaleBufs) sc = 0, sc_phase ^= 1;
                }
            }
            if (!ok) break;
            // the products with this Q are done (S of the last tile stood behind them): the next one
            // may come in while the last P V runs
            have = walk.next(s);
            if (have && i < s.q_tiles) put_q(s);
            if (!(ok = warp_wait(&sh.abort, &sh.o_full[i], o_phase, a.err))) break;
            o_phase ^= 1;
            tc_fence_after();
            const bool whole = cur.t0 == 0 && cur.t1 == cur.it.tiles;
            const int64_t at = (static_cast<int64_t>(cur.sq.q0) + tok) * a.n_q + cur.h * p.G + (abs_row - tok * p.G);
            const int64_t part = static_cast<int64_t>(attn_slot(c, cur.t0 == 0)) * p.mb + row;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float m2 = m == -INFINITY ? -INFINITY : fmaf(m, c2, -attn_bias<INT8>());
#pragma unroll
            for (int j = 0; j < DIM; j += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32_start(to + j, o);
                tmem_ld_wait(o);
                if (live && whole && bd_in(kBkAttn, at, a.T * a.n_q)) {
                    uint4* dst = reinterpret_cast<uint4*>(a.out + at * DIM + j);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv);
                        dst[e / 8] = l == 0.0f ? make_uint4(0, 0, 0, 0) : make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (live && !whole && bd_in(kBkAttn, part, 2ll * p.blocks * p.mb)) {
                    uint4* dst = reinterpret_cast<uint4*>(p.part_o + part * DIM + j);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) dst[e / 4] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
            if (live) {
                if (!whole)
                    p.part_ml[part] = make_float2(m2, l);
                else if (a.lse)
                    a.lse[at] = attn_lse(m2, l);
            }
            __syncwarp();
            tc_fence_before();
        }
    } else if (warp < 12) {
        reg_dec<S::kOtherRegs>();
        if (warp == 8) {
            // ---------------------------------------------------- TMA
            constexpr int kRing = INT8 ? S::kRaw : S::kBufs;
            uint64_t* full = INT8 ? sh.raw_full : sh.full;
            uint64_t* empty = INT8 ? sh.raw_empty : sh.empty;
            const int box_rows = cache.page;  // at most 128
            const int pages_per_tile = kTile / box_rows;
            int buf = 0, sc = 0;
            uint32_t phase = 0, sc_phase = 0;
            bool ok = true;
            while (ok && walk.next(s)) {
                const int32_t* table = a.table + static_cast<int64_t>(s.it.seq) * a.max_pages;
                const int pages = (s.sq.len + cache.page - 1) >> cache.page_shift;
                for (int t = s.t0; t < s.t1 && ok; ++t) {
                    // lane j looks after the j-th page of the tile
                    const int at = t * pages_per_tile + lane;
                    const bool mine = lane < pages_per_tile && at < pages;
                    int page = 0;
                    if (mine) {
                        page = table[at];
                        if (page < 0 || page >= cache.n_pages) {
                            raise_error(a.err, kErrBadIndex);
                            page = 0;
                        }
                    }
                    const int outer = page * n_kv + s.h;
                    const uint32_t rows = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, mine)) * box_rows);
                    if constexpr (INT8) {
                        if (!(ok = warp_wait(&sh.abort, &sh.sc_empty[sc], sc_phase ^ 1, a.err))) break;
                        if (lane == 0) mbar_arrive_expect_tx(&sh.sc_full[sc], rows * 8);
                        __syncwarp();
                        if (mine) {
                            uint8_t* dst = dyn + S::kOffScale + sc * 2 * kTile * 4 + lane * box_rows * 4;
                            const int64_t vec = static_cast<int64_t>(outer) << cache.page_shift;
                            bulk_g2s(dst, cache.k_scale + vec, box_rows * 4, &sh.sc_full[sc]);
                            bulk_g2s(dst + kTile * 4, cache.v_scale + vec, box_rows * 4, &sh.sc_full[sc]);
                        }
                        if (++sc == S::kScaleBufs) sc = 0, sc_phase ^= 1;
                    }
                    for (int kv = 0; kv < 2; ++kv) {
                        if (!(ok = warp_wait(&sh.abort, &empty[buf], phase ^ 1, a.err))) break;
                        if (lane == 0) mbar_arrive_expect_tx(&full[buf], rows * DIM * (INT8 ? 1 : 2));
                        __syncwarp();
                        if (mine) {
                            const CUtensorMap* map = kv ? &cp.v_map : &cp.k_map;
                            if constexpr (INT8) {
                                tma_load_3d(dyn + S::kOffRaw + buf * S::kRawBytes + lane * box_rows * DIM, map, 0, 0,
                                            outer, &full[buf]);
                            } else {
#pragma unroll
                                for (int half = 0; half < S::kHalves; ++half)
                                    tma_load_3d(dyn + S::kOffBufs + buf * S::kTileBytes + half * S::kHalfBytes +
                                                    lane * box_rows * 128,
                                                map, 64 * half, 0, outer, &full[buf]);
                            }
                        }
                        if (++buf == kRing) buf = 0, phase ^= 1;
                    }
                }
            }
            if (!ok) {
                // given up: leave only when the copies in flight have landed
                for (int b = 0; b < kRing; ++b) mbar_wait_bounded(&full[b], b < buf ? phase : phase ^ 1);
                if constexpr (INT8)
                    for (int b = 0; b < S::kScaleBufs; ++b)
                        mbar_wait_bounded(&sh.sc_full[b], b < sc ? sc_phase : sc_phase ^ 1);
            }
        } else if (warp == 9) {
            // ---------------------------------------------------- MMA
            constexpr uint32_t kIdescS = idesc_bf16_f32(kQRows, kTile);
            constexpr uint32_t kIdescO = idesc_bf16_f32(kQRows, DIM) | (1u << 16);  // V: rows along the contracted index
            const uint32_t q_addr = smem_u32(dyn), buf_addr = smem_u32(dyn + S::kOffBufs);
            int buf = 0;
            uint32_t phase = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            bool ok = true;
            const auto product_s = [&](int i, int b) {
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < DIM / 16; ++k) {
                        const uint32_t off = (k >> 2) * S::kHalfBytes + (k & 3) * 32;
                        mma_ss(tmem + i * 128, smem_desc_sw128(q_addr + i * S::kQBytes + off),
                               smem_desc_sw128(buf_addr + b * S::kTileBytes + off), kIdescS, k > 0);
                    }
                    mma_commit(&sh.s_full[i]);
                }
                __syncwarp();
            };
            const auto free_buf = [&](int b) {
                if (elect_one()) mma_commit(&sh.empty[b]);
                __syncwarp();
            };
            const auto take = [&](int* b) {  // the next tile of the ring
                ok = warp_wait(&sh.abort, &sh.full[buf], phase, a.err);
                tc_fence_after();
                *b = buf;
                if (++buf == S::kBufs) buf = 0, phase ^= 1;
                return ok;
            };
            while (ok && walk.next(s)) {
                int bk = 0, bv = 0;
                if (!take(&bk)) break;
                for (int i = 0; i < s.q_tiles && ok; ++i) {
                    if (!(ok = warp_wait(&sh.abort, &sh.q_full[i], q_phase[i], a.err))) break;
                    q_phase[i] ^= 1;
                    tc_fence_after();
                    product_s(i, bk);
                }
                if (!ok) break;
                free_buf(bk);
                for (int t = s.t0; t < s.t1 && ok; ++t) {
                    const bool more = t + 1 < s.t1;
                    if (!take(&bv)) break;
                    if constexpr (!INT8) {
                        // what lies past the sequence may be anything, NaN included: zeros
                        // instead, so that probabilities of 0 times it stay 0
                        const int valid = s.sq.len - t * kTile;
                        if (valid < kTile) {
                            uint8_t* vt = dyn + S::kOffBufs + bv * S::kTileBytes;
                            for (int x = (valid > 0 ? valid : 0) * 8 + lane; x < kTile * 8; x += 32)
#pragma unroll
                                for (int half = 0; half < S::kHalves; ++half)
                                    *reinterpret_cast<uint4*>(vt + half * S::kHalfBytes + x * 16) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    if (more && !take(&bk)) break;
                    for (int i = 0; i < s.q_tiles; ++i) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (!(ok = ok && warp_wait(&sh.abort, &sh.p_full[i][half], p_phase[i], a.err))) continue;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int k = 4 * half; k < 4 * half + 4; ++k)
                                    mma_ts(tmem + kTmemO + i * DIM, tmem + i * 128 + 8 * k,
                                           smem_desc_mn_sw128(buf_addr + bv * S::kTileBytes + k * 2048, S::kHalfBytes),
                                           kIdescO, t > s.t0 || k > 0);
                                if (half == 1 && !more) mma_commit(&sh.o_full[i]);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                        p_phase[i] ^= 1;
                        if (more) product_s(i, bk);
                    }
                    if (!ok) break;
                    free_buf(bv);
                    if (more) free_buf(bk);
                }
            }
            // nothing of this block's products is in flight when its tensor memory is given back
            if (elect_one()) mma_commit(&sh.done);
            __syncwarp();
            mbar_wait_bounded(&sh.done, 0);
        }
    } else {
        reg_dec<S::kOtherRegs>();
        if constexpr (INT8) {
            // -------------------------------------------------------- codes to bf16 tiles
            int raw = 0, buf = 0;
            uint32_t raw_phase = 0, phase = 0;
            bool ok = true;
            const int tid = threadIdx.x & 127;
            constexpr int kChunks = DIM / 16;  // 16-byte chunks of codes of a key
            while (ok && walk.next(s)) {
                for (int n = 2 * (s.t1 - s.t0); n > 0; --n) {
                    if (!(ok = warp_wait(&sh.abort, &sh.raw_full[raw], raw_phase, a.err))) break;
                    if (!(ok = warp_wait(&sh.abort, &sh.empty[buf], phase ^ 1, a.err))) break;
                    const uint8_t* src = dyn + S::kOffRaw + raw * S::kRawBytes;
                    uint8_t* dst = dyn + S::kOffBufs + buf * S::kTileBytes;
#pragma unroll 4
                    for (int x = tid; x < kTile * kChunks; x += 128) {
                        const int key = x / kChunks, ch = x % kChunks;
                        const uint4 w = *reinterpret_cast<const uint4*>(src + x * 16);
                        const uint4 lo = make_uint4(codes_bf16x2(w.x, 0x4140), codes_bf16x2(w.x, 0x4342),
                                                    codes_bf16x2(w.y, 0x4140), codes_bf16x2(w.y, 0x4342));
                        const uint4 hi = make_uint4(codes_bf16x2(w.z, 0x4140), codes_bf16x2(w.z, 0x4342),
                                                    codes_bf16x2(w.w, 0x4140), codes_bf16x2(w.w, 0x4342));
                        uint8_t* half = dst + (ch >> 2) * S::kHalfBytes + key * 128;
                        const int e = ((2 * (ch & 3)) ^ (key & 7)) << 4, o = ((2 * (ch & 3) + 1) ^ (key & 7)) << 4;
                        // lanes of the upper half store their odd chunk first: no two of eight
                        // neighbouring lanes meet in a bank
                        const bool odd_first = ch >= 4;
                        *reinterpret_cast<uint4*>(half + (odd_first ? o : e)) = odd_first ? hi : lo;
                        *reinterpret_cast<uint4*>(half + (odd_first ? e : o)) = odd_first ? lo : hi;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.full[buf]);
                        mbar_arrive(&sh.raw_empty[raw]);
                    }
                    if (++raw == S::kRaw) raw = 0, raw_phase ^= 1;
                    if (++buf == S::kBufs) buf = 0, phase ^= 1;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, kTmemCols);
}

template <int DIM, bool INT8>
cudaError_t launch_chunk_shape(const AttnParams& p, cudaStream_t stream)
{
    using S = ChunkShape<DIM, INT8>;
    static std::atomic<size_t> smem_set[kHostMaxDevices];
    const KvPages& kv = p.a.cache;
    ChunkParams cp{};
    cp.p = p;
    const uint64_t outer = static_cast<uint64_t>(kv.n_pages) * kv.n_kv;
    for (int i = 0; i < 2; ++i)
        if (!encode_tma_3d(i ? &cp.v_map : &cp.k_map,
                           INT8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, INT8 ? 1 : 2,
                           i ? kv.v : kv.k, DIM, kv.page, outer, INT8 ? DIM : 64, kv.page,
                           INT8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    const size_t smem = S::kBytes + 1024;
    const void* kernel = reinterpret_cast<const void*>(attn_chunk_kernel<DIM, INT8>);
    cudaError_t err = ensure_dynamic_smem(kernel, smem, smem_set);
    if (err != cudaSuccess) return err;
    // the warpgroups' register split draws on what the block was launched
    // with; a build whose kernel has fewer registers would wait for them
    static std::atomic<int> regs{0};
    int n = regs.load(std::memory_order_acquire);
    if (n == 0) {
        cudaFuncAttributes attr{};
        if ((err = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return err;
        n = attr.numRegs;
        regs.store(n, std::memory_order_release);
    }
    if (n * (S::kThreads / 128) < 2 * S::kSoftRegs + (S::kThreads / 128 - 2) * S::kOtherRegs)
        return cudaErrorInvalidConfiguration;
    launch_dep(err, attn_chunk_kernel<DIM, INT8>, dim3(p.blocks), dim3(S::kThreads), smem, stream, cp);
    return err;
}

}  // namespace

BD_BOUNDS_TAKE(bounds_take_attention_chunk)

cudaError_t launch_attention_chunk(const AttnParams& p, cudaStream_t stream)
{
    if (p.a.cache.dim == 128)
        return p.a.cache.int8 ? launch_chunk_shape<128, true>(p, stream) : launch_chunk_shape<128, false>(p, stream);
    return p.a.cache.int8 ? launch_chunk_shape<64, true>(p, stream) : launch_chunk_shape<64, false>(p, stream);
}

}  // namespace bd
