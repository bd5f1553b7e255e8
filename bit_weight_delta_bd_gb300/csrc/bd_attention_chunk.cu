// Attention over the paged KV cache for chunks of new tokens, on the tcgen05
// tensor cores (the formulas and the dealing of the work: bd_attention.cuh).
//
// An item is 256 query rows of one kv head for each CTA (two query tiles of
// 128); its keys are read in tiles of 128 by TMA and multiplied in steps of 64.
// Per step and query tile
//   S = Q K^T       128 x 64, operands in shared memory, fp32 in tensor memory
//   P = exp2(c S - m)   one thread per row: maximum, probabilities, denominator
//   O += P V        P as bf16 in tensor memory (over S), V in shared memory
// S has two places, so that S of step j + 1 is there before P of step j is
// done and neither the tensor cores nor the exponentials wait for the other:
// with one place of 128 keys a query tile's products and exponentials took
// turns, 3350 cycles for 128 keys and 256 rows of which the tensor cores
// worked 2300.
//
// Pairs.  With head_dim 128 and sequences of more than 256 rows two CTAs work
// on an item of 512: the even one's products cover both (M = 256), and each
// holds half of the operand that they share, 32 keys of each step of K and 64
// dims of V.  What bounds a single CTA is its shared memory (a step of 64 reads
// Q twice as often as one of 128 would, and the 64-key product then runs at 3/4
// of its rate); a pair reads 3/4 of that, and int8 tiles are converted once for
// 512 rows.  A chunk of 4096 tokens over 8192 keys, 64/8 heads: bf16 885 us by
// single CTAs and 812 by pairs, int8 1245 and 1110.  (O written by whole
// sectors, a row per thread, takes 5 us less of any call: 765 .. 820 us for the
// bf16 chunk as the clocks allow, 1670 to 1800 TFLOP/s.)
// Sequences of up to 256 rows would fill a pair's first query tile at most,
// which takes as long as both: 8 sequences of 4 tokens over 4000 int8 keys take
// 45 us by single CTAs and 68 by pairs.  With head_dim 64 half of V's dims
// would leave 64-byte rows: single CTAs, 717 us for bf16 and 1122 for int8,
// which by their number should be the exponentials' time (as many as with
// head_dim 128, for half the products; no measurement sets them apart).
//
// The running maximum that P is formed with lags behind the true one by at
// most 2^8 (a row's sums are rescaled in tensor memory only when its maximum
// grew by more than 8 in units of log2; the fp32 sums have room for that
// factor), so that rescaling is rare after a row's first steps.
// A warp for each query tile issues its products, P V of step j and then S of
// step j + 2.
//
// Int8 keys and values: TMA brings the codes, a fourth warpgroup turns them
// into tiles of numbers (exactly: K to fp16 and V to bf16), once for all
// query tiles; the scales multiply S and P in the softmax's registers.  Q
// enters that product in fp16, scaled by a power of two per row, as in the
// decode kernel; P stays bf16, whose range the sums of a row's smallest
// probabilities need.  Within each group of four dims the tiles hold them in
// the order 0, 2, 1, 3, in which the codes come out of a register.  The
// softmax bounds this kernel: without its reads of the scales (32 of 16 bytes
// per step and warp, in the way of the products' operands) and the conversion
// it would take 934 us, and without the softmax 757.  (Four lanes to a row, a
// quarter of the scales each, shuffles for the maximum: 1260 us; two warpgroups
// to a row: slower as well.)
//
// Warps: 0..3 and 4..7 softmax of query tiles 0 and 1 (and loading Q, and
// writing O); 8 TMA; 9 and 10 MMA of query tiles 0 and 1 (of a pair: the even
// CTA's); 11 passes on that a pair's tiles are there (bf16: landed, int8: the
// odd CTA's converted); 12..15 conversion (int8).
#include <cuda_fp16.h>

#include <type_traits>

#include "bd_attention.cuh"
#include "bd_tcgen05.cuh"
#include "bd_tma.h"

namespace bd {
namespace {

constexpr int kTile = 128;       // keys of a tile
constexpr int kQRows = 128;      // rows of a query tile
constexpr int kStep = 64;        // keys of a step
constexpr float kLag = 8.0f;     // how far (log2) a row's maximum may run ahead of the one in use

struct ChunkParams {
    // [n_pages * n_kv][page][dim]; boxes of 128 bytes (int8 V of a pair, and head_dim 64: 64) x page rows, K of a
    // pair up to 32
    CUtensorMap k_map, v_map;
    AttnParams p;
};

template <int DIM, bool INT8, bool PAIR>
struct ChunkShape {
    static constexpr bool kPair = PAIR;
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kThreads = INT8 ? 512 : 384;
    static constexpr bool kSmall = PAIR || DIM == 64;  // tiles of 16 KB
    static constexpr int kBufs = INT8 ? (kSmall ? 6 : 3) : kSmall ? 8 : 5;  // bf16 tiles in shared memory
    static constexpr int kRaw = INT8 ? (kSmall ? 6 : 3) : 0;                // tiles of codes
    static constexpr int kScaleBufs = INT8 ? (kSmall ? 4 : 3) : 0;          // scales of a key tile, K and V
    // a CTA's part of a tile: in a pair half the keys of each step of K, half the dims of V
    static constexpr int kKeysK = kTile / kCtas, kDimsV = DIM / kCtas;
    static constexpr int kTileBytes = kTile * DIM * 2 / kCtas;
    static constexpr int kRawBytes = kTile * DIM / kCtas;
    static constexpr int kQBytes = kQRows * DIM * 2;
    static constexpr int kOffBufs = 2 * kQBytes;
    static constexpr int kOffRaw = kOffBufs + kBufs * kTileBytes;
    static constexpr int kOffScale = kOffRaw + kRaw * kRawBytes;
    static constexpr int kBytes = kOffScale + kScaleBufs * 2 * kTile * 4;
    // registers of a softmax thread, and of the others: the sum over the
    // warpgroups is what the block was launched with
    static constexpr int kSoftRegs = INT8 ? 168 : 208;
    static constexpr int kOtherRegs = 88;
    static_assert(2 * kSoftRegs + (INT8 ? 2 : 1) * kOtherRegs <= (INT8 ? 4 * 128 : 3 * 168), "register split");
};

constexpr int kMaxBufs = 8, kMaxRaw = 6, kMaxScales = 4;

struct ChunkShared {
    uint64_t full[kMaxBufs], empty[kMaxBufs];    // bf16 tiles (full: of both CTAs, in the even one)
    uint64_t landed[kMaxBufs];                   // this CTA's part of them (pairs; int8: the odd one's)
    uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];     // tiles of codes
    uint64_t sc_full[kMaxScales], sc_empty[kMaxScales];  // scales
    uint64_t q_full[2], o_full[2];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2];  // by query tile (and place)
    uint64_t done;
    uint32_t tmem;
    volatile int abort;
};

// all of it dynamic: the tiles start on a 1024-byte boundary without padding
template <typename Shape>
constexpr size_t chunk_smem()
{
    static_assert(Shape::kBytes + sizeof(ChunkShared) <= 227 * 1024, "shared memory");
    return Shape::kBytes + sizeof(ChunkShared);
}

constexpr int kSoftWarps = 8, kTmaWarp = 8, kMmaWarp = 9, kPassWarp = 11, kConvertWarp = 12;

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;  // S at 128 i + 64 b (query tile i, place b), O tiles from 256 on

// A wait of a whole warp; false (for all lanes) once the block has given up,
// which the end of the kernel reports.
__device__ __forceinline__ bool warp_wait(volatile int* abort_flag, uint64_t* bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (*abort_flag) return false;
    if (__all_sync(0xffffffffu, mbar_wait_sleeping(bar, parity))) return true;
    *abort_flag = 1;
    return false;
}

// Barriers of a pair: an arrival at the even CTA's (for tensor memory, and for
// tiles that TMA has brought), a wait for arrivals of both, and the tensor
// cores' arrival at both.
template <bool PAIR>
__device__ __forceinline__ void arrive_even(uint64_t* bar)
{
    if constexpr (PAIR) mbar_arrive_remote(bar, 0);
    else mbar_arrive(bar);
}
// The same for what this CTA's threads have written to its shared memory, which
// the even CTA's products are to read: released at cluster scope by the odd
// CTA, since an arrival of CTA scope orders none of it there.
template <bool PAIR>
__device__ __forceinline__ void arrive_even_written(uint64_t* bar, int rank)
{
    if (PAIR && rank != 0) mbar_arrive_remote_release(bar, 0);
    else mbar_arrive(bar);
}
template <bool PAIR>
__device__ __forceinline__ void wait_both(volatile int* abort_flag, uint64_t* bar, uint32_t parity)
{
    if (warp_wait(abort_flag, bar, parity) && PAIR) (void)mbar_try_wait_cluster(bar, parity);  // for its scope
}
template <bool PAIR>
__device__ __forceinline__ void commit_both(uint64_t* bar)
{
    if constexpr (PAIR) mma_commit_pair(bar, 3);
    else mma_commit(bar);
}

template <bool PAIR>
__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR) mma_ts_pair(d, a, b, idesc, accumulate);
    else mma_ts(d, a, b, idesc, accumulate);
}
template <bool PAIR>
__device__ __forceinline__ void mma_from_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR) mma_ss_pair(d, a, b, idesc, accumulate);
    else mma_ss(d, a, b, idesc, accumulate);
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

__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15])::"memory");
}

__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t (&v)[16])
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

// What lies past the sequence in a tile of V may be anything, NaN included:
// zeros from key `valid` on instead, so that probabilities of 0 times it stay
// 0.  DIMS: that the CTA holds.  By a warp.  Returns whether it wrote any.
template <int DIMS>
__device__ __forceinline__ bool zero_past(uint8_t* v, int valid, int lane)
{
    if (valid >= kTile) return false;
#pragma unroll 1
    for (int x = (valid > 0 ? valid : 0) * 8 + lane; x < kTile * 8; x += 32)
#pragma unroll
        for (int d = 0; d < DIMS; d += 64)
            *reinterpret_cast<uint4*>(v + (d / 64) * kTile * 128 + x * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    return true;
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

// Two codes, bytes 0 and 2 of r, as a pair of fp16 (see bd_attention.cu).
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t r)
{
    const uint32_t x = (r & 0x00FF00FFu) ^ 0x64806480u, offset = 0xE480E480u;  // 1152 + code, -1152
    const __half2 d = __hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&offset));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// Two codes, bytes 0 and 2 of r, as a pair of bf16: with c the byte, 0x4300 |
// (c & 0x7f) is 128 + (c & 0x7f), 0x4300 | (c & 0x80) is 128 or 256, and the
// difference is the code.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t r)
{
    const uint32_t hi = (r & 0x007F007Fu) | 0x43004300u, lo = (r & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&hi), *reinterpret_cast<const __nv_bfloat162*>(&lo));
    return *reinterpret_cast<const uint32_t*>(&d);
}

template <bool HALF>
__device__ __forceinline__ uint2 codes4(uint32_t r)  // in the order 0, 2, 1, 3
{
    if constexpr (HALF) return make_uint2(codes_f16x2(r), codes_f16x2(r >> 8));
    return make_uint2(codes_bf16x2(r), codes_bf16x2(r >> 8));
}

// A tile of codes as a tile of numbers, 16-byte chunks of 16 codes, by the 128
// threads of a warpgroup.  Eight neighbouring lanes take four chunks of two
// keys whose numbers differ in the bits (5: the lowest and the third; 64-byte
// rows: the lowest) that put both their reads from TMA's swizzled tile of
// codes and their writes to the swizzled tile of numbers into different banks.
// Later chunks of a thread lie 16 (32) keys on, at the same place of the swizzle.
// DIM: codes of a row; KEYS: rows of the tile.
template <int DIM, int KEYS, bool HALF>
__device__ __forceinline__ void convert_tile(const uint8_t* src, uint8_t* dst, int tid)
{
    constexpr int kKeys = 128 * 16 / DIM;  // keys of one round
    constexpr int kRounds = KEYS / kKeys;
    const int warp = tid >> 5, c = tid & 3, odd = (tid >> 2) & 1, rest = (tid >> 3) & 3;
    int key, ch;
    if constexpr (DIM == 128) {
        // the warp's 4 keys of 16: {b, b ^ 5}, b = 2 (warp & 1) + {0, 1}, in the 8 keys of warp >> 1
        ch = c + 4 * (rest & 1);
        key = 8 * (warp >> 1) + ((2 * (warp & 1) + (rest >> 1)) ^ (odd ? 5 : 0));
    } else {
        ch = c;
        key = 8 * warp + 2 * rest + odd;
    }
    const uint8_t* from = src + key * DIM + ((DIM == 128 ? ch ^ (key & 7) : ch ^ ((key >> 1) & 3)) << 4);
    uint8_t* row = dst + (ch >> 2) * (KEYS * 128) + key * 128;
    uint8_t* to_lo = row + (((2 * (ch & 3)) ^ (key & 7)) << 4);
    uint8_t* to_hi = row + (((2 * (ch & 3) + 1) ^ (key & 7)) << 4);
    uint4 w = *reinterpret_cast<const uint4*>(from);
#pragma unroll 2
    for (int i = 0; i < kRounds; ++i) {
        uint4 next = w;
        if (i + 1 < kRounds) next = *reinterpret_cast<const uint4*>(from + (i + 1) * kKeys * DIM);
        const uint2 a = codes4<HALF>(w.x), b = codes4<HALF>(w.y), d = codes4<HALF>(w.z), e = codes4<HALF>(w.w);
        *reinterpret_cast<uint4*>(to_lo + i * kKeys * 128) = make_uint4(a.x, a.y, b.x, b.y);
        *reinterpret_cast<uint4*>(to_hi + i * kKeys * 128) = make_uint4(d.x, d.y, e.x, e.y);
        w = next;
    }
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
        s.sq = attn_seq(p, s.it.seq, false);
        s.rows = s.sq.n_new * p.G - s.it.row0;
        u += s.t1 - s.t0;
        if (s.t1 == s.it.tiles && s.h == n_kv - 1) ++item;
        // known for uniform
        s.t0 = __shfl_sync(0xffffffffu, s.t0, 0);
        s.t1 = __shfl_sync(0xffffffffu, s.t1, 0);
        s.rows = __shfl_sync(0xffffffffu, s.rows, 0);
        s.sq.len = __shfl_sync(0xffffffffu, s.sq.len, 0);
        s.q_tiles = s.rows > p.mb / 2 ? 2 : 1;
        return true;
    }
};

// Row `row` (of the item) of a segment's Q; null past the item's rows.
template <int DIM>
__device__ __forceinline__ const uint4* q_row(const AttnParams& p, const Segment& s, int row)
{
    const AttentionArgs& a = p.a;
    if (row >= s.rows || row >= p.mb) return nullptr;
    const int abs_row = s.it.row0 + row, tok = abs_row / p.G;
    return reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(s.sq.q0) + tok) * a.q_stride +
                                          static_cast<int64_t>(s.h * p.G + (abs_row - tok * p.G)) * DIM);
}

__device__ __forceinline__ void prefetch_l2(const void* p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ float abs_max8(float big, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        big = max3(big, fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u)));
    return big;
}

// The power of two at or below |x|, kept within 2^-100 .. 2^100.
__device__ __forceinline__ float unit_of(float x)
{
    return __uint_as_float(__float_as_uint(fminf(fmaxf(x, 7.9e-31f), 1.2e30f)) & 0x7F800000u);
}

// A warp's 32 rows, from row r0 on, of the query tile that starts at the
// item's row tile_row, into shared memory (K-major, 128-byte swizzle, halves
// of 64 dims); rows past the item are zeros.  Neighbouring lanes take neighbouring 16 bytes, eight loads in
// flight (a row per lane, two in flight, cost 6 us per item, and twice that
// where int8 looked for the maximum first).  A negative scale is taken into
// Q's sign; int8: fp16, over the row's power of two, dims in the codes' order.
// Returns what the products of row r0 + lane are to be multiplied by.
template <int DIM, bool INT8>
__device__ __forceinline__ float load_q(const AttnParams& p, const Segment& s, int tile_row, int r0, int lane, uint8_t* dst)
{
    constexpr int kLanes = DIM / 8, kRowsAtOnce = 32 / kLanes, kBatch = 8;
    const uint64_t own = reinterpret_cast<uint64_t>(q_row<DIM>(p, s, tile_row + r0 + lane));
    const uint32_t flip = p.a.scale < 0.0f ? 0x80008000u : 0u;
    const int c = lane & (kLanes - 1), sub = lane / kLanes;
    float back = 1.0f;
#pragma unroll 1
    for (int g = 0; g < 32; g += kBatch * kRowsAtOnce) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint64_t at = __shfl_sync(0xffffffffu, own, g + k * kRowsAtOnce + sub);
            v[k] = make_uint4(0, 0, 0, 0);
            if (at) v[k] = __ldg(reinterpret_cast<const uint4*>(at) + c);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = r0 + g + k * kRowsAtOnce + sub;
            uint4 x = v[k];
            x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
            if constexpr (INT8) {
                float big = abs_max8(0.0f, x);
#pragma unroll
                for (int o = 1; o < kLanes; o *= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                const float unit = unit_of(big), f = 16384.0f / unit;
#pragma unroll
                for (int e = 0; e < kRowsAtOnce; ++e) {
                    const float of = __shfl_sync(0xffffffffu, unit, e * kLanes);
                    if (lane == g + k * kRowsAtOnce + e) back = of / 16384.0f;
                }
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float x0 = __uint_as_float(w[e] << 16) * f, x1 = __uint_as_float(w[e] & 0xFFFF0000u) * f;
                    const float x2 = __uint_as_float(w[e + 1] << 16) * f;
                    const float x3 = __uint_as_float(w[e + 1] & 0xFFFF0000u) * f;
                    const __half2 even = __floats2half2_rn(x0, x2), odd = __floats2half2_rn(x1, x3);
                    o[e] = *reinterpret_cast<const uint32_t*>(&even);
                    o[e + 1] = *reinterpret_cast<const uint32_t*>(&odd);
                }
                x = make_uint4(o[0], o[1], o[2], o[3]);
            }
            *reinterpret_cast<uint4*>(dst + (c >> 3) * (kQRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
        }
    }
    return back;
}

template <int DIM, bool INT8, bool PAIR>
__global__ void __launch_bounds__(ChunkShape<DIM, INT8, PAIR>::kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ ChunkParams cp)
{
    using S = ChunkShape<DIM, INT8, PAIR>;
    constexpr bool kPair = PAIR;
    extern __shared__ __align__(1024) uint8_t dyn[];
    ChunkShared& sh = *reinterpret_cast<ChunkShared*>(dyn + S::kBytes);
    const AttnParams& p = cp.p;
    const AttentionArgs& a = p.a;
    const KvPages& cache = a.cache;
    // (taken from lane 0, so that the compiler knows it for uniform: the
    // branches below, and the descriptors that the MMA warp forms in them)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kBufs; ++i) {
            // (int8: four warps of the even CTA, and what the odd one passes on)
            mbar_init(&sh.full[i], INT8 ? 3 + S::kCtas : S::kCtas);
            mbar_init(&sh.empty[i], 2);
            mbar_init(&sh.landed[i], INT8 ? 4 : 1);
        }
        for (int i = 0; i < S::kRaw; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
        }
        for (int i = 0; i < S::kScaleBufs; ++i) {
            mbar_init(&sh.sc_full[i], 1);
            mbar_init(&sh.sc_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 4 * S::kCtas);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sh.s_full[i][b], 1);
                mbar_init(&sh.p_full[i][b], 4 * S::kCtas);
            }
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.done, 2);
        sh.abort = 0;
        fence_mbarrier_init();
    }
    if (warp == kMmaWarp) {
        if constexpr (kPair) tmem_alloc_pair(&sh.tmem, kTmemCols);
        else tmem_alloc(&sh.tmem, kTmemCols);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync_all();  // the other's barriers are there before anything arrives at them
    tc_fence_after();
    grid_dependency_wait();

    const uint32_t tmem = sh.tmem;
    const AttnHeader head = *p.head;
    const int n_kv = cache.n_kv;
    const int64_t units = static_cast<int64_t>(head.tiles) * n_kv;
    const int active = attn_active(units, p.blocks);
    const int rank = kPair ? __shfl_sync(0xffffffffu, static_cast<int>(cluster_ctarank()), 0) : 0;
    const int c = blockIdx.x / S::kCtas;
    Walk walk{p, 0, 0, 0};
    if (c < active) {
        walk.u = attn_first(units, active, c);
        walk.end = attn_first(units, active, c + 1);
        walk.item = attn_find_item(p.items, head.n_items, n_kv, walk.u);
    }
    if (threadIdx.x == 0 && rank == 0) {
        AttnJoin j{};
        if (c < active) {
            const AttnItem it = p.items[walk.item];
            const int64_t first = static_cast<int64_t>(it.before) * n_kv;
            const int h = attn_div(walk.u - first, it.tiles);
            j = attn_join_of(units, active, c, walk.u, first + static_cast<int64_t>(h) * it.tiles, it.tiles,
                             attn_seq(p, it.seq, false), p.G, it.row0, h);
        }
        p.joins[c] = j;
    }
    __syncwarp();
    Segment s;

    if (warp < kSoftWarps) {
        // -------------------------------------------------------- softmax of query tile i
        reg_inc<S::kSoftRegs>();
        const int i = warp >> 2;
        const int r = 32 * (warp & 3) + lane;  // this thread's row of the tile
        const int tile_row = (i * S::kCtas + rank) * kQRows;  // the tile's first row of the item
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + i * 128, to = tmem + lanes + kTmemO + i * DIM;
        uint8_t* q_smem = dyn + i * S::kQBytes;
        float unit = 1.0f;  // of this thread's row of the Q in shared memory
        const bool out_sectors = on_sector(a.out);
        uint32_t s_phase = 0, o_phase = 0, pv_phase = 0, sc_phase = 0;
        int sc = 0;
        // After a timeout (reported) the waits return at once and the loops run out on what is there.
        // (Each part of the loop stands once, and its rare parts are rolled: the code that runs has to
        // fit the instruction cache, or the warps wait for their instructions.)
        bool ran = false, whole = false, live = false;  // of the segment whose sums are still to be written
        int64_t at = 0;
        float m = -INFINITY, l = 0.0f, m2 = 0.0f;
        for (;;) {
            // the products with the last Q are done (S of its last tile stood behind them): the next
            // one may come in while the last P V runs
            const bool have = walk.next(s);
            const bool runs = have && i < s.q_tiles;
            if (runs) {
                unit = load_q<DIM, INT8>(p, s, tile_row, r - lane, lane, q_smem);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_even_written<kPair>(&sh.q_full[i], rank);
            }
            if (ran) {
                warp_wait(&sh.abort, &sh.o_full[i], o_phase);
                o_phase ^= 1;
                tc_fence_after();
                live = live && bd_in(kBkAttn, at, whole ? a.T * a.n_q : 2ll * p.blocks * p.mb);
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
                for (int j = 0; j < DIM; j += 16) {
                    uint32_t o[16];
                    __syncwarp();
                    tmem_ld16_wait(to + j, o);
                    if constexpr (INT8) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {  // back from the order 0, 2, 1, 3
                            const uint32_t x = o[e + 1];
                            o[e + 1] = o[e + 2];
                            o[e + 2] = x;
                        }
                    }
                    if (live && whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            w[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
                            if (l == 0.0f) w[k] = 0u;
                        }
                        uint16_t* dst = a.out + at * DIM + j;
                        if (out_sectors) {
                            store_32(dst, w);
                        } else {
                            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            const uint32_t w[8] = {o[e],     o[e + 1], o[e + 2], o[e + 3],
                                                   o[e + 4], o[e + 5], o[e + 6], o[e + 7]};
                            store_32(p.part_o + at * DIM + j + e, w);
                        }
                    }
                }
                if (live) {
                    if (!whole)
                        p.part_ml[at] = make_float2(m2, l);
                    else if (a.lse)
                        a.lse[at] = attn_lse(m2, l);
                }
                __syncwarp();
                tc_fence_before();
            }
            if (!have) break;
            ran = runs;
            if (!runs) {
                // no rows here: only the scales' slots have to be handed on
                if constexpr (INT8) {
                    for (int t = s.t0; t < s.t1; ++t) {
                        if (!warp_wait(&sh.abort, &sh.sc_full[sc], sc_phase)) break;
                        if (lane == 0) mbar_arrive(&sh.sc_empty[sc]);
                        if (++sc == S::kScaleBufs) sc = 0, sc_phase ^= 1;
                    }
                }
                continue;
            }
            const int row = tile_row + r;
            live = row < s.rows && row < p.mb;
            int seen = 0;
            {
                const int abs_row = s.it.row0 + row, tok = live ? abs_row / p.G : 0;
                if (live) seen = attn_seen(s.sq, tok, a.causal);
                whole = s.t0 == 0 && s.t1 == s.it.tiles;
                at = whole ? (static_cast<int64_t>(s.sq.q0) + tok) * a.n_q + s.h * p.G + (abs_row - tok * p.G)
                           : static_cast<int64_t>(attn_slot(c, s.t0 == 0)) * p.mb + row;
            }
            // what the tile's first row sees (the others see at least as much): below it no mask
            const int all_seen = attn_seen(s.sq, (s.it.row0 + tile_row) / p.G, a.causal);
            // (a scale of 0 would make NaN of a masked score)
            const float c2 = fmaxf(fabsf(a.scale) * kLog2e * unit, 1e-30f);
            m = -INFINITY;
            l = 0.0f;
#pragma unroll 1
            for (int j = 2 * s.t0; j < 2 * s.t1; ++j) {
                const int b = j & 1;
                warp_wait(&sh.abort, &sh.s_full[i][b], s_phase);
                tc_fence_after();
                uint32_t v[64];
                tmem_ld32_start(ts + 64 * b, v);
                tmem_ld32_start(ts + 64 * b + 32, v + 32);
                const float *ks = nullptr, *vs = nullptr;
                if constexpr (INT8) {
                    if (b == 0) warp_wait(&sh.abort, &sh.sc_full[sc], sc_phase);
                    ks = reinterpret_cast<const float*>(dyn + S::kOffScale) + sc * 2 * kTile + kStep * b;
                    vs = ks + kTile;
                }
                tmem_ld_wait(v);
                tmem_ld_wait(v + 32);
                if constexpr (INT8) {
#pragma unroll
                    for (int e = 0; e < 64; e += 4) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(ks + e);
                        const float2 x = unpack2(mul2(f32x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), f.x));
                        const float2 y =
                            unpack2(mul2(f32x2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), f.y));
                        v[e] = __float_as_uint(x.x), v[e + 1] = __float_as_uint(x.y);
                        v[e + 2] = __float_as_uint(y.x), v[e + 3] = __float_as_uint(y.y);
                    }
                }
                if ((j + 1) * kStep > all_seen) {
                    const int left = seen - j * kStep;  // keys of the step that the row sees
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (e >= left) v[e] = 0xFF800000u;  // -infinity
                    if constexpr (INT8) {
                        // scales past the sequence may be anything, NaN included: zeros instead (every
                        // warp writes them, each before it reads)
                        const int valid = s.sq.len - j * kStep;
                        float* z = const_cast<float*>(vs);
                        if (lane >= valid) z[lane] = 0.0f;
                        if (lane + 32 >= valid) z[lane + 32] = 0.0f;
                        fence_proxy_async_smem();  // before TMA's next scales in this place
                    }
                    __syncwarp();
                }
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
#pragma unroll
                for (int e = 8; e < 64; e += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = max3(mx[k], __uint_as_float(v[e + 2 * k]), __uint_as_float(v[e + 2 * k + 1]));
                const float mt = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                // the first step sets the maximum; later it moves when it has grown by kLag
                const bool grow = mt > m && (mt - m) * c2 > kLag;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = !grow ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - mt) * c2);
                    if (grow) m = mt;
                    l *= f;
                    if (j > 2 * s.t0) {
                        // P V of the step before has to be done (S of this step says it of the one before that)
                        warp_wait(&sh.abort, &sh.pv_done[i], pv_phase ^ 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < DIM; d += 16) {
                            uint32_t o[16];
                            tmem_ld16_wait(to + d, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16_start(to + d, o);
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.0f : fmaf(-m, c2, attn_bias<INT8>());
                uint64_t sum[2] = {0, 0};  // pairs of zeros
                const uint64_t c22 = f32x2(c2, c2), nm2 = f32x2(nm, nm);
#pragma unroll
                for (int e0 = 0; e0 < 64; e0 += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        [[maybe_unused]] ulonglong2 f{};
                        if constexpr (INT8) f = *reinterpret_cast<const ulonglong2*>(vs + e0 + e);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int x = e0 + e + 2 * k;
                            float2 pr =
                                unpack2(fma2(f32x2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), c22, nm2));
                            pr.x = ex2(pr.x);
                            pr.y = ex2(pr.y);
                            const uint64_t pp = f32x2(pr.x, pr.y);
                            sum[k] = add2(sum[k], pp);
                            if constexpr (INT8) pr = unpack2(mul2(pp, k ? f.y : f.x));
                            pk[e / 2 + k] = pack_bf16x2(pr.x, pr.y);
                        }
                    }
                    tmem_st16_start(ts + 64 * b + e0 / 2, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive_even<kPair>(&sh.p_full[i][b]);
                    if constexpr (INT8)
                        if (b) mbar_arrive(&sh.sc_empty[sc]);
                }
                if (b) s_phase ^= 1;
                pv_phase ^= 1;
                if constexpr (INT8)
                    if (b && ++sc == S::kScaleBufs) sc = 0, sc_phase ^= 1;
                const float2 s2 = unpack2(add2(sum[0], sum[1]));
                l += s2.x + s2.y;
            }
            m2 = m == -INFINITY ? -INFINITY : fmaf(m, c2, -attn_bias<INT8>());
        }
    } else if (warp < kConvertWarp) {
        reg_dec<S::kOtherRegs>();
        if (warp == kTmaWarp) {
            // ---------------------------------------------------- TMA
            constexpr int kRing = INT8 ? S::kRaw : S::kBufs;
            uint64_t* full = INT8 ? sh.raw_full : kPair ? sh.landed : sh.full;
            uint64_t* empty = INT8 ? sh.raw_empty : sh.empty;
            const int pages_per_tile = kTile / cache.page;  // (at most 128 keys a page)
            // K of a pair: boxes of up to 32 keys, the CTA's half of each step of 64
            const int box_k = kPair && cache.page > 32 ? 32 : cache.page;
            const int boxes_k = S::kKeysK / box_k, boxes_step = kPair ? 32 / box_k : 0;
            int buf = 0, sc = 0;
            uint32_t phase = 0, sc_phase = 0;
            bool ok = true;
            while (ok && walk.next(s)) {
                // the segment's Q on its way to the L2 cache while the tiles before it are worked on
#pragma unroll 1
                for (int r = lane; r < 2 * kQRows; r += 32)
                    if (const uint4* q = q_row<DIM>(p, s, ((r >> 7) * S::kCtas + rank) * kQRows + (r & 127))) {
                        prefetch_l2(q);
                        if constexpr (DIM == 128) prefetch_l2(q + 8);
                    }
                __syncwarp();
                const int32_t* table = a.table + static_cast<int64_t>(s.it.seq) * a.max_pages;
                const int pages = (s.sq.len + cache.page - 1) >> cache.page_shift;
                for (int t = s.t0; t < s.t1 && ok; ++t) {
                    // lane j looks after the j-th page of the tile, and the j-th box of K
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
                    const uint32_t rows =
                        static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, mine)) * cache.page);
                    int key_k = lane * cache.page;  // of the tile
                    if constexpr (kPair) {
                        const int step = lane / boxes_step;
                        key_k = (step & 1) * kStep + 32 * rank + (lane - step * boxes_step) * box_k;
                    }
                    const int of = key_k >> cache.page_shift;  // the lane with the box's page
                    const int outer_k = __shfl_sync(0xffffffffu, outer, of & 31);
                    const bool mine_k = lane < boxes_k && t * pages_per_tile + of < pages;
                    const uint32_t rows_k =
                        static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, mine_k)) * box_k);
                    if constexpr (INT8) {
                        if (!(ok = warp_wait(&sh.abort, &sh.sc_empty[sc], sc_phase ^ 1))) break;
                        if (lane == 0) mbar_arrive_expect_tx(&sh.sc_full[sc], rows * 8);
                        __syncwarp();
                        if (mine) {
                            uint8_t* dst = dyn + S::kOffScale + sc * 2 * kTile * 4 + lane * cache.page * 4;
                            const int64_t vec = static_cast<int64_t>(outer) << cache.page_shift;
                            bulk_g2s(dst, cache.k_scale + vec, cache.page * 4, &sh.sc_full[sc]);
                            bulk_g2s(dst + kTile * 4, cache.v_scale + vec, cache.page * 4, &sh.sc_full[sc]);
                        }
                        if (++sc == S::kScaleBufs) sc = 0, sc_phase ^= 1;
                    }
                    for (int kv = 0; kv < 2; ++kv) {
                        if (!(ok = warp_wait(&sh.abort, &empty[buf], phase ^ 1))) break;
                        constexpr int kBytes = INT8 ? 1 : 2;
                        if (lane == 0)
                            mbar_arrive_expect_tx(&full[buf], (kv ? rows * S::kDimsV : rows_k * DIM) * kBytes);
                        __syncwarp();
                        uint8_t* dst = dyn + (INT8 ? S::kOffRaw + buf * S::kRawBytes : S::kOffBufs + buf * S::kTileBytes);
                        if (kv == 0 && mine_k) {
                            const int row = key_k & (cache.page - 1), to = lane * box_k;
                            if constexpr (INT8) {
                                tma_load_3d(dst + to * DIM, &cp.k_map, 0, row, outer_k, &full[buf]);
                            } else {
#pragma unroll
                                for (int d = 0; d < DIM; d += 64)
                                    tma_load_3d(dst + (d / 64) * S::kKeysK * 128 + to * 128, &cp.k_map, d, row, outer_k,
                                                &full[buf]);
                            }
                        }
                        if (kv == 1 && mine) {
                            const int to = lane * cache.page;
                            if constexpr (INT8) {
                                tma_load_3d(dst + to * S::kDimsV, &cp.v_map, rank * S::kDimsV, 0, outer, &full[buf]);
                            } else {
#pragma unroll
                                for (int d = 0; d < S::kDimsV; d += 64)
                                    tma_load_3d(dst + (d / 64) * kTile * 128 + to * 128, &cp.v_map,
                                                rank * S::kDimsV + d, 0, outer, &full[buf]);
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
        } else if (warp < kMmaWarp + 2 && rank == 0) {
            // ---------------------------------------------------- MMA of query tile i
            constexpr int kRows = kQRows * S::kCtas;
            constexpr uint32_t kIdescS = INT8 ? idesc_f16_f32(kRows, kStep) : idesc_bf16_f32(kRows, kStep);
            // V: rows along the contracted index
            constexpr uint32_t kIdescO = idesc_bf16_f32(kRows, DIM) | (1u << 16);
            const int i = warp - kMmaWarp;
            const uint32_t q_addr = smem_u32(dyn + i * S::kQBytes), buf_addr = smem_u32(dyn + S::kOffBufs);
            const uint32_t ts = tmem + i * 128, to = tmem + kTmemO + i * DIM;
            int buf = 0;
            uint32_t phase = 0, q_phase = 0, p_phase = 0;
            const auto wait = [&](uint64_t* bar, uint32_t parity) { wait_both<kPair>(&sh.abort, bar, parity); };
            const auto take = [&]() {  // the next tile of the ring
                const int b = buf;
                wait(&sh.full[b], phase);
                if (++buf == S::kBufs) buf = 0, phase ^= 1;
                return b;
            };
            // (after a timeout, which is reported, the waits return at once and the loop runs out)
            while (walk.next(s)) {
                if (i >= s.q_tiles) {
                    // nothing to multiply: the tiles are only handed on
#pragma unroll 1
                    for (int n = 2 * (s.t1 - s.t0); n > 0; --n) {
                        const int b = take();
                        if (lane < S::kCtas) mbar_arrive_remote(&sh.empty[b], lane);
                    }
                    continue;
                }
                wait(&sh.q_full[i], q_phase);
                q_phase ^= 1;
                int bv = 0, bk = 0;
                // turn j: P V of step j - 2, then S of step j
#pragma unroll 1
                for (int j = 2 * s.t0; j < 2 * s.t1 + 2; ++j) {
                    const int b = j & 1;
                    const bool pv = j >= 2 * s.t0 + 2, qk = j < 2 * s.t1;
                    if (pv && b == 0) {
                        bv = take();
                        if constexpr (!INT8 && !kPair)
                            zero_past<S::kDimsV>(dyn + S::kOffBufs + bv * S::kTileBytes,
                                                 s.sq.len - (j - 2) * kStep, lane);
                    }
                    if (qk && b == 0) bk = take();
                    if (pv) {
                        wait(&sh.p_full[i][b], p_phase);
                        if (b) p_phase ^= 1;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        if (pv) {
                            const uint64_t v_desc =
                                smem_desc_mn_sw128(buf_addr + bv * S::kTileBytes + b * kStep * 128, kTile * 128);
#pragma unroll
                            for (int k = 0; k < kStep / 16; ++k)
                                mma_from_tmem<kPair>(to, ts + 64 * b + 8 * k, v_desc + k * (2048 >> 4), kIdescO,
                                                     j > 2 * s.t0 + 2 || k > 0);
                            commit_both<kPair>(&sh.pv_done[i]);
                            if (b) commit_both<kPair>(&sh.empty[bv]);
                            if (j == 2 * s.t1 + 1) commit_both<kPair>(&sh.o_full[i]);
                        }
                        if (qk) {
                            const uint64_t q_desc = smem_desc_sw128(q_addr);
                            const uint64_t k_desc =
                                smem_desc_sw128(buf_addr + bk * S::kTileBytes + b * (S::kKeysK / 2) * 128);
#pragma unroll
                            for (int k = 0; k < DIM / 16; ++k) {
                                const uint32_t in = (k & 3) * 32;
                                mma_from_smem<kPair>(ts + 64 * b, q_desc + (((k >> 2) * kQRows * 128 + in) >> 4),
                                                     k_desc + (((k >> 2) * S::kKeysK * 128 + in) >> 4), kIdescS, k > 0);
                            }
                            commit_both<kPair>(&sh.s_full[i][b]);
                            if (b) commit_both<kPair>(&sh.empty[bk]);
                        }
                    }
                    __syncwarp();
                }
            }
            // nothing of this warp's products is in flight when the tensor memory is given back
            if (elect_one()) commit_both<kPair>(&sh.done);
            __syncwarp();
            mbar_wait_bounded(&sh.done, 0);
        } else if (kPair && warp == kPassWarp && (!INT8 || rank != 0)) {
            // ---------------------------------------------------- this CTA's parts are there
            // A release at cluster scope waits for the warp's writes on their way: by the converting
            // warps themselves an int8 chunk of 4096 over 8192 keys takes 1211 us, by this warp, which
            // writes next to nothing, 1112 (8 mixed chunks: 386 and 335).
            int buf = 0;
            uint32_t phase = 0;
            bool ok = true;
            while (ok && walk.next(s)) {
#pragma unroll 1
                for (int n = 0; n < 2 * (s.t1 - s.t0); ++n) {  // K and V in turn
                    if (!(ok = warp_wait(&sh.abort, &sh.landed[buf], phase))) break;
                    bool written = INT8;
                    if (!INT8 && (n & 1))
                        written = zero_past<S::kDimsV>(dyn + S::kOffBufs + buf * S::kTileBytes,
                                                       s.sq.len - (s.t0 + n / 2) * kTile, lane);
                    if (lane == 0) {
                        if (written) arrive_even_written<kPair>(&sh.full[buf], rank);
                        else arrive_even<kPair>(&sh.full[buf]);
                    }
                    if (++buf == S::kBufs) buf = 0, phase ^= 1;
                }
            }
        }
    } else {
        reg_dec<S::kOtherRegs>();
        if constexpr (INT8) {
            // -------------------------------------------------------- codes to bf16 tiles
            int raw = 0, buf = 0;
            uint32_t raw_phase = 0, phase = 0;
            bool ok = true;
            const int tid = threadIdx.x & 127;
            while (ok && walk.next(s)) {
                for (int n = 2 * (s.t1 - s.t0); n > 0; --n) {
                    if (!(ok = warp_wait(&sh.abort, &sh.raw_full[raw], raw_phase))) break;
                    if (!(ok = warp_wait(&sh.abort, &sh.empty[buf], phase ^ 1))) break;
                    const uint8_t* src = dyn + S::kOffRaw + raw * S::kRawBytes;
                    uint8_t* dst = dyn + S::kOffBufs + buf * S::kTileBytes;
                    if (n & 1) convert_tile<S::kDimsV, kTile, false>(src, dst, tid);  // V
                    else convert_tile<DIM, S::kKeysK, true>(src, dst, tid);           // K
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(kPair && rank != 0 ? &sh.landed[buf] : &sh.full[buf]);
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
    if constexpr (kPair) cluster_sync_all();  // the products read both CTAs' memory: neither ends before they have
    tc_fence_after();
    if (threadIdx.x == 0 && sh.abort) raise_error(a.err, kErrTimeout);
    if (warp == kMmaWarp) {
        if constexpr (kPair) tmem_dealloc_pair(tmem, kTmemCols);
        else tmem_dealloc(tmem, kTmemCols);
    }
}

template <int DIM, bool INT8, bool PAIR>
cudaError_t launch_chunk_shape(const AttnParams& p, cudaStream_t stream)
{
    using S = ChunkShape<DIM, INT8, PAIR>;
    static std::atomic<size_t> smem_set[kHostMaxDevices];
    const KvPages& kv = p.a.cache;
    ChunkParams cp{};
    cp.p = p;
    const uint64_t outer = static_cast<uint64_t>(kv.n_pages) * kv.n_kv;
    const auto type = INT8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const auto swizzle = [](int bytes) { return bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B; };
    const int bytes = INT8 ? 1 : 2, cols_k = INT8 ? DIM : 64, cols_v = INT8 ? S::kDimsV : 64;
    const int box_k = S::kPair && kv.page > 32 ? 32 : kv.page;
    if (!encode_tma_3d(&cp.k_map, type, bytes, kv.k, DIM, kv.page, outer, cols_k, box_k, swizzle(cols_k * bytes)) ||
        !encode_tma_3d(&cp.v_map, type, bytes, kv.v, DIM, kv.page, outer, cols_v, kv.page, swizzle(cols_v * bytes)))
        return cudaErrorInvalidValue;
    constexpr size_t smem = chunk_smem<S>();
    const void* kernel = reinterpret_cast<const void*>(attn_chunk_kernel<DIM, INT8, PAIR>);
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
    launch_dep_clusters(err, attn_chunk_kernel<DIM, INT8, PAIR>, dim3(p.blocks * S::kCtas), dim3(S::kThreads), S::kCtas, smem,
                        stream, cp);
    return err;
}

}  // namespace

BD_BOUNDS_TAKE(bounds_take_attention_chunk)

cudaError_t launch_attention_chunk(const AttnParams& p, cudaStream_t stream)
{
    const bool int8 = p.a.cache.int8 != 0;
    if (p.mb == kPairRows) {
        return int8 ? launch_chunk_shape<128, true, true>(p, stream) : launch_chunk_shape<128, false, true>(p, stream);
    }
    if (p.a.cache.dim == 128)
        return int8 ? launch_chunk_shape<128, true, false>(p, stream) : launch_chunk_shape<128, false, false>(p, stream);
    return int8 ? launch_chunk_shape<64, true, false>(p, stream) : launch_chunk_shape<64, false, false>(p, stream);
}

}  // namespace bd
