// The norms around a block: the RMS norm of what the block gives, its gate, the
// sum with the residual, and the RMS norm that the next block takes,
//   n = x (mean x^2 + eps)^(-1/2) post_gain_{vid}     (n = x without post_gain)
//   h = residual_scale r + block_scale gate n
//   y = h (mean h^2 + eps)^(-1/2) gain_{vid}
// with h rounded to bf16 and y to bf16, fp32 or e4m3 with a scale per row.
//
// Bound by the bytes: x, r (and a gate of each token) are read once, h and y
// written once.  A block, or for short rows a warp, works on a row at a time
// and keeps it in registers; it meets twice, for the sum of x^2 and for that of
// h^2.  (One meeting would do with the sums of x^2, r^2, x r and their weights,
// but where h is what is left of two large terms, the sum of its squares would
// be what is left of theirs.)  While a row is worked on the next one is on its
// way.  The largest |y|, which the 8-bit output's scale needs, is |h gain|'s
// largest times the row's factor, so it comes with the second sum.
#include <cuda_fp8.h>

#include <atomic>
#include <cmath>

#include "bd_device.cuh"
#include "bd_tma.h"

namespace bd {
namespace {

constexpr int kOutBf16 = 0, kOutF32 = 1, kOutE4m3 = 2;
constexpr int kMaxThreads = 1024;

struct BlockNormParams {
    BlockNormArgs a;
};

__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t f32_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&y)[8])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(f32_bf16x2(y[0], y[1]), f32_bf16x2(y[2], y[3]), f32_bf16x2(y[4], y[5]),
                                              f32_bf16x2(y[6], y[7]));
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// the larger of two, NaN if either is NaN (fmaxf would drop it)
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum of s and maximum of m (NaN if one is) over the row's threads, in a fixed
// order; all of them get both.
template <bool WARP, bool MAX>
__device__ __forceinline__ float2 row_reduce(float s, float m, float2* red)
{
    const auto warp_reduce = [&]() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            if constexpr (MAX) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
    };
    warp_reduce();
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        if (lane == 0) red[warp] = make_float2(s, m);
        __syncthreads();
        const float2 v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
        s = v.x;
        m = v.y;
        warp_reduce();
    }
    return make_float2(s, m);
}

// 8 elements of the block's output, the residual and the gate
struct Raw {
    uint4 x, r, g;
};

// A token's gains and gate.
struct Rows {
    const uint16_t *post, *gain, *gate;
};

__device__ __forceinline__ Rows rows_of(const BlockNormArgs& a, int64_t t, bool report)
{
    Rows w{a.post_gain, a.gain, a.gate};
    if (a.vid) {
        const int v = a.vid[t];
        if (v >= 0 && v < a.V) {
            w.gain = a.gains[v];
            if (a.post_gain) w.post = a.post_gains[v];
        } else if (v != -1 && report) {
            raise_error(a.err, kErrBadVariant);
        }
    }
    if (a.gate && a.gate_rows > 1) {
        int64_t i = a.gate_idx ? a.gate_idx[t] : t;
        if (i < 0 || i >= a.gate_rows) {
            if (report) raise_error(a.err, kErrBadIndex);
            i = 0;
        }
        w.gate = a.gate + i * a.d;
    } else if (a.gate_idx && report && a.gate_idx[t] != 0) {
        raise_error(a.err, kErrBadIndex);
    }
    return w;
}

__device__ __forceinline__ void load_raw(const BlockNormArgs& a, int64_t at, const uint16_t* gate, int64_t g, Raw& w)
{
    w.x = w.r = w.g = make_uint4(0, 0, 0, 0);
    if (bd_in_range(kBkBlockNorm, at, 8, a.T * a.d)) {
        w.x = *reinterpret_cast<const uint4*>(a.x + at);
        w.r = *reinterpret_cast<const uint4*>(a.residual + at);
        if (gate) w.g = *reinterpret_cast<const uint4*>(gate + 8 * g);
    }
}

__device__ __forceinline__ float add_squares(float s, uint4 u)
{
    float f[8];
    unpack8(u, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(f[e], f[e], s);
    return s;
}

// h of 8 elements; rstd and the gain of the norm after the block, if there is one
__device__ __forceinline__ void form_h(const BlockNormArgs& a, const Raw& w, const uint16_t* post, int64_t g, float rstd,
                                       float (&h)[8])
{
    unpack8(w.x, h);
    if (post) {
        float p[8];
        unpack8(*reinterpret_cast<const uint4*>(post + 8 * g), p);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = h[e] * rstd * p[e];
    }
    if (a.gate) {
        float q[8];
        unpack8(w.g, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] *= q[e];
    }
    float r[8];
    unpack8(w.r, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = fmaf(a.block_scale, h[e], a.residual_scale * r[e]);
}

// 8 elements of h, from element `at` of the matrix on, and of the norm's output.
template <int OUT>
__device__ __forceinline__ void put_group(const BlockNormArgs& a, int64_t at, const uint16_t* gain, const float (&z)[8],
                                          float mult, float code)
{
    if (!bd_in_range(kBkBlockNorm, at, 8, a.T * a.d)) return;
    if (a.residual_out) store_bf16(a.residual_out + at, z);
    float y[8];
    unpack8(*reinterpret_cast<const uint4*>(gain), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = z[e] * mult * y[e];
    if constexpr (OUT == kOutBf16) {
        store_bf16(static_cast<uint16_t*>(a.out) + at, y);
    } else if constexpr (OUT == kOutF32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
        o[0] = make_float4(y[0], y[1], y[2], y[3]);
        o[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + at) =
            make_uint2(e4m3x4(y[0] * code, y[1] * code, y[2] * code, y[3] * code),
                       e4m3x4(y[4] * code, y[5] * code, y[6] * code, y[7] * code));
    }
}

// NG: groups of 8 elements that a thread keeps (0: the row is longer than the
// block can keep, and h is formed again from its terms in each pass).
template <int NG, int OUT>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_kernel(const __grid_constant__ BlockNormParams p)
{
    // the first sum's, and the second's by turns: a warp may still read the last row's
    __shared__ float2 red[3][32];
    const BlockNormArgs& a = p.a;
    const int64_t groups = a.d / 8;
    const int first = threadIdx.x, step = blockDim.x;
    const int64_t rows_step = gridDim.x;
    int64_t t = blockIdx.x;
    constexpr int kKeep = NG > 0 ? NG : 1;
    constexpr bool kAhead = NG > 0 && NG <= 2;  // the next row is loaded early (with four groups, registers are short)
    Raw raw[kKeep];
    Rows rows{}, next{};
    const auto load_row = [&](int64_t r, Rows& w) {
        w = rows_of(a, r, first == 0);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int64_t g = first + static_cast<int64_t>(i) * step;
            if (g < groups) load_raw(a, r * a.d + 8 * g, w.gate, g, raw[i]);
        }
    };

    grid_launch_dependents();
    grid_dependency_wait();
    if (kAhead && t < a.T) load_row(t, next);
    for (int turn = 0; t < a.T; t += rows_step, turn ^= 1) {
        if constexpr (kAhead) rows = next;
        else load_row(t, rows);
        const int64_t row = t * a.d;

        // ---- the norm after the block
        float rstd = 1.0f;
        if (rows.post) {
            float ss = 0.0f;
            if constexpr (NG > 0) {
#pragma unroll
                for (int i = 0; i < NG; ++i)
                    if (first + static_cast<int64_t>(i) * step < groups) ss = add_squares(ss, raw[i].x);
            } else {
                for (int64_t g = first; g < groups; g += step)
                    if (bd_in_range(kBkBlockNorm, row + 8 * g, 8, a.T * a.d))
                        ss = add_squares(ss, *reinterpret_cast<const uint4*>(a.x + row + 8 * g));
            }
            rstd = rsqrtf(row_reduce<false, false>(ss, 0.0f, red[0]).x / static_cast<float>(a.d) + a.eps);
        }

        // ---- h, the sum of its squares, and the largest |h gain|
        float ss = 0.0f, amax = 0.0f;
        const auto add_up = [&](int64_t g, const float (&h)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[e], h[e], ss);
            if constexpr (OUT == kOutE4m3) {
                float w[8];
                unpack8(*reinterpret_cast<const uint4*>(rows.gain + 8 * g), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(h[e] * w[e]));
            }
        };
        float h[kKeep][8];
        if constexpr (NG > 0) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t g = first + static_cast<int64_t>(i) * step;
                if (g < groups) form_h(a, raw[i], rows.post, g, rstd, h[i]);
            }
            if constexpr (kAhead)
                if (t + rows_step < a.T) load_row(t + rows_step, next);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t g = first + static_cast<int64_t>(i) * step;
                if (g < groups) add_up(g, h[i]);
            }
        } else {
            for (int64_t g = first; g < groups; g += step) {
                load_raw(a, row + 8 * g, rows.gate, g, raw[0]);
                form_h(a, raw[0], rows.post, g, rstd, h[0]);
                add_up(g, h[0]);
            }
        }
        const float2 both = row_reduce<false, OUT == kOutE4m3>(ss, amax, red[1 + turn]);
        const float mult = rsqrtf(both.x / static_cast<float>(a.d) + a.eps);
        float code = 1.0f;
        if constexpr (OUT == kOutE4m3) {
            amax = max_nan(both.y * mult, 1e-30f);
            code = 448.0f / amax;
            if (first == 0) a.scale[t] = amax / 448.0f;
        }

        // ---- out
        const auto put = [&](int64_t g, const float (&z)[8]) {
            put_group<OUT>(a, row + 8 * g, rows.gain + 8 * g, z, mult, code);
        };
        if constexpr (NG > 0) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t g = first + static_cast<int64_t>(i) * step;
                if (g < groups) put(g, h[i]);
            }
        } else {
            // each thread reads a group again before it writes the same group
            // of residual_out, which may be x's or the residual's buffer
            for (int64_t g = first; g < groups; g += step) {
                load_raw(a, row + 8 * g, rows.gate, g, raw[0]);
                form_h(a, raw[0], rows.post, g, rstd, h[0]);
                put(g, h[0]);
            }
        }
    }
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
// a pair of bf16
__device__ __forceinline__ uint64_t pair(uint32_t w)
{
    return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Many rows: x, r and gates of a token's own come as bulk copies into a ring in
// shared memory, a few rows ahead of the one that is worked on, so that neither
// the meetings nor the registers say how much is on its way.  A row is a block's,
// or of up to 128 groups a warp's, with a ring of its own and no meeting; a stage
// is free again when the sum of the row's h^2 is there, which all have put their
// parts into.  What is kept of a row from there on is h gain.  With three stages
// or more the sum of the next row's x^2 is formed in the same meeting, one for each
// row; with two the next row would have to be there before the one after it is
// asked for (4096 x 8192 gated e4m3: 59.5 us with one meeting, 57.5 with two; bf16
// with one gate and three stages 51.7 and 54.0).
// Gates that tokens share come through the ring as well: read where they are used,
// which leaves room for a third stage, 20011 rows of 1000 take 47.5 us for 35.8 (on
// their way early, with the gains: 42.6).  Seven, six or five warps of a block in
// place of eight, with a longer ring each: 37.1, 40.1 and 44.8.
constexpr int kRingMaxStages = 8;
constexpr int kRingWarps = 8;  // rows of a block where a row is a warp's

// Blocks of an SM that the registers allow for, of up to `block` threads.
constexpr int ring_blocks(int ng, int block, bool warp) { return warp ? 6 - ng : 1024 / block; }

// Sums of a and b, and the largest m, over the row's threads.  (m is the bits of a
// magnitude, whose order is that of the numbers, with NaN above all.)
template <bool WARP, bool MAX>
__device__ __forceinline__ float3 ring_reduce(float a, float b, uint32_t m, float4* red)
{
    const auto warp_reduce = [&]() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if constexpr (MAX) m = __reduce_max_sync(0xffffffffu, m);
    };
    warp_reduce();
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        if (lane == 0) red[warp] = make_float4(a, b, __uint_as_float(m), 0.0f);
        __syncthreads();
        const float4 v = lane < warps ? red[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        a = v.x;
        b = v.y;
        m = __float_as_uint(v.z);
        warp_reduce();
    }
    return make_float3(a, b, __uint_as_float(m));
}

struct RingParams {
    BlockNormArgs a;
    int stages, row_bytes;  // of a row's ring; bytes of a row of x
};

template <int NG, int OUT, int BLOCK, bool WARP>
__global__ void __launch_bounds__(BLOCK, ring_blocks(NG, BLOCK, WARP)) block_norm_ring_kernel(const __grid_constant__ RingParams p)
{
    constexpr int kRows = WARP ? kRingWarps : 1;  // of the block at a time
    extern __shared__ __align__(128) uint8_t ring_all[];
    // by turns: a warp may still read the last row's; and the one of a meeting that the other lies between
    __shared__ float4 red[3][32];
    __shared__ uint64_t full_all[kRows][kRingMaxStages];
    __shared__ volatile int given_up;
    __shared__ int64_t unfilled[kRows];  // given up: the first row that was not asked for any more
    const BlockNormArgs& a = p.a;
    const int which = WARP ? threadIdx.x >> 5 : 0;
    const int first = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    const int groups = static_cast<int>(a.d / 8);
    const bool own_gates = a.gate && a.gate_rows > 1;
    const int stage_bytes = p.row_bytes * (own_gates ? 3 : 2);
    uint8_t* const ring = ring_all + static_cast<size_t>(which) * p.stages * stage_bytes;
    uint64_t* const full = full_all[which];
    const int64_t rows_step = static_cast<int64_t>(gridDim.x) * kRows;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows + which;

    grid_launch_dependents();
    if (first == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        unfilled[which] = a.T;
        if (which == 0) given_up = 0;
        fence_mbarrier_init();
    }
    __syncthreads();
    grid_dependency_wait();

    // the row of a gate that token t takes
    const auto gate_row = [&](int64_t t) {
        if (t >= a.T) return static_cast<int64_t>(0);
        int64_t i = a.gate_idx ? a.gate_idx[t] : t;
        if (i < 0 || i >= a.gate_rows) {
            raise_error(a.err, kErrBadIndex);
            i = 0;
        }
        return i;
    };
    // by the row's first thread: row t into stage s.  Not once a wait was given up, which this thread knows of before it
    // gets to a stage whose copies may still be on their way.
    const auto fill = [&](int64_t t, int s, int64_t gate_at) {
        if (t >= a.T) return;
        if (given_up) {
            if (t < unfilled[which]) unfilled[which] = t;
            return;
        }
        uint8_t* dst = ring + static_cast<size_t>(s) * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_g2s(dst, a.x + t * a.d, p.row_bytes, &full[s]);
        bulk_g2s(dst + p.row_bytes, a.residual + t * a.d, p.row_bytes, &full[s]);
        if (own_gates) bulk_g2s(dst + 2 * p.row_bytes, a.gate + gate_at * a.d, p.row_bytes, &full[s]);
    };
    int64_t gate_next = 0;  // of the row that the next refill brings
    if (first == 0) {
        for (int s = 0; s < p.stages; ++s) fill(t0 + s * rows_step, s, own_gates ? gate_row(t0 + s * rows_step) : 0);
        if (own_gates) gate_next = gate_row(t0 + p.stages * rows_step);
    }
    int vid_next = a.vid && t0 < a.T ? a.vid[t0] : -1;
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    // waits for row t, and returns this thread's part of the sum of its x^2
    const auto squares = [&](int s, uint32_t ph) {
        // (given up, which is reported: what is there is worked on)
        if (!mbar_try_wait(&full[s], ph) && !given_up && !mbar_wait_sleeping(&full[s], ph)) {
            given_up = 1;
            raise_error(a.err, kErrTimeout);
        }
        if (!a.post_gain) return 0.0f;
        const uint4* xs = reinterpret_cast<const uint4*>(ring + static_cast<size_t>(s) * stage_bytes);
        uint64_t ss = 0;  // a pair of zeros
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            if (first + i * step >= groups) continue;
            const uint4 x = xs[first + i * step];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t f = pair(w[e]);
                ss = fma2(f, f, ss);
            }
        }
        const float2 s2 = unpack2(ss);
        return s2.x + s2.y;
    };
    const bool ahead = p.stages >= 3;
    float x_sum = 0.0f;
    if (ahead && t0 < a.T) x_sum = ring_reduce<WARP, false>(0.0f, squares(0, 0), 0u, red[1]).y;
    for (int64_t t = t0; t < a.T; t += rows_step, turn ^= 1) {
        const uint16_t *post = a.post_gain, *gain = a.gain;
        if (a.vid) {
            const int v = vid_next;
            if (v >= 0 && v < a.V) {
                gain = a.gains[v];
                if (post) post = a.post_gains[v];
            } else if (v != -1 && first == 0) {
                raise_error(a.err, kErrBadVariant);
            }
            if (t + rows_step < a.T) vid_next = a.vid[t + rows_step];
        }
        if (first == 0 && a.gate_idx && !own_gates && a.gate_idx[t] != 0) raise_error(a.err, kErrBadIndex);
        const uint4* xs = reinterpret_cast<const uint4*>(ring + static_cast<size_t>(stage) * stage_bytes);
        const uint4* rs = xs + groups;
        const uint4* gs = own_gates ? rs + groups : reinterpret_cast<const uint4*>(a.gate);
        uint4 post_gain[NG];  // on its way while the row is waited for
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            post_gain[i] = make_uint4(0, 0, 0, 0);
            if (post && first + i * step < groups)
                post_gain[i] = *(reinterpret_cast<const uint4*>(post) + first + i * step);
        }
        if (!ahead) {
            x_sum = squares(stage, phase);
            if (post) x_sum = ring_reduce<WARP, false>(0.0f, x_sum, 0u, red[2]).y;
        }
        const float c = post ? a.block_scale * rsqrtf(x_sum / static_cast<float>(a.d) + a.eps) : a.block_scale;
        const uint64_t c2 = f32x2(c, c), rs2 = f32x2(a.residual_scale, a.residual_scale);
        uint64_t ss = 0, z[NG][4];  // h gain
        uint32_t most = 0;  // the bits of the largest |h gain|
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int g = first + i * step;
            if (g >= groups) continue;
            const uint4 x = xs[g], r = rs[g], wg = *(reinterpret_cast<const uint4*>(gain) + g);
            const uint4 pg = post_gain[i];
            uint4 gate = make_uint4(0, 0, 0, 0);
            if (a.gate) gate = gs[g];
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, rw[4] = {r.x, r.y, r.z, r.w};
            const uint32_t pw[4] = {pg.x, pg.y, pg.z, pg.w}, gw[4] = {gate.x, gate.y, gate.z, gate.w};
            const uint32_t ww[4] = {wg.x, wg.y, wg.z, wg.w};
            uint32_t hw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint64_t n = mul2(pair(xw[e]), c2);
                if (post) n = mul2(n, pair(pw[e]));
                const uint64_t rr = mul2(pair(rw[e]), rs2);
                // (a gate multiplies, and joins the residual, in one rounding)
                const uint64_t h = a.gate ? fma2(n, pair(gw[e]), rr) : fma2(n, f32x2(1.0f, 1.0f), rr);
                ss = fma2(h, h, ss);
                z[i][e] = mul2(h, pair(ww[e]));
                const float2 hf = unpack2(h);
                hw[e] = f32_bf16x2(hf.x, hf.y);
                if constexpr (OUT == kOutE4m3) {
                    const float2 zf = unpack2(z[i][e]);
                    most = max(most, max(__float_as_uint(fabsf(zf.x)), __float_as_uint(fabsf(zf.y))));
                }
            }
            if (a.residual_out && bd_in_range(kBkBlockNorm, t * a.d + 8 * g, 8, a.T * a.d))
                *reinterpret_cast<uint4*>(a.residual_out + t * a.d + 8 * g) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        }
        const float2 s = unpack2(ss);
        const int following = stage + 1 == p.stages ? 0 : stage + 1;
        const float x_part = ahead && t + rows_step < a.T ? squares(following, following ? phase : phase ^ 1) : 0.0f;
        const float3 both = ring_reduce<WARP, OUT == kOutE4m3>(s.x + s.y, x_part, most, red[turn]);
        x_sum = both.y;
        if (first == 0) {  // all threads have read their part of the row
            fill(t + p.stages * rows_step, stage, gate_next);
            if (own_gates) gate_next = gate_row(t + (p.stages + 1) * rows_step);
        }
        const float mult = rsqrtf(both.x / static_cast<float>(a.d) + a.eps);
        [[maybe_unused]] float amax = 0.0f;
        if constexpr (OUT == kOutE4m3) {
            amax = max_nan(both.z * mult, 1e-30f);
            if (first == 0) a.scale[t] = amax / 448.0f;
        }
        // 8 bits: y 448 / max |y| in one factor; in two for a row so small that the one leaves fp32's range.
        float to_out = mult;
        if constexpr (OUT == kOutE4m3) {
            to_out = amax > 1e-30f ? 448.0f / both.z : mult * (448.0f / amax);
            if (__builtin_expect(to_out == INFINITY, 0)) {
                const uint64_t y2 = f32x2(mult, mult);
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[i][e] = mul2(z[i][e], y2);
                to_out = 448.0f / amax;
            }
        }
        const uint64_t m2 = f32x2(to_out, to_out);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int g = first + i * step;
            if (g >= groups) continue;
            const int64_t at = t * a.d + 8 * g;
            if (!bd_in_range(kBkBlockNorm, at, 8, a.T * a.d)) continue;
            float2 y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = unpack2(mul2(z[i][e], m2));
            }
            if constexpr (OUT == kOutBf16) {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
                    make_uint4(f32_bf16x2(y[0].x, y[0].y), f32_bf16x2(y[1].x, y[1].y), f32_bf16x2(y[2].x, y[2].y),
                               f32_bf16x2(y[3].x, y[3].y));
            } else if constexpr (OUT == kOutF32) {
                float* o = static_cast<float*>(a.out) + at;
                const uint4 lo = make_uint4(__float_as_uint(y[0].x), __float_as_uint(y[0].y), __float_as_uint(y[1].x),
                                            __float_as_uint(y[1].y));
                const uint4 hi = make_uint4(__float_as_uint(y[2].x), __float_as_uint(y[2].y), __float_as_uint(y[3].x),
                                            __float_as_uint(y[3].y));
                if (on_sector(a.out)) {
                    store_32(o, lo, hi);
                } else {
                    reinterpret_cast<uint4*>(o)[0] = lo;
                    reinterpret_cast<uint4*>(o)[1] = hi;
                }
            } else {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + at) = make_uint2(
                    e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y), e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y));
            }
        }
        if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    // given up: leave only when the copies in flight have landed, each stage's last ones
    __syncthreads();
    if (given_up && first < p.stages && t0 < a.T) {
        const int64_t rows = (unfilled[which] - t0 + rows_step - 1) / rows_step;  // that were, in the order of the stages
        if (rows > first) mbar_wait_bounded(&full[first], (rows - first - 1) / p.stages & 1);
    }
}

template <int NG, int BLOCK, bool WARP>
cudaError_t launch_ring(const BlockNormArgs& a, int threads, int sm_count, cudaStream_t stream)
{
    static std::atomic<size_t> smem_set[3][kHostMaxDevices];
    RingParams p{a, 0, static_cast<int>(a.d) * 2};
    // blocks of an SM: by its threads, and by the registers of a block that may have up to BLOCK of them
    const int by_registers = ring_blocks(NG, BLOCK, WARP) * (BLOCK / threads);
    const int per_sm = 2048 / threads < by_registers ? 2048 / threads : by_registers;
    const int rows = WARP ? kRingWarps : 1;
    const size_t stage = static_cast<size_t>(p.row_bytes) * (a.gate && a.gate_rows > 1 ? 3 : 2) * rows;
    const size_t room = (228u * 1024u) / per_sm - 3u * 1024u;
    p.stages = static_cast<int>(room / stage);
    if (p.stages > kRingMaxStages) p.stages = kRingMaxStages;
    if (p.stages < 2) return cudaErrorInvalidConfiguration;  // (rows that long do not come here)
    const size_t smem = stage * p.stages;
    const int64_t blocks = (a.T + rows - 1) / rows, resident = static_cast<int64_t>(sm_count) * per_sm;
    const dim3 grid(static_cast<unsigned>(blocks < resident ? blocks : resident));
    const auto go = [&](auto kernel, std::atomic<size_t>* set) {
        cudaError_t err = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem, set);
        launch_dep(err, kernel, grid, dim3(threads), smem, stream, p);
        return err;
    };
    if (a.out_dtype == kOutBf16) return go(block_norm_ring_kernel<NG, kOutBf16, BLOCK, WARP>, smem_set[0]);
    if (a.out_dtype == kOutF32) return go(block_norm_ring_kernel<NG, kOutF32, BLOCK, WARP>, smem_set[1]);
    return go(block_norm_ring_kernel<NG, kOutE4m3, BLOCK, WARP>, smem_set[2]);
}

template <int NG>
cudaError_t launch_groups(const BlockNormParams& p, int threads, int sm_count, cudaStream_t stream)
{
    cudaError_t err = cudaSuccess;
    const int64_t resident = static_cast<int64_t>(sm_count) * (2048 / threads);  // 2048 threads for each SM
    const dim3 grid(static_cast<unsigned>(p.a.T < resident ? p.a.T : resident));
    if (p.a.out_dtype == kOutBf16)
        launch_dep(err, block_norm_kernel<NG, kOutBf16>, grid, dim3(threads), 0, stream, p);
    else if (p.a.out_dtype == kOutF32)
        launch_dep(err, block_norm_kernel<NG, kOutF32>, grid, dim3(threads), 0, stream, p);
    else
        launch_dep(err, block_norm_kernel<NG, kOutE4m3>, grid, dim3(threads), 0, stream, p);
    return err;
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int sm_count, cudaStream_t stream)
{
    if (a.T == 0) return cudaSuccess;
    BlockNormParams p{a};
    const int64_t groups = a.d / 8;
    const auto threads_for = [&](int ng) {
        const int64_t n = (groups + ng - 1) / ng;
        return static_cast<int>((n + 31) / 32 * 32);
    };
    // Few rows: as many threads on a row as it has groups, for its latency.
    // Many: a warp for short rows, else two groups a thread.
    // The ring's kernel has block_scale and the first norm's factor, 2^-64 .. 2^74, in one number: not where that may
    // leave fp32's range (scales past 2^30 and 2^-30, far from those in use).
    const float bs = fabsf(a.block_scale);
    const bool few = a.T <= 2 * sm_count || (bs != 0.0f && (bs < 0x1p-30f || bs > 0x1p30f));
    if (!few && groups <= 32) return launch_ring<1, 32 * kRingWarps, true>(a, 32 * kRingWarps, sm_count, stream);
    if (!few && groups <= 64) return launch_ring<2, 32 * kRingWarps, true>(a, 32 * kRingWarps, sm_count, stream);
    if (!few && groups <= 128) return launch_ring<4, 32 * kRingWarps, true>(a, 32 * kRingWarps, sm_count, stream);
    if (!few && groups <= 1024) return launch_ring<2, 512, false>(a, threads_for(2), sm_count, stream);
    if (!few && groups <= 2048) return launch_ring<2, 1024, false>(a, threads_for(2), sm_count, stream);
    if (groups <= kMaxThreads) return launch_groups<1>(p, threads_for(1), sm_count, stream);
    if (groups <= 2 * kMaxThreads) return launch_groups<2>(p, threads_for(2), sm_count, stream);
    if (groups <= 4 * kMaxThreads) return launch_groups<4>(p, threads_for(4), sm_count, stream);
    return launch_groups<0>(p, kMaxThreads, sm_count, stream);
}

BD_BOUNDS_TAKE(bounds_take_block_norm)

}  // namespace bd
