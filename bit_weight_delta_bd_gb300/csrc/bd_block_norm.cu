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

#include "bd_device.cuh"

namespace bd {
namespace {

constexpr int kOutBf16 = 0, kOutF32 = 1, kOutE4m3 = 2;
constexpr int kMaxThreads = 1024;
constexpr int kThreads = 512;
constexpr int kWarpRows = 8;  // rows of a block where a row is a warp's

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

// NG: groups of 8 elements that a thread keeps (0: the row is longer than the
// block can keep, and h is formed again from its terms in each pass).
template <int NG, int OUT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kMaxThreads, WARP ? 2 : 1)
    block_norm_kernel(const __grid_constant__ BlockNormParams p)
{
    // the first sum's, and the second's by turns: a warp may still read the last row's
    __shared__ float2 red[3][32];
    const BlockNormArgs& a = p.a;
    const int64_t groups = a.d / 8;
    const int first = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    const int64_t rows_step = static_cast<int64_t>(gridDim.x) * (WARP ? kWarpRows : 1);
    int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    constexpr int kKeep = NG > 0 ? NG : 1;
    constexpr bool kAhead = !WARP && NG > 0 && NG <= 2;  // the next row is loaded early (with four groups, registers are short)
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
            rstd = rsqrtf(row_reduce<WARP, false>(ss, 0.0f, red[0]).x / static_cast<float>(a.d) + a.eps);
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
        const float2 both = row_reduce<WARP, OUT == kOutE4m3>(ss, amax, red[1 + turn]);
        const float mult = rsqrtf(both.x / static_cast<float>(a.d) + a.eps);
        float code = 1.0f;
        if constexpr (OUT == kOutE4m3) {
            amax = max_nan(both.y * mult, 1e-30f);
            code = 448.0f / amax;
            if (first == 0) a.scale[t] = amax / 448.0f;
        }

        // ---- out
        const auto put = [&](int64_t g, const float (&z)[8]) {
            const int64_t at = row + 8 * g;
            if (!bd_in_range(kBkBlockNorm, at, 8, a.T * a.d)) return;
            if (a.residual_out) store_bf16(a.residual_out + at, z);
            float y[8];
            unpack8(*reinterpret_cast<const uint4*>(rows.gain + 8 * g), y);
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

template <int NG, bool WARP>
cudaError_t launch_groups(const BlockNormParams& p, int threads, int sm_count, cudaStream_t stream)
{
    cudaError_t err = cudaSuccess;
    // 2048 threads for each SM; rows that are a warp's, all at once
    const int64_t blocks = WARP ? (p.a.T + kWarpRows - 1) / kWarpRows : p.a.T;
    const int64_t resident = WARP ? blocks : static_cast<int64_t>(sm_count) * (2048 / threads);
    const dim3 grid(static_cast<unsigned>(blocks < resident ? blocks : resident));
    if (p.a.out_dtype == kOutBf16)
        launch_dep(err, block_norm_kernel<NG, kOutBf16, WARP>, grid, dim3(threads), 0, stream, p);
    else if (p.a.out_dtype == kOutF32)
        launch_dep(err, block_norm_kernel<NG, kOutF32, WARP>, grid, dim3(threads), 0, stream, p);
    else
        launch_dep(err, block_norm_kernel<NG, kOutE4m3, WARP>, grid, dim3(threads), 0, stream, p);
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
    const bool few = a.T <= 2 * sm_count;
    if (!few && groups <= 32) return launch_groups<1, true>(p, 32 * kWarpRows, sm_count, stream);
    if (!few && groups <= 64) return launch_groups<2, true>(p, 32 * kWarpRows, sm_count, stream);
    if (groups <= (few ? kMaxThreads : kThreads)) return launch_groups<1, false>(p, threads_for(1), sm_count, stream);
    if (groups <= 2 * kMaxThreads) return launch_groups<2, false>(p, threads_for(2), sm_count, stream);
    if (groups <= 4 * kMaxThreads) return launch_groups<4, false>(p, threads_for(4), sm_count, stream);
    return launch_groups<0, false>(p, kMaxThreads, sm_count, stream);
}

BD_BOUNDS_TAKE(bounds_take_block_norm)

}  // namespace bd
