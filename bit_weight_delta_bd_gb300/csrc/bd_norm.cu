// RMS norm with the residual's addition and, for tokens of several variants,
// each token's own gain:
//   h = x + r,   y = h * (mean h^2 + eps)^(-1/2) * gain_{vid}
// and y rounded to bf16, fp32 or e4m3 with a scale per row.
//
// A block works on a row at a time (many rows of up to 512 elements: a warp does);
// a thread keeps its groups of 8 elements of h in registers between the sum of
// squares and the output, so x and r are read once and h and y written once:
// the kernel is bound by those bytes.  While a row is added up the next one is
// already on its way, so that the block's meeting does not leave memory idle.
// The largest |y| of a row, which the 8-bit output's scale needs, is |h
// gain|'s largest times the row's factor, so it is found in the same pass as
// the sum and the block meets once.
#include <cuda_fp8.h>

#include "bd_device.cuh"

namespace bd {
namespace {

constexpr int kOutBf16 = 0, kOutF32 = 1, kOutE4m3 = 2;
constexpr int kNormMaxThreads = 1024;
constexpr int kNormThreads = 512;
constexpr int kWarpRows = 8;  // rows of a block where a row is a warp's

struct NormParams {
    NormArgs a;
};

__device__ __forceinline__ float2 bf16x2_f32(uint32_t u)
{
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t f32_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
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
template <bool WARP>
__device__ __forceinline__ float2 row_reduce(float s, float m, float2* red)
{
    const auto warp_reduce = [&]() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
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

// 8 elements of x and of the residual
struct Raw {
    uint4 u, r;
};

__device__ __forceinline__ void load_raw(const NormArgs& a, int64_t at, Raw& w)
{
    w.u = w.r = make_uint4(0, 0, 0, 0);
    if (bd_in_range(kBkNorm, at, 8, a.T * a.d)) {
        w.u = *reinterpret_cast<const uint4*>(a.x + at);
        if (a.residual) w.r = *reinterpret_cast<const uint4*>(a.residual + at);
    }
}

// their sums h
__device__ __forceinline__ void form_h(const NormArgs& a, const Raw& w, float (&h)[8])
{
    const uint4 u = w.u, r = w.r;
    const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_f32(uu[i]);
        h[2 * i] = f.x;
        h[2 * i + 1] = f.y;
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_f32(rr[i]);
            h[2 * i] += f.x;
            h[2 * i + 1] += f.y;
        }
    }
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

__device__ __forceinline__ void load_gain(const uint16_t* gain, int64_t g, float (&w)[8])
{
    const uint4 v = *reinterpret_cast<const uint4*>(gain + 8 * g);
    const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_f32(vv[i]);
        w[2 * i] = f.x;
        w[2 * i + 1] = f.y;
    }
}

// NG: groups of 8 elements that a thread keeps (0: the row is longer than
// the block can keep, and h is formed again from x and r in each pass).
template <int NG, int OUT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kNormMaxThreads, WARP ? 4 : 1)
    rms_norm_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float2 red[2][32];  // by turns: a warp may still read the last row's
    const NormArgs& a = p.a;
    const int64_t groups = a.d / 8;
    const int first = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    const int64_t rows_step = static_cast<int64_t>(gridDim.x) * (WARP ? kWarpRows : 1);
    int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    constexpr int kKeep = NG > 0 ? NG : 1;
    float h[kKeep][8];
    Raw raw[kKeep];
    constexpr bool kAhead = !WARP && NG <= 2;  // the next row is loaded early (with four groups, registers are short)
    const auto load_row = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int64_t g = first + static_cast<int64_t>(i) * step;
            if (g < groups) load_raw(a, r * a.d + 8 * g, raw[i]);
        }
    };

    grid_launch_dependents();
    grid_dependency_wait();
    if (kAhead && t < a.T) load_row(t);
    for (int turn = 0; t < a.T; t += rows_step, turn ^= 1) {
        if constexpr (!kAhead) load_row(t);
        const int64_t row = t * a.d;
        const uint16_t* gain = a.gain;
        if (a.vid) {
            const int v = a.vid[t];
            if (v >= 0 && v < a.V)
                gain = a.gains[v];
            else if (v != -1 && first == 0)
                raise_error(a.err, kErrBadVariant);
        }

        float ss = 0.0f, amax = 0.0f;
        const auto add_up = [&](int64_t g, const float (&x)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
            if constexpr (OUT == kOutE4m3) {
                float w[8];
                load_gain(gain, g, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(x[e] * w[e]));
            }
        };
        if constexpr (NG > 0) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t g = first + static_cast<int64_t>(i) * step;
                if (g < groups) form_h(a, raw[i], h[i]);
            }
            if constexpr (kAhead)
                if (t + rows_step < a.T) load_row(t + rows_step);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t g = first + static_cast<int64_t>(i) * step;
                if (g < groups) add_up(g, h[i]);
            }
        } else {
            for (int64_t g = first; g < groups; g += step) {
                load_raw(a, row + 8 * g, raw[0]);
                form_h(a, raw[0], h[0]);
                add_up(g, h[0]);
            }
        }
        const float2 both = row_reduce<WARP>(ss, amax, red[turn]);
        const float rstd = rsqrtf(both.x / static_cast<float>(a.d) + a.eps);
        float mult = 1.0f;
        if constexpr (OUT == kOutE4m3) {
            amax = max_nan(both.y * rstd, 1e-30f);
            mult = 448.0f / amax;
            if (first == 0) a.scale[t] = amax / 448.0f;
        }

        const auto put = [&](int64_t g, const float (&x)[8]) {
            const int64_t at = row + 8 * g;
            if (!bd_in_range(kBkNorm, at, 8, a.T * a.d)) return;
            if (a.residual_out) store_bf16(a.residual_out + at, x);
            float y[8];
            load_gain(gain, g, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e] * rstd * y[e];
            if constexpr (OUT == kOutBf16) {
                store_bf16(static_cast<uint16_t*>(a.out) + at, y);
            } else if constexpr (OUT == kOutF32) {
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
                o[0] = make_float4(y[0], y[1], y[2], y[3]);
                o[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + at) =
                    make_uint2(e4m3x4(y[0] * mult, y[1] * mult, y[2] * mult, y[3] * mult),
                               e4m3x4(y[4] * mult, y[5] * mult, y[6] * mult, y[7] * mult));
            }
        };
        if constexpr (NG > 0) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t g = first + static_cast<int64_t>(i) * step;
                if (g < groups) put(g, h[i]);
            }
        } else {
            // each thread reads a group of x and r again before it writes the
            // same group of residual_out, which may be either's buffer
            for (int64_t g = first; g < groups; g += step) {
                load_raw(a, row + 8 * g, raw[0]);
                form_h(a, raw[0], h[0]);
                put(g, h[0]);
            }
        }
    }
}

template <int NG, bool WARP>
cudaError_t launch_groups(const NormParams& p, int threads, int sm_count, cudaStream_t stream)
{
    cudaError_t err = cudaSuccess;
    // 2048 threads for each SM; rows that are a warp's, all at once
    const int64_t blocks = WARP ? (p.a.T + kWarpRows - 1) / kWarpRows : p.a.T;
    const int64_t resident = WARP ? blocks : static_cast<int64_t>(sm_count) * (2048 / threads);
    const dim3 grid(static_cast<unsigned>(blocks < resident ? blocks : resident));
    if (p.a.out_dtype == kOutBf16)
        launch_dep(err, rms_norm_kernel<NG, kOutBf16, WARP>, grid, dim3(threads), 0, stream, p);
    else if (p.a.out_dtype == kOutF32)
        launch_dep(err, rms_norm_kernel<NG, kOutF32, WARP>, grid, dim3(threads), 0, stream, p);
    else
        launch_dep(err, rms_norm_kernel<NG, kOutE4m3, WARP>, grid, dim3(threads), 0, stream, p);
    return err;
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int sm_count, cudaStream_t stream)
{
    if (a.T == 0) return cudaSuccess;
    NormParams p{a};
    const int64_t groups = a.d / 8;
    const auto threads_for = [&](int ng) {
        const int64_t n = (groups + ng - 1) / ng;
        return static_cast<int>((n + 31) / 32 * 32);
    };
    // Few rows: as many threads on a row as it has groups, for its latency.
    // Many: a warp for short rows, else two groups a thread (4096 rows of 8192:
    // bf16 41.7 us and e4m3 38.2 with 512 threads, 43.6 and 42.2 with 1024 and
    // one group, 53.7 and 56.0 with 256 and four; 8192 of 16384: 176 and 155
    // with 1024, 201 and 212 with 512 and four).
    const bool few = a.T <= 2 * sm_count;
    if (!few && groups <= 32) return launch_groups<1, true>(p, 32 * kWarpRows, sm_count, stream);
    if (!few && groups <= 64) return launch_groups<2, true>(p, 32 * kWarpRows, sm_count, stream);
    if (groups <= (few ? kNormMaxThreads : kNormThreads))
        return launch_groups<1, false>(p, threads_for(1), sm_count, stream);
    if (groups <= 2 * kNormMaxThreads) return launch_groups<2, false>(p, threads_for(2), sm_count, stream);
    if (groups <= 4 * kNormMaxThreads) return launch_groups<4, false>(p, threads_for(4), sm_count, stream);
    return launch_groups<0, false>(p, kNormMaxThreads, sm_count, stream);
}

BD_BOUNDS_TAKE(bounds_take_norm)

}  // namespace bd
