// RMS norm with the residual's addition and, for tokens of several variants,
// each token's own gain:
//   h = x + r,   y = h * (mean h^2 + eps)^(-1/2) * gain_{vid}
// and y rounded to bf16, fp32 or e4m3 with a scale per row.
//
// One block per row; a thread keeps its groups of 8 elements of h in
// registers between the sum of squares and the output, so x and r are read
// once and h and y written once: the kernel is bound by those bytes.
#include <cuda_fp8.h>

#include "bd_device.cuh"

namespace bd {
namespace {

constexpr int kOutBf16 = 0, kOutF32 = 1, kOutE4m3 = 2;
constexpr int kNormMaxThreads = 1024;

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

struct SumOp {
    static __device__ __forceinline__ float zero() { return 0.0f; }
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct MaxOp {
    static __device__ __forceinline__ float zero() { return 0.0f; }
    static __device__ __forceinline__ float of(float a, float b) { return max_nan(a, b); }
};

// Reduction over the block in a fixed order; every thread gets the result.
template <typename Op>
__device__ __forceinline__ float block_reduce(float v, float* red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = Op::of(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : Op::zero();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = Op::of(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// h of group g (8 elements) of a row
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t at, float (&h)[8])
{
    uint4 u = make_uint4(0, 0, 0, 0), r = make_uint4(0, 0, 0, 0);
    if (bd_in_range(kBkNorm, at, 8, a.T * a.d)) {
        u = *reinterpret_cast<const uint4*>(a.x + at);
        if (a.residual) r = *reinterpret_cast<const uint4*>(a.residual + at);
    }
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

__device__ __forceinline__ void times_gain(const uint16_t* gain, int64_t g, float rstd, float (&h)[8])
{
    const uint4 w = *reinterpret_cast<const uint4*>(gain + 8 * g);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_f32(ww[i]);
        h[2 * i] = h[2 * i] * rstd * f.x;
        h[2 * i + 1] = h[2 * i + 1] * rstd * f.y;
    }
}

// NG: groups of 8 elements that a thread keeps (0: the row is longer than
// the block can keep, and h is formed again from x and r in each pass).
template <int NG, int OUT>
__global__ void __launch_bounds__(kNormMaxThreads) rms_norm_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float red[2][32];
    const NormArgs& a = p.a;
    const int64_t groups = a.d / 8;
    const int64_t t = blockIdx.x;
    const int64_t row = t * a.d;
    constexpr int kKeep = NG > 0 ? NG : 1;
    float h[kKeep][8];

    grid_launch_dependents();
    grid_dependency_wait();

    const uint16_t* gain = a.gain;
    if (a.vid) {
        const int v = a.vid[t];
        if (v >= 0 && v < a.V)
            gain = a.gains[v];
        else if (v != -1 && threadIdx.x == 0)
            raise_error(a.err, kErrBadVariant);
    }

    float ss = 0.0f;
    if constexpr (NG > 0) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int64_t g = threadIdx.x + static_cast<int64_t>(i) * blockDim.x;
            if (g < groups) {
                load_h(a, row + 8 * g, h[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
    } else {
        for (int64_t g = threadIdx.x; g < groups; g += blockDim.x) {
            load_h(a, row + 8 * g, h[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[0][e], h[0][e], ss);
        }
    }
    ss = block_reduce<SumOp>(ss, red[0]);
    const float rstd = rsqrtf(ss / static_cast<float>(a.d) + a.eps);

    float mult = 1.0f;
    if constexpr (OUT == kOutE4m3) {
        float amax = 0.0f;
        if constexpr (NG > 0) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t g = threadIdx.x + static_cast<int64_t>(i) * blockDim.x;
                if (g >= groups) continue;
                if (a.residual_out) store_bf16(a.residual_out + row + 8 * g, h[i]);
                times_gain(gain, g, rstd, h[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(h[i][e]));
            }
        } else {
            for (int64_t g = threadIdx.x; g < groups; g += blockDim.x) {
                load_h(a, row + 8 * g, h[0]);
                times_gain(gain, g, rstd, h[0]);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(h[0][e]));
            }
        }
        amax = block_reduce<MaxOp>(amax, red[1]);
        amax = max_nan(amax, 1e-30f);
        mult = 448.0f / amax;
        if (threadIdx.x == 0) a.scale[t] = amax / 448.0f;
    }

    const auto put = [&](int64_t g, float (&y)[8]) {
        const int64_t at = row + 8 * g;
        if (!bd_in_range(kBkNorm, at, 8, a.T * a.d)) return;
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
            const int64_t g = threadIdx.x + static_cast<int64_t>(i) * blockDim.x;
            if (g >= groups) continue;
            if constexpr (OUT != kOutE4m3) {
                if (a.residual_out) store_bf16(a.residual_out + row + 8 * g, h[i]);
                times_gain(gain, g, rstd, h[i]);
            }
            put(g, h[i]);
        }
    } else {
        // each thread reads a group of x and r again before it writes the
        // same group of residual_out, which may be either's buffer
        for (int64_t g = threadIdx.x; g < groups; g += blockDim.x) {
            load_h(a, row + 8 * g, h[0]);
            if (a.residual_out) store_bf16(a.residual_out + row + 8 * g, h[0]);
            times_gain(gain, g, rstd, h[0]);
            put(g, h[0]);
        }
    }
}

template <int NG>
cudaError_t launch_groups(const NormParams& p, int threads, cudaStream_t stream)
{
    cudaError_t err = cudaSuccess;
    const dim3 grid(static_cast<unsigned>(p.a.T));
    if (p.a.out_dtype == kOutBf16)
        launch_dep(err, rms_norm_kernel<NG, kOutBf16>, grid, dim3(threads), 0, stream, p);
    else if (p.a.out_dtype == kOutF32)
        launch_dep(err, rms_norm_kernel<NG, kOutF32>, grid, dim3(threads), 0, stream, p);
    else
        launch_dep(err, rms_norm_kernel<NG, kOutE4m3>, grid, dim3(threads), 0, stream, p);
    return err;
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int /*sm_count*/, cudaStream_t stream)
{
    if (a.T == 0) return cudaSuccess;
    NormParams p{a};
    const int64_t groups = a.d / 8;
    const auto threads_for = [&](int ng) {
        const int64_t n = (groups + ng - 1) / ng;
        return static_cast<int>((n + 31) / 32 * 32);
    };
    if (groups <= kNormMaxThreads) return launch_groups<1>(p, threads_for(1), stream);
    if (groups <= 2 * kNormMaxThreads) return launch_groups<2>(p, threads_for(2), stream);
    if (groups <= 4 * kNormMaxThreads) return launch_groups<4>(p, threads_for(4), stream);
    return launch_groups<0>(p, kNormMaxThreads, stream);
}

BD_BOUNDS_TAKE(bounds_take_norm)

}  // namespace bd
