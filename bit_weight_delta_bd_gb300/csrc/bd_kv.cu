// The paged KV cache: rotary positions with the write into the cache, and
// reading the cache back.  Both kernels only move data (a few operations per
// element) and are bound by the bytes they read and write.
//
// Int8 codes.  Per (token, kv head): scale = max(max |x|, 1e-30) / 127 and
// code = round-half-even(x / scale), both with IEEE divisions.  The rotation
// rounds each product and each sum by itself (no contraction to fused
// multiply-adds), so codes and scales are those of the formula evaluated
// operation by operation in fp32, whatever computes them.
#include "bd_device.cuh"

namespace bd {
namespace {

constexpr int rope_threads(bool int8) { return int8 ? 64 : 32; }  // of a block at most
constexpr int kUnit = 16;  // elements of a head that one thread handles

__device__ __forceinline__ void unpack8(uint4 u, float* f)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float* f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 codes of x / scale as 8 bytes (the first element lowest)
__device__ __forceinline__ uint2 codes8(const float* x, float scale)
{
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int c = __float2int_rn(__fdiv_rn(x[i], scale));
        c = c < -127 ? -127 : c > 127 ? 127 : c;
        w[i / 4] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * (i % 4));
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct RopeParams {
    RopeArgs a;
};

// A thread handles 16 elements of a head: the 8 pairs (i, i + rot/2) from
// i = 8 u on, or elements 16 u .. 16 u + 15 (interleaved pairs, the part past
// rot, and v).  Its unit u stays the same for all heads it visits, so the
// cosines and sines are read once per token.  UPH = dim / 16 units per head;
// a block is one token (grid x) and one part of its heads (grid y), blockDim /
// UPH heads a pass.  What bounds it is how many tokens an SM works on at a
// time, since each waits for its position, then its table row, then its heads:
// small blocks, a head's successor loaded before it is worked on, and the first
// heads before the position is there.  One head ahead, or two where codes are
// formed, since more registers leave fewer blocks.  4096 tokens, 64/8 heads of
// 128: bf16 29.9 us, 5.7 TB/s, with 32 threads (64 threads 30.0, with two ahead
// 34.0, three 38.5; 256 threads 37.9; the position first 33.2), and 5 ragged
// prompts of up to 1201 tokens, 48 heads of 64, 11.6 us (64 threads 12.5);
// int8 and read back 37.9 us with 64 threads (32 threads 45.6; one ahead 39.5;
// loads only after the work on those before 40.5).
template <int UPH, bool INT8>
__global__ void __launch_bounds__(rope_threads(INT8)) rope_append_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kDim = UPH * kUnit;
    constexpr int kAhead = INT8 ? 2 : 1;  // heads that a thread has loaded, or is loading
    const RopeArgs& a = p.a;
    const int u = threadIdx.x % UPH;
    const int64_t t = blockIdx.x;
    const int n_kv = a.cache.n_kv;
    const int heads = a.n_q + 2 * n_kv;
    const int per_pass = blockDim.x / UPH, step = gridDim.y * per_pass;

    grid_launch_dependents();
    grid_dependency_wait();

    // this unit's elements, and whether they turn
    const bool turns = 16 * u < a.rot;
    const int first = turns && !a.interleaved ? 8 * u : 16 * u;
    const int second = turns && !a.interleaved ? 8 * u + a.rot / 2 : 16 * u + 8;

    uint4 raw[kAhead][2];
    const auto load = [&](int h, uint4 (&to)[2]) {
        if (h >= heads) return;
        const bool is_v = h >= a.n_q + n_kv;
        const uint16_t* src = h < a.n_q ? a.q + t * a.q_stride + static_cast<int64_t>(h) * kDim
                              : is_v    ? a.v + t * a.v_stride + static_cast<int64_t>(h - a.n_q - n_kv) * kDim
                                        : a.k + t * a.k_stride + static_cast<int64_t>(h - a.n_q) * kDim;
        to[0] = *reinterpret_cast<const uint4*>(src + (is_v ? 16 * u : first));
        to[1] = *reinterpret_cast<const uint4*>(src + (is_v ? 16 * u + 8 : second));
    };
    const int head0 = blockIdx.y * per_pass + threadIdx.x / UPH;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(head0 + i * step, raw[i]);

    float c[8], s[8];
    if (turns) {
        const int pair0 = 8 * u;
        int64_t pos[kMaxAxes];
#pragma unroll
        for (int x = 0; x < kMaxAxes; ++x) {
            pos[x] = x < a.n_axes ? a.pos[t * a.n_axes + x] : 0;
            if (pos[x] < 0 || pos[x] >= a.n_pos) {
                raise_error(a.err, kErrBadIndex);
                pos[x] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int x = a.axis_of_pair[pair0 + i];
            const int64_t at = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
            const float2 cs = *(reinterpret_cast<const float2*>(a.tab) + at * (a.rot / 2) + pair0 + i);
            c[i] = cs.x;
            s[i] = cs.y;
        }
    }
    const int64_t slots = a.cache.n_pages * a.cache.page;
    int64_t slot = a.slot[t];
    if (slot < -1 || slot >= slots) {
        if (threadIdx.x == 0) raise_error(a.err, kErrBadIndex);
        slot = -1;
    }
    const int64_t page = slot >> a.cache.page_shift, place = slot & (a.cache.page - 1);

    // all lanes of a warp run the same number of passes (the reductions use the full warp)
    const auto work = [&](int h, const uint4 (&from)[2]) {
        const bool live = h < heads;
        const bool is_q = h < a.n_q, is_v = h >= a.n_q + n_kv;
        const int e0 = is_v ? 16 * u : first, e1 = is_v ? 16 * u + 8 : second;
        float x[16];
        unpack8(from[0], x);
        unpack8(from[1], x + 8);
        if (turns && !is_v) {
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p0 = x[2 * i], p1 = x[2 * i + 1];
                    x[2 * i] = __fsub_rn(__fmul_rn(p0, c[i]), __fmul_rn(p1, s[i]));
                    x[2 * i + 1] = __fadd_rn(__fmul_rn(p1, c[i]), __fmul_rn(p0, s[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p0 = x[i], p1 = x[8 + i];
                    x[i] = __fsub_rn(__fmul_rn(p0, c[i]), __fmul_rn(p1, s[i]));
                    x[8 + i] = __fadd_rn(__fmul_rn(p1, c[i]), __fmul_rn(p0, s[i]));
                }
            }
        }
        if (live && is_q) {
            uint16_t* dst = a.q_out + t * a.q_out_stride + static_cast<int64_t>(h) * kDim;
            *reinterpret_cast<uint4*>(dst + e0) = pack8(x);
            *reinterpret_cast<uint4*>(dst + e1) = pack8(x + 8);
        }
        if constexpr (INT8) {
            if (__all_sync(0xffffffffu, !live || is_q)) return;
            float amax = 0.0f;
            if (live && !is_q) {
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(x[i]));
            }
#pragma unroll
            for (int o = 1; o < UPH; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (live && !is_q && slot >= 0) {
                const float scale = __fdiv_rn(max_nan(amax, 1e-30f), 127.0f);
                const int hk = is_v ? h - a.n_q - n_kv : h - a.n_q;
                const int64_t vec = ((page * n_kv + hk) << a.cache.page_shift) + place;
                if (bd_in(kBkRope, vec, slots * n_kv)) {
                    uint8_t* dst = static_cast<uint8_t*>(is_v ? a.cache.v : a.cache.k) + vec * kDim;
                    *reinterpret_cast<uint2*>(dst + e0) = codes8(x, scale);
                    *reinterpret_cast<uint2*>(dst + e1) = codes8(x + 8, scale);
                    if (u == 0) (is_v ? a.cache.v_scale : a.cache.k_scale)[vec] = scale;
                }
            }
        } else if (live && !is_q && slot >= 0) {
            const int hk = is_v ? h - a.n_q - n_kv : h - a.n_q;
            const int64_t vec = ((page * n_kv + hk) << a.cache.page_shift) + place;
            if (bd_in(kBkRope, vec, slots * n_kv)) {
                uint16_t* dst = static_cast<uint16_t*>(is_v ? a.cache.v : a.cache.k) + vec * kDim;
                *reinterpret_cast<uint4*>(dst + e0) = pack8(x);
                *reinterpret_cast<uint4*>(dst + e1) = pack8(x + 8);
            }
        }
    };
    for (int h0 = blockIdx.y * per_pass; h0 < heads; h0 += kAhead * step) {
        const int h = h0 + threadIdx.x / UPH;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (h0 + i * step >= heads) break;
            const uint4 now[2] = {raw[i][0], raw[i][1]};
            load(h + (i + kAhead) * step, raw[i]);
            work(h + i * step, now);
        }
    }
}

// ------------------------------------------------------------------------------- read

constexpr int kReadThreads = 256;
constexpr int kReadRows = 8;  // output rows of a block

struct KvReadParams {
    KvReadArgs a;
};

// A block gathers kReadRows consecutive output rows: their places in the
// cache are looked up first (a binary search in kv_off per row), then all
// threads copy units of 16 elements, two at a time: 8 sequences of up to 8192
// int8 tokens, 8 heads of 128, in 48.4 us, 6.1 TB/s (51.6 one at a time); bf16
// 59.4 us, 6.6 TB/s, by whole sectors (62.5 by halves of 16 bytes).
template <int UPH, bool INT8>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const __grid_constant__ KvReadParams p)
{
    constexpr int kDim = UPH * kUnit;
    __shared__ int64_t base[kReadRows];  // page * n_kv * page + place of the token; -1: zeros, -2: leave the row
    const KvReadArgs& a = p.a;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kReadRows;

    grid_launch_dependents();
    grid_dependency_wait();

    if (threadIdx.x < kReadRows) {
        const int64_t r = row0 + threadIdx.x;
        int64_t b = -2;
        if (r < a.rows && r < a.kv_off[a.n_seq]) {
            int64_t lo = 0, hi = a.n_seq;  // the last s with kv_off[s] <= r
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (a.kv_off[mid] <= r) lo = mid;
                else hi = mid;
            }
            const int64_t j = r - a.kv_off[lo];
            b = -1;
            const int64_t at = j >> a.cache.page_shift;
            if (j >= 0 && at < a.max_pages) {
                const int64_t pg = a.table[lo * a.max_pages + at];
                if (pg >= 0 && pg < a.cache.n_pages)
                    b = ((pg * a.cache.n_kv) << a.cache.page_shift) + (j & (a.cache.page - 1));
            }
            if (b < 0) raise_error(a.err, kErrBadIndex);
        }
        base[threadIdx.x] = b;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x >= 32) {
        // offsets out of order, or tokens that there are no rows for (by the warps that have nothing to look up)
        bool bad = false;
        for (int64_t s = threadIdx.x - 32; s < a.n_seq; s += kReadThreads - 32) {
            const int32_t o = a.kv_off[s], e = a.kv_off[s + 1];
            bad = bad || e < o || (s == 0 && o != 0) || e > a.rows;
        }
        if (bad) raise_error(a.err, kErrBadIndex);
    }
    __syncthreads();

    const int per_row = a.cache.n_kv * UPH;  // units of one row of k (or v)
    const int64_t vecs = (a.cache.n_pages * a.cache.n_kv) << a.cache.page_shift;
    const bool is_v = blockIdx.y != 0;
    const void* pool = is_v ? a.cache.v : a.cache.k;
    const float* scales = is_v ? a.cache.v_scale : a.cache.k_scale;
    uint16_t* out = is_v ? a.v_out : a.k_out;
    // (int8 has no registers to spare for eight at once: 50.5 us for 48.4)
    [[maybe_unused]] const bool sectors = on_sector(pool) && on_sector(out);
    // two units at a time: both loads before either is converted
    const int units = kReadRows * per_row;
    for (int i0 = threadIdx.x; i0 < units; i0 += 2 * kReadThreads) {
        uint4 lo[2], hi[2];
        float scale[2];
        int64_t to[2];  // of the output, or -1
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = i0 + k * kReadThreads;
            const int r = i / per_row, j = i - r * per_row;
            const int64_t b = i < units ? base[r] : -2;
            const int h = j / UPH, u = j % UPH;
            to[k] = b == -2 ? -1 : ((row0 + r) * a.cache.n_kv + h) * kDim + 16 * u;
            lo[k] = hi[k] = make_uint4(0, 0, 0, 0);
            scale[k] = 0.0f;
            const int64_t vec = b + (static_cast<int64_t>(h) << a.cache.page_shift);
            if (b >= 0 && bd_in(kBkKvRead, vec, vecs)) {
                if constexpr (INT8) {
                    lo[k] = ld_stream_v4(static_cast<const uint8_t*>(pool) + vec * kDim + 16 * u);
                    scale[k] = __ldg(scales + vec);
                } else {
                    const uint16_t* src = static_cast<const uint16_t*>(pool) + vec * kDim + 16 * u;
                    if (sectors) {
                        load_32(src, lo[k], hi[k]);
                    } else {
                        lo[k] = ld_stream_v4(src);
                        hi[k] = ld_stream_v4(src + 8);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (to[k] < 0 || !bd_in_range(kBkKvRead, to[k], 16, a.rows * a.cache.n_kv * kDim)) continue;
            if constexpr (INT8) {
                const uint32_t ww[4] = {lo[k].x, lo[k].y, lo[k].z, lo[k].w};
                float f[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    f[e] = static_cast<float>(static_cast<int8_t>(ww[e / 4] >> (8 * (e % 4)))) * scale[k];
                lo[k] = pack8(f);
                hi[k] = pack8(f + 8);
            }
            uint16_t* dst = out + to[k];
            if (!INT8 && sectors) {
                store_32(dst, lo[k], hi[k]);
            } else {
                *reinterpret_cast<uint4*>(dst) = lo[k];
                *reinterpret_cast<uint4*>(dst + 8) = hi[k];
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, int sm_count, cudaStream_t stream)
{
    if (a.T == 0) return cudaSuccess;
    RopeParams p{a};
    // as few passes as so many threads allow, all about equally full
    const int uph = a.cache.dim / kUnit, heads = a.n_q + 2 * a.cache.n_kv;
    const int most = rope_threads(a.cache.int8) / uph;
    const int passes = (heads + most - 1) / most, per_pass = (heads + passes - 1) / passes;
    const int threads = (per_pass * uph + 31) / 32 * 32;
    // few tokens: the passes of a token are split over blocks until the GPU has about 8 blocks per SM
    const int real = (heads + threads / uph - 1) / (threads / uph);
    int64_t split = (8ll * sm_count + a.T - 1) / a.T;
    if (split > real) split = real;
    if (split < 1) split = 1;
    const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(split));
    cudaError_t err = cudaSuccess;
    if (a.cache.dim == 128)
        launch_dep(err, a.cache.int8 ? rope_append_kernel<8, true> : rope_append_kernel<8, false>, grid,
                   dim3(threads), 0, stream, p);
    else
        launch_dep(err, a.cache.int8 ? rope_append_kernel<4, true> : rope_append_kernel<4, false>, grid,
                   dim3(threads), 0, stream, p);
    return err;
}

cudaError_t launch_kv_read(const KvReadArgs& a, int /*sm_count*/, cudaStream_t stream)
{
    if (a.rows == 0) return cudaSuccess;
    KvReadParams p{a};
    const dim3 grid(static_cast<unsigned>((a.rows + kReadRows - 1) / kReadRows), 2);
    cudaError_t err = cudaSuccess;
    if (a.cache.dim == 128)
        launch_dep(err, a.cache.int8 ? kv_read_kernel<8, true> : kv_read_kernel<8, false>, grid, dim3(kReadThreads),
                   0, stream, p);
    else
        launch_dep(err, a.cache.int8 ? kv_read_kernel<4, true> : kv_read_kernel<4, false>, grid, dim3(kReadThreads),
                   0, stream, p);
    return err;
}

BD_BOUNDS_TAKE(bounds_take_kv)

}  // namespace bd
