// C ABI of libbitdelta.so: argument checks, workspace layout and dispatch to
// the sm_103a kernels.  Every entry point is declared and documented in
// include/bitdelta.h.
#include <atomic>
#include <cstring>

#include "../../include/bitdelta.h"
#include "bd_internal.h"

namespace {

constexpr int kVersion = 10000;  // 1.0.0
constexpr size_t kWsHeader = 256;  // error word + padding; scratch starts here

// The calling thread's last failed CUDA result (bd_last_cuda_error).
thread_local int g_last_cuda_error = 0;

// Per-device cache of (compute capability, SM count).
constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_cc[kMaxDevices];
std::atomic<int> g_dev_sms[kMaxDevices];

bd_status device_info(int* sm_count)
{
    int dev = 0;
    if (const int cs_ = bd::cuda_status(cudaGetDevice(&dev))) return static_cast<bd_status>(cs_);
    if (dev < 0 || dev >= kMaxDevices) return BD_ERR_DEVICE;
    int cc = g_dev_cc[dev].load(std::memory_order_acquire);
    if (cc == 0) {
        int major = 0, minor = 0, sms = 0;
        cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return static_cast<bd_status>(bd::cuda_status(e));
        cc = major * 10 + minor;
        g_dev_sms[dev].store(sms, std::memory_order_relaxed);
        g_dev_cc[dev].store(cc, std::memory_order_release);
    }
    if (cc != 103) return BD_ERR_DEVICE;
    *sm_count = g_dev_sms[dev].load(std::memory_order_relaxed);
    return BD_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

bd_status check_d_in(int64_t d_in) { return (d_in > 0 && d_in % 128 == 0) ? BD_OK : BD_ERR_UNSUPPORTED_SHAPE; }

bd_status check_ws(const void* ws, size_t ws_bytes, size_t need)
{
    if (!ws || ws_bytes < need) return BD_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return BD_ERR_MISALIGNED;
    return BD_OK;
}

bd_status launched(cudaError_t e) { return static_cast<bd_status>(bd::cuda_status(e)); }

uint32_t* err_word(void* ws) { return static_cast<uint32_t*>(ws); }

}  // namespace

int bd::cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return BD_OK;
    g_last_cuda_error = static_cast<int>(e);
    return BD_ERR_CUDA;
}

extern "C" {

int bd_version(void) { return kVersion; }

int bd_last_cuda_error(void) { return g_last_cuda_error; }

const char* bd_cuda_error_string(int code)
{
    const char* name = cudaGetErrorName(static_cast<cudaError_t>(code));
    return name ? name : "unknown CUDA error";
}

const char* bd_status_string(bd_status s)
{
    switch (s) {
        case BD_OK: return "BD_OK";
        case BD_ERR_INVALID_ARG: return "BD_ERR_INVALID_ARG: invalid argument";
        case BD_ERR_UNSUPPORTED_SHAPE: return "BD_ERR_UNSUPPORTED_SHAPE: d_in must be a positive multiple of 128";
        case BD_ERR_MISALIGNED: return "BD_ERR_MISALIGNED: pointer alignment rule broken";
        case BD_ERR_BAD_VARIANT: return "BD_ERR_BAD_VARIANT: variant id outside [-1, V)";
        case BD_ERR_NONFINITE: return "BD_ERR_NONFINITE: non-finite delta in compression";
        case BD_ERR_CUDA: return "BD_ERR_CUDA: CUDA runtime error";
        case BD_ERR_TIMEOUT: return "BD_ERR_TIMEOUT: an in-kernel wait timed out";
        case BD_ERR_WORKSPACE: return "BD_ERR_WORKSPACE: workspace missing or too small";
        case BD_ERR_DEVICE: return "BD_ERR_DEVICE: current device is not compute capability 10.3";
        case BD_ERR_BOUNDS: return "BD_ERR_BOUNDS: a kernel met an index outside its buffer (bounds-checked build)";
        case BD_ERR_BAD_INDEX:
            return "BD_ERR_BAD_INDEX: a position, slot, page, length or offset outside its range";
    }
    return "BD_ERR_UNKNOWN";
}

// ------------------------------------------------------------------ compress

size_t bd_compress_workspace_size(int64_t d_out, int64_t /*d_in*/, int alpha_mode)
{
    if (d_out < 0) return 0;
    size_t n = kWsHeader;
    if (alpha_mode == BD_ALPHA_PER_MATRIX) {
        const size_t ctas = static_cast<size_t>((d_out + bd::kCompressRowsPerCta - 1) / bd::kCompressRowsPerCta);
        n += ctas * sizeof(double);
    }
    return (n + 255) & ~static_cast<size_t>(255);
}

bd_status bd_compress(const uint16_t* w_base, const uint16_t* w_ft, int64_t d_out, int64_t d_in, int alpha_mode,
                      uint32_t* signs, float* alpha, void* ws, size_t ws_bytes, void* stream)
{
    BD_NVTX_RANGE("bd_compress");
    if (alpha_mode != BD_ALPHA_PER_MATRIX && alpha_mode != BD_ALPHA_PER_ROW) return BD_ERR_INVALID_ARG;
    if (d_out < 0) return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_d_in(d_in)) return s;
    if (bd_status s = check_ws(ws, ws_bytes, bd_compress_workspace_size(d_out, d_in, alpha_mode))) return s;
    if (d_out == 0) return BD_OK;
    if (!w_base || !w_ft || !signs || !alpha) return BD_ERR_INVALID_ARG;
    if (!aligned(w_base, 16) || !aligned(w_ft, 16) || !aligned(signs, 16) || !aligned(alpha, 4))
        return BD_ERR_MISALIGNED;
    const size_t wbytes = static_cast<size_t>(d_out) * d_in * 2;
    const size_t sbytes = static_cast<size_t>(d_out) * (d_in / 8);
    const size_t abytes = (alpha_mode == BD_ALPHA_PER_ROW ? static_cast<size_t>(d_out) : 1u) * 4;
    if (overlaps(signs, sbytes, w_base, wbytes) || overlaps(signs, sbytes, w_ft, wbytes) ||
        overlaps(alpha, abytes, w_base, wbytes) || overlaps(alpha, abytes, w_ft, wbytes) ||
        overlaps(signs, sbytes, alpha, abytes) || overlaps(ws, ws_bytes, signs, sbytes) ||
        overlaps(ws, ws_bytes, alpha, abytes))
        return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    auto* partials = reinterpret_cast<double*>(static_cast<char*>(ws) + kWsHeader);
    return launched(bd::launch_compress(w_base, w_ft, d_out, d_in, alpha_mode == BD_ALPHA_PER_ROW, signs, alpha,
                                        partials, err_word(ws), static_cast<cudaStream_t>(stream)));
}

bd_status bd_debug_reconstruct(const uint16_t* w_base, const uint32_t* signs, const float* alpha, int alpha_mode,
                               int64_t d_out, int64_t d_in, float* w_eff, void* stream)
{
    BD_NVTX_RANGE("bd_debug_reconstruct");
    if (alpha_mode != BD_ALPHA_PER_MATRIX && alpha_mode != BD_ALPHA_PER_ROW) return BD_ERR_INVALID_ARG;
    if (d_out < 0) return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_d_in(d_in)) return s;
    if (d_out == 0) return BD_OK;
    if (!w_base || !signs || !alpha || !w_eff) return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    return launched(bd::launch_debug_reconstruct(w_base, signs, alpha, alpha_mode == BD_ALPHA_PER_ROW, d_out, d_in,
                                                 w_eff, static_cast<cudaStream_t>(stream)));
}

bd_status bd_materialize(const uint16_t* w_base, const uint32_t* signs, const float* alpha, int alpha_mode,
                         int64_t d_out, int64_t d_in, uint16_t* w_eff, void* stream)
{
    BD_NVTX_RANGE("bd_materialize");
    if (alpha_mode != BD_ALPHA_PER_MATRIX && alpha_mode != BD_ALPHA_PER_ROW) return BD_ERR_INVALID_ARG;
    if (d_out < 0) return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_d_in(d_in)) return s;
    if (d_out == 0) return BD_OK;
    if (!w_base || !signs || !alpha || !w_eff) return BD_ERR_INVALID_ARG;
    if (!aligned(w_base, 16) || !aligned(w_eff, 16) || !aligned(signs, 4) || !aligned(alpha, 4))
        return BD_ERR_MISALIGNED;
    const size_t wbytes = static_cast<size_t>(d_out) * static_cast<size_t>(d_in) * 2;
    const size_t abytes = (alpha_mode == BD_ALPHA_PER_ROW ? static_cast<size_t>(d_out) : 1u) * 4;
    if (overlaps(w_eff, wbytes, w_base, wbytes) || overlaps(w_eff, wbytes, signs, wbytes / 16) ||
        overlaps(w_eff, wbytes, alpha, abytes))
        return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    return launched(bd::launch_materialize(w_base, signs, alpha, alpha_mode == BD_ALPHA_PER_ROW, d_out, d_in, w_eff,
                                           sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ MonoSoup merge

size_t bd_monosoup_workspace_size(int64_t d_out, int64_t d_in, int32_t k, int32_t rank, int32_t l)
{
    if (d_out < 0 || d_in < 0 || k < 1 || rank < 0 || l < 1) return 0;
    return bd::monosoup_workspace_size(d_out, d_in, k, rank, l);
}

bd_status bd_monosoup_merge(const uint16_t* w_base, const uint16_t* const* w_ft, int32_t k, int64_t d_out,
                            int64_t d_in, int32_t rank, int32_t l, int32_t power_iters, const float* omega,
                            void* w_merged, int out_dtype, void* ws, size_t ws_bytes, void* stream)
{
    BD_NVTX_RANGE("bd_monosoup_merge");
    if (out_dtype != BD_OUT_BF16 && out_dtype != BD_OUT_F32) return BD_ERR_INVALID_ARG;
    if (k < 1 || k > BD_MAX_VARIANTS || rank < 0 || l < 4 || l > bd::monosoup_max_l() || l % 4 != 0 || rank > l ||
        power_iters < 0 || power_iters > 16)
        return BD_ERR_INVALID_ARG;
    if (d_out < 0) return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_d_in(d_in)) return s;
    if (d_out == 0) return BD_OK;
    if (!w_base || !w_ft || !w_merged || (rank > 0 && !omega)) return BD_ERR_INVALID_ARG;
    const size_t wbytes = static_cast<size_t>(d_out) * static_cast<size_t>(d_in) * 2;
    const size_t obytes = wbytes * (out_dtype == BD_OUT_F32 ? 2 : 1);
    if (!aligned(w_base, 16) || !aligned(w_merged, 16) || (omega && !aligned(omega, 16))) return BD_ERR_MISALIGNED;
    if (overlaps(w_merged, obytes, w_base, wbytes)) return BD_ERR_INVALID_ARG;
    for (int32_t i = 0; i < k; ++i) {
        if (!w_ft[i]) return BD_ERR_INVALID_ARG;
        if (!aligned(w_ft[i], 16)) return BD_ERR_MISALIGNED;
        if (overlaps(w_merged, obytes, w_ft[i], wbytes)) return BD_ERR_INVALID_ARG;
    }
    if (omega && overlaps(w_merged, obytes, omega, static_cast<size_t>(d_in) * l * 4)) return BD_ERR_INVALID_ARG;
    if (bd_status s = check_ws(ws, ws_bytes, bd::monosoup_workspace_size(d_out, d_in, k, rank, l))) return s;
    if (overlaps(ws, ws_bytes, w_merged, obytes)) return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    bd::MonoSoupArgs a{};
    a.w_base = w_base;
    a.w_ft = w_ft;
    a.k = k;
    a.d_out = d_out;
    a.d_in = d_in;
    a.rank = rank;
    a.l = l;
    a.power_iters = power_iters;
    a.omega = omega;
    a.out = w_merged;
    a.out_f32 = out_dtype == BD_OUT_F32;
    a.ws = ws;
    a.err = err_word(ws);
    a.sm_count = sms;
    return launched(bd::launch_monosoup(a, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ linear

size_t bd_linear_workspace_size(int64_t /*T*/, int64_t /*d_out*/, int64_t /*d_in*/) { return kWsHeader; }

static bd_status check_linear_common(const uint16_t* x, int64_t T, const uint16_t* w_base, int64_t d_out,
                                     int64_t d_in, void* y, int out_dtype, void* ws, size_t ws_bytes, size_t ws_need)
{
    if (out_dtype != BD_OUT_BF16 && out_dtype != BD_OUT_F32) return BD_ERR_INVALID_ARG;
    if (T < 0 || d_out < 0) return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_d_in(d_in)) return s;
    if (bd_status s = check_ws(ws, ws_bytes, ws_need)) return s;
    if (T == 0 || d_out == 0) return BD_OK;
    if (!x || !w_base || !y) return BD_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w_base, 16) || !aligned(y, 16)) return BD_ERR_MISALIGNED;
    const size_t ybytes = static_cast<size_t>(T) * d_out * (out_dtype == BD_OUT_F32 ? 4 : 2);
    if (overlaps(y, ybytes, x, static_cast<size_t>(T) * d_in * 2) ||
        overlaps(y, ybytes, w_base, static_cast<size_t>(d_out) * d_in * 2) || overlaps(y, ybytes, ws, ws_bytes))
        return BD_ERR_INVALID_ARG;
    return BD_OK;
}

bd_status bd_linear(const uint16_t* x, int64_t T, const uint16_t* w_base, const uint32_t* signs, const float* alpha,
                    int alpha_mode, int64_t d_out, int64_t d_in, void* y, int out_dtype, void* ws, size_t ws_bytes,
                    void* stream)
{
    BD_NVTX_RANGE("bd_linear");
    if (alpha_mode != BD_ALPHA_PER_MATRIX && alpha_mode != BD_ALPHA_PER_ROW) return BD_ERR_INVALID_ARG;
    if (bd_status s = check_linear_common(x, T, w_base, d_out, d_in, y, out_dtype, ws, ws_bytes,
                                          bd_linear_workspace_size(T, d_out, d_in)))
        return s;
    if (T == 0 || d_out == 0) return BD_OK;
    if (!signs || !alpha) return BD_ERR_INVALID_ARG;
    if (!aligned(signs, 16) || !aligned(alpha, 4)) return BD_ERR_MISALIGNED;
    const size_t ybytes = static_cast<size_t>(T) * d_out * (out_dtype == BD_OUT_F32 ? 4 : 2);
    const size_t abytes = (alpha_mode == BD_ALPHA_PER_ROW ? static_cast<size_t>(d_out) : 1u) * 4;
    if (overlaps(y, ybytes, signs, static_cast<size_t>(d_out) * (d_in / 8)) || overlaps(y, ybytes, alpha, abytes))
        return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t ysz = out_dtype == BD_OUT_F32 ? 4 : 2;

    if (T > bd::kSkinnyMaxTokens && bd::prefill_available()) {
        bd::PrefillArgs p{};
        p.x = x; p.w_base = w_base; p.signs = signs; p.alpha = alpha;
        p.per_row = alpha_mode == BD_ALPHA_PER_ROW;
        p.T = T; p.d_out = d_out; p.d_in = d_in; p.y = y; p.out_f32 = out_dtype == BD_OUT_F32;
        p.err = err_word(ws);
        return launched(bd::launch_prefill(p, sms, st));
    }
    // decode kernel over groups of up to 64 tokens
    for (int64_t t0 = 0; t0 < T; t0 += bd::kSkinnyMaxTokens) {
        bd::SkinnyArgs a{};
        a.x = x + t0 * d_in;
        a.w_base = w_base;
        a.signs = signs;
        a.alpha = alpha;
        a.T = (T - t0) < bd::kSkinnyMaxTokens ? (T - t0) : bd::kSkinnyMaxTokens;
        a.d_out = d_out; a.d_in = d_in;
        a.per_row = alpha_mode == BD_ALPHA_PER_ROW;
        a.y = static_cast<char*>(y) + static_cast<size_t>(t0) * d_out * ysz;
        a.out_f32 = out_dtype == BD_OUT_F32;
        a.err = err_word(ws);
        if (bd_status s = launched(bd::launch_skinny(a, st))) return s;
    }
    return BD_OK;
}

// Multi-variant workspace for one group of up to 64 tokens: the error word,
// then (at 1 KiB) the zero-padded per-variant x tiles of the sign phases and
// the per-token partial corrections.
namespace {

struct MultiWs {
    size_t xp, corr, total;
};

MultiWs multi_ws_layout(int64_t T, int32_t V, int64_t d_in)
{
    const int64_t group = bd::multi_group_tokens(V);
    const int64_t tg = T < group ? T : group;
    const auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    MultiWs w{};
    w.xp = 1024;
    const size_t ptiles = static_cast<size_t>(bd::multi_max_ptiles(static_cast<int>(tg), V));
    w.corr = w.xp + up(ptiles * 8 * static_cast<size_t>(d_in) * 2);
    w.total = w.corr + up(static_cast<size_t>(tg) * static_cast<size_t>(bd::multi_corr_splits(d_in)) * 4);
    return w;
}

// From this many tokens on, bd_linear_multi runs the grouped tensor-core
// prefill (one 256-token block per variant segment piece) instead of the
// decode kernel on 64-token groups: at 512 tokens over 14 variants the plan
// has at most 17 blocks per row block against 8 decode groups that each
// re-read W_base.
constexpr int64_t kMultiPrefillMinT = 512;

bool use_grouped_prefill(int64_t T) { return T >= kMultiPrefillMinT && bd::prefill_available(); }

// Grouped prefill workspace: the error word, then the router's perm [T] and
// seg_off [V + 2], the block plan and x in sorted order [T][d_in].
struct GroupedWs {
    size_t perm, seg, plan, xs, total;
};

GroupedWs grouped_ws_layout(int64_t T, int32_t V, int64_t d_in)
{
    const auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    GroupedWs w{};
    w.perm = 1024;
    w.seg = w.perm + up(static_cast<size_t>(T) * 4);
    w.plan = w.seg + up(static_cast<size_t>(V + 2) * 4);
    w.xs = w.plan + up(static_cast<size_t>(bd::grouped_prefill_blocks(T, V)) * 16);
    w.total = w.xs + up(static_cast<size_t>(T) * static_cast<size_t>(d_in) * 2);
    return w;
}

}  // namespace

size_t bd_linear_multi_workspace_size(int64_t T, int32_t V, int64_t /*d_out*/, int64_t d_in)
{
    if (T < 0 || d_in < 0 || V < 1 || V > BD_MAX_VARIANTS) return kWsHeader;
    if (use_grouped_prefill(T)) return grouped_ws_layout(T, V, d_in).total;
    return multi_ws_layout(T, V, d_in).total;
}

bd_status bd_linear_multi(const uint16_t* x, int64_t T, const int32_t* vid, int32_t V,
                          const uint32_t* const* signs_tab, const float* const* alpha_tab, int alpha_mode,
                          const uint16_t* w_base, int64_t d_out, int64_t d_in, void* y, int out_dtype, void* ws,
                          size_t ws_bytes, void* stream)
{
    BD_NVTX_RANGE("bd_linear_multi");
    if (alpha_mode != BD_ALPHA_PER_MATRIX && alpha_mode != BD_ALPHA_PER_ROW) return BD_ERR_INVALID_ARG;
    if (V < 1 || V > BD_MAX_VARIANTS) return BD_ERR_INVALID_ARG;
    if (bd_status s = check_linear_common(x, T, w_base, d_out, d_in, y, out_dtype, ws, ws_bytes,
                                          bd_linear_multi_workspace_size(T, V, d_out, d_in)))
        return s;
    if (T == 0 || d_out == 0) return BD_OK;
    if (!vid || !signs_tab || !alpha_tab) return BD_ERR_INVALID_ARG;
    if (!aligned(vid, 4)) return BD_ERR_MISALIGNED;
    const size_t ybytes = static_cast<size_t>(T) * d_out * (out_dtype == BD_OUT_F32 ? 4 : 2);
    const size_t abytes = (alpha_mode == BD_ALPHA_PER_ROW ? static_cast<size_t>(d_out) : 1u) * 4;
    for (int v = 0; v < V; ++v) {
        if (!signs_tab[v] || !alpha_tab[v]) return BD_ERR_INVALID_ARG;
        if (!aligned(signs_tab[v], 16) || !aligned(alpha_tab[v], 4)) return BD_ERR_MISALIGNED;
        if (overlaps(y, ybytes, signs_tab[v], static_cast<size_t>(d_out) * (d_in / 8)) ||
            overlaps(y, ybytes, alpha_tab[v], abytes))
            return BD_ERR_INVALID_ARG;
    }
    if (overlaps(y, ybytes, vid, static_cast<size_t>(T) * 4)) return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (use_grouped_prefill(T)) {
        if (T > INT32_MAX) return BD_ERR_UNSUPPORTED_SHAPE;
        const GroupedWs lay = grouped_ws_layout(T, V, d_in);
        char* w = static_cast<char*>(ws);
        bd::GroupedPrefillArgs g{};
        g.x = x;
        g.perm = reinterpret_cast<int32_t*>(w + lay.perm);
        g.seg_off = reinterpret_cast<int32_t*>(w + lay.seg);
        g.w_base = w_base;
        for (int v = 0; v < V; ++v) {
            g.signs[v] = signs_tab[v];
            g.alpha[v] = alpha_tab[v];
        }
        g.V = V;
        g.per_row = alpha_mode == BD_ALPHA_PER_ROW;
        g.T = T;
        g.d_out = d_out;
        g.d_in = d_in;
        g.y = y;
        g.out_f32 = out_dtype == BD_OUT_F32;
        g.err = err_word(ws);
        g.xs = reinterpret_cast<uint16_t*>(w + lay.xs);
        g.plan = reinterpret_cast<int4*>(w + lay.plan);
        if (bd_status s = launched(bd::launch_route(vid, T, V, reinterpret_cast<int32_t*>(w + lay.perm),
                                                    reinterpret_cast<int32_t*>(w + lay.seg), g.err, st)))
            return s;
        return launched(bd::launch_prefill_grouped(g, st));
    }
    const size_t ysz = out_dtype == BD_OUT_F32 ? 4 : 2;
    const int64_t group = bd::multi_group_tokens(V);
    const MultiWs lay = multi_ws_layout(T, V, d_in);
    for (int64_t t0 = 0; t0 < T; t0 += group) {
        bd::MultiArgs a{};
        a.x = x + t0 * d_in;
        a.vid = vid + t0;
        a.w_base = w_base;
        a.T = (T - t0) < group ? (T - t0) : group;
        a.d_out = d_out; a.d_in = d_in; a.V = V;
        a.per_row = alpha_mode == BD_ALPHA_PER_ROW;
        for (int v = 0; v < V; ++v) {
            a.signs[v] = signs_tab[v];
            a.alpha[v] = alpha_tab[v];
        }
        a.y = static_cast<char*>(y) + static_cast<size_t>(t0) * d_out * ysz;
        a.out_f32 = out_dtype == BD_OUT_F32;
        a.err = err_word(ws);
        a.xp = reinterpret_cast<uint8_t*>(static_cast<char*>(ws) + lay.xp);
        a.corr = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.corr);
        if (bd_status s = launched(bd::launch_multi(a, st))) return s;
    }
    return BD_OK;
}

// ------------------------------------------------------------------ router

size_t bd_route_workspace_size(int64_t /*T*/, int32_t /*V*/) { return kWsHeader; }

bd_status bd_route(const int32_t* vid, int64_t T, int32_t V, int32_t* perm, int32_t* seg_off, void* ws,
                   size_t ws_bytes, void* stream)
{
    BD_NVTX_RANGE("bd_route");
    if (V < 0 || V > BD_MAX_VARIANTS) return BD_ERR_INVALID_ARG;
    if (T < 0 || T > INT32_MAX) return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_ws(ws, ws_bytes, bd_route_workspace_size(T, V))) return s;
    if (!seg_off || (T > 0 && (!vid || !perm))) return BD_ERR_INVALID_ARG;
    if (!aligned(seg_off, 4) || (T > 0 && (!aligned(vid, 4) || !aligned(perm, 4)))) return BD_ERR_MISALIGNED;
    if (overlaps(perm, static_cast<size_t>(T) * 4, vid, static_cast<size_t>(T) * 4) ||
        overlaps(seg_off, static_cast<size_t>(V + 2) * 4, vid, static_cast<size_t>(T) * 4) ||
        overlaps(seg_off, static_cast<size_t>(V + 2) * 4, perm, static_cast<size_t>(T) * 4))
        return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    return launched(bd::launch_route(vid, T, V, perm, seg_off, err_word(ws), static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ norm

size_t bd_rms_norm_workspace_size(int64_t /*T*/, int64_t /*d*/) { return kWsHeader; }

bd_status bd_rms_norm(const uint16_t* x, const uint16_t* residual, int64_t T, int64_t d, const uint16_t* gain,
                      const int32_t* vid, int32_t V, const uint16_t* const* gain_tab, float eps,
                      uint16_t* residual_out, void* out, int out_dtype, float* scale, void* ws, size_t ws_bytes,
                      void* stream)
{
    BD_NVTX_RANGE("bd_rms_norm");
    if (out_dtype != BD_OUT_BF16 && out_dtype != BD_OUT_F32 && out_dtype != BD_OUT_E4M3) return BD_ERR_INVALID_ARG;
    if (V < 0 || V > BD_MAX_VARIANTS || !(eps >= 0.0f)) return BD_ERR_INVALID_ARG;
    if (T < 0 || T > INT32_MAX || d <= 0 || d % 8 != 0) return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_ws(ws, ws_bytes, bd_rms_norm_workspace_size(T, d))) return s;
    if (T == 0) return BD_OK;
    if (!x || !gain || !out || (out_dtype == BD_OUT_E4M3) != (scale != nullptr)) return BD_ERR_INVALID_ARG;
    if (vid && V > 0 && !gain_tab) return BD_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(gain, 16) ||
        !aligned(out, 16) || !aligned(vid, 4) || !aligned(scale, 4))
        return BD_ERR_MISALIGNED;
    const size_t n = static_cast<size_t>(T) * static_cast<size_t>(d), g = static_cast<size_t>(d) * 2;
    const size_t obytes = n * (out_dtype == BD_OUT_F32 ? 4 : out_dtype == BD_OUT_BF16 ? 2 : 1);
    const size_t tbytes = static_cast<size_t>(T) * 4;
    const auto written_over = [&](const void* in, size_t bytes) {  // by an output other than residual_out
        return overlaps(out, obytes, in, bytes) || overlaps(scale, tbytes, in, bytes);
    };
    if (written_over(x, n * 2) || written_over(residual, n * 2) || written_over(residual_out, n * 2) ||
        written_over(gain, g) || written_over(vid, tbytes) || written_over(ws, ws_bytes) ||
        overlaps(out, obytes, scale, tbytes) || overlaps(residual_out, n * 2, gain, g) ||
        overlaps(residual_out, n * 2, vid, tbytes) || overlaps(residual_out, n * 2, ws, ws_bytes) ||
        (residual_out != x && overlaps(residual_out, n * 2, x, n * 2)) ||
        (residual_out != residual && overlaps(residual_out, n * 2, residual, n * 2)))
        return BD_ERR_INVALID_ARG;
    bd::NormArgs a{};
    if (vid) {
        for (int32_t v = 0; v < V; ++v) {
            if (!gain_tab[v]) return BD_ERR_INVALID_ARG;
            if (!aligned(gain_tab[v], 16)) return BD_ERR_MISALIGNED;
            if (written_over(gain_tab[v], g) || overlaps(residual_out, n * 2, gain_tab[v], g))
                return BD_ERR_INVALID_ARG;
            a.gains[v] = gain_tab[v];
        }
    }
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    a.x = x;
    a.residual = residual;
    a.residual_out = residual_out;
    a.gain = gain;
    a.vid = vid;
    a.V = V;
    a.T = T;
    a.d = d;
    a.eps = eps;
    a.out = out;
    a.out_dtype = out_dtype;
    a.scale = scale;
    a.err = err_word(ws);
    return launched(bd::launch_rms_norm(a, sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ norms around a block

size_t bd_block_norm_workspace_size(int64_t /*T*/, int64_t /*d*/) { return kWsHeader; }

bd_status bd_block_norm(const uint16_t* x, const uint16_t* residual, int64_t T, int64_t d, const uint16_t* post_gain,
                        const uint16_t* const* post_gain_tab, const uint16_t* gate, int64_t gate_rows,
                        const int32_t* gate_idx, float block_scale, float residual_scale, const uint16_t* gain,
                        const uint16_t* const* gain_tab, const int32_t* vid, int32_t V, float eps,
                        uint16_t* residual_out, void* out, int out_dtype, float* scale, void* ws, size_t ws_bytes,
                        void* stream)
{
    BD_NVTX_RANGE("bd_block_norm");
    if (out_dtype != BD_OUT_BF16 && out_dtype != BD_OUT_F32 && out_dtype != BD_OUT_E4M3) return BD_ERR_INVALID_ARG;
    if (V < 0 || V > BD_MAX_VARIANTS || !(eps >= 0.0f)) return BD_ERR_INVALID_ARG;
    if (!(block_scale - block_scale == 0.0f) || !(residual_scale - residual_scale == 0.0f))
        return BD_ERR_INVALID_ARG;  // not finite
    if (T < 0 || T > INT32_MAX || d <= 0 || d % 8 != 0 || gate_rows < 0 || gate_rows > INT32_MAX)
        return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_ws(ws, ws_bytes, bd_block_norm_workspace_size(T, d))) return s;
    if (T == 0) return BD_OK;
    if (!x || !residual || !gain || !out || (out_dtype == BD_OUT_E4M3) != (scale != nullptr)) return BD_ERR_INVALID_ARG;
    if (vid && V > 0 && (!gain_tab || (post_gain && !post_gain_tab))) return BD_ERR_INVALID_ARG;
    // without gate_idx: one gate for all tokens, or each token's own
    if (gate ? gate_rows < 1 || (!gate_idx && gate_rows != 1 && gate_rows != T) : gate_idx != nullptr)
        return BD_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(gain, 16) ||
        !aligned(post_gain, 16) || !aligned(gate, 16) || !aligned(gate_idx, 4) || !aligned(out, 16) ||
        !aligned(vid, 4) || !aligned(scale, 4))
        return BD_ERR_MISALIGNED;
    const size_t n = static_cast<size_t>(T) * static_cast<size_t>(d), g = static_cast<size_t>(d) * 2;
    const size_t obytes = n * (out_dtype == BD_OUT_F32 ? 4 : out_dtype == BD_OUT_BF16 ? 2 : 1);
    const size_t tbytes = static_cast<size_t>(T) * 4, gbytes = static_cast<size_t>(gate_rows) * g;
    const auto written_over = [&](const void* in, size_t bytes) {  // by an output other than residual_out
        return overlaps(out, obytes, in, bytes) || overlaps(scale, tbytes, in, bytes);
    };
    const auto met = [&](const void* in, size_t bytes) {  // by any output
        return written_over(in, bytes) || overlaps(residual_out, n * 2, in, bytes);
    };
    if (written_over(x, n * 2) || written_over(residual, n * 2) || written_over(residual_out, n * 2) || met(gain, g) ||
        met(post_gain, g) || met(gate, gbytes) || met(gate_idx, tbytes) || met(vid, tbytes) || met(ws, ws_bytes) ||
        overlaps(out, obytes, scale, tbytes) || (residual_out != x && overlaps(residual_out, n * 2, x, n * 2)) ||
        (residual_out != residual && overlaps(residual_out, n * 2, residual, n * 2)))
        return BD_ERR_INVALID_ARG;
    bd::BlockNormArgs a{};
    if (vid) {
        for (int32_t v = 0; v < V; ++v) {
            for (const uint16_t* w : {gain_tab[v], post_gain ? post_gain_tab[v] : gain_tab[v]}) {
                if (!w) return BD_ERR_INVALID_ARG;
                if (!aligned(w, 16)) return BD_ERR_MISALIGNED;
                if (met(w, g)) return BD_ERR_INVALID_ARG;
            }
            a.gains[v] = gain_tab[v];
            if (post_gain) a.post_gains[v] = post_gain_tab[v];
        }
    }
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    a.x = x;
    a.residual = residual;
    a.residual_out = residual_out;
    a.post_gain = post_gain;
    a.gain = gain;
    a.gate = gate;
    a.gate_rows = gate_rows;
    a.gate_idx = gate_idx;
    a.vid = vid;
    a.V = V;
    a.block_scale = block_scale;
    a.residual_scale = residual_scale;
    a.T = T;
    a.d = d;
    a.eps = eps;
    a.out = out;
    a.out_dtype = out_dtype;
    a.scale = scale;
    a.err = err_word(ws);
    return launched(bd::launch_block_norm(a, sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ paged KV cache

// A cache's shape, pointers and alignment; *out is what the kernels take.
static bd_status check_kv_pages(const bd_kv_pages* c, bd::KvPages* out)
{
    if (!c) return BD_ERR_INVALID_ARG;
    if (c->dtype != BD_KV_BF16 && c->dtype != BD_KV_INT8 && c->dtype != BD_KV_INT4) return BD_ERR_INVALID_ARG;
    int shift = 4;
    while (shift < 7 && (1 << shift) < c->page_size) ++shift;
    if ((1 << shift) != c->page_size || (c->head_dim != 64 && c->head_dim != 128) || c->n_kv < 1 || c->n_kv > 1024 ||
        c->n_pages < 0 || c->n_pages > INT32_MAX / c->n_kv || c->n_pages > INT32_MAX / c->page_size)
        return BD_ERR_UNSUPPORTED_SHAPE;
    const bool codes = c->dtype != BD_KV_BF16;
    if (!c->k || !c->v || (codes && (!c->k_scale || !c->v_scale))) return BD_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || (codes && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))))
        return BD_ERR_MISALIGNED;
    *out = bd::KvPages{c->k, c->v, codes ? c->k_scale : nullptr, codes ? c->v_scale : nullptr, c->n_pages, c->page_size,
                       shift, c->n_kv, c->head_dim, c->dtype == BD_KV_INT8, c->dtype == BD_KV_INT4};
    return BD_OK;
}

static size_t kv_vectors(const bd::KvPages& c)
{
    return static_cast<size_t>(c.n_pages) * static_cast<size_t>(c.n_kv) * static_cast<size_t>(c.page);
}

// Whether [p, p + n) meets any buffer of the cache.
static bool meets_cache(const bd::KvPages& c, const void* p, size_t n)
{
    const size_t vec = kv_vectors(c), dim = static_cast<size_t>(c.dim);
    const size_t bytes = vec * (c.int4 ? dim / 2 : c.int8 ? dim : 2 * dim), sb = vec * (c.int4 ? dim / 32 : 1) * 4;
    return overlaps(p, n, c.k, bytes) || overlaps(p, n, c.v, bytes) || overlaps(p, n, c.k_scale, sb) ||
           overlaps(p, n, c.v_scale, sb);
}

// Bytes from the first to the last element of T strided rows.
static size_t span_bytes(int64_t T, int64_t stride, int64_t row)
{
    return (static_cast<size_t>(T - 1) * static_cast<size_t>(stride) + static_cast<size_t>(row)) * 2;
}

size_t bd_rope_append_workspace_size(int64_t /*T*/) { return kWsHeader; }

bd_status bd_rope_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                         int64_t v_stride, int64_t T, int32_t n_q, const int32_t* pos, int32_t n_axes,
                         const uint8_t* axis_of_pair, const float* rope_tab, int64_t n_pos, int32_t rot_dim,
                         int interleaved, const int32_t* slot, const bd_kv_pages* cache, uint16_t* q_out,
                         int64_t q_out_stride, void* ws, size_t ws_bytes, void* stream)
{
    BD_NVTX_RANGE("bd_rope_append");
    bd::RopeArgs a{};
    if (bd_status s = check_kv_pages(cache, &a.cache)) return s;
    const int64_t dim = a.cache.dim, kv_row = a.cache.n_kv * dim, q_row = n_q * dim;
    if (T < 0 || T > INT32_MAX || n_q < 0 || n_q > 65536 || rot_dim < 0 || rot_dim % 16 != 0 || rot_dim > dim)
        return BD_ERR_UNSUPPORTED_SHAPE;
    if (k_stride < kv_row || v_stride < kv_row || k_stride % 8 || v_stride % 8 ||
        (n_q > 0 && (q_stride < q_row || q_out_stride < q_row || q_stride % 8 || q_out_stride % 8)))
        return BD_ERR_UNSUPPORTED_SHAPE;
    if (n_axes < 1 || n_axes > BD_MAX_AXES) return BD_ERR_INVALID_ARG;
    if (bd_status s = check_ws(ws, ws_bytes, bd_rope_append_workspace_size(T))) return s;
    for (int i = 0; axis_of_pair && i < rot_dim / 2; ++i) {
        if (axis_of_pair[i] >= n_axes) return BD_ERR_INVALID_ARG;
        a.axis_of_pair[i] = axis_of_pair[i];
    }
    if (T == 0) return BD_OK;
    if (!k || !v || !slot || (n_q > 0 && (!q || !q_out)) || (rot_dim > 0 && (!pos || !rope_tab || n_pos < 1)))
        return BD_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || (n_q > 0 && (!aligned(q, 16) || !aligned(q_out, 16))) ||
        !aligned(rope_tab, 16) || !aligned(pos, 4) || !aligned(slot, 4))
        return BD_ERR_MISALIGNED;
    const size_t tbytes = static_cast<size_t>(T) * 4;
    const size_t kb = span_bytes(T, k_stride, kv_row), vb = span_bytes(T, v_stride, kv_row);
    const size_t pb = rot_dim > 0 ? tbytes * n_axes : 0;
    const size_t rb = rot_dim > 0 ? static_cast<size_t>(n_pos) * rot_dim * 4 : 0;
    if (meets_cache(a.cache, k, kb) || meets_cache(a.cache, v, vb) || meets_cache(a.cache, slot, tbytes) ||
        meets_cache(a.cache, ws, ws_bytes) || meets_cache(a.cache, pos, pb) || meets_cache(a.cache, rope_tab, rb))
        return BD_ERR_INVALID_ARG;
    if (n_q > 0) {
        const size_t qb = span_bytes(T, q_stride, q_row), ob = span_bytes(T, q_out_stride, q_row);
        const bool in_place = q_out == q && q_out_stride == q_stride;
        // in place, k and v may lie between q's rows (slices of one product): their columns are apart
        const auto apart = [&](const uint16_t* p, int64_t stride) {
            if (stride != q_out_stride) return false;
            const int64_t d = reinterpret_cast<intptr_t>(p) - reinterpret_cast<intptr_t>(q_out);
            const int64_t row = stride * 2, at = ((d % row) + row) % row;
            return at >= q_row * 2 && at + kv_row * 2 <= row;
        };
        if (meets_cache(a.cache, q, qb) || meets_cache(a.cache, q_out, ob) || overlaps(q_out, ob, slot, tbytes) ||
            overlaps(q_out, ob, ws, ws_bytes) || overlaps(q_out, ob, pos, pb) || overlaps(q_out, ob, rope_tab, rb) ||
            (overlaps(q_out, ob, k, kb) && !apart(k, k_stride)) || (overlaps(q_out, ob, v, vb) && !apart(v, v_stride)) ||
            (!in_place && overlaps(q_out, ob, q, qb)))
            return BD_ERR_INVALID_ARG;
    }
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.T = T;
    a.n_q = n_q;
    a.pos = pos;
    a.n_axes = n_axes;
    a.tab = rope_tab;
    a.n_pos = n_pos;
    a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    a.slot = slot;
    a.q_out = q_out;
    a.err = err_word(ws);
    return launched(bd::launch_rope_append(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t bd_kv_read_workspace_size(int64_t /*rows*/) { return kWsHeader; }

bd_status bd_kv_read(const bd_kv_pages* cache, const int32_t* page_table, int64_t max_pages, const int32_t* kv_off,
                     int64_t n_seq, int64_t rows, uint16_t* k_out, uint16_t* v_out, void* ws, size_t ws_bytes,
                     void* stream)
{
    BD_NVTX_RANGE("bd_kv_read");
    bd::KvReadArgs a{};
    if (bd_status s = check_kv_pages(cache, &a.cache)) return s;
    if (n_seq < 0 || n_seq > INT32_MAX || rows < 0 || rows > INT32_MAX || max_pages < 0 ||
        max_pages > INT32_MAX / a.cache.page)
        return BD_ERR_UNSUPPORTED_SHAPE;
    if (bd_status s = check_ws(ws, ws_bytes, bd_kv_read_workspace_size(rows))) return s;
    if (n_seq == 0 || rows == 0) return BD_OK;
    if (!page_table || !kv_off || !k_out || !v_out) return BD_ERR_INVALID_ARG;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(page_table, 4) || !aligned(kv_off, 4))
        return BD_ERR_MISALIGNED;
    const size_t ob = static_cast<size_t>(rows) * static_cast<size_t>(a.cache.n_kv) * a.cache.dim * 2;
    const size_t pb = static_cast<size_t>(n_seq) * static_cast<size_t>(max_pages) * 4;
    const size_t fb = static_cast<size_t>(n_seq + 1) * 4;
    for (const void* o : {static_cast<const void*>(k_out), static_cast<const void*>(v_out)})
        if (meets_cache(a.cache, o, ob) || overlaps(o, ob, page_table, pb) || overlaps(o, ob, kv_off, fb) ||
            overlaps(o, ob, ws, ws_bytes))
            return BD_ERR_INVALID_ARG;
    if (overlaps(k_out, ob, v_out, ob)) return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    a.table = page_table;
    a.max_pages = max_pages;
    a.kv_off = kv_off;
    a.n_seq = n_seq;
    a.rows = rows;
    a.k_out = k_out;
    a.v_out = v_out;
    a.err = err_word(ws);
    return launched(bd::launch_kv_read(a, sms, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ attention

size_t bd_attention_workspace_size(int64_t T, int64_t n_seq, int32_t n_q, int32_t n_kv, int32_t head_dim)
{
    if (T < 0 || n_seq < 0 || n_kv < 1 || n_q < n_kv || (head_dim != 64 && head_dim != 128)) return kWsHeader;
    return bd::attention_workspace_size(T, n_seq, n_q, n_kv, head_dim);
}

bd_status bd_attention(const uint16_t* q, int64_t q_stride, const int32_t* q_off, int64_t T, int64_t n_seq,
                       int64_t max_new, int32_t n_q, const bd_kv_pages* cache, const int32_t* page_table,
                       int64_t max_pages, const int32_t* kv_len, float scale, int causal, uint16_t* out, float* lse,
                       void* ws, size_t ws_bytes, void* stream)
{
    BD_NVTX_RANGE("bd_attention");
    bd::AttentionArgs a{};
    if (bd_status s = check_kv_pages(cache, &a.cache)) return s;
    if (n_q < 1 || n_q % a.cache.n_kv != 0 || n_q > 65536 || T < 0 || n_seq < 0 || max_new < 0 || max_pages < 0 ||
        n_seq > INT32_MAX / 2 || max_pages > INT32_MAX / a.cache.page || T > INT32_MAX / n_q)
        return BD_ERR_UNSUPPORTED_SHAPE;
    const int64_t row = static_cast<int64_t>(n_q) * a.cache.dim;
    if (q_stride < row || q_stride % 8) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!(scale - scale == 0.0f)) return BD_ERR_INVALID_ARG;  // not finite
    if (bd_status s = check_ws(ws, ws_bytes, bd_attention_workspace_size(T, n_seq, n_q, a.cache.n_kv, a.cache.dim)))
        return s;
    if (T == 0 || n_seq == 0) return BD_OK;
    // a bad page is replaced by page 0, and the tensor maps need an extent: there has to be one
    if (a.cache.n_pages == 0) return BD_ERR_UNSUPPORTED_SHAPE;
    if (!q || !q_off || !kv_len || !out || (!page_table && max_pages > 0)) return BD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(q_off, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4) ||
        !aligned(lse, 4))
        return BD_ERR_MISALIGNED;
    const size_t qb = span_bytes(T, q_stride, row);
    const size_t ob = static_cast<size_t>(T) * static_cast<size_t>(row) * 2, lb = static_cast<size_t>(T) * n_q * 4;
    const size_t pb = static_cast<size_t>(n_seq) * static_cast<size_t>(max_pages) * 4;
    const size_t fb = static_cast<size_t>(n_seq + 1) * 4;
    const auto written_over = [&](const void* in, size_t n) { return overlaps(out, ob, in, n) || overlaps(lse, lb, in, n); };
    if (written_over(q, qb) || written_over(q_off, fb) || written_over(kv_len, fb - 4) || written_over(page_table, pb) ||
        written_over(ws, ws_bytes) || meets_cache(a.cache, out, ob) || meets_cache(a.cache, lse, lb) ||
        meets_cache(a.cache, ws, ws_bytes) || overlaps(out, ob, lse, lb) || overlaps(ws, ws_bytes, q, qb) ||
        overlaps(ws, ws_bytes, q_off, fb) || overlaps(ws, ws_bytes, kv_len, fb - 4) ||
        overlaps(ws, ws_bytes, page_table, pb))
        return BD_ERR_INVALID_ARG;
    int sms = 0;
    if (bd_status s = device_info(&sms)) return s;
    a.q = q;
    a.q_stride = q_stride;
    a.q_off = q_off;
    a.T = T;
    a.n_seq = n_seq;
    a.max_new = max_new;
    a.n_q = n_q;
    a.table = page_table;
    a.max_pages = max_pages;
    a.kv_len = kv_len;
    a.scale = scale;
    a.causal = causal != 0;
    a.out = out;
    a.lse = lse;
    a.ws = ws;
    a.err = err_word(ws);
    a.sm_count = sms;
    return launched(bd::launch_attention(a, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ async errors

int bd_debug_bounds_check(uint32_t* kernels)
{
    const uint32_t f = bd::bounds_take_compress() | bd::bounds_take_skinny() | bd::bounds_take_multi() |
                       bd::bounds_take_prefill() | bd::bounds_take_route() | bd::bounds_take_materialize() |
                       bd::bounds_take_monosoup() | bd::bounds_take_norm() | bd::bounds_take_block_norm() |
                       bd::bounds_take_kv() |
                       bd::bounds_take_attention() | bd::bounds_take_attention_chunk();
    if (kernels) *kernels = f;
    if (f == ~0u) return BD_ERR_CUDA;
    return f ? BD_ERR_BOUNDS : BD_OK;
}

int bd_debug_bounds_enabled(void)
{
#ifdef BD_DEBUG_BOUNDS
    return 1;
#else
    return 0;
#endif
}

bd_status bd_check_async(void* ws, void* stream)
{
    if (!ws) return BD_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return BD_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    if (const int cs_ = bd::cuda_status(cudaMemcpyAsync(&word, ws, sizeof word, cudaMemcpyDeviceToHost, st))) return static_cast<bd_status>(cs_);
    if (const int cs_ = bd::cuda_status(cudaStreamSynchronize(st))) return static_cast<bd_status>(cs_);
    if (word == 0) return BD_OK;
    const uint32_t zero = 0;
    if (const int cs_ = bd::cuda_status(cudaMemcpyAsync(ws, &zero, sizeof zero, cudaMemcpyHostToDevice, st))) return static_cast<bd_status>(cs_);
    if (const int cs_ = bd::cuda_status(cudaStreamSynchronize(st))) return static_cast<bd_status>(cs_);
    if (word & (1u << BD_ERR_TIMEOUT)) return BD_ERR_TIMEOUT;
    if (word & (1u << BD_ERR_BAD_VARIANT)) return BD_ERR_BAD_VARIANT;
    if (word & (1u << BD_ERR_BAD_INDEX)) return BD_ERR_BAD_INDEX;
    if (word & (1u << BD_ERR_NONFINITE)) return BD_ERR_NONFINITE;
    return BD_ERR_CUDA;
}

}  // extern "C"
