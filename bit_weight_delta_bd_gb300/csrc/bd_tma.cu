// TMA tensor-map encoding (see bd_tma.h).
#include <cstring>
#include <mutex>
#include <unordered_map>

#include "bd_tma.h"

namespace bd {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

struct MapKey {
    uintptr_t base;
    uint64_t cols, rows, row_bytes;
    uint32_t box_cols, box_rows;
    int dtype, swizzle;
    uint32_t rank = 2;    // 2, 3 (contiguous slices) or 4 (rows in parts)
    uint64_t outer = 1;
    uint32_t parts = 1;
    bool operator==(const MapKey& o) const
    {
        return base == o.base && cols == o.cols && rows == o.rows && row_bytes == o.row_bytes &&
               box_cols == o.box_cols && box_rows == o.box_rows && dtype == o.dtype && swizzle == o.swizzle &&
               rank == o.rank && outer == o.outer && parts == o.parts;
    }
};

struct MapKeyHash {
    size_t operator()(const MapKey& k) const
    {
        uint64_t h = 1469598103934665603ull;
        const uint64_t v[11] = {static_cast<uint64_t>(k.base), k.cols, k.rows, k.row_bytes, k.box_cols, k.box_rows,
                               static_cast<uint64_t>(k.dtype), static_cast<uint64_t>(k.swizzle), k.rank, k.outer,
                               k.parts};
        for (uint64_t x : v) h = (h ^ x) * 1099511628211ull;
        return static_cast<size_t>(h);
    }
};

constexpr size_t kMapCacheMax = 4096;

}  // namespace

namespace {

// A map of the key's rank.  No map of another rank stands in for an array with
// an extent of 0: the encoder refuses that.
bool encode(CUtensorMap* map, const MapKey& key)
{
    thread_local std::unordered_map<MapKey, CUtensorMap, MapKeyHash> cache;
    auto it = cache.find(key);
    if (it != cache.end()) {
        std::memcpy(map, &it->second, sizeof(CUtensorMap));
        return true;
    }
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const bool split = key.rank == 4;
    const cuuint64_t part_bytes = key.row_bytes / key.parts, slice = key.rows * key.row_bytes;
    const cuuint64_t dims[4] = {split ? key.cols / key.parts : key.cols, key.rows, split ? key.parts : key.outer,
                                key.outer};
    const cuuint64_t strides[3] = {key.row_bytes, split ? part_bytes : slice, slice};
    const cuuint32_t box[4] = {key.box_cols, key.box_rows, split ? key.parts : 1, 1};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    if (fn(map, static_cast<CUtensorMapDataType>(key.dtype), key.rank, reinterpret_cast<void*>(key.base), dims, strides,
           box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, static_cast<CUtensorMapSwizzle>(key.swizzle),
           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    if (cache.size() >= kMapCacheMax) cache.clear();
    cache.emplace(key, *map);
    return true;
}

}  // namespace

bool encode_tma_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, uint64_t cols, uint64_t rows,
                   uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    return encode(map, MapKey{reinterpret_cast<uintptr_t>(base), cols, rows, row_bytes, box_cols, box_rows,
                              static_cast<int>(dtype), static_cast<int>(swizzle)});
}

bool encode_tma_3d(CUtensorMap* map, CUtensorMapDataType dtype, uint32_t elem_bytes, const void* base, uint64_t cols,
                   uint64_t rows, uint64_t outer, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    return encode(map, MapKey{reinterpret_cast<uintptr_t>(base), cols, rows, cols * elem_bytes, box_cols, box_rows,
                              static_cast<int>(dtype), static_cast<int>(swizzle), 3, outer});
}

bool encode_tma_parts(CUtensorMap* map, CUtensorMapDataType dtype, uint32_t elem_bytes, const void* base, uint64_t cols,
                      uint64_t rows, uint64_t outer, uint32_t parts, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    return encode(map, MapKey{reinterpret_cast<uintptr_t>(base), cols, rows, cols * elem_bytes,
                              static_cast<uint32_t>(cols / parts), box_rows, static_cast<int>(dtype),
                              static_cast<int>(swizzle), 4, outer, parts});
}

cudaError_t ensure_dynamic_smem(const void* kernel, size_t bytes, std::atomic<size_t>* per_device)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kHostMaxDevices) return cudaErrorInvalidDevice;
    if (per_device[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
    // all of the unified L1/shared storage as shared memory, so that as many
    // CTAs (and thread-block clusters) as the shared memory allows are resident
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) per_device[dev].store(bytes, std::memory_order_release);
    return e;
}

}  // namespace bd
