// lod_host.cuh -- host helpers shared by the files that implement the C entry
// points: the thread-local error text, pointer checks and tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <initializer_list>
#include <utility>

#include "lod.h"

namespace lod {
namespace host {

// Record the calling thread's error text (lod_last_error) and return `code`.
int32_t fail(int32_t code, const char* fmt, ...);
int32_t cuda_fail(cudaError_t e, const char* what);
// Forget the calling thread's error text; returns LOD_OK.
int32_t ok();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A per-call buffer the kernels read or write in place: memory of the current
// device, managed memory, or page-locked host memory mapped at the same
// address (cudaHostAlloc / cudaMallocHost under unified addressing: the
// kernels then move its bytes over the host link themselves).  Pageable host
// memory and another device's memory are refused before anything is enqueued.
int32_t check_visible(const void* ptr, const char* name, int* host = nullptr);
int32_t check_visible_all(std::initializer_list<std::pair<const void*, const char*>> bufs);

// Tiled tensor map of `rank` dimensions with boxes of box_cols x box_rows
// elements (128-byte rows, 128-byte swizzle).
int32_t encode_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides_bytes,
                   cuuint32_t box_rows = 128, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   cuuint32_t box_cols = 64);

// Streaming multiprocessors of the current device.
int num_sms();

// The checks every entry point of the dense cache makes of lod_params and of
// K, V and their strides (LOD_OK, or the error recorded).
int32_t check_params(const lod_params* p);
int32_t check_cache(const lod_params* p, const void* K, const void* V, const int64_t* kv_strides);

}  // namespace host
}  // namespace lod
