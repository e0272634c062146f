// Host-side helpers shared by the training operators' translation units: the
// calling thread's error message, argument checks, tensor maps and launches.
// Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "fadam_ops.h"

namespace fadam_ops {

// Records the message for fadam_ops_last_error() and returns `st`.
fadam_status fail(fadam_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fadam_status cuda_fail(cudaError_t e, const char* what);
void clear_error();

inline int elem_size(int32_t dt) {
  return dt == FADAM_DT_F32 ? 4 : dt == FADAM_DT_BF16 || dt == FADAM_DT_F16 ? 2 : 0;
}
inline bool is_16bit(int32_t dt) { return dt == FADAM_DT_BF16 || dt == FADAM_DT_F16; }
inline bool misaligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// Facts of the current device, looked up once per device.
struct DeviceFacts {
  int sm_count;
  int* status;  // device word that a wait which gave up sets to FADAM_ETIMEOUT
};
fadam_status device_facts(DeviceFacts* out);

// A [rows, inner] row-major matrix of 16-bit elements, `ld` elements from one
// row to the next, read in boxes of box_rows x 64 elements with the 128-byte
// swizzle.  Elements outside the matrix read as zero.
fadam_status matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t inner, int64_t ld,
                        int box_rows);
// What a matrix needs for that: a 16-byte aligned base and row stride.
inline bool bulk_readable(const void* base, int64_t ld) {
  return !misaligned(base, 16) && ld % 8 == 0;
}

// Launches a kernel that may begin while the launch before it on the stream
// still runs: it sets itself up and calls chain_wait() (ops_device.cuh) before
// it touches memory.  A chain's setup and launch latency then lie under its
// predecessor's end.
template <class... Params, class... Args>
fadam_status launch_chained(const char* what, void (*kernel)(Params...), int64_t grid, int block,
                            size_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(unsigned(grid));
  config.blockDim = dim3(unsigned(block));
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&config, kernel, std::forward<Args>(args)...);
  return e == cudaSuccess ? FADAM_OK : cuda_fail(e, what);
}

// Hands out consecutive 256-byte aligned pieces of a workspace; with a NULL
// base it only adds up their sizes.
struct Carver {
  char* base;
  size_t used = 0;
  void* take(size_t bytes) {
    void* p = base ? base + used : nullptr;
    used += (bytes + 255) / 256 * 256;
    return p;
  }
};

}  // namespace fadam_ops
