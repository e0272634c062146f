// Host-side helpers of the training operators: error messages, device facts
// and tensor maps.
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "ops_internal.h"

// Set by a kernel whose bounded wait gave up; read by fadam_ops_status.
static __device__ int g_ops_status;
// What fadam_ops_status found there.  Read and cleared in one step: what is set
// in between by a launch of another thread is left for the next call.
static __device__ int g_ops_status_taken;
static __global__ void take_status_kernel() { g_ops_status_taken = atomicExch(&g_ops_status, 0); }

namespace fadam_ops {

namespace {
thread_local char t_error[512];
constexpr int kMaxDevices = 64;
std::mutex g_mutex;
DeviceFacts g_facts[kMaxDevices];
bool g_known[kMaxDevices];

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);
Encode find_encode() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return nullptr;
  }
  return found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(fn) : nullptr;
}
}  // namespace

fadam_status fail(fadam_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_error, sizeof t_error, fmt, ap);
  va_end(ap);
  return st;
}

fadam_status cuda_fail(cudaError_t e, const char* what) {
  snprintf(t_error, sizeof t_error, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  (void)cudaGetLastError();  // clear a non-sticky error so later calls start clean
  return FADAM_ECUDA;
}

void clear_error() { t_error[0] = 0; }

fadam_status device_facts(DeviceFacts* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(FADAM_ELIMIT, "device %d beyond %d", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_known[dev]) {
    DeviceFacts f{};
    e = cudaDeviceGetAttribute(&f.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    void* word = nullptr;
    e = cudaGetSymbolAddress(&word, g_ops_status);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress");
    f.status = static_cast<int*>(word);
    g_facts[dev] = f;
    g_known[dev] = true;
  }
  *out = g_facts[dev];
  return FADAM_OK;
}

fadam_status matrix_map(CUtensorMap* map, const void* base, int64_t rows, int64_t inner, int64_t ld,
                        int box_rows) {
  static const Encode encode = find_encode();
  if (!encode) return fail(FADAM_ECUDA, "the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {64, cuuint32_t(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  // the type only fixes the element size: nothing is converted on the way
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(FADAM_ECUDA, "cuTensorMapEncodeTiled: %d for a %lld x %lld matrix of stride %lld",
                int(r), (long long)rows, (long long)inner, (long long)ld);
  return FADAM_OK;
}

}  // namespace fadam_ops

extern "C" const char* fadam_ops_last_error(void) { return fadam_ops::t_error; }

extern "C" fadam_status fadam_ops_status(int32_t* device_status) {
  using namespace fadam_ops;
  clear_error();
  if (!device_status) return fail(FADAM_EINVAL, "device_status is NULL");
  int word = 0;
  // all streams of the device: the default one does not wait for non-blocking ones
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) {
    std::lock_guard<std::mutex> lock(g_mutex);
    take_status_kernel<<<1, 1>>>();
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, g_ops_status_taken, sizeof word);
  }
  if (e != cudaSuccess) return cuda_fail(e, "fadam_ops_status");
  *device_status = word;
  return FADAM_OK;
}
