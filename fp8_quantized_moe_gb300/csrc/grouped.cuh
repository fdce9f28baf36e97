// What the grouped kernels on block-scaled 8-bit operands share: tensor maps,
// device queries and the waits of issuing warps.  (Included by several translation units; everything is local to each.)
#pragma once

#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxGroups = 1024;
constexpr int kMaxDevices = 256;  // host-side per-device caches

// One lane of the warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Whether the phase has completed, asked without waiting (try_wait may wait microseconds).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait of a whole warp that issues loads or MMAs.  Such a warp runs its loop with
// all lanes, and only the issuing instructions are one lane's: what they take (addresses,
// descriptors) is then the warp's, in uniform registers, and a stage costs half the clocks
// of a loop that one lane runs alone (tgmm_fp8_mx without MMAs: 190 against 340 ns a stage).
__device__ __forceinline__ bool wait_uniform(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 64;\n\t"
      "@q bra AGAIN;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, ok != 0)) return true;
  return __all_sync(0xffffffffu, mbar_wait_bounded_idle(bar, parity, abort_flag, kWaitLimitNs));
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A byte matrix [rows, cols] of row pitch `pitch` for boxes of box_rows x 128
// bytes in the 128-byte swizzle, or as they lie; reads past the extents return zeros.
inline bool make_map_u8(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t pitch,
                        uint32_t box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
  cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device, or -1 where it is not an sm_103 (or on an error), and its SMs; asked
// of the runtime once a device (half a microsecond a call otherwise).
inline int sm103_device(int* sms) {
  static std::atomic<int> known[kMaxDevices];  // 0: not asked yet; -1: another device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      return -1;
    if (major != 10 || minor != 3) n = -1;
    known[dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return n > 0 ? dev : -1;
}

// Let `kernel` have `bytes` of dynamic shared memory on device `dev`: once a device.
struct SmemLimit {
  std::atomic<bool> done[kMaxDevices];
  template <class K>
  cudaError_t set(K kernel, size_t bytes, int dev) {
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
  }
};

}  // namespace
}  // namespace moe
