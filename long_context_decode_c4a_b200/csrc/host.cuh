// host.cuh -- host-side helpers shared by the files that implement the C ABI: argument-check macros,
// the thread's error text, device attributes, workspace checks and launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <utility>

#include "csa.h"

namespace csa {

// Record the calling thread's error text (csa_last_error) and return `code`.
int fail(int code, const char* fmt, ...);

#define CSA_CHECK_ARG(cond, ...)                                   \
  do {                                                             \
    if (!(cond)) return fail(CSA_ERR_INVALID_ARG, __VA_ARGS__);    \
  } while (0)
#define CSA_CHECK_SUP(cond, ...)                                   \
  do {                                                             \
    if (!(cond)) return fail(CSA_ERR_UNSUPPORTED, __VA_ARGS__);    \
  } while (0)
#define CSA_CUDA(call)                                                                     \
  do {                                                                                     \
    cudaError_t e_ = (call);                                                               \
    if (e_ != cudaSuccess) return fail(CSA_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct DeviceInfo {
  int sms = 0;
  int max_smem = 0;
  bool attrs_set = false;
};

// Launch with programmatic stream serialization: the kernel may begin launching while the
// previous kernel on the stream runs; it calls pdl_wait() before touching global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Attributes of the current device (looked up once per device, kernels' shared memory limits set).
int device_info(DeviceInfo** out);

// Splits of a query's candidates that an attention workspace is sized for, and the bytes of their partials.
int attn_ws_splits(long long queries);
size_t attn_part_bytes(long long queries, int splits);

inline int log2_int(int x) {
  int k = 0;
  while ((1 << k) < x) ++k;
  return k;
}

// A page table and a cache behind it, for B requests: e4m3 rows of 512 (quantised) or bf16 rows.
int check_table(const csa_page_table* pt, int B);
int check_paged(const csa_page_table* pt, const csa_paged_cache* c, int B, bool quantised);

// Bytes of a CSA_WS_PAGES workspace.
size_t pages_ws_bytes(long long slots, long long max_pages, long long num_pages);

// The workspace is present, 256-byte aligned and at least `need` bytes.
int check_ws(const void* ws, size_t ws_bytes, size_t need);

}  // namespace csa
