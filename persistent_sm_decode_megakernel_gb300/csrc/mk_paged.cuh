// Shared by the paged-cache operators (append, attention, page updates, beam selection):
// launches as programmatic dependents, the device status word, type conversions.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <exception>
#include <string>

#include "../../include/mk.h"

namespace mk {

void set_last_error(const std::string& msg);  // defined beside mk_last_error

enum PagedOp : int { PO_APPEND = 1, PO_ATTEND = 2, PO_UPDATE = 3, PO_COMPACT = 4, PO_SELECT = 5 };

inline mk_status paged_fail(mk_status s, const std::string& m) {
  set_last_error(m);
  return s;
}

// The body of a C entry point: whatever it throws (memory that a descriptor asks for and the
// host does not have) becomes a status.
template <typename F>
inline mk_status c_entry(F&& body) noexcept {
  try {
    return body();
  } catch (const std::exception& e) {
    try {
      set_last_error(std::string("host: ") + e.what());
    } catch (...) {
    }
  } catch (...) {
  }
  return MK_ERR_INVALID;
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// whether vectors of `dim` elements at strides s0 (n0 of them) and s1 (n1) lie over one another for certain
inline bool overlaps(long long n0, long long s0, long long n1, long long s1, long long dim) {
  const long long a0 = s0 < 0 ? -s0 : s0, a1 = s1 < 0 ? -s1 : s1;
  return (n0 > 1 && a0 < dim) || (n1 > 1 && a1 < dim) || (n0 > 1 && n1 > 1 && a0 == a1);
}
inline size_t round16(size_t x) { return (x + 15) & ~size_t(15); }

// Every kernel of these operators is launched as a programmatic dependent of what precedes
// it in the stream and waits for that (pdl_wait) before it touches memory: its launch
// overlaps the previous kernel's tail, the order of the data stays the stream's.
template <typename... Params, typename... Args>
inline mk_status launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, void* stream,
                                  const char* what, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return paged_fail(MK_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  return MK_OK;
}

// multiprocessors of the current device (looked up once per device)
mk_status sm_count(int* n);
// the checks on a page view that every operator over pages applies: "" when usable
std::string check_view(const mk_page_view* c);
// whether the attention can count its work over that many rows of the table: "" when it can
std::string check_line(const mk_page_view* c, long long n_rows, int window);

#ifdef __CUDACC__
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// keeps the first error found (of several found at the same time, one of them)
__device__ __noinline__ static void report(int32_t* status, int code, int op, int row, int value) {
  if (status != nullptr && atomicCAS(status, 0, code) == 0) {
    status[1] = op;
    status[2] = row;
    status[3] = value;
  }
}

template <typename T>
struct Conv;
template <>
struct Conv<float> {
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <>
struct Conv<__half> {
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <>
struct Conv<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};

// what is read once need not stay in L1
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 8 consecutive elements of memory (16-byte aligned), as they lie there
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = ldg_stream(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void gather(const T* p) {  // wherever p lies
#pragma unroll
    for (int i = 0; i < 8; ++i) reinterpret_cast<T*>(w)[i] = p[i];
  }
  __device__ __forceinline__ void up(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Conv<T>::up(reinterpret_cast<const T*>(w)[i]);
  }
};
// two floats rounded to a pair of 16-bit values in one word
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
#endif

}  // namespace mk
