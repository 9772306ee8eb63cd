// Shared by the language-model entry points (pp_grammar.cu, pp_logits.cu,
// pp_embed.cu): element types, id loads and 16-byte packs.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pp.h"

namespace ppl {

constexpr uint64_t MAX_DIM = (uint64_t(1) << 31) - 65536;

inline pp_rc rc_of(cudaError_t e) {
  if (e == cudaSuccess) return PP_OK;
  return e == cudaErrorMemoryAllocation ? PP_ENOMEM : PP_ECUDA;
}
inline bool ftype_ok(int t) { return t >= PP_F32 && t <= PP_BF16; }
inline bool itype_ok(int t) { return t >= PP_U8 && t <= PP_I64; }
inline size_t fsize(int t) { return t == PP_F32 ? 4 : 2; }
inline size_t isize(int t) { return t == PP_I64 ? 8 : t == PP_I32 ? 4 : 1; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// The id at index i as int64.
__device__ __forceinline__ int64_t load_id(const void* p, int type, uint64_t i) {
  switch (type) {
    case PP_U8: return static_cast<const uint8_t*>(p)[i];
    case PP_I8: return static_cast<const int8_t*>(p)[i];
    case PP_I32: return static_cast<const int32_t*>(p)[i];
    default: return static_cast<const int64_t*>(p)[i];
  }
}

// f(position, id) for the ids at positions first, first + step, ... below n,
// BATCH loads on their way at a time (a load per iteration would wait for
// each: the id feeds a shared-memory atomic that later loads stay behind).
template <int BATCH, class I, class F>
__device__ __forceinline__ void for_ids_of(const I* p, uint64_t stride, uint32_t first, uint32_t n, uint32_t step, F&& f) {
  const I* q = p + first * stride;
  const uint64_t d = step * stride;
  uint64_t i = first;
  for (; i + uint64_t(BATCH - 1) * step < n; i += uint64_t(BATCH) * step, q += BATCH * d) {
    I v[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) v[k] = q[k * d];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) f(uint32_t(i) + k * step, v[k]);
  }
  I v[BATCH];
#pragma unroll
  for (int k = 0; k < BATCH; ++k)
    if (i + uint64_t(k) * step < n) v[k] = q[k * d];
#pragma unroll
  for (int k = 0; k < BATCH; ++k)
    if (i + uint64_t(k) * step < n) f(uint32_t(i) + k * step, v[k]);
}
template <int BATCH, class F>
__device__ __forceinline__ void for_ids(const void* p, int type, uint64_t stride, uint32_t first, uint32_t n, uint32_t step, F&& f) {
  switch (type) {
    case PP_U8: return for_ids_of<BATCH>(static_cast<const uint8_t*>(p), stride, first, n, step, f);
    case PP_I8: return for_ids_of<BATCH>(static_cast<const int8_t*>(p), stride, first, n, step, f);
    case PP_I32: return for_ids_of<BATCH>(static_cast<const int32_t*>(p), stride, first, n, step, f);
    default: return for_ids_of<BATCH>(static_cast<const int64_t*>(p), stride, first, n, step, f);
  }
}

// The barrier of a thread-block cluster.  A block's shared memory may be
// accessed by others once it has started: every thread arrives when its kernel
// begins and waits before the first such access, by which time the others'
// arrivals are long over.  cluster_sync also orders memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// N elements moved in accesses of at most 16 bytes (p aligned to that).
template <class T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
  T v[N];
};

}  // namespace ppl
