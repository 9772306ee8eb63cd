// pp_token_probs: a model's logits as probabilities, by a temperature and cut
// to each row's k most likely tokens.
//
// A cluster of blocks takes a row, each a part of it, which it reads once into
// shared memory; the largest value, the sum of the exponentials and the
// k-th largest value are found there, and the probabilities are written.  The
// blocks exchange their largest value and their sum relative to it once.
//
// The k-th largest is found digit by digit from the top of the values' bits in
// the order of their values: a count of each digit over the values that agree
// with the digits found, added up over the cluster.  Values that tie with it
// are kept from the lowest token on, so the last one's place is found the same
// way among their places.
#include <algorithm>
#include <cstring>

#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using ppl::to_f;

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int CLUSTER = 8;
constexpr uint32_t RESIDENT_MOST = 200 * 1024;  // bytes of a block's part

struct ProbArgs {
  const void* in;
  float* out;
  const float* temperature;
  const int32_t* top_k;
  uint64_t in_stride, out_stride;
  uint32_t n_vocab, blocks, part;
  int32_t resident;
};

// Floats in an order of unsigned integers; 0 is lost (NaN is taken out before).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 is 0
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t KEY_LOST = 0x007FFFFFu;  // key_of(-infinity)

__device__ __forceinline__ float remote_f(const float* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote_u(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The exponential of (f - top) / temperature, f at most top; c: 2 log2(e) over
// the temperature.  Halves, since the difference of two floats may not be one;
// an infinite difference gives 0, under an infinite temperature too (-200: 0).
__device__ __forceinline__ float share(float f, float top, float c) {
  return f == top ? 1.f : exp2f(fmaxf((f * 0.5f - top * 0.5f) * c, -200.f));
}

struct Shared {
  float part_max, part_sum;
  uint32_t part_first;  // the first token with part_max
  float wmax[WARPS], wsum[WARPS];
  uint32_t wfirst[WARPS];
  uint32_t digit, above;
  uint32_t hist[8][256];
};

// The digit in which the want-th element (from 1, from the largest digit down)
// lies, over the cluster; above: how many elements have larger digits.
__device__ __forceinline__ void digit_of(Shared& sh, int pass, uint32_t blocks, uint32_t want) {
  ppl::cluster_sync();  // every block's counts are there
  if (threadIdx.x < 32) {
    const uint32_t lane = threadIdx.x;
    uint32_t n[8], sum = 0;  // of the digits 255 - 8 lane - k
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      n[k] = 0;
      for (uint32_t b = 0; b < blocks; ++b) n[k] += remote_u(&sh.hist[pass][255 - 8 * lane - k], b);
      sum += n[k];
    }
    uint32_t run = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(~0u, run, d);
      if (lane >= uint32_t(d)) run += y;
    }
    run -= sum;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (run < want && want <= run + n[k]) {
        sh.digit = 255 - 8 * lane - k;
        sh.above = run;
      }
      run += n[k];
    }
  }
  __syncthreads();
}

template <class T>
__global__ void __launch_bounds__(THREADS) probs_kernel(const ProbArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ Shared sh;
  constexpr int VEC = 16 / sizeof(T);
  const uint32_t rank = blockIdx.x % a.blocks, r = blockIdx.x / a.blocks;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const T* in = static_cast<const T*>(a.in) + r * a.in_stride;
  float* out = a.out + r * a.out_stride;
  // places count from the 16-byte boundary at or before the row's start
  const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(in) / sizeof(T) % VEC);
  const uint32_t all = a.n_vocab + shift;
  const uint32_t from = rank * a.part, to = min(from + a.part, all);
  const uint32_t lo = max(from, shift);  // this block's: places lo .. to - 1
  T* buf = reinterpret_cast<T*>(raw);
  if (a.resident) {
    for (uint32_t v = threadIdx.x * VEC; v < a.part; v += THREADS * VEC) {
      const uint32_t j = from + v;
      if (j >= shift && j + VEC <= all) {
        *reinterpret_cast<uint4*>(buf + v) = *reinterpret_cast<const uint4*>(in - shift + j);
      } else {
        for (int k = 0; k < VEC; ++k)
          if (j + k >= shift && j + k < all) buf[v + k] = in[j + k - shift];
      }
    }
    for (uint32_t i = threadIdx.x; i < 8 * 256; i += THREADS) sh.hist[i / 256][i % 256] = 0;
    __syncthreads();
  } else {
    for (uint32_t i = threadIdx.x; i < 8 * 256; i += THREADS) sh.hist[i / 256][i % 256] = 0;
    __syncthreads();
  }
  const T* x = a.resident ? buf - from : in - shift;  // by place
  auto value = [&](uint32_t j) { return fmaxf(to_f(x[j]), -INFINITY); };  // NaN: -infinity
  const float t = a.temperature ? a.temperature[r] : 1.f;
  const bool greedy = !(t > 0x1p-125f);  // below, c is not a float
  const float c = 2.88539008f / t;
  // ---- the k-th largest
  uint32_t least = 0, last = ~0u;  // keys above `least` are kept, and those equal to it at places up to `last`
  const int32_t k = a.top_k ? a.top_k[r] : 0;
  if (k > 0 && uint32_t(k) < a.n_vocab && !greedy) {
    uint32_t want = uint32_t(k), known = 0, mask = 0;
    int pass = 0;
    for (int at = 24; at >= 0; at -= 8, ++pass) {
      for (uint32_t j = lo + threadIdx.x; j < to; j += THREADS) {
        const uint32_t q = key_of(value(j));
        if ((q & mask) == known) atomicAdd(&sh.hist[pass][q >> at & 255], 1);
      }
      digit_of(sh, pass, a.blocks, want);
      known |= sh.digit << at;
      mask |= 255u << at;
      want -= sh.above;
      __syncthreads();
    }
    least = known;
    // of the values that tie, the `want` lowest places
    uint32_t place = 0;
    mask = 0;
    for (int at = 24; at >= 0; at -= 8, ++pass) {
      for (uint32_t j = lo + threadIdx.x; j < to; j += THREADS)
        if (key_of(value(j)) == least) {
          const uint32_t q = ~j;
          if ((q & mask) == place) atomicAdd(&sh.hist[pass][q >> at & 255], 1);
        }
      digit_of(sh, pass, a.blocks, want);
      place |= sh.digit << at;
      mask |= 255u << at;
      want -= sh.above;
      __syncthreads();
    }
    last = ~place;
  }
  auto kept = [&](float f, uint32_t j) {
    const uint32_t q = key_of(f);
    return q > KEY_LOST && (q > least || (q == least && j <= last));
  };
  // ---- the largest value and the sum relative to it
  float m = -INFINITY;
  for (uint32_t j = lo + threadIdx.x; j < to; j += THREADS) m = fmaxf(m, value(j));
#pragma unroll
  for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  if (lane == 0) sh.wmax[warp] = m;
  __syncthreads();
  m = sh.wmax[lane % WARPS];
#pragma unroll
  for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  float s = 0.f;
  uint32_t first = ~0u;
  for (uint32_t j = lo + threadIdx.x; j < to; j += THREADS) {
    const float f = value(j);
    if (greedy) {
      if (f == m) first = min(first, j);
    } else if (kept(f, j)) {
      s += share(f, m, c);
    }
  }
#pragma unroll
  for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
  first = __reduce_min_sync(~0u, first);
  if (lane == 0) sh.wsum[warp] = s, sh.wfirst[warp] = first;
  __syncthreads();
  if (warp == 0) {
    s = lane < WARPS ? sh.wsum[lane] : 0.f;
#pragma unroll
    for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
    first = __reduce_min_sync(~0u, lane < WARPS ? sh.wfirst[lane] : ~0u);
    if (lane == 0) sh.part_max = m, sh.part_sum = s, sh.part_first = first;
  }
  ppl::cluster_sync();
  float top = -INFINITY, total = 0.f;
  uint32_t best = ~0u;
  for (uint32_t b = 0; b < a.blocks; ++b) top = fmaxf(top, remote_f(&sh.part_max, b));
  for (uint32_t b = 0; b < a.blocks; ++b) {
    const float pm = remote_f(&sh.part_max, b);
    total += remote_f(&sh.part_sum, b) * share(pm, top, c);
    if (pm == top) best = min(best, remote_u(&sh.part_first, b));
  }
  ppl::cluster_sync();  // no block ends before the others have read it
  const float inv = total > 0.f ? 1.f / total : 0.f;
  for (uint32_t j = lo + threadIdx.x; j < to; j += THREADS) {
    const float f = value(j);
    float p;
    if (greedy) p = j == best && top > -INFINITY ? 1.f : 0.f;
    else p = kept(f, j) ? share(f, top, c) * inv : 0.f;
    out[j - shift] = p;
  }
}

template <class T>
cudaError_t launch(ProbArgs& a, uint64_t n_rows, cudaStream_t stream) {
  static ppi::DeviceOnce once;
  int dev;
  cudaError_t e = ppi::current_device(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&](int) {
    return cudaFuncSetAttribute(probs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(RESIDENT_MOST));
  });
  if (e != cudaSuccess) return e;
  constexpr uint32_t VEC = 16 / sizeof(T);
  const uint32_t n = a.n_vocab + VEC - 1;
  uint32_t blocks = 1;
  while (blocks < CLUSTER && ((n / blocks) * sizeof(T) > 65536 || (n_rows * blocks < 304 && n / (blocks * 2) >= 2048))) blocks *= 2;
  a.blocks = blocks;
  a.part = ((n + blocks - 1) / blocks + VEC - 1) / VEC * VEC;
  a.resident = a.part * sizeof(T) <= RESIDENT_MOST;
  cudaLaunchAttribute at;
  std::memset(&at, 0, sizeof at);
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(n_rows * blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = a.resident ? a.part * sizeof(T) : 0;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, probs_kernel<T>, static_cast<const ProbArgs>(a));
}

}  // namespace

extern "C" pp_rc pp_token_probs(const void* d_logits, pp_ftype type, size_t n_rows, size_t n_vocab,
                                size_t logits_stride, const float* d_temperature, const int32_t* d_top_k,
                                float* d_probs, size_t probs_stride, cudaStream_t stream) {
  if (!ppl::ftype_ok(type)) return PP_EINVAL;
  if (n_rows && n_vocab && (!d_logits || !d_probs)) return PP_EINVAL;
  if (n_rows > 1 && (probs_stride < n_vocab || (d_logits == d_probs && logits_stride != probs_stride))) return PP_EINVAL;
  if (d_logits && d_logits == d_probs && type != PP_F32) return PP_EINVAL;
  if (!ppl::aligned(d_logits, ppl::fsize(type)) || !ppl::aligned(d_probs, 4) || !ppl::aligned(d_temperature, 4) || !ppl::aligned(d_top_k, 4))
    return PP_EINVAL;
  if (n_rows >= ppl::MAX_DIM / CLUSTER || n_vocab >= (size_t(1) << 30)) return PP_ETOOLARGE;
  if (!n_rows || !n_vocab) return PP_OK;
  ProbArgs a;
  std::memset(&a, 0, sizeof a);
  a.in = d_logits;
  a.out = d_probs;
  a.temperature = d_temperature;
  a.top_k = d_top_k;
  a.in_stride = logits_stride;
  a.out_stride = probs_stride;
  a.n_vocab = uint32_t(n_vocab);
  cudaError_t e;
  switch (type) {
    case PP_F32: e = launch<float>(a, n_rows, stream); break;
    case PP_F16: e = launch<__half>(a, n_rows, stream); break;
    default: e = launch<__nv_bfloat16>(a, n_rows, stream); break;
  }
  return ppl::rc_of(e);
}
