// pp_logits: penalties for repeated tokens, biases and a grammar's mask on a
// model's logits, in one pass over them.
//
// A block takes one row's slice of the vocabulary.  It counts the row's
// history tokens that fall into its slice in shared memory (bit 31: the
// token was seen at all, bits 0-30: how often it was answered), keeps the
// last bias entry of each of its tokens there too, and then every thread
// turns its logits from registers.  The counts need no memory of their own
// and no second kernel, and no order of the atomics changes a count.
#include <algorithm>
#include <cstring>

#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using ppl::from_f;
using ppl::load_id;
using ppl::Pack;
using ppl::to_f;

constexpr int THREADS = 256;
constexpr uint32_t SEEN = 0x80000000u;

struct LogitArgs {
  const void* in;
  void* out;
  uint64_t in_stride, out_stride;
  uint32_t n_vocab, n_slices;
  uint32_t shift;  // VEC > 1: elements between a 16-byte boundary and row 0
  pp_logit_opts o;
};

// Rows start at any element, so a vector access begins at a multiple of VEC
// of a place counted from the last 16-byte boundary before the row: `lead`
// elements before column 0.
template <class T, int VEC>
__device__ __forceinline__ uint32_t row_lead(uint32_t shift, uint64_t stride, uint64_t row) {
  return uint32_t((shift + row * stride) % VEC);
}

__device__ __forceinline__ int64_t cut(int64_t x, int64_t hi) { return x < 0 ? 0 : x < hi ? x : hi; }

// counts[j] for the history tokens at columns first + j, j < size
__device__ void count_history(const pp_logit_opts& o, uint64_t row, int64_t first, uint32_t size,
                              uint32_t* counts) {
  const int64_t h = o.d_history_row ? o.d_history_row[row] : int64_t(row);
  if (h < 0 || uint64_t(h) >= o.history_rows) return;
  const int64_t len = o.d_history_len ? cut(o.d_history_len[row], o.history_cols) : o.history_cols;
  const int64_t given = o.d_prompt_len ? cut(o.d_prompt_len[row], o.history_cols) : 0;
  const uint64_t base = uint64_t(h) * o.history_stride;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < len; t += THREADS) {
    const int64_t tok = load_id(o.d_history, o.history_type, base + t);
    const int64_t j = tok - first;
    if (tok >= 0 && j >= 0 && j < size) {
      if (t >= given) atomicAdd(&counts[j], 1u);
      else atomicOr(&counts[j], SEEN);
    }
  }
}

// slot[j] = 1 + the last bias entry of column first + j
__device__ void find_biases(const pp_logit_opts& o, uint64_t row, int64_t first, uint32_t size,
                            uint32_t* slot) {
  const int64_t lo = cut(o.d_bias_offsets[row], o.n_bias), hi = cut(o.d_bias_offsets[row + 1], o.n_bias);
  for (int64_t e = lo + threadIdx.x; e < hi; e += THREADS) {
    const int64_t tok = o.d_bias_tokens[e], j = tok - first;
    if (tok >= 0 && j >= 0 && j < size) atomicMax(&slot[j], uint32_t(e + 1));
  }
}

template <class T, int VEC, int NV, bool HIST, bool BIAS, bool MASK>
__global__ void __launch_bounds__(THREADS) logits_kernel(const __grid_constant__ LogitArgs p) {
  constexpr uint32_t SLICE = THREADS * VEC * NV;
  extern __shared__ uint32_t sh[];
  uint32_t* counts = sh;
  uint32_t* slot = sh + (HIST ? SLICE : 0);
  const pp_logit_opts& o = p.o;
  const uint64_t row = blockIdx.x / p.n_slices;
  const uint32_t slice = blockIdx.x % p.n_slices;
  const uint32_t lead = VEC > 1 ? row_lead<T, VEC>(p.shift, p.in_stride, row) : 0;
  const int64_t first = int64_t(slice) * SLICE - lead;  // column of the slice's element 0
  const T* in = static_cast<const T*>(p.in) + row * p.in_stride;
  T* out = static_cast<T*>(p.out) + row * p.out_stride;
  const uint32_t* words = nullptr;
  if (MASK) {
    const uint32_t s = o.d_state[row * o.state_stride];
    if (s < uint32_t(o.n_states)) words = o.d_allowed + s * o.allowed_stride;
  }
  // the logits, ahead of everything that waits
  constexpr uint32_t ALL = (1u << VEC) - 1;
  Pack<T, VEC> x[NV];
  uint32_t need[NV];  // bit k: element k is a column that the grammar allows
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = first + int64_t(i * THREADS + threadIdx.x) * VEC;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (c + k >= 0 && c + k < p.n_vocab) m |= 1u << k;
    if (MASK && m) {
      uint32_t w = 0;
      if (words) {
        const int64_t b = c < 0 ? 0 : c;
        const uint32_t last = (p.n_vocab - 1) / 32, k = uint32_t(b / 32);
        w = __funnelshift_r(words[k], words[k < last ? k + 1 : k], uint32_t(b % 32)) << (b - c);
      }
      m &= w;
    }
    need[i] = m;
    if (m == ALL || (VEC > 1 && m && c >= 0 && c + VEC <= p.n_vocab)) {
      x[i] = *reinterpret_cast<const Pack<T, VEC>*>(in + c);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (m >> k & 1) x[i].v[k] = in[c + k];
    }
  }
  if (HIST || BIAS) {
    for (uint32_t j = threadIdx.x; j < SLICE * ((HIST ? 1 : 0) + (BIAS ? 1 : 0)); j += THREADS) sh[j] = 0;
    __syncthreads();
    if (HIST) count_history(o, row, first, SLICE, counts);
    if (BIAS) find_biases(o, row, first, SLICE, slot);
    __syncthreads();
  }
  const float rep = HIST && o.d_repetition ? o.d_repetition[row] : 1.f;
  const float pres = HIST && o.d_presence ? o.d_presence[row] : 0.f;
  const float freq = HIST && o.d_frequency ? o.d_frequency[row] : 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t j = (i * THREADS + threadIdx.x) * VEC;
    const int64_t c = first + j;
    Pack<T, VEC> y;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      y.v[k] = from_f<T>(-INFINITY);
      if (need[i] >> k & 1) {
        y.v[k] = x[i].v[k];
        const uint32_t n = HIST ? counts[j + k] : 0, e = BIAS ? slot[j + k] : 0;
        if (n | e) {
          float f = to_f(x[i].v[k]);
          if (n) {
            const float said = float(n & ~SEEN);
            f = f > 0.f ? f / rep : f * rep;
            if (n & ~SEEN) f = f - freq * said - pres;
          }
          if (e) f += o.d_bias_values[e - 1];
          y.v[k] = from_f<T>(f);
        }
      }
    }
    if (VEC == 1 || (c >= 0 && c + VEC <= p.n_vocab)) {
      if (VEC > 1 || c < p.n_vocab) *reinterpret_cast<Pack<T, VEC>*>(out + c) = y;
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (c + k >= 0 && c + k < p.n_vocab) out[c + k] = y.v[k];
    }
  }
}

template <class T, int VEC, int NV>
cudaError_t launch_kind(LogitArgs& p, uint64_t n_rows, bool hist, bool bias, bool mask,
                        cudaStream_t stream) {
  constexpr uint32_t SLICE = THREADS * VEC * NV;
  p.n_slices = uint32_t((uint64_t(p.n_vocab) + (VEC - 1) + SLICE - 1) / SLICE);
  const uint64_t blocks = n_rows * p.n_slices;
  if (blocks >= (uint64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  const size_t smem = SLICE * 4 * ((hist ? 1 : 0) + (bias ? 1 : 0));
  auto go = [&](auto kernel) {
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
      if (e != cudaSuccess) return e;
    }
    kernel<<<unsigned(blocks), THREADS, smem, stream>>>(p);
    return cudaGetLastError();
  };
  switch ((hist ? 4 : 0) + (bias ? 2 : 0) + (mask ? 1 : 0)) {
    case 0: return go(logits_kernel<T, VEC, NV, false, false, false>);
    case 1: return go(logits_kernel<T, VEC, NV, false, false, true>);
    case 2: return go(logits_kernel<T, VEC, NV, false, true, false>);
    case 3: return go(logits_kernel<T, VEC, NV, false, true, true>);
    case 4: return go(logits_kernel<T, VEC, NV, true, false, false>);
    case 5: return go(logits_kernel<T, VEC, NV, true, false, true>);
    case 6: return go(logits_kernel<T, VEC, NV, true, true, false>);
    default: return go(logits_kernel<T, VEC, NV, true, true, true>);
  }
}

template <class T>
cudaError_t launch_type(LogitArgs& p, uint64_t n_rows, bool hist, bool bias, bool mask,
                        cudaStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  // 16-byte accesses need input and output rows at the same place of a
  // 16-byte line; any other pair goes element by element
  const uint64_t a = reinterpret_cast<uintptr_t>(p.in) / sizeof(T) % VEC;
  const uint64_t b = reinterpret_cast<uintptr_t>(p.out) / sizeof(T) % VEC;
  if (a == b && (n_rows == 1 || p.in_stride % VEC == p.out_stride % VEC)) {
    p.shift = uint32_t(a);
    return launch_kind<T, VEC, 2>(p, n_rows, hist, bias, mask, stream);
  }
  return launch_kind<T, 1, 8>(p, n_rows, hist, bias, mask, stream);
}

}  // namespace

extern "C" pp_rc pp_logits(const void* d_in, pp_ftype type, size_t n_rows, size_t n_vocab,
                           size_t in_stride, const pp_logit_opts* opts, void* d_out,
                           size_t out_stride, cudaStream_t stream) {
  if (!ppl::ftype_ok(type)) return PP_EINVAL;
  if (n_rows && n_vocab && (!d_in || !d_out)) return PP_EINVAL;
  if (n_rows > 1 && (out_stride < n_vocab || (d_in == d_out && in_stride != out_stride))) return PP_EINVAL;
  if (!ppl::aligned(d_in, ppl::fsize(type)) || !ppl::aligned(d_out, ppl::fsize(type))) return PP_EINVAL;
  LogitArgs p;
  std::memset(&p, 0, sizeof p);
  if (opts) p.o = *opts;
  const pp_logit_opts& o = p.o;
  if (o.d_history) {
    if (!ppl::itype_ok(o.history_type)) return PP_EINVAL;
    if (o.history_cols >= ppl::MAX_DIM || o.history_rows >= ppl::MAX_DIM) return PP_ETOOLARGE;
  }
  const bool bias = o.d_bias_offsets && o.n_bias;
  if (bias && (!o.d_bias_tokens || !o.d_bias_values)) return PP_EINVAL;
  if (o.n_bias >= ppl::MAX_DIM) return PP_ETOOLARGE;
  const bool mask = o.d_allowed != nullptr;
  if (mask && (!o.d_state || o.n_states < 1 || o.n_states > PP_MAX_STATES ||
               o.allowed_stride < (n_vocab + 31) / 32))
    return PP_EINVAL;
  if (n_rows >= ppl::MAX_DIM || n_vocab >= ppl::MAX_DIM) return PP_ETOOLARGE;
  if (!n_rows || !n_vocab) return PP_OK;
  p.in = d_in;
  p.out = d_out;
  p.in_stride = in_stride;
  p.out_stride = out_stride;
  p.n_vocab = uint32_t(n_vocab);
  const bool hist = o.d_history && o.history_cols && (o.d_repetition || o.d_presence || o.d_frequency);
  cudaError_t e;
  switch (type) {
    case PP_F32: e = launch_type<float>(p, n_rows, hist, bias, mask, stream); break;
    case PP_F16: e = launch_type<__half>(p, n_rows, hist, bias, mask, stream); break;
    default: e = launch_type<__nv_bfloat16>(p, n_rows, hist, bias, mask, stream); break;
  }
  if (e == cudaErrorInvalidConfiguration) return PP_ETOOLARGE;
  return ppl::rc_of(e);
}
