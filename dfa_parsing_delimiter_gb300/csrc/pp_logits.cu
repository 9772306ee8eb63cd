// pp_logits: penalties for repeated tokens, biases and a grammar's mask on a
// model's logits, in one pass over them.
//
// A block takes one row's slice of the vocabulary, a thread's first logits
// already on their way while the row's history is counted in shared memory: a
// bit for each token of the slice that was seen, and how often it was
// answered.  Then the slice streams by in 16-byte vectors that only meet the
// mask, and last the marked logits, a thread each, are turned and written
// over.  They are read again for that: what the grammar allows has just been
// written unchanged, so it is there also if the result takes the logits'
// place.  The counts need no memory of their own and no second kernel, and no
// order of the atomics changes a count.
//
// 512 rows of 131075 f16 with histories of up to 8191, biases and a grammar
// take 79 us, of which the stream alone is 44 (its 268 MB at the copy rate:
// 40), the mask 4, counting and turning 25 and the biases 7; bound by the
// latency of a block's steps one after the other, so many blocks at once (four
// on a multiprocessor) count for more than loads in flight in each.
//
// What was measured against it (512 rows of 131075 f16, histories of 8191,
// biases, a grammar): turning marked elements within their vectors takes 8
// times the instructions, since at 2 in 100 marked nearly every warp has one;
// sharing the history among a cluster's blocks, which count in each other's
// shared memory, 272 us against 144 us for every block reading all of it.
#include <algorithm>
#include <cstring>

#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using ppl::from_f;
using ppl::to_f;

constexpr int THREADS = 512, BLOCKS = 4;  // a multiprocessor
constexpr int NV = 2;  // vectors that a thread holds

struct LogitArgs {
  const void* in;
  void* out;
  uint64_t in_stride, out_stride;
  uint32_t n_vocab;
  uint32_t shift;     // VEC > 1: elements between a 16-byte boundary and row 0
  uint32_t slice;     // elements a block takes, a multiple of 128
  uint32_t n_slices;  // of a row
  pp_logit_opts o;
};

__device__ __forceinline__ int64_t cut(int64_t x, int64_t hi) { return x < 0 ? 0 : x < hi ? x : hi; }

// How often each of a slice's tokens was answered, HIST bits each (16, for
// histories of fewer than 2^16 tokens, or 32); 0: there is no history.
template <int HIST>
struct Counts {
  static __host__ __device__ constexpr uint32_t words(uint32_t slice) { return HIST == 16 ? slice / 2 : HIST ? slice : 0; }
  static __device__ __forceinline__ void add(uint32_t* c, uint32_t j) {
    if (HIST == 16) atomicAdd(c + j / 2, j & 1 ? 0x10000u : 1u);
    else atomicAdd(c + j, 1u);
  }
  static __device__ __forceinline__ uint32_t get(const uint32_t* c, uint32_t j) {
    return HIST == 16 ? reinterpret_cast<const uint16_t*>(c)[j] : c[j];
  }
};

// A row's history: where it is, its length, and how much of it was given.
struct History {
  const char* line;
  uint32_t len, given;
};
__device__ __forceinline__ History history_of(const pp_logit_opts& o, uint64_t row) {
  const int64_t h = o.d_history_row ? o.d_history_row[row] : int64_t(row);
  History r;
  r.len = uint32_t(o.d_history_len ? cut(o.d_history_len[row], o.history_cols) : o.history_cols);
  r.given = uint32_t(o.d_prompt_len ? cut(o.d_prompt_len[row], o.history_cols) : 0);
  if (h < 0 || uint64_t(h) >= o.history_rows || !o.d_history) r.len = 0;
  r.line = static_cast<const char*>(o.d_history) +
           uint64_t(h) * o.history_stride * (o.history_type == PP_I64 ? 8 : o.history_type == PP_I32 ? 4 : 1);
  return r;
}

// A row's biases.
struct Biases {
  const int32_t* tokens;
  const float* values;
  uint32_t n;
};
__device__ __forceinline__ Biases biases_of(const pp_logit_opts& o, uint64_t row) {
  if (!o.d_bias_offsets) return {nullptr, nullptr, 0};
  const int64_t lo = cut(o.d_bias_offsets[row], o.n_bias), hi = cut(o.d_bias_offsets[row + 1], o.n_bias);
  return {o.d_bias_tokens + lo, o.d_bias_values + lo, hi > lo ? uint32_t(hi - lo) : 0};
}

template <int HIST>
__device__ __forceinline__ void count_history(const History& h, int type, int first, uint32_t size, uint32_t* counts,
                                              uint32_t* marks) {
  ppl::for_ids<4>(h.line, type, 1, threadIdx.x, h.len, THREADS, [&](uint32_t t, auto tok) {
    if (sizeof(tok) == 8 && uint64_t(tok) >= 0x7FFFFFFFu) return;
    const uint32_t j = uint32_t(tok) - uint32_t(first);  // before the slice: past its end
    if (j >= size) return;
    atomicOr(&marks[j / 32], 1u << (j % 32));
    if (t >= h.given) Counts<HIST>::add(counts, j);
  });
}

// -infinity in a word of a 16-byte vector.
template <class T> struct Bits;
template <> struct Bits<float> { static constexpr uint32_t NEG = 0xFF800000u; };
template <> struct Bits<__half> { static constexpr uint32_t NEG = 0xFC00FC00u; };
template <> struct Bits<__nv_bfloat16> { static constexpr uint32_t NEG = 0xFF80FF80u; };

// -infinity where bit k of need is 0.  Of 16-bit elements a word holds two:
// four bits of need go to the signs of four bytes, and a byte permute spreads
// two of the signs over the word's halves.
template <class T>
__device__ __forceinline__ uint4 forbid(uint4 v, uint32_t need) {
  uint32_t keep[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int q = 0; q < 4; ++q) keep[q] = 0u - (need >> q & 1);
  } else {
    const uint32_t lo = (need & 15) * 0x10204080u, hi = (need >> 4) * 0x10204080u;
    asm("prmt.b32 %0, %1, %1, 0x9988;" : "=r"(keep[0]) : "r"(lo));
    asm("prmt.b32 %0, %1, %1, 0xBBAA;" : "=r"(keep[1]) : "r"(lo));
    asm("prmt.b32 %0, %1, %1, 0x9988;" : "=r"(keep[2]) : "r"(hi));
    asm("prmt.b32 %0, %1, %1, 0xBBAA;" : "=r"(keep[3]) : "r"(hi));
  }
  const uint32_t neg = Bits<T>::NEG;
  return make_uint4((v.x & keep[0]) | (neg & ~keep[0]), (v.y & keep[1]) | (neg & ~keep[1]),
                    (v.z & keep[2]) | (neg & ~keep[2]), (v.w & keep[3]) | (neg & ~keep[3]));
}

// The 32 bits of `bits` from column c on (c > -32).
__device__ __forceinline__ uint32_t allowed_from(const uint32_t* bits, int c, int n_vocab) {
  if (c < 0) return bits[0] << -c;
  const uint32_t w = uint32_t(c) / 32, last = uint32_t(n_vocab - 1) / 32;
  return __funnelshift_r(bits[w], bits[min(w + 1, last)], c);
}

// f(j) for the set bits j of marks that `without` (if any) has not, restricted
// to columns that exist and that `bits` (if masked) allows; first: the column
// of bit 0.  A warp takes 64
// words at a time, two a lane, and deals their set bits out to its lanes.
template <class F>
__device__ __forceinline__ void for_marked(const uint32_t* marks, const uint32_t* without, uint32_t n_words, int first, int n_vocab, bool masked,
                                           const uint32_t* bits, F&& f) {
  const int lane = threadIdx.x & 31;
  for (uint32_t w0 = threadIdx.x / 32 * 64; w0 < n_words; w0 += THREADS * 2) {
    uint32_t set[2] = {0, 0};
    if (w0 + 2 * lane < n_words) {
      const uint2 two = *reinterpret_cast<const uint2*>(marks + w0 + 2 * lane);
      set[0] = two.x;
      set[1] = two.y;
      if (without) {
        set[0] &= ~without[w0 + 2 * lane];
        set[1] &= ~without[w0 + 2 * lane + 1];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (set[h]) {
        const int c = first + int(w0 + 2 * lane + h) * 32;
        if (c < 0) set[h] &= c > -32 ? ~0u << -c : 0;
        if (c + 32 > n_vocab) set[h] &= c < n_vocab ? ~0u >> (c + 32 - n_vocab) : 0;
        if (masked && set[h]) set[h] &= bits ? allowed_from(bits, c, n_vocab) : 0;
      }
    const uint32_t half = __popc(set[0]), own = half + __popc(set[1]);
    uint32_t upto = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t up = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += up;
    }
    const uint32_t all = __shfl_sync(~0u, upto, 31), halves = (upto - own) << 8 | half;
    for (uint32_t i0 = 0; i0 < all; i0 += 32) {
      const uint32_t i = i0 + lane;
      int q = 0;  // the lane that has the i-th set bit: the first with upto > i
#pragma unroll
      for (int d = 16; d; d /= 2)
        if (__shfl_sync(~0u, upto, q + d - 1) <= i) q += d;
      const uint32_t of = __shfl_sync(~0u, halves, q & 31);
      const uint32_t a = __shfl_sync(~0u, set[0], q & 31), b = __shfl_sync(~0u, set[1], q & 31);
      uint32_t nth = i - (of >> 8);
      const bool second = nth >= (of & 0xFF);
      if (second) nth -= of & 0xFF;
      if (i < all) {
        uint32_t word = second ? b : a;
        int k = second ? 32 : 0;  // its nth set bit
#pragma unroll
        for (int d = 16; d; d /= 2) {
          const uint32_t low = __popc(word & ((1u << d) - 1));
          if (nth >= low) {
            nth -= low;
            word >>= d;
            k += d;
          }
        }
        f(int((w0 + 2 * q) * 32 + k));
      }
      __syncwarp();
    }
  }
}

// A logit under its row's penalties; said: how often its token was answered.
struct Penalties {
  float rep, pres, freq;
  __device__ __forceinline__ Penalties(const pp_logit_opts& o, bool history, uint64_t row)
      : rep(history && o.d_repetition ? o.d_repetition[row] : 1.f),
        pres(history && o.d_presence ? o.d_presence[row] : 0.f),
        freq(history && o.d_frequency ? o.d_frequency[row] : 0.f) {}
  __device__ __forceinline__ float on(float f, uint32_t said) const {
    f = f > 0.f ? f / rep : f * rep;
    return said ? f - freq * float(said) - pres : f;
  }
};

// The biases of a row some of whose tokens have several entries, of which the
// last counts: THREADS of the list at a time, from its end, and a bit for each
// token that a later lot had.  Entries of one lot for one token clash on their
// bit; only those are compared with the lot's later entries, a warp for each.
// So this is linear in the list, where a search of what follows each entry
// took 102 ms for 100000 entries with one pair among them (75 us without a
// pair, 132 us with it).  As a function of its own it costs every row of the
// kernel with biases 1 % (its calls' stack), inlined nothing.
template <class T, int HIST>
__device__ __forceinline__ void repeated_biases(const LogitArgs& p, uint64_t row, int first, uint32_t* counts) {
  const uint32_t n_marks = p.slice / 32, lane = threadIdx.x & 31;
  const uint32_t* marks = counts + Counts<HIST>::words(p.slice);
  uint32_t* done = counts + Counts<HIST>::words(p.slice) + (HIST ? n_marks : 0);
  const T* in = static_cast<const T*>(p.in) + row * p.in_stride;
  T* out = static_cast<T*>(p.out) + row * p.out_stride;
  const uint32_t* bits = nullptr;
  if (p.o.d_allowed) {
    const uint32_t s = p.o.d_state[row * p.o.state_stride];
    if (s < uint32_t(p.o.n_states)) bits = p.o.d_allowed + s * p.o.allowed_stride;
  }
  const Biases bias = biases_of(p.o, row);
  const Penalties pen(p.o, HIST != 0, row);
  for (uint32_t w = threadIdx.x; w < n_marks; w += THREADS) done[w] = 0;
  __syncthreads();
  for (uint32_t top = bias.n, base; top; top = base) {
    base = top > THREADS ? top - THREADS : 0;
    const uint32_t e = base + threadIdx.x;
    const int tok = e < top ? bias.tokens[e] : -1;
    const uint32_t j = uint32_t(tok) - uint32_t(first), bit = 1u << (j % 32);
    bool last = tok >= 0 && tok < int(p.n_vocab) && j < p.slice && !(done[j / 32] & bit);
    __syncthreads();
    const bool clash = last && atomicOr(&done[j / 32], bit) & bit;
    if (__syncthreads_or(clash)) {
      if (clash) atomicAnd(&done[j / 32], ~bit);  // now clear for all entries of such a token
      __syncthreads();
      const bool shared = last && !(done[j / 32] & bit);
      __syncthreads();
      if (shared) atomicOr(&done[j / 32], bit);
      for (uint32_t todo = __ballot_sync(~0u, shared); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1, same = __shfl_sync(~0u, tok, src);
        bool later = false;
        for (uint32_t k = e + src + 1; k < top; k += 32) later |= bias.tokens[k] == same;
        if (__any_sync(~0u, later) && int(lane) == src) last = false;
      }
      __syncthreads();
    }
    if (last && (!p.o.d_allowed || (bits && (bits[uint32_t(tok) / 32] >> (tok & 31) & 1)))) {
      float f = to_f(in[tok]);
      if (HIST && marks[j / 32] >> (j % 32) & 1) f = pen.on(f, Counts<HIST>::get(counts, j));
      out[tok] = from_f<T>(f + bias.values[e]);
    }
  }
}

// Rows start at any element, so a vector access begins at a multiple of VEC
// of a place counted from the last 16-byte boundary before the row, `lead`
// elements before column 0; a row's incomplete first and last vectors go
// element by element, as everything does with VEC 1.
template <class T, int VEC, int HIST, bool BIAS, bool MASK>
__global__ void __launch_bounds__(THREADS, BLOCKS) logits_kernel(const __grid_constant__ LogitArgs p) {
  constexpr uint32_t ALL = (1u << VEC) - 1;
  using C = Counts<HIST>;
  extern __shared__ __align__(16) uint32_t counts[];
  __shared__ uint32_t twice;  // some token has several bias entries
  const uint32_t n_marks = p.slice / 32;
  uint32_t* marks = counts + C::words(p.slice);        // tokens of the history
  uint32_t* biased = marks + (HIST ? n_marks : 0);     // tokens with a bias
  const pp_logit_opts& o = p.o;
  const uint64_t row = blockIdx.x / p.n_slices;
  const uint32_t nth = blockIdx.x - uint32_t(row) * p.n_slices;
  const int lead = VEC > 1 ? int((p.shift + row * p.in_stride) % VEC) : 0;
  const int n_vocab = int(p.n_vocab);
  const int first = int(nth * p.slice) - lead;  // column of the slice's element 0
  const T* in = static_cast<const T*>(p.in) + row * p.in_stride;
  T* out = static_cast<T*>(p.out) + row * p.out_stride;
  const bool masked = MASK && o.d_allowed;
  const uint32_t* bits = nullptr;
  if (masked) {
    const uint32_t s = o.d_state[row * o.state_stride];
    if (s < uint32_t(o.n_states)) bits = o.d_allowed + s * o.allowed_stride;
  }

  History h;
  if (HIST) h = history_of(o, row);
  Biases bias = {};
  if (BIAS) bias = biases_of(o, row);

  // the complete vectors of the row that this slice holds: v_lo .. v_hi - 1
  const int n_vec = int(p.slice) / VEC;
  const int v_lo = first < 0 ? 1 : 0, v_hi = min(n_vec, (n_vocab - first) / VEC);
  // this thread's first one, and how many vectors from there to v_hi; its
  // vectors are THREADS apart, whole words of bits, so that its place within
  // a word stays
  const int c_first = first + (v_lo + int(threadIdx.x)) * VEC;
  int left = VEC > 1 ? v_hi - v_lo - int(threadIdx.x) : 0;
  const uint4* src = reinterpret_cast<const uint4*>(in + c_first);
  uint4* dst = reinterpret_cast<uint4*>(out + c_first);
  const uint32_t* word = bits + uint32_t(c_first) / 32;
  const uint32_t shift = uint32_t(c_first) % 32;
  const bool across = shift + VEC > 32;  // into the next word
  uint4 x[NV];
  uint32_t need[NV];  // bit k: the grammar allows element k
  // what the grammar forbids is not even read
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * THREADS < left) {
        need[i] = ALL;
        if (masked) {
          uint32_t lo = 0, hi = 0;
          if (bits) {
            lo = word[i * (THREADS * VEC / 32)];
            if (across) hi = word[i * (THREADS * VEC / 32) + 1];
          }
          need[i] = __funnelshift_r(lo, hi, shift) & ALL;
        }
        if (need[i]) x[i] = src[i * THREADS];
      }
  };
  if (VEC > 1) load();
  if (HIST || BIAS) {
    const uint32_t n = C::words(p.slice) + n_marks * ((HIST ? 1 : 0) + (BIAS ? 1 : 0));  // a multiple of 4
    for (uint32_t j = threadIdx.x * 4; j < n; j += THREADS * 4)
      *reinterpret_cast<uint4*>(counts + j) = make_uint4(0, 0, 0, 0);
    if (BIAS && threadIdx.x == 0) twice = 0;
    __syncthreads();
    if (BIAS)
      ppl::for_ids_of<1>(bias.tokens, 1, THREADS - 1 - threadIdx.x, bias.n, THREADS, [&](uint32_t, int32_t tok) {
        const uint32_t j = uint32_t(tok) - uint32_t(first);
        if (tok < 0 || j >= p.slice) return;
        if (atomicOr(&biased[j / 32], 1u << (j % 32)) >> (j % 32) & 1) twice = 1;
      });
    if (HIST) count_history<HIST>(h, o.history_type, first, p.slice, counts, marks);
  }
  // element j of the slice by itself
  auto single = [&](int j) {
    const int c = first + j;
    if (c < 0 || c >= n_vocab) return;
    const bool fine = !masked || (bits && (bits[uint32_t(c) / 32] >> (c & 31) & 1));
    out[c] = fine ? in[c] : from_f<T>(-INFINITY);
  };
  if (VEC == 1)
    for (int j = threadIdx.x; j < int(p.slice); j += THREADS) single(j);
  while (VEC > 1 && left > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * THREADS < left) dst[i * THREADS] = masked ? forbid<T>(x[i], need[i]) : x[i];
    src += NV * THREADS;
    dst += NV * THREADS;
    word += NV * THREADS * VEC / 32;
    left -= NV * THREADS;
    load();
  }
  if (VEC > 1) {  // the incomplete vectors: before v_lo and from v_hi on
    if (first < 0 && int(threadIdx.x) < VEC) single(threadIdx.x);
    if (v_hi < n_vec && v_hi >= v_lo && int(threadIdx.x) >= THREADS - VEC) single(v_hi * VEC + threadIdx.x - (THREADS - VEC));
  }
  if (!HIST && !BIAS) return;
  __syncthreads();
  const Penalties pen(o, HIST != 0, row);
  auto turn = [&](int j, bool seen) {
    const float f = to_f(in[first + j]);
    return HIST && seen ? pen.on(f, C::get(counts, j)) : f;
  };
  if (HIST)  // but for tokens with a bias, which come next
    for_marked(marks, BIAS ? biased : nullptr, n_marks, first, n_vocab, masked, bits,
               [&](int j) { out[first + j] = from_f<T>(turn(j, true)); });
  if (BIAS && twice) {
    __syncthreads();  // the marked logits are done with the bits of the biases
    repeated_biases<T, HIST>(p, row, first, counts);
  } else if (BIAS) {
    bias = biases_of(o, row);  // again, rather than kept in registers meanwhile
    // from the last thread on: the first warps have the marks
    for (uint32_t e = THREADS - 1 - threadIdx.x; e < bias.n; e += THREADS) {
      const int tok = bias.tokens[e];
      const uint32_t j = uint32_t(tok) - uint32_t(first);
      if (tok < 0 || tok >= n_vocab || j >= p.slice) continue;
      if (masked && !(bits && (bits[uint32_t(tok) / 32] >> (tok & 31) & 1))) continue;
      out[tok] = from_f<T>(turn(j, HIST && marks[j / 32] >> (j % 32) & 1) + bias.values[e]);
    }
  }
}

constexpr uint32_t SLICE_MOST = 24576 + 128;  // 55 KiB with counts of 16 bits: BLOCKS of them fit
constexpr uint32_t SLICE_LEAST = 1024;
constexpr size_t SMEM_MOST = SLICE_MOST * 4 + SLICE_MOST / 4;

template <class T, int VEC, int HIST, bool BIAS, bool MASK>
cudaError_t launch_one(const LogitArgs& p, uint64_t blocks, cudaStream_t stream) {
  static ppi::DeviceOnce once;
  auto kernel = logits_kernel<T, VEC, HIST, BIAS, MASK>;
  int dev;
  cudaError_t e = ppi::current_device(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&](int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM_MOST));
  });
  if (e != cudaSuccess) return e;
  const size_t smem = 4 * (Counts<HIST>::words(p.slice) + p.slice / 32 * ((HIST ? 1 : 0) + (BIAS ? 1 : 0)));
  kernel<<<unsigned(blocks), THREADS, smem, stream>>>(p);
  return cudaGetLastError();
}

template <class T, int VEC>
cudaError_t launch_kind(LogitArgs& p, uint64_t n_rows, int hist, bool bias, bool mask, cudaStream_t stream) {
  // Slices of up to SLICE_MOST tokens, since every block reads its row's
  // history; smaller ones where there are few rows, as many as run at once
  // (four on each of 152 multiprocessors; for 64 rows of 131072, 9 slices
  // take 10.9 us and 14, two waves, 14.6), but none of fewer than SLICE_LEAST
  // tokens.
  const uint64_t n = uint64_t(p.n_vocab) + VEC - 1;
  const uint64_t s = std::max((n + 24575) / 24576, std::min(std::max<uint64_t>(608 / n_rows, 1), (n + SLICE_LEAST - 1) / SLICE_LEAST));
  p.slice = uint32_t(((n + s - 1) / s + 127) / 128 * 128);  // whole words of marks, in fours
  p.n_slices = uint32_t((n + p.slice - 1) / p.slice);
  const uint64_t blocks = n_rows * p.n_slices;
  if (blocks >= (uint64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  if constexpr (VEC == 1) {  // the rare pair of unlike alignments: one kernel for all
    return launch_one<T, 1, 32, true, true>(p, blocks, stream);
  } else {
    switch (hist / 16 * 4 + (bias ? 2 : 0) + (mask ? 1 : 0)) {
      case 0: return launch_one<T, VEC, 0, false, false>(p, blocks, stream);
      case 1: return launch_one<T, VEC, 0, false, true>(p, blocks, stream);
      case 2: return launch_one<T, VEC, 0, true, false>(p, blocks, stream);
      case 3: return launch_one<T, VEC, 0, true, true>(p, blocks, stream);
      case 4: return launch_one<T, VEC, 16, false, false>(p, blocks, stream);
      case 5: return launch_one<T, VEC, 16, false, true>(p, blocks, stream);
      case 6: return launch_one<T, VEC, 16, true, false>(p, blocks, stream);
      case 7: return launch_one<T, VEC, 16, true, true>(p, blocks, stream);
      case 8: return launch_one<T, VEC, 32, false, false>(p, blocks, stream);
      case 9: return launch_one<T, VEC, 32, false, true>(p, blocks, stream);
      case 10: return launch_one<T, VEC, 32, true, false>(p, blocks, stream);
      default: return launch_one<T, VEC, 32, true, true>(p, blocks, stream);
    }
  }
}

template <class T>
cudaError_t launch_type(LogitArgs& p, uint64_t n_rows, int hist, bool bias, bool mask, cudaStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  // 16-byte accesses need input and output rows at the same place of a
  // 16-byte line; any other pair goes element by element
  const uint64_t a = reinterpret_cast<uintptr_t>(p.in) / sizeof(T) % VEC;
  const uint64_t b = reinterpret_cast<uintptr_t>(p.out) / sizeof(T) % VEC;
  if (a == b && (n_rows == 1 || p.in_stride % VEC == p.out_stride % VEC)) {
    p.shift = uint32_t(a);
    return launch_kind<T, VEC>(p, n_rows, hist, bias, mask, stream);
  }
  return launch_kind<T, 1>(p, n_rows, hist, bias, mask, stream);
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
  const bool some = o.d_bias_offsets && o.n_bias;
  if (some && (!o.d_bias_tokens || !o.d_bias_values)) return PP_EINVAL;
  if (o.n_bias >= ppl::MAX_DIM) return PP_ETOOLARGE;
  const bool mask = o.d_allowed != nullptr;
  if (mask && (!o.d_state || o.n_states < 1 || o.n_states > PP_MAX_STATES ||
               o.allowed_stride < (n_vocab + 31) / 32))
    return PP_EINVAL;
  if (n_rows >= ppl::MAX_DIM || n_vocab >= (size_t(1) << 30)) return PP_ETOOLARGE;
  if (!n_rows || !n_vocab) return PP_OK;
  if (o.d_history && !ppl::aligned(o.d_history, ppl::isize(o.history_type))) return PP_EINVAL;
  for (const void* four : {static_cast<const void*>(o.d_history_row), static_cast<const void*>(o.d_history_len),
                           static_cast<const void*>(o.d_prompt_len), static_cast<const void*>(o.d_repetition),
                           static_cast<const void*>(o.d_presence), static_cast<const void*>(o.d_frequency),
                           static_cast<const void*>(o.d_bias_offsets), static_cast<const void*>(o.d_bias_tokens),
                           static_cast<const void*>(o.d_bias_values), static_cast<const void*>(o.d_allowed)})
    if (!ppl::aligned(four, 4)) return PP_EINVAL;
  p.in = d_in;
  p.out = d_out;
  p.in_stride = in_stride;
  p.out_stride = out_stride;
  p.n_vocab = uint32_t(n_vocab);
  int hist = 0;
  if (o.d_history && o.history_cols && (o.d_repetition || o.d_presence || o.d_frequency)) hist = o.history_cols < 0x10000 ? 16 : 32;
  else p.o.d_history = nullptr;
  const bool bias = some;
  if (!bias) p.o.d_bias_offsets = nullptr;
  cudaError_t e;
  switch (type) {
    case PP_F32: e = launch_type<float>(p, n_rows, hist, bias, mask, stream); break;
    case PP_F16: e = launch_type<__half>(p, n_rows, hist, bias, mask, stream); break;
    default: e = launch_type<__nv_bfloat16>(p, n_rows, hist, bias, mask, stream); break;
  }
  if (e == cudaErrorInvalidConfiguration) return PP_ETOOLARGE;
  return ppl::rc_of(e);
}
