// pp_token_probs: a model's logits as probabilities, by a temperature and cut
// to each row's k most likely tokens.
//
// A row is read once and written once: bound by memory, at six or eight bytes a
// token.  A cluster of blocks shares it, since a block cannot hold a long row, and
// holds it on the chip between the reading and the writing:
//
//   plain_kernel  rows without a cut.  Parts lie in shared memory; largest value,
//                 sum of exponentials relative to it, one exchange of the two
//                 through distributed shared memory, probabilities.  2560 rows of
//                 50001 f32: 173 us (5.9 TB/s; with the parts in registers, two
//                 blocks a multiprocessor, 213 at the time), 512 of 131075 bf16: 73.
//   cut_kernel    rows with a cut.  Parts lie in registers (in shared memory the
//                 steps below read them again each time: 512 rows of 131075 f16 111
//                 us instead of 104, 64 rows of 131072 bf16 24 instead of 19).  At
//                 least k values of a row reach the least of the blocks' k_part-th
//                 largest thread maxima, and not many more: those are listed, and
//                 every block finds the k-th largest in all lists, digit by digit
//                 of its bits in the order of values, then, of values that tie, the
//                 last place that is kept.  All else is zero and is written before.
//                 Bound by the latency of a block's steps one after the other (some
//                 twenty barriers, three of them of the cluster).
//   long_kernel   rows that eight blocks cannot hold: the steps read them again
//                 (64 rows of 900001 bf16 297 us, with a cut 1130).
//
// Which tokens are kept is exact, whatever 32 bits make of the exponentials.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using ppl::from_f;
using ppl::to_f;

constexpr int LONG_THREADS = 512, LONG_WARPS = LONG_THREADS / 32;
constexpr int CLUSTER = 8;   // blocks at most
constexpr int MID = 512;     // threads of a block that has a part of a longer row
constexpr int LARGE = 1024;  // and of the longest rows with a cut
constexpr int NV_MOST = 9;   // 16-byte vectors of a thread, in registers
// Bytes of a part in shared memory, so that four blocks share a multiprocessor: 512 rows
// of 80000 f32 60 us by six blocks, 65 by five of 62 KiB and 71 by eight; 2560 of 50001 f32
// 173 by four, 182 by three of 65 KiB; but 512 of 131075 f32 107 by eight and 104 by seven
// of 73 KiB.  Three share one where one block or two then hold the row: 4096 rows of 32000
// f32 174 us by two blocks, 190 by three, and bf16 123 by one, 140 by two.
constexpr uint32_t PART_MOST = 56320, PART_OF_TWO = 66048;
constexpr uint32_t RESIDENT_MOST = 200 * 1024;  // where a block has a multiprocessor for itself

struct ProbArgs {
  const void* in;
  float* out;
  const float* temperature;
  const int32_t* top_k;
  uint64_t in_stride, out_stride;
  uint32_t n_vocab, n_rows, blocks, part;
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

// ------------------------------------------------------------ rows of any length
struct Shared {
  float part_max, part_sum;
  uint32_t part_first;  // the first token with part_max
  float wmax[LONG_WARPS], wsum[LONG_WARPS];
  uint32_t wfirst[LONG_WARPS];
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
__global__ void __launch_bounds__(LONG_THREADS) long_kernel(const ProbArgs a) {
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
    for (uint32_t v = threadIdx.x * VEC; v < a.part; v += LONG_THREADS * VEC) {
      const uint32_t j = from + v;
      if (j >= shift && j + VEC <= all) {
        *reinterpret_cast<uint4*>(buf + v) = *reinterpret_cast<const uint4*>(in - shift + j);
      } else {
        for (int k = 0; k < VEC; ++k)
          if (j + k >= shift && j + k < all) buf[v + k] = in[j + k - shift];
      }
    }
    for (uint32_t i = threadIdx.x; i < 8 * 256; i += LONG_THREADS) sh.hist[i / 256][i % 256] = 0;
    __syncthreads();
  } else {
    for (uint32_t i = threadIdx.x; i < 8 * 256; i += LONG_THREADS) sh.hist[i / 256][i % 256] = 0;
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
      for (uint32_t j = lo + threadIdx.x; j < to; j += LONG_THREADS) {
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
      for (uint32_t j = lo + threadIdx.x; j < to; j += LONG_THREADS)
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
  for (uint32_t j = lo + threadIdx.x; j < to; j += LONG_THREADS) m = fmaxf(m, value(j));
#pragma unroll
  for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  if (lane == 0) sh.wmax[warp] = m;
  __syncthreads();
  m = sh.wmax[lane % LONG_WARPS];
#pragma unroll
  for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  float s = 0.f;
  uint32_t first = ~0u;
  for (uint32_t j = lo + threadIdx.x; j < to; j += LONG_THREADS) {
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
    s = lane < LONG_WARPS ? sh.wsum[lane] : 0.f;
#pragma unroll
    for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
    first = __reduce_min_sync(~0u, lane < LONG_WARPS ? sh.wfirst[lane] : ~0u);
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
  for (uint32_t j = lo + threadIdx.x; j < to; j += LONG_THREADS) {
    const float f = value(j);
    float p;
    if (greedy) p = j == best && top > -INFINITY ? 1.f : 0.f;
    else p = kept(f, j) ? share(f, top, c) * inv : 0.f;
    out[j - shift] = p;
  }
}

// ------------------------------------------------------------ rows with a cut
constexpr int entries_of(int threads) { return threads > 128 ? 4 : 8; }  // listed candidates a thread

// The THREADS threads of a row: a block, or for short rows one of its groups.
// Groups that begin together run the same instructions at nearly the same
// time, which matters here: the code is long and straight, and warps at other
// places in it wait for one another's instructions (8192 rows of 5000 bf16: 162 us
// four to a block, 184 in blocks of their own, at the time; now 108).
template <int THREADS>
__device__ __forceinline__ uint32_t tid() { return threadIdx.x % THREADS; }
template <int THREADS>
constexpr int GROUPS_OF = THREADS > 128 ? 1 : 4;
template <int THREADS>
__device__ __forceinline__ void row_sync() {
  if constexpr (GROUPS_OF<THREADS> == 1) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.x / THREADS), "n"(THREADS) : "memory");
}
// The same for a row's cluster: groups have none.
template <int THREADS>
__device__ __forceinline__ void all_sync() {
  if constexpr (GROUPS_OF<THREADS> == 1) ppl::cluster_sync();
  else row_sync<THREADS>();
}

template <int THREADS>
struct Fast {
  static constexpr int WARPS = THREADS / 32, ENTRIES = entries_of(THREADS), LIST = THREADS * ENTRIES;
  // of every block of the cluster, written by it
  unsigned long long sums[WARPS];
  float part_max[CLUSTER], part_sum[CLUSTER], part_bound[CLUSTER];
  uint32_t part_first[CLUSTER], part_n[CLUSTER];
  float wf[2][WARPS];
  uint32_t wu[WARPS];
  uint32_t bin, above, in_bin;
  uint32_t hist[256], all[256];
  uint32_t listed;
  uint2 list[LIST];  // the block's candidates: values and places
};

__device__ __forceinline__ uint32_t there(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  return a;
}
__device__ __forceinline__ void put(uint32_t a, float x) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory"); }
__device__ __forceinline__ void put(uint32_t a, uint32_t x) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory"); }

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
  return x;
}
__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x += __shfl_xor_sync(~0u, x, d);
  return x;
}
__device__ __forceinline__ float float_of(uint32_t key) { return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

// The digit (a warp's work) that the want-th element from the largest digit
// down has, how many have larger ones and how many it.
template <class S, class F>
__device__ __forceinline__ void find_digit(S& sh, uint32_t want, F&& count) {
  const uint32_t lane = threadIdx.x % 32;
  uint32_t c[8], sum = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum += c[k] = count(255 - 8 * lane - k);
  uint32_t run = sum;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t y = __shfl_up_sync(~0u, run, d);
    if (lane >= uint32_t(d)) run += y;
  }
  run -= sum;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (run < want && want <= run + c[k]) {
      sh.bin = 255 - 8 * lane - k;
      sh.above = run;
      sh.in_bin = c[k];
    }
    run += c[k];
  }
}

// The counts of all the cluster's blocks, in sh.all.  Every block has counted before, and
// may count again after the next all_sync.
template <int THREADS>
__device__ __forceinline__ void add_up(Fast<THREADS>& sh, uint32_t blocks) {
  for (uint32_t i = tid<THREADS>(); i < 256; i += THREADS) {
    uint32_t n[CLUSTER];
#pragma unroll
    for (uint32_t b = 0; b < CLUSTER; ++b) n[b] = b < blocks ? remote_u(&sh.hist[i], b) : 0;
#pragma unroll
    for (uint32_t b = 1; b < CLUSTER; ++b) n[0] += n[b];
    sh.all[i] = n[0];
  }
  row_sync<THREADS>();
}

// A digit of the want-th largest of the threads' entries; count(add) calls add
// with the digit of each of the thread's that are in question.
template <int THREADS, class F>
__device__ __forceinline__ void next_digit(Fast<THREADS>& sh, uint32_t want, F&& count) {
  for (uint32_t i = tid<THREADS>(); i < 256; i += THREADS) sh.hist[i] = 0;
  row_sync<THREADS>();
  count([&](uint32_t digit) { atomicAdd(&sh.hist[digit], 1); });
  row_sync<THREADS>();
  if (tid<THREADS>() < 32) find_digit(sh, want, [&](uint32_t d) { return sh.hist[d]; });
  row_sync<THREADS>();
}

// A thread's vectors of a block's part of a row.  Places count from the 16-byte
// boundary at or before the row's start; what is outside the row is -infinity.
template <class T, int THREADS, int NV>
struct Part {
  static constexpr int VEC = 16 / sizeof(T), N = NV;
  // a key's lowest bits, which all values of a sign share
  static constexpr int LOW = sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 13 : 16;
  using Vec = ppl::Pack<T, VEC>;
  Vec x[NV];
  uint32_t begin;       // place of the first vector
  int full, whole, n;   // the first whole vector, the one after the last whole one, all with values
  int slots;            // vectors that some thread has
  uint32_t shift, all;  // the row's first place, and the one after its last

  __device__ __forceinline__ uint32_t at(int i) const { return begin + i * THREADS * VEC; }

  __device__ __forceinline__ void load(const T* in, uint32_t from, uint32_t part, uint32_t n_vocab) {
    shift = uint32_t(reinterpret_cast<uintptr_t>(in) / sizeof(T) % VEC);
    all = n_vocab + shift;
    begin = from + tid<THREADS>() * VEC;
    const uint32_t to = min(from + part, all);
    constexpr uint32_t STEP = THREADS * VEC;
    slots = from < to ? (to - from + STEP - 1) / STEP : 0;
    n = begin < to ? (to - begin + STEP - 1) / STEP : 0;
    full = begin < shift ? 1 : 0;
    whole = begin + VEC <= to ? (to - VEC - begin) / STEP + 1 : 0;
    const T none = from_f<T>(-INFINITY);
    const T* p = in + (int64_t(begin) - shift);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) x[i].v[k] = none;
      if (i >= full && i < whole) x[i] = *reinterpret_cast<const Vec*>(p + i * int(STEP));
    }
    // the incomplete vectors, where the row begins and ends
#pragma unroll 1
    for (int e = full ? 0 : whole; e < n; e = e < whole && whole < n ? whole : n) {
      const uint32_t j = at(e);
      Vec edge;
#pragma unroll
      for (int k = 0; k < VEC; ++k) edge.v[k] = j + k >= shift && j + k < all ? in[int64_t(j) + k - shift] : none;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == e) x[i] = edge;
    }
  }
  // What was computed from the values is not kept for the next pass over them:
  // in 32 bits they would not fit the registers.
  __device__ __forceinline__ void forget() {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&x[i]);
        asm volatile("" : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]));
      }
    }
  }
  template <class F>
  __device__ __forceinline__ void each(F&& f) {
    forget();
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i < slots) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) f(to_f(x[i].v[k]), at(i) + k);
      }
  }
  template <class F>
  __device__ __forceinline__ void change(F&& f) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i < slots) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[i].v[k] = from_f<T>(f(to_f(x[i].v[k]), at(i) + k));
      }
  }
  // The inputs' and the outputs' boundaries agree where their strides do.
  __device__ __forceinline__ bool wide(const float* out) const { return (reinterpret_cast<uintptr_t>(out) / 4 - shift) % VEC == 0; }
  // f(i, p) fills the VEC probabilities p of vector i.
  template <class F>
  __device__ __forceinline__ void write(float* out, F&& f) {
    forget();
    const bool wide = this->wide(out);
    float* to = out + (int64_t(begin) - shift);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i >= n) break;
      constexpr int STEP = THREADS * VEC;
      float p[VEC];
      f(i, p);
      if (wide && i >= full && i < whole) {
        if constexpr (VEC == 8)
          asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + i * STEP), "f"(p[0]), "f"(p[1]), "f"(p[2]), "f"(p[3]),
                       "f"(p[4]), "f"(p[5]), "f"(p[6]), "f"(p[7]) : "memory");
        else
          *reinterpret_cast<float4*>(to + i * STEP) = make_float4(p[0], p[1], p[2], p[3]);
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if (at(i) + k >= shift && at(i) + k < all) to[i * STEP + k] = p[k];
      }
    }
  }
};

// What is kept: keys above `least`, and those equal to it at places up to `last`.
struct Cut {
  uint32_t least, last;
};

// This thread's entries of all the blocks' lists, in which every block finds the same.
// Those of a row's only block stay in its list.
template <int THREADS>
struct Entries {
  static constexpr int MOST = Fast<THREADS>::ENTRIES;
  static constexpr bool HELD = GROUPS_OF<THREADS> == 1;
  float value[HELD ? MOST : 1];
  uint32_t place[HELD ? MOST : 1];
  int n;
  const uint2* list;
  uint32_t total;

  __device__ __forceinline__ Entries(Fast<THREADS>& sh, uint32_t all) : n(0), list(sh.list), total(all) {
    if constexpr (HELD) {
#pragma unroll
      for (int e = 0; e < MOST; ++e) {
        uint32_t i = tid<THREADS>() + e * THREADS, b = 0;
        if (i < total) {
          for (uint32_t m; i >= (m = sh.part_n[b]); ++b) i -= m;
          uint32_t v;
          asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v), "=r"(place[e]) : "r"(there(&sh.list[i], b)) : "memory");
          value[e] = __uint_as_float(v);
          ++n;
        }
      }
    }
  }
  // f(value, place, number of the entry)
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    if constexpr (HELD) {
#pragma unroll
      for (int e = 0; e < MOST; ++e)
        if (e < n) f(value[e], place[e], tid<THREADS>() + e * THREADS);
    } else {
#pragma unroll 1
      for (uint32_t i = tid<THREADS>(); i < total; i += THREADS) f(__uint_as_float(list[i].x), list[i].y, i);
    }
  }
};

// The values for which `pick` holds go to the block's list, in any order.  They are few, so
// they are only marked in the pass over the values, and read again for the list: a
// branch for each value makes a kernel of code that is not at hand when it is needed.
template <class P, int THREADS, class T, class F>
__device__ __forceinline__ void list_where(P& part, Fast<THREADS>& sh, const T* in, F&& pick) {
  constexpr int WORDS = (P::N * P::VEC + 31) / 32;
  uint32_t marks[WORDS] = {};
  part.forget();
#pragma unroll
  for (int i = 0; i < P::N; ++i)
    if (i < part.slots)
#pragma unroll
    for (int k = 0; k < P::VEC; ++k)
      if (pick(to_f(part.x[i].v[k]))) marks[(i * P::VEC + k) / 32] |= 1u << (i * P::VEC + k) % 32;
#pragma unroll
  for (int w = 0; w < WORDS; ++w)
    for (; marks[w]; marks[w] &= marks[w] - 1) {
      const int e = w * 32 + __ffs(marks[w]) - 1;
      const uint32_t j = part.at(e / P::VEC) + e % P::VEC, at = atomicAdd(&sh.listed, 1);
      if (at < Fast<THREADS>::LIST) sh.list[at] = make_uint2(__float_as_uint(to_f(in[int64_t(j) - part.shift])), j);
    }
}

// The cut that keeps `want` of the total listed values, all from reach to top.
template <class P, int THREADS>
__device__ __forceinline__ Cut cut_among(Fast<THREADS>& sh, const Entries<THREADS>& entries, uint32_t want, float top, float reach, uint32_t places) {
  constexpr int LOW = P::LOW;
  const uint32_t hi = key_of(top) >> LOW, lo = key_of(reach) >> LOW;
  Cut cut = {lo, ~0u};  // all candidates
  uint32_t in_bin = entries.total;
  if (in_bin <= want) return cut;
  // digit by digit below the bits that all candidates share; then, of those that tie, the places
  int bits = 32 - __clz(hi ^ lo), side = 0;
  uint32_t found = bits == 32 ? 0 : hi >> bits << bits;
  const int place_bits = 32 - __clz(places);
  const uint32_t inside = ~(~0u << place_bits);
#pragma unroll 1
  while (true) {
    if (want == in_bin || bits == 0) {  // all that agree so far are kept, or the last bit is known
      if (side) {
        cut.last = ~found & inside;
        return cut;
      }
      cut.least = found;
      if (want == in_bin) return cut;
      side = 1;
      found = 0;
      bits = place_bits;
    }
    const int at = max(bits - 8, 0);
    const uint32_t mask = bits == 32 ? 0 : ~0u << bits, low = (1u << (bits - at)) - 1;
    next_digit<THREADS>(sh, want, [&](auto&& add) {
      entries.each([&](float f, uint32_t j, uint32_t) {
        const uint32_t key = key_of(f) >> LOW, q = side ? ~j & inside : key;
        if ((!side || key == cut.least) && (q & mask) == found) add(q >> at & low);
      });
    });
    found |= sh.bin << at;
    want -= sh.above;
    in_bin = sh.in_bin;
    bits = at;
  }
}

// The cut of any length.  The values from the largest to the least are counted in 256
// steps of equal height, and those in the step that the cut goes through are listed.
// Where the lists have no room for them, their digits are counted over all values of
// the cluster.  A function of its own, since its registers would crowd out the values
// elsewhere.
template <class T, int THREADS, int NV>
__device__ __noinline__ Cut cut_of_all(const T* in, uint32_t from, uint32_t size, uint32_t n_vocab, Fast<THREADS>& sh, uint32_t rank,
                                       uint32_t blocks, uint32_t want) {
  using P = Part<T, THREADS, NV>;
  constexpr int WARPS = THREADS / 32, LIST = Fast<THREADS>::LIST;
  const uint32_t lane = tid<THREADS>() % 32, warp = tid<THREADS>() / 32;
  P part;
  part.load(in, from, size, n_vocab);
  float top = -INFINITY, low = INFINITY;
  part.each([&](float f, uint32_t) {
    top = fmaxf(top, f);
    if (f > -INFINITY) low = fminf(low, f);
  });
  top = warp_max(top);
  low = -warp_max(-low);
  row_sync<THREADS>();  // all are done with what was there
  if (lane == 0) sh.wf[0][warp] = top, sh.wf[1][warp] = low;
  if (tid<THREADS>() == 0) sh.listed = 0;
  for (uint32_t i = tid<THREADS>(); i < 256; i += THREADS) sh.hist[i] = 0;
  row_sync<THREADS>();
  top = warp_max(sh.wf[0][lane % WARPS]);
  low = -warp_max(-sh.wf[1][lane % WARPS]);
  all_sync<THREADS>();  // nor does another block read this one's from before
  if (tid<THREADS>() < blocks) {
    put(there(&sh.part_max[rank], tid<THREADS>()), top);
    put(there(&sh.part_bound[rank], tid<THREADS>()), low);
  }
  all_sync<THREADS>();
  for (uint32_t b = 0; b < blocks; ++b) {
    top = fmaxf(top, sh.part_max[b]);
    low = fminf(low, sh.part_bound[b]);
  }
  const float height = 255.f / (top - low);
  if (height > 0.f && height < INFINITY) {  // not so where all are equal, or too far from one another
    // steps never rise as values fall, whatever is rounded
    auto step = [&](float f) { return 255 - min(int((top - f) * height), 255); };
    part.each([&](float f, uint32_t) {
      if (f > -INFINITY) atomicAdd(&sh.hist[step(f)], 1);
    });
    all_sync<THREADS>();  // every block's counts are there
    if (tid<THREADS>() == 0) sh.in_bin = 0;
    row_sync<THREADS>();
    add_up(sh, blocks);
    if (tid<THREADS>() < 32) find_digit(sh, want, [&](uint32_t d) { return sh.all[d]; });
    row_sync<THREADS>();
    const uint32_t total = sh.in_bin, left = want - sh.above;
    const int bin = sh.bin;
    if (total == 0) return {0, ~0u};  // fewer finite values than are to be kept
    if (total <= LIST) {
      float reach = top, high = low;
      list_where(part, sh, in, [&](float f) { return f > -INFINITY && step(f) == bin; });
      row_sync<THREADS>();
      if (tid<THREADS>() < blocks) put(there(&sh.part_n[rank], tid<THREADS>()), sh.listed);
      all_sync<THREADS>();
      const Entries<THREADS> entries(sh, total);
      entries.each([&](float f, uint32_t, uint32_t) { reach = fminf(reach, f), high = fmaxf(high, f); });
      reach = -warp_max(-reach);
      high = warp_max(high);
      if (lane == 0) sh.wf[0][warp] = high, sh.wf[1][warp] = reach;
      all_sync<THREADS>();  // and every block has read what it needs of the others
      high = warp_max(sh.wf[0][lane % WARPS]);
      reach = -warp_max(-sh.wf[1][lane % WARPS]);
      row_sync<THREADS>();  // all have read wf, which the caller writes next: where the step is kept whole no other barrier comes between
      return cut_among<P>(sh, entries, left, high, reach, part.all);
    }
    all_sync<THREADS>();  // the counts are read
  }
  Cut cut = {0, ~0u};
  const int place_bits = 32 - __clz(part.all);
  // side 0: the values; side 1: the places of those that tie, where not all are kept
  uint32_t found = 0;
  int bits = 32 - P::LOW, side = 0;
  while (true) {
    const int at = max(bits - 8, 0);
    const uint32_t mask = bits == 32 ? 0 : ~0u << bits, low = (1u << (bits - at)) - 1;
    for (uint32_t i = tid<THREADS>(); i < 256; i += THREADS) sh.hist[i] = 0;
    row_sync<THREADS>();
    part.each([&](float f, uint32_t j) {
      uint32_t q = key_of(fmaxf(f, -INFINITY)) >> P::LOW;
      bool in = !side || q == cut.least;
      if (side) q = ~j & ~(~0u << place_bits);
      in = in && (q & mask) == found;
      if (in) atomicAdd(&sh.hist[q >> at & low], 1);
    });
    all_sync<THREADS>();  // every block's counts are there
    add_up(sh, blocks);
    if (tid<THREADS>() < 32) find_digit(sh, want, [&](uint32_t d) { return sh.all[d]; });
    all_sync<THREADS>();  // and read
    found |= sh.bin << at;
    want -= sh.above;
    bits = at;
    const bool whole = want == sh.in_bin;  // all that agree so far are kept
    if (!whole && bits > 0) continue;
    if (side) {
      cut.last = ~found & ~(~0u << place_bits);
      return cut;
    }
    cut.least = found;
    if (whole) return cut;
    side = 1;
    found = 0;
    bits = place_bits;
  }
}

// The probabilities of a cut row, where the blocks' lists have room for what
// reaches a bound that at least top_k values reach; false where not.
template <class P, int THREADS, int G, class T>
__device__ __forceinline__ bool write_cut(P& part, Fast<THREADS>& sh, uint32_t rank, uint32_t blocks, uint32_t top_k, float m,
                                          const float (&maxima)[G], float c, const T* in, uint32_t size, float* out) {
  constexpr int LIST = Fast<THREADS>::LIST, LOW = P::LOW;
  const uint32_t k_part = (top_k + blocks - 1) / blocks;
  const bool every = k_part > THREADS * G;  // only where the lists have room for the row
  if (every && part.all > LIST) return false;
  // Each block's k_part-th largest of its threads' (or vectors') maxima (its key's upper half): at least
  // k_part of its values reach that, so top_k of the row reach the least of them.  A block
  // with fewer than that finds -infinity.
  uint32_t bound = 0, want = k_part;
  for (int at = 24; at >= 16 && !every; at -= 8) {
    next_digit<THREADS>(sh, want, [&](auto&& add) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const uint32_t key = key_of(maxima[i]);
        if (at == 24 || key >> 24 == bound >> 24) add(key >> at & 255);
      }
    });
    bound |= sh.bin << at;
    want -= sh.above;
  }
  if (tid<THREADS>() < blocks) {
    put(there(&sh.part_max[rank], tid<THREADS>()), m);
    put(there(&sh.part_bound[rank], tid<THREADS>()), bound > KEY_LOST ? float_of(bound) : -3.402823466e38f);
  }
  if (tid<THREADS>() == 0) sh.listed = 0;
  all_sync<THREADS>();
  float reach = INFINITY, top = -INFINITY;
  for (uint32_t b = 0; b < blocks; ++b) {
    top = fmaxf(top, sh.part_max[b]);
    reach = fminf(reach, sh.part_bound[b]);
  }
  // the candidates, in any order
  list_where(part, sh, in, [&](float f) { return f >= reach; });
  row_sync<THREADS>();
  const uint32_t mine = sh.listed;
  if (tid<THREADS>() < blocks) put(there(&sh.part_n[rank], tid<THREADS>()), mine);
  all_sync<THREADS>();
  uint32_t total = 0, own = 0;
  for (uint32_t b = 0; b < blocks; ++b) {
    if (b < rank) own += sh.part_n[b];
    total += sh.part_n[b];
  }
  if (total > LIST) return false;
  const Entries<THREADS> entries(sh, total);
  if constexpr (GROUPS_OF<THREADS> == 1) ppl::cluster_arrive_release();  // this block has read what it needs of the others
  // Zeros everywhere: the few others are written over them once they are known.
  if (part.wide(out)) {
    part.write(out, [&](int, float* p) {
#pragma unroll
      for (int k = 0; k < P::VEC; ++k) p[k] = 0.f;
    });
  } else {  // so that a warp's lie side by side (512 rows of 131075 f16: 115 us, and 315 vector by vector)
    const uint32_t from = part.begin - tid<THREADS>() * P::VEC;
#pragma unroll 4
    for (uint32_t j = max(from, part.shift) + tid<THREADS>(); j < min(from + size, part.all); j += THREADS) out[j - part.shift] = 0.f;
  }
  const Cut cut = cut_among<P>(sh, entries, top_k, top, reach, part.all);
  auto kept = [&](float f, uint32_t j) {
    const uint32_t key = key_of(f) >> LOW;
    return key > cut.least || (key == cut.least && j <= cut.last);
  };
  // The lists' order is not the same each time, so the sum is one of whole numbers: units
  // of 2^-44, of exponentials up to 1 of which one is.
  unsigned long long s = 0;
  entries.each([&](float f, uint32_t j, uint32_t) {
    if (!kept(f, j)) return;
    const float high = share(f, top, c) * 0x1p22f;
    const uint32_t whole = __float2uint_rz(high);
    s += (uint64_t(whole) << 22) + __float2uint_rz((high - float(whole)) * 0x1p22f);
  });
#pragma unroll
  for (int d = 16; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
  if (tid<THREADS>() % 32 == 0) sh.sums[tid<THREADS>() / 32] = s;
  row_sync<THREADS>();
  s = sh.sums[tid<THREADS>() % (THREADS / 32)];
#pragma unroll
  for (int d = THREADS / 64; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
  const float factor = s ? 1.f / (float(uint32_t(s >> 32)) * 0x1p-12f + float(uint32_t(s)) * 0x1p-44f) : 0.f;
  entries.each([&](float f, uint32_t j, uint32_t i) {  // over the zeros: there were barriers since
    if (i - own < mine && kept(f, j)) out[int64_t(j) - part.shift] = share(f, top, c) * factor;
  });
  if constexpr (GROUPS_OF<THREADS> == 1) ppl::cluster_wait();
  return true;
}

template <class T, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS* GROUPS_OF<THREADS>, 1024 / (THREADS * GROUPS_OF<THREADS>)) cut_kernel(const ProbArgs a) {
  constexpr int GROUPS = GROUPS_OF<THREADS>;
  if constexpr (GROUPS == 1) ppl::cluster_arrive();
  constexpr int VEC = 16 / sizeof(T), WARPS = THREADS / 32;
  using P = Part<T, THREADS, NV>;
  __shared__ Fast<THREADS> shared[GROUPS];
  const uint32_t group = threadIdx.x / THREADS;
  Fast<THREADS>& sh = shared[group];
  const uint32_t rank = blockIdx.x % a.blocks, r = blockIdx.x / a.blocks * GROUPS + group;
  if (r >= a.n_rows) return;
  const uint32_t lane = tid<THREADS>() % 32, warp = tid<THREADS>() / 32;
  float* out = a.out + r * a.out_stride;
  const float t = a.temperature ? a.temperature[r] : 1.f;
  const int32_t top_k = a.top_k[r];
  const T* in = static_cast<const T*>(a.in) + r * a.in_stride;
  P part;
  part.load(in, rank * a.part, a.part, a.n_vocab);
  const bool greedy = !(t > 0x1p-125f);  // below, c is not a float
  const float c = 2.88539008f / t;
  constexpr int G = THREADS > 128 ? 1 : NV;  // maxima a thread: more where there are few threads
  float m = -INFINITY, maxima[G];
#pragma unroll
  for (int i = 0; i < G; ++i) maxima[i] = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i < part.slots) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) maxima[i % G] = fmaxf(maxima[i % G], to_f(part.x[i].v[k]));
    }
#pragma unroll
  for (int i = 0; i < G; ++i) m = fmaxf(m, maxima[i]);
  m = warp_max(m);
  if (lane == 0) sh.wf[0][warp] = m;
  row_sync<THREADS>();
  m = warp_max(sh.wf[0][lane % WARPS]);
  if constexpr (GROUPS == 1) ppl::cluster_wait();  // every block has started
  const bool some = top_k > 0 && uint32_t(top_k) < a.n_vocab && !greedy;
  Cut cut = {0, ~0u};
  if (some) {
    if (write_cut(part, sh, rank, a.blocks, uint32_t(top_k), m, maxima, c, in, a.part, out)) return;
    cut = cut_of_all<T, THREADS, NV>(in, rank * a.part, a.part, a.n_vocab, sh, rank, a.blocks, uint32_t(top_k));
    part.load(in, rank * a.part, a.part, a.n_vocab);  // again, rather than kept in registers meanwhile
  }
  // ---- the sum relative to the block's largest value, and the first place that has it
  // Kept, in floats: above all that tie, or of those that tie up to the last place.  (KEY_LOST
  // and what is beyond infinity's key make NaN, which nothing reaches.)
  const uint32_t tie = cut.least << P::LOW, over = (cut.least + 1) << P::LOW;
  float from_tie = tie > KEY_LOST ? float_of(tie) : -3.402823466e38f, from_over = over > KEY_LOST ? float_of(over) : INFINITY;
  auto kept = [&](float f, uint32_t j) { return f >= from_over || (f >= from_tie && j <= cut.last); };
  float half = -0.5f * m;
  if (m == INFINITY && !greedy) {  // the infinities that are kept become 0, the rest -infinity, and the largest 0
    part.change([&](float f, uint32_t j) { return f == m && kept(f, j) ? 0.f : -INFINITY; });
    half = 0.f;
    from_tie = -3.402823466e38f;
    from_over = INFINITY;
    cut.last = ~0u;
  }
  // share(f, m, c), where all are kept and where not: loops for each (512 rows of 131075 bf16 without a cut 86 us, and
  // 102 where every value is compared)
  auto of_all = [&](float f, uint32_t) { return fmaxf(fmaf(f, 0.5f, half) * c, -200.f); };
  auto of_kept = [&](float f, uint32_t j) { return kept(f, j) ? of_all(f, j) : -200.f; };
  float s = 0.f;
  uint32_t first = ~0u;
  auto sum = [&](auto&& exponent) {
    if constexpr (sizeof(T) == 4) {  // in the values' place
      part.change([&](float f, uint32_t j) {
        const float e = exp2f(exponent(f, j));
        s += e;
        return e;
      });
    } else {
      part.each([&](float f, uint32_t j) {
        float e;  // below 2^-126: 0, beside a 1 in the sum
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(exponent(f, j)));
        s += e;
      });
    }
  };
  if (greedy) part.each([&](float f, uint32_t j) { first = f == m ? min(first, j) : first; });
  else if (some) sum(of_kept);
  else sum(of_all);
  s = warp_add(s);
  first = __reduce_min_sync(~0u, first);
  if (lane == 0) sh.wf[1][warp] = s, sh.wu[warp] = first;
  row_sync<THREADS>();
  if (warp == 0) {
    s = warp_add(lane < WARPS ? sh.wf[1][lane] : 0.f);
    first = __reduce_min_sync(~0u, lane < WARPS ? sh.wu[lane] : ~0u);
    if (lane < a.blocks) {
      put(there(&sh.part_max[rank], lane), m);
      put(there(&sh.part_sum[rank], lane), s);
      put(there(&sh.part_first[rank], lane), first);
    }
  }
  all_sync<THREADS>();
  float top = -INFINITY;
  for (uint32_t b = 0; b < a.blocks; ++b) top = fmaxf(top, sh.part_max[b]);
  float total = 0.f;
  uint32_t best = ~0u;
  for (uint32_t b = 0; b < a.blocks; ++b) {
    total += sh.part_sum[b] * share(sh.part_max[b], top, c);
    if (sh.part_max[b] == top) best = min(best, sh.part_first[b]);
  }
  if (greedy) {
    if (!(top > -INFINITY)) best = ~0u;
    part.write(out, [&](int i, float* p) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) p[k] = part.at(i) + k == best ? 1.f : 0.f;
    });
    return;
  }
  const float factor = total > 0.f ? share(m, top, c) / total : 0.f;
  auto write = [&](auto&& exponent) {
    part.write(out, [&](int i, float* p) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float f = to_f(part.x[i].v[k]);
        p[k] = (sizeof(T) == 4 ? f : exp2f(exponent(f, part.at(i) + k))) * factor;
      }
    });
  };
  if (sizeof(T) == 2 && some) write(of_kept);
  else write(of_all);
}

// ------------------------------------------------------------ rows without a cut
// A block's part of a row lies in shared memory, each thread's vectors where only
// it reads them: copies, largest value, sum and writing have no barrier between
// them but for the exchange of the largest values and the sums.  Few registers and
// short loops: as many blocks at once as hide one another's latencies.
template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) plain_kernel(const ProbArgs a) {
  ppl::cluster_arrive();
  constexpr int VEC = 16 / sizeof(T), WARPS = THREADS / 32;
  constexpr int STEP = THREADS * VEC;
  using Vec = ppl::Pack<T, VEC>;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ float part_max[CLUSTER], part_sum[CLUSTER], wmax[WARPS], wsum[WARPS];
  __shared__ uint32_t part_first[CLUSTER], wfirst[WARPS];
  const uint32_t rank = blockIdx.x % a.blocks, r = blockIdx.x / a.blocks;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const T* in = static_cast<const T*>(a.in) + r * a.in_stride;
  float* out = a.out + r * a.out_stride;
  // places count from the 16-byte boundary at or before the row's start
  const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(in) / sizeof(T) % VEC);
  const uint32_t all = a.n_vocab + shift, to = min((rank + 1) * a.part, all), begin = rank * a.part + threadIdx.x * VEC;
  const int n = begin < to ? (to - begin + STEP - 1) / STEP : 0;  // vectors with values
  const int full = begin < shift ? 1 : 0;                         // the first whole one
  const int whole = begin + VEC <= to ? (to - VEC - begin) / STEP + 1 : 0;  // the one after the last whole one
  Vec* x = reinterpret_cast<Vec*>(raw) + threadIdx.x;
  {
    const T* p = in + (int64_t(begin) - shift);
    uint32_t slot = uint32_t(__cvta_generic_to_shared(x));
#pragma unroll 4
    for (int i = full; i < whole; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + i * THREADS * 16), "l"(p + int64_t(i) * STEP) : "memory");
    // the incomplete vectors, where the row begins and ends
    for (int e = full ? 0 : whole; e < n; e = e < whole && whole < n ? whole : n) {
      const uint32_t j = begin + e * STEP;
#pragma unroll
      for (int k = 0; k < VEC; ++k) x[e * THREADS].v[k] = j + k >= shift && j + k < all ? in[int64_t(j) + k - shift] : from_f<T>(-INFINITY);
    }
  }
  const float t = a.temperature ? a.temperature[r] : 1.f;
  const bool greedy = !(t > 0x1p-125f);  // below, c is not a float
  const float c = 2.88539008f / t;
  asm volatile("cp.async.wait_all;" ::: "memory");
  float m = -INFINITY;
#pragma unroll 2
  for (int i = 0; i < n; ++i) {
    const Vec v = x[i * THREADS];
#pragma unroll
    for (int k = 0; k < VEC; ++k) m = fmaxf(m, to_f(v.v[k]));
  }
  m = warp_max(m);
  if (lane == 0) wmax[warp] = m;
  __syncthreads();
  m = warp_max(wmax[lane % WARPS]);
  // share(f, m, c) for a finite m.  Nothing is added to an exponent to keep small numbers within a float's
  // range: beside 64 the likeliest tokens would lose 3 bits.
  const float half = -0.5f * m;
  auto exponent = [&](float f) { return fmaxf(fmaf(f, 0.5f, half) * c, -200.f); };
  const bool endless = m == INFINITY;
  float s = 0.f;
  uint32_t first = ~0u;
  if (greedy) {
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) first = to_f(x[i * THREADS].v[k]) == m ? min(first, begin + i * STEP + k) : first;
  } else if (endless) {
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) s += to_f(x[i * THREADS].v[k]) == m ? 1.f : 0.f;
  } else {
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const Vec v = x[i * THREADS];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float e;  // below 2^-126: 0, beside a 1 in the sum
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(exponent(to_f(v.v[k]))));
        s += e;
      }
    }
  }
  s = warp_add(s);
  first = __reduce_min_sync(~0u, first);
  if (lane == 0) wsum[warp] = s, wfirst[warp] = first;
  __syncthreads();
  ppl::cluster_wait();  // every block has started
  if (warp == 0) {
    s = warp_add(lane < WARPS ? wsum[lane] : 0.f);
    first = __reduce_min_sync(~0u, lane < WARPS ? wfirst[lane] : ~0u);
    if (lane < a.blocks) {
      put(there(&part_max[rank], lane), m);
      put(there(&part_sum[rank], lane), s);
      put(there(&part_first[rank], lane), first);
    }
  }
  ppl::cluster_sync();
  float top = -INFINITY, total = 0.f;
  uint32_t best = ~0u;
  for (uint32_t b = 0; b < a.blocks; ++b) top = fmaxf(top, part_max[b]);
  for (uint32_t b = 0; b < a.blocks; ++b) {
    total += part_sum[b] * share(part_max[b], top, c);
    if (part_max[b] == top && top > -INFINITY) best = min(best, part_first[b]);
  }
  const float factor = total > 0.f ? share(m, top, c) / total : 0.f;
  // the inputs' and the outputs' boundaries agree where their strides do
  const bool wide = (reinterpret_cast<uintptr_t>(out) / 4 - shift) % VEC == 0;
  auto write = [&](auto&& probability) {
    // Elsewhere value by value, so that a warp's lie side by side: 512 rows of 131075 f16 81 us, 72 where the
    // boundaries agree (226 with the values of a vector one after the other, at the time).
    if (!wide) {
      const uint32_t from = rank * a.part;
      const T* y = reinterpret_cast<const T*>(raw);
      __syncthreads();
#pragma unroll 4
      for (uint32_t j = max(from, shift) + threadIdx.x; j < to; j += THREADS) out[j - shift] = probability(to_f(y[j - from]), j);
      return;
    }
    float* q = out + (int64_t(begin) - shift);
#pragma unroll 2
    for (int i = 0; i < n; ++i, q += STEP) {
      const Vec v = x[i * THREADS];
      float p[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) p[k] = probability(to_f(v.v[k]), begin + i * STEP + k);
      if (i >= full && i < whole) {
        if constexpr (VEC == 8)
          asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "f"(p[0]), "f"(p[1]), "f"(p[2]), "f"(p[3]), "f"(p[4]),
                       "f"(p[5]), "f"(p[6]), "f"(p[7]) : "memory");
        else
          *reinterpret_cast<float4*>(q) = make_float4(p[0], p[1], p[2], p[3]);
      } else {
        const uint32_t j = begin + i * STEP;
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if (j + k >= shift && j + k < all) q[k] = p[k];
      }
    }
  };
  // each kind of row with loops of its own (one loop for all three, its values' exponentials kept in their place
  // where they are floats: 2560 x 50001 f32 179 us, 512 x 131075 bf16 88)
  if (greedy) write([&](float, uint32_t j) { return j == best ? 1.f : 0.f; });
  else if (endless) write([&](float f, uint32_t) { return f == m ? factor : 0.f; });
  else write([&](float f, uint32_t) { return exp2f(exponent(f)) * factor; });
}

template <class K>
cudaError_t launch_as(K kernel, const ProbArgs& a, uint64_t n_rows, int threads, uint32_t smem, cudaStream_t stream, int groups = 1) {
  cudaLaunchAttribute at;
  std::memset(&at, 0, sizeof at);
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = a.blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((n_rows + groups - 1) / groups * a.blocks));
  cfg.blockDim = dim3(threads * groups);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <class T, int THREADS_>
cudaError_t launch_cut(const ProbArgs& a, uint64_t n_rows, uint32_t vectors, cudaStream_t stream) {
  const uint32_t nv = (vectors + THREADS_ - 1) / THREADS_;
  if (nv <= 2) return launch_as(cut_kernel<T, THREADS_, 2>, a, n_rows, THREADS_, 0, stream, GROUPS_OF<THREADS_>);
  if (nv <= 5) return launch_as(cut_kernel<T, THREADS_, 5>, a, n_rows, THREADS_, 0, stream, GROUPS_OF<THREADS_>);
  return launch_as(cut_kernel<T, THREADS_, NV_MOST>, a, n_rows, THREADS_, 0, stream, GROUPS_OF<THREADS_>);
}

// A kernel whose parts lie in shared memory.
template <class K>
cudaError_t launch_in_shared(K kernel, ppi::DeviceOnce& once, const ProbArgs& a, uint64_t n_rows, int threads, uint32_t smem, cudaStream_t stream) {
  int dev;
  cudaError_t e = ppi::current_device(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&](int) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(RESIDENT_MOST)); });
  if (e != cudaSuccess) return e;
  return launch_as(kernel, a, n_rows, threads, smem, stream);
}

template <class T>
cudaError_t launch(ProbArgs& a, uint64_t n_rows, cudaStream_t stream) {
  constexpr uint32_t VEC = 16 / sizeof(T);
  static ppi::DeviceOnce once[3];
  const uint32_t vectors = (a.n_vocab + 2 * VEC - 2) / VEC;  // at any alignment
  // Short rows, and enough of them to fill the device: 128 threads each (8192 rows of 5000 bf16
  // with a cut: 108 us; with a block of 512 threads each 206, at 128 then 184).
  const bool small = vectors <= 128 * NV_MOST && (n_rows >= 608 || vectors <= 256);
  uint32_t blocks = 1;
  auto part = [&] {
    const uint32_t each = (vectors + blocks - 1) / blocks;
    a.blocks = blocks;
    a.part = each * VEC;
    return each;
  };
  auto more = [&] {
    while (blocks * 2 <= CLUSTER && n_rows * blocks * 2 <= 264 && vectors >= blocks * 2 * MID) blocks *= 2;
  };
  if (small) {
    part();
    if (a.top_k) return launch_cut<T, 128>(a, n_rows, vectors, stream);
    return launch_in_shared(plain_kernel<T, 128>, once[0], a, n_rows, 128, vectors * 16, stream);
  }
  if (a.top_k) {
    // as many blocks as hold the row, of a power of two or not (512 rows of 80000 f32: 102 us by five,
    // 133 by eight; 2560 of 50001: 287 by three, 335 by four); more while all of them run at once (64
    // rows of 131072 bf16: 33 us in clusters of four, one wave, and 41 of eight, two, at the time; now 19)
    const uint32_t threads = vectors <= MID * NV_MOST * CLUSTER ? MID : LARGE;
    blocks = std::min((vectors + threads * NV_MOST - 1) / (threads * NV_MOST), uint32_t(CLUSTER));
    more();
    const uint32_t each = part();
    if (each <= MID * NV_MOST) return launch_cut<T, MID>(a, n_rows, each, stream);
    // a multiprocessor a block (64 rows of 200064 f32, k = 50: 38 us, 185 in long_kernel; of 500000 bf16 81 and 651)
    if (each <= LARGE * NV_MOST) return launch_as(cut_kernel<T, LARGE, NV_MOST>, a, n_rows, LARGE, 0, stream);
  } else {
    const uint32_t most = (vectors <= PART_OF_TWO / 16 * 2 ? PART_OF_TWO : PART_MOST) / 16;
    blocks = std::min((vectors + most - 1) / most, uint32_t(CLUSTER));
    more();
    const uint32_t each = part();
    if (each <= RESIDENT_MOST / 16) return launch_in_shared(plain_kernel<T, MID>, once[1], a, n_rows, MID, each * 16, stream);
  }
  blocks = CLUSTER;
  const uint32_t each = part();
  a.resident = each <= RESIDENT_MOST / 16;
  return launch_in_shared(long_kernel<T>, once[2], a, n_rows, LONG_THREADS, a.resident ? each * 16 : 0, stream);
}

}  // namespace

extern "C" pp_rc pp_token_probs(const void* d_logits, pp_ftype type, size_t n_rows, size_t n_vocab,
                                size_t logits_stride, const float* d_temperature, const int32_t* d_top_k,
                                float* d_probs, size_t probs_stride, cudaStream_t stream) {
  if (!ppl::ftype_ok(type)) return PP_EINVAL;
  if (n_rows >= ppl::MAX_DIM / CLUSTER || n_vocab >= (size_t(1) << 30)) return PP_ETOOLARGE;
  if (!n_rows || !n_vocab) return PP_OK;
  if (!d_logits || !d_probs) return PP_EINVAL;
  if (n_rows > 1 && (probs_stride < n_vocab || (d_logits == d_probs && logits_stride != probs_stride))) return PP_EINVAL;
  if (d_logits == d_probs && type != PP_F32) return PP_EINVAL;
  if (!ppl::aligned(d_logits, ppl::fsize(type)) || !ppl::aligned(d_probs, 4) || !ppl::aligned(d_temperature, 4) || !ppl::aligned(d_top_k, 4))
    return PP_EINVAL;
  ProbArgs a;
  std::memset(&a, 0, sizeof a);
  a.in = d_logits;
  a.out = d_probs;
  a.temperature = d_temperature;
  a.top_k = d_top_k;
  a.in_stride = logits_stride;
  a.out_stride = probs_stride;
  a.n_vocab = uint32_t(n_vocab);
  a.n_rows = uint32_t(n_rows);
  cudaError_t e;
  switch (type) {
    case PP_F32: e = launch<float>(a, n_rows, stream); break;
    case PP_F16: e = launch<__half>(a, n_rows, stream); break;
    default: e = launch<__nv_bfloat16>(a, n_rows, stream); break;
  }
  return ppl::rc_of(e);
}
