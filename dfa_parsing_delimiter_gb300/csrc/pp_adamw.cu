// pp_adamw: one AdamW step over many tensors, states in 32 or in 8 bits.
//
// A warp takes a tile of 256 consecutive elements of one tensor: parameter,
// gradient and both states are read once, stepped in registers and written
// once.  Nothing is read twice and nothing is shared between tiles but the
// step's constants.  With 32-bit states it is bound by memory, 20 to 28 bytes an
// element: 131072 x 2048 f32 1125 us (6.7 TB/s; with accesses of 16 bytes, not
// 32, 1220), 32M bf16 with 32-bit copies 142 us (6.3 TB/s).
//
// With 8-bit states a tile is also what shares an exponent: the largest one is a
// warp reduction, and the codes come from the registers that the step left.  It is
// bound by instructions (some 85 an element, half of them logic, which runs at half
// the rate: hashing, codes in and out) and by loads that too few warps wait for:
// 159M elements of f32 with bf16 gradients 443 us (floor 327), and 154 for reading the
// states' values back (140).  What got both there, 597 us together: the next tile
// fetched into the cache ahead (634 us, without 705), arithmetic on two floats at a
// time (615), roots and quotients that flush (597), multiply-adds for shifts and
// additions (714 with them and approximate quotients, 906 before).
//
// The tensors' addresses are kernel parameters (up to 640 tensors a launch):
// nothing to copy to the device, so a step is one launch and can be captured.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using ppl::from_f;
using ppl::to_f;

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int TILE = PP_ADAMW_BLOCK, EACH = TILE / 32;  // elements of a warp and of a lane
// Blocks that a multiprocessor holds (159M, 8 bits: 714 us, 746 with five, 835 with three, at the time)
// and that a launch has for each.
constexpr int RESIDENT = 4, BLOCKS = 8;

struct Item {
  void* param;
  const void* grad;
  uint64_t n;
  uint64_t first;       // of the state's elements
  uint32_t tile_begin;  // of the launch's tiles
  float decay;
  int32_t param_type, grad_type;
};

struct Common {
  void* m;
  void* v;
  uint8_t* m_exp;
  uint8_t* v_exp;
  float* master;
  int32_t* counters;  // steps done; blocks that are through with this one
  const float* lr_at;
  const float* scale_at;
  const float* skip_at;
  float lr, b1, c1, b2, c2, eps;  // c: 1 - b, rounded once
  float log_b1, log_b2;
  uint32_t n_items, n_tiles, chunk, seed;
  int32_t nearest, last;
  int32_t wide;  // the states lie at 32-byte addresses
};

template <int CAP>
struct Args {
  Common c;
  Item item[CAP];
};
static_assert(sizeof(Args<640>) < 32764, "kernel parameters");

// A hash of 32 bits: odd multipliers from the fractions of the roots of 2 and
// 3, between shifts that bring high bits down.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ x >> 16;
}

// EACH values of a lane.  In a whole tile at 32-byte addresses a lane's are
// EACH consecutive ones; otherwise, element by element, those at lane, lane +
// 32, ... so that a warp's accesses lie side by side.
__device__ __forceinline__ void read_whole(const float* p, float* x) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]) : "l"(p) : "memory");
}
__device__ __forceinline__ void write_whole(float* p, const float* x) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]),
               "f"(x[5]), "f"(x[6]), "f"(x[7]) : "memory");
}
template <class T>
__device__ __forceinline__ void read_whole(const T* p, float* x) {
  const ppl::Pack<T, EACH> q = *reinterpret_cast<const ppl::Pack<T, EACH>*>(p);
#pragma unroll
  for (int i = 0; i < EACH; ++i) x[i] = to_f(q.v[i]);
}
template <class T>
__device__ __forceinline__ void write_whole(T* p, const float* x) {
  ppl::Pack<T, EACH> q;
#pragma unroll
  for (int i = 0; i < EACH; ++i) q.v[i] = from_f<T>(x[i]);
  *reinterpret_cast<ppl::Pack<T, EACH>*>(p) = q;
}
template <bool WHOLE, class T>
__device__ __forceinline__ void read(const T* p, uint32_t lane, uint32_t n, float* x) {
  if constexpr (WHOLE) {
    read_whole(p + lane * EACH, x);
  } else {
#pragma unroll
    for (int k = 0; k < EACH; ++k) x[k] = lane + k * 32 < n ? to_f(p[lane + k * 32]) : 0.f;
  }
}
template <bool WHOLE, class T>
__device__ __forceinline__ void write(T* p, uint32_t lane, uint32_t n, const float* x) {
  if constexpr (WHOLE) {
    write_whole(p + lane * EACH, x);
  } else {
#pragma unroll
    for (int k = 0; k < EACH; ++k)
      if (lane + k * 32 < n) p[lane + k * 32] = from_f<T>(x[k]);
  }
}
template <bool WHOLE>
__device__ __forceinline__ void read_any(const void* p, int type, uint64_t at, uint32_t lane, uint32_t n, float* x) {
  switch (type) {
    case PP_F32: return read<WHOLE>(static_cast<const float*>(p) + at, lane, n, x);
    case PP_F16: return read<WHOLE>(static_cast<const __half*>(p) + at, lane, n, x);
    default: return read<WHOLE>(static_cast<const __nv_bfloat16*>(p) + at, lane, n, x);
  }
}
template <bool WHOLE>
__device__ __forceinline__ void write_any(void* p, int type, uint64_t at, uint32_t lane, uint32_t n, const float* x) {
  switch (type) {
    case PP_F32: return write<WHOLE>(static_cast<float*>(p) + at, lane, n, x);
    case PP_F16: return write<WHOLE>(static_cast<__half*>(p) + at, lane, n, x);
    default: return write<WHOLE>(static_cast<__nv_bfloat16*>(p) + at, lane, n, x);
  }
}

// Two floats at a time.
struct Two {
  unsigned long long v;
  __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Two operator*(Two a, Two b) {
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
  return a;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.v) : "l"(b.v), "l"(c.v));
  return a;
}

// ------------------------------------------------------------ 8-bit states
// A tile's values share the exponent E (a float's exponent field) of their
// largest magnitude.  A code is the top of the float whose exponent field is
// shifted so that E becomes TOP: 4 bits of exponent and a sign for the mean
// (TOP 14), 5 for the square (TOP 30, no sign), 3 of mantissa; what underflows
// the shifted field is a subnormal float and so a subnormal code.  A value
// that rounds up from the largest still has a code.
//
// The shift is a product with a power of two.  One that is not a float (E above
// TOP + 126, values of 2^(TOP - 1) and more) is split into two, which is rare enough
// for loops of its own.
constexpr int TOP_M = 14, TOP_V = 30;
__device__ __forceinline__ float pow2(int field) { return __int_as_float(field << 23); }
__device__ __forceinline__ uint32_t byte_of(uint2 c, int k) { return __byte_perm(k < 4 ? c.x : c.y, 0, 0x4440 | (k & 3)); }

template <int TOP>
__device__ __forceinline__ void decode_all(uint2 c, uint32_t e, float* x) {
  constexpr int MOST = TOP + 127;  // 2^(E - TOP) is a float up to here
  const float scale = e == 255 ? __int_as_float(0x7FC00000) : e ? pow2(min(int(e), MOST) + 127 - TOP) : 0.f;
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    uint32_t bits;
    if (TOP == TOP_M) {  // the code in the highest byte, its sign kept by the shift
      const uint32_t high = __byte_perm(k < 4 ? c.x : c.y, 0, 0x0444 | (k & 3) << 12);
      bits = uint32_t(int32_t(high) >> 4) & 0x87F00000u;
    } else {
      bits = byte_of(c, k) << 20;
    }
    x[k] = __uint_as_float(bits);
  }
#pragma unroll
  for (int k = 0; k < EACH; k += 2) (Two(x[k], x[k + 1]) * Two(scale)).get(x[k], x[k + 1]);
  if (e > MOST && e != 255) {
#pragma unroll
    for (int k = 0; k < EACH; ++k) x[k] *= pow2(int(e) - MOST + 127);
  }
}

// A lane's codes, as 8 bytes; the tile's exponent in e.  x is lost.  random: 16
// bits (for the mean the high ones, for the square the low ones) for each, or half a step.
template <int TOP>
__device__ __forceinline__ uint2 encode(float* x, const uint32_t* random, uint32_t& e) {
  constexpr int MOST = TOP + 126;  // 2^(TOP - E) is a float up to here
  uint32_t most = 0;
#pragma unroll
  for (int k = 0; k < EACH; ++k) most = max(most, TOP == TOP_M ? __float_as_uint(x[k]) * 2 : __float_as_uint(x[k]));
  most = __reduce_max_sync(~0u, most);
  const int field = max(int(TOP == TOP_M ? most >> 24 : most >> 23 & 255), 1);
  e = field < 254 ? field : 255;
  if (e == 255) return make_uint2(0, 0);
  if (field > MOST) {
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const float y = x[k] * pow2(127 + MOST - field);
      x[k] = TOP == TOP_V && x[k] > 0.f ? fmaxf(y, 0x1p-149f) : y;  // a square that is above 0 stays so, for the code below
    }
  }
  const float scale = pow2(127 + TOP - min(field, MOST));
  // A multiply-add where an addition and a shift would do: logic runs at half the rate.
  uint32_t y[EACH], t[EACH];
#pragma unroll
  for (int k = 0; k < EACH; k += 2) {
    float a, b;
    (Two(x[k], x[k + 1]) * Two(scale)).get(a, b);
    y[k] = __float_as_uint(a);
    y[k + 1] = __float_as_uint(b);
  }
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    t[k] = (TOP == TOP_M ? random[k] >> 16 : random[k] & 0xFFFFu) * 16 + y[k];
    if (TOP == TOP_V && x[k] > 0.f) t[k] = max(t[k], 1u << 20);  // a square never rounds to zero: the step divides by its root
    t[k] *= 16;  // the code in the highest byte
  }
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    w[k] = __byte_perm(__byte_perm(t[4 * k], t[4 * k + 1], 0x0073), __byte_perm(t[4 * k + 2], t[4 * k + 3], 0x0073), 0x5410);
    if (TOP == TOP_M)  // seven bits; the eighth is the sign
      w[k] |= 0x80808080u & __byte_perm(__byte_perm(y[4 * k], y[4 * k + 1], 0x0073), __byte_perm(y[4 * k + 2], y[4 * k + 3], 0x0073), 0x5410);
  }
  return make_uint2(w[0], w[1]);
}
template <bool WHOLE>
__device__ __forceinline__ uint2 read_codes(const uint8_t* p, uint32_t lane, uint32_t n) {
  if constexpr (WHOLE) {
    return *reinterpret_cast<const uint2*>(p + lane * EACH);
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < EACH; ++k)
      if (lane + k * 32 < n) w[k / 4] |= uint32_t(p[lane + k * 32]) << (k % 4 * 8);
    return make_uint2(w[0], w[1]);
  }
}
template <bool WHOLE>
__device__ __forceinline__ void write_codes(uint8_t* p, uint32_t lane, uint32_t n, uint2 c) {
  if constexpr (WHOLE) {
    *reinterpret_cast<uint2*>(p + lane * EACH) = c;
  } else {
#pragma unroll
    for (int k = 0; k < EACH; ++k)
      if (lane + k * 32 < n) p[lane + k * 32] = uint8_t((k < 4 ? c.x : c.y) >> (k % 4 * 8));
  }
}

// The square root and the quotient of the step are each within 2^-22 of their
// values, as is the rate: what a parameter changes by is exact to 20 bits or so.
// FLUSH: numbers below 2^-126 count as zero, which takes fewer instructions (159M
// elements, 8 bits, and their values: 597 us, 615 without).  Of a square that is a root of 2^-63,
// times 1 / sqrt(1 - beta2^t), at most 2^-22 of an eps of 2^-41 times that and more.  A rate
// times a mean below 2^-126 is lost, or has lost bits without FLUSH: what it would change is 2^-126
// over the divisor.
template <bool FLUSH>
__device__ __forceinline__ float root_of(float x) {
  float y;
  if constexpr (FLUSH) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  else asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool FLUSH>
__device__ __forceinline__ float quotient(float x, float y) {
  if constexpr (!FLUSH) return __fdividef(x, y);
  float q;
  asm("div.approx.ftz.f32 %0, %1, %2;" : "=f"(q) : "f"(x), "f"(y));
  return q;
}

struct Constants {
  float lr, scale, rate, root;  // root: of 1 / (1 - beta2^t)
  uint32_t key;
  bool flush;
};

// A lane's elements, a step on.
template <bool FLUSH>
__device__ __forceinline__ void step_values(const Common& c, const Constants& d, float keep, float* p, const float* g, float* m, float* v) {
#pragma unroll
  for (int k = 0; k < EACH; k += 2) {
    const Two x = Two(g[k], g[k + 1]) * Two(d.scale);
    // each product and sum rounded by itself: the states are the formula's, bit by bit
    // (sums by themselves: two packed ones become a fused one)
    float more[2], above[2], below[2];
    (Two(m[k], m[k + 1]) * Two(c.b1)).get(m[k], m[k + 1]);
    (x * Two(c.c1)).get(more[0], more[1]);
    m[k] = __fadd_rn(m[k], more[0]);
    m[k + 1] = __fadd_rn(m[k + 1], more[1]);
    (Two(v[k], v[k + 1]) * Two(c.b2)).get(v[k], v[k + 1]);
    (x * x * Two(c.c2)).get(more[0], more[1]);
    v[k] = __fadd_rn(v[k], more[0]);
    v[k + 1] = __fadd_rn(v[k + 1], more[1]);
    (Two(m[k], m[k + 1]) * Two(-d.rate)).get(above[0], above[1]);
    fma2(Two(root_of<FLUSH>(v[k]), root_of<FLUSH>(v[k + 1])), Two(d.root), Two(c.eps)).get(below[0], below[1]);
    fma2(Two(p[k], p[k + 1]), Two(keep), Two(quotient<FLUSH>(above[0], below[0]), quotient<FLUSH>(above[1], below[1]))).get(p[k], p[k + 1]);
  }
}

// One tile of n elements, at `at` of its tensor.
template <int BITS, bool WHOLE>
__device__ __forceinline__ void step_tile(const Common& c, const Constants& d, const Item& t, uint64_t at, uint32_t n) {
  const uint32_t lane = threadIdx.x % 32;
  const uint64_t s = t.first + at;
  float p[EACH], g[EACH], m[EACH], v[EACH];
  read_any<WHOLE>(t.grad, t.grad_type, at, lane, n, g);
  if (BITS == 32) {
    read<WHOLE>(static_cast<const float*>(c.m) + s, lane, n, m);
    read<WHOLE>(static_cast<const float*>(c.v) + s, lane, n, v);
  }
  uint2 cm, cv;
  uint32_t em, ev;
  if (BITS == 8) {
    cm = read_codes<WHOLE>(static_cast<const uint8_t*>(c.m) + s, lane, n);
    cv = read_codes<WHOLE>(static_cast<const uint8_t*>(c.v) + s, lane, n);
    em = c.m_exp[s / TILE];
    ev = c.v_exp[s / TILE];
  }
  if (c.master) read<WHOLE>(c.master + s, lane, n, p);
  else read_any<WHOLE>(t.param, t.param_type, at, lane, n, p);
  if (BITS == 8 && WHOLE && at + (WARPS + 1) * TILE <= t.n) {
    // the warp's next tile on its way to the cache: registers for it would cost warps
    constexpr uint32_t NEXT = WARPS * TILE;
    const uint32_t i = NEXT + lane * EACH;
    auto fetch = [](const void* q) { asm volatile("prefetch.global.L2 [%0];" ::"l"(q)); };
    fetch(static_cast<const char*>(t.grad) + (at + i) * (t.grad_type == PP_F32 ? 4 : 2));
    fetch(c.master ? reinterpret_cast<const char*>(c.master + s + i) : static_cast<const char*>(t.param) + (at + i) * (t.param_type == PP_F32 ? 4 : 2));
    fetch(static_cast<const uint8_t*>(c.m) + s + i);
    fetch(static_cast<const uint8_t*>(c.v) + s + i);
  }
  if (BITS == 8) {
    decode_all<TOP_M>(cm, em, m);
    decode_all<TOP_V>(cv, ev, v);
  }
  const float keep = 1.f - d.lr * t.decay;
  if (d.flush) step_values<true>(c, d, keep, p, g, m, v);
  else step_values<false>(c, d, keep, p, g, m, v);
  write_any<WHOLE>(t.param, t.param_type, at, lane, n, p);
  if (c.master) write<WHOLE>(c.master + s, lane, n, p);
  if (BITS == 32) {
    write<WHOLE>(static_cast<float*>(c.m) + s, lane, n, m);
    write<WHOLE>(static_cast<float*>(c.v) + s, lane, n, v);
    return;
  }
  uint32_t random[EACH];
  if (c.nearest) {
#pragma unroll
    for (int k = 0; k < EACH; ++k) random[k] = 0x80008000u;
  } else {
    // 32 hashed bits an element, half for each state; within a tile places differ in other bits than its
    // first, so they are joined by exclusive or
    const uint32_t place = (uint32_t(s) | (WHOLE ? lane * EACH : lane)) ^ mix(d.key + uint32_t(s >> 32));
#pragma unroll
    for (int k = 0; k < EACH; ++k) random[k] = mix(place ^ (WHOLE ? k : k * 32));
  }
  if (!WHOLE) {
#pragma unroll
    for (int k = 0; k < EACH; ++k)
      if (lane + k * 32 >= n) m[k] = v[k] = 0.f;  // no part of the tile's exponents
  }
  cm = encode<TOP_M>(m, random, em);
  cv = encode<TOP_V>(v, random, ev);
  write_codes<WHOLE>(static_cast<uint8_t*>(c.m) + s, lane, n, cm);
  write_codes<WHOLE>(static_cast<uint8_t*>(c.v) + s, lane, n, cv);
  if (lane == 0) {
    c.m_exp[s / TILE] = uint8_t(em);
    c.v_exp[s / TILE] = uint8_t(ev);
  }
}

template <int BITS, int CAP>
__global__ void __launch_bounds__(THREADS, RESIDENT) adamw_kernel(const __grid_constant__ Args<CAP> a) {
  const Common& c = a.c;
  if (c.skip_at && *c.skip_at != 0.f) return;
  const int step = c.counters[0] + 1;
  Constants d;
  d.lr = c.lr_at ? *c.lr_at : c.lr;
  d.scale = c.scale_at ? *c.scale_at : 1.f;
  // 1 - b^t without a difference of nearly equal numbers
  d.rate = d.lr / -expm1f(float(step) * c.log_b1);
  d.root = 1.f / sqrtf(-expm1f(float(step) * c.log_b2));
  d.key = mix(mix(c.seed) + uint32_t(step));
  d.flush = c.eps >= d.root * 0x1p-41f;
  // a block takes c.chunk tiles a turn, for which a tensor is looked up once
  for (uint32_t chunk = blockIdx.x * c.chunk; chunk < c.n_tiles; chunk += gridDim.x * c.chunk) {
    uint32_t i = 0;  // the last tensor that begins at or before the chunk
    for (uint32_t size = c.n_items; size > 1;) {
      const uint32_t half = size / 2;
      if (a.item[i + half].tile_begin <= chunk) i += half;
      size -= half;
    }
    const uint32_t stop = min(chunk + c.chunk, c.n_tiles);
    for (uint32_t tile = chunk + threadIdx.x / 32; tile < stop; tile += WARPS) {
      while (i + 1 < c.n_items && a.item[i + 1].tile_begin <= tile) ++i;
      const Item& t = a.item[i];
      const uint64_t at = uint64_t(tile - t.tile_begin) * TILE;
      const uint32_t n = uint32_t(t.n - at < TILE ? t.n - at : TILE);
      // 32 bytes an access, or element by element (67M elements, 32-bit states: f32 287 and 286 us, bf16 229
      // and 243; 8-bit states: f32 241 and 291, bf16 213 and 261)
      if (n == TILE && c.wide && (reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad)) % 32 == 0)
        step_tile<BITS, true>(c, d, t, at, n);
      else
        step_tile<BITS, false>(c, d, t, at, n);
    }
  }
  if (!c.last) return;
  // the block that is through last counts the step: by then every block has read the count
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(&c.counters[1], 1) == int(gridDim.x) - 1) {
    c.counters[1] = 0;
    c.counters[0] = step;
  }
}

template <class T, bool WHOLE>
__global__ void __launch_bounds__(THREADS) values_kernel(const uint8_t* m, const uint8_t* m_exp, const uint8_t* v,
                                                         const uint8_t* v_exp, uint32_t n_tiles, T* m_out, T* v_out) {
  const uint32_t lane = threadIdx.x % 32;
  for (uint32_t tile = blockIdx.x * WARPS + threadIdx.x / 32; tile < n_tiles; tile += gridDim.x * WARPS) {
    const uint64_t s = uint64_t(tile) * TILE;
    float x[EACH];
    if (m_out) {
      decode_all<TOP_M>(read_codes<WHOLE>(m + s, lane, TILE), m_exp[tile], x);
      write<WHOLE>(m_out + s, lane, TILE, x);
    }
    if (v_out) {
      decode_all<TOP_V>(read_codes<WHOLE>(v + s, lane, TILE), v_exp[tile], x);
      write<WHOLE>(v_out + s, lane, TILE, x);
    }
  }
}

cudaError_t grid_for(uint64_t tiles, uint32_t each, unsigned* grid) {
  int sms;
  const cudaError_t e = ppi::sm_count(&sms);
  *grid = unsigned(std::min<uint64_t>(std::max<uint64_t>((tiles + each - 1) / each, 1), uint64_t(sms) * BLOCKS));
  return e;
}

template <int CAP>
cudaError_t launch(const Common& c, const Item* items, int bits, cudaStream_t stream) {
  Args<CAP> a;
  a.c = c;
  std::memcpy(a.item, items, c.n_items * sizeof(Item));
  unsigned grid;
  const cudaError_t e = grid_for(c.n_tiles, c.chunk, &grid);
  if (e != cudaSuccess) return e;
  if (bits == 32) adamw_kernel<32, CAP><<<grid, THREADS, 0, stream>>>(a);
  else adamw_kernel<8, CAP><<<grid, THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

bool state_ok(const pp_adamw_state* s) {
  if (!s || (s->bits != 32 && s->bits != 8)) return false;
  if (s->n % TILE != 0) return false;
  if (s->n && (!s->d_exp_avg || !s->d_exp_avg_sq)) return false;
  if (!ppl::aligned(s->d_exp_avg, 16) || !ppl::aligned(s->d_exp_avg_sq, 16)) return false;
  return s->bits == 32 || !s->n || (s->d_exp_avg_exponent && s->d_exp_avg_sq_exponent);
}

}  // namespace

extern "C" pp_rc pp_adamw(const pp_adamw_tensor* tensors, size_t n_tensors, const pp_adamw_state* state,
                          const pp_adamw_opts* o, cudaStream_t stream) {
  if (!state_ok(state) || !o || (n_tensors && !tensors)) return PP_EINVAL;
  if (!state->d_counters || !ppl::aligned(state->d_counters, 4) || !ppl::aligned(state->d_master, 16)) return PP_EINVAL;
  if (!(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) || !(o->eps >= 0) || !std::isfinite(float(o->eps))) return PP_EINVAL;
  if (!o->d_lr && !(o->lr >= 0 && std::isfinite(float(o->lr)))) return PP_EINVAL;
  if (!ppl::aligned(o->d_lr, 4) || !ppl::aligned(o->d_grad_scale, 4) || !ppl::aligned(o->d_skip, 4)) return PP_EINVAL;
  if (state->n / TILE >= ppl::MAX_DIM) return PP_ETOOLARGE;
  for (size_t i = 0; i < n_tensors; ++i) {
    const pp_adamw_tensor& t = tensors[i];
    if (!ppl::ftype_ok(t.param_type) || !ppl::ftype_ok(t.grad_type) || !std::isfinite(t.weight_decay)) return PP_EINVAL;
    if (t.first % TILE != 0 || t.first > state->n || t.n > state->n - t.first) return PP_EINVAL;
    if (t.n && (!t.d_param || !t.d_grad || !ppl::aligned(t.d_param, ppl::fsize(t.param_type)) ||
                !ppl::aligned(t.d_grad, ppl::fsize(t.grad_type))))
      return PP_EINVAL;
  }
  Common c;
  std::memset(&c, 0, sizeof c);
  c.m = state->d_exp_avg;
  c.v = state->d_exp_avg_sq;
  c.m_exp = state->d_exp_avg_exponent;
  c.v_exp = state->d_exp_avg_sq_exponent;
  c.master = state->d_master;
  c.counters = state->d_counters;
  c.lr_at = o->d_lr;
  c.scale_at = o->d_grad_scale;
  c.skip_at = o->d_skip;
  c.lr = float(o->lr);
  c.b1 = float(o->beta1);
  c.c1 = float(1 - o->beta1);
  c.b2 = float(o->beta2);
  c.c2 = float(1 - o->beta2);
  c.eps = float(o->eps);
  c.log_b1 = float(std::log(o->beta1));
  c.log_b2 = float(std::log(o->beta2));
  c.seed = state->seed;
  c.nearest = state->nearest;
  c.wide = ppl::aligned(c.m, 32) && ppl::aligned(c.v, 32) && ppl::aligned(c.master, 32);
  constexpr size_t MOST = 640;
  Item items[MOST];
  size_t i = 0;
  do {  // once also without tensors: the step counts
    uint64_t tiles = 0;
    uint32_t n = 0;
    for (; i < n_tensors && n < MOST; ++i) {
      const pp_adamw_tensor& t = tensors[i];
      if (!t.n) continue;
      items[n++] = {t.d_param, t.d_grad, t.n, t.first, uint32_t(tiles), t.weight_decay, t.param_type, t.grad_type};
      tiles += (t.n + TILE - 1) / TILE;
      if (tiles >= ppl::MAX_DIM) return PP_ETOOLARGE;  // only where tensors share state
    }
    c.n_items = n;
    c.n_tiles = uint32_t(tiles);
    // up to 16 tiles a warp and turn, and eight turns a resident block: the next tile of a turn is
    // fetched ahead (159M elements, 8 bits, and their values: 634 us, and 660 with turns of 4 tiles)
    c.chunk = uint32_t(std::min<uint64_t>(std::max<uint64_t>(tiles / (152 * RESIDENT * 8 * WARPS), 1), 16)) * WARPS;
    c.last = i == n_tensors;
    // few tensors as fewer parameters: a launch for 9 takes the host 7.8 us, and 9.0 with all 31 KB
    const cudaError_t e = n <= 128 ? launch<128>(c, items, state->bits, stream) : launch<MOST>(c, items, state->bits, stream);
    if (e != cudaSuccess) return ppl::rc_of(e);
  } while (i < n_tensors);
  return PP_OK;
}

extern "C" pp_rc pp_adamw_values(const pp_adamw_state* state, pp_ftype type, void* d_exp_avg, void* d_exp_avg_sq,
                                 cudaStream_t stream) {
  if (!state_ok(state) || state->bits != 8 || !ppl::ftype_ok(type)) return PP_EINVAL;
  if (!ppl::aligned(d_exp_avg, 16) || !ppl::aligned(d_exp_avg_sq, 16)) return PP_EINVAL;
  if (state->n / TILE >= ppl::MAX_DIM) return PP_ETOOLARGE;
  if (!state->n || (!d_exp_avg && !d_exp_avg_sq)) return PP_OK;
  const uint32_t tiles = uint32_t(state->n / TILE);
  unsigned grid;
  const cudaError_t e = grid_for(tiles, WARPS, &grid);
  if (e != cudaSuccess) return ppl::rc_of(e);
  const uint8_t* m = static_cast<const uint8_t*>(state->d_exp_avg);
  const uint8_t* v = static_cast<const uint8_t*>(state->d_exp_avg_sq);
  const bool wide = ppl::aligned(d_exp_avg, 32) && ppl::aligned(d_exp_avg_sq, 32);
  auto go = [&](auto kernel, auto* mo, auto* vo) {
    kernel<<<grid, THREADS, 0, stream>>>(m, state->d_exp_avg_exponent, v, state->d_exp_avg_sq_exponent, tiles, mo, vo);
  };
  switch (type) {
    case PP_F32: go(wide ? values_kernel<float, true> : values_kernel<float, false>, static_cast<float*>(d_exp_avg), static_cast<float*>(d_exp_avg_sq)); break;
    case PP_F16: go(wide ? values_kernel<__half, true> : values_kernel<__half, false>, static_cast<__half*>(d_exp_avg), static_cast<__half*>(d_exp_avg_sq)); break;
    default: go(wide ? values_kernel<__nv_bfloat16, true> : values_kernel<__nv_bfloat16, false>, static_cast<__nv_bfloat16*>(d_exp_avg), static_cast<__nv_bfloat16*>(d_exp_avg_sq)); break;
  }
  return ppl::rc_of(cudaGetLastError());
}
