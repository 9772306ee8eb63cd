// pp_verify_drafts: drafted tokens against the target's probabilities, and the
// token after the last accepted one.
//
// A draft d of probability q is accepted where u * q < p, so with chance min(1,
// p / q); the first that is not is replaced by a token drawn from what the
// draft left of the target, max(p - q, 0), which makes every token one of the
// target's.  After a fully accepted draft the token comes from the target.
//
// A draw compares a random number with running sums over the vocabulary, and a
// sum of floats would depend on its order.  Probabilities count here as whole
// numbers of 2^-unit_bits (2^-45 for 131072 tokens): their sums are exact, so
// the token is the same however the row is shared out.
//
// A cluster of blocks takes a request.  Each block finds the accepted drafts for
// itself, sums its part of the row (of both rows after a draft that is not
// accepted), a segment a warp, and gives the sum to the other blocks; the block
// whose part holds the drawn sum looks for the token in that warp's segment.
//
// Bound by memory where there are many requests, and by the latency of its steps
// (two rounds of loads for the drafts, the sum, the exchange, the token) where
// there are few: 512 requests of 5 drafts and 131075 f32 tokens 75 us (372 MB, 5.0
// TB/s), 64 of 7 sure drafts and 131072 tokens 10 us, one of 4 and 32000 tokens 5.6.
//
// What was measured against it (512 requests): a ring of asynchronous copies for
// each warp 134 to 185 us where registers took 98 at the time, since the buffers
// leave room for fewer blocks; 64-bit conversions 323 us instead of 142; the token
// looked for by the segment's warp alone 109 us instead of 91.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using ppl::to_f;

constexpr int THREADS = 256, RESIDENT = 4, WARPS = THREADS / 32;
constexpr int CLUSTER = 8;  // blocks at most
// Loads of each row that a thread has on their way; blocks that a multiprocessor holds
// then.  512 x 131075: 75 us with 16 and four blocks, 90 with 8 and six.
constexpr int UNROLL = 16;
constexpr int FEW = 8;      // tokens of a thread that looks for one

struct VerifyArgs {
  const void* target;
  const void* probs;
  const void* drafts;
  const int32_t* target_row;
  const int32_t* probs_row;
  const int32_t* lengths;
  const float* accept;
  const float* sample;
  int32_t* tokens;
  int32_t* counts;
  uint64_t target_stride, probs_stride, drafts_stride, accept_stride, tokens_stride;
  uint32_t target_rows, probs_rows, n_drafts, n_vocab;
  uint32_t blocks, part;  // blocks of a cluster, tokens of a block
  int32_t draft_type;
  int32_t unit_bits;
  float scale;
};

// A probability's float: NaN counts as 0, values outside [0, 1] are cut.
template <class T>
__device__ __forceinline__ float prob(const T* p) { return __saturatef(to_f(*p)); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

// A probability in units, in PARTS digits of base 2^23.  Conversions to 64 bits
// run at 2 a clock and multiprocessor here, so there are none: 2^23 is added, rounding
// down, to what the digit is the whole part of, which leaves the digit in the low bits.
// The rest is exact, and so is its product with 2^23.
template <int PARTS>
struct Units {
  uint32_t digit[PARTS];  // each plus the bits of 2^23
  __device__ __forceinline__ Units(float p, float scale) {  // scale: 2^(unit_bits - 23 (PARTS - 1))
    constexpr float BASE = 8388608.f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const float up = __fmaf_rd(p, scale, BASE);
      digit[k] = __float_as_uint(up);
      if (k + 1 < PARTS) {
        p = fmaf(p, scale, BASE - up);
        scale = BASE;
      }
    }
  }
};

// A sum of such numbers, less others of as many: the bits of 2^23 cancel.
template <int PARTS>
struct Sum {
  int32_t digit[PARTS];
  __device__ __forceinline__ Sum() {
#pragma unroll
    for (int k = 0; k < PARTS; ++k) digit[k] = 0;
  }
  __device__ __forceinline__ void add(const Units<PARTS>& a, const Units<PARTS>& b) {
#pragma unroll
    for (int k = 0; k < PARTS; ++k) digit[k] += int32_t(a.digit[k] - b.digit[k]);
  }
  __device__ __forceinline__ uint64_t value() const {
    int64_t v = 0;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) v = v * (1 << 23) + digit[k];
    return uint64_t(v);
  }
};

// Tokens lo .. hi - 1 of a row: what token v weighs is P less Q where P is more.
// LESS: there is a q.  A token `gone` weighs nothing.
template <class T, int PARTS, bool LESS>
struct Segment {
  const T* p;
  const T* q;
  uint32_t lo, hi, gone;
  float scale;

  __device__ __forceinline__ void add(Sum<PARTS>& s, float a, float b) const {
    const Units<PARTS> x(a, scale), y(LESS ? b : 0.f, scale);
    // P is more than Q only where p is more than q
    if (!LESS || a > b) s.add(x, y);
  }
  __device__ __forceinline__ uint64_t weight(uint32_t v) const {
    Sum<PARTS> s;
    if (v < hi && v != gone) add(s, prob(p + v), LESS ? prob(q + v) : 0.f);
    return s.value();
  }
  __device__ __forceinline__ uint64_t sum() const {
    const uint32_t lane = threadIdx.x % 32;
    uint64_t total = 0;
    uint32_t v = lo + lane;
    auto batch = [&](bool whole) {
      float a[UNROLL], b[UNROLL];
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) a[i] = whole || v + i * 32 < hi ? prob(p + v + i * 32) : 0.f;
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) b[i] = LESS && (whole || v + i * 32 < hi) ? prob(q + v + i * 32) : 0.f;
      Sum<PARTS> s;  // digits below 2^23, UNROLL of them: no overflow
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) add(s, a[i], b[i]);
      total += s.value();
    };
    const uint32_t whole = hi > lo ? (hi - lo) / (UNROLL * 32) : 0;
    for (uint32_t k = 0; k < whole; ++k, v += UNROLL * 32) batch(true);
    if (v - lane < hi) batch(false);
    total = warp_sum(total);
    if (gone >= lo && gone < hi) {
      Sum<PARTS> s;
      add(s, prob(p + gone), LESS ? prob(q + gone) : 0.f);
      total -= s.value();
    }
    return total;
  }
  // The lowest token at which the running sum passes t, less than the whole, goes to *out.  All threads of the
  // block, each with a few tokens one behind the other, so that one scan over the threads does.
  __device__ __forceinline__ void pick(uint64_t t, uint64_t (&sums)[WARPS], int32_t* out) const {
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (uint32_t at = lo; at < hi; at += THREADS * FEW) {
      const uint32_t v = at + threadIdx.x * FEW;
      uint64_t w[FEW], x = 0;
#pragma unroll
      for (int i = 0; i < FEW; ++i) x += w[i] = weight(v + i);
      uint64_t run = x;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint64_t y = __shfl_up_sync(~0u, run, d);
        if (lane >= uint32_t(d)) run += y;
      }
      __syncthreads();  // all are done with what was in sums
      if (lane == 31) sums[warp] = run;
      __syncthreads();
      uint64_t before = run - x, all = 0;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        if (k < int(warp)) before += sums[k];
        all += sums[k];
      }
      if (t >= before && t - before < x) {
        t -= before;
        uint32_t k = 0;
#pragma unroll
        for (int i = 0; i < FEW; ++i) {  // the first whose running sum passes t
          const bool over = t < w[i];
          if (over) break;
          t -= w[i];
          ++k;
        }
        *out = int32_t(v + k);
      }
      if (t < all) return;  // for the thread that has just written, too: t is less than x then
      t -= all;
    }
  }
};

template <class T, bool SURE, int PARTS>
__global__ void __launch_bounds__(THREADS, RESIDENT) verify_kernel(const VerifyArgs a) {
  ppl::cluster_arrive();
  __shared__ uint64_t totals[2][CLUSTER];  // of the blocks, twice: by what the draft left, and by the target
  __shared__ uint64_t sums[WARPS];
  __shared__ uint32_t s_accepted, s_rejected, s_token;
  const uint32_t rank = blockIdx.x % a.blocks, r = blockIdx.x / a.blocks;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const T* target = static_cast<const T*>(a.target);
  const T* probs = static_cast<const T*>(a.probs);
  auto draft = [&](int i) { return ppl::load_id(a.drafts, a.draft_type, r * a.drafts_stride + i); };
  // what does not hang on one another is loaded at once
  const int most = int(a.n_drafts);
  const float u_sample = a.sample[r];
  int64_t d = -1;
  float u = 0.f;
  if (warp == 0 && int(lane) < most) {
    d = draft(lane);
    u = a.accept[r * a.accept_stride + lane];
  }
  const int64_t first = a.target_row ? int64_t(a.target_row[r]) : int64_t(r) * (a.n_drafts + 1);
  const int64_t qfirst = SURE ? 0 : a.probs_row ? int64_t(a.probs_row[r]) : int64_t(r) * a.n_drafts;
  const int n = a.lengths ? max(0, min(most, a.lengths[r])) : most;
  auto row = [&](int64_t i) -> const T* { return i >= 0 && i < int64_t(a.target_rows) ? target + uint64_t(i) * a.target_stride : nullptr; };
  auto qrow = [&](int64_t i) -> const T* { return i >= 0 && i < int64_t(a.probs_rows) ? probs + uint64_t(i) * a.probs_stride : nullptr; };
  if (warp == 0) {
    int accepted = n;
    int64_t token = -1;  // the draft that is not accepted
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + int(lane);
      bool bad = false;
      if (i < n) {
        if (i0) {
          d = draft(i);
          u = a.accept[r * a.accept_stride + i];
        }
        const T* p = row(first + i);
        const T* q = SURE ? nullptr : qrow(qfirst + i);
        bad = true;
        if (d >= 0 && d < int64_t(a.n_vocab) && p && (SURE || q)) {
          // 24 bits by 24 bits: the product is exact
          const float pd = prob(p + d), qd = SURE ? 1.f : prob(q + d);
          bad = !(u >= 0.f && double(u) * double(qd) < double(pd));
        }
      }
      const uint32_t some = __ballot_sync(~0u, bad);
      if (some) {
        accepted = i0 + __ffs(some) - 1;
        token = __shfl_sync(~0u, d, __ffs(some) - 1);
        break;
      }
    }
    if (lane == 0) {
      s_accepted = accepted;
      s_rejected = accepted < n;
      s_token = token >= 0 && token < int64_t(a.n_vocab) ? uint32_t(token) : ~0u;
    }
  }
  __syncthreads();
  const int j = int(s_accepted);
  bool lost = s_rejected != 0;
  const T* p = row(first + j);
  const T* q = !SURE && lost ? qrow(qfirst + j) : nullptr;
  uint32_t gone = SURE && lost ? s_token : ~0u;
  const uint32_t begin = min(rank * a.part, a.n_vocab), end = min(begin + a.part, a.n_vocab);
  const uint32_t each = (a.part + WARPS * 32 - 1) / (WARPS * 32) * 32;
  const uint32_t lo = min(begin + warp * each, end), hi = min(lo + each, end);
  uint64_t total = 0, before = 0, mine = 0;  // of all blocks, of those before this one, this block's
  const Segment<T, PARTS, true> less = {p, q, lo, hi, gone, a.scale};
  for (int round = 0; round < 2; ++round) {
    uint64_t s = 0;
    if (p) s = round || SURE || !q ? Segment<T, PARTS, false>{p, nullptr, lo, hi, round ? ~0u : gone, a.scale}.sum() : less.sum();
    if (lane == 0) sums[warp] = s;
    __syncthreads();
    if (round == 0) ppl::cluster_wait();
    if (warp == 0) {
      mine = warp_sum(lane < WARPS ? sums[lane] : 0);
      if (lane < a.blocks) {
        uint32_t to;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(uint32_t(__cvta_generic_to_shared(&totals[round][rank]))), "r"(lane));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(mine) : "memory");
      }
    }
    ppl::cluster_sync();
    total = before = 0;
    for (uint32_t b = 0; b < a.blocks; ++b) {
      if (b < rank) before += totals[round][b];
      if (b == rank) mine = totals[round][b];
      total += totals[round][b];
    }
    if (total || !lost) break;
    // the draft left nothing: the target's own probabilities
    lost = false;
    q = nullptr;
    gone = ~0u;
  }
  int32_t* out = a.tokens + r * a.tokens_stride;
  if (rank == 0) {
    for (int i = threadIdx.x; i <= int(a.n_drafts); i += THREADS)
      if (i != j || !total) out[i] = i < j ? int32_t(draft(i)) : -1;
    if (threadIdx.x == 0) a.counts[r] = j + (total ? 1 : 0);
  }
  if (!total) return;
  // the random number in units of 2^-31 of the total
  const uint32_t w = u_sample > 0.f ? (u_sample < 1.f ? uint32_t(u_sample * 2147483648.f) : 0x7FFFFFFFu) : 0;
  uint64_t t = __umul64hi(total, w) << 33 | (total * w) >> 31;
  if (t < before || t - before >= mine) return;
  t -= before;
  uint32_t k = 0;  // which warp's segment
  for (; t >= sums[k]; ++k) t -= sums[k];
  const uint32_t from = min(begin + k * each, end), to = min(from + each, end);
  if (SURE || !q) Segment<T, PARTS, false>{p, nullptr, from, to, gone, a.scale}.pick(t, sums, out + j);
  else Segment<T, PARTS, true>{p, q, from, to, gone, a.scale}.pick(t, sums, out + j);
}

template <class T, bool SURE, int PARTS>
cudaError_t launch(VerifyArgs& a, uint64_t n_requests, cudaStream_t stream) {
  // a block for each half of 152 multiprocessors' room at least, if with only 2048 tokens
  // each; beyond that as long as a block has 16384 tokens, for its steps cost it as
  // much time as some thousands of them (256 x 50001: two blocks a request 15 us, four 17;
  // 512 x 131075: four 75 us, two 80, three and five 77, eight 83)
  uint32_t blocks = 1;
  while (blocks < CLUSTER && n_requests * blocks < 1025 && a.n_vocab / (blocks * 2) >= (n_requests * blocks < 304 ? 2048 : 16384)) blocks *= 2;
  a.blocks = blocks;
  a.part = ((a.n_vocab + blocks - 1) / blocks + 31) / 32 * 32;
  cudaLaunchAttribute at;
  std::memset(&at, 0, sizeof at);
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(n_requests * blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, SURE, PARTS>, static_cast<const VerifyArgs>(a));
}

template <class T>
cudaError_t launch_type(VerifyArgs& a, uint64_t n, cudaStream_t stream) {
  // the highest of PARTS digits is at most 2^23
  if (a.unit_bits <= 46) {
    a.scale = std::ldexp(1.f, a.unit_bits - 23);
    return a.probs ? launch<T, false, 2>(a, n, stream) : launch<T, true, 2>(a, n, stream);
  }
  a.scale = std::ldexp(1.f, a.unit_bits - 46);
  return a.probs ? launch<T, false, 3>(a, n, stream) : launch<T, true, 3>(a, n, stream);
}

}  // namespace

extern "C" pp_rc pp_verify_drafts(const void* d_target, pp_ftype type, size_t target_rows, size_t n_vocab,
                                  size_t target_stride, const void* d_drafts, pp_itype draft_type,
                                  size_t n_requests, size_t n_drafts, size_t drafts_stride,
                                  const float* d_accept, size_t accept_stride, const float* d_sample,
                                  const pp_draft_opts* opts, int32_t* d_tokens, size_t tokens_stride,
                                  int32_t* d_counts, cudaStream_t stream) {
  if (!ppl::ftype_ok(type) || !ppl::itype_ok(draft_type)) return PP_EINVAL;
  pp_draft_opts o;
  std::memset(&o, 0, sizeof o);
  if (opts) o = *opts;
  if (n_requests >= ppl::MAX_DIM / CLUSTER || n_drafts >= (size_t(1) << 24) || n_vocab >= (size_t(1) << 30) || target_rows >= ppl::MAX_DIM ||
      o.probs_rows >= ppl::MAX_DIM)
    return PP_ETOOLARGE;
  if (!n_requests) return PP_OK;
  if (!n_vocab || !d_sample || !d_tokens || !d_counts || (target_rows && !d_target)) return PP_EINVAL;
  if (n_drafts && (!d_drafts || !d_accept)) return PP_EINVAL;
  if (n_requests > 1 && tokens_stride < n_drafts + 1) return PP_EINVAL;
  const size_t fs = ppl::fsize(type);
  if (!ppl::aligned(d_target, fs) || !ppl::aligned(o.d_probs, fs) || !ppl::aligned(d_drafts, ppl::isize(draft_type))) return PP_EINVAL;
  for (const void* four : {static_cast<const void*>(d_accept), static_cast<const void*>(d_sample), static_cast<const void*>(d_tokens),
                           static_cast<const void*>(d_counts), static_cast<const void*>(o.d_probs_row),
                           static_cast<const void*>(o.d_target_row), static_cast<const void*>(o.d_lengths)})
    if (!ppl::aligned(four, 4)) return PP_EINVAL;
  VerifyArgs a;
  std::memset(&a, 0, sizeof a);
  a.target = d_target;
  a.probs = n_drafts ? o.d_probs : nullptr;
  a.drafts = d_drafts;
  a.target_row = o.d_target_row;
  a.probs_row = o.d_probs_row;
  a.lengths = o.d_lengths;
  a.accept = d_accept;
  a.sample = d_sample;
  a.tokens = d_tokens;
  a.counts = d_counts;
  a.target_stride = target_stride;
  a.probs_stride = o.probs_stride;
  a.drafts_stride = drafts_stride;
  a.accept_stride = accept_stride;
  a.tokens_stride = tokens_stride;
  a.target_rows = uint32_t(target_rows);
  a.probs_rows = uint32_t(o.probs_rows);
  a.n_drafts = uint32_t(n_drafts);
  a.n_vocab = uint32_t(n_vocab);
  a.draft_type = draft_type;
  // n_vocab probabilities of at most 1 sum to less than 2^62 units
  a.unit_bits = 62;
  for (size_t v = n_vocab - 1; v; v >>= 1) --a.unit_bits;
  cudaError_t e;
  switch (type) {
    case PP_F32: e = launch_type<float>(a, n_requests, stream); break;
    case PP_F16: e = launch_type<__half>(a, n_requests, stream); break;
    default: e = launch_type<__nv_bfloat16>(a, n_requests, stream); break;
  }
  return ppl::rc_of(e);
}
