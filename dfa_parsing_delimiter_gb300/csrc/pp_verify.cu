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
// itself, sums its part of the row, a segment a warp, and gives the sum to the
// other blocks; the warp whose segment holds the drawn sum reads it again.
#include <algorithm>
#include <cstring>

#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using ppl::to_f;

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int CLUSTER = 8;  // blocks at most
constexpr int UNROLL = 8;

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
  float unit;  // 2^unit_bits
};

// A probability's float: NaN counts as 0, values outside [0, 1] are cut.
template <class T>
__device__ __forceinline__ float prob(const T* p) { return fminf(fmaxf(to_f(*p), 0.f), 1.f); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

// What token v of the row weighs.  SURE: the draft's probability is all at one
// token.  left: the draft's part is taken off.
template <class T, bool SURE>
__device__ __forceinline__ uint64_t weight(const T* p, const T* q, uint32_t v, uint32_t gone, float unit) {
  const uint64_t a = __float2ull_rz(prob(p + v) * unit);
  if (SURE) return v == gone ? 0 : a;
  const uint64_t b = q ? __float2ull_rz(prob(q + v) * unit) : 0;
  return a > b ? a - b : 0;
}

// The sum of this warp's segment.
template <class T, bool SURE>
__device__ __forceinline__ uint64_t segment_sum(const T* p, const T* q, uint32_t lo, uint32_t hi, uint32_t gone, float unit) {
  uint64_t s = 0;
  uint32_t v = lo + threadIdx.x % 32;
  for (; v + (UNROLL - 1) * 32 < hi; v += UNROLL * 32) {
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) s += weight<T, SURE>(p, q, v + k * 32, gone, unit);
  }
  for (; v < hi; v += 32) s += weight<T, SURE>(p, q, v, gone, unit);
  return warp_sum(s);
}

// The lowest token of the segment at which the running sum passes t.
template <class T, bool SURE>
__device__ __forceinline__ uint32_t segment_pick(const T* p, const T* q, uint32_t lo, uint32_t hi, uint32_t gone, float unit, uint64_t t) {
  const uint32_t lane = threadIdx.x % 32;
  for (uint32_t at = lo; at < hi; at += 32) {
    const uint32_t v = at + lane;
    uint64_t x = v < hi ? weight<T, SURE>(p, q, v, gone, unit) : 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint64_t y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    const uint32_t past = __ballot_sync(~0u, x > t);
    if (past) return at + __ffs(past) - 1;
    t -= __shfl_sync(~0u, x, 31);
  }
  return lo;  // not reached: the segment's sum is above t
}

template <class T, bool SURE>
__global__ void __launch_bounds__(THREADS) verify_kernel(const VerifyArgs a) {
  ppl::cluster_arrive();
  __shared__ uint64_t totals[2][CLUSTER];  // of the blocks, twice: by what the draft left, and by the target
  __shared__ uint64_t sums[WARPS];
  __shared__ uint32_t s_accepted, s_rejected, s_token;
  const uint32_t rank = blockIdx.x % a.blocks, r = blockIdx.x / a.blocks;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const T* target = static_cast<const T*>(a.target);
  const T* probs = static_cast<const T*>(a.probs);
  const int64_t first = a.target_row ? int64_t(a.target_row[r]) : int64_t(r) * (a.n_drafts + 1);
  const int64_t qfirst = SURE ? 0 : a.probs_row ? int64_t(a.probs_row[r]) : int64_t(r) * a.n_drafts;
  int n = int(a.n_drafts);
  if (a.lengths) n = max(0, min(n, a.lengths[r]));
  auto row = [&](int64_t i) -> const T* { return i >= 0 && i < int64_t(a.target_rows) ? target + uint64_t(i) * a.target_stride : nullptr; };
  auto qrow = [&](int64_t i) -> const T* { return i >= 0 && i < int64_t(a.probs_rows) ? probs + uint64_t(i) * a.probs_stride : nullptr; };
  auto draft = [&](int i) { return ppl::load_id(a.drafts, a.draft_type, r * a.drafts_stride + i); };
  if (warp == 0) {
    int accepted = n;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + int(lane);
      bool bad = false;
      if (i < n) {
        const int64_t d = draft(i);
        const float u = a.accept[r * a.accept_stride + i];
        const T* p = row(first + i);
        const T* q = SURE ? nullptr : qrow(qfirst + i);
        bad = true;
        if (d >= 0 && d < int64_t(a.n_vocab) && p && (SURE || q)) {
          // 24 bits by 24 bits: the product is exact
          const double share = SURE ? double(u) : double(u) * double(prob(q + d));
          bad = !(u >= 0.f && share < double(prob(p + d)));
        }
      }
      const uint32_t some = __ballot_sync(~0u, bad);
      if (some) {
        accepted = i0 + __ffs(some) - 1;
        break;
      }
    }
    if (lane == 0) {
      s_accepted = accepted;
      s_rejected = accepted < n;
      const int64_t d = accepted < n ? draft(accepted) : -1;
      s_token = d >= 0 && d < int64_t(a.n_vocab) ? uint32_t(d) : ~0u;
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
  for (int round = 0; round < 2; ++round) {
    const uint64_t s = p ? segment_sum<T, SURE>(p, q, lo, hi, gone, a.unit) : 0;
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
  const float u = a.sample[r];
  const uint32_t w = u > 0.f ? (u < 1.f ? uint32_t(u * 2147483648.f) : 0x7FFFFFFFu) : 0;
  uint64_t t = __umul64hi(total, w) << 33 | (total * w) >> 31;
  if (t < before || t - before >= mine) return;
  t -= before;
  for (int k = 0; k < WARPS; ++k) {  // which warp's segment
    const uint64_t s = sums[k];
    if (t < s) {
      if (int(warp) == k) {
        const uint32_t v = segment_pick<T, SURE>(p, q, lo, hi, gone, a.unit, t);
        if (lane == 0) out[j] = int32_t(v);
      }
      return;
    }
    t -= s;
  }
}

template <class T, bool SURE>
cudaError_t launch(VerifyArgs& a, uint64_t n_requests, cudaStream_t stream) {
  // as many blocks a request as fill 152 multiprocessors four times, none of
  // fewer than 2048 tokens
  uint32_t blocks = 1;
  while (blocks < CLUSTER && n_requests * blocks < 608 && a.n_vocab / (blocks * 2) >= 2048) blocks *= 2;
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
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, SURE>, static_cast<const VerifyArgs>(a));
}

template <class T>
cudaError_t launch_type(VerifyArgs& a, uint64_t n, cudaStream_t stream) {
  return a.probs ? launch<T, false>(a, n, stream) : launch<T, true>(a, n, stream);
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
  int bits = 62;
  for (size_t v = n_vocab - 1; v; v >>= 1) --bits;
  a.unit = float(uint64_t(1) << bits);
  cudaError_t e;
  switch (type) {
    case PP_F32: e = launch_type<float>(a, n_requests, stream); break;
    case PP_F16: e = launch_type<__half>(a, n_requests, stream); break;
    default: e = launch_type<__nv_bfloat16>(a, n_requests, stream); break;
  }
  return ppl::rc_of(e);
}
