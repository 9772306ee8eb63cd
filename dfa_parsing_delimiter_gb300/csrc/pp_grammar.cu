// A vocabulary under a DFA (pp_vocab_grammar) and the DFA's states along
// token sequences (pp_grammar_states).
//
// A token is a short input of the DFA, so what it does is a state-transition
// vector (ParPaRaw Section 3.1): lane s holds the state reached from s.  A
// vector fits a 64-bit word, 16 nibbles; composing two is the parser's byte
// permute (stv16_compose).  Over tokens instead of bytes the same scan gives
// the state at every place of a sequence.
#include <cstring>

#include "pp_internal.h"
#include "pp_lm.cuh"
#include "pp_stv16.cuh"

namespace {

using namespace ppd;
using ppl::load_id;

struct VocabDfa {
  uint8_t byte_to_group[256];
  uint64_t row[PP_MAX_GROUPS];  // nibble s of row g: delta[g][s]
  uint32_t live;                // states from which an accepting state can be reached
  uint32_t accept;              // accepting ones among them
  int32_t n_states;
};

struct VocabArgs {
  const int32_t* offsets;
  const uint8_t* chars;
  int64_t chars_len;
  uint32_t n_vocab;
  int64_t end;
  uint64_t* vectors;
  uint32_t* allowed;
  uint64_t stride;
};

constexpr int VOCAB_THREADS = 256;
constexpr int VOCAB_LONG = 64;  // bytes from which a warp reads a token together

__device__ __forceinline__ Stv16 vocab_walk(const uint8_t* p, int64_t n, const Stv16* step) {
  Stv16 a = stv16_id();
  for (int64_t k = 0; k < n; ++k) a = stv16_compose(a, step[p[k]]);
  return a;
}

// A thread per token: its bytes composed one by one, then a ballot per state
// writes 32 tokens' bits.  A token of VOCAB_LONG bytes or more is read by
// its whole warp, a piece a lane, and the pieces are composed in order.
__global__ void __launch_bounds__(VOCAB_THREADS)
vocab_kernel(const __grid_constant__ VocabArgs p, const __grid_constant__ VocabDfa dfa) {
  __shared__ Stv16 step[256];
  step[threadIdx.x] = stv16_unpack(dfa.row[dfa.byte_to_group[threadIdx.x]]);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const uint64_t v = uint64_t(blockIdx.x) * VOCAB_THREADS + threadIdx.x;
  const bool there = v < p.n_vocab;
  int64_t lo = 0, n = 0;
  if (there) {
    lo = p.offsets[v];
    const int64_t hi = p.offsets[v + 1];
    n = lo >= 0 && hi >= lo && hi <= p.chars_len ? hi - lo : 0;
  }
  const bool ends = there && int64_t(v) == p.end;
  if (ends) n = 0;
  Stv16 a = stv16_id();
  if (n < VOCAB_LONG) a = vocab_walk(p.chars + lo, n, step);
  for (uint32_t todo = __ballot_sync(FULL, n >= VOCAB_LONG); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    const int64_t at = __shfl_sync(FULL, lo, src), all = __shfl_sync(FULL, n, src);
    const int64_t each = (all + 31) / 32, b = min(int64_t(lane) * each, all);
    Stv16 g = vocab_walk(p.chars + at + b, min(each, all - b), step);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const Stv16 up = shfl_up16(g, d);
      if (lane >= d) g = stv16_compose(up, g);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = __shfl_sync(FULL, g.w[k], 31);
      if (lane == src) a.w[k] = w;
    }
  }
  const uint64_t vec = stv16_pack(a);
  if (there) p.vectors[v] = vec;
  uint32_t mine = 0;
  for (int s = 0; s < dfa.n_states; ++s) {
    const uint32_t set = ends ? dfa.accept >> s : n > 0 && (dfa.live >> s & 1) ? dfa.live >> nib_apply(vec, s) : 0;
    const uint32_t word = __ballot_sync(FULL, set & 1);
    if (lane == s) mine = word;
  }
  const uint64_t w = v / 32;
  if (lane < dfa.n_states && w < p.stride) p.allowed[lane * p.stride + w] = mine;
}

// ------------------------------------------------------------------ states
struct StateArgs {
  const uint64_t* vectors;
  uint32_t n_vocab;
  int32_t n_states;
  const void* tokens;
  int32_t type;
  uint32_t n_rows, n_cols;
  uint64_t tstride;
  const int32_t* lengths;
  const uint8_t* start;
  uint64_t start_stride;
  uint8_t start_state;
  uint8_t* states;
  uint64_t sstride;
};

__device__ __forceinline__ uint32_t first_state(const StateArgs& p, uint64_t row) {
  const uint32_t s = p.start ? p.start[row * p.start_stride] : p.start_state;
  return s < uint32_t(p.n_states) ? s : PP_STATE_NONE;
}
__device__ __forceinline__ uint32_t row_length(const StateArgs& p, uint64_t row) {
  return p.lengths ? uint32_t(min(max(p.lengths[row], 0), int32_t(p.n_cols))) : p.n_cols;
}

// Few tokens a row (STATES_SHORT or fewer): a thread walks its row.
constexpr uint32_t STATES_SHORT = 16;
__global__ void __launch_bounds__(128) states_short_kernel(const __grid_constant__ StateArgs p) {
  const uint64_t row = uint64_t(blockIdx.x) * 128 + threadIdx.x;
  if (row >= p.n_rows) return;
  uint32_t s = first_state(p, row);
  const uint32_t len = row_length(p, row);
  uint8_t* out = p.states + row * p.sstride;
  out[0] = uint8_t(s);
  for (uint32_t t = 0; t < p.n_cols; ++t) {
    if (t < len && s != PP_STATE_NONE) {
      const int64_t tok = load_id(p.tokens, p.type, row * p.tstride + t);
      s = tok >= 0 && tok < p.n_vocab ? nib_apply(p.vectors[tok], s) : PP_STATE_NONE;
    }
    out[t + 1] = uint8_t(s);
  }
}

// Longer rows: the blocks of a cluster share a row, a part each.  A thread
// composes K tokens' vectors, the warp scans them, the block composes its
// warps' totals; each block tells the later ones its part's total, and after
// a cluster barrier the state that enters a part is known and passes through
// the warps' totals to the threads.  A part of up to STATES_THREADS x K
// tokens keeps its vectors in registers between the two steps; a longer one
// reads them twice.
constexpr int STATES_THREADS = 1024, STATES_WARPS = 32, STATES_BLOCKS = 8;

struct StateShared {
  uint64_t total[STATES_WARPS];  // the warps' vectors
  uint32_t lost[STATES_WARPS];   // a token outside the vocabulary among a warp's
  uint64_t part[STATES_BLOCKS];  // the earlier blocks' vectors, written by them
  uint32_t part_lost[STATES_BLOCKS];
  uint64_t tile;
  uint32_t tile_lost;
};

// One tile's vectors into registers and its warps' totals into shared memory.
template <int K, class I>
__device__ __forceinline__ void states_tile(const StateArgs& p, const I* tokens, uint64_t t0, uint64_t len,
                                            uint64_t (&vec)[K], uint32_t* bad, Stv16* before, uint32_t* dead,
                                            StateShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  int64_t tok[K];
#pragma unroll
  for (int k = 0; k < K; ++k) tok[k] = t0 + k < len ? int64_t(tokens[t0 + k]) : -1;
  *bad = K;  // this thread's first token outside the vocabulary
#pragma unroll
  for (int k = K - 1; k >= 0; --k) {
    const bool fine = tok[k] >= 0 && tok[k] < p.n_vocab;
    vec[k] = fine ? p.vectors[tok[k]] : 0xFEDCBA9876543210ull;  // the identity
    if (!fine && t0 + k < len) *bad = k;
  }
  Stv16 a = stv16_id();
  if (t0 < len) {
#pragma unroll
    for (int k = 0; k < K; ++k) a = stv16_compose(a, stv16_unpack(vec[k]));
  }
  __syncwarp();
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const Stv16 up = shfl_up16(a, d);
    if (lane >= d) a = stv16_compose(up, a);
  }
  *before = shfl_up16(a, 1);
  *dead = __ballot_sync(FULL, *bad < K);
  if (lane == 31) {
    sh.total[warp] = stv16_pack(a);
    sh.lost[warp] = *dead;
  }
}

template <int K, class I>
__device__ void states_row(const StateArgs& p, uint32_t blocks, uint32_t each, StateShared& sh, uint32_t* staged) {
  constexpr uint32_t TILE = STATES_THREADS * K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint64_t row = blockIdx.x / blocks;
  const uint32_t rank = blockIdx.x % blocks;
  const uint64_t begin = min(uint64_t(rank) * each, uint64_t(p.n_cols)), end = min(begin + each, uint64_t(p.n_cols));
  const uint64_t len = min(uint64_t(row_length(p, row)), end);
  const I* tokens = static_cast<const I*>(p.tokens) + row * p.tstride;
  uint8_t* out = p.states + row * p.sstride;
  uint64_t vec[K];
  uint32_t bad, dead, s = first_state(p, row);
  Stv16 before;
  if (rank == 0 && threadIdx.x == 0) out[0] = uint8_t(s);
  if (blocks > 1) {
    // the part's total, by warp 0
    Stv16 all = stv16_id();
    uint32_t gone = 0;
    for (uint64_t base = begin; base < end; base += TILE) {
      states_tile<K>(p, tokens, base + uint64_t(threadIdx.x) * K, len, vec, &bad, &before, &dead, sh);
      __syncthreads();
      if (warp == 0) {
        Stv16 a = stv16_unpack(sh.total[lane]);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const Stv16 up = shfl_up16(a, d);
          if (lane >= d) a = stv16_compose(up, a);
        }
        all = stv16_compose(all, a);  // lane 31 has them all
        gone |= __ballot_sync(FULL, sh.lost[lane] != 0);
      }
      if (base + TILE < end) __syncthreads();
    }
    if (warp == 0 && lane == 31)
      for (uint32_t q = rank + 1; q < blocks; ++q) {
        const uint64_t v = stv16_pack(all);
        uint32_t a, b;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(uint32_t(__cvta_generic_to_shared(&sh.part[rank]))), "r"(q));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(uint32_t(__cvta_generic_to_shared(&sh.part_lost[rank]))), "r"(q));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(b), "r"(gone) : "memory");
      }
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
    for (uint32_t q = 0; q < rank; ++q)
      if (s != PP_STATE_NONE) s = sh.part_lost[q] ? uint32_t(PP_STATE_NONE) : nib_apply(sh.part[q], s);
  }
  const bool kept = blocks > 1 && end - begin <= TILE;  // the one tile's vectors are still here
  for (uint64_t base = begin; base < end; base += TILE) {
    const uint64_t t0 = base + uint64_t(threadIdx.x) * K;
    if (!kept) {
      states_tile<K>(p, tokens, t0, len, vec, &bad, &before, &dead, sh);
      __syncthreads();
    }
    uint32_t q = s;
    for (int w = 0; w < STATES_WARPS; ++w) {
      if (w == warp) q = s;
      if (s != PP_STATE_NONE) s = sh.lost[w] ? uint32_t(PP_STATE_NONE) : nib_apply(sh.total[w], s);
    }
    if (q != PP_STATE_NONE && lane > 0) q = stv16_apply(before, q);
    if (dead & ((1u << lane) - 1)) q = PP_STATE_NONE;
#pragma unroll
    for (int g = 0; g < K / 4; ++g) {
      uint32_t four = 0;
#pragma unroll
      for (int k = 4 * g; k < 4 * g + 4; ++k) {
        if (uint32_t(k) >= bad) q = PP_STATE_NONE;
        if (q != PP_STATE_NONE) q = nib_apply(vec[k], q);
        four |= q << (8 * (k - 4 * g));
      }
      staged[threadIdx.x * (K / 4) + g] = four;
    }
    __syncthreads();
    // the tile's states, which begin at any byte, in words of memory
    uint8_t* to = out + base + 1;
    const uint32_t n = uint32_t(min(uint64_t(TILE), end - base));
    const uint32_t skip = min(uint32_t(-reinterpret_cast<intptr_t>(to)) & 3u, n), words = (n - skip) / 4;
    for (uint32_t w = threadIdx.x; w < words; w += STATES_THREADS)
      reinterpret_cast<uint32_t*>(to + skip)[w] = __funnelshift_r(staged[w], staged[w + 1], 8 * skip);
    const uint32_t rest = n - skip - 4 * words;
    if (threadIdx.x < skip) to[threadIdx.x] = reinterpret_cast<uint8_t*>(staged)[threadIdx.x];
    if (threadIdx.x < rest) to[n - rest + threadIdx.x] = reinterpret_cast<uint8_t*>(staged)[n - rest + threadIdx.x];
    if (base + TILE < end) __syncthreads();
  }
}

template <int K>
__global__ void __launch_bounds__(STATES_THREADS, 1)
states_kernel(const __grid_constant__ StateArgs p, uint32_t blocks, uint32_t each) {
  __shared__ StateShared sh;
  __shared__ __align__(16) uint32_t staged[STATES_THREADS * K / 4 + 1];
  switch (p.type) {
    case PP_U8: return states_row<K, uint8_t>(p, blocks, each, sh, staged);
    case PP_I8: return states_row<K, int8_t>(p, blocks, each, sh, staged);
    case PP_I32: return states_row<K, int32_t>(p, blocks, each, sh, staged);
    default: return states_row<K, int64_t>(p, blocks, each, sh, staged);
  }
}

cudaError_t launch_states(const StateArgs& p, cudaStream_t stream) {
  // a cluster shares a row while there are fewer blocks than 152
  // multiprocessors and a part keeps 1024 tokens
  uint32_t blocks = 1;
  while (blocks < STATES_BLOCKS && uint64_t(p.n_rows) * blocks < 152 && p.n_cols / (2 * blocks) >= 1024) blocks *= 2;
  const uint32_t each = uint32_t((uint64_t(p.n_cols) + blocks - 1) / blocks);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  std::memset(&at, 0, sizeof at);
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.gridDim = dim3(p.n_rows * blocks);
  cfg.blockDim = dim3(STATES_THREADS);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, each <= STATES_THREADS * 4 ? states_kernel<4> : states_kernel<16>, p, blocks, each);
}

// Per state, whether an accepting state can be reached from it without
// passing through the invalid state.
uint32_t live_states(const pp_dfa_desc* d) {
  uint32_t in = 0, live = 0;
  for (int s = 0; s < d->n_states; ++s)
    if (s != d->invalid_state) in |= 1u << s;
  uint32_t used = 0;  // groups that some byte has
  for (int b = 0; b < 256; ++b) used |= 1u << d->byte_to_group[b];
  live = d->accept_mask & in;
  for (uint32_t before = ~live; before != live;) {
    before = live;
    for (int s = 0; s < d->n_states; ++s)
      for (int g = 0; g < d->n_groups; ++g)
        if ((in >> s & 1) && (used >> g & 1) && (live >> d->delta[g][s] & 1)) live |= 1u << s;
  }
  return live;
}

}  // namespace

extern "C" {

pp_rc pp_vocab_grammar(const int32_t* d_offsets, const uint8_t* d_chars, size_t chars_len,
                       size_t n_vocab, const pp_dfa_desc* dfa, int64_t end_token,
                       uint64_t* d_vectors, uint32_t* d_allowed, size_t allowed_stride,
                       cudaStream_t stream) {
  if (!ppi::generic_dfa_ok(dfa) || (chars_len && !d_chars)) return PP_EINVAL;
  if (n_vocab && (!d_offsets || !d_vectors || !d_allowed)) return PP_EINVAL;
  if (end_token < -1 || (end_token >= 0 && uint64_t(end_token) >= n_vocab)) return PP_EINVAL;
  if (n_vocab >= ppl::MAX_DIM) return PP_ETOOLARGE;
  if (allowed_stride < (n_vocab + 31) / 32) return PP_EINVAL;
  if (!n_vocab) return PP_OK;
  VocabDfa g;
  std::memset(&g, 0, sizeof g);
  std::memcpy(g.byte_to_group, dfa->byte_to_group, 256);
  for (int r = 0; r < PP_MAX_GROUPS; ++r)
    for (int s = 0; s < PP_MAX_STATES; ++s) {
      const uint64_t to = r < dfa->n_groups && s < dfa->n_states ? dfa->delta[r][s] : s;
      g.row[r] |= to << (4 * s);
    }
  g.live = live_states(dfa);
  g.accept = dfa->accept_mask & g.live;
  g.n_states = dfa->n_states;
  const VocabArgs p = {d_offsets, d_chars, int64_t(chars_len), uint32_t(n_vocab), end_token,
                       d_vectors, d_allowed, allowed_stride};
  const uint64_t blocks = (n_vocab + VOCAB_THREADS - 1) / VOCAB_THREADS;
  vocab_kernel<<<unsigned(blocks), VOCAB_THREADS, 0, stream>>>(p, g);
  return ppl::rc_of(cudaGetLastError());
}

pp_rc pp_grammar_states(const uint64_t* d_vectors, size_t n_vocab, int n_states,
                        const void* d_tokens, pp_itype token_type, size_t n_rows, size_t n_cols,
                        size_t tokens_stride, const int32_t* d_lengths, const uint8_t* d_start,
                        size_t start_stride, uint8_t start_state, uint8_t* d_states,
                        size_t states_stride, cudaStream_t stream) {
  if (n_states < 1 || n_states > PP_MAX_STATES || !ppl::itype_ok(token_type)) return PP_EINVAL;
  if (n_rows && (!d_states || (n_cols && (!d_tokens || (n_vocab && !d_vectors))))) return PP_EINVAL;
  if (n_rows > 1 && states_stride < n_cols + 1) return PP_EINVAL;
  if (n_rows >= ppl::MAX_DIM || n_cols >= ppl::MAX_DIM || n_vocab >= ppl::MAX_DIM)
    return PP_ETOOLARGE;
  if (!n_rows) return PP_OK;
  const StateArgs p = {d_vectors, uint32_t(n_vocab), n_states, d_tokens, token_type,
                       uint32_t(n_rows), uint32_t(n_cols), tokens_stride, d_lengths, d_start,
                       start_stride, start_state, d_states, states_stride};
  if (n_cols <= STATES_SHORT)
    states_short_kernel<<<unsigned((n_rows + 127) / 128), 128, 0, stream>>>(p);
  else
    return ppl::rc_of(launch_states(p, stream));
  return ppl::rc_of(cudaGetLastError());
}

}  // extern "C"
