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

// State-transition vectors of DFAs with up to 8 states: the low half of the
// 16-lane form of pp_stv16.cuh, at 8 instead of 28 instructions a
// composition.  Map<16> is that form itself.
template <int S> struct Map;
template <> struct Map<16> {
  using Packed = uint64_t;
  Stv16 g;
  static constexpr Packed ID = 0xFEDCBA9876543210ull;
  static __device__ __forceinline__ Map id() { return {stv16_id()}; }
  static __device__ __forceinline__ Map unpack(Packed v) { return {stv16_unpack(v)}; }
  __device__ __forceinline__ Packed pack() const { return stv16_pack(g); }
  __device__ __forceinline__ Map then(const Map& b) const { return {stv16_compose(g, b.g)}; }
  __device__ __forceinline__ Map up(int d) const { return {shfl_up16(g, d)}; }
  __device__ __forceinline__ uint32_t apply(uint32_t s) const { return stv16_apply(g, s); }
  static __device__ __forceinline__ Packed load(const uint64_t* v, uint64_t i) { return v[i]; }
};
template <> struct Map<8> {
  using Packed = uint32_t;
  uint32_t w[2];  // lanes 0-3, 4-7, a byte each
  static constexpr Packed ID = 0x76543210u;
  static __device__ __forceinline__ Map id() { return {{0x03020100u, 0x07060504u}}; }
  static __device__ __forceinline__ Map unpack(Packed v) {
    const uint32_t ev = v & 0x0F0F0F0Fu, od = (v >> 4) & 0x0F0F0F0Fu;
    return {{prmt(ev, od, 0x5140u), prmt(ev, od, 0x7362u)}};
  }
  __device__ __forceinline__ Packed pack() const { return prmt(w[0] | (w[0] >> 4), w[1] | (w[1] >> 4), 0x6420u); }
  __device__ __forceinline__ Map then(const Map& b) const {
    Map r;
#pragma unroll
    for (int k = 0; k < 2; ++k) r.w[k] = prmt(b.w[0], b.w[1], prmt(w[k] | (w[k] >> 4), 0u, 0x0020u));
    return r;
  }
  __device__ __forceinline__ Map up(int d) const {
    return {{__shfl_up_sync(FULL, w[0], d), __shfl_up_sync(FULL, w[1], d)}};
  }
  __device__ __forceinline__ uint32_t apply(uint32_t s) const { return ((s & 4 ? w[1] : w[0]) >> (8 * (s & 3))) & 0xFFu; }
  static __device__ __forceinline__ Packed load(const uint64_t* v, uint64_t i) {
    return reinterpret_cast<const uint32_t*>(v)[2 * i];  // the low half
  }
};

// Inclusive scan of a warp's maps.
template <class M>
__device__ __forceinline__ M warp_scan(M a) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int d = 1; d < 32; d *= 2) {
    const M up = a.up(d);
    if (lane >= d) a = up.then(a);
  }
  return a;
}

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

template <class M>
__device__ __forceinline__ M vocab_walk(const uint8_t* p, int64_t n, const M* step) {
  M a = M::id();
  for (int64_t k = 0; k < n; ++k) a = a.then(step[p[k]]);
  return a;
}

// The vectors of a warp's 32 tokens (n bytes at lo each, one behind the
// other, `all` in total, at most VOCAB_BYTES): every lane composes an equal
// share of the bytes, whatever tokens they belong to.  What a lane has of the
// token that it begins in is completed by a segmented scan of what the lanes
// before it left open.  marks: the tokens' last bytes; done: the vectors of
// the tokens that have bytes, in order.
constexpr uint32_t VOCAB_BYTES = 2048;
template <class M>
__device__ __forceinline__ typename M::Packed vocab_share(const uint8_t* p, uint32_t at, uint32_t n, uint32_t all,
                                                          const M* step, uint32_t* marks, typename M::Packed* done) {
  const int lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1;
  marks[lane] = marks[lane + 32] = 0;
  __syncwarp();
  if (n) atomicOr(&marks[(at + n - 1) / 32], 1u << ((at + n - 1) % 32));
  const uint32_t some = __ballot_sync(FULL, n > 0), each = (all + 31) / 32;
  __syncwarp();
  const uint32_t begin = min(lane * each, all), end = min(begin + each, all);
  int l = 0;  // the token that holds byte `begin`: the first that ends after it
#pragma unroll
  for (int d = 16; d; d /= 2)
    if (__shfl_sync(FULL, at + n, l + d - 1) <= begin) l += d;
  uint32_t r = __popc(some & ((1u << (l & 31)) - 1)), first = r;
  M a = M::id(), head = a;
  bool ended = false;  // the lane's first token
  for (uint32_t k = begin; k < end; ++k) {
    a = a.then(step[p[k]]);
    if (marks[k / 32] >> (k % 32) & 1) {
      if (ended) done[r] = a.pack();
      else head = a;
      ended = true;
      a = M::id();
      ++r;
    }
  }
  __syncwarp();
  uint32_t cut = ended;  // a holds what is open since an end, not since the lane's first byte
#pragma unroll 1
  for (int d = 1; d < 32; d *= 2) {
    const M up = a.up(d);
    const uint32_t up_cut = __shfl_up_sync(FULL, cut, d);
    if (lane >= d && !cut) {
      a = up.then(a);
      cut = up_cut;
    }
  }
  const M open = a.up(1);
  if (ended) done[first] = lane ? open.then(head).pack() : head.pack();
  __syncwarp();
  return n ? done[__popc(some & below)] : M::ID;
}

// A warp's 32 tokens together where they lie one behind the other with no
// more than VOCAB_BYTES bytes, as in any ordinary vocabulary; else a thread a
// token, but tokens of VOCAB_LONG bytes or more by their whole warp, a piece
// a lane, the pieces composed in order.  Then a ballot per state writes 32
// tokens' bits.
//
// Bound by instructions: 262144 tokens of 8 bytes on average under 16 states
// take 9.9 M of a warp, 6.0 M of them on the ALU pipe (71 % of its rate), in 15
// us; a third are the compositions of bytes and of the scan, the rest the
// bytes, the marks, the branch at a token's end and the ballots around them.
// With a thread a token a warp takes as long as its longest token: 24 us.
template <int S>
__global__ void __launch_bounds__(VOCAB_THREADS)
vocab_kernel(const __grid_constant__ VocabArgs p, const __grid_constant__ VocabDfa dfa) {
  using M = Map<S>;
  __shared__ M step[256];
  __shared__ uint32_t marks[VOCAB_THREADS / 32][VOCAB_BYTES / 32];
  __shared__ typename M::Packed done[VOCAB_THREADS / 32][32];
  step[threadIdx.x] = M::unpack(typename M::Packed(dfa.row[dfa.byte_to_group[threadIdx.x]]));
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
  const int64_t lo0 = __shfl_sync(FULL, lo, 0), hi = lo + n, before = __shfl_up_sync(FULL, hi, 1);
  const int64_t all = __shfl_sync(FULL, hi, 31) - lo0;
  const bool together = __all_sync(FULL, there && (lane == 0 || lo == before)) && all <= VOCAB_BYTES;
  typename M::Packed packed;
  if (together) {
    packed = vocab_share<M>(p.chars + lo0, uint32_t(lo - lo0), uint32_t(n), uint32_t(all), step, marks[threadIdx.x / 32],
                            done[threadIdx.x / 32]);
  } else {
    packed = (n < VOCAB_LONG ? vocab_walk(p.chars + lo, n, step) : M::id()).pack();
    for (uint32_t todo = __ballot_sync(FULL, n >= VOCAB_LONG); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int64_t at = __shfl_sync(FULL, lo, src), size = __shfl_sync(FULL, n, src);
      const int64_t each = (size + 31) / 32, b = min(int64_t(lane) * each, size);
      const M g = warp_scan(vocab_walk(p.chars + at + b, min(each, size - b), step));
      const typename M::Packed whole = __shfl_sync(FULL, g.pack(), 31);
      if (lane == src) packed = whole;
    }
  }
  if (ends) {
    n = 0;
    packed = M::ID;
  }
  const uint64_t vec = S == 8 ? 0xFEDCBA9800000000ull | packed : packed;
  if (there) p.vectors[v] = vec;
  // bit s: state s allows the token
  uint32_t set = 0;
#pragma unroll
  for (int s = 0; s < S; ++s) set |= (dfa.live >> (uint32_t(packed >> (4 * s)) & 15) & 1) << s;
  set = ends ? dfa.accept : n > 0 ? set & dfa.live : 0;
  uint32_t mine = 0;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const uint32_t word = __ballot_sync(FULL, set >> s & 1);
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

// Few tokens a row, or many rows: a thread walks its row, the vectors of
// STATES_BATCH tokens on their way at a time.  That takes 0.28 us a column
// while the rows fit the machine, and a block a row 0.0135 us a row (of up to
// 2560 tokens): 8192 rows of 64 tokens take 21 us here and 113 there, 2048
// rows of 256 75 and 33, so rows of up to a 20th of their number go here.
constexpr uint32_t STATES_SHORT = 16, STATES_MANY = 20;
constexpr int STATES_BATCH = 4;
__global__ void __launch_bounds__(128) states_short_kernel(const __grid_constant__ StateArgs p) {
  const uint64_t row = uint64_t(blockIdx.x) * 128 + threadIdx.x;
  if (row >= p.n_rows) return;
  uint32_t s = first_state(p, row);
  const uint32_t len = row_length(p, row);
  uint8_t* out = p.states + row * p.sstride;
  out[0] = uint8_t(s);
  for (uint32_t t = 0; t < p.n_cols; t += STATES_BATCH) {
    int64_t tok[STATES_BATCH];
    uint64_t vec[STATES_BATCH];
#pragma unroll
    for (int k = 0; k < STATES_BATCH; ++k) tok[k] = t + k < len ? load_id(p.tokens, p.type, row * p.tstride + t + k) : -1;
#pragma unroll
    for (int k = 0; k < STATES_BATCH; ++k) vec[k] = tok[k] >= 0 && tok[k] < p.n_vocab ? p.vectors[tok[k]] : 0;
#pragma unroll
    for (int k = 0; k < STATES_BATCH; ++k) {
      if (t + k < len && s != PP_STATE_NONE)
        s = tok[k] >= 0 && tok[k] < p.n_vocab ? nib_apply(vec[k], s) : PP_STATE_NONE;
      if (t + k < p.n_cols) out[t + k + 1] = uint8_t(s);
    }
  }
}

// Longer rows: the blocks of a cluster share a row, a part each.  A thread
// composes K tokens' vectors, the warp scans them, the block composes its
// warps' totals; each block tells the later ones its part's total, and after
// a cluster barrier the state that enters a part is known and passes through
// the warps' totals to the threads.  A part of up to STATES_THREADS x K
// tokens keeps its vectors in registers between the two steps; a longer one
// reads them twice.
//
// Bound by the latency of its steps, barriers first (16 rows of 65537 tokens
// under 5 states: 13.4 us, issue 38 %), not by memory.  Two blocks share a
// multiprocessor, so that clusters of 16 fill the machine (with one, only 15
// clusters of 8 run at once, and 16 rows take two waves, 27 us).  Threads a
// block: more of them hold a longer part in one tile, whose tokens are read
// once, and pay more for their barriers.  16 rows under 5 and 16 states, us:
//   tokens a row   20000        50000        65537        100000       200000
//   512 threads     9.1, 12.0   12.2, 15.9   26.8, 40.3   30.7, 44.7   55.2, 84.0
//   640            10.1, 13.3   13.4, 18.6   14.1, 19.5   32.4, 51.3   49.9, 78.0
//   768            12.0, 15.8   15.4, 18.3   16.5, 19.3   37.9, 55.5   59.4, 85.5
// (one tile up to 65536, 81920 and 98304).  The 16-lane form of 8 tokens a
// thread spills 88 bytes at the 48 registers that two blocks leave.
constexpr int STATES_THREADS = 640, STATES_WARPS = STATES_THREADS / 32, STATES_BLOCKS = 16;

struct StateShared {
  uint64_t total[STATES_WARPS];  // the warps' vectors, then those of all up to each
  uint32_t lost[STATES_WARPS];   // a token outside the vocabulary among a warp's
  uint32_t lost_mask;            // bit w: warp w has one
  uint64_t part[STATES_BLOCKS];  // the earlier blocks' vectors, written by them
  uint32_t part_lost[STATES_BLOCKS];
};

// One tile's vectors into registers, and the vectors from the tile's begin to
// each warp's end into shared memory.
template <class M, int K, class I>
__device__ __forceinline__ void states_tile(const StateArgs& p, const I* tokens, uint32_t t0, uint32_t len,
                                            typename M::Packed (&vec)[K], uint32_t* bad, M* before, uint32_t* dead,
                                            StateShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  I tok[K];
#pragma unroll
  for (int k = 0; k < K; ++k) tok[k] = t0 + k < len ? tokens[t0 + k] : I(0);
  *bad = K;  // this thread's first token outside the vocabulary
#pragma unroll
  for (int k = K - 1; k >= 0; --k) {
    // an id below 0 turns into one past the vocabulary
    const bool there = t0 + k < len, fine = sizeof(I) == 8 ? uint64_t(tok[k]) < p.n_vocab : uint32_t(tok[k]) < p.n_vocab;
    vec[k] = there && fine ? M::load(p.vectors, uint32_t(tok[k])) : M::ID;
    if (there && !fine) *bad = k;
  }
  M a = M::id();
  if (t0 < len) {
#pragma unroll
    for (int k = 0; k < K; ++k) a = a.then(M::unpack(vec[k]));
  }
  __syncwarp();
  a = warp_scan(a);
  *before = a.up(1);
  *dead = __ballot_sync(FULL, *bad < K);
  if (lane == 31) {
    sh.total[warp] = a.pack();
    sh.lost[warp] = *dead;
  }
  __syncthreads();
  if (warp == 0) {
    const bool in = lane < STATES_WARPS;
    const M t = warp_scan(in ? M::unpack(typename M::Packed(sh.total[lane])) : M::id());
    const uint32_t mask = __ballot_sync(FULL, in && sh.lost[lane] != 0);
    if (in) sh.total[lane] = t.pack();
    if (lane == 0) sh.lost_mask = mask;
  }
  __syncthreads();
}

template <class M, int K, class I>
__device__ void states_row(const StateArgs& p, uint32_t blocks, uint32_t each, StateShared& sh, uint32_t* staged) {
  using Packed = typename M::Packed;
  constexpr uint32_t TILE = STATES_THREADS * K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint64_t row = blockIdx.x / blocks;
  const uint32_t rank = blockIdx.x % blocks;
  const uint32_t begin = uint32_t(min(uint64_t(rank) * each, uint64_t(p.n_cols)));
  const uint32_t end = uint32_t(min(uint64_t(begin) + each, uint64_t(p.n_cols)));
  const uint32_t len = min(row_length(p, row), end);
  const I* tokens = static_cast<const I*>(p.tokens) + row * p.tstride;
  uint8_t* out = p.states + row * p.sstride;
  Packed vec[K];
  uint32_t bad = K, dead = 0, gone = 0, s = first_state(p, row);
  M before = M::id(), all = M::id();
  if (blocks > 1) ppl::cluster_arrive();
  if (rank == 0 && threadIdx.x == 0) out[0] = uint8_t(s);
  const bool kept = blocks > 1 && end - begin <= TILE;  // one tile, whose vectors stay
#pragma unroll 1
  for (int pass = blocks > 1 ? 0 : 1; pass < 2; ++pass) {
#pragma unroll 1
    for (uint32_t base = begin; base < end; base += TILE) {  // TILE is far below 2^16: no overflow
      const uint32_t t0 = base + threadIdx.x * K;
      if (pass == 0 || !kept) states_tile(p, tokens, t0, len, vec, &bad, &before, &dead, sh);
      const M whole = M::unpack(Packed(sh.total[STATES_WARPS - 1]));
      const uint32_t lost = sh.lost_mask;
      if (pass == 0) {
        all = all.then(whole);
        gone |= lost;
        if (base + TILE < end) __syncthreads();
        continue;
      }
      uint32_t q = s;
      if (q != PP_STATE_NONE) {
        if (warp > 0) q = nib_apply(sh.total[warp - 1], q);
        if (lane > 0) q = before.apply(q);
      }
      if ((lost & ((1u << warp) - 1)) || (dead & ((1u << lane) - 1))) q = PP_STATE_NONE;
      if (q != PP_STATE_NONE && bad == K) {
#pragma unroll
        for (int g = 0; g < K / 4; ++g) {
          uint32_t four = 0;
#pragma unroll
          for (int k = 4 * g; k < 4 * g + 4; ++k) {
            q = uint32_t(vec[k] >> (4 * q)) & 15;
            four |= q << (8 * (k - 4 * g));
          }
          staged[threadIdx.x * (K / 4) + g] = four;
        }
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (uint32_t(k) >= bad) q = PP_STATE_NONE;
          if (q != PP_STATE_NONE) q = uint32_t(vec[k] >> (4 * q)) & 15;
          reinterpret_cast<uint8_t*>(staged)[threadIdx.x * K + k] = uint8_t(q);
        }
      }
      if (s != PP_STATE_NONE) s = lost ? uint32_t(PP_STATE_NONE) : whole.apply(s);
      __syncthreads();
      // the tile's states, which begin at any byte, in words of memory
      uint8_t* to = out + uint64_t(base) + 1;
      const uint32_t n = min(TILE, end - base);
      const uint32_t skip = min(uint32_t(-reinterpret_cast<intptr_t>(to)) & 3u, n), words = (n - skip) / 4;
      for (uint32_t w = threadIdx.x; w < words; w += STATES_THREADS)
        reinterpret_cast<uint32_t*>(to + skip)[w] = __funnelshift_r(staged[w], staged[w + 1], 8 * skip);
      const uint32_t rest = n - skip - 4 * words;
      if (threadIdx.x < skip) to[threadIdx.x] = reinterpret_cast<uint8_t*>(staged)[threadIdx.x];
      if (threadIdx.x < rest) to[n - rest + threadIdx.x] = reinterpret_cast<uint8_t*>(staged)[n - rest + threadIdx.x];
      if (base + TILE < end) __syncthreads();
    }
    if (pass == 0) {
      ppl::cluster_wait();  // the later blocks have started
      if (warp == 0 && uint32_t(lane) > rank && uint32_t(lane) < blocks) {  // a lane per later block
        const uint64_t v = all.pack();
        uint32_t a, b;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(uint32_t(__cvta_generic_to_shared(&sh.part[rank]))), "r"(lane));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(uint32_t(__cvta_generic_to_shared(&sh.part_lost[rank]))), "r"(lane));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(b), "r"(gone) : "memory");
      }
      ppl::cluster_sync();
#pragma unroll 4
      for (uint32_t q = 0; q < rank; ++q) {
        const uint32_t next = uint32_t(sh.part[q] >> (4 * (s & 15))) & 15;
        s = s == PP_STATE_NONE || sh.part_lost[q] ? uint32_t(PP_STATE_NONE) : next;
      }
    }
  }
}

template <int S, int K>
__global__ void __launch_bounds__(STATES_THREADS, 2)
states_kernel(const __grid_constant__ StateArgs p, uint32_t blocks, uint32_t each) {
  __shared__ StateShared sh;
  __shared__ __align__(16) uint32_t staged[STATES_THREADS * K / 4 + 1];
  switch (p.type) {
    case PP_U8: return states_row<Map<S>, K, uint8_t>(p, blocks, each, sh, staged);
    case PP_I8: return states_row<Map<S>, K, int8_t>(p, blocks, each, sh, staged);
    case PP_I32: return states_row<Map<S>, K, int32_t>(p, blocks, each, sh, staged);
    default: return states_row<Map<S>, K, int64_t>(p, blocks, each, sh, staged);
  }
}
using StatesKernel = void (*)(StateArgs, uint32_t, uint32_t);
const StatesKernel STATES_KERNEL[4] = {states_kernel<8, 4>, states_kernel<8, 8>, states_kernel<16, 4>, states_kernel<16, 8>};

cudaLaunchConfig_t states_config(uint32_t blocks, uint32_t grid, cudaLaunchAttribute* at, cudaStream_t stream) {
  std::memset(at, 0, sizeof *at);
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = blocks;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(STATES_THREADS);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

cudaError_t launch_states(const StateArgs& p, cudaStream_t stream) {
  static ppi::DeviceOnce once;
  static uint32_t most[ppi::MAX_DEVICES];  // blocks of the largest cluster
  int dev;
  cudaError_t e = ppi::current_device(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [](int d) {
    cudaError_t e = cudaSuccess;
    for (int k = 0; k < 4 && e == cudaSuccess; ++k)
      e = cudaFuncSetAttribute(STATES_KERNEL[k], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = states_config(STATES_BLOCKS, STATES_BLOCKS, &at, nullptr);
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, STATES_KERNEL[3], &cfg);
    most[d] = n > 0 ? STATES_BLOCKS : 8;
    return e;
  });
  if (e != cudaSuccess) return e;
  // a cluster shares a row while there are fewer than two blocks for each of
  // 152 multiprocessors and a part keeps 1024 tokens
  uint32_t blocks = 1;
  while (blocks < most[dev] && uint64_t(p.n_rows) * blocks < 304 && p.n_cols / (2 * blocks) >= 1024) blocks *= 2;
  if (uint64_t(p.n_rows) * blocks >= (uint64_t(1) << 31)) blocks = 1;
  const uint32_t each = uint32_t((uint64_t(p.n_cols) + blocks - 1) / blocks);
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = states_config(blocks, p.n_rows * blocks, &at, stream);
  return cudaLaunchKernelEx(&cfg, STATES_KERNEL[(p.n_states > 8 ? 2 : 0) + (each > STATES_THREADS * 4 ? 1 : 0)], p, blocks, each);
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
  if (!ppl::aligned(d_offsets, 4) || !ppl::aligned(d_vectors, 8) || !ppl::aligned(d_allowed, 4)) return PP_EINVAL;
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
  if (dfa->n_states <= 8) vocab_kernel<8><<<unsigned(blocks), VOCAB_THREADS, 0, stream>>>(p, g);
  else vocab_kernel<16><<<unsigned(blocks), VOCAB_THREADS, 0, stream>>>(p, g);
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
  if (!ppl::aligned(d_vectors, 8) || !ppl::aligned(d_tokens, ppl::isize(token_type)) || !ppl::aligned(d_lengths, 4))
    return PP_EINVAL;
  const StateArgs p = {d_vectors, uint32_t(n_vocab), n_states, d_tokens, token_type,
                       uint32_t(n_rows), uint32_t(n_cols), tokens_stride, d_lengths, d_start,
                       start_stride, start_state, d_states, states_stride};
  if (n_cols <= STATES_SHORT || n_cols * STATES_MANY <= n_rows)
    states_short_kernel<<<unsigned((n_rows + 127) / 128), 128, 0, stream>>>(p);
  else
    return ppl::rc_of(launch_states(p, stream));
  return ppl::rc_of(cudaGetLastError());
}

}  // extern "C"
