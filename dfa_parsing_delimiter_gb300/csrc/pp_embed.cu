// Rows of a table by id (pp_embed) and the gradient for the table
// (pp_embed_grad).
//
// The gradient of a gather is a scatter-add; to sum in a fixed order and
// without atomics on values, the positions are sorted by id with a stable
// radix sort of (id, position), and the sorted list is cut into chunks of
// equal length.  A warp walks a chunk for 256 columns, adds the rows of each
// run of equal ids in registers and writes the sum once.  A run that ends by
// the end of the next chunk is finished by the chunk it begins in; a longer
// one leaves a partial sum per chunk, added up in order by a last kernel.
// Up to SMALL_IDS positions one kernel does it all (small_kernel).  Up to
// SORT_CAP positions one thread-block cluster sorts in distributed
// shared memory, while the first blocks of the next kernel write the zeros
// of the rows that no id names; more go through global memory in passes.
#include <algorithm>
#include <cstring>

#include "pp_device.cuh"
#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using namespace ppd;
using ppl::cluster_arrive;
using ppl::cluster_sync;
using ppl::cluster_wait;
using ppl::from_f;
using ppl::load_id;
using ppl::Pack;
using ppl::to_f;

constexpr int UNIT = 8;  // columns a thread moves at once

template <class F>
cudaError_t with_type(int t, F&& f) {
  switch (t) {
    case PP_F32: return f(float{});
    case PP_F16: return f(__half{});
    default: return f(__nv_bfloat16{});
  }
}

// ------------------------------------------------------------------ lookup
struct EmbedArgs {
  const void* ids;
  int32_t type;
  uint64_t id_stride;
  uint32_t n;
  const void* table;
  uint32_t n_vocab, dim;
  uint64_t tstride;
  float scale;
  int64_t pad;
  void* out;
  uint64_t ostride;
};

// blockDim.x threads move a row, blockDim.y rows a block; U columns a thread
// and step (8 where rows are aligned to 16 bytes in both arrays), AHEAD
// steps' loads on their way before the first store: the compiler cannot know
// that the arrays do not overlap.
//
// 65536 rows of 4096 f32 to bf16: 953 MB in 149 us, 94 % of the copy rate;
// rows that several ids name are partly read again (463 MB for 292).
constexpr int EMBED_THREADS = 256, AHEAD = 4;
template <class T, class O, int U>
__global__ void __launch_bounds__(EMBED_THREADS) embed_kernel(const __grid_constant__ EmbedArgs p) {
  const uint64_t i = uint64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (i >= p.n) return;
  const int64_t id = load_id(p.ids, p.type, i * p.id_stride);
  const bool there = id >= 0 && id < p.n_vocab && id != p.pad;
  const T* row = static_cast<const T*>(p.table) + (there ? uint64_t(id) * p.tstride : 0);
  O* out = static_cast<O*>(p.out) + i * p.ostride;
  const uint64_t step = uint64_t(blockDim.x) * U;
  for (uint64_t c = uint64_t(threadIdx.x) * U; c < p.dim; c += step * AHEAD) {
    Pack<T, U> x[AHEAD];
#pragma unroll
    for (int g = 0; g < AHEAD; ++g)
      if (there && c + g * step + U <= p.dim) x[g] = *reinterpret_cast<const Pack<T, U>*>(row + c + g * step);
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) {
      const uint64_t at = c + g * step;
      if (at + U <= p.dim) {
        Pack<O, U> y;
#pragma unroll
        for (int k = 0; k < U; ++k) y.v[k] = from_f<O>(there ? to_f(x[g].v[k]) * p.scale : 0.f);
        *reinterpret_cast<Pack<O, U>*>(out + at) = y;
      } else if (U > 1) {
        for (uint64_t k = at; k < p.dim; ++k) out[k] = from_f<O>(there ? to_f(row[k]) * p.scale : 0.f);
      }
    }
  }
}

// Whether every row of an array begins on a 16-byte boundary.
bool rows_aligned(const void* p, size_t size, uint64_t stride, uint64_t rows) {
  return ppl::aligned(p, 16) && (rows <= 1 || stride * size % 16 == 0);
}

template <class T, class O>
cudaError_t launch_embed(const EmbedArgs& p, cudaStream_t stream) {
  const bool wide = rows_aligned(p.table, sizeof(T), p.tstride, p.n_vocab) &&
                    rows_aligned(p.out, sizeof(O), p.ostride, p.n);
  const uint32_t steps = wide ? (p.dim + UNIT - 1) / UNIT : p.dim;
  // threads a row: enough for one step each, but with a large n only a
  // quarter, whose AHEAD steps are loaded at once (65536 rows of 4096: 152
  // us against 156)
  const uint32_t want = p.n >= 2048 ? (steps + AHEAD - 1) / AHEAD : steps;
  uint32_t x = 1;
  while (x < EMBED_THREADS && x < want) x *= 2;
  const dim3 block(x, EMBED_THREADS / x);
  const unsigned grid = unsigned((uint64_t(p.n) + block.y - 1) / block.y);
  if (wide) embed_kernel<T, O, UNIT><<<grid, block, 0, stream>>>(p);
  else embed_kernel<T, O, 1><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------- sort by id
// Least significant digit first; each pass counts the digits of every tile,
// scans each digit's counts over the tiles and moves the pairs, whose block
// adds up the digits before.  Keys: the id, or n_vocab for a position that
// takes no part (sorted last).
constexpr int SORT_THREADS = 512, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ITEMS = 8;  // pairs a thread
constexpr uint32_t SORT_TILE = SORT_THREADS * SORT_ITEMS;
constexpr int DIGIT_BITS = 9, DIGITS = 1 << DIGIT_BITS;
static_assert(DIGITS == SORT_THREADS, "a thread per digit");

struct SortArgs {
  const void* ids;  // first pass: the ids; else null
  int32_t type;
  uint64_t id_stride;
  uint32_t n, n_vocab;
  int64_t pad;
  const uint32_t *key_in, *pos_in;
  uint32_t *key_out, *pos_out;
  uint32_t* counts;  // [1 << bits][n_tiles], then [1 << bits] totals
  uint32_t n_tiles;
  int shift, bits;
};

__device__ __forceinline__ uint32_t key_of(const SortArgs& p, int64_t id) {
  return id >= 0 && id < p.n_vocab && id != p.pad ? uint32_t(id) : p.n_vocab;
}
__device__ __forceinline__ uint32_t sort_key(const SortArgs& p, uint64_t i) {
  return p.ids ? key_of(p, load_id(p.ids, p.type, i * p.id_stride)) : p.key_in[i];
}

// This thread's keys of a tile: warp w has SORT_ITEMS x 32 consecutive ones.
__device__ __forceinline__ void tile_keys(const SortArgs& p, uint64_t first, uint32_t (&key)[SORT_ITEMS]) {
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) key[k] = first + k * 32 < p.n ? sort_key(p, first + k * 32) : 0;
}

// Exclusive scan of a value a thread over the block's SORT_THREADS threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  uint32_t inc = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t up = __shfl_up_sync(FULL, inc, d);
    if (lane >= d) inc += up;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  uint32_t before = inc - x;
  for (int w = 0; w < warp; ++w) before += sums[w];
  return before;
}

__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(const __grid_constant__ SortArgs p) {
  __shared__ uint32_t count[DIGITS];
  count[threadIdx.x] = 0;
  const uint64_t first = uint64_t(blockIdx.x) * SORT_TILE + threadIdx.x / 32 * (SORT_ITEMS * 32) + (threadIdx.x & 31);
  uint32_t key[SORT_ITEMS];
  tile_keys(p, first, key);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k)
    if (first + k * 32 < p.n) atomicAdd(&count[key[k] >> p.shift & ((1u << p.bits) - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < 1u << p.bits) p.counts[uint64_t(threadIdx.x) * p.n_tiles + blockIdx.x] = count[threadIdx.x];
}

// A block per digit: its counts become the pairs with it in earlier tiles.
__global__ void __launch_bounds__(SORT_THREADS) sort_scan_kernel(const __grid_constant__ SortArgs p) {
  __shared__ uint32_t sums[SORT_WARPS];
  __shared__ uint32_t last;
  uint32_t* counts = p.counts + uint64_t(blockIdx.x) * p.n_tiles;
  uint32_t run = 0;
  for (uint32_t base = 0; base < p.n_tiles; base += SORT_THREADS) {
    const uint32_t t = base + threadIdx.x, x = t < p.n_tiles ? counts[t] : 0;
    const uint32_t before = block_scan(x, sums);
    if (t < p.n_tiles) counts[t] = run + before;
    if (threadIdx.x == SORT_THREADS - 1) last = before + x;
    __syncthreads();
    run += last;
    __syncthreads();
  }
  if (threadIdx.x == 0) p.counts[(uint64_t(1) << p.bits) * p.n_tiles + blockIdx.x] = run;
}

// Stable move: equal digits of a warp are ranked by ballots, in order.
__global__ void __launch_bounds__(SORT_THREADS) sort_move_kernel(const __grid_constant__ SortArgs p) {
  __shared__ uint32_t place[SORT_WARPS][DIGITS];
  __shared__ uint32_t sums[SORT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint32_t n_bins = 1u << p.bits;
  for (int w = 0; w < SORT_WARPS; ++w) place[w][threadIdx.x] = 0;
  const uint64_t first = uint64_t(blockIdx.x) * SORT_TILE + warp * (SORT_ITEMS * 32) + lane;
  uint32_t key[SORT_ITEMS], rank[SORT_ITEMS];
  tile_keys(p, first, key);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const bool there = first + k * 32 < p.n;
    const uint32_t d = key[k] >> p.shift & (n_bins - 1);
    uint32_t same = __ballot_sync(FULL, there);
    for (int b = 0; b < p.bits; ++b) {
      const uint32_t set = __ballot_sync(FULL, d >> b & 1);
      same &= d >> b & 1 ? set : ~set;
    }
    const uint32_t before = place[warp][d], below = __popc(same & ((1u << lane) - 1));
    rank[k] = before + below;
    __syncwarp();
    if (there && below == 0) place[warp][d] = before + __popc(same);
    __syncwarp();
  }
  const uint32_t total = threadIdx.x < n_bins ? p.counts[uint64_t(n_bins) * p.n_tiles + threadIdx.x] : 0;
  uint32_t run = block_scan(total, sums);  // and all ranks are in
  if (threadIdx.x < n_bins) {
    run += p.counts[uint64_t(threadIdx.x) * p.n_tiles + blockIdx.x];
    for (int w = 0; w < SORT_WARPS; ++w) {
      const uint32_t c = place[w][threadIdx.x];
      place[w][threadIdx.x] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k)
    if (first + k * 32 < p.n) {
      const uint32_t to = place[warp][key[k] >> p.shift & (n_bins - 1)] + rank[k];
      p.key_out[to] = key[k];
      p.pos_out[to] = p.ids ? uint32_t(first + k * 32) : p.pos_in[first + k * 32];
    }
}

// ------------------------------------------------------------ zero rows
// The kernels of one pp_embed_grad follow each other by programmatic
// dependent launch: each lets the next one's blocks start early, and a block
// that needs what the kernel before wrote waits for that one's end first.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct ZeroArgs {
  void* out;
  uint64_t row_bytes, stride_bytes;  // of a row of the gradient
  uint32_t n_vocab;
  int32_t wide;       // rows in whole 16-byte pieces
  int32_t elem_size;  // otherwise: 2 or 4
};

// Rows base + i, i < span, whose bit is clear become zeros; every thread of
// the block takes part.
template <int THREADS>
__device__ void zero_rows(const ZeroArgs& z, const uint32_t* bits, uint64_t base, uint32_t span) {
  const uint32_t units = uint32_t(z.wide ? z.row_bytes / 16 : z.row_bytes / z.elem_size);
  uint32_t per = 1;  // threads a row
  while (per < THREADS && per < units) per *= 2;
  const uint32_t me = threadIdx.x % per;
  for (uint32_t i = threadIdx.x / per; i < span; i += THREADS / per) {
    if (bits[i / 32] >> (i % 32) & 1) continue;
    char* row = static_cast<char*>(z.out) + (base + i) * z.stride_bytes;
    if (z.wide)
      for (uint32_t u = me; u < units; u += per) reinterpret_cast<uint4*>(row)[u] = make_uint4(0, 0, 0, 0);
    else if (z.elem_size == 4)
      for (uint32_t u = me; u < units; u += per) reinterpret_cast<uint32_t*>(row)[u] = 0;
    else
      for (uint32_t u = me; u < units; u += per) reinterpret_cast<uint16_t*>(row)[u] = 0;
  }
}

// From a sorted list: a thread looks for each of ZERO_SPAN rows.
constexpr int ZERO_SPAN = 256;
__global__ void __launch_bounds__(256)
zero_kernel(const __grid_constant__ ZeroArgs z, const uint32_t* key, uint32_t n) {
  __shared__ uint32_t bits[ZERO_SPAN / 32];
  const uint64_t base = uint64_t(blockIdx.x) * ZERO_SPAN, v = base + threadIdx.x;
  uint32_t lo = 0, hi = n;  // the first index whose key is v or more
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (key[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  const uint32_t word = __ballot_sync(FULL, lo < n && key[lo] == v);
  if ((threadIdx.x & 31) == 0) bits[threadIdx.x / 32] = word;
  __syncthreads();
  zero_rows<256>(z, bits, base, uint32_t(min(uint64_t(ZERO_SPAN), z.n_vocab - base)));
}

// From the ids themselves: block `me` of `all` looks at its share of the rows
// against every id, `SPAN` rows at a time (bits: that many).
constexpr uint32_t SPAN = 1u << 18;
template <int THREADS>
__device__ __noinline__ void zero_scan(const ZeroArgs& z, const SortArgs& s, uint32_t me, uint32_t all, uint32_t* bits) {
  const uint64_t each = (z.n_vocab + all - 1) / all;
  const uint64_t v0 = me * each, v1 = min(v0 + each, uint64_t(z.n_vocab));
  // from a place of its own on, as blocks that read the same ids at the same
  // time wait for the same lines
  const uint32_t turn = uint32_t(uint64_t(s.n) * me / all);
  for (uint64_t base = v0; base < v1; base += SPAN) {
    const uint32_t span = uint32_t(min(uint64_t(SPAN), v1 - base));
    for (uint32_t w = threadIdx.x; w * 32 < span; w += THREADS) bits[w] = 0;
    __syncthreads();
    auto mark = [&](uint32_t, auto id) {
      // an id below 0 turns into one far past the span
      const uint64_t j = sizeof(id) == 8 ? uint64_t(id) - base : uint32_t(id) - uint32_t(base);
      if (j < span) atomicOr(&bits[j / 32], 1u << (j % 32));
    };
    ppl::for_ids<8>(s.ids, s.type, s.id_stride, turn + threadIdx.x, s.n, THREADS, mark);
    ppl::for_ids<8>(s.ids, s.type, s.id_stride, threadIdx.x, turn, THREADS, mark);
    __syncthreads();
    const uint64_t pad = uint64_t(s.pad) - base;  // has no gradient, so its row is zeros
    if (pad < span && threadIdx.x == 0) bits[pad / 32] &= ~(1u << (pad % 32));
    __syncthreads();
    zero_rows<THREADS>(z, bits, base, span);
    __syncthreads();
  }
}

// ------------------------------------------------- sort in one cluster
// Block r of the cluster holds pairs r PER .. (r + 1) PER - 1 of the list,
// PER = 1024 ITEMS.  Per pass a block ranks its pairs' digits (per warp by
// ballots, in order), tells every block its digit totals, and after a
// cluster barrier each pair goes straight to its place in the shared memory
// of the block that owns it (the last pass: to global memory).  Bound by the
// latency of its steps: 131072 pairs in two passes of 9 bits take 29 us, 8192
// take 9, hidden behind the zeros but when the result is accumulated.  The
// passes through global memory take three kernels each, 42 us for 140000 pairs.
constexpr int CS_THREADS = 1024, CS_WARPS = 32, CS_BITS = 9, CS_BINS = 1 << CS_BITS;
constexpr int CS_BLOCKS = 16, CS_ITEMS = 8;
constexpr uint32_t SORT_CAP = CS_THREADS * CS_ITEMS * CS_BLOCKS;

struct ClusterArgs {
  SortArgs s;  // key_out, pos_out: the sorted list
  int32_t blocks, bits, passes;
  uint32_t* n_long;  // [2], set to 0 for the sums
};

__device__ __forceinline__ uint32_t smem_of(const void* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

template <int ITEMS>
__global__ void __launch_bounds__(CS_THREADS, 1) cluster_sort_kernel(const __grid_constant__ ClusterArgs p) {
  constexpr uint32_t PER = CS_THREADS * ITEMS;
  extern __shared__ uint2 item[];  // [PER], then the arrays below
  uint32_t* totals = reinterpret_cast<uint32_t*>(item + PER);                  // [CS_BLOCKS][CS_BINS]
  uint16_t* place = reinterpret_cast<uint16_t*>(totals + CS_BLOCKS * CS_BINS);  // [CS_WARPS][CS_BINS]
  __shared__ uint32_t start[CS_BINS];
  __shared__ uint32_t sums[CS_BINS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  cluster_arrive();
  let_next_start();
  const uint32_t rank = blockIdx.x, n_bins = 1u << p.bits;
  if (rank == 0 && threadIdx.x == 0) p.n_long[0] = p.n_long[1] = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    for (uint32_t k = threadIdx.x; k < CS_WARPS * CS_BINS / 2; k += CS_THREADS)
      reinterpret_cast<uint32_t*>(place)[k] = 0;
    uint2 it[ITEMS];
    uint16_t nth[ITEMS];
    const uint32_t i0 = warp * (32 * ITEMS) + lane;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)  // past the list's end: after everything else
      it[k] = pass ? item[i0 + k * 32] : make_uint2(p.s.n_vocab, rank * PER + i0 + k * 32);
    if (!pass) {
      auto read = [&](auto* ids) {
        int64_t id[ITEMS];
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) id[k] = it[k].y < p.s.n ? int64_t(ids[it[k].y * p.s.id_stride]) : -1;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) it[k].x = key_of(p.s, id[k]);
      };
      switch (p.s.type) {
        case PP_U8: read(static_cast<const uint8_t*>(p.s.ids)); break;
        case PP_I8: read(static_cast<const int8_t*>(p.s.ids)); break;
        case PP_I32: read(static_cast<const int32_t*>(p.s.ids)); break;
        default: read(static_cast<const int64_t*>(p.s.ids)); break;
      }
    }
    __syncthreads();
    uint16_t* mine = place + warp * CS_BINS;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t d = it[k].x >> shift & (n_bins - 1);
      uint32_t same = FULL;
      for (int b = 0; b < p.bits; ++b) {
        const uint32_t set = __ballot_sync(FULL, d >> b & 1);
        same &= d >> b & 1 ? set : ~set;
      }
      const uint32_t before = mine[d], below = __popc(same & ((1u << lane) - 1));
      nth[k] = uint16_t(before + below);
      __syncwarp();
      if (below == 0) mine[d] = uint16_t(before + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    if (!pass) cluster_wait();  // all blocks have started
    if (threadIdx.x < n_bins) {  // the warps' counts to places within the block
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < CS_WARPS; ++w) {
        const uint32_t c = place[w * CS_BINS + threadIdx.x];
        place[w * CS_BINS + threadIdx.x] = uint16_t(run);
        run += c;
      }
      for (int q = 0; q < p.blocks; ++q)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(smem_of(&totals[rank * CS_BINS + threadIdx.x], q)), "r"(run) : "memory");
    }
    cluster_sync();
    uint32_t all = 0, before = 0, inc = 0;
    if (threadIdx.x < CS_BINS) {
      if (threadIdx.x < n_bins)
        for (int q = 0; q < p.blocks; ++q) {
          const uint32_t c = totals[q * CS_BINS + threadIdx.x];
          if (q < int(rank)) before += c;
          all += c;
        }
      inc = all;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t up = __shfl_up_sync(FULL, inc, d);
        if (lane >= d) inc += up;
      }
      if (lane == 31) sums[warp] = inc;
    }
    __syncthreads();
    if (threadIdx.x < CS_BINS) {
      for (int w = 0; w < warp; ++w) before += sums[w];
      start[threadIdx.x] = before + inc - all;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const uint32_t d = it[k].x >> shift & (n_bins - 1);
      const uint32_t to = start[d] + mine[d] + nth[k];
      if (pass + 1 < p.passes) {
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(smem_of(&item[to % PER], to / PER)), "r"(it[k].x), "r"(it[k].y) : "memory");
      } else if (to < p.s.n) {
        p.s.key_out[to] = it[k].x;
        p.s.pos_out[to] = it[k].y;
      }
    }
    if (pass + 1 < p.passes) cluster_sync();
  }
}

constexpr size_t cluster_smem(int items) {
  return size_t(CS_THREADS) * items * 8 + CS_BLOCKS * CS_BINS * 4 + CS_WARPS * CS_BINS * 2;
}

// ------------------------------------------------------------ sums of runs
struct SumArgs {
  const uint32_t *key, *pos;  // sorted by (key, position)
  uint32_t n, n_vocab;
  const void* grad;
  uint64_t gstride;
  uint32_t dim, slices;  // columns, and groups of SUM_COLS of them
  float scale;
  int32_t accumulate;
  void* out;
  uint64_t ostride;
  float* part;  // [n_chunks][2][width]: sums of a chunk's first and last run
  uint64_t width;
  uint32_t n_chunks, chunk;
  uint32_t* n_long;  // [2]: long runs, and those that blocks share
  uint2* longs;  // the chunk that each begins in, and its id; the shared ones from the end on
  uint32_t n_zero;           // blocks that write zeros, before those that sum
  ZeroArgs z;
  SortArgs s;
};

constexpr int SUM_WARPS = 16, JOIN_WARPS = 8;
constexpr int SUM_COLS = 32 * UNIT;  // columns a warp
constexpr uint32_t NO_KEY = 0xFFFFFFFFu;

// A lane's columns of the 32 N from c0 on: N consecutive ones (WIDE: aligned
// rows) or every 32nd one (any rows), n of which exist.
template <bool WIDE, int N = UNIT>
struct Cols {
  static constexpr int STEP = WIDE ? 1 : 32;
  uint32_t first;
  int n;
  __device__ __forceinline__ Cols(uint32_t c0, uint32_t dim) {
    const uint32_t lane = threadIdx.x & 31;
    first = c0 + lane * (WIDE ? N : 1);
    const int left = int(dim) - int(first);
    n = left <= 0 ? 0 : min((left + STEP - 1) / STEP, N);
  }
};

// Loads and stores of a lane's columns; row: at its first one.
template <class T, bool WIDE, int N>
__device__ __forceinline__ void load_row(const T* row, int n, Pack<T, N>& x) {
  if (WIDE && n == N) {
    x = *reinterpret_cast<const Pack<T, N>*>(row);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) x.v[k] = k < n ? row[k * Cols<WIDE>::STEP] : from_f<T>(0.f);
  }
}

template <class O, bool WIDE, int N>
__device__ __forceinline__ void store_row(O* row, int n, const float (&x)[N]) {
  if (WIDE && n == N) {
    Pack<O, N> v;
#pragma unroll
    for (int k = 0; k < N; ++k) v.v[k] = from_f<O>(x[k]);
    *reinterpret_cast<Pack<O, N>*>(row) = v;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < n) row[k * Cols<WIDE>::STEP] = from_f<O>(x[k]);
  }
}

template <class O, bool WIDE, int N>
__device__ __forceinline__ void write_sum(const SumArgs& p, uint32_t id, const Cols<WIDE, N>& at, float (&a)[N]) {
  O* row = static_cast<O*>(p.out) + (uint64_t(id) * p.ostride + at.first);
#pragma unroll
  for (int k = 0; k < N; ++k) a[k] *= p.scale;
  if (p.accumulate) {
    Pack<O, N> old;
    load_row<O, WIDE>(row, at.n, old);
#pragma unroll
    for (int k = 0; k < N; ++k) a[k] += to_f(old.v[k]);
  }
  store_row<O, WIDE>(row, at.n, a);
}

// 16, 8 or 4 bytes from global to shared memory, asynchronously.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(a), "l"(from), "n"(BYTES) : "memory");
}

// Rows on their way to a warp: a ring of DEPTH rows of 32 N columns in shared
// memory, BYTES in all.  A lane copies its own columns and reads them back
// itself, so nothing synchronises.  The lanes' pieces of up to 16 bytes
// (WIDE) or their elements lie side by side.
template <class T, bool WIDE, int BYTES, int N = UNIT>
struct Ring {
  static constexpr int PIECE = !WIDE ? int(sizeof(T)) : N * sizeof(T) < 16 ? int(N * sizeof(T)) : 16;
  static constexpr int EACH = PIECE / int(sizeof(T));  // elements a piece
  static constexpr uint32_t ROW = 32 * N * sizeof(T), DEPTH = BYTES / ROW, END = DEPTH * ROW;
  char* mine;
  uint32_t in = 0, out = 0;  // where the next row is copied to, and read from
  __device__ __forceinline__ explicit Ring(char* warp) : mine(warp + (threadIdx.x & 31) * PIECE) {}
  static __device__ __forceinline__ constexpr int place(int k) { return k / EACH * 32 * PIECE + k % EACH * int(sizeof(T)); }
  // one group of copies a call; row null: none
  __device__ __forceinline__ void copy(const T* row, int n) {
    if (row) {
      if (WIDE && n == N) {
#pragma unroll
        for (int k = 0; k < N; k += EACH) copy_async<PIECE < 4 ? 4 : PIECE>(mine + in + place(k), row + k);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          T* to = reinterpret_cast<T*>(mine + in + place(k));
          if (k >= n) *to = from_f<T>(0.f);
          else if (sizeof(T) == 4) copy_async<4>(to, row + k * Cols<WIDE, N>::STEP);
          else *to = row[k * Cols<WIDE, N>::STEP];
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    in = in + ROW == END ? 0 : in + ROW;
  }
  // the oldest row, with DEPTH - 1 groups after it, is added to a
  __device__ __forceinline__ void add(float (&a)[N]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
#pragma unroll
    for (int g = 0; g < N; g += EACH) {
      const Pack<T, EACH> x = *reinterpret_cast<const Pack<T, EACH>*>(mine + out + place(g));
#pragma unroll
      for (int k = 0; k < EACH; ++k) a[g + k] += to_f(x.v[k]);
    }
    out = out + ROW == END ? 0 : out + ROW;
  }
};

// Long runs that reach this many chunks after their first are listed apart.
// 128 measured the same on Zipf ids (271 us a call against 272); 64 is the least
// that gives each warp of a group a piece.
constexpr uint32_t JOIN_SHARE = 64;
// Where piece q of the run that begins in chunk c lies, for column 0.
__device__ __forceinline__ float* piece_of(const SumArgs& p, uint64_t c, uint32_t q) {
  return p.part + (q ? 2 * (c + q) : 2 * c + 1) * p.width;
}
// How many blocks have left their sums of that run for the columns from c0
// on: in the next chunk's second row, which is free since the run fills the
// chunk.  Set to 0 where the run is listed.
__device__ __forceinline__ uint32_t* joined(const SumArgs& p, uint64_t c, uint32_t c0) {
  return reinterpret_cast<uint32_t*>(p.part + (2 * (c + 1) + 1) * p.width + c0);
}

// Of the sorted list, chunk c holds [c L, (c + 1) L), L <= 32.  A run is long
// if it begins in chunk c and goes on past the end of chunk c + 1.  A warp
// per chunk and SUM_COLS columns; the chunk's keys and the next one's are in
// its lanes, and RING_BYTES of rows are on their way.
// The first n_zero blocks write the rows that no id names.  They need the
// ids alone and so run beside the sort; the sums follow on the slots that
// they leave, and the memory is never idle.
//
// 131072 rows of 2048 bf16 for 131072 Zipf ids: 1.59 GB in 253 us, 92 % of
// the copy rate (zeros 794 MB, rows read 537 MB, sums 280 MB); bound by
// memory.  A run's sum is written in one place of a loop that is not
// unrolled: with 8 rows in registers and as many places the code does not
// fit the instruction cache, and the sums alone take 347 us instead of 120.
constexpr int RING_BYTES = 3072;  // a warp; 4096 measures the same, 2048 up to 6 % slower on f32
template <class T, class O, bool WIDE>
__global__ void __launch_bounds__(SUM_WARPS * 32, 2) sum_kernel(const __grid_constant__ SumArgs p) {
  using R = Ring<T, WIDE, RING_BYTES>;  // 6 rows, of 32-bit values 3
  __shared__ __align__(16) char ring_mem[SUM_WARPS][RING_BYTES];
  const int lane = threadIdx.x & 31;
  let_next_start();
  if (blockIdx.x < p.n_zero) {
    static_assert(sizeof ring_mem >= SPAN / 8, "the ring's memory holds the rows' bits");
    zero_scan<SUM_WARPS * 32>(p.z, p.s, blockIdx.x, p.n_zero, reinterpret_cast<uint32_t*>(&ring_mem[0][0]));
    wait_for_previous();  // so that the end of this kernel is the end of both
    return;
  }
  const uint64_t me = uint64_t(blockIdx.x - p.n_zero) * SUM_WARPS + threadIdx.x / 32;
  const uint64_t c = me / p.slices;
  const uint32_t c0 = uint32_t(me % p.slices) * SUM_COLS;
  const Cols<WIDE> at(c0, p.dim);
  wait_for_previous();
  if (c >= p.n_chunks) return;
  const uint32_t L = p.chunk, n = p.n;
  const uint32_t lo = uint32_t(c) * L, size = min(L, n - lo);
  const bool in0 = uint32_t(lane) < size, in1 = uint32_t(lane) < L && uint64_t(lo) + L + lane < n;
  const uint32_t key0 = in0 ? p.key[lo + lane] : NO_KEY, key1 = in1 ? p.key[lo + L + lane] : NO_KEY;
  const uint32_t pos0 = in0 ? p.pos[lo + lane] : 0, pos1 = in1 ? p.pos[lo + L + lane] : 0;
  const uint32_t prev = lo ? p.key[lo - 1] : NO_KEY, prev2 = lo > L ? p.key[lo - L - 1] : NO_KEY;
  const uint32_t far = uint64_t(lo) + 2 * L < n ? p.key[lo + 2 * L] : NO_KEY;
  const uint64_t share = lo + uint64_t(JOIN_SHARE) * L;
  const uint32_t beyond = c0 == 0 && share < n ? p.key[share] : NO_KEY;
  const uint32_t first = __shfl_sync(FULL, key0, 0), last = __shfl_sync(FULL, key0, size - 1);
  const uint32_t next = __shfl_sync(FULL, key1, 0);
  const bool goes_on = prev == first;                                  // the first run began earlier
  const bool head = goes_on && (prev2 == first || next == first);      // and is long
  uint32_t i = goes_on && !head ? __popc(__ballot_sync(FULL, in0 && key0 == first)) : 0;
  uint32_t end = __popc(__ballot_sync(FULL, key0 < p.n_vocab));
  const bool crosses = size == L && next == last && last < p.n_vocab && !(goes_on && first == last);
  const bool tail = crosses && far == last;  // the last run is long and begins here
  if (crosses && !tail) end += __popc(__ballot_sync(FULL, key1 == last));
  if (tail && lane == 0) {
    *joined(p, c, c0) = 0;
    const bool shared = beyond == last;
    if (c0 == 0) {
      const uint32_t at = atomicAdd(p.n_long + shared, 1u);
      p.longs[shared ? p.n_chunks - 1 - at : at] = make_uint2(uint32_t(c), last);
    }
  }
  if (i >= end) return;
  const T* grad = static_cast<const T*>(p.grad) + at.first;
  float* part = p.part + 2 * c * p.width + at.first;
  float a[UNIT] = {};
  bool piece = head;  // the current run is the long one that began earlier
  uint32_t id = __shfl_sync(FULL, key0, i);
  R ring(ring_mem[threadIdx.x / 32]);
  auto copy = [&](uint32_t e) {
    const T* row = nullptr;
    if (e < end) row = grad + uint64_t(__shfl_sync(FULL, e < L ? pos0 : pos1, e < L ? e : e - L)) * p.gstride;
    ring.copy(row, at.n);
  };
  for (uint32_t k = 0; k + 1 < R::DEPTH; ++k) copy(i + k);
#pragma unroll 1
  for (; i < end; ++i) {
    copy(i + R::DEPTH - 1);
    const uint32_t now = __shfl_sync(FULL, i < L ? key0 : key1, i < L ? i : i - L);
    if (now != id) {
      if (piece) store_row<float, WIDE>(part, at.n, a);
      else write_sum<O, WIDE>(p, id, at, a);
      piece = false;
      id = now;
#pragma unroll
      for (int j = 0; j < UNIT; ++j) a[j] = 0.f;
    }
    ring.add(a);
  }
  if (piece || tail) store_row<float, WIDE>(part + (piece ? 0 : p.width), at.n, a);
  else write_sum<O, WIDE>(p, id, at, a);
}

// Adds the pieces of each long run for SUM_COLS columns: a block per run, its
// warps one piece after another by turns.  Runs of more than JOIN_SHARE pieces
// (a padding id that nothing masks, the first of a Zipf law) are cut among the
// JOIN_GROUP blocks of a group; each leaves its sum in the place of its first
// piece, and the last one to do so adds the sums, in order.  Bound by latency,
// and for long runs by what a block with so few loads in flight reads (50 GB/s;
// a multiprocessor reads 137 with 1024 threads of eight 16-byte loads).  An id
// that half of 131072 positions of 2048 columns name: 190 us a call, 222 with
// one block a run.  Two loads in flight a lane: more cost registers, and so blocks (131072
// Zipf ids of 2048 columns: 268 us a call with 2, 272 with 4, 274 with 6).
constexpr int JOIN_BLOCKS = 256, JOIN_GROUP = 8, JOIN_LOADS = 2;

template <class O, bool WIDE>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 4) join_kernel(const __grid_constant__ SumArgs p) {
  static_assert(JOIN_GROUP == JOIN_WARPS, "a warp adds a block's sum in the end");
  static_assert(JOIN_SHARE + 1 >= JOIN_GROUP * JOIN_WARPS, "a piece for each warp of a group");
  __shared__ float part[JOIN_WARPS][SUM_COLS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint32_t rank = blockIdx.x % JOIN_GROUP, groups = gridDim.x / JOIN_GROUP;
  const uint64_t L = p.chunk;
  const Cols<WIDE> cols(blockIdx.y * SUM_COLS, p.dim);
  wait_for_previous();
  const uint2 n_long = *reinterpret_cast<const uint2*>(p.n_long);
  uint32_t r = blockIdx.x, h = groups - 1 - blockIdx.x / JOIN_GROUP;
  const uint2 own = r < p.n_chunks ? p.longs[r] : make_uint2(0, 0);  // beside n_long, whether there is one or not
#pragma unroll 1
  for (;;) {
    // first the shared runs, by the groups whose blocks have the fewest others
    const bool shared = h < n_long.y;
    if (!shared && r >= n_long.x) break;
    uint2 run = own;
    if (shared) run = p.longs[p.n_chunks - 1 - h];
    else if (r != blockIdx.x) run = p.longs[r];
    const uint64_t c = run.x;
    const uint32_t id = run.y, step = shared ? JOIN_GROUP * JOIN_WARPS : JOIN_WARPS;
    uint32_t q = shared ? rank * JOIN_WARPS + warp : warp;
    // the first piece comes beside the keys, whether the run has it or not
    Pack<float, UNIT> x0;
    if (c + q < p.n_chunks) load_row<float, WIDE>(piece_of(p, c, q) + cols.first, cols.n, x0);
    uint32_t n;  // pieces in the chunks after the one that the run begins in
    if (shared) {
      h += groups;
      n = JOIN_SHARE;
      uint32_t most = uint32_t(p.n_chunks - 1 - c);
      while (n < most) {  // each probe leaves a 257th
        const uint32_t far = (most - n + blockDim.x - 1) / blockDim.x, at = n + (threadIdx.x + 1) * far;
        const uint32_t m = __syncthreads_count(at <= most && p.key[(c + at) * L] == id);
        n += m * far;
        most = min(most, n + far - 1);
      }
    } else {
      r += gridDim.x;
      const uint64_t at = (c + 1 + threadIdx.x) * L;
      n = __syncthreads_count(threadIdx.x < JOIN_SHARE && at < p.n && p.key[at] == id);
    }
    float a[UNIT];
#pragma unroll
    for (int k = 0; k < UNIT; ++k) a[k] = q <= n ? x0.v[k] : 0.f;
    for (q += step; q <= n; q += JOIN_LOADS * step) {
      Pack<float, UNIT> x[JOIN_LOADS];
#pragma unroll
      for (int j = 0; j < JOIN_LOADS; ++j)
        if (q + j * step <= n) load_row<float, WIDE>(piece_of(p, c, q + j * step) + cols.first, cols.n, x[j]);
#pragma unroll
      for (int j = 0; j < JOIN_LOADS; ++j)
        if (q + j * step <= n) {
#pragma unroll
          for (int k = 0; k < UNIT; ++k) a[k] += x[j].v[k];
        }
    }
    bool end = !shared;
#pragma unroll 1
    for (;;) {
#pragma unroll
      for (int k = 0; k < UNIT; ++k) part[warp][k * 32 + lane] = a[k];
      __syncthreads();
      bool go_on = false;
      if (warp == 0) {
#pragma unroll
        for (int k = 0; k < UNIT; ++k)
          for (int w = 1; w < JOIN_WARPS; ++w) a[k] += part[w][k * 32 + lane];
        if (end) {
          write_sum<O, WIDE>(p, id, cols, a);
        } else {
          store_row<float, WIDE>(piece_of(p, c, rank * JOIN_WARPS) + cols.first, cols.n, a);
          __threadfence();
          __syncwarp();
          if (lane == 0) go_on = atomicAdd(joined(p, c, blockIdx.y * SUM_COLS), 1u) == JOIN_GROUP - 1;
          __threadfence();
        }
      }
      if (!__syncthreads_or(go_on)) break;
      __threadfence();
      load_row<float, WIDE>(piece_of(p, c, warp * JOIN_WARPS) + cols.first, cols.n, x0);  // a block's sum
#pragma unroll
      for (int k = 0; k < UNIT; ++k) a[k] = x0.v[k];
      end = true;
    }
  }
}

// ------------------------------------------------------------ small batches
// Up to SMALL_IDS ids in one launch without scratch: every block that sums
// sorts the (id, position) pairs for itself (bitonic, in shared memory) and
// has 64 columns, its warps equal shares of the sorted list.  So few columns,
// two a lane, since a block of this size reads 50 to 70 GB/s and each has all
// rows of its columns.  The pieces of runs that cross shares are kept in shared
// memory and added in order by the warp that a run begins in.  Other blocks
// write zero rows as in sum_kernel.
//
// Rows of 256 f32 or 2048 bf16 for 4000 ids: 128 ids take 7 and 13 us, and 15
// and 13 in three kernels, a call from Python 8 and 14 against 19 and 18; 512
// ids 14 and 24, and 16 and 17 in three kernels.
constexpr int SMALL_IDS = 384, SMALL_PAIRS = 512;
constexpr int SMALL_UNIT = 2, SMALL_COLS = 32 * SMALL_UNIT;
constexpr int SMALL_RING = 2048;  // bytes a warp

template <class T, class O, bool WIDE>
__global__ void __launch_bounds__(SUM_WARPS * 32, 2) small_kernel(const __grid_constant__ SumArgs p) {
  using R = Ring<T, WIDE, SMALL_RING, SMALL_UNIT>;
  constexpr uint32_t THREADS = SUM_WARPS * 32;
  __shared__ __align__(16) char small_mem[SUM_WARPS * SMALL_RING];  // the rings; zero rows: the bits
  __shared__ uint64_t pair[SMALL_PAIRS];                            // key << 32 | position
  static_assert(sizeof small_mem >= SPAN / 8, "the rings' memory holds the rows' bits");
  if (blockIdx.x < p.n_zero) return zero_scan<THREADS>(p.z, p.s, blockIdx.x, p.n_zero, reinterpret_cast<uint32_t*>(small_mem));
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32, n = p.n;
  const Cols<WIDE, SMALL_UNIT> at((blockIdx.x - p.n_zero) * SMALL_COLS, p.dim);
  uint32_t size = 2;
  while (size < n) size *= 2;
  for (uint32_t i = threadIdx.x; i < size; i += THREADS)
    pair[i] = i < n ? uint64_t(sort_key(p.s, i)) << 32 | i : ~0ull;
  for (uint32_t k = 2; k <= size; k *= 2)
    for (uint32_t j = k / 2; j; j /= 2) {
      __syncthreads();
      for (uint32_t t = threadIdx.x; t < size / 2; t += THREADS) {
        const uint32_t a = 2 * t - (t & (j - 1)), b = a + j;
        const uint64_t x = pair[a], y = pair[b];
        if ((x > y) == ((a & k) == 0)) {
          pair[a] = y;
          pair[b] = x;
        }
      }
    }
  __syncthreads();
  auto key = [&](uint32_t i) { return uint32_t(pair[i] >> 32); };
  uint32_t m = 0, top = n;  // the ids that take part: the first key of n_vocab
  while (m < top) {
    const uint32_t mid = (m + top) / 2;
    if (key(mid) < p.n_vocab) m = mid + 1;
    else top = mid;
  }
  const uint32_t each = (m + SUM_WARPS - 1) / SUM_WARPS;
  auto share = [&](uint32_t w) { return min(w * each, m); };
  const uint32_t lo = share(warp), hi = share(warp + 1);
  // this share's first run began before it, its last one goes on after it
  const bool head = lo < hi && lo > 0 && key(lo - 1) == key(lo);
  const bool tail = lo < hi && hi < m && key(hi) == key(hi - 1) && !(head && key(lo) == key(hi - 1));
  const T* grad = static_cast<const T*>(p.grad) + at.first;
  R ring(small_mem + warp * SMALL_RING);
  auto copy = [&](uint32_t e) { ring.copy(e < hi ? grad + uint64_t(uint32_t(pair[e])) * p.gstride : nullptr, at.n); };
  float a[SMALL_UNIT] = {}, first[SMALL_UNIT] = {};
  bool piece = head;
  uint32_t id = lo < hi ? key(lo) : 0;
  for (uint32_t k = 0; k + 1 < R::DEPTH; ++k) copy(lo + k);
#pragma unroll 1
  for (uint32_t i = lo; i < hi; ++i) {
    copy(i + R::DEPTH - 1);
    const uint32_t now = key(i);
    if (now != id) {
      if (!piece) write_sum<O, WIDE>(p, id, at, a);
#pragma unroll
      for (int j = 0; j < SMALL_UNIT; ++j) {
        if (piece) first[j] = a[j];
        a[j] = 0.f;
      }
      piece = false;
      id = now;
    }
    ring.add(a);
  }
  if (piece) {  // one run is all of the share
#pragma unroll
    for (int j = 0; j < SMALL_UNIT; ++j) first[j] = a[j];
  } else if (lo < hi && !tail) {
    write_sum<O, WIDE>(p, id, at, a);
  }
  // the pieces that other warps add up: the first run's, where the ring was
  __syncwarp();
  float* mine = reinterpret_cast<float*>(small_mem + warp * SMALL_RING);
#pragma unroll
  for (int j = 0; j < SMALL_UNIT; ++j) mine[j * 32 + lane] = first[j];
  __syncthreads();
  if (!tail) return;
  for (uint32_t w = warp + 1; w < SUM_WARPS && share(w) < m && key(share(w)) == id; ++w) {
    const float* piece_of = reinterpret_cast<const float*>(small_mem + w * SMALL_RING);
#pragma unroll
    for (int j = 0; j < SMALL_UNIT; ++j) a[j] += piece_of[j * 32 + lane];
  }
  write_sum<O, WIDE>(p, id, at, a);
}

// Keep freed stream-ordered memory in the device's default pool across
// calls (the pool otherwise returns it to the system at every synchronize).
cudaError_t keep_pool_memory() {
  static ppi::DeviceOnce once;
  int dev;
  const cudaError_t e = ppi::current_device(&dev);
  if (e != cudaSuccess) return e;
  return once.run(dev, [](int d) {
    cudaMemPool_t pool;
    const cudaError_t e = cudaDeviceGetDefaultMemPool(&pool, d);
    if (e != cudaSuccess) return e;
    uint64_t keep = ~0ull;
    return cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
  });
}

// Per device: attributes of the cluster sort, and its largest cluster.
constexpr int CLUSTER_ITEMS[3] = {1, 2, 8};
using ClusterKernel = void (*)(ClusterArgs);
const ClusterKernel CLUSTER_KERNEL[3] = {cluster_sort_kernel<1>, cluster_sort_kernel<2>, cluster_sort_kernel<8>};

cudaLaunchConfig_t cluster_config(int kind, int blocks, cudaLaunchAttribute* at, cudaStream_t stream) {
  std::memset(at, 0, sizeof *at);
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = blocks;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(CS_THREADS);
  cfg.dynamicSmemBytes = cluster_smem(CLUSTER_ITEMS[kind]);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

cudaError_t cluster_setup(int* blocks) {
  static ppi::DeviceOnce once;
  static int most[ppi::MAX_DEVICES];
  int dev;
  cudaError_t e = ppi::current_device(&dev);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [](int d) {
    for (int k = 0; k < 3; ++k) {
      cudaError_t e = cudaFuncSetAttribute(CLUSTER_KERNEL[k], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           int(cluster_smem(CLUSTER_ITEMS[k])));
      if (e == cudaSuccess) e = cudaFuncSetAttribute(CLUSTER_KERNEL[k], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = cluster_config(2, CS_BLOCKS, &at, nullptr);
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, CLUSTER_KERNEL[2], &cfg);
    most[d] = n > 0 ? CS_BLOCKS : 8;  // 8 blocks run on any device
    return e;
  });
  *blocks = most[dev];
  return e;
}

int key_bits(uint32_t n_vocab) {
  int bits = 1;
  while (bits < 32 && (uint64_t(n_vocab) >> bits)) ++bits;
  return bits;
}

cudaError_t launch_cluster_sort(ClusterArgs& p, int blocks, cudaStream_t stream) {
  // pairs a thread: the fewest that the blocks hold, as the sort is bound by
  // its steps' latencies
  const uint32_t n = p.s.n, threads = uint32_t(CS_THREADS * blocks);
  const int kind = n <= threads ? 0 : n <= 2 * threads ? 1 : 2;
  int c = 1;
  while (c < blocks && uint32_t(CLUSTER_ITEMS[kind] * CS_THREADS * c) < n) c *= 2;
  const int bits = key_bits(p.s.n_vocab);
  p.passes = (bits + CS_BITS - 1) / CS_BITS;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.blocks = c;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = cluster_config(kind, c, &at, stream);
  return cudaLaunchKernelEx(&cfg, CLUSTER_KERNEL[kind], p);
}

cudaError_t launch_sort(SortArgs s, uint32_t* key[2], uint32_t* pos[2], int* at, cudaStream_t stream) {
  const int bits = key_bits(s.n_vocab), passes = (bits + DIGIT_BITS - 1) / DIGIT_BITS;
  s.bits = (bits + passes - 1) / passes;
  int to = 0;
  for (int pass = 0; pass < passes; ++pass) {
    s.shift = pass * s.bits;
    s.key_out = key[to];
    s.pos_out = pos[to];
    sort_count_kernel<<<s.n_tiles, SORT_THREADS, 0, stream>>>(s);
    sort_scan_kernel<<<1u << s.bits, SORT_THREADS, 0, stream>>>(s);
    sort_move_kernel<<<s.n_tiles, SORT_THREADS, 0, stream>>>(s);
    s.ids = nullptr;
    s.key_in = key[to];
    s.pos_in = pos[to];
    to ^= 1;
  }
  *at = to ^ 1;
  return cudaGetLastError();
}

template <class K>
cudaError_t launch_next(K kernel, dim3 grid, dim3 block, const SumArgs& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class T, class O>
bool wide_rows(const SumArgs& p) {
  return rows_aligned(p.grad, sizeof(T), p.gstride, p.n) && rows_aligned(p.out, sizeof(O), p.ostride, p.n_vocab);
}

template <class T, class O, bool WIDE>
cudaError_t launch_small(const SumArgs& p, cudaStream_t stream) {
  const uint32_t sums = p.n ? (p.dim + SMALL_COLS - 1) / SMALL_COLS : 0;
  small_kernel<T, O, WIDE><<<p.n_zero + sums, SUM_WARPS * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class T, class O>
cudaError_t launch_sums(const SumArgs& p, cudaStream_t stream) {
  const bool wide = wide_rows<T, O>(p);
  const unsigned grid = unsigned(p.n_zero + (uint64_t(p.n_chunks) * p.slices + SUM_WARPS - 1) / SUM_WARPS);
  const uint32_t runs = std::min(p.n_chunks, std::max(uint32_t(JOIN_BLOCKS), 152 * 8 / p.slices));
  const dim3 join((runs + JOIN_GROUP - 1) / JOIN_GROUP * JOIN_GROUP, p.slices);
  cudaError_t e = launch_next(wide ? sum_kernel<T, O, true> : sum_kernel<T, O, false>, grid, SUM_WARPS * 32, p, stream);
  if (e == cudaSuccess)
    e = launch_next(wide ? join_kernel<O, true> : join_kernel<O, false>, join, JOIN_WARPS * 32, p, stream);
  return e;
}

// What a gradient's sorted list and partial sums take, in 32-bit words.
struct GradPlan {
  uint32_t slices, chunk, n_chunks, n_tiles;
  size_t width, parts, longs, pairs, counts;
  bool one;  // one cluster sorts
  size_t bytes() const { return 4 * (parts + 4 + longs + (one ? 2 : 4) * pairs + (one ? 0 : counts)); }
};

GradPlan grad_plan(size_t n, size_t dim, int cluster_blocks) {
  GradPlan g;
  g.slices = uint32_t((dim + SUM_COLS - 1) / SUM_COLS);
  // chunks of 32 where they make enough warps to fill the machine (24 on
  // each of 152 multiprocessors), else shorter ones: 8192 rows of 1024 take
  // 34 us in chunks of 8, 37 in 16 and 45 in 32; but shorter ones leave more
  // pieces of long runs, and 100000 rows of 512 for 1000 ids take 95 us in
  // chunks of 32, 109 in 16 and 119 in 8
  g.chunk = 32;
  while (g.chunk > 8 && uint64_t(n) / g.chunk * g.slices < 152 * 24) g.chunk /= 2;
  g.n_chunks = uint32_t((n + g.chunk - 1) / g.chunk);
  g.n_tiles = uint32_t((n + SORT_TILE - 1) / SORT_TILE);
  g.one = n <= uint64_t(SORT_CAP) / CS_BLOCKS * cluster_blocks;
  g.width = (dim + 7) / 8 * 8;
  g.parts = size_t(g.n_chunks) * 2 * g.width;
  g.longs = (size_t(g.n_chunks) + 1) / 2 * 4;  // in fours
  g.pairs = (n + 3) / 4 * 4;
  g.counts = (size_t(g.n_tiles) + 1) * DIGITS;
  return g;
}

// pp_embed_grad and its form with the caller's scratch (given).
pp_rc embed_grad(const void* d_ids, pp_itype id_type, size_t id_stride, size_t n, const void* d_grad, pp_ftype grad_type,
                 size_t grad_stride, size_t n_vocab, size_t dim, float scale, int64_t padding_id, int accumulate, void* d_out,
                 pp_ftype out_type, size_t out_stride, bool given, void* scratch, size_t scratch_bytes, cudaStream_t stream) {
  if (!ppl::itype_ok(id_type) || !ppl::ftype_ok(grad_type) || !ppl::ftype_ok(out_type)) return PP_EINVAL;
  if (n_vocab && dim && (!d_out || (n && (!d_ids || !d_grad)))) return PP_EINVAL;
  if (n_vocab > 1 && out_stride < dim) return PP_EINVAL;
  if (!ppl::aligned(d_ids, ppl::isize(id_type)) || !ppl::aligned(d_grad, ppl::fsize(grad_type)) ||
      !ppl::aligned(d_out, ppl::fsize(out_type)))
    return PP_EINVAL;
  if (n >= ppl::MAX_DIM || n_vocab >= ppl::MAX_DIM || dim >= ppl::MAX_DIM) return PP_ETOOLARGE;
  if (dim > uint64_t(65535) * SUM_COLS) return PP_ETOOLARGE;  // the grid's second dimension
  if (!n_vocab || !dim || (!n && accumulate)) return PP_OK;
  if (given && (scratch_bytes < pp_embed_grad_scratch(n, n_vocab, dim) || !ppl::aligned(scratch, 16) ||
                (!scratch && pp_embed_grad_scratch(n, n_vocab, dim))))
    return PP_EINVAL;
  int n_sm;
  cudaError_t e = ppi::sm_count(&n_sm);
  if (e != cudaSuccess) return ppl::rc_of(e);
  const size_t size = ppl::fsize(out_type);
  int blocks = CS_BLOCKS;
  if (n > SMALL_IDS && (e = cluster_setup(&blocks)) != cudaSuccess) return ppl::rc_of(e);
  const GradPlan plan = grad_plan(n, dim, blocks);
  SumArgs p;
  std::memset(&p, 0, sizeof p);
  p.n = uint32_t(n);
  p.n_vocab = uint32_t(n_vocab);
  p.grad = d_grad;
  p.gstride = grad_stride;
  p.dim = uint32_t(dim);
  p.scale = scale;
  p.accumulate = accumulate;
  p.out = d_out;
  p.ostride = out_stride;
  p.slices = plan.slices;
  p.width = plan.width;
  p.chunk = plan.chunk;
  p.n_chunks = plan.n_chunks;
  if (uint64_t(p.n_chunks) * p.slices / SUM_WARPS >= ppl::MAX_DIM) return PP_ETOOLARGE;
  ZeroArgs z;
  z.out = d_out;
  z.row_bytes = dim * size;
  z.stride_bytes = out_stride * size;
  z.n_vocab = uint32_t(n_vocab);
  z.wide = z.row_bytes % 16 == 0 && rows_aligned(d_out, size, out_stride, n_vocab);
  z.elem_size = int(size);
  SortArgs s;
  std::memset(&s, 0, sizeof s);
  s.ids = d_ids;
  s.type = id_type;
  s.id_stride = id_stride;
  s.n = uint32_t(n);
  s.n_vocab = uint32_t(n_vocab);
  s.pad = padding_id;
  if (!accumulate) {  // two blocks a multiprocessor, but none for less than 64 KiB
    p.z = z;
    p.s = s;
    p.n_zero = uint32_t(std::min<uint64_t>(2 * n_sm, n_vocab * dim * size / 65536 + 1));
  }
  if (n <= SMALL_IDS) {
    p.s = s;
    return ppl::rc_of(with_type(grad_type, [&](auto t) {
      return with_type(out_type, [&](auto o) {
        using T = decltype(t);
        using O = decltype(o);
        return wide_rows<T, O>(p) ? launch_small<T, O, true>(p, stream) : launch_small<T, O, false>(p, stream);
      });
    }));
  }
  s.n_tiles = plan.n_tiles;
  if (!given) {
    if ((e = keep_pool_memory()) != cudaSuccess) return ppl::rc_of(e);
    e = cudaMallocAsync(&scratch, plan.bytes(), stream);
    if (e != cudaSuccess) return ppl::rc_of(e);
  }
  p.part = static_cast<float*>(scratch);
  uint32_t* u = reinterpret_cast<uint32_t*>(p.part + plan.parts);
  p.n_long = u;
  p.longs = reinterpret_cast<uint2*>(u + 4);
  u += 4 + plan.longs;
  uint32_t* key[2] = {u, u + 2 * plan.pairs};
  uint32_t* pos[2] = {u + plan.pairs, u + 3 * plan.pairs};
  s.counts = u + 4 * plan.pairs;
  int at = 0;
  if (plan.one) {
    ClusterArgs c;
    c.s = s;
    c.s.key_out = key[0];
    c.s.pos_out = pos[0];
    c.n_long = p.n_long;
    e = launch_cluster_sort(c, blocks, stream);
  } else {
    p.n_zero = 0;  // from the sorted list
    e = cudaMemsetAsync(p.n_long, 0, 8, stream);
    if (e == cudaSuccess) e = launch_sort(s, key, pos, &at, stream);
    if (e == cudaSuccess && !accumulate) {
      zero_kernel<<<unsigned((n_vocab + ZERO_SPAN - 1) / ZERO_SPAN), 256, 0, stream>>>(z, key[at], s.n);
      e = cudaGetLastError();
    }
  }
  p.key = key[at];
  p.pos = pos[at];
  if (e == cudaSuccess)
    e = with_type(grad_type, [&](auto t) {
      return with_type(out_type, [&](auto o) { return launch_sums<decltype(t), decltype(o)>(p, stream); });
    });
  const cudaError_t ef = given ? cudaSuccess : cudaFreeAsync(scratch, stream);
  return ppl::rc_of(e == cudaSuccess ? ef : e);
}

}  // namespace

extern "C" {

pp_rc pp_embed(const void* d_ids, pp_itype id_type, size_t id_stride, size_t n,
               const void* d_table, pp_ftype table_type, size_t n_vocab, size_t dim,
               size_t table_stride, float scale, int64_t padding_id, void* d_out,
               pp_ftype out_type, size_t out_stride, cudaStream_t stream) {
  if (!ppl::itype_ok(id_type) || !ppl::ftype_ok(table_type) || !ppl::ftype_ok(out_type)) return PP_EINVAL;
  if (n && dim && (!d_ids || !d_out || (n_vocab && !d_table))) return PP_EINVAL;
  if (n > 1 && out_stride < dim) return PP_EINVAL;
  if (!ppl::aligned(d_ids, ppl::isize(id_type)) || !ppl::aligned(d_table, ppl::fsize(table_type)) ||
      !ppl::aligned(d_out, ppl::fsize(out_type)))
    return PP_EINVAL;
  if (n >= ppl::MAX_DIM || n_vocab >= ppl::MAX_DIM || dim >= ppl::MAX_DIM) return PP_ETOOLARGE;
  if (!n || !dim) return PP_OK;
  const EmbedArgs p = {d_ids, id_type, id_stride, uint32_t(n), d_table, uint32_t(n_vocab),
                       uint32_t(dim), table_stride, scale, padding_id, d_out, out_stride};
  return ppl::rc_of(with_type(table_type, [&](auto t) {
    return with_type(out_type, [&](auto o) { return launch_embed<decltype(t), decltype(o)>(p, stream); });
  }));
}

size_t pp_embed_grad_scratch(size_t n, size_t n_vocab, size_t dim) {
  if (n <= SMALL_IDS || !n_vocab || !dim || n >= ppl::MAX_DIM || dim >= ppl::MAX_DIM) return 0;
  return grad_plan(n, dim, CS_BLOCKS / 2).bytes();  // no less than with clusters of CS_BLOCKS
}

pp_rc pp_embed_grad(const void* d_ids, pp_itype id_type, size_t id_stride, size_t n,
                    const void* d_grad, pp_ftype grad_type, size_t grad_stride, size_t n_vocab,
                    size_t dim, float scale, int64_t padding_id, int accumulate, void* d_out,
                    pp_ftype out_type, size_t out_stride, cudaStream_t stream) {
  return embed_grad(d_ids, id_type, id_stride, n, d_grad, grad_type, grad_stride, n_vocab, dim, scale, padding_id,
                    accumulate, d_out, out_type, out_stride, false, nullptr, 0, stream);
}

pp_rc pp_embed_grad_noalloc(const void* d_ids, pp_itype id_type, size_t id_stride, size_t n,
                            const void* d_grad, pp_ftype grad_type, size_t grad_stride, size_t n_vocab,
                            size_t dim, float scale, int64_t padding_id, int accumulate, void* d_out,
                            pp_ftype out_type, size_t out_stride, void* d_scratch, size_t scratch_bytes,
                            cudaStream_t stream) {
  return embed_grad(d_ids, id_type, id_stride, n, d_grad, grad_type, grad_stride, n_vocab, dim, scale, padding_id,
                    accumulate, d_out, out_type, out_stride, true, d_scratch, scratch_bytes, stream);
}

}  // extern "C"
