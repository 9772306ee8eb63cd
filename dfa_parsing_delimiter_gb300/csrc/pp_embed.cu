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
#include <algorithm>
#include <cstring>

#include "pp_device.cuh"
#include "pp_internal.h"
#include "pp_lm.cuh"

namespace {

using namespace ppd;
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
// and step (8 where rows are aligned to 16 bytes in both arrays).
template <class T, class O, int U>
__global__ void __launch_bounds__(256) embed_kernel(const __grid_constant__ EmbedArgs p) {
  const uint64_t i = uint64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (i >= p.n) return;
  const int64_t id = load_id(p.ids, p.type, i * p.id_stride);
  const bool there = id >= 0 && id < p.n_vocab && id != p.pad;
  const T* row = static_cast<const T*>(p.table) + (there ? uint64_t(id) * p.tstride : 0);
  O* out = static_cast<O*>(p.out) + i * p.ostride;
  for (uint64_t c = uint64_t(threadIdx.x) * U; c < p.dim; c += uint64_t(blockDim.x) * U) {
    if (U > 1 && c + U <= p.dim) {
      Pack<T, U> x;
      Pack<O, U> y;
      if (there) x = *reinterpret_cast<const Pack<T, U>*>(row + c);
#pragma unroll
      for (int k = 0; k < U; ++k) y.v[k] = from_f<O>(there ? to_f(x.v[k]) * p.scale : 0.f);
      *reinterpret_cast<Pack<O, U>*>(out + c) = y;
    } else {
      for (uint64_t k = c; k < c + U && k < p.dim; ++k)
        out[k] = from_f<O>(there ? to_f(row[k]) * p.scale : 0.f);
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
  uint32_t x = 1;
  while (x < 256 && x < steps) x *= 2;
  const dim3 block(x, 256 / x);
  const unsigned grid = unsigned((uint64_t(p.n) + block.y - 1) / block.y);
  if (wide) embed_kernel<T, O, UNIT><<<grid, block, 0, stream>>>(p);
  else embed_kernel<T, O, 1><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------- sort by id
// Least significant digit first; each pass counts the digits of every tile,
// scans the counts by (digit, tile) and moves the pairs.  Keys: the id, or
// n_vocab for a position that takes no part (sorted last).
constexpr int SORT_THREADS = 256, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ITEMS = 16;  // pairs a thread
constexpr uint32_t SORT_TILE = SORT_THREADS * SORT_ITEMS;
constexpr int DIGIT_BITS = 8, DIGITS = 1 << DIGIT_BITS;

struct SortArgs {
  const void* ids;  // first pass: the ids; else null
  int32_t type;
  uint64_t id_stride;
  uint32_t n, n_vocab;
  int64_t pad;
  const uint32_t *key_in, *pos_in;
  uint32_t *key_out, *pos_out;
  uint32_t* counts;  // [DIGITS][n_tiles]
  uint32_t n_tiles;
  int shift;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& p, uint64_t i) {
  if (!p.ids) return p.key_in[i];
  const int64_t id = load_id(p.ids, p.type, i * p.id_stride);
  return id >= 0 && id < p.n_vocab && id != p.pad ? uint32_t(id) : p.n_vocab;
}

__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(const __grid_constant__ SortArgs p) {
  __shared__ uint32_t count[DIGITS];
  count[threadIdx.x] = 0;
  __syncthreads();
  const uint64_t base = uint64_t(blockIdx.x) * SORT_TILE;
#pragma unroll 4
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const uint64_t i = base + k * SORT_THREADS + threadIdx.x;
    if (i < p.n) atomicAdd(&count[sort_key(p, i) >> p.shift & (DIGITS - 1)], 1u);
  }
  __syncthreads();
  p.counts[uint64_t(threadIdx.x) * p.n_tiles + blockIdx.x] = count[threadIdx.x];
}

// Exclusive scan of the counts in place, one block.
__global__ void __launch_bounds__(1024) sort_scan_kernel(uint32_t* counts, uint64_t n) {
  __shared__ uint32_t total[32];
  __shared__ uint32_t carry;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (uint64_t base = 0; base < n; base += 4096) {
    uint32_t v[4], sum = 0;
    const uint64_t at = base + threadIdx.x * 4;
    for (int k = 0; k < 4; ++k) {
      v[k] = at + k < n ? counts[at + k] : 0;
      sum += v[k];
    }
    uint32_t inc = sum;
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t up = __shfl_up_sync(FULL, inc, d);
      if (lane >= d) inc += up;
    }
    if (lane == 31) total[warp] = inc;
    __syncthreads();
    uint32_t run = carry;
    for (int w = 0; w < warp; ++w) run += total[w];
    run += inc - sum;
    for (int k = 0; k < 4; ++k)
      if (at + k < n) {
        counts[at + k] = run;
        run += v[k];
      }
    __syncthreads();
    if (threadIdx.x == 1023) carry = run;
    __syncthreads();
  }
}

// Stable move: warp w of the block owns SORT_ITEMS x 32 consecutive pairs,
// ranks equal digits by match and adds them up per warp in order.
__global__ void __launch_bounds__(SORT_THREADS) sort_move_kernel(const __grid_constant__ SortArgs p) {
  __shared__ uint32_t place[SORT_WARPS][DIGITS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int w = 0; w < SORT_WARPS; ++w) place[w][threadIdx.x] = 0;
  __syncthreads();
  const uint64_t base = uint64_t(blockIdx.x) * SORT_TILE + warp * (SORT_ITEMS * 32) + lane;
  uint32_t key[SORT_ITEMS], rank[SORT_ITEMS];
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) key[k] = base + k * 32 < p.n ? sort_key(p, base + k * 32) : 0;
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const bool there = base + k * 32 < p.n;
    const uint32_t d = there ? key[k] >> p.shift & (DIGITS - 1) : DIGITS;
    const uint32_t same = __match_any_sync(FULL, d);
    if (there) rank[k] = place[warp][d] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (there && lane == 31 - __clz(same)) place[warp][d] = rank[k] + 1;
    __syncwarp();
  }
  __syncthreads();
  uint32_t run = p.counts[uint64_t(threadIdx.x) * p.n_tiles + blockIdx.x];
  for (int w = 0; w < SORT_WARPS; ++w) {
    const uint32_t c = place[w][threadIdx.x];
    place[w][threadIdx.x] = run;
    run += c;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k)
    if (base + k * 32 < p.n) {
      const uint32_t to = place[warp][key[k] >> p.shift & (DIGITS - 1)] + rank[k];
      p.key_out[to] = key[k];
      p.pos_out[to] = p.ids ? uint32_t(base + k * 32) : p.pos_in[base + k * 32];
    }
}

// ------------------------------------------------------------ sums of runs
struct SumArgs {
  const uint32_t *key, *pos;  // sorted by (key, position)
  uint32_t n, n_vocab;
  const void* grad;
  uint64_t gstride;
  uint32_t dim;
  float scale;
  int32_t accumulate;
  void* out;
  uint64_t ostride;
  float* part;  // [n_chunks][2][dim]: sums of a chunk's first and last run
  uint32_t n_chunks, chunk;
};

constexpr int SUM_WARPS = 8;
constexpr int SUM_COLS = 32 * UNIT;  // columns a warp

// Columns of a warp: a lane has 8 consecutive ones (aligned rows) or every
// 32nd one (any rows).
template <bool WIDE>
__device__ __forceinline__ uint64_t col_of(uint64_t c0, int k) {
  const int lane = threadIdx.x & 31;
  return WIDE ? c0 + lane * UNIT + k : c0 + lane + 32 * k;
}

template <class T, bool WIDE>
__device__ __forceinline__ void load_row(const T* row, uint64_t c0, uint32_t dim, float (&x)[UNIT]) {
  if (WIDE && col_of<WIDE>(c0, UNIT) <= dim) {
    const Pack<T, UNIT> v = *reinterpret_cast<const Pack<T, UNIT>*>(row + col_of<WIDE>(c0, 0));
#pragma unroll
    for (int k = 0; k < UNIT; ++k) x[k] = to_f(v.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < UNIT; ++k) x[k] = col_of<WIDE>(c0, k) < dim ? to_f(row[col_of<WIDE>(c0, k)]) : 0.f;
  }
}

template <class O, bool WIDE>
__device__ __forceinline__ void store_row(O* row, uint64_t c0, uint32_t dim, const float (&x)[UNIT]) {
  if (WIDE && col_of<WIDE>(c0, UNIT) <= dim) {
    Pack<O, UNIT> v;
#pragma unroll
    for (int k = 0; k < UNIT; ++k) v.v[k] = from_f<O>(x[k]);
    *reinterpret_cast<Pack<O, UNIT>*>(row + col_of<WIDE>(c0, 0)) = v;
  } else {
#pragma unroll
    for (int k = 0; k < UNIT; ++k)
      if (col_of<WIDE>(c0, k) < dim) row[col_of<WIDE>(c0, k)] = from_f<O>(x[k]);
  }
}

template <class O, bool WIDE>
__device__ __forceinline__ void write_sum(const SumArgs& p, uint32_t id, uint64_t c0, float (&a)[UNIT]) {
  O* row = static_cast<O*>(p.out) + uint64_t(id) * p.ostride;
#pragma unroll
  for (int k = 0; k < UNIT; ++k) a[k] *= p.scale;
  if (p.accumulate) {
    float old[UNIT];
    load_row<O, WIDE>(row, c0, p.dim, old);
#pragma unroll
    for (int k = 0; k < UNIT; ++k) a[k] += old[k];
  }
  store_row<O, WIDE>(row, c0, p.dim, a);
}

// Of the sorted list, chunk c holds [c L, (c + 1) L).  A run is long if it
// begins in chunk c and goes on past the end of chunk c + 1.
struct Runs {
  const uint32_t* key;
  uint64_t n, L;
  // whether the run that holds index i (the first of chunk c > 0) began
  // before it
  __device__ bool goes_on(uint64_t c) const { return c > 0 && c * L < n && key[c * L - 1] == key[c * L]; }
  // whether the run that crosses from chunk c - 1 into chunk c is long
  __device__ bool long_into(uint64_t c) const {
    const uint32_t id = key[c * L];
    if (c >= 2 && key[(c - 1) * L - 1] == id) return true;          // began before chunk c - 1
    return (c + 1) * L < n && key[(c + 1) * L] == id;               // passes the end of chunk c
  }
};

template <class T, class O, bool WIDE>
__global__ void __launch_bounds__(SUM_WARPS * 32) sum_kernel(const __grid_constant__ SumArgs p) {
  const uint64_t c = blockIdx.x;
  const uint64_t c0 = (uint64_t(blockIdx.y) * SUM_WARPS + threadIdx.x / 32) * SUM_COLS;
  if (c0 >= p.dim) return;
  const Runs runs = {p.key, p.n, p.chunk};
  const uint64_t L = p.chunk, lo = c * L, hi = min(lo + L, uint64_t(p.n));
  const T* grad = static_cast<const T*>(p.grad);
  uint64_t i = lo;
  float a[UNIT], x[UNIT];
  bool part = false;  // the current run is a piece of a long one
  if (runs.goes_on(c)) {
    part = runs.long_into(c);
    if (!part)  // finished by the chunk before
      while (i < hi && p.key[i] == p.key[lo]) ++i;
  }
  while (i < hi) {
    const uint32_t id = p.key[i];
    if (id >= p.n_vocab) break;
#pragma unroll
    for (int k = 0; k < UNIT; ++k) a[k] = 0.f;
    const bool head = part;
    // to the run's end, which is past the chunk's where that makes it whole
    const bool tail = !head && (c + 2) * L < p.n && p.key[(c + 2) * L] == id;
    const uint64_t end = head || tail ? hi : min(hi + L, uint64_t(p.n));
    for (; i < end && p.key[i] == id; ++i) {
      load_row<T, WIDE>(grad + uint64_t(p.pos[i]) * p.gstride, c0, p.dim, x);
#pragma unroll
      for (int k = 0; k < UNIT; ++k) a[k] += x[k];
    }
    if (head || tail) store_row<float, WIDE>(p.part + (2 * c + (tail ? 1 : 0)) * uint64_t((p.dim + 7) / 8 * 8), c0, p.dim, a);
    else write_sum<O, WIDE>(p, id, c0, a);
    part = false;
  }
}

// Adds the pieces of the long run that begins in chunk c, in order.
template <class O, bool WIDE>
__global__ void __launch_bounds__(SUM_WARPS * 32) join_kernel(const __grid_constant__ SumArgs p) {
  const uint64_t c = blockIdx.x, L = p.chunk;
  const uint64_t c0 = (uint64_t(blockIdx.y) * SUM_WARPS + threadIdx.x / 32) * SUM_COLS;
  if (c0 >= p.dim || (c + 2) * L >= p.n) return;
  const uint32_t id = p.key[(c + 1) * L - 1];
  if (id >= p.n_vocab || p.key[(c + 2) * L] != id) return;
  if (c > 0 && p.key[c * L - 1] == id) return;  // it began earlier
  const uint64_t width = (p.dim + 7) / 8 * 8;
  float a[UNIT], x[UNIT];
  load_row<float, WIDE>(p.part + (2 * c + 1) * width, c0, p.dim, a);
  for (uint64_t d = c + 1; d * L < p.n && p.key[d * L] == id; ++d) {
    load_row<float, WIDE>(p.part + 2 * d * width, c0, p.dim, x);
#pragma unroll
    for (int k = 0; k < UNIT; ++k) a[k] += x[k];
  }
  write_sum<O, WIDE>(p, id, c0, a);
}

// Rows of ids that do not occur become zeros.
template <class O, bool WIDE>
__global__ void __launch_bounds__(256) fill_kernel(const __grid_constant__ SumArgs p) {
  const uint64_t v = blockIdx.x;
  uint32_t lo = 0, hi = p.n;  // the first sorted index whose key is v or more
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (p.key[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  if (lo < p.n && p.key[lo] == v) return;
  const float zero[UNIT] = {};
  O* row = static_cast<O*>(p.out) + v * p.ostride;
  for (uint64_t c0 = (threadIdx.x / 32) * SUM_COLS; c0 < p.dim; c0 += 8 * SUM_COLS)
    store_row<O, WIDE>(row, c0, p.dim, zero);
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

cudaError_t launch_sort(SortArgs s, uint32_t* key[2], uint32_t* pos[2], int* at, cudaStream_t stream) {
  int bits = 1;
  while (bits < 32 && (uint64_t(s.n_vocab) >> bits)) ++bits;
  int to = 0;
  for (int shift = 0; shift < bits; shift += DIGIT_BITS) {
    s.shift = shift;
    s.key_out = key[to];
    s.pos_out = pos[to];
    sort_count_kernel<<<s.n_tiles, SORT_THREADS, 0, stream>>>(s);
    sort_scan_kernel<<<1, 1024, 0, stream>>>(s.counts, uint64_t(s.n_tiles) * DIGITS);
    sort_move_kernel<<<s.n_tiles, SORT_THREADS, 0, stream>>>(s);
    s.ids = nullptr;
    s.key_in = key[to];
    s.pos_in = pos[to];
    to ^= 1;
  }
  *at = to ^ 1;
  return cudaGetLastError();
}

template <class T, class O>
cudaError_t launch_sums(const SumArgs& p, cudaStream_t stream) {
  const bool wide = rows_aligned(p.grad, sizeof(T), p.gstride, p.n) &&
                    rows_aligned(p.out, sizeof(O), p.ostride, p.n_vocab);
  const unsigned y = unsigned((uint64_t(p.dim) + SUM_COLS * SUM_WARPS - 1) / (SUM_COLS * SUM_WARPS));
  const dim3 grid(p.n_chunks, y);
  if (!p.accumulate) {
    if (wide) fill_kernel<O, true><<<p.n_vocab, 256, 0, stream>>>(p);
    else fill_kernel<O, false><<<p.n_vocab, 256, 0, stream>>>(p);
  }
  if (!p.n) return cudaGetLastError();
  if (wide) {
    sum_kernel<T, O, true><<<grid, SUM_WARPS * 32, 0, stream>>>(p);
    if (p.n_chunks > 2) join_kernel<O, true><<<grid, SUM_WARPS * 32, 0, stream>>>(p);
  } else {
    sum_kernel<T, O, false><<<grid, SUM_WARPS * 32, 0, stream>>>(p);
    if (p.n_chunks > 2) join_kernel<O, false><<<grid, SUM_WARPS * 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
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

pp_rc pp_embed_grad(const void* d_ids, pp_itype id_type, size_t id_stride, size_t n,
                    const void* d_grad, pp_ftype grad_type, size_t grad_stride, size_t n_vocab,
                    size_t dim, float scale, int64_t padding_id, int accumulate, void* d_out,
                    pp_ftype out_type, size_t out_stride, cudaStream_t stream) {
  if (!ppl::itype_ok(id_type) || !ppl::ftype_ok(grad_type) || !ppl::ftype_ok(out_type)) return PP_EINVAL;
  if (n_vocab && dim && (!d_out || (n && (!d_ids || !d_grad)))) return PP_EINVAL;
  if (n_vocab > 1 && out_stride < dim) return PP_EINVAL;
  if (!ppl::aligned(d_ids, ppl::isize(id_type)) || !ppl::aligned(d_grad, ppl::fsize(grad_type)) ||
      !ppl::aligned(d_out, ppl::fsize(out_type)))
    return PP_EINVAL;
  if (n >= ppl::MAX_DIM || n_vocab >= ppl::MAX_DIM || dim >= ppl::MAX_DIM) return PP_ETOOLARGE;
  if (dim > uint64_t(65535) * SUM_COLS * SUM_WARPS) return PP_ETOOLARGE;  // the grid's second dimension
  if (!n_vocab || !dim || (!n && accumulate)) return PP_OK;
  cudaError_t e = keep_pool_memory();
  if (e != cudaSuccess) return ppl::rc_of(e);
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
  p.chunk = 64;
  p.n_chunks = uint32_t((n + p.chunk - 1) / p.chunk);
  SortArgs s;
  std::memset(&s, 0, sizeof s);
  s.ids = d_ids;
  s.type = id_type;
  s.id_stride = id_stride;
  s.n = uint32_t(n);
  s.n_vocab = uint32_t(n_vocab);
  s.pad = padding_id;
  s.n_tiles = uint32_t((n + SORT_TILE - 1) / SORT_TILE);
  const size_t width = (dim + 7) / 8 * 8;
  const size_t counts = size_t(s.n_tiles) * DIGITS, pairs = (n + 3) / 4 * 4;
  const size_t parts = p.n_chunks > 2 ? size_t(p.n_chunks) * 2 * width : 0;
  void* scratch = nullptr;
  e = cudaMallocAsync(&scratch, 4 * (parts + 4 * pairs + counts) + 16, stream);
  if (e != cudaSuccess) return ppl::rc_of(e);
  p.part = static_cast<float*>(scratch);
  uint32_t* u = reinterpret_cast<uint32_t*>(p.part + parts);
  uint32_t* key[2] = {u, u + pairs};
  uint32_t* pos[2] = {u + 2 * pairs, u + 3 * pairs};
  s.counts = u + 4 * pairs;
  int at = 0;
  if (n) e = launch_sort(s, key, pos, &at, stream);
  p.key = key[at];
  p.pos = pos[at];
  if (e == cudaSuccess)
    e = with_type(grad_type, [&](auto t) {
      return with_type(out_type, [&](auto o) { return launch_sums<decltype(t), decltype(o)>(p, stream); });
    });
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  return ppl::rc_of(e == cudaSuccess ? ef : e);
}

}  // extern "C"
