// embed_tokens.cu -- the embedding lookup over vocabulary shards and its gradient.
//
//   out_t = scale table[token_t]          (a word of another number gives 0)
//   dtable_w = scale sum of dout_t over the t with token_t = w, in order of t
//
// Both are bound by memory. The lookup takes a warp for 2 KiB of a row: its four
// 16-byte loads a lane are in flight at once, and a few tokens still make many warps.
//
// The gradient sums in an order that no run changes, with no atomics on values: the
// pairs (word, t) are sorted, and a warp sums a chunk of 32 (few tokens: 8) sorted
// tokens by 256 columns, its loads in flight eight at a time. A word whose tokens lie
// in one chunk is stored at once; of others each chunk leaves its part, and the
// chunk where such a word begins adds the parts up, in order, in a kernel behind.
// A pair is one 64-bit number, no two alike, so any way of sorting gives the same
// order: blocks sort tiles of 8192 in shared memory, and if there are several, each
// pair's place is its place in its tile and its places by bisection in the others.
// Where the tables are not added to, the blocks beside the sorting ones fill them
// with zeros meanwhile; rows of words that occur are written once more.
#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {
namespace {

constexpr int kSortThreads = 512;
constexpr int kTile = 8192;  // pairs of a tile: 64 KiB
constexpr uint64_t kNone = ~0ull;

__device__ __forceinline__ int shard_of(const int64_t* first, int nranks, int64_t word) {
  int r = 0;
  while (r + 1 < nranks && first[r + 1] <= word) r++;
  return r;
}

template <typename T>
__global__ void __launch_bounds__(256) embed_kernel(const __grid_constant__ EmbedArgs a) {
  constexpr int kLoads = 4, kSpan = kLoads * 32 * 16 / (int)sizeof(T);  // elements of a warp
  constexpr int kEach = 16 / (int)sizeof(T);
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = unit / a.spans;
  const int d0 = (int)(unit % a.spans) * kSpan + lane * kEach;
  if (t >= a.tokens) return;
  const int64_t word = a.tokens_in[t];
  const bool there = word >= 0 && word < a.first[a.nranks];
  const int r = shard_of(a.first, a.nranks, word);
  const T* row = (const T*)a.tables[r] + (there ? (word - a.first[r]) * a.row_stride[r] : 0);
  T* out = (T*)a.out + t * a.out_stride;
  uint4 u[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; i++) {
    const int d = d0 + i * 32 * kEach;
    u[i] = make_uint4(0, 0, 0, 0);
    if (there && d < a.hidden) u[i] = *reinterpret_cast<const uint4*>(row + d);
  }
#pragma unroll
  for (int i = 0; i < kLoads; i++) {
    const int d = d0 + i * 32 * kEach;
    if (d >= a.hidden) continue;
    uint32_t* x = reinterpret_cast<uint32_t*>(&u[i]);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if (sizeof(T) == 4) x[j] = there ? __float_as_uint(__uint_as_float(x[j]) * a.scale) : 0u;
      else x[j] = there ? bf16_pair(bf16_lo(x[j]) * a.scale, bf16_hi(x[j]) * a.scale) : 0u;
    }
    *reinterpret_cast<uint4*>(out + d) = u[i];
  }
}

// Blocks 0 .. tiles - 1 sort a tile each; the others fill the tables with zeros.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ EmbedBwdArgs a) {
  extern __shared__ uint64_t pair[];
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  if ((int)blockIdx.x >= a.tiles) {
    const int64_t warps = (int64_t)(gridDim.x - a.tiles) * (kSortThreads / 32);
    const int lane = threadIdx.x & 31;
    int r = 0;
    for (int64_t w = (int64_t)(blockIdx.x - a.tiles) * (kSortThreads / 32) + (threadIdx.x >> 5); w < a.first[a.nranks];
         w += warps) {
      while (a.first[r + 1] <= w) r++;
      float* row = a.dtables[r] + (w - a.first[r]) * a.drow_stride[r];
      for (int d = lane * 4; d < a.hidden; d += 128) *reinterpret_cast<float4*>(row + d) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const int64_t at = (int64_t)blockIdx.x * kTile;
  const int count = (int)min((int64_t)kTile, a.tokens - at);
  int size = 2;
  while (size < count) size *= 2;
  for (int i = threadIdx.x; i < size; i += kSortThreads) {
    const int64_t word = i < count ? a.tokens_in[at + i] : -1;
    pair[i] = word >= 0 && word < a.first[a.nranks] ? (uint64_t)word << 32 | (uint64_t)(at + i) : kNone;
  }
  for (int k = 2; k <= size; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < size / 2; i += kSortThreads) {
        const int lo = (i & ~(j - 1)) * 2 | (i & (j - 1)), hi = lo | j;
        const uint64_t x = pair[lo], y = pair[hi];
        if ((x > y) == ((lo & k) == 0)) {
          pair[lo] = y;
          pair[hi] = x;
        }
      }
    }
  }
  __syncthreads();
  uint64_t* to = a.tiles == 1 ? a.sorted : a.sorted_tiles;
  for (int i = threadIdx.x; i < count; i += kSortThreads) to[at + i] = pair[i];
}

// Tiles to one row of pairs. Tokens that ask for nothing are alike: their order is of no matter, they stay behind.
__global__ void __launch_bounds__(256) embed_merge_kernel(const __grid_constant__ EmbedBwdArgs a) {
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens) return;
  const uint64_t x = a.sorted_tiles[i];
  const int mine = (int)(i / kTile);
  int64_t place = i % kTile;
  for (int t = 0; t < a.tiles; t++) {
    if (t == mine) continue;
    const uint64_t* tile = a.sorted_tiles + (int64_t)t * kTile;
    int lo = 0, hi = (int)min((int64_t)kTile, a.tokens - (int64_t)t * kTile);
    while (lo < hi) {  // pairs of the tile below x; of those alike (none's) the ones in tiles ahead
      const int mid = (lo + hi) >> 1;
      const uint64_t y = tile[mid];
      if (y < x || (y == x && t < mine)) lo = mid + 1;
      else hi = mid;
    }
    place += lo;
  }
  a.sorted[place] = x;
}

__device__ __forceinline__ uint32_t word_of(uint64_t pair) { return (uint32_t)(pair >> 32); }

__device__ __forceinline__ void store_sum(const EmbedBwdArgs& a, uint32_t word, int d, float (&sum)[8]) {
  const int r = shard_of(a.first, a.nranks, word);
  float* row = a.dtables[r] + ((int64_t)word - a.first[r]) * a.drow_stride[r] + d;
  Pack8<float> x;
  float v[8] = {};
  if (a.accumulate) {
    x.load(row);
    x.widen(v);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = fmaf(sum[i], a.scale, v[i]);
  x.narrow(v);
  x.store(row);
}

// Where chunk c leaves its part of a word that began ahead of it (side 0) or goes on behind it (side 1).
__device__ __forceinline__ float* part_of(const EmbedBwdArgs& a, int64_t c, int side, int d) {
  return a.parts + (c * 2 + side) * a.hidden + d;
}

template <typename T, int C>
__global__ void __launch_bounds__(256) embed_sum_kernel(const __grid_constant__ EmbedBwdArgs a) {
  constexpr int kAhead = 8;
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t c = unit / a.spans, i0 = c * C;
  const int d = (int)(unit % a.spans) * 256 + lane * 8;
  if (i0 >= a.tokens) return;
  // the chunk's pairs, a lane each, and the words next to it
  const uint64_t mine = lane < C && i0 + lane < a.tokens ? a.sorted[i0 + lane] : kNone;
  const uint32_t before = i0 > 0 ? word_of(a.sorted[i0 - 1]) : ~0u;
  const uint32_t behind = i0 + C < a.tokens ? word_of(a.sorted[i0 + C]) : ~0u;
  float sum[8] = {};
  uint32_t word = word_of(__shfl_sync(~0u, mine, 0));
  bool head = word == before;  // the present word began in a chunk ahead
  if (word == ~0u) return;
#pragma unroll
  for (int b = 0; b < C; b += kAhead) {
    Pack8<T> x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      const uint64_t p = __shfl_sync(~0u, mine, b + i);
      x[i].zero();
      if (word_of(p) != ~0u && d < a.hidden) x[i].load_stream((const T*)a.dout + (int64_t)(uint32_t)p * a.dout_stride + d);
    }
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      const uint32_t next = word_of(__shfl_sync(~0u, mine, b + i));
      if (next != word) {
        if (d < a.hidden && word != ~0u) {
          if (head) {
            Pack8<float> y;
            y.narrow(sum);
            y.store(part_of(a, c, 0, d));
          } else {
            store_sum(a, word, d, sum);
          }
        }
        head = false;
        word = next;
#pragma unroll
        for (int j = 0; j < 8; j++) sum[j] = 0.f;
      }
      float v[8];
      x[i].widen(v);
#pragma unroll
      for (int j = 0; j < 8; j++) sum[j] += v[j];
    }
  }
  if (word == ~0u || d >= a.hidden) return;
  if (head || word == behind) {
    Pack8<float> y;
    y.narrow(sum);
    y.store(part_of(a, c, head ? 0 : 1, d));
  } else {
    store_sum(a, word, d, sum);
  }
}

// The parts of each word that lies in several chunks, by the chunk in which it begins.
template <int C>
__global__ void __launch_bounds__(256) embed_join_kernel(const __grid_constant__ EmbedBwdArgs a) {
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t c = unit / a.spans, end = (c + 1) * C;
  const int d = (int)(unit % a.spans) * 256 + lane * 8;
  if (end >= a.tokens || d >= a.hidden) return;
  const uint32_t word = word_of(a.sorted[end - 1]);
  if (word == ~0u || word_of(a.sorted[end]) != word) return;
  if (word_of(a.sorted[c * C]) == word && c > 0 && word_of(a.sorted[c * C - 1]) == word) return;  // it began ahead
  float sum[8], v[8];
  Pack8<float> x;
  x.load(part_of(a, c, 1, d));
  x.widen(sum);
  for (int64_t k = c + 1; k * C < a.tokens && word_of(a.sorted[k * C]) == word; k++) {
    x.load(part_of(a, k, 0, d));
    x.widen(v);
#pragma unroll
    for (int j = 0; j < 8; j++) sum[j] += v[j];
  }
  store_sum(a, word, d, sum);
}

template <typename T, int C>
cudaError_t sums(EmbedBwdArgs& a, cudaStream_t stream) {
  void* params[] = {&a};
  const int64_t units = div_up(a.tokens, C) * a.spans;
  const dim3 grid((unsigned)div_up(units, 8));
  const cudaError_t e = launch_op((const void*)embed_sum_kernel<T, C>, grid, 256, 0, stream, params);
  if (e != cudaSuccess || a.tokens <= C) return e;
  return launch_op((const void*)embed_join_kernel<C>, grid, 256, 0, stream, params);
}

// Chunks of 32 tokens leave less to join; of 8, where they would make too few warps.
bool short_chunks(int64_t tokens, int hidden) { return div_up(tokens, 32) * div_up(hidden, 256) < 152 * 16; }

}  // namespace

int64_t embed_tokens_scratch_bytes(int64_t tokens, int hidden) {
  const int chunk = short_chunks(tokens, hidden) ? 8 : 32;
  return 2 * align_up(tokens * 8, 256) + div_up(tokens, chunk) * 2 * hidden * 4;
}

cudaError_t launch_embed_tokens(EmbedArgs& a, cudaStream_t stream) {
  const int es = a.dtype == 0 ? 4 : 2;
  a.spans = (int)div_up((int64_t)a.hidden * es, 2048);
  void* params[] = {&a};
  const void* fn = a.dtype == 0 ? (const void*)embed_kernel<float> : (const void*)embed_kernel<uint16_t>;
  return launch_op(fn, dim3((unsigned)div_up(a.tokens * a.spans, 8)), 256, 0, stream, params);
}

cudaError_t launch_embed_tokens_bwd(EmbedBwdArgs& a, cudaStream_t stream) {
  char* scratch = a.ws + kOpScratchOffset;
  a.sorted = (uint64_t*)scratch;
  a.sorted_tiles = (uint64_t*)(scratch + align_up(a.tokens * 8, 256));
  a.parts = (float*)(scratch + 2 * align_up(a.tokens * 8, 256));
  a.tiles = (int)div_up(a.tokens, kTile);
  a.spans = (int)div_up(a.hidden, 256);
  int blocks = 0;
  cudaError_t e = resident_blocks((const void*)embed_sort_kernel, kSortThreads, kTile * 8, &blocks);
  if (e != cudaSuccess) return e;
  const int zeros = a.accumulate ? 0 : (int)(a.first[a.nranks] < blocks * 16 ? div_up(a.first[a.nranks], 16) : blocks);
  if (a.tiles + zeros == 0) return cudaSuccess;
  void* params[] = {&a};
  e = launch_op((const void*)embed_sort_kernel, dim3((unsigned)(a.tiles + zeros)), kSortThreads, kTile * 8, stream, params);
  if (e != cudaSuccess || a.tokens == 0) return e;
  if (a.tiles > 1) {
    e = launch_op((const void*)embed_merge_kernel, dim3((unsigned)div_up(a.tokens, 256)), 256, 0, stream, params);
    if (e != cudaSuccess) return e;
  }
  const bool few = short_chunks(a.tokens, a.hidden);
  if (a.dtype == 0) return few ? sums<float, 8>(a, stream) : sums<float, 32>(a, stream);
  return few ? sums<uint16_t, 8>(a, stream) : sums<uint16_t, 32>(a, stream);
}

}  // namespace rar
