// embed_tokens.cu -- the embedding lookup over vocabulary shards and its gradient.
//
//   out_t = scale table[token_t]          (a word of another number gives 0)
//   dtable_w = scale sum of dout_t over the t with token_t = w, in order of t
//
// Both are bound by memory. The lookup takes a warp for 2 KiB of a row: its four
// 16-byte loads a lane are in flight at once, and a few tokens still make many warps.
// 16384 tokens of 7168 bf16 elements take 54 us, 6.2 TB/s.
//
// The gradient sums in an order that no run changes, with no atomics on values: the
// pairs (word, t) are sorted, and a warp sums a chunk of 32 (few tokens: 8) sorted
// tokens by 256 columns, its loads in flight eight at a time. A word whose tokens lie
// in one chunk is stored at once; the parts of others meet in shared memory, eight
// chunks a block, and of words of several blocks in a kernel behind, always in order.
// A pair is one 64-bit number, no two alike, so any way of sorting gives the same
// order: blocks sort tiles in shared memory (32 pairs in a warp's lanes, then runs merge by
// bisection), and if there are several, each pair's place is its place in its tile and
// its places by bisection in the others.
// Where the tables are not added to, the rows of words that do not occur are filled with
// zeros, so that every row is written once: some by blocks beside the sort and the merge,
// which leave most SMs free, and find their words in the tokens as they are; the others
// by warps of the sums' kernel, which look their words up in the sorted pairs. (Filling
// whole tables beside the sorting blocks, and rows that occur again, took 187 us where the
// warps took 170.) 16385 tokens of 4096 elements, 32008 words, take 130 us, the floor of
// the bytes 97; 300 tokens of 512 elements, with nothing sorted and in one launch, 5.8.
#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {
namespace {

constexpr int kChunks = 8;  // of a block, a warp each
constexpr int kSortThreads = 512, kMergeThreads = 512;
constexpr int kMergePairs = 24576;  // of whole tiles, in a merging block's shared memory
// Pairs of a tile: bisection in shared memory bounds its sort (8192 took 80 us), and the
// number of tiles the merge's.
constexpr int kSmallTile = 1024, kLargeTile = 4096;
constexpr int64_t kManyPairs = 65536;  // with small tiles no more than 64 of them
constexpr int kClearBlocks = 152;  // that clear rows beside others; twice as many fit beside the sort
constexpr int kFewTokens = 512;
constexpr uint64_t kNone = (uint64_t)~0u << 32;  // with the token's number: a token of no word

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

// Rows of 0 for the words from first to end that no token asks for, by block number
// `block` of `blocks`, from the tokens as they come: a block marks those of its words that
// occur, so many at a time. Warps take a row each.
__device__ __forceinline__ void clear_absent(const EmbedBwdArgs& a, int64_t first, int64_t end, int block, int blocks) {
  constexpr int kWords = 4096;
  __shared__ uint32_t occurs[kWords / 32];
  const int64_t to = first + (end - first) * (block + 1) / blocks;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int64_t from = first + (end - first) * block / blocks; from < to; from += kWords) {
    const int count = (int)min((int64_t)kWords, to - from);
    for (int i = threadIdx.x; i < kWords / 32; i += blockDim.x) occurs[i] = 0;
    __syncthreads();
    constexpr int kAhead = 16;
    for (int64_t t0 = threadIdx.x; t0 < a.tokens; t0 += kAhead * blockDim.x) {
      int32_t x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int64_t t = t0 + i * blockDim.x;
        x[i] = t < a.tokens ? a.tokens_in[t] : -1;
      }
#pragma unroll
      for (int i = 0; i < kAhead; i++) {
        const int64_t w = x[i] - from;
        if (w >= 0 && w < count) atomicOr(&occurs[w >> 5], 1u << (w & 31));
      }
    }
    __syncthreads();
    for (int w = threadIdx.x >> 5; w < count; w += warps) {
      if (occurs[w >> 5] >> (w & 31) & 1) continue;
      const int64_t word = from + w;
      const int r = shard_of(a.first, a.nranks, word);
      float4* const row = reinterpret_cast<float4*>(a.dtables[r] + (word - a.first[r]) * a.drow_stride[r]);
#pragma unroll 8
      for (int d = lane; d < a.hidden / 4; d += 32) row[d] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
  }
}

// A block sorts a tile; those behind them clear rows.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ EmbedBwdArgs a) {
  extern __shared__ uint64_t pair[];
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  if ((int)blockIdx.x >= a.tiles) {
    clear_absent(a, 0, a.clear_first, (int)blockIdx.x - a.tiles, (int)gridDim.x - a.tiles);
    return;
  }
  const int64_t at = (int64_t)blockIdx.x * a.tile;
  const int count = (int)min((int64_t)a.tile, a.tokens - at);
  // warps sort 32 pairs each, by exchanges between lanes; then runs merge two by two
  uint64_t *from = pair, *into = pair + a.tile;
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i - lane < count; i += kSortThreads) {
    const int64_t word = i < count ? a.tokens_in[at + i] : -1;
    uint64_t x = (word >= 0 && word < a.first[a.nranks] ? (uint64_t)word << 32 : kNone) | (uint64_t)(at + i);
#pragma unroll
    for (int k = 2; k <= 32; k *= 2) {
#pragma unroll
      for (int j = k / 2; j > 0; j /= 2) {
        const uint64_t y = __shfl_xor_sync(~0u, x, j);
        const bool low = (lane & j) == 0, up = (lane & k) == 0;
        if (low == up ? y < x : y > x) x = y;
      }
    }
    from[i] = x;
  }
  for (int run = 32; run < count; run *= 2) {
    __syncthreads();
    // a pair's place among both runs: its own, and by bisection how many of the other run are ahead of it
#pragma unroll 4
    for (int i = threadIdx.x; i < count; i += kSortThreads) {
      const uint64_t x = from[i];
      const int base = i & ~(2 * run - 1), other = (i & run) != 0 ? base : base + run;
      int lo = 0, hi = max(0, min(run, count - other));
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const uint64_t y = from[other + mid];
        if (y < x) lo = mid + 1;
        else hi = mid;
      }
      into[base + (i & (run - 1)) + lo] = x;
    }
    uint64_t* const t = from;
    from = into;
    into = t;
  }
  __syncthreads();
  uint64_t* to = a.tiles == 1 ? a.sorted : a.sorted_tiles;
  for (int i = threadIdx.x; i < count; i += kSortThreads) to[at + i] = from[i];
}

// Tiles to one row of pairs, a thread a pair; tokens that ask for nothing stay behind.
// Blocks behind those that merge clear rows.
// Blocks bisect in shared memory, 192 KiB of tiles at a time: in global memory, with a
// tenth of the pairs in L1 at first, 17 tiles took 36 us.
__global__ void __launch_bounds__(kMergeThreads) embed_merge_kernel(const __grid_constant__ EmbedBwdArgs a) {
  extern __shared__ uint64_t pair[];
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int blocks = (int)((a.tokens + kMergeThreads - 1) / kMergeThreads);
  if ((int)blockIdx.x >= blocks) {
    clear_absent(a, a.clear_first, a.clear_end, (int)blockIdx.x - blocks, (int)gridDim.x - blocks);
    return;
  }
  const int64_t i = (int64_t)blockIdx.x * kMergeThreads + threadIdx.x;
  const bool live = i < a.tokens;
  const uint64_t x = live ? a.sorted_tiles[i] : 0;
  const int64_t mine = i / a.tile;
  int64_t place = i - mine * a.tile;
  for (int64_t from = 0; from < a.tokens; from += kMergePairs) {
    const int count = (int)min((int64_t)kMergePairs, a.tokens - from);
    __syncthreads();
#pragma unroll 8
    for (int j = threadIdx.x; j < count; j += kMergeThreads) pair[j] = a.sorted_tiles[from + j];
    __syncthreads();
    constexpr int kAtOnce = 4;  // tiles that are searched side by side
    for (int t0 = 0; t0 < count; t0 += kAtOnce * a.tile) {
      int at[kAtOnce], end[kAtOnce], start[kAtOnce];  // the tiles' pairs below x end before `at`
#pragma unroll
      for (int k = 0; k < kAtOnce; k++) {
        start[k] = at[k] = min(t0 + k * a.tile, count);
        end[k] = (from + start[k]) / a.tile == mine ? start[k] : min(start[k] + a.tile, count);
      }
      for (int step = a.tile; step > 0; step >>= 1) {
#pragma unroll
        for (int k = 0; k < kAtOnce; k++)
          if (at[k] + step <= end[k] && pair[at[k] + step - 1] < x) at[k] += step;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; k++) place += at[k] - start[k];
    }
  }
  if (live) a.sorted[place] = x;
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

// Where block c's chunks leave their part of a word that began ahead of them (side 0) or goes on behind them (side 1).
__device__ __forceinline__ float* part_of(const EmbedBwdArgs& a, int64_t c, int side, int d) {
  return a.parts + (c * 2 + side) * a.hidden + d;
}

// The first of the sorted pairs whose word is not below `word`; a warp, 32 probes at a time.
__device__ __forceinline__ int64_t first_of(const EmbedBwdArgs& a, uint32_t word) {
  int64_t lo = 0, hi = a.tokens;  // it is in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) >> 5, probe = lo + (int64_t)(threadIdx.x & 31) * step;
    const int below = __popc(__ballot_sync(~0u, probe < hi && word_of(a.sorted[probe < hi ? probe : lo]) < word));
    if (below == 0) return lo;
    const int64_t from = lo + (int64_t)(below - 1) * step;  // the last probe below
    hi = min(hi, from + step);
    lo = from + 1;
  }
  return lo;
}

// Rows of 0 for the words from `first` on that no token asks for, at most 32; a warp.
__device__ __forceinline__ void clear_words(const EmbedBwdArgs& a, int64_t first, int count) {
  const int lane = threadIdx.x & 31;
  const int64_t mine = first + lane;
  const auto number = [](int64_t word) { return (uint32_t)min(word, (int64_t)1 << 31); };  // tokens' are below 2^31
  int64_t lo = first_of(a, number(first));
  const int64_t end = first_of(a, number(min(first + count, a.first[a.nranks])));
  bool absent = false;
  if (lane < count && mine < a.first[a.nranks]) {
    int64_t hi = end;  // the first pair of the word or a later one
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (word_of(a.sorted[mid]) < number(mine)) lo = mid + 1;
      else hi = mid;
    }
    absent = lo >= end || word_of(a.sorted[lo]) != number(mine);
  }
  for (uint32_t left = __ballot_sync(~0u, absent); left != 0; left &= left - 1) {
    const int64_t word = first + __ffs(left) - 1;
    const int r = shard_of(a.first, a.nranks, word);
    float4* const row = reinterpret_cast<float4*>(a.dtables[r] + (word - a.first[r]) * a.drow_stride[r]);
#pragma unroll 8
    for (int d = lane; d < a.hidden / 4; d += 32) row[d] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

template <typename T, int C>
__global__ void __launch_bounds__(256) embed_sum_kernel(const __grid_constant__ EmbedBwdArgs a) {
  constexpr int kAhead = 8;
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  if (blockIdx.x >= a.sum_blocks) {
    const int64_t first = a.clear_end + ((int64_t)(blockIdx.x - a.sum_blocks) * kChunks + warp) * a.clear_rows;
    if (first < a.first[a.nranks]) clear_words(a, first, a.clear_rows);
    return;
  }
  // parts of a word that began ahead of a warp's chunk, and of one that begins in it and goes on behind it; whether the
  // first is the whole chunk and goes on
  __shared__ __align__(16) float head_part[kChunks][256], tail_part[kChunks][256];
  __shared__ int goes_on[kChunks];
  const int64_t block = blockIdx.x / a.spans, c = block * kChunks + warp, i0 = c * C;
  const int d = (int)(blockIdx.x % a.spans) * 256 + lane * 8;
  // the chunk's pairs, a lane each, and the words next to it
  const uint64_t mine = lane < C && i0 + lane < a.tokens ? a.sorted[i0 + lane] : kNone;
  const uint32_t before = i0 > 0 && i0 <= a.tokens ? word_of(a.sorted[i0 - 1]) : ~0u;
  const uint32_t behind = i0 + C < a.tokens ? word_of(a.sorted[i0 + C]) : ~0u;
  float sum[8] = {};
  uint32_t word = word_of(__shfl_sync(~0u, mine, 0));
  const bool began_ahead = word != ~0u && word == before;
  bool head = began_ahead;  // the present word did
  Pack8<float> y;
#pragma unroll
  for (int b = 0; b < C; b += kAhead) {
    if (word == ~0u) break;
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
        if (word != ~0u) {
          if (head) {
            y.narrow(sum);
            y.store(&head_part[warp][lane * 8]);
          } else if (d < a.hidden) {
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
  const bool on = word != ~0u && word == behind;  // the last word goes on
  if (head || on) {
    y.narrow(sum);
    y.store(head ? &head_part[warp][lane * 8] : &tail_part[warp][lane * 8]);
  } else if (word != ~0u && d < a.hidden) {
    store_sum(a, word, d, sum);
  }
  if (lane == 0) goes_on[warp] = head && on;
  __syncthreads();
  if (d >= a.hidden) return;
  // the block's parts of a word, one after another
  const bool begins = on && !head;  // here, and goes on
  if (!begins && !(warp == 0 && began_ahead)) return;
  for (int which = 0; which < 2; which++) {
    if (which == 0 ? !(warp == 0 && began_ahead) : !begins) continue;
    float v[8];
    y.load(which == 0 ? &head_part[0][lane * 8] : &tail_part[warp][lane * 8]);
    y.widen(sum);
    int w = warp;
    bool more = which == 0 ? goes_on[0] != 0 : true;
    while (more && w + 1 < kChunks) {
      w++;
      y.load(&head_part[w][lane * 8]);
      y.widen(v);
#pragma unroll
      for (int j = 0; j < 8; j++) sum[j] += v[j];
      more = goes_on[w] != 0;
    }
    if (which == 0 || more) {
      y.narrow(sum);
      y.store(part_of(a, block, which, d));
    } else {
      store_sum(a, word, d, sum);
    }
  }
}

// The parts of each word that lies in several blocks' chunks of B tokens, by the block in which it begins.
template <int B>
__global__ void __launch_bounds__(256) embed_join_kernel(const __grid_constant__ EmbedBwdArgs a) {
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t c = unit / a.spans, end = (c + 1) * B;
  const int d = (int)(unit % a.spans) * 256 + lane * 8;
  if (end >= a.tokens) return;
  const uint32_t word = word_of(a.sorted[end - 1]), next = word_of(a.sorted[end]), first = word_of(a.sorted[c * B]),
                 ahead = c > 0 ? word_of(a.sorted[c * B - 1]) : ~0u;
  if (word == ~0u || next != word) return;
  if (first == word && ahead == word) return;  // it began ahead
  float sum[8], v[8];
  Pack8<float> x;
  x.zero();
  if (d < a.hidden) x.load(part_of(a, c, 1, d));
  x.widen(sum);
  // 32 blocks at a time: how many of them begin with the word, then their parts, eight under way
  for (int64_t k0 = c + 1;; k0 += 32) {
    const int64_t k = k0 + lane;
    const uint32_t on = __ballot_sync(~0u, k * B < a.tokens && word_of(a.sorted[k * B]) == word);
    const int count = __popc(on);
    for (int i0 = 0; i0 < count; i0 += 8) {
      Pack8<float> y[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        y[i].zero();
        if (i0 + i < count && d < a.hidden) y[i].load(part_of(a, k0 + i0 + i, 0, d));
      }
#pragma unroll
      for (int i = 0; i < 8; i++) {
        y[i].widen(v);
#pragma unroll
        for (int j = 0; j < 8; j++) sum[j] += v[j];
      }
    }
    if (count < 32) break;
  }
  if (d >= a.hidden) return;
  store_sum(a, word, d, sum);
}

// Few tokens, with nothing sorted: a block a token and 256 columns, which is over if its word
// has come before, and else finds the word's other tokens and sums their rows, eight warps
// a part of them each if there are more than eight. Blocks behind these clear rows.
template <typename T>
__global__ void __launch_bounds__(256) embed_few_kernel(const __grid_constant__ EmbedBwdArgs a) {
  __shared__ int same[kFewTokens], found[kFewTokens / 32];
  __shared__ __align__(16) float part[kChunks][256];
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  if (blockIdx.x >= a.sum_blocks) {
    clear_absent(a, 0, a.clear_end, (int)(blockIdx.x - a.sum_blocks), (int)(gridDim.x - a.sum_blocks));
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tokens = (int)a.tokens, i = (int)blockIdx.x / a.spans;
  const int d = (int)blockIdx.x % a.spans * 256 + lane * 8;
  const int32_t word = a.tokens_in[i];
  if (word < 0 || word >= a.first[a.nranks]) return;
  // warp by warp 32 tokens: which have the word
  bool before = false;
  uint32_t mine[kFewTokens / 256];
#pragma unroll
  for (int k = 0; k < kFewTokens / 256; k++) {
    const int j = k * 256 + threadIdx.x;
    const bool match = j < tokens && a.tokens_in[j] == word;
    before |= match && j < i;
    mine[k] = __ballot_sync(~0u, match);
    if (lane == 0) found[k * kChunks + warp] = __popc(mine[k]);
  }
  if (__syncthreads_or(before)) return;
  int count = 0;
#pragma unroll
  for (int k = 0; k < kFewTokens / 32; k++) {
    if (k % kChunks == warp && (mine[k / kChunks] >> lane & 1) != 0)
      same[count + __popc(mine[k / kChunks] & ((1u << lane) - 1))] = k * 32 + lane;
    count += found[k];
  }
  __syncthreads();
  const int warps = count > kChunks ? kChunks : 1;
  if (warp >= warps) return;
  const int end = count * (warp + 1) / warps;
  float sum[8] = {}, v[8];
  for (int k0 = count * warp / warps; k0 < end; k0 += 8) {
    Pack8<T> x[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      x[k].zero();
      if (k0 + k < end && d < a.hidden) x[k].load_stream((const T*)a.dout + (int64_t)same[k0 + k] * a.dout_stride + d);
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
      x[k].widen(v);
#pragma unroll
      for (int j = 0; j < 8; j++) sum[j] += v[j];
    }
  }
  if (warps > 1) {
    Pack8<float> y;
    y.narrow(sum);
    y.store(&part[warp][lane * 8]);
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < kChunks; w++) {
      y.load(&part[w][lane * 8]);
      y.widen(v);
#pragma unroll
      for (int j = 0; j < 8; j++) sum[j] += v[j];
    }
  }
  if (d < a.hidden) store_sum(a, (uint32_t)word, d, sum);
}

template <typename T, int C>
cudaError_t sums(EmbedBwdArgs& a, cudaStream_t stream) {
  void* params[] = {&a};
  constexpr int B = C * kChunks;
  const int64_t units = div_up(a.tokens, B) * a.spans;
  a.sum_blocks = units;
  // a warp's rows: 32 KiB of them, one at least
  a.clear_rows = (int)(8192 / a.hidden < 1 ? 1 : 8192 / a.hidden > 32 ? 32 : 8192 / a.hidden);
  const int64_t clears = a.accumulate ? 0 : div_up(a.first[a.nranks] - a.clear_end, (int64_t)a.clear_rows * kChunks);
  const cudaError_t e =
      launch_op((const void*)embed_sum_kernel<T, C>, dim3((unsigned)(units + clears)), 32 * kChunks, 0, stream, params);
  if (e != cudaSuccess || a.tokens <= B) return e;
  return launch_op((const void*)embed_join_kernel<B>, dim3((unsigned)div_up(units, 8)), 256, 0, stream, params);
}

// Every block of few tokens reads them all, and most rows are one block's work: at 1600 blocks
// (100 tokens of 4096 elements) 31 us where the sort takes 34, at 300 tokens of 512 elements
// 11 and 18, but at 4096 (256 of 4096) 24 and 22, at 8192 (512 of 4096) 23 and 18.
bool few_tokens(int64_t tokens, int spans) { return tokens <= kFewTokens && tokens * spans <= 152 * 16; }

// Chunks of 32 tokens leave less to join; of 8, where they would make too few warps.
constexpr int64_t kShortChunks = 152 * 16;
bool short_chunks(int64_t tokens, int hidden) { return div_up(tokens, 32) * div_up(hidden, 256) < kShortChunks; }

}  // namespace

// Enough for every call of so many tokens or fewer.
int64_t embed_tokens_scratch_bytes(int64_t tokens, int hidden) {
  const int64_t few = (int64_t)(kShortChunks - 1) / div_up(hidden, 256) * 32, blocks = div_up(tokens < few ? tokens : few, 8 * kChunks),
                more = div_up(tokens, 32 * kChunks);
  return 2 * align_up(tokens * 8, 256) + (blocks > more ? blocks : more) * 2 * hidden * 4;
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
  a.tile = a.tokens <= kManyPairs ? kSmallTile : kLargeTile;
  a.tiles = (int)div_up(a.tokens, a.tile);
  a.spans = (int)div_up(a.hidden, 256);
  if (a.accumulate && a.tokens == 0) return cudaSuccess;
  const int64_t words = a.first[a.nranks];
  // Where most words do not occur, rows to clear beside the sort, and half of them beside the
  // merge: as many as these take; the sums' kernel reads meanwhile, and is better at it
  // (16385 tokens, 32008 words of 4096 elements: none 142 us, a fifth 139, a third 133, all 154;
  // 50000 tokens, 2000 words of 1024: none 100 us, a third 104).
  a.clear_end = a.accumulate || a.tokens > kManyPairs || words <= a.tokens ? 0 : a.tiles > 1 ? words / 3 : words;
  a.clear_first = a.tiles > 1 ? a.clear_end / 2 : a.clear_end;
  auto clearing = [&](int64_t rows, int64_t most) {  // blocks, of 16 KiB or more
    const int64_t n = div_up(rows * a.hidden, 4096);
    return n < most ? n : most;
  };
  void* params[] = {&a};
  if (few_tokens(a.tokens, a.spans)) {
    a.clear_end = a.accumulate ? 0 : words;
    a.sum_blocks = a.tokens * a.spans;
    return launch_op(a.dtype == 0 ? (const void*)embed_few_kernel<float> : (const void*)embed_few_kernel<uint16_t>,
                     dim3((unsigned)(a.sum_blocks + clearing(a.clear_end, 8 * kClearBlocks))), 32 * kChunks, 0, stream, params);
  }
  int blocks = 0;
  cudaError_t e = resident_blocks((const void*)embed_sort_kernel, kSortThreads, 2 * kLargeTile * 8, &blocks);
  if (e != cudaSuccess) return e;
  e = launch_op((const void*)embed_sort_kernel, dim3((unsigned)(a.tiles + clearing(a.clear_first, 2 * kClearBlocks))), kSortThreads,
                2 * a.tile * 8, stream, params);
  if (e != cudaSuccess) return e;
  if (a.tiles > 1) {
    e = resident_blocks((const void*)embed_merge_kernel, kMergeThreads, kMergePairs * 8, &blocks);
    if (e != cudaSuccess) return e;
    const int64_t merging = div_up(a.tokens, kMergeThreads), others = merging < kClearBlocks / 2 ? merging : kClearBlocks / 2;
    e = launch_op((const void*)embed_merge_kernel,
                  dim3((unsigned)(merging + clearing(a.clear_end - a.clear_first, kClearBlocks - others))), kMergeThreads,
                  kMergePairs * 8, stream, params);
    if (e != cudaSuccess) return e;
  }
  const bool few = short_chunks(a.tokens, a.hidden);
  if (a.dtype == 0) return few ? sums<float, 8>(a, stream) : sums<float, 32>(a, stream);
  return few ? sums<uint16_t, 8>(a, stream) : sums<uint16_t, 32>(a, stream);
}

}  // namespace rar
