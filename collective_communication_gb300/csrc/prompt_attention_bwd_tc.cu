// prompt_attention_bwd_tc.cu -- the gradient of the attention over whole prompts in
// bf16 on the fifth-generation tensor cores, for head sizes up to 128 and up to 128
// query heads a key head.
//
//   P = 2^(scale log2(e) Q K^T - lse log2(e)),  dS = P (dO V^T - delta),  delta = O . dO
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two kernels that both recompute P: one by rows for dQ (three products a tile), one by
// keys for dK and dV (four); a small one ahead of them works out delta. One kernel
// with five products would have to add dQ up across blocks, in an order that changes
// from run to run, or in passes over partial sums of dQ in memory.
//
// A row is a query head of the group of a token, as in the forward kernel, so dK and
// dV of a key head are sums over the rows of a tile like any others. Tiles are 128 by
// 128; scores, dO V^T and the sums are in tensor memory (at a head size of 128 all of
// it); P and dS are rounded to bf16 (2^-8 of themselves) into the place of what they
// came from, and are left operands from there. The keys' kernel has S transposed, keys
// as rows, so that P^T and dS^T come out as left operands too.
//
// O is rounded to bf16, and its rounding goes into delta: over few keys, where O is as
// large as the values, by as much as the result's own rounding. Rows whose whole tile
// sees one tile of keys take delta from sum P (dO V^T) instead, which is at hand there.
//
// Four warpgroups work out the weights, a quarter of the columns each: a thread has 32
// columns of a row (with two, of 64 columns a thread, the two steps of a tile of keys
// took 3900 cycles of latency where its products take 2048). The products' order keeps
// the tensor cores busy meanwhile:
//   rows:  S(j+1) | dS(j) ready: dP(j+1), dQ += dS(j) K(j) | ...
//   keys:  P(i) ready: dV += P(i) dO, S(i+1) | dS(i) ready: dK += dS(i) Q, dP(i+1) | ...
// Blocks stay, one an SM, and take items (a tile of rows, or of keys) from a counter;
// a warp finds the next one while the last is under way, and its first tiles are copied.
//
// Measured: 8192 tokens of one sequence, 16 query heads on 4 key heads of 64: 542 us, 0.9 PFLOP/s of the
// seven products. What bounds it is the weights' chain, from scores through two roundings to the last
// product, as long for half the products of a head size of 128: tensor cores 36 % of the time, issue
// slots 37 to 48 %. Keys have two buffers of scores there, so that the next tile's are ready when the
// weights are done with this one (one buffer, as tensor memory allows at 128: 561 us, 536 with two, before
// warps decided together whether a wait had run out, which costs 2 %).
// 4097 tokens of 9 sequences, 32 query heads on 8 key heads of 128: 151 us, 16 of them
// delta (cold; out and dout from memory); the keys that most rows see are 27 tiles of rows
// where an SM has 20 on average. Queries of the next item ahead in a buffer of their own,
// for fewer tiles of keys and values, took as long, and 800 us for 715 (8192
// tokens, 16 query heads on 2 key heads of 128; 727 now).
#include <type_traits>

#include "prompt_attention.cuh"
#include "rar_launch.h"
#include "tensor_core.cuh"

namespace rar {
namespace {

using namespace tc;

constexpr int kWeightWarps = 16, kThreads = 32 * (kWeightWarps + 4);
constexpr int kTile = 128;   // rows, and keys
constexpr int kColumns = 32;  // of a thread
constexpr int kCopyWarp = kWeightWarps, kProductWarp = kCopyWarp + 1, kItemWarp = kCopyWarp + 2, kNumbersWarp = kCopyWarp + 3;
constexpr int kItemSlots = 2;
constexpr int kNextItem = kOpCounters - 1, kDoneBlocks = kOpCounters - 2;  // counters of the workspace
constexpr float kLog2e = 1.4426950408889634f;

struct Maps {
  CUtensorMap q[kMaxRanks], k[kMaxRanks], v[kMaxRanks], dout[kMaxRanks];
};

template <int DP>
struct Layout {
  static constexpr int kSlab = kTile * 128;
  static constexpr int kBytes = kSlab * (DP / 64);  // a tile of bf16 rows
  static constexpr int kKeyStages = DP == 64 ? 4 : 3, kValueStages = DP == 64 ? 4 : 2;  // of the rows' kernel
  static constexpr int kRowStages = DP == 64 ? 4 : 2;                                  // of the keys' kernel: Q and dO
  static constexpr int kRowsShared = (2 + kKeyStages + kValueStages) * kBytes + 1024;
  static constexpr int kKeysShared = (2 + 2 * kRowStages) * kBytes + 1024;
};

struct Item {
  int there;             // 0: no more
  int rank, head;        // key head
  int sequence, length;  // the sequence's first token in the step, and its tokens
  int from, count;       // first token or key of the item in the sequence, and how many
  int part;
};

// Numbers of items, in tiles of `unit` tokens, and what their rows are split into.
struct Work {
  int64_t slots;
  int unit;
  KeyParts split;
};

// Item number n in order; 0 if there is none, -1 if there are no more (a whole warp).
__device__ __forceinline__ int find_item(const PromptBwdArgs& a, const Work& work, ItemOrder& order, bool ordered, bool by_keys,
                                         uint32_t n, Item* item) {
  const uint32_t lanes = (uint32_t)(a.kv_heads * a.nranks), parts = (uint32_t)work.split.parts, whole = n / parts, slot = whole / lanes;
  const int lane_of = (int)(whole - slot * lanes);
  item->part = (int)(n - whole * parts);
  item->head = lane_of % a.kv_heads;
  item->rank = lane_of / a.kv_heads;
  PromptSequence seq;
  int tile;
  if (ordered) {
    if (!order.advance(slot, work.unit, by_keys, &seq.index, &tile)) return -1;
    seq.first = __shfl_sync(~0u, order.first, seq.index);
    seq.length = __shfl_sync(~0u, order.length, seq.index);
  } else if (!find_sequence(a.starts, a.sequences, a.tokens, 1, work.unit, by_keys ? slot : work.slots - 1 - slot, &seq, &tile)) {
    return 0;
  }
  item->sequence = seq.first;
  item->length = seq.length;
  item->from = tile * work.unit;
  item->count = min(work.unit, seq.length - item->from);
  item->there = 1;
  return 1;
}

// The warp that finds items for the others, from those with the most work on: rows that
// see many keys, or keys that many rows see.
__device__ __forceinline__ void serve_items(const PromptBwdArgs& a, const Work& work, bool by_keys, uint32_t magic,
                                            Item* items, uint64_t* full, uint64_t* empty, volatile Limit* limit) {
  const int lane = threadIdx.x & 31;
  uint32_t* const counters = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes);
  const uint32_t all = (uint32_t)(work.slots * work.split.parts * a.kv_heads * a.nranks);
  ItemOrder order;
  const bool ordered = order.begin(a.starts, a.sequences, a.tokens, work.unit);
  // without a workspace there are no items: the others wait for the first one, not for the header
  const bool ready = magic == kOpMagic;
  if (!ready && lane == 0) op_report(a.ws, kErrWorkspace);
  uint32_t n = ready ? blockIdx.x : all;
  for (int i = 0;;) {
    Item item;
    const int found = n < all ? find_item(a, work, order, ordered, by_keys, n, &item) : -1;
    if (found < 0) item.there = 0;
    if (found != 0) {
      if (!wait_warp(&empty[i % kItemSlots], (i / kItemSlots & 1) ^ 1, limit)) break;
      if (lane == 0) {
        items[i % kItemSlots] = item;
        arrive(&full[i % kItemSlots]);
      }
      i++;
    }
    if (found < 0) break;
    uint32_t next = 0;
    if (lane == 0) next = atomicAdd(&counters[kNextItem], 1);
    n = gridDim.x + __shfl_sync(~0u, next, 0);
  }
  // the last block to have no more sets the counters back
  if (ready && lane == 0 && atom_add_acq_rel_u32(&counters[kDoneBlocks], 1) == gridDim.x - 1) {
    counters[kNextItem] = 0;
    counters[kDoneBlocks] = 0;
  }
}

// What another warp reads of item i; false at the end.
struct Taken {
  int rank, head, sequence, length, from, count, part;
};
__device__ __forceinline__ bool take_item(int i, const Item* items, uint64_t* full, uint64_t* empty, volatile Limit* limit, Taken* t) {
  if (!wait_warp(&full[i % kItemSlots], i / kItemSlots & 1, limit)) return false;
  const Item& item = items[i % kItemSlots];
  const int there = uniform(item.there);
  if (there) {
    t->rank = uniform(item.rank);
    t->head = uniform(item.head);
    t->sequence = uniform(item.sequence);
    t->length = uniform(item.length);
    t->from = uniform(item.from);
    t->count = uniform(item.count);
    t->part = uniform(item.part);
  }
  __syncwarp();
  if (there && (threadIdx.x & 31) == 0) arrive(&empty[i % kItemSlots]);
  return there != 0;
}

// Rows from `first` on of a tile in shared memory become 0, before products run over them; one warp.
template <int DP>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int first) {
  for (int r = first * 8 + (threadIdx.x & 31); r < kTile * 8; r += 32)
    for (int h = 0; h < DP / 64; h++) *reinterpret_cast<uint4*>(tile + h * Layout<DP>::kSlab + r * 16) = make_uint4(0, 0, 0, 0);
}

// Sums of a row from tensor memory: the slice's quarter of its elements.
template <int DP>
struct Quarter {
  uint32_t o[DP / 4];
  __device__ __forceinline__ void load(uint32_t at, int slice) {
    if (DP == 128) tmem_load32(at + slice * 32, o);
    else tmem_load16(at + slice * 16, o);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < DP / 4; i++) o[i] = 0;
  }
  __device__ __forceinline__ void store_part(float* row, int slice, float by, int D) const {
#pragma unroll
    for (int i = 0; i < DP / 4; i += 4) {
      const int d = slice * (DP / 4) + i;
      if (d < D)
        store4(row + d, __uint_as_float(o[i]) * by, __uint_as_float(o[i + 1]) * by, __uint_as_float(o[i + 2]) * by,
               __uint_as_float(o[i + 3]) * by);
    }
  }
  __device__ __forceinline__ void store(uint16_t* row, int slice, float by, int D) const {
#pragma unroll
    for (int i = 0; i < DP / 4; i += 8) {
      const int d = slice * (DP / 4) + i;
      if (d >= D) continue;
      Pack8<uint16_t> x;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] = __uint_as_float(o[i + k]) * by;
      x.narrow(v);
      x.store(row + d);
    }
  }
};

// One arrival of the warp, after its lanes' stores to tensor memory.
__device__ __forceinline__ void arrive_warp(uint64_t* b) {
  stores_done();
  fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(b);
}

__device__ __forceinline__ void end_block(char* ws, volatile Limit* limit, int warp) {
  __syncwarp();
  fence_before();
  __syncthreads();
  if (limit->dead) {
    // a wait ran out: copies and products that are still under way have ended by the time this has passed
    const uint64_t until = global_timer_ns() + 10000000ull;
    while (global_timer_ns() < until) {}
    if (threadIdx.x == 0) op_report(ws, kErrTimeout);
  }
  __syncthreads();
  if (warp == kCopyWarp) {
    fence_after();
    tmem_free(0, 512);
  }
}

__device__ __forceinline__ float* deltas_of(const PromptBwdArgs& a, int rank) {
  return reinterpret_cast<float*>(a.ws + kOpScratchOffset) + (int64_t)rank * a.tokens * a.q_heads;
}

// delta of every row: DP / 8 lanes a row, 16 bytes a lane of each tensor.
template <int DP>
__global__ void __launch_bounds__(256) prompt_delta_kernel(const __grid_constant__ PromptBwdArgs a) {
  constexpr int kLanes = DP / 8, kAtOnce = 32 / kLanes, kUnroll = 4;
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int lane = threadIdx.x & 31, rank = blockIdx.y, d = lane % kLanes * 8, D = a.head_dim;
  const int rows = a.tokens * a.q_heads;
  const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * (kAtOnce * kUnroll) + lane / kLanes;
  Pack8<uint16_t> x[kUnroll], y[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; i++) {
    const int64_t r = first + i * kAtOnce;
    x[i].zero();
    y[i].zero();
    if (r < rows && d < D) {
      const int64_t token = r / a.q_heads, head = r % a.q_heads;
      x[i].load_stream((const uint16_t*)a.out[rank] + token * a.out_stride + head * a.out_head + d);
      y[i].load_stream((const uint16_t*)a.dout[rank] + token * a.dout_stride + head * a.dout_head + d);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; i++) {
    float u[8], v[8], sum = 0.f;
    x[i].widen(u);
    y[i].widen(v);
#pragma unroll
    for (int k = 0; k < 8; k++) sum = fmaf(u[k], v[k], sum);
#pragma unroll
    for (int k = 1; k < kLanes; k *= 2) sum += __shfl_xor_sync(~0u, sum, k);
    const int64_t r = first + i * kAtOnce;
    if (d == 0 && r < rows) deltas_of(a, rank)[r] = sum;
  }
}

// Products with P and dS may take what their roundings leave as well, which lies behind them. The roundings are as large as
// the result's, and stay so over any number of keys: dq is off by 2.4e-3 of its norm in long sequences, by 2.8e-3 in one of 2
// tokens, where its own rounding is 1.66e-3. With the rests that is all there is, but for another three products
// of seven: 148 -> 178 us for 4097 packed tokens of 128 elements, 550 -> 694 for 8192 of 64. Those have them that are a small
// part of such a call, and whose products are over before anything else is in a call of their own (1.5 to 3.5 us of 18 to
// 33): dq of rows that see one tile of keys, dk and dv of sequences of one. What a sequence gets depends on
// its own length alone, not on what it is packed with.
template <int DP>
__global__ void __launch_bounds__(kThreads, 1) prompt_rows_tc_kernel(const __grid_constant__ PromptBwdArgs a,
                                                                     const __grid_constant__ Maps maps,
                                                                     const __grid_constant__ Work work) {
  using L = Layout<DP>;
  constexpr int KS = L::kKeyStages, VS = L::kValueStages;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (shared_address(raw) & 1023));
  __shared__ uint64_t q_full, q_empty, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], dp_full, ds_ready, dq_full, dq_free,
      sums_half, sums_full,
      item_full[kItemSlots], item_empty[kItemSlots];
  __shared__ Item items[kItemSlots];
  __shared__ uint32_t tmem_at;
  __shared__ Limit limit_at;
  volatile Limit* const limit = &limit_at;
  __shared__ float sums[2][kTile];
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    limit->dead = 0;
    limit->ns = a.wait_ns;
    barrier_init(&q_full, 1);
    barrier_init(&q_empty, 1);
    for (int i = 0; i < KS; i++) {
      barrier_init(&k_full[i], 1);
      barrier_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; i++) {
      barrier_init(&v_full[i], 1);
      barrier_init(&v_empty[i], 1);
    }
    barrier_init(&dp_full, 1);
    barrier_init(&ds_ready, kWeightWarps);
    barrier_init(&dq_full, 1);
    barrier_init(&dq_free, kWeightWarps);
    barrier_init(&sums_half, kWeightWarps / 2);
    barrier_init(&sums_full, kWeightWarps / 2);
    for (int i = 0; i < kItemSlots; i++) {
      barrier_init(&item_full[i], 1);
      barrier_init(&item_empty[i], kWeightWarps + 2);
    }
    barriers_ready();
  }
  const uint32_t magic = op_start(a.ws);
  if (warp == kCopyWarp) tmem_alloc(&tmem_at, 512);
  __syncthreads();
  constexpr uint32_t s_at = 0, dp_at = 256, dq_at = 384;  // all of tensor memory, from 0 on; S: two buffers of 128 columns
  uint8_t *const q_tile = smem, *const g_tile = smem + L::kBytes, *const k_ring = smem + 2 * L::kBytes,
          *const v_ring = k_ring + KS * L::kBytes;
  const int group = a.q_heads / a.kv_heads, D = a.head_dim, per_tile = kTile / group, steps = (D + 15) / 16;

  if (warp == kItemWarp) {
    serve_items(a, work, false, magic, items, item_full, item_empty, limit);
  } else if (warp == kNumbersWarp) {
    if (blockIdx.x == 0) check_starts(a.starts, a.sequences, a.tokens, a.ws, lane, 32);
  } else if (warp == kCopyWarp) {
    int n = 0;  // tiles of keys so far
    for (int i = 0;; i++) {
      Taken t;
      if (!take_item(i, items, item_full, item_empty, limit, &t)) break;
      const int tiles = (t.from + t.count + kTile - 1) / kTile;
      bool fine = true;
      for (int j = 0; j < tiles && fine; j++, n++) {
        const int k = n % KS, v = n % VS;
        if (!(fine = wait_warp(&k_empty[k], (n / KS & 1) ^ 1, limit))) break;
        if (lane == 0) {
          arrive_expect(&k_full[k], L::kBytes);
          for (int h = 0; h < DP / 64; h++)
            copy_3d(k_ring + k * L::kBytes + h * L::kSlab, &maps.k[t.rank], h * 64, t.head, t.sequence + j * kTile, &k_full[k]);
        }
        if (!(fine = wait_warp(&v_empty[v], (n / VS & 1) ^ 1, limit))) break;
        if (lane == 0) {
          arrive_expect(&v_full[v], L::kBytes);
          for (int h = 0; h < DP / 64; h++)
            copy_3d(v_ring + v * L::kBytes + h * L::kSlab, &maps.v[t.rank], h * 64, t.head, t.sequence + j * kTile, &v_full[v]);
        }
        if (j == 0) {
          if (!(fine = wait_warp(&q_empty, (i & 1) ^ 1, limit))) break;
          if (lane == 0) {
            arrive_expect(&q_full, (uint32_t)(2 * per_tile * group * 128 * (DP / 64)));
            for (int h = 0; h < DP / 64; h++) {
              copy_3d(q_tile + h * L::kSlab, &maps.q[t.rank], h * 64, t.head * group, t.sequence + t.from, &q_full);
              copy_3d(g_tile + h * L::kSlab, &maps.dout[t.rank], h * 64, t.head * group, t.sequence + t.from, &q_full);
            }
          }
        }
      }
      if (!fine) break;
    }
  } else if (warp == kProductWarp) {
    const uint32_t q_at = shared_address(q_tile), g_at = shared_address(g_tile), k_at = shared_address(k_ring),
                   v_at = shared_address(v_ring);
    const uint32_t lead = elect_one();
    int base = 0;  // tiles of keys of the items before
    for (int i = 0;; i++) {
      Taken t;
      if (!take_item(i, items, item_full, item_empty, limit, &t)) break;
      const int tiles = (t.from + t.count + kTile - 1) / kTile;
      auto score = [&](int j) {  // S of key tile j; keys that are none are 0, for the product with dS
        const int n = base + j, stage = n % KS;
        if (!wait_warp(&k_full[stage], n / KS & 1, limit)) return false;
        if (t.length - j * kTile < kTile) {
          clear_rows<DP>(k_ring + stage * L::kBytes, t.length - j * kTile);
          stores_to_products();
          __syncwarp();
        }
        fence_after();
        rows_by_rows<DP / 16, L::kSlab>(lead, s_at + (n & 1) * 128, q_at, k_at + stage * L::kBytes, kTile, steps);
        return true;
      };
      auto value = [&](int j) {  // dO V^T
        const int n = base + j, stage = n % VS;
        if (!wait_warp(&v_full[stage], n / VS & 1, limit)) return false;
        fence_after();
        rows_by_rows<DP / 16, L::kSlab>(lead, dp_at, g_at, v_at + stage * L::kBytes, kTile, steps);
        commit(lead, &dp_full);
        commit(lead, &v_empty[stage]);
        if (j + 1 == tiles) commit(lead, &q_empty);
        return true;
      };
      bool fine = wait_warp(&q_full, i & 1, limit) && score(0) && value(0);
      for (int j = 0; j < tiles && fine; j++) {
        const int n = base + j;
        const bool more = j + 1 < tiles;
        if (more && !(fine = score(j + 1))) break;
        if (j == 0 && i > 0 && !(fine = wait_warp(&dq_free, (i - 1) & 1, limit))) break;  // dQ of the item before has been read
        if (!(fine = wait_warp(&ds_ready, n & 1, limit))) break;
        fence_after();
        if (more && !(fine = value(j + 1))) break;
        weights_by_rows<2, kColumns>(lead, dq_at, s_at + (n & 1) * 128, k_at + n % KS * L::kBytes, steps * 16, j > 0, L::kSlab);
        if (tiles == 1)
          weights_by_rows<2, kColumns>(lead, dq_at, s_at + (n & 1) * 128 + kColumns / 2, k_at + n % KS * L::kBytes, steps * 16, true, L::kSlab);
        commit(lead, &k_empty[n % KS]);
        if (!more) commit(lead, &dq_full);
      }
      if (!fine) break;
      base += tiles;
    }
  } else if (warp < kWeightWarps) {
    const int slice = warp >> 2;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
    const int row = threadIdx.x & 127, token = row / group, in_group = row % group;
    const float scale2 = a.scale * kLog2e;
    int n = 0, summed = 0;  // tiles of keys, and items whose rows see one, so far
    for (int i = 0;; i++) {
      Taken t;
      if (!take_item(i, items, item_full, item_empty, limit, &t) || (a.fault == kFaultWeights && warp == 0)) break;
      const int tiles = (t.from + t.count + kTile - 1) / kTile, query = t.head * group + in_group;
      const bool mine = token < t.count;
      const int64_t at_token = (int64_t)t.sequence + t.from + token, at = at_token * a.q_heads + query;
      float lse2 = 0.f, delta = 0.f;
      if (mine) {
        lse2 = a.lse[t.rank][at] * kLog2e;
        delta = deltas_of(a, t.rank)[at];
      }
      const int sees = t.from + (mine ? token : 0) + 1;
      const int least = __reduce_min_sync(~0u, sees);
      const F2 scale_pair = f2(scale2, scale2), lse_pair = f2(-lse2, -lse2);
      // the score gradients of key tile j; ONE: it is all that the rows see
      auto work_out = [&](auto one, int j) {
        constexpr bool ONE = decltype(one)::value;
        if (!wait(&dp_full, n & 1, limit)) return false;  // S of the tile was issued ahead of it
        fence_after();
        const uint32_t from = s_at + (n & 1) * 128 + quarter + slice * kColumns;
        uint32_t s[kColumns], dp[kColumns];
        tmem_load32(from, s);
        tmem_load32(dp_at + quarter + slice * kColumns, dp);
        loads_done();
        const int upto = sees - j * kTile - slice * kColumns;
        const bool cut = (j + 1) * kTile > least;
#pragma unroll
        for (int c = 0; c < kColumns; c += 2) {
          float2 p = unpack(fma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale_pair, lse_pair));
          s[c] = __float_as_uint(exp2_fast(p.x));
          s[c + 1] = __float_as_uint(exp2_fast(p.y));
        }
        if (cut) {
#pragma unroll
          for (int c = 0; c < kColumns; c++) {
            if (c >= upto) s[c] = dp[c] = 0;
          }
          // the one score of a row that sees one key has no gradient, whatever roundings leave of dp - delta; NaN stays
          if (sees == 1) s[0] = __float_as_uint(__uint_as_float(s[0]) * 0.f);
        }
        if (ONE) {
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < kColumns; c++) sum = fmaf(__uint_as_float(s[c]), __uint_as_float(dp[c]), sum);
          // slices 2 and 3 hand theirs to 0 and 1, and those the two sums to all; the next item's come after dQ of this one,
          // for which all warps have to be through here
          if (slice >= 2) {
            sums[slice - 2][row] = sum;
            __syncwarp();
            if (lane == 0) arrive(&sums_half);
          } else {
            if (!wait(&sums_half, summed & 1, limit)) return false;
            sums[slice][row] += sum;
            __syncwarp();
            if (lane == 0) arrive(&sums_full);
          }
          if (!wait(&sums_full, summed & 1, limit)) return false;
          summed++;
          delta = sums[0][row] + sums[1][row];
          if (mine && slice == 0) deltas_of(a, t.rank)[at] = delta;
        }
        const F2 delta_pair = f2(-delta, -delta);
#pragma unroll
        for (int c = 0; c < kColumns; c += 2) {
          const F2 d = add2(f2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])), delta_pair);
          const float2 ds = unpack(mul2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), d));
          if (ONE) dp[c] = __float_as_uint(ds.x), dp[c + 1] = __float_as_uint(ds.y);
          s[c / 2] = bf16_pair(ds.x, ds.y);
        }
        tmem_store16(from, s);
        if (ONE) {
#pragma unroll
          for (int c = 0; c < kColumns; c += 2) s[c / 2] = bf16_rest(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1]), s[c / 2]);
          tmem_store16(from + kColumns / 2, s);
        }
        arrive_warp(&ds_ready);
        n++;
        return true;
      };
      bool fine = true;
      if (tiles == 1) fine = work_out(std::true_type{}, 0);
      else
        for (int j = 0; j < tiles && fine; j++) fine = work_out(std::false_type{}, j);
      if (!fine || !wait(&dq_full, i & 1, limit)) break;
      fence_after();
      Quarter<DP> o;
      o.load(dq_at + quarter, slice);
      loads_done();
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(&dq_free);
      if (mine) o.store((uint16_t*)a.dq[t.rank] + at_token * a.dq_stride + query * a.dq_head, slice, a.scale, D);
    }
  }
  end_block(a.ws, limit, warp);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) prompt_keys_tc_kernel(const __grid_constant__ PromptBwdArgs a,
                                                                     const __grid_constant__ Maps maps,
                                                                     const __grid_constant__ Work work) {
  using L = Layout<DP>;
  constexpr int NS = L::kRowStages, SB = DP == 64 ? 2 : 1;  // SB: buffers of scores, what tensor memory has room for
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (shared_address(raw) & 1023));
  __shared__ uint64_t kv_full, kv_empty, full[NS], empty[NS], s_full[SB], p_ready[SB], dp_full, ds_ready, sums_full, sums_free,
      item_full[kItemSlots], item_empty[kItemSlots];
  __shared__ Item items[kItemSlots];
  __shared__ uint32_t tmem_at;
  __shared__ Limit limit_at;
  volatile Limit* const limit = &limit_at;
  __shared__ __align__(16) float numbers[NS][2][kTile];  // -lse log2(e) and -delta of a tile's rows
  __shared__ uint8_t token_of[kTile];
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int group = a.q_heads / a.kv_heads;
  if (threadIdx.x == 0) {
    limit->dead = 0;
    limit->ns = a.wait_ns;
    barrier_init(&kv_full, 1);
    barrier_init(&kv_empty, 1);
    for (int i = 0; i < NS; i++) {
      barrier_init(&full[i], 2);
      barrier_init(&empty[i], 1 + kWeightWarps);
    }
    // of each buffer: a warp may be through with the next tile's scores while another has not read these
    for (int i = 0; i < SB; i++) {
      barrier_init(&s_full[i], 1);
      barrier_init(&p_ready[i], kWeightWarps);
    }
    barrier_init(&dp_full, 1);
    barrier_init(&ds_ready, kWeightWarps);
    barrier_init(&sums_full, 1);
    barrier_init(&sums_free, kWeightWarps);
    for (int i = 0; i < kItemSlots; i++) {
      barrier_init(&item_full[i], 1);
      barrier_init(&item_empty[i], kWeightWarps + 3);
    }
    barriers_ready();
  }
  if (threadIdx.x < kTile) token_of[threadIdx.x] = (uint8_t)(threadIdx.x / group);
  const uint32_t magic = op_start(a.ws);
  if (warp == kCopyWarp) tmem_alloc(&tmem_at, 512);
  __syncthreads();
  constexpr uint32_t s_at = 0, dp_at = SB * 128, dv_at = dp_at + 128, dk_at = dv_at + DP;  // all of tensor memory, from 0 on
  uint8_t *const k_tile = smem, *const v_tile = smem + L::kBytes, *const ring = smem + 2 * L::kBytes;  // a stage: Q, dO
  const int D = a.head_dim, per_tile = kTile / group, steps = (D + 15) / 16;
  // tiles of rows, of all that see the item's keys the part's
  auto tile_of = [&](const Taken& t, int part) {
    const int first = t.from / per_tile, count = (t.length + per_tile - 1) / per_tile - first;
    return first + (int)((int64_t)count * part / work.split.parts);
  };
  auto first_tile = [&](const Taken& t) { return tile_of(t, t.part); };
  auto last_tile = [&](const Taken& t) { return tile_of(t, t.part + 1); };
  auto rests_of = [&](const Taken& t) { return t.length <= kTile; };

  if (warp == kItemWarp) {
    serve_items(a, work, true, magic, items, item_full, item_empty, limit);
  } else if (warp == kCopyWarp) {
    int n = 0, some = 0;  // tiles of rows, and items that have some, so far
    for (int i = 0;; i++) {
      Taken t;
      if (!take_item(i, items, item_full, item_empty, limit, &t)) break;
      const int begin = first_tile(t), end = last_tile(t);
      bool fine = true;
      for (int x = begin; x < end && fine; x++, n++) {
        const int stage = n % NS;
        if (!(fine = wait_warp(&empty[stage], (n / NS & 1) ^ 1, limit))) break;
        if (lane == 0) {
          arrive_expect(&full[stage], (uint32_t)(2 * per_tile * group * 128 * (DP / 64)));
          for (int h = 0; h < DP / 64; h++) {
            copy_3d(ring + stage * 2 * L::kBytes + h * L::kSlab, &maps.q[t.rank], h * 64, t.head * group,
                    t.sequence + x * per_tile, &full[stage]);
            copy_3d(ring + (stage * 2 + 1) * L::kBytes + h * L::kSlab, &maps.dout[t.rank], h * 64, t.head * group,
                    t.sequence + x * per_tile, &full[stage]);
          }
        }
        if (x == begin) {
          if (!(fine = wait_warp(&kv_empty, (some & 1) ^ 1, limit))) break;
          if (lane == 0) {
            arrive_expect(&kv_full, 2 * L::kBytes);
            for (int h = 0; h < DP / 64; h++) {
              copy_3d(k_tile + h * L::kSlab, &maps.k[t.rank], h * 64, t.head, t.sequence + t.from, &kv_full);
              copy_3d(v_tile + h * L::kSlab, &maps.v[t.rank], h * 64, t.head, t.sequence + t.from, &kv_full);
            }
          }
        }
      }
      if (!fine) break;
      some += begin < end;
    }
  } else if (warp == kNumbersWarp) {
    int n = 0;
    for (int i = 0;; i++) {
      Taken t;
      if (!take_item(i, items, item_full, item_empty, limit, &t)) break;
      const int begin = first_tile(t), end = last_tile(t);
      const float *const lse = a.lse[t.rank], *const deltas = deltas_of(a, t.rank);
      float l[4], d[4];
      auto read = [&](int x) {  // a tile ahead
#pragma unroll
        for (int y = 0; y < 4; y++) {
          const int r = lane + 32 * y, token = x * per_tile + token_of[r];
          const bool there = token_of[r] < per_tile && token < t.length && x < end;
          const int64_t at = ((int64_t)t.sequence + token) * a.q_heads + t.head * group + r - token_of[r] * group;
          l[y] = there ? lse[at] * -kLog2e : 0.f;
          d[y] = there ? -deltas[at] : 0.f;
        }
      };
      read(begin);
      bool fine = true;
      for (int x = begin; x < end; x++, n++) {
        const int stage = n % NS;
        if (!(fine = wait_warp(&empty[stage], (n / NS & 1) ^ 1, limit))) break;
#pragma unroll
        for (int y = 0; y < 4; y++) {
          numbers[stage][0][lane + 32 * y] = l[y];
          numbers[stage][1][lane + 32 * y] = d[y];
        }
        __syncwarp();
        if (lane == 0) arrive(&full[stage]);
        read(x + 1);
      }
      if (!fine) break;
    }
  } else if (warp == kProductWarp) {
    const uint32_t k_at = shared_address(k_tile), v_at = shared_address(v_tile), ring_at = shared_address(ring);
    const uint32_t lead = elect_one();
    int base = 0, some = 0;  // tiles of rows, and items that have some, so far
    for (int i = 0;; i++) {
      Taken t;
      if (!take_item(i, items, item_full, item_empty, limit, &t)) break;
      const int begin = first_tile(t), end = last_tile(t);
      const bool rests = rests_of(t);
      if (begin == end) continue;
      auto score = [&](int x) {  // S^T of a tile of rows; rows that are none are 0, for the products with P and dS
        const int n = base + x - begin, stage = n % NS;
        if (!wait_warp(&full[stage], n / NS & 1, limit)) return false;
        const int rows = min(per_tile, t.length - x * per_tile) * group;
        if (rows < kTile) {
          clear_rows<DP>(ring + stage * 2 * L::kBytes, rows);
          clear_rows<DP>(ring + (stage * 2 + 1) * L::kBytes, rows);
          stores_to_products();
          __syncwarp();
        }
        fence_after();
        rows_by_rows<DP / 16, L::kSlab>(lead, s_at + n % SB * 128, k_at, ring_at + stage * 2 * L::kBytes, kTile, steps);
        commit(lead, &s_full[n % SB]);
        return true;
      };
      auto value = [&](int x) {  // V dO^T
        rows_by_rows<DP / 16, L::kSlab>(lead, dp_at, v_at, ring_at + ((base + x - begin) % NS * 2 + 1) * L::kBytes, kTile, steps);
        commit(lead, &dp_full);
        if (x + 1 == end) commit(lead, &kv_empty);
      };
      bool fine = wait_warp(&kv_full, some & 1, limit) && score(begin);
      if (!fine) break;
      value(begin);
      if (SB > 1 && begin + 1 < end && !score(begin + 1)) break;
      // sums of the item before have been read
      if (some > 0 && !wait_warp(&sums_free, (some - 1) & 1, limit)) break;
      for (int x = begin; x < end; x++) {
        const int n = base + x - begin, stage = n % NS;
        const bool more = x + 1 < end;
        if (!(fine = wait_warp(&p_ready[n % SB], n / SB & 1, limit))) break;
        fence_after();
        weights_by_rows<2, kColumns>(lead, dv_at, s_at + n % SB * 128, ring_at + (stage * 2 + 1) * L::kBytes, steps * 16, x > begin, L::kSlab);
        if (rests)
          weights_by_rows<2, kColumns>(lead, dv_at, s_at + n % SB * 128 + kColumns / 2, ring_at + (stage * 2 + 1) * L::kBytes, steps * 16, true,
                                       L::kSlab);
        if (x + SB < end && !(fine = score(x + SB))) break;
        if (!(fine = wait_warp(&ds_ready, n & 1, limit))) break;
        fence_after();
        weights_by_rows<2, kColumns>(lead, dk_at, dp_at, ring_at + stage * 2 * L::kBytes, steps * 16, x > begin, L::kSlab);
        if (rests)
          weights_by_rows<2, kColumns>(lead, dk_at, dp_at + kColumns / 2, ring_at + stage * 2 * L::kBytes, steps * 16, true, L::kSlab);
        commit(lead, &empty[stage]);
        if (!more) commit(lead, &sums_full);
        if (more) value(x + 1);
      }
      if (!fine) break;
      base += end - begin;
      some++;
    }
  } else if (warp < kWeightWarps) {
    const int slice = warp >> 2, c0 = slice * kColumns;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;
    const int row = threadIdx.x & 127;
    const F2 scale_pair = f2(a.scale * kLog2e, a.scale * kLog2e);
    int n = 0, some = 0;
    for (int i = 0;; i++) {
      Taken t;
      if (!take_item(i, items, item_full, item_empty, limit, &t) || (a.fault == kFaultWeights && warp == 0)) break;
      const int begin = first_tile(t), end = last_tile(t), key = t.from + row;
      // weights and score gradients of a tile of rows
      auto work_out = [&](auto with_rests, int x) {
        constexpr bool RESTS = decltype(with_rests)::value;
        const int stage = n % NS;
        // the rows' numbers, and their scores
        if (!wait(&full[stage], n / NS & 1, limit)) return false;
        if (!wait(&s_full[n % SB], n / SB & 1, limit)) return false;
        fence_after();
        const uint32_t from = s_at + n % SB * 128 + quarter + c0, dp_from = dp_at + quarter + c0;
        uint32_t s[kColumns], w[kColumns / 2];
        tmem_load32(from, s);
        loads_done();
        const int rows = min(per_tile, t.length - x * per_tile) * group;
        const bool cut = rows < kTile || x * per_tile < t.from + kTile - 1;
        const float4* l = reinterpret_cast<const float4*>(numbers[stage][0] + c0);
        const float4* d = reinterpret_cast<const float4*>(numbers[stage][1] + c0);
#pragma unroll
        for (int c = 0; c < kColumns; c += 4) {
          const float4 y = l[c / 4];
          const float2 p = unpack(fma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale_pair, f2(y.x, y.y)));
          const float2 q = unpack(fma2(f2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), scale_pair, f2(y.z, y.w)));
          s[c] = __float_as_uint(exp2_fast(p.x));
          s[c + 1] = __float_as_uint(exp2_fast(p.y));
          s[c + 2] = __float_as_uint(exp2_fast(q.x));
          s[c + 3] = __float_as_uint(exp2_fast(q.y));
        }
        if (cut) {
          const int before = key - x * per_tile;  // tokens of the tile ahead of the key
#pragma unroll
          for (int c = 0; c < kColumns; c++)
            if (c0 + c >= rows || (int)token_of[c0 + c] < before) s[c] = 0;
        }
#pragma unroll
        for (int c = 0; c < kColumns; c += 2) w[c / 2] = bf16_pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        tmem_store16(from, w);
        if (RESTS) {
#pragma unroll
          for (int c = 0; c < kColumns; c += 2) w[c / 2] = bf16_rest(__uint_as_float(s[c]), __uint_as_float(s[c + 1]), w[c / 2]);
          tmem_store16(from + kColumns / 2, w);
        }
        arrive_warp(&p_ready[n % SB]);
        if (!wait(&dp_full, n & 1, limit)) return false;
        fence_after();
        uint32_t g[kColumns];
        tmem_load32(dp_from, g);
        loads_done();
        if (x == 0) {  // rows of the first token, which see one key: its score has no gradient, NaN stays
#pragma unroll
          for (int c = 0; c < kColumns; c++)
            if (c0 + c < group) s[c] = __float_as_uint(__uint_as_float(s[c]) * 0.f);
        }
        // four of the scores' gradients as bf16 pairs
        auto gradients = [&](int c, float2* u, float2* v) {
          const float4 y = d[c / 4];
          *u = unpack(mul2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                           add2(f2(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), f2(y.x, y.y))));
          *v = unpack(mul2(f2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                           add2(f2(__uint_as_float(g[c + 2]), __uint_as_float(g[c + 3])), f2(y.z, y.w))));
          w[c / 2] = bf16_pair(u->x, u->y);
          w[c / 2 + 1] = bf16_pair(v->x, v->y);
        };
        float2 u, v;
        if (RESTS) {
#pragma unroll
          for (int c = 0; c < kColumns; c += 4) {
            gradients(c, &u, &v);
            s[c / 2] = bf16_rest(u.x, u.y, w[c / 2]);  // in the place of weights that have had their turn
            s[c / 2 + 1] = bf16_rest(v.x, v.y, w[c / 2 + 1]);
          }
          tmem_store16(dp_from + kColumns / 2, s);
        } else {
#pragma unroll
          for (int c = 0; c < kColumns; c += 4) gradients(c, &u, &v);
        }
        tmem_store16(dp_from, w);
        arrive_warp(&ds_ready);
        if (lane == 0) arrive(&empty[stage]);  // the rows' numbers have been read
        n++;
        return true;
      };
      bool fine = true;
      if (rests_of(t))
        for (int x = begin; x < end && fine; x++) fine = work_out(std::true_type{}, x);
      else
        for (int x = begin; x < end && fine; x++) fine = work_out(std::false_type{}, x);
      if (!fine) break;
      Quarter<DP> dk, dv;
      if (begin < end) {
        if (!wait(&sums_full, some & 1, limit)) break;
        some++;
        fence_after();
        dk.load(dk_at + quarter, slice);
        dv.load(dv_at + quarter, slice);
        loads_done();
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(&sums_free);
      } else {
        dk.zero();
        dv.zero();
      }
      if (row < t.count) {
        const int64_t token = (int64_t)t.sequence + key;
        if (work.split.parts > 1) {
          const int64_t each = key_part_floats(a.nranks, a.tokens, a.kv_heads, D);
          float* const to = work.split.sums + 2 * t.part * each + (((int64_t)t.rank * a.tokens + token) * a.kv_heads + t.head) * D;
          dk.store_part(to, slice, a.scale, D);
          dv.store_part(to + each, slice, 1.f, D);
        } else {
          dk.store((uint16_t*)a.dk[t.rank] + token * a.dk_stride + t.head * a.dk_head, slice, a.scale, D);
          dv.store((uint16_t*)a.dv[t.rank] + token * a.dv_stride + t.head * a.dv_head, slice, 1.f, D);
        }
      }
    }
  }
  end_block(a.ws, limit, warp);
}

template <int DP>
cudaError_t launch(const PromptBwdArgs& a, cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads, per_tile = kTile / group, D = a.head_dim;
  const void *rows = (const void*)prompt_rows_tc_kernel<DP>, *keys = (const void*)prompt_keys_tc_kernel<DP>;
  int blocks = 0;
  cudaError_t e = resident_blocks(rows, kThreads, Layout<DP>::kRowsShared, &blocks);
  if (e == cudaSuccess) e = resident_blocks(keys, kThreads, Layout<DP>::kKeysShared, &blocks);
  static thread_local Maps maps;
  for (int r = 0; r < a.nranks && e == cudaSuccess; r++) {
    e = make_map(&maps.q[r], a.q[r], D, a.q_heads, a.tokens, a.q_head * 2, a.q_stride * 2, group, per_tile);
    if (e == cudaSuccess)
      e = make_map(&maps.dout[r], a.dout[r], D, a.q_heads, a.tokens, a.dout_head * 2, a.dout_stride * 2, group, per_tile);
    if (e == cudaSuccess) e = make_map(&maps.k[r], a.k[r], D, a.kv_heads, a.tokens, a.k_head * 2, a.k_stride * 2, 1, kTile);
    if (e == cudaSuccess) e = make_map(&maps.v[r], a.v[r], D, a.kv_heads, a.tokens, a.v_head * 2, a.v_stride * 2, 1, kTile);
  }
  if (e != cudaSuccess) return e;
  PromptBwdArgs copy = a;
  void* delta_params[] = {&copy};
  const int64_t a_block = 8 * 4 * (32 / (DP / 8));  // rows
  // (no row of 128 tokens or fewer has a second tile of keys: the rows' kernel works out all deltas)
  if (a.tokens > kTile)
    e = launch_op((const void*)prompt_delta_kernel<DP>,
                  dim3((unsigned)div_up((int64_t)a.tokens * a.q_heads, a_block), (unsigned)a.nranks), 256, 0, stream, delta_params);
  for (int which = 0; which < 2 && e == cudaSuccess; which++) {
    Work work;
    work.unit = which == 0 ? per_tile : kTile;
    work.slots = prompt_slots(a.tokens, a.sequences, 1, work.unit);
    work.split.parts = 1;
    if (which == 1)
      work.split.parts = key_parts(work.slots * a.kv_heads * a.nranks, blocks < kPromptSplitBlocks ? blocks : kPromptSplitBlocks,
                                   likely_keys(a.tokens, a.sequences) / (2 * per_tile), kLeastRowTilesFew, kLeastRowTiles);
    work.split.sums = (float*)(a.ws + kOpScratchOffset + align_up((int64_t)a.nranks * a.tokens * a.q_heads * 4, 256));
    const int64_t all = work.slots * work.split.parts * a.kv_heads * a.nranks;
    void* params[] = {&copy, &maps, &work};
    e = launch_op(which == 0 ? rows : keys, dim3((unsigned)(all < blocks ? all : blocks)), kThreads,
                  which == 0 ? Layout<DP>::kRowsShared : Layout<DP>::kKeysShared, stream, params);
    if (e == cudaSuccess && work.split.parts > 1) e = launch_prompt_key_parts(a, work.split, stream);
  }
  return e;
}

}  // namespace

cudaError_t launch_prompt_attention_bwd_tc(const PromptBwdArgs& a, cudaStream_t stream) {
  return a.head_dim <= 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace rar
