// prompt_attention_tc.cu -- attention over whole prompts in bf16 on the fifth-
// generation tensor cores, for head sizes up to 128 and up to 128 query heads a key head.
//
//   S = Q K^T,  P = 2^(scale log2(e) S - m),  O += P V,  l += row sums of P
//
// with the running maximum m of a row; out = O / l, lse = (m + log2 l) ln 2. A row is a
// query head of the group of a token, so a tile's 128 rows are floor(128 / group)
// tokens, and K and V are read once for all heads of the group.
//
// A block has two tiles of rows (an item) and walks over tiles of 128 keys. One warp
// copies (TMA), one issues products, and a warpgroup for each tile of rows turns S into
// P: a thread a row, so that the softmax needs no exchange between threads. While one
// tile's weights are being worked out, the other's products run. S and O are in tensor
// memory (2 x 128 and 2 x head size columns); P takes the place of the S that it came
// from, as bf16, and is the left operand of P V from there; products with the first half
// of a tile's weights run while the second half is worked out. Weights are rounded to bf16
// for that product; their sum l is of the unrounded ones. The rounding is as large as the
// result's own, over few keys or many: out is off by 1.9 to 2.1e-3 of its norm, where its own
// rounding is 1.6e-3. What it leaves would take a second product: 686 -> 977 us for 16384
// tokens, 115 -> 147 for 8192 packed ones, 306 -> 422 for chunks. A cached request of one tile of
// rows (128 / group new tokens: drafts behind a long context) has it (20.4 -> 22.4 us for five
// tokens behind 30011, 58 -> 73 for eight such requests; 2.3e-3 -> 1.7e-3), so that these tokens come out as close as one by one from
// decode_attention.cu, which has it too. The second tile's columns are free there.
//
// Blocks stay, one an SM, and take items from a counter, those with the most keys
// first. A fourth warp takes them ahead and finds out what they are, so
// that queries, keys and values of the next item are copied, and its scores worked out,
// while the last one's results are still being stored.
//
// m moves only if a score is more than 8 above it (in base 2): weights up to 2^8 lose
// nothing in binary32, and O is read and rescaled for almost no tile. Products run in
// the order in which they are issued, so the S of the next tile that a warpgroup
// sees says that P V of the last one has been added too.
//
// Few rows over many keys (the verification of drafted tokens behind a long context)
// would leave most SMs idle: where the items would be at most half of the SMs, each
// one's keys are split over several, which leave O, m and l unscaled as binary32, and a
// second kernel adds them up in the order of the keys, a block a row, or a warp a row
// where there are few parts (prompt_attention.cu).
//
// Measured: 16384 tokens of one sequence, 16 query heads on 2 key heads of 128: 613 us in runs of
// milliseconds, 650 to 695 in longer ones with lower clocks, 1.58 to 1.79 PFLOP/s, where a plain
// matrix product makes 1.95 in a burst and 1.73 over seconds; chunks of 2048 tokens behind up to 8192
// cached ones, 64 heads on 8, pages of 16: 294 to 304 us, tensor cores 70 % of the time. 8192 tokens in
// 17 sequences: 115 us, tensor cores 41 %: items are over before the chain of their products and weights has
// filled the SM, and reading and writing rows takes 45 us of it at the memory's rate.
// Heads of 64 take 515 us for the 16384 tokens: the exponentials bound them, as many
// for half the products. Five tokens behind 30011 take 23 us, a chain of a block's start,
// its share of the keys and the join; 97 tokens 8, a chain of one tile: the first item
// 1.5 us, copies 0.6, scores 0.4, weights 1.1, the product 0.4, rows 0.6.
#include <type_traits>

#include "prompt_attention.cuh"
#include "rar_launch.h"
#include "tensor_core.cuh"

namespace rar {
namespace {

using namespace tc;

// Where keys and values are, and how they are copied: dense, in pages by TMA, or in
// pages by the lanes of a fourth warpgroup. TMA takes a box a page (two for heads of 72 to
// 120), and with small pages a tile's boxes take longer to issue than its products to run;
// lanes take as long whatever the pages are. Chunks of 2048 tokens of 6 requests behind up to
// 8192, 64 / 8 heads, us by TMA in pages of 8, 16 and 32 tokens, and by lanes: heads of 40 293,
// 253, 253 and 285; of 64 293, 260, 258 and 280; of 80 474, 312, 276 and 323; of 120 478, 321,
// 300 and 350; of 128 328, 301, 300 and 339.
enum Form { kDense, kPages, kLanes };
// Two softmax warpgroups, one of which each warp has a part of its own, and the one that
// copies keys and values. The registers that a block starts with (168 a thread of 384,
// 128 of 512) are shared out anew: what the others leave, the softmax takes.
template <int FORM>
struct Threads {
  static constexpr int kCount = FORM == kLanes ? 512 : 384, kStart = FORM == kLanes ? 128 : 168;
  static constexpr int kFew = FORM == kLanes ? 48 : 72, kMany = FORM == kLanes ? 208 : 216;
  static_assert(kFew * (kCount / 128 - 2) + 2 * kMany <= kStart * (kCount / 128), "no more than the block was launched with");
};
constexpr int kRows = 128, kKeys = 128;
constexpr int kCopyWarp = 8, kProductWarp = 9, kItemWarp = 10, kStoreWarp = 11, kCacheWarp = 12;
constexpr int kItemSlots = 2, kLostSlots = 8;
constexpr int kNextItem = kOpCounters - 1, kDoneBlocks = kOpCounters - 2;  // counters of the workspace
constexpr float kLog2e = 1.4426950408889634f;

struct Maps {
  CUtensorMap q[kMaxRanks], k[kMaxRanks], v[kMaxRanks], out[kMaxRanks];  // k, v: of dense keys
};

template <int DP>
struct Layout {
  static constexpr int kSlab = kRows * 128;              // 64 elements of 128 rows
  static constexpr int kTile = kSlab * (DP / 64);
  static constexpr int kQueries = 3;                     // tiles of queries: the item's, and one of the next
  static constexpr int kStages = DP == 64 ? 8 : 4;       // tiles of keys or values
  static constexpr int kShared = (kQueries + kStages) * kTile + 1024;
  // With half the columns for O, weights have columns of their own, and the S of the next tile need not wait for P V.
  static constexpr bool kApart = DP == 64;
};

struct Split {
  int64_t slots, items;
  int parts;    // that an item's keys are split into
  float* sums;  // per item and part: 2 x 128 rows of DP binary32, then m and l of each
};
// of 2 x 128 rows with m and l
template <int DP>
constexpr int64_t kPartFloats = 2 * kRows * (DP + 2);

struct Item {
  int there;        // 0: no more
  int rank, head;   // key head
  int sequence, keys;
  int first, before;  // the first row's token in the step, and its position
  int tokens[2];    // of each tile of rows
  int begin, end;   // tiles of keys
  int last[2];      // a tile of rows walks from begin to here
  int part;
  int rests;        // weights keep what their rounding leaves
  int64_t index;    // of the item, parts aside
};

// Item number n in order; 0 if there is none, -1 if there are no more (a whole warp).
// Numbers are below 2^31, and in 32 bits for short prompts: divisions in 64 are half of the time that the first item takes.
template <int FORM>
__device__ __forceinline__ int find_item(const PromptArgs& a, const Split& split, ItemOrder& order, bool ordered, uint32_t n,
                                         Item* item) {
  const int per_tile = kRows / (a.q_heads / a.kv_heads);
  const uint32_t whole = n / (uint32_t)split.parts, lanes = (uint32_t)(a.kv_heads * a.nranks), slot = whole / lanes;
  item->part = (int)(n - whole * (uint32_t)split.parts);
  const int lane_of = (int)(whole - slot * lanes);
  item->head = lane_of % a.kv_heads;
  item->rank = lane_of / a.kv_heads;
  PromptSequence seq;
  int pair;
  if (ordered) {
    if (!order.advance(slot, 2 * per_tile, false, &seq.index, &pair)) return -1;
    seq.first = __shfl_sync(~0u, order.first, seq.index);
    seq.length = __shfl_sync(~0u, order.length, seq.index);
    seq.before = __shfl_sync(~0u, order.before, seq.index);
    seq.keys = __shfl_sync(~0u, order.keys, seq.index);
  } else {
    // the last tokens of a sequence see the most keys: they come first
    if (!find_sequence(a.starts, a.sequences, a.tokens, 1, 2 * per_tile, split.slots - 1 - slot, &seq, &pair)) return 0;
    if (FORM != kDense) cached_sequence(a, &seq);
  }
  const int token0 = pair * 2 * per_tile;  // of the sequence
  item->rests = FORM != kDense && seq.length <= per_tile;
  item->index = (int64_t)(seq.first / (2 * per_tile) + seq.index + pair) * lanes + lane_of;  // by number, as the join finds it
  item->sequence = seq.index;
  item->keys = seq.keys;
  item->first = seq.first + token0;
  item->before = seq.before + token0;
  int tiles[2];
#pragma unroll
  for (int t = 0; t < 2; t++) {
    const int tokens = max(0, min(per_tile, seq.length - token0 - t * per_tile));
    const int sees = min(item->before + t * per_tile + tokens, seq.keys);
    tiles[t] = tokens > 0 && sees > 0 ? (sees + kKeys - 1) / kKeys : 0;
    item->tokens[t] = tokens;
  }
  const int most = max(tiles[0], tiles[1]);
  // (most is below 2^24, parts 152 or fewer)
  item->begin = (int)((uint32_t)most * (uint32_t)item->part / (uint32_t)split.parts);
  item->end = (int)((uint32_t)most * (uint32_t)(item->part + 1) / (uint32_t)split.parts);
#pragma unroll
  for (int t = 0; t < 2; t++) item->last[t] = max(item->begin, min(tiles[t], item->end));
  item->there = 1;
  return 1;
}

template <int DP, int FORM>
__global__ void __launch_bounds__(Threads<FORM>::kCount, 1) prompt_tc_kernel(const __grid_constant__ PromptArgs a,
                                                                const __grid_constant__ Maps maps,
                                                                const __grid_constant__ Split split) {
  using L = Layout<DP>;
  constexpr int NS = L::kStages, NQ = L::kQueries;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (shared_address(raw) & 1023));
  __shared__ uint64_t q_full[NQ], q_empty[NQ], full[NS], empty[NS], s_full[2], s_read[2], p_half[2], p_full[2], pv_done[2], o_full[2],
      o_free[2], out_ready[2],
      item_full[kItemSlots], item_empty[kItemSlots];
  __shared__ Item items[kItemSlots];
  __shared__ uint32_t tmem_at, lost[kLostSlots][4];
  __shared__ Limit limit_at;
  volatile Limit* const limit = &limit_at;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    limit->dead = 0;
    limit->ns = a.wait_ns;
    for (int i = 0; i < NQ; i++) {
      barrier_init(&q_full[i], 1);
      barrier_init(&q_empty[i], 1);
    }
    for (int i = 0; i < NS; i++) {
      barrier_init(&full[i], FORM == kLanes ? 4 : 1);
      barrier_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      barrier_init(&s_full[i], 1);
      barrier_init(&s_read[i], 4);
      barrier_init(&pv_done[i], 1);
      barrier_init(&p_half[i], kRows);
      barrier_init(&p_full[i], kRows);
      barrier_init(&o_full[i], 1);
      barrier_init(&o_free[i], kRows);
      barrier_init(&out_ready[i], kRows);
    }
    for (int i = 0; i < kItemSlots; i++) {
      barrier_init(&item_full[i], 1);
      barrier_init(&item_empty[i], FORM == kLanes ? 15 : 11);  // the warps that read it: all but the one that writes it
    }
    barriers_ready();
  }
  if (warp == kCopyWarp && lane == 0) {  // the descriptors of the first item
    const int first = (int)(blockIdx.x / split.parts % (a.kv_heads * a.nranks)) / a.kv_heads;
    prefetch_map(&maps.q[first]);
    prefetch_map(&maps.out[first]);
    if (FORM != kLanes) {
      prefetch_map(&maps.k[first]);
      prefetch_map(&maps.v[first]);
    }
  }
  const uint32_t magic = op_start(a.ws);
  const int group = a.q_heads / a.kv_heads, D = a.head_dim;
  const int per_tile = kRows / group;  // tokens of a tile
  if (warp == kCopyWarp) tmem_alloc(&tmem_at, 512);
  ItemOrder order;
  bool ordered = false;
  if (warp == kItemWarp) {
    ordered = order.begin(a.starts, a.sequences, a.tokens, 2 * per_tile);
    if (FORM != kDense && ordered && order.items > 0) {  // (a request with no new tokens is not looked at)
      PromptSequence seq = {lane, order.first, order.length, 0, order.length};
      cached_sequence(a, &seq);
      order.before = seq.before;
      order.keys = seq.keys;
    }
  }
  __syncthreads();
  constexpr uint32_t tmem = 0;  // all of it, so it begins at 0
  constexpr uint32_t s_at[2] = {tmem, tmem + 128}, o_at[2] = {tmem + 256, tmem + 256 + DP};
  constexpr uint32_t p_at[2] = {L::kApart ? tmem + 384 : s_at[0], L::kApart ? tmem + 448 : s_at[1]};
  // of the first tile of rows, where there is no second one: the second's place, or the other half of S
  constexpr uint32_t rest_at = L::kApart ? p_at[1] : p_at[0] + 64;
  uint8_t* const ring = smem + NQ * L::kTile;
  const uint32_t all = (uint32_t)(split.items * split.parts);
  // a tile of keys is slab by slab, or where a box holds whole rows of pages, eight rows of both slabs after one another
  const bool grouped = FORM == kPages && DP == 128 && D == DP;
  const uint32_t kv_slab = grouped ? kGroup : L::kSlab, kv_group = grouped ? kGroup * (DP / 64) : kGroup;
  const int steps = (D + 15) / 16;
  // With one item a block, its softmax warps store the results: a TMA store takes 1 us longer to be done, and there is
  // nothing to do meanwhile.
  const bool alone = all <= gridDim.x;

  if (warp >= kCopyWarp) give_registers<Threads<FORM>::kFew>();
  if (warp == kItemWarp) {
    uint32_t* const counters = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes);
    // without a workspace there are no items: the others wait for the first one, not for the header
    const bool ready = magic == kOpMagic;
    if (!ready && lane == 0) op_report(a.ws, kErrWorkspace);
    uint32_t n = ready ? blockIdx.x : all;
    for (int i = 0;;) {
      Item item;
      int found = n < all ? find_item<FORM>(a, split, order, ordered, n, &item) : -1;
      if (found < 0) item.there = 0;
      if (found != 0) {
        if (!wait_warp(&item_empty[i % kItemSlots], (i / kItemSlots & 1) ^ 1, limit)) break;
        if (lane == 0) {
          items[i % kItemSlots] = item;
          arrive(&item_full[i % kItemSlots]);
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
  } else if (warp == kCopyWarp) {
    int stage = 0, queries = 0, seen = 0;  // seen: tiles of keys of the items before
    uint32_t phase = 0;
    for (int i = 0;; i++) {
      if (!wait_warp(&item_full[i % kItemSlots], i / kItemSlots & 1, limit)) break;
      const Item& item = items[i % kItemSlots];
      const int there = uniform(item.there);
      if (!there) break;
      const int rank = uniform(item.rank), head = uniform(item.head), first = uniform(item.first), begin = uniform(item.begin),
                end = uniform(item.end), keys = uniform(item.keys),
                base = first - uniform(item.before);  // of the sequence, if its keys are dense
      const int32_t* const row_pages = a.table + uniform(item.sequence) * a.table_stride;
      const int last[2] = {uniform(item.last[0]), uniform(item.last[1])};
      __syncwarp();
      if (lane == 0) arrive(&item_empty[i % kItemSlots]);
      auto query = [&](int t) {
        const int at = queries % NQ;
        if (!wait_warp(&q_empty[at], (queries / NQ & 1) ^ 1, limit)) return false;
        if (lane == 0) {
          arrive_expect(&q_full[at], (uint32_t)(per_tile * group * 128 * (DP / 64)));
          for (int h = 0; h < DP / 64; h++)
            copy_3d(smem + at * L::kTile + h * L::kSlab, &maps.q[rank], h * 64, head * group, first + t * per_tile, &q_full[at]);
        }
        queries++;
        return true;
      };
      bool fine = true;
      if (last[0] > begin) fine = query(0);
      if (FORM == kLanes) {
        if (fine && last[1] > begin) fine = query(1);
        if (!fine) break;
        continue;
      }
      // a page, or 128 tokens of a larger one, is a lane's; read a tile ahead, INT32_MIN where there is no key
      const int box = FORM == kPages ? min(kKeys, 1 << a.page_shift) : kKeys;
      auto page_of = [&](int j) {
        const int key = j * kKeys + lane * box;
        return FORM == kPages && lane * box < kKeys && j < end && key < keys ? row_pages[key >> a.page_shift] : INT32_MIN;
      };
      int next_page = page_of(begin);
      for (int j = begin; j < end && fine; j++) {
        const int page = next_page;
        next_page = page_of(j + 1);
        const bool copied = (unsigned)page < (unsigned)a.num_pages;
        const int count = FORM == kPages ? __popc(__ballot_sync(~0u, copied)) : 0;
        for (int which = 0; which < 2; which++) {
          if (!(fine = wait_warp(&empty[stage], phase ^ 1, limit))) break;
          uint8_t* const to = ring + stage * L::kTile;
          const CUtensorMap* const map = which == 0 ? &maps.k[rank] : &maps.v[rank];
          if (FORM == kDense) {
            if (lane == 0) {
              arrive_expect(&full[stage], L::kTile);
              for (int h = 0; h < DP / 64; h++)
                copy_3d(to + h * L::kSlab, map, h * 64, head, base + j * kKeys, &full[stage]);
            }
          } else {
            if (which == 0) {
              const bool none = page != INT32_MIN && !copied;
              uint32_t bad[4] = {0, 0, 0, 0};
              if (__any_sync(~0u, none)) {
                if (none) op_report(a.ws, kErrCapacity);
#pragma unroll
                for (int r = 0; r < 4; r++) {  // rows of the tile that such a page would have filled
                  uint32_t bits = 0;
                  if (none)
                    for (int y = lane * box; y < (lane + 1) * box; y++)
                      if (y >> 5 == r) bits |= 1u << (y & 31);
                  bad[r] = __reduce_or_sync(~0u, bits);
                }
              }
              if (lane == 0) {
#pragma unroll
                for (int r = 0; r < 4; r++) lost[(seen + j - begin) % kLostSlots][r] = bad[r];
              }
            }
            __syncwarp();
            if (lane == 0) arrive_expect(&full[stage], (uint32_t)(count * box * 128 * (DP / 64)));
            __syncwarp();
            if (copied) {
              const int off = (j * kKeys + lane * box) & ((1 << a.page_shift) - 1), plane = page * a.kv_heads + head;
              if (grouped)
                copy_4d(to + lane * box * (128 * (DP / 64)), map, 0, 0, 0, ((plane << a.page_shift) + off) >> 3, &full[stage]);
              else
                for (int h = 0; h < DP / 64; h++)
                  copy_3d(to + h * L::kSlab + lane * box * 128, map, h * 64, off, plane, &full[stage]);
            }
            __syncwarp();
          }
          if (++stage == NS) {
            stage = 0;
            phase ^= 1;
          }
          if (j == begin && which == 0 && last[1] > begin && !(fine = query(1))) break;
        }
      }
      if (!fine) break;
      seen += end - begin;
    }
  } else if (FORM == kLanes && warp >= kCacheWarp) {
    // Keys and values of a cache's pages, 32 rows of a tile a warp, 16 bytes a lane, in the
    // places where TMA would put them. Rows of no key, or of a page that is none, are 0; so
    // are elements past the head.
    constexpr int kPieces = DP / 8, kAtOnce = 32 / kPieces;  // lanes of a row, rows of an instruction
    const int mine = (warp - kCacheWarp) * 32, piece = lane % kPieces;
    const bool inside = piece * 8 < D;
    // (rows of an instruction differ in the bits of a row's swizzle below those of its first one)
    const uint32_t to = shared_address(ring) + (piece >> 3) * L::kSlab + (mine + lane / kPieces) * 128 +
                        (((piece & 7) ^ (lane / kPieces)) << 4);
    int stage = 0, oldest = 0, pending = 0, seen = 0;  // pending: tiles from `oldest` on whose copies are under way
    uint32_t phase = 0;
    auto hand_over = [&] {  // the oldest of them, which has come in
      stores_to_products();
      __syncwarp();
      if (lane == 0) arrive(&full[oldest]);
      oldest = oldest + 1 == NS ? 0 : oldest + 1;
      pending--;
    };
    auto drain = [&] {
      if (pending == 2) {
        copies_done<1>();
        hand_over();
      }
      if (pending == 1) {
        copies_done<0>();
        hand_over();
      }
    };
    for (int i = 0;; i++) {
      if (pending > 0 && !__all_sync(~0u, ended(&item_full[i % kItemSlots], i / kItemSlots & 1))) drain();
      if (!wait_warp(&item_full[i % kItemSlots], i / kItemSlots & 1, limit)) break;
      const Item& item = items[i % kItemSlots];
      const int there = uniform(item.there);
      if (!there) break;
      const int head = uniform(item.head), keys = uniform(item.keys), begin = uniform(item.begin), end = uniform(item.end);
      const int32_t* row_pages = a.table + uniform(item.sequence) * a.table_stride;
      const uint16_t *const k = (const uint16_t*)a.k[uniform(item.rank)], *const v = (const uint16_t*)a.v[uniform(item.rank)];
      __syncwarp();
      if (lane == 0) arrive(&item_empty[i % kItemSlots]);
      auto page_of = [&](int j) {  // of the lane's row, a tile ahead
        const int key = j * kKeys + mine + lane;
        return j < end && key < keys ? row_pages[key >> a.page_shift] : 0;
      };
      bool fine = true;
      int next_page = page_of(begin);
      for (int j = begin; j < end && fine; j++) {
        const int key = j * kKeys + mine + lane, page = next_page;
        next_page = page_of(j + 1);
        const bool there = (unsigned)page < (unsigned)a.num_pages;
        const int row = key < keys && there
                            ? ((page * a.kv_heads + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1))
                            : -1;
        const uint32_t bad = __ballot_sync(~0u, key < keys && !there);
        if (bad != 0 && lane == 0) op_report(a.ws, kErrCapacity);
        for (int which = 0; which < 2; which++) {
          if (!__all_sync(~0u, ended(&empty[stage], phase ^ 1))) {
            drain();  // nobody would make room for what is not there yet
            if (!(fine = wait_warp(&empty[stage], phase ^ 1, limit))) break;
          }
          if (which == 0 && lane == 0) lost[(seen + j - begin) % kLostSlots][warp - kCacheWarp] = bad;
          const uint16_t* const from = (which == 0 ? k : v) + piece * 8;
          const uint32_t place = to + stage * L::kTile;
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += kAtOnce) {
            const int at = __shfl_sync(~0u, row, r0 + lane / kPieces);
            copy_16((place + r0 * 128) ^ ((r0 & 7) << 4), from + (int64_t)max(at, 0) * D, at >= 0 && inside ? 16 : 0);
          }
          copies_of_a_tile();
          if (++pending == 3) {
            copies_done<2>();
            hand_over();
          }
          if (++stage == NS) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!fine) break;
      seen += end - begin;
    }
    drain();
  } else if (warp == kStoreWarp) {
    if (blockIdx.x == 0) check_starts(a.starts, a.sequences, a.tokens, a.ws, lane, 32);
    int queries = 0, results[2] = {0, 0};
    for (int i = 0;; i++) {
      if (!wait_warp(&item_full[i % kItemSlots], i / kItemSlots & 1, limit)) break;
      const Item& item = items[i % kItemSlots];
      const int there = uniform(item.there);
      if (!there) break;
      const int rank = uniform(item.rank), head = uniform(item.head), first = uniform(item.first), begin = uniform(item.begin);
      const int last[2] = {uniform(item.last[0]), uniform(item.last[1])},
                tokens[2] = {uniform(item.tokens[0]), uniform(item.tokens[1])};
      __syncwarp();
      if (lane == 0) arrive(&item_empty[i % kItemSlots]);
      bool fine = true;
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (!fine || last[t] <= begin) continue;
        const int at = queries++ % NQ;
        if (!(fine = wait_warp(&out_ready[t], results[t]++ & 1, limit))) break;
        if (lane == 0) {
          if (tokens[t] == per_tile && split.parts == 1 && !alone) {
            for (int h = 0; h < DP / 64 && h * 64 < D; h++)
              store_3d(&maps.out[rank], h * 64, head * group, first + t * per_tile, smem + at * L::kTile + h * L::kSlab);
            stores_read();
          }
          arrive(&q_empty[at]);
        }
        __syncwarp();
      }
      if (!fine) break;
    }
    if (lane == 0) stores_written();
  } else if (warp == kProductWarp) {
    const uint32_t lead = elect_one();
    const int n_out = steps * 16;
    const uint32_t q_at = shared_address(smem), ring_at = shared_address(ring);
    int stage = 0, queries = 0, seen = 0;
    int walked[2] = {0, 0}, results[2] = {0, 0};  // tiles of keys, and items, of each tile of rows so far
    uint32_t phase = 0;
    for (int i = 0;; i++) {
      if (!wait_warp(&item_full[i % kItemSlots], i / kItemSlots & 1, limit)) break;
      const Item& item = items[i % kItemSlots];
      const int there = uniform(item.there);
      if (!there) break;
      const int begin = uniform(item.begin), end = uniform(item.end), keys = uniform(item.keys), rests = uniform(item.rests);
      const int last[2] = {uniform(item.last[0]), uniform(item.last[1])};
      __syncwarp();
      if (lane == 0) arrive(&item_empty[i % kItemSlots]);
      if (begin >= end) continue;
      int q_slot[2];
#pragma unroll
      for (int t = 0; t < 2; t++) q_slot[t] = last[t] > begin ? queries++ : 0;
      // the S of a key tile for a tile of rows that sees it
      auto score = [&](int t, uint32_t k_at) {
        rows_by_rows<DP / 16, L::kSlab>(lead, s_at[t], q_at + (uint32_t)(q_slot[t] % NQ) * L::kTile, k_at, kKeys, steps, kv_slab, kv_group);
        commit(lead, &s_full[t]);
      };
      // V of key tile j is there; rows with no key would be multiplied by weights of 0, and may hold a NaN
      auto values = [&](int j, int stage, uint32_t phase) {
        if (!wait_warp(&full[stage], phase, limit)) return false;
        const int left = keys - j * kKeys;
        const uint32_t* const holes_of = lost[(seen + j - begin) % kLostSlots];
        const bool holes = FORM == kPages && __any_sync(~0u, lane < 4 && holes_of[lane & 3] != 0);
        if (FORM != kLanes && (left < kKeys || holes)) {
          for (int r = lane; r < kKeys; r += 32)
            if (r >= left || (holes && (holes_of[r >> 5] >> (r & 31) & 1)))
              for (int h = 0; h < DP / 64; h++)
                for (int c = 0; c < 8; c++)
                  *reinterpret_cast<uint4*>(ring + stage * L::kTile + h * kv_slab + (r >> 3) * kv_group + (r & 7) * 128 + c * 16) =
                      make_uint4(0, 0, 0, 0);
          stores_to_products();
          __syncwarp();
        }
        return true;
      };
      // stages: K of the first tile, then V of a tile and K of the next in turn
      bool fine = wait_warp(&full[stage], phase, limit);
      const int first_stage = stage;
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (!fine || last[t] <= begin) continue;
        if (!(fine = wait_warp(&q_full[q_slot[t] % NQ], q_slot[t] / NQ & 1, limit))) break;
        fence_after();
        score(t, ring_at + first_stage * L::kTile);
      }
      if (!fine) break;
      commit(lead, &empty[first_stage]);
      if (++stage == NS) {
        stage = 0;
        phase ^= 1;
      }
      if (!values(begin, stage, phase)) break;
      int v_stage = stage;
      uint32_t v_phase = phase;
      for (int j = begin; j < end && fine; j++) {
        const bool more = j + 1 < end;
        const int k_stage = v_stage + 1 == NS ? 0 : v_stage + 1;
        const uint32_t k_phase = v_phase ^ (k_stage == 0);
        const int next_stage = k_stage + 1 == NS ? 0 : k_stage + 1;
        const uint32_t next_phase = k_phase ^ (next_stage == 0);
        if (L::kApart && more) {
          if (!(fine = wait_warp(&full[k_stage], k_phase, limit))) break;
#pragma unroll
          for (int t = 0; t < 2; t++) {
            if (!fine || j + 1 >= last[t]) continue;
            if (!(fine = wait_warp(&s_read[t], walked[t] & 1, limit))) break;
            fence_after();
            score(t, ring_at + k_stage * L::kTile);
          }
          if (!fine) break;
          commit(lead, &empty[k_stage]);
        }
#pragma unroll
        for (int t = 0; t < 2; t++) {
          if (j < last[t]) {
            // O of the item before has been read
            if (j == begin && results[t] > 0 && !(fine = wait_warp(&o_free[t], (results[t] - 1) & 1, limit))) break;
            if (!(fine = wait_warp(&p_half[t], walked[t] & 1, limit))) break;
            fence_after();
            weights_by_rows<8, 0, 0, 4>(lead, o_at[t], p_at[t], ring_at + v_stage * L::kTile, n_out, j > begin, kv_slab, kv_group);
            if (FORM != kDense && t == 0 && rests)
              weights_by_rows<8, 0, 0, 4>(lead, o_at[0], rest_at, ring_at + v_stage * L::kTile, n_out, true, kv_slab, kv_group);
            if (!(fine = wait_warp(&p_full[t], walked[t] & 1, limit))) break;
            fence_after();
            weights_by_rows<8, 0, 4, 8>(lead, o_at[t], p_at[t], ring_at + v_stage * L::kTile, n_out, true, kv_slab, kv_group);
            if (FORM != kDense && t == 0 && rests)
              weights_by_rows<8, 0, 4, 8>(lead, o_at[0], rest_at, ring_at + v_stage * L::kTile, n_out, true, kv_slab, kv_group);
            walked[t]++;
            if (L::kApart) commit(lead, &pv_done[t]);
            if (j + 1 == last[t]) {
              commit(lead, &o_full[t]);
              results[t]++;
            }
          }
          // what the warp waits for beside the weights, it waits for while products run
          if (!L::kApart && more && t == 0 && !(fine = wait_warp(&full[k_stage], k_phase, limit))) break;
          if (more && t == 1 && !(fine = values(j + 1, next_stage, next_phase))) break;
          if (!L::kApart && j + 1 < last[t]) {
            fence_after();
            score(t, ring_at + k_stage * L::kTile);
          }
        }
        if (!fine) break;
        commit(lead, &empty[v_stage]);
        if (!L::kApart && more) commit(lead, &empty[k_stage]);
        // behind the item's last V: the next item's first K
        stage = more ? next_stage : k_stage;
        phase = more ? next_phase : k_phase;
        v_stage = next_stage;
        v_phase = next_phase;
      }
      if (!fine) break;
      seen += end - begin;
    }
  } else if (warp < kCopyWarp) {
    take_registers<Threads<FORM>::kMany>();
    const int t = warp >> 2;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
    const int row = threadIdx.x & 127, token = row / group, in_group = row % group;
    // of a negative scale or none, the scores are turned or cleared first, so that the largest is the one that counts
    const float scale2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
    const float turn = a.scale < 0.f ? -1.f : 0.f;
    int walked = 0, results = 0, seen = 0, queries = 0;  // queries: tiles of queries of both tiles of rows
    for (int i = 0;; i++) {
      if (!wait(&item_full[i % kItemSlots], i / kItemSlots & 1, limit)) break;
      const Item& item = items[i % kItemSlots];
      if (!item.there || (a.fault == kFaultWeights && warp == 0)) break;
      const int begin = item.begin, end = item.end, last = item.last[t];
      const bool rests = item.rests;
      const int q_slot = (queries + (t == 1 && item.last[0] > begin)) % NQ;
      queries += (item.last[0] > begin) + (item.last[1] > begin);
      const int tokens = item.tokens[t];
      const bool mine = token < tokens;
      // rows that are none see what the tile's first row sees: they hold anything, and nobody reads them
      const int sees = min(item.before + t * per_tile + (mine ? token : 0) + 1, item.keys);
      const int query = item.head * group + in_group, rank = item.rank, part = item.part;
      const int64_t at_token = (int64_t)item.first + t * per_tile + token, index = item.index;
      __syncwarp();
      if (lane == 0) arrive(&item_empty[i % kItemSlots]);
      int least = sees;  // of the warp
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) least = min(least, __shfl_xor_sync(~0u, least, d));
      float m = -INFINITY, l = 0.f;
      bool fine = true;
      for (int j = begin; j < last; j++) {
        if (!(fine = wait(&s_full[t], walked & 1, limit))) break;
        walked++;
        fence_after();
        uint32_t s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_load32(s_at[t] + quarter + c, s + c);
        loads_done();
        if (L::kApart) {
          fence_before();
          __syncwarp();
          if (lane == 0) arrive(&s_read[t]);
        }
        if (!(a.scale > 0.f)) {
#pragma unroll
          for (int c = 0; c < kKeys; c++) s[c] = __float_as_uint(__uint_as_float(s[c]) * turn);
        }
        const uint32_t* holes_of = lost[(seen + j - begin) % kLostSlots];
        const bool holes = FORM != kDense && (holes_of[0] | holes_of[1] | holes_of[2] | holes_of[3]) != 0;
        if ((j + 1) * kKeys > least || holes) {
          const int upto = sees - j * kKeys;
#pragma unroll
          for (int c = 0; c < kKeys; c++) {
            bool there = c < upto;
            if (FORM != kDense && holes) there = there && !(holes_of[c >> 5] >> (c & 31) & 1);
            if (!there) s[c] = 0xff800000u;
          }
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; i++) top[i] = __uint_as_float(s[i]);
#pragma unroll
        for (int c = 4; c < kKeys; c += 4)
#pragma unroll
          for (int i = 0; i < 4; i++) top[i] = fmaxf(top[i], __uint_as_float(s[c + i]));
        const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // the last tile's weights have been read, and O has them
        if (L::kApart && j > begin) {
          if (!(fine = wait(&pv_done[t], walked & 1, limit))) break;
          fence_after();
        }
        const float high = best * scale2;
        // (rows that are none have no say: what they hold would change how the others are rounded)
        if (__any_sync(~0u, mine && high > m + 8.f)) {
          const float next = fmaxf(m, high);
          const float keep = next == -INFINITY ? 1.f : exp2_fast(m - next);
          m = next;
          l *= keep;
          if (j > begin) {
            uint32_t o[16];
#pragma unroll 1
            for (int c = 0; c < DP; c += 16) {
              tmem_load16(o_at[t] + quarter + c, o);
              loads_done();
#pragma unroll
              for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
              tmem_store16(o_at[t] + quarter + c, o);
            }
          }
        }
        const float by = m == -INFINITY ? 0.f : m;  // nothing seen so far: the weights are 0
        F2 sum = f2(0.f, 0.f), more = f2(0.f, 0.f);
        const F2 scale_pair = f2(scale2, scale2), by_pair = f2(-by, -by);
        // products with the first half of the weights run while the second half is worked out
        auto half = [&](auto with_rests, int h) {
          constexpr bool RESTS = decltype(with_rests)::value;
          uint32_t left[RESTS ? 16 : 1];
#pragma unroll
          for (int c = h * 64; c < h * 64 + 64; c += 4) {
            float2 x = unpack(fma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale_pair, by_pair));
            float2 y = unpack(fma2(f2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), scale_pair, by_pair));
            x.x = exp2_fast(x.x);
            x.y = exp2_fast(x.y);
            y.x = exp2_fast(y.x);
            y.y = exp2_fast(y.y);
            sum = add2(sum, f2(x.x, x.y));
            more = add2(more, f2(y.x, y.y));
            s[c / 2] = bf16_pair(x.x, x.y);
            s[c / 2 + 1] = bf16_pair(y.x, y.y);
            if (RESTS) {
              left[c / 2 % 16] = bf16_rest(x.x, x.y, s[c / 2]);
              left[c / 2 % 16 + 1] = bf16_rest(y.x, y.y, s[c / 2 + 1]);
              if (c % 32 == 28) tmem_store16(rest_at + quarter + c / 32 * 16, left);
            }
          }
          tmem_store32(p_at[t] + quarter + 32 * h, s + 32 * h);
          stores_done();
          fence_before();
          arrive(h == 0 ? &p_half[t] : &p_full[t]);
        };
        if (FORM != kDense && rests) {
          half(std::true_type{}, 0);
          half(std::true_type{}, 1);
        } else {
          half(std::false_type{}, 0);
          half(std::false_type{}, 1);
        }
        const float2 u = unpack(add2(sum, more));
        l += u.x + u.y;
      }
      if (!fine) break;
      seen += end - begin;
      const bool some = last > begin;  // O has been written
      if (some) {
        if (!wait(&o_full[t], results & 1, limit)) break;
        results++;
        fence_after();
      }
      const float by = l == 0.f ? 0.f : 1.f / l;
      uint16_t* const out = (uint16_t*)a.out[rank] + at_token * a.out_stride + query * a.out_head;
      float* const sums = split.sums + (index * split.parts + part) * kPartFloats<DP> + t * kRows * (DP + 2);
      if (!some) {
        for (int c = 0; c < D && mine && split.parts == 1; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
      } else {
        uint32_t o[DP];
#pragma unroll
        for (int c = 0; c < DP; c += 32) tmem_load32(o_at[t] + quarter + c, o + c);
        loads_done();
        fence_before();
        arrive(&o_free[t]);
        if (split.parts > 1) {  // a part of the keys: O as it is
          if (mine) {
#pragma unroll
            for (int c = 0; c < DP; c += 4)
              if (c < D) *reinterpret_cast<uint4*>(sums + row * DP + c) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
          }
        } else {
          // to the queries' place in shared memory, from where the store warp's TMA takes a
          // whole tile; a warp stores its rows of one that the sequence does not fill itself, or of a block's only item
          if (l == 0.f) {  // no weight at all: 0, whatever the values are
#pragma unroll
            for (int c = 0; c < DP; c++) o[c] = 0;
          }
          uint8_t* const place = smem + q_slot * L::kTile + row * 128;
          const F2 by_pair = f2(by, by);
#pragma unroll
          for (int c = 0; c < DP; c += 8) {
            uint4 x;
            uint32_t* to = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const float2 v = unpack(mul2(f2(__uint_as_float(o[c + 2 * k]), __uint_as_float(o[c + 2 * k + 1])), by_pair));
              to[k] = bf16_pair(v.x, v.y);
            }
            *reinterpret_cast<uint4*>(place + (c >> 6) * L::kSlab + (((c >> 3 & 7) ^ (row & 7)) << 4)) = x;
          }
          stores_to_products();
          if (tokens != per_tile || alone) {
            __syncwarp();
            constexpr int kPieces = DP / 8, kAtOnce = 32 / kPieces;  // lanes of a row, rows of an instruction
            const int piece = lane % kPieces;
            const uint8_t* from = smem + q_slot * L::kTile + (row - lane) * 128 + (piece >> 3) * L::kSlab;
#pragma unroll 4
            for (int r0 = 0; r0 < 32; r0 += kAtOnce) {
              const int r = r0 + lane / kPieces;
              uint16_t* const to = (uint16_t*)__shfl_sync(~0u, mine ? (unsigned long long)out : 0ull, r);
              const uint4 x = *reinterpret_cast<const uint4*>(from + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
              if (to != nullptr && piece * 8 < D) *reinterpret_cast<uint4*>(to + piece * 8) = x;
            }
          }
        }
        arrive(&out_ready[t]);
      }
      if (mine && split.parts > 1) {
        sums[kRows * DP + row] = m;
        sums[kRows * (DP + 1) + row] = l;
      } else if (mine && a.lse[rank] != nullptr) {
        a.lse[rank][at_token * a.q_heads + query] = (m + log2f(l)) / kLog2e;
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (limit->dead) {
    // a wait ran out: copies and products that are still under way have ended by the time this has passed
    const uint64_t until = global_timer_ns() + 10000000ull;
    while (global_timer_ns() < until) {}
    if (threadIdx.x == 0) op_report(a.ws, kErrTimeout);
  }
  __syncthreads();
  if (warp == kCopyWarp) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

// The parts of a row's keys, a block a row: each of its four warps adds up every fourth
// part, all their loads under way at once, and the four sums join in the warps' order.
template <int DP>
__global__ void __launch_bounds__(128) prompt_join_kernel(const __grid_constant__ PromptArgs a,
                                                          const __grid_constant__ Split split) {
  constexpr int E = DP / 32, kMost = kPromptSplitBlocks / 4, kBatch = 20;  // elements of a lane, parts of a warp
  __shared__ float partial[4][DP];
  const uint32_t magic = op_start(a.ws);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = (int)(blockIdx.x % (2 * kRows)), t = r / kRows, row = r % kRows;
  const int group = a.q_heads / a.kv_heads, D = a.head_dim, per_tile = kRows / group, token = row / group;
  const int64_t index = blockIdx.x / (2 * kRows), lanes = (int64_t)a.kv_heads * a.nranks;
  const float* const sums = split.sums + index * split.parts * kPartFloats<DP> + t * kRows * (DP + 2);
  float m[kPromptSplitBlocks / 32 + 1], l[kPromptSplitBlocks / 32 + 1];
#pragma unroll
  for (int i = 0; i <= kPromptSplitBlocks / 32; i++) {
    const int k = i * 32 + lane;
    m[i] = k < split.parts ? sums[k * kPartFloats<DP> + kRows * DP + row] : -INFINITY;
    l[i] = k < split.parts ? sums[k * kPartFloats<DP> + kRows * (DP + 1) + row] : 0.f;
  }
  PromptSequence seq;
  int pair;
  if (!op_ready(a.ws, magic) || token >= per_tile) return;
  if (!find_sequence(a.starts, a.sequences, a.tokens, 1, 2 * per_tile, index / lanes, &seq, &pair)) return;
  const int at = pair * 2 * per_tile + t * per_tile + token;  // the row's token in the sequence
  if (at >= seq.length) return;
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i <= kPromptSplitBlocks / 32; i++) top = fmaxf(top, m[i]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
#pragma unroll
  for (int i = 0; i <= kPromptSplitBlocks / 32; i++) {
    // now the part's weight; below 0: a part with no weight at all has left nothing. (One of NaN scores alone has a
    // sum of NaN, and no maximum.)
    m[i] = l[i] == 0.f ? -1.f : exp2_fast(m[i] - top);
    if (!(m[i] < 0.f)) sum = fmaf(l[i], m[i], sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  float v[E] = {};
#pragma unroll 1
  for (int k0 = 0; k0 < kMost && k0 * 4 < split.parts; k0 += kBatch) {
    float x[kBatch][E], w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; k++) {
      const int part = (k0 + k) * 4 + warp;
      w[k] = -1.f;
#pragma unroll
      for (int i = 0; i <= kPromptSplitBlocks / 32; i++) {
        const float y = __shfl_sync(~0u, m[i], part & 31);
        if (part >> 5 == i) w[k] = y;
      }
      const float* p = sums + part * kPartFloats<DP> + row * DP + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float2 y = make_float2(0.f, 0.f);
        if (!(w[k] < 0.f) && part < split.parts) y = *reinterpret_cast<const float2*>(p + e);
        x[k][e] = y.x;
        x[k][e + 1] = y.y;
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; k++)
#pragma unroll
      for (int e = 0; e < E; e++) v[e] = fmaf(x[k][e], w[k] < 0.f ? 0.f : w[k], v[e]);
  }
#pragma unroll
  for (int e = 0; e < E; e++) partial[warp][lane * E + e] = v[e];
  __syncthreads();
  const int lane_of = (int)(index % lanes), head = lane_of % a.kv_heads, rank = lane_of / a.kv_heads;
  const int64_t at_token = (int64_t)seq.first + at;
  const int query = head * group + row % group, d = threadIdx.x * 2;
  const float by = sum == 0.f ? 0.f : 1.f / sum;
  if (d < D) {
    float y[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const float z = (partial[0][d + e] + partial[1][d + e]) + (partial[2][d + e] + partial[3][d + e]);
      y[e] = sum == 0.f ? 0.f : z * by;
    }
    *reinterpret_cast<uint32_t*>((uint16_t*)a.out[rank] + at_token * a.out_stride + query * a.out_head + d) = bf16_pair(y[0], y[1]);
  }
  if (threadIdx.x == 0 && a.lse[rank] != nullptr) a.lse[rank][at_token * a.q_heads + query] = (top + log2f(sum)) / kLog2e;
}

template <int DP, int FORM>
cudaError_t launch(const PromptArgs& a, cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads, per_tile = kRows / group, D = a.head_dim;
  const void* fn = (const void*)prompt_tc_kernel<DP, FORM>;
  int blocks = 0;
  cudaError_t e = resident_blocks(fn, Threads<FORM>::kCount, Layout<DP>::kShared, &blocks);
  if (e != cudaSuccess) return e;
  static thread_local Maps maps;
  for (int r = 0; r < a.nranks && e == cudaSuccess; r++) {
    e = make_map(&maps.q[r], a.q[r], D, a.q_heads, a.tokens, a.q_head * 2, a.q_stride * 2, group, per_tile);
    if (e == cudaSuccess) e = make_map(&maps.out[r], a.out[r], D, a.q_heads, a.tokens, a.out_head * 2, a.out_stride * 2, group, per_tile);
    for (int which = 0; which < 2 && e == cudaSuccess; which++) {
      CUtensorMap* map = which == 0 ? &maps.k[r] : &maps.v[r];
      const void* base = which == 0 ? a.k[r] : a.v[r];
      const int64_t page = (int64_t)1 << a.page_shift, planes = (int64_t)a.num_pages * a.kv_heads, box = page < kKeys ? page : kKeys;
      if (FORM == kDense)
        e = make_map(map, base, D, a.kv_heads, a.tokens, (which == 0 ? a.k_head : a.v_head) * 2,
                     (which == 0 ? a.k_stride : a.v_stride) * 2, 1, kKeys);
      else if (FORM == kPages && DP == 128 && D == DP)
        e = make_grouped_map(map, base, D, planes * page, (int)box / 8);
      else if (FORM == kPages)
        e = make_map(map, base, D, page, planes, D * 2, page * D * 2, (int)box, 1);
    }
  }
  if (e != cudaSuccess) return e;
  Split split;
  split.slots = prompt_slots(a.tokens, a.sequences, 1, 2 * per_tile);
  split.items = split.slots * a.kv_heads * a.nranks;
  split.sums = (float*)(a.ws + kOpScratchOffset);
  split.parts = 1;
  // tiles of keys that an item may have
  const int64_t most = div_up(FORM != kDense ? (int64_t)a.max_blocks << a.page_shift : likely_keys(a.tokens, a.sequences), kKeys);
  if (split.items * 2 <= kPromptSplitBlocks) {
    const int64_t room = kPromptSplitBlocks / split.items, wanted = div_up(most, 2);
    split.parts = (int)(room < wanted ? room : wanted);
  }
  const int64_t all = split.items * split.parts;
  PromptArgs copy = a;
  void* params[] = {&copy, &maps, &split};
  e = launch_op(fn, dim3((unsigned)(all < blocks ? all : blocks)), Threads<FORM>::kCount, Layout<DP>::kShared, stream, params);
  if (e != cudaSuccess || split.parts == 1) return e;
  if (split.parts <= kFewParts)
    return launch_prompt_join_few(a, {split.sums, split.parts, kRows, DP, 1, kPartFloats<DP>, split.slots}, stream);
  void* join_params[] = {&copy, &split};
  return launch_op((const void*)prompt_join_kernel<DP>, dim3((unsigned)(split.items * 2 * kRows)), 128, 0, stream, join_params);
}

}  // namespace

cudaError_t launch_prompt_attention_tc(const PromptArgs& a, cudaStream_t stream) {
  const bool small = a.head_dim <= 64;
  if (a.table == nullptr) return small ? launch<64, kDense>(a, stream) : launch<128, kDense>(a, stream);
  if (a.page_shift >= (a.head_dim == 128 ? 3 : 4)) return small ? launch<64, kPages>(a, stream) : launch<128, kPages>(a, stream);
  return small ? launch<64, kLanes>(a, stream) : launch<128, kLanes>(a, stream);
}

}  // namespace rar
