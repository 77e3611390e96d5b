// prompt_attention.cuh -- what the forms of the attention over whole prompts share:
// arguments, and the way from a block's number to its rows.
//
// The query heads that share a key head are rows of one tile: row r of a sequence is
// head r % group of its token r / group. Sequences are packed along the tokens, and
// only the device knows where they start. A tile holds `unit` of something that a
// sequence has `per` of a token (rows, or tokens); sequence s takes the numbers from
// slot(s) = floor(starts[s] per / unit) + s on. That leaves it at least
// ceil(length per / unit) numbers, since floor(x + y) >= floor(x) + ceil(y) - 1, so a
// grid of slot(last) + 1 blocks, whose size the host knows, covers any starts, and a
// block finds its sequence by bisection with no sums over the lengths.
#pragma once

#include "op_common.cuh"

namespace rar {

struct PromptArgs {
  const void* q[kMaxRanks];
  const void* k[kMaxRanks];  // [tokens, kv_heads, head_dim], or the paged cache if table is set
  const void* v[kMaxRanks];
  void* out[kMaxRanks];
  float* lse[kMaxRanks];  // null: not wanted
  const int32_t* starts;
  const int32_t* lens;   // of the cached form
  const int32_t* table;  // null: dense keys
  char* ws;
  int64_t q_stride, k_stride, v_stride, out_stride, table_stride;
  int64_t q_head, k_head, v_head, out_head;  // elements from head to head of a token
  float scale;
  int nranks, dtype, tokens, sequences, q_heads, kv_heads, head_dim, page_shift, num_pages, max_blocks;
  uint64_t wait_ns;  // limit of a wait inside a block
  int fault;
};

struct PromptBwdArgs {
  const void* q[kMaxRanks];
  const void* k[kMaxRanks];
  const void* v[kMaxRanks];
  const void* out[kMaxRanks];
  const void* dout[kMaxRanks];
  const float* lse[kMaxRanks];
  void* dq[kMaxRanks];
  void* dk[kMaxRanks];
  void* dv[kMaxRanks];
  const int32_t* starts;
  char* ws;  // scratch: delta, float [ranks, tokens, q_heads]; then what parts leave of dk and dv
  int64_t q_stride, k_stride, v_stride, out_stride, dout_stride, dq_stride, dk_stride, dv_stride;
  int64_t q_head, k_head, v_head, out_head, dout_head, dq_head, dk_head, dv_head;
  float scale;
  int nranks, dtype, tokens, sequences, q_heads, kv_heads, head_dim;
  uint64_t wait_ns;  // limit of a wait inside a block
  int fault;
};

// The rows that see a tile of keys may be split into parts, which then leave their sums:
// float [part, 2 (dk, dv), rank, token, kv_heads, head_dim] behind delta.
struct KeyParts {
  int parts;
  float* sums;
};
__host__ __device__ inline int64_t key_part_floats(int nranks, int64_t tokens, int kv_heads, int head_dim) {
  return (int64_t)nranks * tokens * kv_heads * head_dim;  // of dk, or dv, of a part
}
constexpr int kMostKeyParts = 8;
// Parts for `items` tiles of keys on `blocks` resident blocks, where a key is seen by the rows of `row_tiles` tiles on
// average. Few items are split until there is one a block, into parts of `least_few` tiles of rows or more, or two, of twice
// as many (1000 tokens, 4 key heads of 64: 71 us whole, 51 in three parts, 55 in seven). The items of a long
// sequence differ by the rows that see them, so they are split further, into parts of `least` tiles, for eight a
// block: one of 8192 tokens, 4 key heads of 64, 658 us whole and 554 in four parts; of 4096 tokens, 8 key heads of 128, 64
// tiles of rows or fewer each, 244 whole and 256 in two, for the cost of the parts' sums.
inline int key_parts(int64_t items, int64_t blocks, int64_t row_tiles, int64_t least_few, int64_t least) {
  if (items < 1) items = 1;
  int64_t parts = 1;
  const int64_t waves[] = {1, 2, 8}, tiles[] = {least_few, 2 * least_few, least};
  for (int i = 0; i < 3; i++) {
    const int64_t room = waves[i] * blocks / items, there = row_tiles / tiles[i], n = room < there ? room : there;
    parts = n > parts ? n : parts;
  }
  return parts > kMostKeyParts ? kMostKeyParts : (int)parts;
}
// on the tensor cores, and on the ordinary arithmetic units, where a tile takes 5 to 8 us
constexpr int kLeastRowTilesFew = 2, kLeastRowTiles = 32, kLeastPlainRowTilesFew = 1, kLeastPlainRowTiles = 8;
// Adds them up, in their order.
cudaError_t launch_prompt_key_parts(const PromptBwdArgs& a, const KeyParts& parts, cudaStream_t stream);

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream);
// The forms of bf16 with head sizes up to 128 and groups up to 128 (prompt_attention_tc.cu, prompt_attention_bwd_tc.cu).
cudaError_t launch_prompt_attention_tc(const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_prompt_attention_bwd_tc(const PromptBwdArgs& a, cudaStream_t stream);
constexpr int kPromptSplitBlocks = 152;  // blocks among which few tiles' keys are split: the SMs
constexpr int kPromptParts = 304;        // the same in the form on the ordinary arithmetic units: two blocks an SM
cudaError_t launch_prompt_attention_bwd(const PromptBwdArgs& a, cudaStream_t stream);
int64_t prompt_attention_scratch_bytes(int nranks, int64_t tokens, int q_heads, int kv_heads, int head_dim);

// Where few parts of each row's keys have been left: of item i's part k from sums + (i * parts + k) * part_floats on,
// with tiles of tile_rows rows of row_floats numbers, then their m and l.
struct FewParts {
  const float* sums;
  int parts, tile_rows, row_floats, pairs;  // pairs: items are two tiles, and the ranks' heads of an item lie together
  int64_t part_floats, slots;
};
constexpr int kFewParts = 16;
// Joins them, a warp a row: a block a row, most of its threads idle, took 45 us for 500 tokens of 16 heads.
cudaError_t launch_prompt_join_few(const PromptArgs& a, const FewParts& parts, cudaStream_t stream);
// Keys that one of the dense sequences may have, as far as the host knows: twice the average.
inline int64_t likely_keys(int64_t tokens, int sequences) {
  return sequences < 2 ? tokens : (2 * tokens + sequences - 1) / sequences;
}

// Numbers that cover any starts of `tokens` tokens in `sequences` sequences.
inline int64_t prompt_slots(int64_t tokens, int sequences, int per, int unit) {
  return tokens * per / unit + sequences;
}

// A sequence as its starts and lengths say, with what does not fit left out.
struct PromptSequence {
  int index, first, length;  // its number, first token and tokens in the step
  int before;                // position of its first token; negative where lens is below the step's tokens
  int keys;                  // tokens with a key
};

// Every pair of starts, by `threads` threads from 0 on.
__device__ __forceinline__ void check_starts(const int32_t* starts, int sequences, int tokens, char* ws, int thread,
                                             int threads) {
  bool bad = false;
  for (int s = thread; s < sequences; s += threads) {
    const int a = starts[s], b = starts[s + 1];
    bad |= a < 0 || b < a || b > tokens;
  }
  if (bad) op_report(ws, kErrCapacity);
}

// The sequence that number `slot` belongs to, and which of its tiles it is; false for none.
// A whole warp looks, 32 sequences at a time.
__device__ __forceinline__ bool find_sequence(const int32_t* starts, int sequences, int tokens, int per, int unit,
                                              int64_t slot, PromptSequence* seq, int* tile) {
  int lo = 0, hi = sequences;  // the last s with slot(s) <= slot
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, probe = lo + (int)(threadIdx.x & 31) * step;
    bool below = false;
    if (probe < hi) {
      const int a = starts[probe];
      below = a <= tokens && (int64_t)(a > 0 ? a : 0) * per / unit + probe <= slot;
    }
    const int count = __popc(__ballot_sync(~0u, below));
    lo += (count > 1 ? count - 1 : 0) * step;
    hi = min(hi, lo + step);
  }
  const int a = starts[lo], b = starts[lo + 1];
  if (a < 0 || b < a || b > tokens) return false;
  const int64_t t = slot - ((int64_t)a * per / unit + lo);
  if (t < 0 || t * unit >= (int64_t)(b - a) * per) return false;
  seq->index = lo;
  seq->first = a;
  seq->length = seq->keys = b - a;
  seq->before = 0;
  *tile = (int)t;
  return true;
}

// The cached form: positions and keys from the request's length, of which the step's tokens are the last.
__device__ __forceinline__ void cached_sequence(const PromptArgs& a, PromptSequence* seq) {
  const int len = a.lens[seq->index];
  const int room = a.max_blocks << a.page_shift;
  if (len < 0 || len > room) op_report(a.ws, kErrCapacity);
  seq->before = (len < 0 ? 0 : len) - seq->length;
  seq->keys = len < 0 ? 0 : len < room ? len : room;
}

// The order in which a kernel's items are taken, where there are at most 32 sequences:
// those with the most work first, whatever sequence they are of. A warp steps through
// it, a lane a sequence. An item is `unit` tokens; its work is the keys that its last
// token sees, or (by_keys) the tokens that see its first one. (In the order of the
// numbers, sequences of different lengths left SMs with what they happened to get. The
// order alone took 8192 tokens of 17 sequences from 129 to 120 us, the gradient of 4097
// tokens of 9 from 165 to 151.)
struct ItemOrder {
  int first, length, before, keys;  // of the lane's sequence
  int items, left;                  // of them not taken
  int64_t taken;                    // of all sequences
  int last_sequence, last_tile;     // the last one taken

  __device__ __forceinline__ bool begin(const int32_t* starts, int sequences, int tokens, int unit) {
    first = length = before = keys = items = left = last_sequence = last_tile = 0;
    taken = 0;
    if (sequences > 32) return false;
    const int s = (int)(threadIdx.x & 31);
    if (s < sequences) {
      const int a = starts[s], b = starts[s + 1];
      if (a >= 0 && b >= a && b <= tokens) {
        first = a;
        length = keys = b - a;
        items = (length + unit - 1) / unit;
      }
    }
    left = items;
    return true;
  }
  // Item number n, none below the last one asked for; false if there are no more.
  __device__ __forceinline__ bool advance(int64_t n, int unit, bool by_keys, int* sequence, int* tile) {
    for (; taken <= n; taken++) {
      const int i = by_keys ? items - left : left - 1;
      const int work = left == 0 ? INT32_MIN : by_keys ? length - i * unit : min(before + min((i + 1) * unit, length), keys);
      const int most = __reduce_max_sync(~0u, work);
      if (__all_sync(~0u, left == 0)) return false;
      last_sequence = __ffs(__ballot_sync(~0u, left > 0 && work == most)) - 1;
      last_tile = __shfl_sync(~0u, i, last_sequence);
      if ((int)(threadIdx.x & 31) == last_sequence) left--;
    }
    *sequence = last_sequence;
    *tile = last_tile;
    return true;
  }
};

}  // namespace rar
