// prompt_attention_tc.cu -- attention over whole prompts in bf16 on the fifth-
// generation tensor cores, for head sizes up to 128 and up to 128 query heads a key head.
//
//   S = Q K^T,  P = 2^(scale log2(e) S - m),  O += P V,  l += row sums of P
//
// with the running maximum m of a row; out = O / l, lse = (m + log2 l) ln 2. A row is a
// query head of the group of a token, so a tile's 128 rows are floor(128 / group)
// tokens, and K and V are read once for all heads of the group.
//
// A block has two tiles of rows and walks over tiles of 128 keys. One warp copies (TMA),
// one issues products, and a warpgroup for each tile of rows turns S into P: a thread a
// row, so that the softmax needs no exchange between threads. While one tile's weights
// are being worked out, the other's products run. S and O are in tensor memory (2 x 128
// and 2 x head size columns); P takes the place of the S that it came from, as bf16, and
// is the left operand of P V from there. Weights are rounded to bf16 (2^-8 of
// themselves, in both directions): their sum l is of the unrounded ones, so the
// roundings average out over the keys and stay below the result's own.
//
// m moves only if a score is more than 8 above it (in base 2): weights up to 2^8 lose
// nothing in binary32, and O is read and rescaled for almost no tile. Products run in
// the order in which they are issued, so the S of the next tile that a warpgroup
// sees says that P V of the last one has been added too.
//
// Few rows over many keys (the verification of drafted tokens behind a long context)
// would leave most SMs idle: where the blocks would be fewer than half of the SMs, each
// tile's keys are split over several, which leave O, m and l unscaled as binary32, and
// the one that arrives last adds them up in the order of the keys.
#include <cstdio>

#include "prompt_attention.cuh"
#include "rar_launch.h"
#include "tensor_core.cuh"

namespace rar {
namespace {

using namespace tc;

constexpr int kThreads = 384;  // two softmax warpgroups, and one of which a warp copies and one issues products
// Registers: 384 threads start with 168 each, the third warpgroup leaves 96 of its own to the two others.
constexpr int kFewRegisters = 72, kManyRegisters = 216;
static_assert(kFewRegisters + 2 * kManyRegisters <= 3 * 168, "no more than the block was launched with");
constexpr int kRows = 128, kKeys = 128;
constexpr int kCopyWarp = 8, kProductWarp = 9;
constexpr float kLog2e = 1.4426950408889634f;

struct Maps {
  CUtensorMap q[kMaxRanks], k[kMaxRanks], v[kMaxRanks];
};

template <int DP>
struct Layout {
  static constexpr int kSlab = kRows * 128;              // 64 elements of 128 rows
  static constexpr int kTile = kSlab * (DP / 64);
  static constexpr int kStages = DP == 64 ? 8 : 4;       // tiles of keys or values
  static constexpr int kShared = (2 + kStages) * kTile + 1024;
};

__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(2 * kRows) : "memory"); }

struct Split {
  int parts;      // blocks that share a tile's keys
  float* sums;    // per block: 2 x 128 rows of DP binary32, then m and l of each
};

template <int DP, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) prompt_tc_kernel(const __grid_constant__ PromptArgs a,
                                                                const __grid_constant__ Maps maps, Split split) {
  using L = Layout<DP>;
  constexpr int NS = L::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (shared_address(raw) & 1023));
  __shared__ uint64_t q_full, full[NS], empty[NS], s_full[2], p_half[2], p_full[2], o_full[2];
  __shared__ uint32_t tmem_at, lost[4][4];
  __shared__ int dead_flag, last_flag;
  volatile int* const dead = &dead_flag;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    dead_flag = 0;
    barrier_init(&q_full, 1);
    for (int i = 0; i < NS; i++) {
      barrier_init(&full[i], 1);
      barrier_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      barrier_init(&s_full[i], 1);
      barrier_init(&p_half[i], kRows);
      barrier_init(&p_full[i], kRows);
      barrier_init(&o_full[i], 1);
    }
    barriers_ready();
  }
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_starts(a.starts, a.sequences, a.tokens, a.ws);
  const int group = a.q_heads / a.kv_heads, head = blockIdx.y, rank = blockIdx.z, D = a.head_dim;
  const int per_tile = kRows / group;  // tokens of a tile
  PromptSequence seq;
  int pair;
  // the last tokens of a sequence see the most keys: their blocks start first
  const int part = (int)(blockIdx.x % (unsigned)split.parts);
  const int64_t slot = (gridDim.x / (unsigned)split.parts) - 1 - blockIdx.x / (unsigned)split.parts;
  if (!find_sequence(a.starts, a.sequences, a.tokens, 1, 2 * per_tile, slot, &seq, &pair)) return;
  if (PAGED) cached_sequence(a, &seq);
  const int token0 = pair * 2 * per_tile;  // of the sequence
  int rows_of[2], tiles_of[2];             // tokens of each tile, and tiles of keys that its last one sees
#pragma unroll
  for (int t = 0; t < 2; t++) {
    rows_of[t] = max(0, min(per_tile, seq.length - token0 - t * per_tile));
    const int sees = min(seq.before + token0 + t * per_tile + rows_of[t], seq.keys);
    tiles_of[t] = rows_of[t] > 0 && sees > 0 ? (sees + kKeys - 1) / kKeys : 0;
  }
  const int tiles = max(tiles_of[0], tiles_of[1]);
  const int begin = (int)((int64_t)tiles * part / split.parts), end = (int)((int64_t)tiles * (part + 1) / split.parts);
  if (warp == kCopyWarp) tmem_alloc(&tmem_at, 512);
  __syncthreads();
  constexpr uint32_t tmem = 0;  // all of it, so it begins at 0
  constexpr uint32_t s_at[2] = {tmem, tmem + 128}, o_at[2] = {tmem + 256, tmem + 384};
  uint8_t* const ring = smem + 2 * L::kTile;
  const int steps = (D + 15) / 16;
  const int last[2] = {min(tiles_of[0], end), min(tiles_of[1], end)};  // a tile of rows walks from begin to here

  if (warp >= kCopyWarp) give_registers<kFewRegisters>();
  if (warp == kCopyWarp) {
    if (begin < end) {
      if (lane == 0) {
        prefetch_map(&maps.k[rank]);
        prefetch_map(&maps.v[rank]);
        const int boxes = (last[0] > begin) + (last[1] > begin);
        arrive_expect(&q_full, (uint32_t)(boxes * per_tile * group * 128 * (DP / 64)));
        for (int t = 0; t < 2; t++)
          if (last[t] > begin)
            for (int h = 0; h < DP / 64; h++)
              copy_3d(smem + t * L::kTile + h * L::kSlab, &maps.q[rank], h * 64, head * group,
                      seq.first + token0 + t * per_tile, &q_full);
      }
      int stage = 0;
      uint32_t phase = 0;
      bool fine = true;
      for (int j = begin; j < end && fine; j++) {
        int page = 0, box = kKeys;
        bool there = true;
        if (PAGED) box = min(kKeys, 1 << a.page_shift);
        uint32_t bad[4];
        for (int which = 0; which < 2 && fine; which++) {
          fine = wait(&empty[stage], phase ^ 1, dead);
          uint8_t* to = ring + stage * L::kTile;
          const CUtensorMap* map = which == 0 ? &maps.k[rank] : &maps.v[rank];
          if (!PAGED) {
            if (fine && lane == 0) {
              arrive_expect(&full[stage], L::kTile);
              for (int h = 0; h < DP / 64; h++)
                copy_3d(to + h * L::kSlab, map, h * 64, head, seq.first + j * kKeys, &full[stage]);
            }
          } else if (fine) {
            // a box a page (or 128 tokens of a larger one); boxes past the keys, and pages that are none, are not copied
            const int boxes = kKeys / box;
            if (which == 0) bad[0] = bad[1] = bad[2] = bad[3] = 0;
            int count = 0;
            for (int b0 = 0; b0 < boxes; b0 += 32) {
              const int b = b0 + lane, key = j * kKeys + b * box;
              const bool wanted = b < boxes && key < seq.keys;
              page = wanted ? a.table[seq.index * a.table_stride + (key >> a.page_shift)] : 0;
              there = wanted && (unsigned)page < (unsigned)a.num_pages;
              if (wanted && !there) op_report(a.ws, kErrCapacity);
              count += __popc(__ballot_sync(~0u, there));
              if (which == 0 && __any_sync(~0u, wanted && !there)) {
                for (int r = 0; r < 4; r++) {  // rows of the tile that such a page would have filled
                  uint32_t mine = 0;
                  if (wanted && !there)
                    for (int x = b * box; x < (b + 1) * box; x++)
                      if (x >> 5 == r) mine |= 1u << (x & 31);
                  bad[r] |= __reduce_or_sync(~0u, mine);
                }
              }
            }
            if (which == 0 && lane == 0)
              for (int r = 0; r < 4; r++) lost[j & 3][r] = bad[r];
            __syncwarp();
            if (lane == 0) arrive_expect(&full[stage], (uint32_t)(count * box * 128 * (DP / 64)));
            __syncwarp();
            for (int b0 = 0; b0 < boxes; b0 += 32) {
              const int b = b0 + lane, key = j * kKeys + b * box;
              const bool wanted = b < boxes && key < seq.keys;
              if (!wanted) continue;
              page = a.table[seq.index * a.table_stride + (key >> a.page_shift)];
              if ((unsigned)page >= (unsigned)a.num_pages) continue;
              for (int h = 0; h < DP / 64; h++)
                copy_3d(to + h * L::kSlab + b * box * 128, map, h * 64, key & ((1 << a.page_shift) - 1),
                        page * a.kv_heads + head, &full[stage]);
            }
          }
          if (++stage == NS) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == kProductWarp) {
    const int from = uniform(begin), to = uniform(end), upto[2] = {uniform(last[0]), uniform(last[1])}, keys_of = uniform(seq.keys);
    if (from < to) {
      const uint32_t lead = elect_one();
      const int n_out = steps * 16;
      const uint32_t q_at = shared_address(smem), ring_at = shared_address(ring);
      // the S of a key tile for a tile of rows that sees it
      auto score = [&](int t, uint32_t k_at) {
        rows_by_rows<DP / 16, L::kSlab>(lead, s_at[t], q_at + t * L::kTile, k_at, kKeys, steps);
        commit(lead, &s_full[t]);
      };
      // V of key tile j is there; rows with no key would be multiplied by weights of 0, and may hold a NaN
      auto values = [&](int j, int stage, uint32_t phase) {
        if (!wait_warp(&full[stage], phase, dead)) return false;
        const int keys = keys_of - j * kKeys;
        const bool holes = PAGED && __any_sync(~0u, lane < 4 && lost[j & 3][lane & 3] != 0);
        if (keys < kKeys || holes) {
          for (int r = lane; r < kKeys; r += 32)
            if (r >= keys || (holes && (lost[j & 3][r >> 5] >> (r & 31) & 1)))
              for (int h = 0; h < DP / 64; h++)
                for (int c = 0; c < 8; c++)
                  *reinterpret_cast<uint4*>(ring + stage * L::kTile + h * L::kSlab + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
          stores_to_products();
          __syncwarp();
        }
        return true;
      };
      // stages: K of the first tile, then V of a tile and K of the next in turn
      bool fine = wait_warp(&q_full, 0, dead) && wait_warp(&full[0], 0, dead);
      if (fine) {
        fence_after();
        for (int t = 0; t < 2; t++)
          if (upto[t] > from) score(t, ring_at);
        commit(lead, &empty[0]);
        fine = values(from, 1, 0);
      }
      int v_stage = 1;
      uint32_t v_phase = 0;
      for (int j = from; j < to && fine; j++) {
        const bool more = j + 1 < to;
        const int k_stage = v_stage + 1 == NS ? 0 : v_stage + 1;
        const uint32_t k_phase = v_phase ^ (k_stage == 0);
        const int next_stage = k_stage + 1 == NS ? 0 : k_stage + 1;
        const uint32_t next_phase = k_phase ^ (next_stage == 0);
#pragma unroll
        for (int t = 0; t < 2; t++) {
          if (j < upto[t]) {
            if (!(fine = wait_warp(&p_half[t], (j - from) & 1, dead))) break;
            fence_after();
            weights_by_rows<L::kSlab, 0, 0, 4>(lead, o_at[t], s_at[t], ring_at + v_stage * L::kTile, n_out, j > from);
            if (!(fine = wait_warp(&p_full[t], (j - from) & 1, dead))) break;
            fence_after();
            weights_by_rows<L::kSlab, 0, 4, 8>(lead, o_at[t], s_at[t], ring_at + v_stage * L::kTile, n_out, true);
            if (j + 1 >= upto[t]) commit(lead, &o_full[t]);
          }
          // what the warp waits for beside the weights, it waits for while products run
          if (more && t == 0 && !(fine = wait_warp(&full[k_stage], k_phase, dead))) break;
          if (more && t == 1 && !(fine = values(j + 1, next_stage, next_phase))) break;
          if (j + 1 < upto[t]) {
            fence_after();
            score(t, ring_at + k_stage * L::kTile);
          }
        }
        if (!fine) break;
        commit(lead, &empty[v_stage]);
        if (more) commit(lead, &empty[k_stage]);
        v_stage = next_stage;
        v_phase = next_phase;
      }
    }
  } else if (warp < kCopyWarp) {
    take_registers<kManyRegisters>();
    const int t = warp >> 2;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
    const int row = threadIdx.x & 127, token = row / group, query = head * group + row % group;
    const bool mine = token < rows_of[t];
    const int64_t at_token = (int64_t)seq.first + token0 + t * per_tile + token;
    // rows that are none see what the tile's first row sees: they hold anything, and nobody reads them
    const int sees = min(seq.before + token0 + t * per_tile + (mine ? token : 0) + 1, seq.keys);
    int least = sees;  // of the warp
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) least = min(least, __shfl_xor_sync(~0u, least, d));
    // of a negative scale or none, the scores are turned or cleared first, so that the largest is the one that counts
    const float scale2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
    const uint32_t turn = a.scale < 0.f ? 0x80000000u : 0u, keep_bits = a.scale == 0.f ? 0u : ~0u;
    float m = -INFINITY, l = 0.f;
    bool fine = true;
    for (int j = begin; j < last[t] && fine; j++) {
      if (!(fine = wait(&s_full[t], (j - begin) & 1, dead))) break;
      fence_after();
      uint32_t s[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) tmem_load32(s_at[t] + quarter + c, s + c);
      loads_done();
      if (!(a.scale > 0.f)) {
#pragma unroll
        for (int c = 0; c < kKeys; c++) s[c] = (s[c] ^ turn) & keep_bits;
      }
      const bool holes = PAGED && (lost[j & 3][0] | lost[j & 3][1] | lost[j & 3][2] | lost[j & 3][3]) != 0;
      if ((j + 1) * kKeys > least || holes) {
        const int upto = sees - j * kKeys;
#pragma unroll
        for (int c = 0; c < kKeys; c++) {
          bool seen = c < upto;
          if (PAGED && holes) seen = seen && !(lost[j & 3][c >> 5] >> (c & 31) & 1);
          if (!seen) s[c] = 0xff800000u;
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
#pragma unroll
      for (int h = 0; h < 2; h++) {
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
        }
        tmem_store32(s_at[t] + quarter + 32 * h, s + 32 * h);
        stores_done();
        fence_before();
        arrive(h == 0 ? &p_half[t] : &p_full[t]);
      }
      const float2 u = unpack(add2(sum, more));
      l += u.x + u.y;
    }
    const bool some = last[t] > begin;  // O has been written
    if (fine && some) {
      fine = wait(&o_full[t], 0, dead);
      fence_after();
    }
    if (fine && split.parts == 1) {
      const float by = l == 0.f ? 0.f : 1.f / l;
      uint16_t* out = (uint16_t*)a.out[rank] + at_token * a.out_stride + (int64_t)query * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (some) {
          tmem_load32(o_at[t] + quarter + c, o);
          loads_done();
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            if (c + i >= D) continue;
            Pack8<uint16_t> x;
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; k++) v[k] = l == 0.f ? 0.f : __uint_as_float(o[i + k]) * by;
            x.narrow(v);
            x.store(out + c + i);
          }
        }
      }
      if (mine && a.lse[rank] != nullptr) a.lse[rank][at_token * a.q_heads + query] = (m + log2f(l)) / kLog2e;
    } else if (fine) {
      // a part of the keys: O, m and l as they are
      const int64_t item = ((int64_t)rank * a.kv_heads + head) * (gridDim.x / (unsigned)split.parts) + slot;
      float* mine_at = split.sums + (item * split.parts + part) * (int64_t)(2 * kRows * (DP + 2)) + t * kRows * (DP + 2);
      mine_at[kRows * DP + row] = m;
      mine_at[kRows * (DP + 1) + row] = l;
      if (some) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_load32(o_at[t] + quarter + c, o);
          loads_done();
          if (!mine) continue;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            if (c + i < D)
              *reinterpret_cast<uint4*>(mine_at + row * DP + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
    }
    fence_before();
    if (split.parts > 1) {
      // the block that arrives last has every part of the tile
      const int64_t item = ((int64_t)rank * a.kv_heads + head) * (gridDim.x / (unsigned)split.parts) + slot;
      __threadfence();
      softmax_barrier();
      if (threadIdx.x == 0) {
        uint32_t* counter = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes) + item;
        last_flag = atom_add_acq_rel_u32(counter, 1) == (uint32_t)split.parts - 1;
        if (last_flag) *counter = 0;
      }
      softmax_barrier();
      if (last_flag && !*dead) {
        __threadfence();
        const float* parts = split.sums + item * split.parts * (int64_t)(2 * kRows * (DP + 2));
        const int chunks = D / 8;
        for (int i = threadIdx.x; i < 2 * kRows * chunks; i += 2 * kRows) {
          const int r = i / chunks, d = (i % chunks) * 8, u = r / kRows, row = r % kRows, token = row / group;
          if (token >= rows_of[u]) continue;
          float top = -INFINITY, sum = 0.f, v[8] = {};
          for (int k = 0; k < split.parts; k++)
            top = fmaxf(top, parts[(int64_t)(2 * k + u) * kRows * (DP + 2) + kRows * DP + row]);
          for (int k = 0; k < split.parts && top != -INFINITY; k++) {
            const float* p = parts + (int64_t)(2 * k + u) * kRows * (DP + 2);
            const float m = p[kRows * DP + row];
            if (m == -INFINITY) continue;
            const float w = exp2_fast(m - top);
            sum = fmaf(p[kRows * (DP + 1) + row], w, sum);
#pragma unroll
            for (int x = 0; x < 8; x++) v[x] = fmaf(p[row * DP + d + x], w, v[x]);
          }
          const int64_t at_token = (int64_t)seq.first + token0 + u * per_tile + token;
          const int query = head * group + row % group;
#pragma unroll
          for (int x = 0; x < 8; x++) v[x] = sum == 0.f ? 0.f : v[x] / sum;
          Pack8<uint16_t> out;
          out.narrow(v);
          out.store((uint16_t*)a.out[rank] + at_token * a.out_stride + (int64_t)query * D + d);
          if (d == 0 && a.lse[rank] != nullptr) a.lse[rank][at_token * a.q_heads + query] = (top + log2f(sum)) / kLog2e;
        }
      }
    }
  }
  __syncthreads();
  if (*dead) {
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

template <int DP, bool PAGED>
cudaError_t launch(const PromptArgs& a, cudaStream_t stream) {
  const int group = a.q_heads / a.kv_heads, per_tile = kRows / group, D = a.head_dim;
  const void* fn = (const void*)prompt_tc_kernel<DP, PAGED>;
  int blocks = 0;
  cudaError_t e = resident_blocks(fn, kThreads, Layout<DP>::kShared, &blocks);
  if (e != cudaSuccess) return e;
  static thread_local Maps maps;
  for (int r = 0; r < a.nranks && e == cudaSuccess; r++) {
    e = make_map(&maps.q[r], a.q[r], D, a.q_heads, a.tokens, D * 2, a.q_stride * 2, group, per_tile);
    for (int which = 0; which < 2 && e == cudaSuccess; which++) {
      CUtensorMap* map = which == 0 ? &maps.k[r] : &maps.v[r];
      const void* base = which == 0 ? a.k[r] : a.v[r];
      const int page = 1 << a.page_shift;
      e = PAGED ? make_map(map, base, D, page, (int64_t)a.num_pages * a.kv_heads, D * 2, (int64_t)page * D * 2,
                           page < kKeys ? page : kKeys, 1)
                : make_map(map, base, D, a.kv_heads, a.tokens, D * 2, (which == 0 ? a.k_stride : a.v_stride) * 2, 1, kKeys);
    }
  }
  if (e != cudaSuccess) return e;
  const int64_t slots = prompt_slots(a.tokens, a.sequences, 1, 2 * per_tile);
  const int64_t items = slots * a.kv_heads * a.nranks;
  // most keys that a tile may see, in tiles
  const int64_t most = div_up(PAGED ? (int64_t)a.max_blocks << a.page_shift : a.tokens, kKeys);
  Split split = {1, (float*)(a.ws + kOpScratchOffset)};
  if (items * 2 <= kPromptSplitBlocks) {
    const int64_t room = kPromptSplitBlocks / items;
    split.parts = (int)(room < div_up(most, 2) ? room : div_up(most, 2));
    if (split.parts < 1) split.parts = 1;
  }
  PromptArgs copy = a;
  void* params[] = {&copy, &maps, &split};
  return launch_op(fn, dim3((unsigned)(slots * split.parts), (unsigned)a.kv_heads, (unsigned)a.nranks), kThreads,
                   Layout<DP>::kShared, stream, params);
}

}  // namespace

cudaError_t launch_prompt_attention_tc(const PromptArgs& a, cudaStream_t stream) {
  const bool paged = a.table != nullptr;
  if (a.head_dim <= 64) return paged ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  return paged ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace rar
