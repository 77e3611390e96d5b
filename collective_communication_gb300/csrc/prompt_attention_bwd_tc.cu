// prompt_attention_bwd_tc.cu -- the gradient of the attention over whole prompts in
// bf16 on the fifth-generation tensor cores, for head sizes up to 128 and up to 128
// query heads a key head.
//
//   P = 2^(scale log2(e) Q K^T - lse log2(e)),  dS = P (dO V^T - delta),  delta = O . dO
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two kernels that both recompute P: one by rows for dQ (three products a tile, and
// delta, which it leaves for the other), one by keys for dK and dV (four). One kernel
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
// Two warpgroups work out the weights, half of the columns each: a thread has 64
// columns of a row. The products' order keeps the tensor cores busy meanwhile:
//   rows:  S(j+1) | dS(j) ready: dP(j+1), dQ += dS(j) K(j) | ...
//   keys:  P(i) ready: dV += P(i) dO, S(i+1) | dS(i) ready: dK += dS(i) Q, dP(i+1) | ...
#include <cstdio>

#include "prompt_attention.cuh"
#include "rar_launch.h"
#include "tensor_core.cuh"

namespace rar {
namespace {

using namespace tc;

constexpr int kThreads = 384;  // two warpgroups for the weights; warps for copies, products, rows' numbers; one is idle
constexpr int kTile = 128;     // rows, and keys
constexpr int kCopyWarp = 8, kProductWarp = 9, kNumbersWarp = 10;
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

// Rows from `first` on of a tile in shared memory become 0, before products run over them; one warp.
template <int DP>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int first) {
  for (int r = first * 8 + (threadIdx.x & 31); r < kTile * 8; r += 32)
    for (int h = 0; h < DP / 64; h++) *reinterpret_cast<uint4*>(tile + h * Layout<DP>::kSlab + r * 16) = make_uint4(0, 0, 0, 0);
}

// A row of sums from tensor memory, half of its elements each for the two warpgroups, scaled and rounded.
template <int DP>
__device__ __forceinline__ void store_half(uint32_t at, int half, float by, bool mine, uint16_t* row, int D) {
#pragma unroll 1
  for (int c = half * (DP / 2); c < (half + 1) * (DP / 2) && c < D; c += 32) {
    uint32_t o[32];
    tmem_load32(at + c, o);
    loads_done();
    if (!mine) continue;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      if (c + i >= D) continue;
      Pack8<uint16_t> x;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] = __uint_as_float(o[i + k]) * by;
      x.narrow(v);
      x.store(row + c + i);
    }
  }
}

__device__ __forceinline__ void end_block(char* ws, volatile int* dead, int warp, uint32_t tmem) {
  fence_before();
  __syncthreads();
  if (*dead) {
    // a wait ran out: copies and products that are still under way have ended by the time this has passed
    const uint64_t until = global_timer_ns() + 10000000ull;
    while (global_timer_ns() < until) {}
    if (threadIdx.x == 0) op_report(ws, kErrTimeout);
  }
  __syncthreads();
  if (warp == kCopyWarp) {
    fence_after();
    tmem_free(tmem, 512);
  }
}

__device__ __forceinline__ void weights_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) prompt_rows_tc_kernel(const __grid_constant__ PromptBwdArgs a,
                                                                     const __grid_constant__ Maps maps) {
  using L = Layout<DP>;
  constexpr int KS = L::kKeyStages, VS = L::kValueStages;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (shared_address(raw) & 1023));
  __shared__ uint64_t q_full, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], dp_full, ds_ready, dq_full;
  __shared__ uint32_t tmem_at;
  __shared__ int dead_flag;
  __shared__ float half_delta[kTile];
  volatile int* const dead = &dead_flag;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    dead_flag = 0;
    barrier_init(&q_full, 1);
    for (int i = 0; i < KS; i++) {
      barrier_init(&k_full[i], 1);
      barrier_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; i++) {
      barrier_init(&v_full[i], 1);
      barrier_init(&v_empty[i], 1);
    }
    barrier_init(&dp_full, 1);
    barrier_init(&ds_ready, 2 * kTile);
    barrier_init(&dq_full, 1);
    barriers_ready();
  }
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_starts(a.starts, a.sequences, a.tokens, a.ws);
  const int group = a.q_heads / a.kv_heads, head = blockIdx.y, rank = blockIdx.z, D = a.head_dim;
  const int per_tile = kTile / group;
  PromptSequence seq;
  int tile;
  // the last rows of a sequence see the most keys: they start first
  if (!find_sequence(a.starts, a.sequences, a.tokens, 1, per_tile, (int64_t)gridDim.x - 1 - blockIdx.x, &seq, &tile)) return;
  const int token0 = tile * per_tile, tokens = min(per_tile, seq.length - token0);
  const int tiles = (token0 + tokens + kTile - 1) / kTile;
  if (warp == kCopyWarp) tmem_alloc(&tmem_at, 512);
  __syncthreads();
  constexpr uint32_t tmem = 0;  // all of it, so it begins at 0
  constexpr uint32_t s_at = tmem, dp_at = tmem + 256, dq_at = tmem + 384;  // S: two buffers of 128 columns
  uint8_t *const q_tile = smem, *const g_tile = smem + L::kBytes, *const k_ring = smem + 2 * L::kBytes,
          *const v_ring = k_ring + KS * L::kBytes;
  const int steps = (D + 15) / 16;

  if (warp == kCopyWarp) {
    if (lane == 0) {
      arrive_expect(&q_full, (uint32_t)(2 * per_tile * group * 128 * (DP / 64)));
      for (int h = 0; h < DP / 64; h++) {
        copy_3d(q_tile + h * L::kSlab, &maps.q[rank], h * 64, head * group, seq.first + token0, &q_full);
        copy_3d(g_tile + h * L::kSlab, &maps.dout[rank], h * 64, head * group, seq.first + token0, &q_full);
      }
      for (int j = 0; j < tiles; j++) {
        if (!wait(&k_empty[j % KS], (j / KS & 1) ^ 1, dead)) break;
        arrive_expect(&k_full[j % KS], L::kBytes);
        for (int h = 0; h < DP / 64; h++)
          copy_3d(k_ring + j % KS * L::kBytes + h * L::kSlab, &maps.k[rank], h * 64, head, seq.first + j * kTile, &k_full[j % KS]);
        if (!wait(&v_empty[j % VS], (j / VS & 1) ^ 1, dead)) break;
        arrive_expect(&v_full[j % VS], L::kBytes);
        for (int h = 0; h < DP / 64; h++)
          copy_3d(v_ring + j % VS * L::kBytes + h * L::kSlab, &maps.v[rank], h * 64, head, seq.first + j * kTile, &v_full[j % VS]);
      }
    }
  } else if (warp == kProductWarp) {
    const uint32_t q_at = shared_address(q_tile), g_at = shared_address(g_tile), k_at = shared_address(k_ring),
                   v_at = shared_address(v_ring);
    const uint32_t lead = elect_one();
    const int count = uniform(tiles), keys_of = uniform(seq.length);
    auto score = [&](int j) {  // S of key tile j; keys that are none are 0, for the product with dS
      if (!wait_warp(&k_full[j % KS], j / KS & 1, dead)) return false;
      if (keys_of - j * kTile < kTile) {
        clear_rows<DP>(k_ring + j % KS * L::kBytes, keys_of - j * kTile);
        stores_to_products();
        __syncwarp();
      }
      fence_after();
      rows_by_rows<DP / 16, L::kSlab>(lead, s_at + (j & 1) * 128, q_at, k_at + j % KS * L::kBytes, kTile, steps);
      return true;
    };
    auto value = [&](int j) {  // dO V^T
      if (!wait_warp(&v_full[j % VS], j / VS & 1, dead)) return false;
      fence_after();
      rows_by_rows<DP / 16, L::kSlab>(lead, dp_at, g_at, v_at + j % VS * L::kBytes, kTile, steps);
      commit(lead, &dp_full);
      commit(lead, &v_empty[j % VS]);
      return true;
    };
    bool fine = wait_warp(&q_full, 0, dead) && score(0) && value(0);
    for (int j = 0; j < count && fine; j++) {
      const bool more = j + 1 < count;
      if (more && !(fine = score(j + 1))) break;
      if (!(fine = wait_warp(&ds_ready, j & 1, dead))) break;
      fence_after();
      if (more && !(fine = value(j + 1))) break;
      weights_by_rows<32>(lead, dq_at, s_at + (j & 1) * 128, k_at + j % KS * L::kBytes, steps * 16, j > 0, L::kSlab);
      commit(lead, &k_empty[j % KS]);
      if (!more) commit(lead, &dq_full);
    }
  } else if (warp < kCopyWarp) {
    const int half = warp >> 2;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;
    const int row = threadIdx.x & 127, token = row / group, query = head * group + row % group;
    const bool mine = token < tokens;
    const int64_t at_token = (int64_t)seq.first + token0 + token, at = at_token * a.q_heads + query;
    // delta, half of the elements each
    float delta = 0.f, lse2 = 0.f;
    if (mine) {
      const uint16_t* o = (const uint16_t*)a.out[rank] + at_token * a.out_stride + (int64_t)query * D;
      const uint16_t* g = (const uint16_t*)a.dout[rank] + at_token * a.dout_stride + (int64_t)query * D;
#pragma unroll 4
      for (int d = half * (DP / 2); d < (half + 1) * (DP / 2); d += 8) {
        if (d >= D) break;
        Pack8<uint16_t> x, y;
        float u[8], v[8];
        x.load(o + d);
        y.load(g + d);
        x.widen(u);
        y.widen(v);
#pragma unroll
        for (int i = 0; i < 8; i++) delta = fmaf(u[i], v[i], delta);
      }
      lse2 = a.lse[rank][at] * kLog2e;
    }
    if (half == 1) half_delta[row] = delta;
    weights_barrier();
    if (half == 0) {
      delta += half_delta[row];
      if (mine) reinterpret_cast<float*>(a.ws + kOpScratchOffset)[(int64_t)rank * a.tokens * a.q_heads + at] = delta;
    }
    weights_barrier();
    if (half == 0) half_delta[row] = delta;
    weights_barrier();
    delta = half_delta[row];
    const int sees = token0 + (mine ? token : 0) + 1;
    int least = sees;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) least = min(least, __shfl_xor_sync(~0u, least, d));
    const F2 scale_pair = f2(a.scale * kLog2e, a.scale * kLog2e), lse_pair = f2(-lse2, -lse2), delta_pair = f2(-delta, -delta);
    bool fine = true;
    for (int j = 0; j < tiles; j++) {
      if (!(fine = wait(&dp_full, j & 1, dead))) break;  // S of the tile was issued ahead of it
      fence_after();
      const uint32_t from = s_at + (j & 1) * 128 + quarter + half * 64;
      uint32_t s[64], dp[64];
      tmem_load32(from, s);
      tmem_load32(from + 32, s + 32);
      tmem_load32(dp_at + quarter + half * 64, dp);
      tmem_load32(dp_at + quarter + half * 64 + 32, dp + 32);
      loads_done();
      const int upto = sees - j * kTile - half * 64;
      const bool cut = (j + 1) * kTile > least;
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        float2 p = unpack(fma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale_pair, lse_pair));
        p.x = exp2_fast(p.x);
        p.y = exp2_fast(p.y);
        const F2 d = add2(f2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])), delta_pair);
        const float2 ds = unpack(mul2(f2(p.x, p.y), d));
        s[c / 2] = bf16_pair(!cut || c < upto ? ds.x : 0.f, !cut || c + 1 < upto ? ds.y : 0.f);
      }
      tmem_store32(from, s);
      stores_done();
      fence_before();
      arrive(&ds_ready);
    }
    if (fine && wait(&dq_full, 0, dead)) {
      fence_after();
      store_half<DP>(dq_at + quarter, half, a.scale, mine, (uint16_t*)a.dq[rank] + at_token * a.dq_stride + (int64_t)query * D, D);
    }
  }
  __syncwarp();
  end_block(a.ws, dead, warp, tmem);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) prompt_keys_tc_kernel(const __grid_constant__ PromptBwdArgs a,
                                                                     const __grid_constant__ Maps maps) {
  using L = Layout<DP>;
  constexpr int NS = L::kRowStages;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (shared_address(raw) & 1023));
  __shared__ uint64_t kv_full, full[NS], empty[NS], s_full, p_ready, dp_full, ds_ready, done;
  __shared__ uint32_t tmem_at;
  __shared__ int dead_flag;
  __shared__ __align__(16) float numbers[NS][2][kTile];  // -lse log2(e) and -delta of a tile's rows
  __shared__ uint8_t token_of[kTile];
  volatile int* const dead = &dead_flag;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int group = a.q_heads / a.kv_heads;
  if (threadIdx.x == 0) {
    dead_flag = 0;
    barrier_init(&kv_full, 1);
    for (int i = 0; i < NS; i++) {
      barrier_init(&full[i], 1 + 32);
      barrier_init(&empty[i], 1 + 2 * kTile);
    }
    barrier_init(&s_full, 1);
    barrier_init(&p_ready, 2 * kTile);
    barrier_init(&dp_full, 1);
    barrier_init(&ds_ready, 2 * kTile);
    barrier_init(&done, 1);
    barriers_ready();
  }
  if (threadIdx.x < kTile) token_of[threadIdx.x] = (uint8_t)(threadIdx.x / group);
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int head = blockIdx.y, rank = blockIdx.z, D = a.head_dim;
  const int per_tile = kTile / group;
  PromptSequence seq;
  int tile;
  // the first keys of a sequence are seen by the most rows: they start first
  if (!find_sequence(a.starts, a.sequences, a.tokens, 1, kTile, blockIdx.x, &seq, &tile)) return;
  const int key0 = tile * kTile, keys = min(kTile, seq.length - key0);
  const int begin = key0 / per_tile, end = (seq.length + per_tile - 1) / per_tile;  // tiles of rows
  if (warp == kCopyWarp) tmem_alloc(&tmem_at, 512);
  __syncthreads();
  constexpr uint32_t tmem = 0;  // all of it, so it begins at 0
  constexpr uint32_t s_at = tmem, dp_at = tmem + 128, dv_at = tmem + 256, dk_at = tmem + 384;
  uint8_t *const k_tile = smem, *const v_tile = smem + L::kBytes, *const ring = smem + 2 * L::kBytes;  // a stage: Q, dO
  const int steps = (D + 15) / 16;

  if (warp == kCopyWarp) {
    if (lane == 0) {
      arrive_expect(&kv_full, 2 * L::kBytes);
      for (int h = 0; h < DP / 64; h++) {
        copy_3d(k_tile + h * L::kSlab, &maps.k[rank], h * 64, head, seq.first + key0, &kv_full);
        copy_3d(v_tile + h * L::kSlab, &maps.v[rank], h * 64, head, seq.first + key0, &kv_full);
      }
      for (int i = begin; i < end; i++) {
        const int n = i - begin, stage = n % NS;
        if (!wait(&empty[stage], (n / NS & 1) ^ 1, dead)) break;
        arrive_expect(&full[stage], (uint32_t)(2 * per_tile * group * 128 * (DP / 64)));
        for (int h = 0; h < DP / 64; h++) {
          copy_3d(ring + stage * 2 * L::kBytes + h * L::kSlab, &maps.q[rank], h * 64, head * group, seq.first + i * per_tile,
                  &full[stage]);
          copy_3d(ring + (stage * 2 + 1) * L::kBytes + h * L::kSlab, &maps.dout[rank], h * 64, head * group,
                  seq.first + i * per_tile, &full[stage]);
        }
      }
    }
  } else if (warp == kNumbersWarp) {
    const float* deltas = reinterpret_cast<const float*>(a.ws + kOpScratchOffset) + (int64_t)rank * a.tokens * a.q_heads;
    float l[4], d[4];
    auto read = [&](int i) {
#pragma unroll
      for (int x = 0; x < 4; x++) {
        const int r = lane + 32 * x, token = i * per_tile + r / group;
        const bool there = r / group < per_tile && token < seq.length && i < end;
        const int64_t at = ((int64_t)seq.first + token) * a.q_heads + head * group + r % group;
        l[x] = there ? a.lse[rank][at] * -kLog2e : 0.f;
        d[x] = there ? -deltas[at] : 0.f;
      }
    };
    read(begin);
    for (int i = begin; i < end; i++) {
      const int n = i - begin, stage = n % NS;
      if (!wait(&empty[stage], (n / NS & 1) ^ 1, dead)) break;
#pragma unroll
      for (int x = 0; x < 4; x++) {
        numbers[stage][0][lane + 32 * x] = l[x];
        numbers[stage][1][lane + 32 * x] = d[x];
      }
      arrive(&full[stage]);
      read(i + 1);
    }
  } else if (warp == kProductWarp) {
    const uint32_t k_at = shared_address(k_tile), v_at = shared_address(v_tile), ring_at = shared_address(ring);
    const uint32_t lead = elect_one();
    const int from = uniform(begin), to = uniform(end), tokens_of = uniform(seq.length);
    auto score = [&](int i) {  // S^T of a tile of rows; rows that are none are 0, for the products with P and dS
      const int n = i - from, stage = n % NS;
      if (!wait_warp(&full[stage], n / NS & 1, dead)) return false;
      const int rows = min(per_tile, tokens_of - i * per_tile) * group;
      if (rows < kTile) {
        clear_rows<DP>(ring + stage * 2 * L::kBytes, rows);
        clear_rows<DP>(ring + (stage * 2 + 1) * L::kBytes, rows);
        stores_to_products();
        __syncwarp();
      }
      fence_after();
      rows_by_rows<DP / 16, L::kSlab>(lead, s_at, k_at, ring_at + stage * 2 * L::kBytes, kTile, steps);
      commit(lead, &s_full);
      return true;
    };
    auto value = [&](int i) {  // V dO^T
      rows_by_rows<DP / 16, L::kSlab>(lead, dp_at, v_at, ring_at + ((i - from) % NS * 2 + 1) * L::kBytes, kTile, steps);
      commit(lead, &dp_full);
    };
    bool fine = wait_warp(&kv_full, 0, dead) && score(from);
    if (fine) value(from);
    for (int i = from; i < to && fine; i++) {
      const int n = i - from, stage = n % NS;
      const bool more = i + 1 < to;
      if (!(fine = wait_warp(&p_ready, n & 1, dead))) break;
      fence_after();
      weights_by_rows<32>(lead, dv_at, s_at, ring_at + (stage * 2 + 1) * L::kBytes, steps * 16, n > 0, L::kSlab);
      if (more && !(fine = score(i + 1))) break;
      if (!(fine = wait_warp(&ds_ready, n & 1, dead))) break;
      fence_after();
      weights_by_rows<32>(lead, dk_at, dp_at, ring_at + stage * 2 * L::kBytes, steps * 16, n > 0, L::kSlab);
      commit(lead, &empty[stage]);
      if (!more) commit(lead, &done);
      if (more) value(i + 1);
    }
  } else if (warp < kCopyWarp) {
    const int half = warp >> 2;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;
    const int row = threadIdx.x & 127;
    const bool mine = row < keys;
    const int key = key0 + row;
    const F2 scale_pair = f2(a.scale * kLog2e, a.scale * kLog2e);
    bool fine = true;
    for (int i = begin; i < end; i++) {
      const int n = i - begin, stage = n % NS;
      if (!(fine = wait(&full[stage], n / NS & 1, dead))) break;  // the rows' numbers
      if (!(fine = wait(&s_full, n & 1, dead))) break;
      fence_after();
      const uint32_t from = s_at + quarter + half * 64, dp_from = dp_at + quarter + half * 64;
      uint32_t s[64], w[32];
      tmem_load32(from, s);
      tmem_load32(from + 32, s + 32);
      loads_done();
      const int rows = min(per_tile, seq.length - i * per_tile) * group;
      const bool cut = rows < kTile || i * per_tile < key0 + kTile - 1;
      const float4* l = reinterpret_cast<const float4*>(numbers[stage][0] + half * 64);
      const float4* d = reinterpret_cast<const float4*>(numbers[stage][1] + half * 64);
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 x = l[c / 4];
        float2 p = unpack(fma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale_pair, f2(x.x, x.y)));
        float2 q = unpack(fma2(f2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), scale_pair, f2(x.z, x.w)));
        p.x = exp2_fast(p.x);
        p.y = exp2_fast(p.y);
        q.x = exp2_fast(q.x);
        q.y = exp2_fast(q.y);
        if (cut) {
          auto seen = [&](int u) {
            const int r = half * 64 + c + u;
            return r < rows && i * per_tile + token_of[r] >= key;
          };
          p.x = seen(0) ? p.x : 0.f;
          p.y = seen(1) ? p.y : 0.f;
          q.x = seen(2) ? q.x : 0.f;
          q.y = seen(3) ? q.y : 0.f;
        }
        s[c] = __float_as_uint(p.x);
        s[c + 1] = __float_as_uint(p.y);
        s[c + 2] = __float_as_uint(q.x);
        s[c + 3] = __float_as_uint(q.y);
        w[c / 2] = bf16_pair(p.x, p.y);
        w[c / 2 + 1] = bf16_pair(q.x, q.y);
      }
      tmem_store32(from, w);
      stores_done();
      fence_before();
      arrive(&p_ready);
      if (!(fine = wait(&dp_full, n & 1, dead))) break;
      fence_after();
#pragma unroll
      for (int b = 0; b < 64; b += 32) {
        uint32_t g[32];
        tmem_load32(dp_from + b, g);
        loads_done();
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 x = d[(b + c) / 4];
          const float2 u = unpack(mul2(f2(__uint_as_float(s[b + c]), __uint_as_float(s[b + c + 1])),
                                       add2(f2(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), f2(x.x, x.y))));
          const float2 v = unpack(mul2(f2(__uint_as_float(s[b + c + 2]), __uint_as_float(s[b + c + 3])),
                                       add2(f2(__uint_as_float(g[c + 2]), __uint_as_float(g[c + 3])), f2(x.z, x.w))));
          w[(b + c) / 2] = bf16_pair(u.x, u.y);
          w[(b + c) / 2 + 1] = bf16_pair(v.x, v.y);
        }
      }
      tmem_store32(dp_from, w);
      stores_done();
      fence_before();
      arrive(&ds_ready);
      arrive(&empty[stage]);  // the rows' numbers have been read
    }
    if (fine && wait(&done, 0, dead)) {
      fence_after();
      const int64_t token = (int64_t)seq.first + key, at = (int64_t)head * D;
      store_half<DP>(dk_at + quarter, half, a.scale, mine, (uint16_t*)a.dk[rank] + token * a.dk_stride + at, D);
      store_half<DP>(dv_at + quarter, half, 1.f, mine, (uint16_t*)a.dv[rank] + token * a.dv_stride + at, D);
    }
  }
  __syncwarp();
  end_block(a.ws, dead, warp, tmem);
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
    e = make_map(&maps.q[r], a.q[r], D, a.q_heads, a.tokens, D * 2, a.q_stride * 2, group, per_tile);
    if (e == cudaSuccess)
      e = make_map(&maps.dout[r], a.dout[r], D, a.q_heads, a.tokens, D * 2, a.dout_stride * 2, group, per_tile);
    if (e == cudaSuccess) e = make_map(&maps.k[r], a.k[r], D, a.kv_heads, a.tokens, D * 2, a.k_stride * 2, 1, kTile);
    if (e == cudaSuccess) e = make_map(&maps.v[r], a.v[r], D, a.kv_heads, a.tokens, D * 2, a.v_stride * 2, 1, kTile);
  }
  if (e != cudaSuccess) return e;
  PromptBwdArgs copy = a;
  void* params[] = {&copy, &maps};
  e = launch_op(rows, dim3((unsigned)prompt_slots(a.tokens, a.sequences, 1, per_tile), (unsigned)a.kv_heads, (unsigned)a.nranks),
                kThreads, Layout<DP>::kRowsShared, stream, params);
  if (e != cudaSuccess) return e;
  return launch_op(keys, dim3((unsigned)prompt_slots(a.tokens, a.sequences, 1, kTile), (unsigned)a.kv_heads, (unsigned)a.nranks),
                   kThreads, Layout<DP>::kKeysShared, stream, params);
}

}  // namespace

cudaError_t launch_prompt_attention_bwd_tc(const PromptBwdArgs& a, cudaStream_t stream) {
  return a.head_dim <= 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace rar
