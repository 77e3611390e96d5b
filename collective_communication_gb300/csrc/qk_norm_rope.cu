// qk_norm_rope.cu -- root-mean-square norm of every query and key head with the
// rotary position in the same pass, and its gradient.
//
//   y = R(pos) (x * r * w),  r = 1 / sqrt(mean(x^2) + eps)
// R turns the pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved, of the
// first rot elements by the angles whose cosines and sines are a row of
// cos_sin; the other elements pass. All of it is binary32, rounded once.
//
// A row of head_dim elements belongs to a group of L lanes, L the power of two
// at or above head_dim / 8, 8 elements a lane: one 16-byte load of bf16 (two of
// f32), the sum of squares and the partner half of a pair by shuffles. A group
// takes a strip of up to kStrip heads of one token, all loaded before the first
// is used, so that the token's angles are read once and kStrip rows are in
// flight a lane. Bound by memory: every element is read once and written once.
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kNrThreads = 256;
constexpr int kStrip = 4;

namespace {

// The eight cosines and sines that a lane's elements need, by element. For the
// half layout sin carries the sign of its place in the pair; for the
// interleaved one cos[j], sin[j] (j < 4) belong to the pair of elements 2j, 2j + 1.
struct Turn {
  float c[8], s[8];
};

template <bool INTER>
__device__ __forceinline__ void load_turn(Turn* t, const float* row, int rot, int d0) {
  const int half = rot >> 1;
  if (d0 >= rot) return;
  if (INTER) {
    const float4 c = *reinterpret_cast<const float4*>(row + (d0 >> 1));
    const float4 s = *reinterpret_cast<const float4*>(row + half + (d0 >> 1));
    t->c[0] = c.x; t->c[1] = c.y; t->c[2] = c.z; t->c[3] = c.w;
    t->s[0] = s.x; t->s[1] = s.y; t->s[2] = s.z; t->s[3] = s.w;
  } else {
    const int j = d0 < half ? d0 : d0 - half;
    const float sign = d0 < half ? -1.f : 1.f;
    const float4 c0 = *reinterpret_cast<const float4*>(row + j), c1 = *reinterpret_cast<const float4*>(row + j + 4);
    const float4 s0 = *reinterpret_cast<const float4*>(row + half + j);
    const float4 s1 = *reinterpret_cast<const float4*>(row + half + j + 4);
    t->c[0] = c0.x; t->c[1] = c0.y; t->c[2] = c0.z; t->c[3] = c0.w;
    t->c[4] = c1.x; t->c[5] = c1.y; t->c[6] = c1.z; t->c[7] = c1.w;
    t->s[0] = sign * s0.x; t->s[1] = sign * s0.y; t->s[2] = sign * s0.z; t->s[3] = sign * s0.w;
    t->s[4] = sign * s1.x; t->s[5] = sign * s1.y; t->s[6] = sign * s1.z; t->s[7] = sign * s1.w;
  }
}

// v <- R v, or R^T v with BACK. All lanes of the warp call it (the partner half
// of a pair comes by shuffle); lanes past rot keep their values.
template <int L, bool INTER, bool BACK>
__device__ __forceinline__ void rotate(float (&v)[8], const Turn& t, int rot, int d0) {
  if (INTER) {
    if (d0 < rot) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float s = BACK ? -t.s[j] : t.s[j];
        const float x = v[2 * j], y = v[2 * j + 1];
        v[2 * j] = x * t.c[j] - y * s;
        v[2 * j + 1] = y * t.c[j] + x * s;
      }
    }
  } else {
    const int step = rot >> 4;  // lanes of half a rotated part
    const int lane = threadIdx.x & (L - 1);
    const int from = lane < step ? lane + step : lane - step;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float p = __shfl_sync(~0u, v[j], from & (L - 1), L);
      if (d0 < rot) v[j] = v[j] * t.c[j] + p * (BACK ? -t.s[j] : t.s[j]);
    }
  }
}

template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d, L);
  return x;
}

}  // namespace

// CACHE: keys and values go to the cache rows of slots (heads of the strip: q,
// k, v); else keys go to k_out (heads: q, k). Block y is the rank.
template <typename T, int L, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int strips,
                                                               int per_strip) {
  if (!op_workspace_ok(a.ws)) return;
  const int rank = blockIdx.y;
  const int lane = threadIdx.x & (L - 1), d0 = lane * 8, D = a.head_dim;
  const uint32_t item = blockIdx.x * (kNrThreads / L) + threadIdx.x / L;
  const bool live = item < (uint32_t)a.tokens * (uint32_t)strips;
  const int token = live ? (int)(item / (uint32_t)strips) : 0;
  const int heads = a.q_heads + (CACHE ? 2 : 1) * a.kv_heads;
  const int h0 = live ? (int)(item - (uint32_t)token * (uint32_t)strips) * per_strip : 0;
  const bool in_row = live && d0 < D;

  const T* row = reinterpret_cast<const T*>(a.qkv[rank]) + (int64_t)token * a.qkv_stride + d0;
  Pack8<T> x[kStrip];
#pragma unroll
  for (int i = 0; i < kStrip; i++) {
    x[i].zero();
    if (in_row && i < per_strip && h0 + i < heads) x[i].load(row + (int64_t)(h0 + i) * D);
  }
  bool bad = false;
  int pos = live ? a.positions[token] : 0;
  if (pos < 0 || pos >= a.max_pos) { bad = true; pos = 0; }
  int64_t slot = 0;
  if (CACHE) {
    slot = live ? a.slots[token] : -1;  // below zero: a padding token, no cache row
    if (slot >= a.num_slots) { bad = true; slot = -1; }
  }
  Turn turn;
  load_turn<INTER>(&turn, a.cos_sin + (int64_t)pos * a.rot, a.rot, d0);

#pragma unroll
  for (int i = 0; i < kStrip; i++) {
    const int h = h0 + i;
    const bool have = i < per_strip && h < heads;
    const bool is_v = CACHE && h >= a.q_heads + a.kv_heads, is_q = h < a.q_heads;
    float v[8], w[8];
    x[i].widen(v);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) sum += v[j] * v[j];
    const float r = rsqrtf(group_sum<L>(sum) / (float)D + a.eps);
    Pack8<T> wp;
    wp.zero();
    if (in_row && have && !is_v) wp.load(reinterpret_cast<const T*>(is_q ? a.q_weight : a.k_weight) + d0);
    wp.widen(w);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = v[j] * r * w[j];
    rotate<L, INTER, false>(v, turn, a.rot, d0);
    if (!in_row || !have) continue;
    if (!is_v) x[i].narrow(v);
    if (is_q) {
      x[i].store(reinterpret_cast<T*>(a.q_out[rank]) + (int64_t)token * a.q_stride + (int64_t)h * D + d0);
    } else if (!CACHE) {
      x[i].store(reinterpret_cast<T*>(a.k_out[rank]) + (int64_t)token * a.k_stride + (int64_t)(h - a.q_heads) * D + d0);
    } else if (slot >= 0) {
      const int kh = h - a.q_heads - (is_v ? a.kv_heads : 0);
      const int64_t page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
      T* cache = reinterpret_cast<T*>(is_v ? a.v_out[rank] : a.k_out[rank]);
      x[i].store(cache + (((page * a.kv_heads + kh) << a.page_shift) + off) * D + d0);
    }
  }
  if (bad) op_report(a.ws, kErrCapacity);
}

// The gradient. z' = R^T dy, dw = sum z' x r, g = z' w, xh = x r,
// dx = r (g - xh mean(g xh)); dv is copied. A group walks over strips; its sums
// for the two weights stay in registers, are added over the block's groups in
// shared memory in group order, and the block that arrives last for its rank
// adds the blocks' partial sums in block order: the same bits every time.
template <typename T, int L, bool INTER>
__global__ void __launch_bounds__(kNrThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdArgs a, int strips,
                                                                   int per_strip) {
  constexpr int kGroups = kNrThreads / L;
  __shared__ float sums[kNrThreads][8];
  __shared__ bool s_last;
  if (!op_workspace_ok(a.ws)) return;
  const int rank = blockIdx.y;
  const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L, d0 = lane * 8, D = a.head_dim;
  const int heads = a.q_heads + 2 * a.kv_heads;
  float wq[8], wk[8], dwq[8], dwk[8];
  Pack8<T> p;
  p.zero();
  if (d0 < D) p.load(reinterpret_cast<const T*>(a.q_weight) + d0);
  p.widen(wq);
  if (d0 < D) p.load(reinterpret_cast<const T*>(a.k_weight) + d0);
  p.widen(wk);
#pragma unroll
  for (int j = 0; j < 8; j++) dwq[j] = dwk[j] = 0.f;
  bool bad = false;
  const uint32_t items = (uint32_t)a.tokens * (uint32_t)strips;
  const uint32_t step = gridDim.x * kGroups;
  for (uint32_t block_item = blockIdx.x * kGroups; block_item < items; block_item += step) {
    const uint32_t item = block_item + group;
    const bool live = item < items;
    const int token = live ? (int)(item / (uint32_t)strips) : 0;
    const int h0 = live ? (int)(item - (uint32_t)token * (uint32_t)strips) * per_strip : 0;
    const bool in_row = live && d0 < D;
    const T* xrow = reinterpret_cast<const T*>(a.qkv[rank]) + (int64_t)token * a.qkv_stride + d0;
    T* drow = reinterpret_cast<T*>(a.dqkv[rank]) + (int64_t)token * a.dqkv_stride + d0;
    Pack8<T> x[kStrip], dy[kStrip];
#pragma unroll
    for (int i = 0; i < kStrip; i++) {
      const int h = h0 + i;
      x[i].zero();
      dy[i].zero();
      if (!in_row || i >= per_strip || h >= heads) continue;
      const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
      const T* g = reinterpret_cast<const T*>(is_q ? a.dq[rank] : is_v ? a.dv[rank] : a.dk[rank]) + d0;
      const int64_t stride = is_q ? a.dq_stride : is_v ? a.dv_stride : a.dk_stride;
      const int gh = is_q ? h : is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
      dy[i].load(g + (int64_t)token * stride + (int64_t)gh * D);
      if (!is_v) x[i].load(xrow + (int64_t)h * D);
    }
    int pos = live ? a.positions[token] : 0;
    if (pos < 0 || pos >= a.max_pos) { bad = true; pos = 0; }
    Turn turn;
    load_turn<INTER>(&turn, a.cos_sin + (int64_t)pos * a.rot, a.rot, d0);
#pragma unroll
    for (int i = 0; i < kStrip; i++) {
      const int h = h0 + i;
      const bool have = i < per_strip && h < heads;
      const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
      float v[8], g[8];
      x[i].widen(v);
      dy[i].widen(g);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j++) sum += v[j] * v[j];
      const float r = rsqrtf(group_sum<L>(sum) / (float)D + a.eps);
      rotate<L, INTER, true>(g, turn, a.rot, d0);
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        v[j] *= r;
        const float dw = g[j] * v[j];  // zero for a value head, whose x was not loaded
        if (is_q) dwq[j] += dw; else dwk[j] += dw;
        g[j] *= is_q ? wq[j] : wk[j];
        dot += g[j] * v[j];
      }
      dot = group_sum<L>(dot) / (float)D;
#pragma unroll
      for (int j = 0; j < 8; j++) g[j] = r * (g[j] - v[j] * dot);
      if (!in_row || !have) continue;
      if (!is_v) dy[i].narrow(g);
      dy[i].store(drow + (int64_t)h * D);
    }
  }
  if (bad) op_report(a.ws, kErrCapacity);

  // partial sums of the block: [block of the rank][q, k][D]
  float* part = reinterpret_cast<float*>(a.ws + kOpScratchOffset) + (int64_t)rank * gridDim.x * 2 * D;
#pragma unroll
  for (int which = 0; which < 2; which++) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; j++) sums[threadIdx.x][j] = which == 0 ? dwq[j] : dwk[j];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kNrThreads) {
      float s = 0.f;
      for (int g = 0; g < kGroups; g++) s += sums[g * L + (d >> 3)][d & 7];
      part[((int64_t)blockIdx.x * 2 + which) * D + d] = s;
    }
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t* counter = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes) + rank;
    s_last = atomicAdd(counter, 1u) == gridDim.x - 1;
    if (s_last) *counter = 0;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int d = threadIdx.x; d < 2 * D; d += kNrThreads) {
    float s = 0.f;
    for (unsigned b = 0; b < gridDim.x; b++) s += __ldcg(part + (int64_t)b * 2 * D + d);
    if (d < D) a.dq_weight[rank][d] = s;
    else a.dk_weight[rank][d - D] = s;
  }
}

namespace {

int lanes_of(int head_dim) {
  int l = 8;
  while (l * 8 < head_dim) l *= 2;
  return l;
}

template <typename T, int L>
const void* forward_of(bool inter, bool cache) {
  return inter ? (cache ? (const void*)norm_rope_kernel<T, L, true, true> : (const void*)norm_rope_kernel<T, L, true, false>)
               : (cache ? (const void*)norm_rope_kernel<T, L, false, true>
                        : (const void*)norm_rope_kernel<T, L, false, false>);
}
template <typename T>
const void* forward_of(int lanes, bool inter, bool cache) {
  return lanes == 8 ? forward_of<T, 8>(inter, cache) : lanes == 16 ? forward_of<T, 16>(inter, cache)
                                                                   : forward_of<T, 32>(inter, cache);
}
template <typename T, int L>
const void* backward_of(bool inter) {
  return inter ? (const void*)norm_rope_bwd_kernel<T, L, true> : (const void*)norm_rope_bwd_kernel<T, L, false>;
}
template <typename T>
const void* backward_of(int lanes, bool inter) {
  return lanes == 8 ? backward_of<T, 8>(inter) : lanes == 16 ? backward_of<T, 16>(inter) : backward_of<T, 32>(inter);
}

}  // namespace

int64_t norm_rope_scratch_bytes(int nranks, int head_dim) {
  const int64_t blocks = imax(kNormRopeBwdBlocks, nranks);
  return blocks * 2 * head_dim * (int64_t)sizeof(float);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.head_dim);
  const bool cache = a.slots != nullptr;
  const int heads = a.q_heads + (cache ? 2 : 1) * a.kv_heads;
  int strips = (int)div_up(heads, kStrip);
  int per_strip = (int)div_up(heads, strips);
  strips = (int)div_up(heads, per_strip);
  const int64_t items = (int64_t)a.tokens * strips;
  dim3 grid((unsigned)div_up(items, kNrThreads / lanes), (unsigned)a.nranks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: qk_norm_rope nranks=%d tokens=%d heads=%d dim=%d rot=%d grid=%ux%u cache=%d\n",
                 a.nranks, a.tokens, heads, a.head_dim, a.rot, grid.x, grid.y, cache ? 1 : 0);
  const void* fn = a.dtype == kF32 ? forward_of<float>(lanes, a.interleaved != 0, cache)
                                   : forward_of<uint16_t>(lanes, a.interleaved != 0, cache);
  void* params[] = {const_cast<NormRopeArgs*>(&a), &strips, &per_strip};
  return cudaLaunchKernel(fn, grid, dim3(kNrThreads), params, 0, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.head_dim);
  const int heads = a.q_heads + 2 * a.kv_heads;
  int strips = (int)div_up(heads, kStrip);
  int per_strip = (int)div_up(heads, strips);
  strips = (int)div_up(heads, per_strip);
  const int64_t items = (int64_t)a.tokens * strips;
  const int64_t blocks = imax(1, imin(div_up(items, kNrThreads / lanes), kNormRopeBwdBlocks / a.nranks));
  dim3 grid((unsigned)blocks, (unsigned)a.nranks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: qk_norm_rope_backward nranks=%d tokens=%d heads=%d dim=%d rot=%d grid=%ux%u\n",
                 a.nranks, a.tokens, heads, a.head_dim, a.rot, grid.x, grid.y);
  const void* fn = a.dtype == kF32 ? backward_of<float>(lanes, a.interleaved != 0)
                                   : backward_of<uint16_t>(lanes, a.interleaved != 0);
  void* params[] = {const_cast<NormRopeBwdArgs*>(&a), &strips, &per_strip};
  return cudaLaunchKernel(fn, grid, dim3(kNrThreads), params, 0, stream);
}

}  // namespace rar
