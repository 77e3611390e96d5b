// qk_norm_rope.cu -- root-mean-square norm of every query and key head with the
// rotary position in the same pass, and its gradient.
//
//   y = R(pos) (x * r * w),  r = 1 / sqrt(mean(x^2) + eps)
// R turns the pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved, of the
// first rot elements by the angles whose cosines and sines are a row of
// cos_sin; the other elements pass. All of it is binary32, rounded once.
//
// A row of head_dim elements belongs to a group of L lanes, L the power of two
// at or above head_dim / 8. A lane holds eight elements as two chunks of four:
// for pairs half a rotation apart the chunks are 4l and rot/2 + 4l, so both
// elements of a pair are in one lane and the rotation exchanges nothing (with
// eight consecutive elements a lane it took eight shuffles a row and the kernel
// was bound by instructions: 108 us where this one takes 60, 8192 tokens of 10
// heads of 128 on 8 ranks); the group's loads still cover whole lines.
// A group takes a strip of a few heads of one token, all loaded before the
// first is used; weights and angles are read once a strip. Bound by memory:
// every element is read once and written once.
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kNrThreads = 256;
template <typename T>
constexpr int kStrip = 4;                 // rows of a forward strip
constexpr int kBwdStrip = 2;              // heads of a backward strip: x and dy of each are in registers
constexpr int kNormRopeBwdBlocks = 1216;  // most blocks of a backward launch, all ranks together

namespace {

// Where a lane's chunks lie and whether they turn.
struct Lane {
  int o0, o1;     // first elements of the two chunks
  int angle;      // index of its first cosine
  bool in, turn;  // inside the row; inside the rotated part
};
template <bool INTER>
__device__ __forceinline__ Lane lane_of(int l, int D, int rot) {
  Lane n;
  n.in = l * 8 < D;
  n.turn = l * 8 < rot;
  n.angle = 4 * l;
  n.o0 = !INTER && n.turn ? 4 * l : 8 * l;
  n.o1 = !INTER && n.turn ? (rot >> 1) + 4 * l : 8 * l + 4;
  return n;
}

// Two chunks of four elements.
template <typename T>
struct Chunks;
template <>
struct Chunks<uint16_t> {
  uint2 a, b;
  __device__ __forceinline__ void load(const uint16_t* row, const Lane& n) {
    a = *reinterpret_cast<const uint2*>(row + n.o0);
    b = *reinterpret_cast<const uint2*>(row + n.o1);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0, 0); }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(b.x); v[5] = bf16_hi(b.x); v[6] = bf16_lo(b.y); v[7] = bf16_hi(b.y);
  }
  __device__ __forceinline__ void narrow(const float (&v)[8]) {
    a = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    b = make_uint2(bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  }
  __device__ __forceinline__ void store(uint16_t* row, const Lane& n) const {
    *reinterpret_cast<uint2*>(row + n.o0) = a;
    *reinterpret_cast<uint2*>(row + n.o1) = b;
  }
};
template <>
struct Chunks<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, const Lane& n) {
    a = *reinterpret_cast<const float4*>(row + n.o0);
    b = *reinterpret_cast<const float4*>(row + n.o1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void narrow(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float* row, const Lane& n) const {
    *reinterpret_cast<float4*>(row + n.o0) = a;
    *reinterpret_cast<float4*>(row + n.o1) = b;
  }
};

// A lane's four angles; (1, 0) where nothing turns.
struct Turn {
  float c[4], s[4];
};
__device__ __forceinline__ Turn load_turn(const float* row, int rot, const Lane& n) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n.turn) {
    c = *reinterpret_cast<const float4*>(row + n.angle);
    s = *reinterpret_cast<const float4*>(row + (rot >> 1) + n.angle);
  }
  return Turn{{c.x, c.y, c.z, c.w}, {s.x, s.y, s.z, s.w}};
}

// v <- R v, or R^T v with BACK.
template <bool INTER, bool BACK>
__device__ __forceinline__ void rotate(float (&v)[8], const Turn& t) {
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const int x = INTER ? 2 * j : j, y = INTER ? 2 * j + 1 : j + 4, step = INTER ? 2 : 1;
    const float2 c = make_float2(t.c[j], t.c[j + 1]);
    const float2 s = BACK ? make_float2(-t.s[j], -t.s[j + 1]) : make_float2(t.s[j], t.s[j + 1]);
    const float2 a = make_float2(v[x], v[x + step]), b = make_float2(v[y], v[y + step]);
    const float2 ra = fma2(b, make_float2(-s.x, -s.y), mul2(a, c)), rb = fma2(a, s, mul2(b, c));
    v[x] = ra.x;
    v[x + step] = ra.y;
    v[y] = rb.x;
    v[y + step] = rb.y;
  }
}

// Sum over a group; groups of a warp may be on different paths.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
  const uint32_t mask = L == 32 ? ~0u : ((1u << (L & 31)) - 1) << (threadIdx.x & 31 & ~(L - 1));
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) x += __shfl_xor_sync(mask, x, d, L);
  return x;
}
__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float2 s = mul2(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
#pragma unroll
  for (int j = 2; j < 8; j += 2) s = fma2(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), s);
  return s.x + s.y;
}
// The lane's weights of a head's kind.
template <typename T>
__device__ __forceinline__ void load_weight(float (&w)[8], const void* p, const Lane& n) {
  Chunks<T> c;
  c.zero();
  if (n.in) c.load(reinterpret_cast<const T*>(p), n);
  c.widen(w);
}

}  // namespace

// Blocks below q_blocks take strips of per_q query heads, the others strips of
// per_kv key heads, with CACHE each followed by the same heads' values; so a
// warp's groups do the same. Keys and values go to the cache rows of slots, or
// keys to k_out. Block y is the rank.
template <typename T, int L, bool INTER, bool CACHE>
__global__ void __launch_bounds__(kNrThreads, sizeof(T) == 2 ? 4 : 3) norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int q_blocks,
                                                               int q_strips, int per_q, int kv_strips, int per_kv) {
  constexpr int kRows = kStrip<T>;
  const uint32_t magic = op_magic(a.ws);
  const int rank = blockIdx.y, D = a.head_dim;
  const Lane n = lane_of<INTER>(threadIdx.x & (L - 1), D, a.rot);
  const bool is_q = blockIdx.x < q_blocks;
  const uint32_t strips = is_q ? q_strips : kv_strips;
  const uint32_t item = (blockIdx.x - (is_q ? 0 : q_blocks)) * (kNrThreads / L) + threadIdx.x / L;
  const bool live = item < (uint32_t)a.tokens * strips;
  const int token = live ? (int)(item / strips) : 0;
  const int strip = live ? (int)(item - (uint32_t)token * strips) : 0;
  const bool in = live && n.in;
  const int h0 = strip * (is_q ? per_q : per_kv);
  const int heads = is_q ? min(per_q, a.q_heads - h0) : min(per_kv, a.kv_heads - h0);
  const int rows = heads * (CACHE && !is_q ? 2 : 1);

  int pos = live ? a.positions[token] : 0;
  int64_t slot = CACHE && live ? a.slots[token] : -1;  // below zero: a padding token, no cache row
  const T* x0 = reinterpret_cast<const T*>(a.qkv[rank]) + (int64_t)token * a.qkv_stride + (h0 + (is_q ? 0 : a.q_heads)) * D;
  const int to_v = (a.kv_heads - heads) * D;  // from the place after a strip's keys to its values
  Chunks<T> x[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i++)
    if (in && i < rows) x[i].load(x0 + i * D + (CACHE && !is_q && i >= heads ? to_v : 0), n);
    else x[i].zero();
  bool bad = false;
  if (pos < 0 || pos >= a.max_pos) { bad = true; pos = 0; }
  if (CACHE && slot >= a.num_slots) { bad = true; slot = -1; }
  const Turn turn = load_turn(a.cos_sin + (int64_t)pos * a.rot, a.rot, n);
  float w[8];
  load_weight<T>(w, is_q ? a.q_weight : a.k_weight, n);
  const float inv = 1.f / (float)D;
  if (!op_ready(a.ws, magic)) return;

  // where the strip's first row goes and how far apart its rows are
  T* out;
  T* out_v = nullptr;
  int64_t apart = D;
  bool kept = true;  // false: a padding token's keys and values
  if (is_q) {
    out = reinterpret_cast<T*>(a.q_out[rank]) + (int64_t)token * a.q_stride + h0 * D;
  } else if (!CACHE) {
    out = reinterpret_cast<T*>(a.k_out[rank]) + (int64_t)token * a.k_stride + h0 * D;
  } else {
    kept = slot >= 0;
    const int64_t page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
    const int64_t at = (((page * a.kv_heads + h0) << a.page_shift) + off) * D;
    out = reinterpret_cast<T*>(a.k_out[rank]) + at;
    out_v = reinterpret_cast<T*>(a.v_out[rank]) + at;
    apart = (int64_t)D << a.page_shift;
  }
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    if (i >= rows) break;
    if (!CACHE || is_q || i < heads) {
      float v[8];
      x[i].widen(v);
      const float r = rsqrt_fast(fmaf(group_sum<L>(dot8(v, v)), inv, a.eps));
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 y = mul2(mul2(make_float2(v[j], v[j + 1]), make_float2(r, r)), make_float2(w[j], w[j + 1]));
        v[j] = y.x;
        v[j + 1] = y.y;
      }
      rotate<INTER, false>(v, turn);
      x[i].narrow(v);
      if (in && kept) x[i].store(out + i * apart, n);
    } else if (in && kept) {
      x[i].store(out_v + (i - heads) * apart, n);
    }
  }
  if (bad) op_report(a.ws, kErrCapacity);
}

// The gradient. z = R^T dy, dw = sum z x r, g = z w, xh = x r,
// dx = r (g - xh mean(g xh)); dv is copied. The first q_blocks blocks of a rank
// walk over strips of query heads, the others over key heads and the same
// heads' values; so one set of weight sums stays in registers. They are added
// over the block's groups in shared memory in group order, and the block that
// arrives last for its rank adds the blocks' partial sums in block order: the
// same bits every time.
template <typename T, int L, bool INTER>
__global__ void __launch_bounds__(kNrThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdArgs a,
                                                                   int q_blocks) {
  constexpr int kGroups = kNrThreads / L;
  __shared__ float sums[kNrThreads][9];
  __shared__ bool s_last;
  const uint32_t magic = op_magic(a.ws);
  const int rank = blockIdx.y, group = threadIdx.x / L, D = a.head_dim;
  const Lane n = lane_of<INTER>(threadIdx.x & (L - 1), D, a.rot);
  const bool is_q = blockIdx.x < q_blocks;
  const uint32_t block = is_q ? blockIdx.x : blockIdx.x - q_blocks, blocks = is_q ? q_blocks : gridDim.x - q_blocks;
  const int kind_heads = is_q ? a.q_heads : a.kv_heads;
  const uint32_t strips = (uint32_t)(kind_heads + kBwdStrip - 1) / kBwdStrip;
  float w[8], dw[8];
  load_weight<T>(w, is_q ? a.q_weight : a.k_weight, n);
#pragma unroll
  for (int j = 0; j < 8; j++) dw[j] = 0.f;
  const float inv = 1.f / (float)D;
  const int64_t g_stride = is_q ? a.dq_stride : a.dk_stride;
  const T* g0 = reinterpret_cast<const T*>(is_q ? a.dq[rank] : a.dk[rank]);
  bool bad = false;
  const uint32_t items = (uint32_t)a.tokens * strips;
  // the next item is loaded while this one is worked on
  struct Item {
    Chunks<T> x[kBwdStrip], dy[kBwdStrip];
    int token, h0, heads, pos;
  };
  const uint32_t step = blocks * kGroups;
  const T* xs = reinterpret_cast<const T*>(a.qkv[rank]);
  auto fetch = [&](uint32_t item) {
    Item t;
    const bool live = item < items;
    t.token = live ? (int)(item / strips) : 0;
    t.h0 = live ? (int)(item - (uint32_t)t.token * strips) * kBwdStrip : 0;
    t.heads = live && n.in ? min(kBwdStrip, kind_heads - t.h0) : 0;
    t.pos = live ? a.positions[t.token] : 0;
    const T* xrow = xs + (int64_t)t.token * a.qkv_stride + (is_q ? t.h0 : a.q_heads + t.h0) * D;
    const T* grow = g0 + (int64_t)t.token * g_stride + t.h0 * D;
#pragma unroll
    for (int i = 0; i < kBwdStrip; i++) {
      t.x[i].zero();
      t.dy[i].zero();
      if (i < t.heads) {
        t.x[i].load(xrow + i * D, n);
        t.dy[i].load(grow + i * D, n);
      }
    }
    return t;
  };
  uint32_t item = block * kGroups + group;
  Item cur = fetch(item);
  if (!op_ready(a.ws, magic)) return;
  for (; item - group < items; item += step) {
    const Item nxt = fetch(item + step);
    if (cur.pos < 0 || cur.pos >= a.max_pos) { bad = true; cur.pos = 0; }
    const Turn turn = load_turn(a.cos_sin + (int64_t)cur.pos * a.rot, a.rot, n);
    T* drow = reinterpret_cast<T*>(a.dqkv[rank]) + (int64_t)cur.token * a.dqkv_stride;
    Chunks<T> dv[kBwdStrip];
    if (!is_q) {
      const T* vrow = reinterpret_cast<const T*>(a.dv[rank]) + (int64_t)cur.token * a.dv_stride + cur.h0 * D;
#pragma unroll
      for (int i = 0; i < kBwdStrip; i++)
        if (i < cur.heads) dv[i].load(vrow + i * D, n);
    }
    const int place = is_q ? cur.h0 : a.q_heads + cur.h0;
#pragma unroll
    for (int i = 0; i < kBwdStrip; i++) {
      float v[8], g[8];
      cur.x[i].widen(v);
      cur.dy[i].widen(g);
      const float r = rsqrt_fast(fmaf(group_sum<L>(dot8(v, v)), inv, a.eps));
      rotate<INTER, true>(g, turn);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        v[j] *= r;
        dw[j] = fmaf(g[j], v[j], dw[j]);  // rows that are not there are zeros
        g[j] *= w[j];
      }
      const float mean = group_sum<L>(dot8(g, v)) * inv;
#pragma unroll
      for (int j = 0; j < 8; j++) g[j] = r * fmaf(-mean, v[j], g[j]);
      if (i >= cur.heads) continue;
      Chunks<T> dx;
      dx.narrow(g);
      dx.store(drow + (place + i) * D, n);
      if (!is_q) dv[i].store(drow + (place + a.kv_heads + i) * D, n);
    }
    cur = nxt;
  }
  if (bad) op_report(a.ws, kErrCapacity);

  // partial sums of the rank's blocks: [block][D], the query blocks first
  float* parts = reinterpret_cast<float*>(a.ws + kOpScratchOffset) + (int64_t)rank * gridDim.x * D;
#pragma unroll
  for (int j = 0; j < 8; j++) sums[threadIdx.x][j] = dw[j];
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kNrThreads) {
    // the lane and chunk that hold element e
    const int half = a.rot >> 1;
    const bool turned = !INTER && e < a.rot;
    const int l = turned ? (e < half ? e : e - half) >> 2 : e >> 3;
    const int j = turned ? (e & 3) + (e < half ? 0 : 4) : e & 7;
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; g++) s += sums[g * L + l][j];
    parts[(int64_t)blockIdx.x * D + e] = s;
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
  // four elements a thread; the threads that share them take every `many`-th block, then join in that order
  const int quads = D >> 2, many = kNrThreads / quads, quad = threadIdx.x % quads, turn_of = threadIdx.x / quads;
  for (int which = 0; which < 2; which++) {
    const int b0 = which == 0 ? 0 : q_blocks, b1 = which == 0 ? q_blocks : (int)gridDim.x;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turn_of < many) {
#pragma unroll 8
      for (int b = b0 + turn_of; b < b1; b += many) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(parts + (int64_t)b * D + quad * 4));
        s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
      }
    }
    __syncthreads();
    sums[threadIdx.x][0] = s.x;
    sums[threadIdx.x][1] = s.y;
    sums[threadIdx.x][2] = s.z;
    sums[threadIdx.x][3] = s.w;
    __syncthreads();
    float* out = which == 0 ? a.dq_weight[rank] : a.dk_weight[rank];
    for (int e = threadIdx.x; e < D; e += kNrThreads) {
      float t = 0.f;
      for (int k = 0; k < many; k++) t += sums[k * quads + (e >> 2)][e & 3];
      out[e] = t;
    }
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
  return (kNormRopeBwdBlocks + 2ll * nranks) * head_dim * (int64_t)sizeof(float);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.head_dim);
  const bool cache = a.slots != nullptr;
  const int rows = a.dtype == kF32 ? kStrip<float> : kStrip<uint16_t>, most_kv = cache ? rows / 2 : rows;
  int q_strips = (int)div_up(a.q_heads, rows), kv_strips = (int)div_up(a.kv_heads, most_kv);
  int per_q = (int)div_up(a.q_heads, q_strips), per_kv = (int)div_up(a.kv_heads, kv_strips);
  q_strips = (int)div_up(a.q_heads, per_q);
  kv_strips = (int)div_up(a.kv_heads, per_kv);
  const int groups = kNrThreads / lanes;
  int q_blocks = (int)div_up((int64_t)a.tokens * q_strips, groups);
  const int kv_blocks = (int)div_up((int64_t)a.tokens * kv_strips, groups);
  dim3 grid((unsigned)(q_blocks + kv_blocks), (unsigned)a.nranks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: qk_norm_rope nranks=%d tokens=%d heads=%d/%d dim=%d rot=%d grid=%ux%u cache=%d\n",
                 a.nranks, a.tokens, a.q_heads, a.kv_heads, a.head_dim, a.rot, grid.x, grid.y, cache ? 1 : 0);
  const void* fn = a.dtype == kF32 ? forward_of<float>(lanes, a.interleaved != 0, cache)
                                   : forward_of<uint16_t>(lanes, a.interleaved != 0, cache);
  void* params[] = {const_cast<NormRopeArgs*>(&a), &q_blocks, &q_strips, &per_q, &kv_strips, &per_kv};
  return cudaLaunchKernel(fn, grid, dim3(kNrThreads), params, 0, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.head_dim), groups = kNrThreads / lanes;
  // blocks of the two kinds in proportion to their bytes: x, dy and dx of a query or key head, dv twice
  const void* fn = a.dtype == kF32 ? backward_of<float>(lanes, a.interleaved != 0)
                                   : backward_of<uint16_t>(lanes, a.interleaved != 0);
  int device = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&device, &sms);
  if (e != cudaSuccess) return e;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, kNrThreads, 0);
  if (e != cudaSuccess) return e;
  const int64_t most = imin(kNormRopeBwdBlocks, (int64_t)sms * per_sm) / a.nranks;
  const int64_t q_items = (int64_t)a.tokens * div_up(a.q_heads, kBwdStrip);
  const int64_t kv_items = (int64_t)a.tokens * div_up(a.kv_heads, kBwdStrip);
  const int64_t share = most * 3 * a.q_heads / (3 * a.q_heads + 5 * a.kv_heads);
  int q_blocks = (int)imax(1, imin(div_up(q_items, groups), share));
  const int kv_blocks = (int)imax(1, imin(div_up(kv_items, groups), most - share));
  dim3 grid((unsigned)(q_blocks + kv_blocks), (unsigned)a.nranks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: qk_norm_rope_backward nranks=%d tokens=%d heads=%d/%d dim=%d rot=%d grid=%ux%u\n",
                 a.nranks, a.tokens, a.q_heads, a.kv_heads, a.head_dim, a.rot, grid.x, grid.y);
  void* params[] = {const_cast<NormRopeBwdArgs*>(&a), &q_blocks};
  return cudaLaunchKernel(fn, grid, dim3(kNrThreads), params, 0, stream);
}

}  // namespace rar
