// prompt_attention.cu -- attention over whole prompts and its gradient on the
// ordinary arithmetic units, for any type, head size and group.
//
//   s = scale q . k over the keys at or before the query's position, p = exp(s - lse),
//   out = sum p v;   with delta = out . dout:   ds = p (dout . v - delta),
//   dq = scale sum ds k,  dk = scale sum ds q,  dv = sum p dout
//
// A block of 256 threads holds BT rows (prompt_attention.cuh) as binary32 in shared
// memory, and reads tiles of BT keys after one another, with the running maximum and
// sum of the softmax in registers. The gradient is two kernels: one by rows, which
// leaves delta behind and sums dq over the keys, one by keys, which sums dk and dv over
// the rows of all query heads of the group. Both recompute p from lse; no sum
// crosses blocks, so results are the same bits every time.
//
// Threads are 16 by 16; thread (ty, tx) has rows ty + 16 i and columns tx + 16 j of a
// tile's scores, and elements 2 tx + 32 c and the next of the rows' results: operands
// come as loads that half a warp shares or that fall on all banks. Products run two at a
// time along the head (scores) or across it (results). What bounds them is the two
// multiply-adds a lane and cycle, and the latency of a tile's loads: keys and values take
// turns in one buffer, so that two blocks fit an SM up to a head size of 128 and one
// works while the other waits (a buffer each and head sizes padded to 64 or 128: 340 us
// for 2777 tokens of 12 heads of 80 where this took 218; with the keys of the largest
// items split, 170 to 197). Over long prompts that is 34 to 40 TFLOP/s forward and 17 to
// 27 for the gradient, of the 75 that the multiply-adds alone could make: issue slots are
// 46 % busy, the rest of the time warps wait for shared memory and for the pipes.
#include <initializer_list>

#include "op_common.cuh"
#include "prompt_attention.cuh"
#include "rar_launch.h"

namespace rar {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(uint16_t* p, float x, float y) { *reinterpret_cast<uint32_t*>(p) = bf16_pair(x, y); }

// Whether the gradient's tiles have buffers of their own and two blocks fit an SM all the same.
template <int DP>
constexpr bool kApart = DP <= 64;

template <int DP, int BT>
struct Shape {
  static constexpr int MT = BT / 16;   // rows, and columns, of a thread
  static constexpr int NC = DP / 32;   // pairs of elements of a result row
  static constexpr int LD = DP + 4;    // floats from row to row: 16-byte loads of 16 rows fall on different banks
  static constexpr int LP = BT + 4;
  static constexpr int kRows = BT * LD, kScores = BT * LP;
};

// BT rows of D elements, widened, zeros past D and where at(row) is null; loads first, then stores.
template <typename T, int DP, int BT, typename At>
__device__ __forceinline__ void load_rows(float* to, int D, At at) {
  constexpr int C = DP / 8, N = BT * C / kThreads;
  static_assert(BT * C % kThreads == 0, "pieces of a thread");
  Pack8<T> x[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int k = threadIdx.x + i * kThreads, row = k / C, d = (k % C) * 8;
    const T* p = at(row);
    x[i].zero();
    if (p != nullptr && d < D) x[i].load(p + d);
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int k = threadIdx.x + i * kThreads, row = k / C, d = (k % C) * 8;
    float v[8];
    x[i].widen(v);
    float* o = to + row * Shape<DP, BT>::LD + d;
    store4(o, v[0], v[1], v[2], v[3]);
    store4(o + 4, v[4], v[5], v[6], v[7]);
  }
}

// s[i][j] = x[ty + 16 i] . y[tx + 16 j]
template <int DP, int BT>
__device__ __forceinline__ void dots(const float* x, const float* y, int D, float (&s)[BT / 16][BT / 16]) {
  using S = Shape<DP, BT>;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  F2 acc[S::MT][S::MT];
#pragma unroll
  for (int i = 0; i < S::MT; i++)
#pragma unroll
    for (int j = 0; j < S::MT; j++) acc[i][j] = f2(0.f, 0.f);
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    float4 a[S::MT], b[S::MT];
#pragma unroll
    for (int i = 0; i < S::MT; i++) {
      a[i] = *reinterpret_cast<const float4*>(x + (ty + 16 * i) * S::LD + d);
      b[i] = *reinterpret_cast<const float4*>(y + (tx + 16 * i) * S::LD + d);
    }
#pragma unroll
    for (int i = 0; i < S::MT; i++)
#pragma unroll
      for (int j = 0; j < S::MT; j++) {
        acc[i][j] = fma2(f2(a[i].x, a[i].y), f2(b[j].x, b[j].y), acc[i][j]);
        acc[i][j] = fma2(f2(a[i].z, a[i].w), f2(b[j].z, b[j].w), acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < S::MT; i++)
#pragma unroll
    for (int j = 0; j < S::MT; j++) {
      const float2 u = unpack(acc[i][j]);
      s[i][j] = u.x + u.y;
    }
}

template <int DP, int BT>
struct Sums {  // elements 2 tx + 32 c and the next of rows ty + 16 i
  using S = Shape<DP, BT>;
  F2 v[S::MT][S::NC];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < S::MT; i++)
#pragma unroll
      for (int c = 0; c < S::NC; c++) v[i][c] = f2(0.f, 0.f);
  }
  __device__ __forceinline__ void scale_row(int i, float by) {
#pragma unroll
    for (int c = 0; c < S::NC; c++) v[i][c] = mul2(v[i][c], f2(by, by));
  }
  // += sum over t of w[ty + 16 i][t] x[t]
  __device__ __forceinline__ void add(const float* w, const float* x) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 2
    for (int t = 0; t < BT; t += 4) {
      float4 u[S::MT];
#pragma unroll
      for (int i = 0; i < S::MT; i++) u[i] = *reinterpret_cast<const float4*>(w + (ty + 16 * i) * S::LP + t);
#pragma unroll
      for (int k = 0; k < 4; k++)
#pragma unroll
        for (int c = 0; c < S::NC; c++) {
          const float2 y = *reinterpret_cast<const float2*>(x + (t + k) * S::LD + 2 * tx + 32 * c);
#pragma unroll
          for (int i = 0; i < S::MT; i++) {
            const float z = k == 0 ? u[i].x : k == 1 ? u[i].y : k == 2 ? u[i].z : u[i].w;
            v[i][c] = fma2(f2(z, z), f2(y.x, y.y), v[i][c]);
          }
        }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store_row(int i, T* row, int D, float by) const {
    const int tx = threadIdx.x & 15;
#pragma unroll
    for (int c = 0; c < S::NC; c++) {
      if (2 * tx + 32 * c >= D) continue;
      const float2 a = unpack(v[i][c]);
      store2(row + 2 * tx + 32 * c, a.x * by, a.y * by);
    }
  }
};

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

// Cache rows of the keys j0 .. j0 + BT - 1 (-1: no key, or a page that is none).
template <int BT>
__device__ __forceinline__ void find_keys(const PromptArgs& a, const PromptSequence& seq, int head, int j0, int64_t* rows) {
  for (int i = threadIdx.x; i < BT; i += kThreads) {
    const int j = j0 + i;
    int64_t row = -1;
    if (j < seq.keys) {
      const int page = a.table[seq.index * a.table_stride + (j >> a.page_shift)];
      if ((unsigned)page < (unsigned)a.num_pages)
        row = (((int64_t)page * a.kv_heads + head) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
      else
        op_report(a.ws, kErrCapacity);
    }
    rows[i] = row;
  }
}

// An item's keys may be split over several blocks, which then leave O, m and l.
struct Split {
  int parts;
  float* sums;  // per item and part: BT rows of DP, then m and l of each
};
template <int DP, int BT>
constexpr int64_t kPartFloats = BT * (DP + 2);

// A block's place: the heads of all ranks side by side, so that the tiles with the most
// work of every head start first.
struct Place {
  int head, rank, part;
  int64_t slot, slots;
  template <typename Args>
  __device__ __forceinline__ Place(const Args& a, int parts) {
    const unsigned lanes = (unsigned)(a.kv_heads * a.nranks), whole = blockIdx.x / (unsigned)parts;
    part = (int)(blockIdx.x % (unsigned)parts);
    head = (int)(whole % lanes) % a.kv_heads;
    rank = (int)(whole % lanes) / a.kv_heads;
    slot = whole / lanes;
    slots = gridDim.x / (unsigned)parts / lanes;
  }
};

template <typename T, int DP, int BT>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) prompt_kernel(const __grid_constant__ PromptArgs a,
                                                                           const __grid_constant__ Split split) {
  using S = Shape<DP, BT>;
  extern __shared__ __align__(16) float shared[];
  float *sq = shared, *sk = sq + S::kRows, *sp = sk + S::kRows;  // sk: keys, then values
  __shared__ int64_t key_row[BT];
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  if (blockIdx.x == 0) check_starts(a.starts, a.sequences, a.tokens, a.ws, threadIdx.x, kThreads);
  const Place place(a, split.parts);
  const int group = a.q_heads / a.kv_heads, head = place.head, rank = place.rank, part = place.part, D = a.head_dim;
  PromptSequence seq;
  int tile;
  // the last tiles of a sequence see the most keys: they start first
  const int64_t slots = place.slots, slot = slots - 1 - place.slot;
  if (!find_sequence(a.starts, a.sequences, a.tokens, group, BT, slot, &seq, &tile)) return;
  const bool paged = a.table != nullptr;
  if (paged) cached_sequence(a, &seq);
  const int row0 = tile * BT;  // of the sequence: tokens * group stays below 2^31 (checked)
  const int rows = min(BT, seq.length * group - row0);
  const T* q = (const T*)a.q[rank];
  auto token_of = [&](int r) { return seq.first + (row0 + r) / group; };
  auto head_of = [&](int r) { return head * group + (row0 + r) % group; };
  load_rows<T, DP, BT>(sq, D, [&](int r) {
    return r < rows ? q + (int64_t)token_of(r) * a.q_stride + (int64_t)head_of(r) * a.q_head : nullptr;
  });
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int sees[S::MT];  // keys that the row sees
  float m[S::MT], l[S::MT];
  Sums<DP, BT> o;
  o.zero();
#pragma unroll
  for (int i = 0; i < S::MT; i++) {
    const int r = ty + 16 * i;
    sees[i] = r < rows ? min(seq.before + (row0 + r) / group + 1, seq.keys) : 0;
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  const int most = min(seq.before + (row0 + rows - 1) / group + 1, seq.keys);
  const float scale2 = a.scale * kLog2e;
  const int64_t tiles = most > 0 ? div_up(most, BT) : 0;
  const int begin = (int)(tiles * part / split.parts) * BT, end = (int)min(tiles * (part + 1) / split.parts * BT, (int64_t)most);
  for (int j0 = begin; j0 < end; j0 += BT) {
    __syncthreads();
    if (paged) {
      find_keys<BT>(a, seq, head, j0, key_row);
      __syncthreads();
    }
    auto key = [&](const void* base, int64_t stride, int64_t head_stride, int r) -> const T* {
      if (paged) return key_row[r] < 0 ? nullptr : (const T*)base + key_row[r] * D;
      return j0 + r < seq.keys ? (const T*)base + (int64_t)(seq.first + j0 + r) * stride + head * head_stride : nullptr;
    };
    load_rows<T, DP, BT>(sk, D, [&](int r) { return key(a.k[rank], a.k_stride, a.k_head, r); });
    __syncthreads();
    float s[S::MT][S::MT];
    dots<DP, BT>(sq, sk, D, s);
    __syncthreads();
    load_rows<T, DP, BT>(sk, D, [&](int r) { return key(a.v[rank], a.v_stride, a.v_head, r); });
#pragma unroll
    for (int i = 0; i < S::MT; i++) {
      float top = m[i];
#pragma unroll
      for (int j = 0; j < S::MT; j++) {
        const int c = tx + 16 * j;
        s[i][j] = j0 + c < sees[i] && (!paged || key_row[c] >= 0) ? s[i][j] * scale2 : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      const float keep = top == -INFINITY ? 1.f : exp2_fast(m[i] - top);
      const float by = top == -INFINITY ? 0.f : top;  // nothing seen so far: the weights are 0
      m[i] = top;
      l[i] *= keep;
      o.scale_row(i, keep);
#pragma unroll
      for (int j = 0; j < S::MT; j++) {
        const float p = exp2_fast(s[i][j] - by);
        l[i] += p;
        sp[(ty + 16 * i) * S::LP + tx + 16 * j] = p;
      }
    }
    __syncthreads();
    o.add(sp, sk);
  }
#pragma unroll
  for (int i = 0; i < S::MT; i++) {
    const int r = ty + 16 * i;
    const float sum = sum16(l[i]);
    if (r >= rows) continue;
    if (split.parts > 1) {
      float* const to =
          split.sums + ((((int64_t)rank * a.kv_heads + head) * slots + slot) * split.parts + part) * kPartFloats<DP, BT>;
      o.store_row(i, to + r * DP, DP, 1.f);
      if (tx == 0) {
        to[BT * DP + r] = m[i];
        to[BT * (DP + 1) + r] = sum;
      }
      continue;
    }
    o.store_row(i, (T*)a.out[rank] + (int64_t)token_of(r) * a.out_stride + (int64_t)head_of(r) * a.out_head, D,
                sum == 0.f ? 0.f : 1.f / sum);
    if (a.lse[rank] != nullptr && tx == 0)
      a.lse[rank][(int64_t)token_of(r) * a.q_heads + head_of(r)] = (m[i] + log2f(sum)) / kLog2e;
  }
}

// The parts of a row's keys, a block a row: groups of threads take every G-th part, a
// pair of elements a thread, and join in order.
template <typename T, int DP, int BT>
__global__ void __launch_bounds__(128) prompt_join_rows_kernel(const __grid_constant__ PromptArgs a,
                                                               const __grid_constant__ Split split, int64_t slots) {
  constexpr int G = 128 / (DP / 2);
  __shared__ float weight[kPromptParts], reduced[8];
  __shared__ float2 partial[G][DP / 2];
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int group = a.q_heads / a.kv_heads, D = a.head_dim, r = (int)(blockIdx.x % BT), lane = threadIdx.x & 31,
            warp = threadIdx.x >> 5;
  const int64_t item = blockIdx.x / BT, slot = item % slots;
  const int head = (int)(item / slots % a.kv_heads), rank = (int)(item / slots / a.kv_heads);
  PromptSequence seq;
  int tile;
  if (!find_sequence(a.starts, a.sequences, a.tokens, group, BT, slot, &seq, &tile)) return;
  const int row = tile * BT + r;
  if (row >= seq.length * group) return;
  const float* const sums = split.sums + item * split.parts * kPartFloats<DP, BT>;
  float top = -INFINITY, sum = 0.f;
  for (int k = threadIdx.x; k < split.parts; k += 128) top = fmaxf(top, sums[k * kPartFloats<DP, BT> + BT * DP + r]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (lane == 0) reduced[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(reduced[0], reduced[1]), fmaxf(reduced[2], reduced[3]));
  for (int k = threadIdx.x; k < split.parts; k += 128) {
    const float* p = sums + k * kPartFloats<DP, BT> + BT * DP + r;
    // below 0: a part with no weight at all has left nothing. (One of NaN scores alone has a sum of NaN, and no maximum.)
    const float w = p[BT] == 0.f ? -1.f : exp2_fast(p[0] - top);
    weight[k] = w;
    if (!(w < 0.f)) sum = fmaf(p[BT], w, sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0) reduced[4 + warp] = sum;
  __syncthreads();
  sum = (reduced[4] + reduced[5]) + (reduced[6] + reduced[7]);
  const int g = threadIdx.x / (DP / 2), d = threadIdx.x % (DP / 2) * 2;
  if (g < G) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int k = g; k < split.parts; k += G) {
      const float w = weight[k];
      const float2 x = *reinterpret_cast<const float2*>(sums + k * kPartFloats<DP, BT> + r * DP + d);
      if (!(w < 0.f)) {
        v.x = fmaf(x.x, w, v.x);
        v.y = fmaf(x.y, w, v.y);
      }
    }
    partial[g][d / 2] = v;
  }
  __syncthreads();
  const int64_t token = seq.first + row / group, query = head * group + row % group;
  if (g == 0 && d < D) {
    float2 v = partial[0][d / 2];
#pragma unroll
    for (int k = 1; k < G; k++) {
      v.x += partial[k][d / 2].x;
      v.y += partial[k][d / 2].y;
    }
    const float by = sum == 0.f ? 0.f : 1.f / sum;
    store2((T*)a.out[rank] + token * a.out_stride + query * a.out_head + d, sum == 0.f ? 0.f : v.x * by, sum == 0.f ? 0.f : v.y * by);
  }
  if (threadIdx.x == 0 && a.lse[rank] != nullptr) a.lse[rank][token * a.q_heads + query] = (top + log2f(sum)) / kLog2e;
}

// The sequence of a token: the last one that begins at or before it. A whole warp looks.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int sequences, int token) {
  int lo = 0, hi = sequences;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, probe = lo + (int)(threadIdx.x & 31) * step;
    const int count = __popc(__ballot_sync(~0u, probe < hi && starts[probe < hi ? probe : lo] <= token));
    lo += (count > 1 ? count - 1 : 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Few parts of a row's keys, a warp a row of all heads and tokens: lanes have a part's
// weight each, and pairs of elements.
template <typename T>
__global__ void __launch_bounds__(128) prompt_join_few_kernel(const __grid_constant__ PromptArgs a,
                                                              const __grid_constant__ FewParts f) {
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int group = a.q_heads / a.kv_heads, D = a.head_dim, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), each = (int64_t)a.tokens * a.q_heads;
  const int rank = (int)(r / each);
  if (rank >= a.nranks) return;
  const int token = (int)(r % each / a.q_heads), query = (int)(r % a.q_heads), head = query / group, in_group = query % group;
  const int s = sequence_of(a.starts, a.sequences, token), first = a.starts[s], end = a.starts[s + 1];
  if (first < 0 || end > a.tokens || token < first || token >= end) return;
  // the item, its tile of rows, and the row in it
  const int at = token - first;
  int64_t item;
  int tile = 0, row;
  if (f.pairs) {
    const int per_tile = f.tile_rows / group, unit = 2 * per_tile;
    item = (int64_t)(first / unit + s + at / unit) * (a.kv_heads * a.nranks) + rank * a.kv_heads + head;
    tile = at % unit / per_tile;
    row = at % per_tile * group + in_group;
  } else {
    const int64_t slot = (int64_t)first * group / f.tile_rows + s + (at * group + in_group) / f.tile_rows;
    item = ((int64_t)rank * a.kv_heads + head) * f.slots + slot;
    row = (at * group + in_group) % f.tile_rows;
  }
  const float* const sums = f.sums + item * f.parts * f.part_floats + (int64_t)tile * f.tile_rows * (f.row_floats + 2);
  const float* const numbers = sums + lane * f.part_floats + f.tile_rows * f.row_floats + row;
  const float m = lane < f.parts ? numbers[0] : -INFINITY, l = lane < f.parts ? numbers[f.tile_rows] : 0.f;
  float top = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  // below 0: a part with no weight at all has left nothing. (One of NaN scores alone has a sum of NaN, and no maximum.)
  const float w = l == 0.f ? -1.f : exp2_fast(m - top);
  float sum = w < 0.f ? 0.f : l * w;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  const float by = sum == 0.f ? 0.f : 1.f / sum;
  T* const out = (T*)a.out[rank] + (int64_t)token * a.out_stride + query * a.out_head;
  for (int d0 = 0; d0 < D; d0 += 64) {
    const int d = d0 + lane * 2;
    float2 x[kFewParts];
#pragma unroll
    for (int k = 0; k < kFewParts; k++) {
      x[k] = make_float2(0.f, 0.f);
      if (__shfl_sync(~0u, w, k) >= 0.f && d < D) x[k] = *reinterpret_cast<const float2*>(sums + k * f.part_floats + row * f.row_floats + d);
    }
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kFewParts; k++) {
      const float y = __shfl_sync(~0u, w, k);
      if (y < 0.f) continue;
      v.x = fmaf(x[k].x, y, v.x);
      v.y = fmaf(x[k].y, y, v.y);
    }
    if (d < D) store2(out + d, sum == 0.f ? 0.f : v.x * by, sum == 0.f ? 0.f : v.y * by);
  }
  if (lane == 0 && a.lse[rank] != nullptr) a.lse[rank][(int64_t)token * a.q_heads + query] = (top + log2f(sum)) / kLog2e;
}

// Weight of a score s. The difference from lse is taken ahead of the base's factor: the weight is off by roundings of the
// difference, not of scores and lse in another base, and is 1 where the two are the same. (With delta from the same dp, 2
// tokens of 2 / 1 heads of 128: dq off by 1.5e-7 of its norm, where it was 3.3e-7.)
__device__ __forceinline__ float weight_of(float s, bool seen, float scale, float lse) {
  return seen ? exp2_fast(fmaf(s, scale, -lse) * kLog2e) : 0.f;
}
// A score that a row sees alone has none (and would have what roundings leave of dp - delta), unless it is no number.
__device__ __forceinline__ float score_gradient(float p, float dp, bool seen, bool alone, float delta) {
  return seen ? p * (dp - delta) * (alone ? 0.f : 1.f) : 0.f;
}

// dq of BT rows, and delta of each for the other kernel. Delta by way of the result has the roundings of other sums than
// dO . v has; over few keys, where the two nearly cancel, they count.
template <typename T, int DP, int BT>
__global__ void __launch_bounds__(kThreads, DP <= 96 ? 2 : 1) prompt_bwd_rows_kernel(const __grid_constant__ PromptBwdArgs a) {
  using S = Shape<DP, BT>;
  extern __shared__ __align__(16) float shared[];
  float *sq = shared, *sg = sq + S::kRows, *sk = sg + S::kRows, *sv = kApart<DP> ? sk + S::kRows : sk,
        *sp = sv + S::kRows;  // values and keys may take turns
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  if (blockIdx.x == 0) check_starts(a.starts, a.sequences, a.tokens, a.ws, threadIdx.x, kThreads);
  const Place place(a, 1);
  const int group = a.q_heads / a.kv_heads, head = place.head, rank = place.rank, D = a.head_dim;
  PromptSequence seq;
  int tile;
  if (!find_sequence(a.starts, a.sequences, a.tokens, group, BT, place.slots - 1 - place.slot, &seq, &tile)) return;
  const int row0 = tile * BT, rows = min(BT, seq.length * group - row0);
  auto token_of = [&](int r) { return (int64_t)(seq.first + (row0 + r) / group); };
  auto head_of = [&](int r) { return (int64_t)(head * group + (row0 + r) % group); };
  auto row_of = [&](const void* base, int64_t stride, int64_t head_stride, int r) {
    return r < rows ? (const T*)base + token_of(r) * stride + head_of(r) * head_stride : nullptr;
  };
  load_rows<T, DP, BT>(sg, D, [&](int r) { return row_of(a.dout[rank], a.dout_stride, a.dout_head, r); });
  load_rows<T, DP, BT>(sk, D, [&](int r) { return row_of(a.out[rank], a.out_stride, a.out_head, r); });
  load_rows<T, DP, BT>(sq, D, [&](int r) { return row_of(a.q[rank], a.q_stride, a.q_head, r); });
  __syncthreads();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int sees[S::MT];
  float lse[S::MT], delta[S::MT];
  Sums<DP, BT> dq;
  dq.zero();
  const int most = (row0 + rows - 1) / group + 1;
  const bool whole = most <= BT;  // all keys of the rows are in one tile: delta is the sum of p (dO . v), at hand there
  float* const deltas = reinterpret_cast<float*>(a.ws + kOpScratchOffset) + (int64_t)rank * a.tokens * a.q_heads;
#pragma unroll
  for (int i = 0; i < S::MT; i++) {
    const int r = ty + 16 * i;
    float x = 0.f;
    for (int d = tx; d < DP; d += 16) x = fmaf(sg[r * S::LD + d], sk[r * S::LD + d], x);
    delta[i] = sum16(x);
    sees[i] = r < rows ? (row0 + r) / group + 1 : 0;
    lse[i] = 0.f;
    if (r < rows) {
      const int64_t at = token_of(r) * a.q_heads + head_of(r);
      lse[i] = a.lse[rank][at];
      if (tx == 0 && !whole) deltas[at] = delta[i];
    }
  }
  for (int j0 = 0; j0 < most; j0 += BT) {
    __syncthreads();
    auto key = [&](const void* base, int64_t stride, int64_t head_stride, int r) {
      return j0 + r < seq.keys ? (const T*)base + (int64_t)(seq.first + j0 + r) * stride + head * head_stride : nullptr;
    };
    float s[S::MT][S::MT], dp[S::MT][S::MT];
    load_rows<T, DP, BT>(sv, D, [&](int r) { return key(a.v[rank], a.v_stride, a.v_head, r); });
    if (kApart<DP>) load_rows<T, DP, BT>(sk, D, [&](int r) { return key(a.k[rank], a.k_stride, a.k_head, r); });
    __syncthreads();
    dots<DP, BT>(sg, sv, D, dp);
    if (!kApart<DP>) {
      __syncthreads();
      load_rows<T, DP, BT>(sk, D, [&](int r) { return key(a.k[rank], a.k_stride, a.k_head, r); });
      __syncthreads();
    }
    dots<DP, BT>(sq, sk, D, s);
#pragma unroll
    for (int i = 0; i < S::MT; i++) {
      const int r = ty + 16 * i;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < S::MT; j++) {
        const bool seen = j0 + tx + 16 * j < sees[i];
        s[i][j] = weight_of(s[i][j], seen, a.scale, lse[i]);
        if (seen) sum = fmaf(s[i][j], dp[i][j], sum);
      }
      if (whole) {
        delta[i] = sum16(sum);
        if (r < rows && tx == 0) deltas[token_of(r) * a.q_heads + head_of(r)] = delta[i];
      }
#pragma unroll
      for (int j = 0; j < S::MT; j++)
        sp[r * S::LP + tx + 16 * j] = score_gradient(s[i][j], dp[i][j], j0 + tx + 16 * j < sees[i], sees[i] == 1, delta[i]);
    }
    __syncwarp();
    dq.add(sp, sk);
  }
#pragma unroll
  for (int i = 0; i < S::MT; i++) {
    const int r = ty + 16 * i;
    if (r < rows) dq.store_row(i, (T*)a.dq[rank] + token_of(r) * a.dq_stride + head_of(r) * a.dq_head, D, a.scale);
  }
}

// dk and dv of BT keys, over the rows of all query heads of the group that see them.
template <typename T, int DP, int BT>
__global__ void __launch_bounds__(kThreads, DP <= 96 ? 2 : 1) prompt_bwd_keys_kernel(const __grid_constant__ PromptBwdArgs a,
                                                                                     const __grid_constant__ KeyParts split) {
  using S = Shape<DP, BT>;
  extern __shared__ __align__(16) float shared[];
  float *sk = shared, *sv = sk + S::kRows, *sq = sv + S::kRows, *sg = kApart<DP> ? sq + S::kRows : sq,
        *sp = sg + S::kRows, *sd = sp + S::kScores;  // Q and dO may take turns
  __shared__ float slse[BT], sdelta[BT];
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const Place place(a, split.parts);
  const int group = a.q_heads / a.kv_heads, head = place.head, rank = place.rank, part = place.part, D = a.head_dim;
  PromptSequence seq;
  int tile;
  // the first keys of a sequence are seen by the most rows: they start first
  if (!find_sequence(a.starts, a.sequences, a.tokens, 1, BT, place.slot, &seq, &tile)) return;
  const int j0 = tile * BT, keys = min(BT, seq.length - j0);
  auto key = [&](const void* base, int64_t stride, int64_t head_stride, int r) {
    return r < keys ? (const T*)base + (int64_t)(seq.first + j0 + r) * stride + head * head_stride : nullptr;
  };
  load_rows<T, DP, BT>(sk, D, [&](int r) { return key(a.k[rank], a.k_stride, a.k_head, r); });
  load_rows<T, DP, BT>(sv, D, [&](int r) { return key(a.v[rank], a.v_stride, a.v_head, r); });
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  Sums<DP, BT> dk, dv;
  dk.zero();
  dv.zero();
  const float* deltas = reinterpret_cast<const float*>(a.ws + kOpScratchOffset) + (int64_t)rank * a.tokens * a.q_heads;
  const int64_t tiles = div_up((int64_t)(seq.length - j0) * group, BT);
  const int first = j0 * group + (int)(tiles * part / split.parts) * BT, last = j0 * group + (int)(tiles * (part + 1) / split.parts) * BT;
  for (int row0 = first; row0 < min(last, seq.length * group); row0 += BT) {
    const int rows = min(BT, seq.length * group - row0);
    auto token_of = [&](int r) { return (int64_t)(seq.first + (row0 + r) / group); };
    auto head_of = [&](int r) { return (int64_t)(head * group + (row0 + r) % group); };
    auto row_of = [&](const void* base, int64_t stride, int64_t head_stride, int r) {
      return r < rows ? (const T*)base + token_of(r) * stride + head_of(r) * head_stride : nullptr;
    };
    __syncthreads();
    load_rows<T, DP, BT>(sq, D, [&](int r) { return row_of(a.q[rank], a.q_stride, a.q_head, r); });
    if (kApart<DP>) load_rows<T, DP, BT>(sg, D, [&](int r) { return row_of(a.dout[rank], a.dout_stride, a.dout_head, r); });
    for (int r = threadIdx.x; r < BT; r += kThreads) {
      const int64_t at = r < rows ? token_of(r) * a.q_heads + head_of(r) : 0;
      slse[r] = r < rows ? a.lse[rank][at] : 0.f;
      sdelta[r] = r < rows ? deltas[at] : 0.f;
    }
    __syncthreads();
    float s[S::MT][S::MT], dp[S::MT][S::MT];  // rows of the tile are keys here, columns the queries
    dots<DP, BT>(sk, sq, D, s);
    if (!kApart<DP>) {
      __syncthreads();
      load_rows<T, DP, BT>(sg, D, [&](int r) { return row_of(a.dout[rank], a.dout_stride, a.dout_head, r); });
      __syncthreads();
    }
    dots<DP, BT>(sv, sg, D, dp);
#pragma unroll
    for (int i = 0; i < S::MT; i++)
#pragma unroll
      for (int j = 0; j < S::MT; j++) {
        const int r = tx + 16 * j, c = ty + 16 * i;
        const bool seen = r < rows && c < keys && j0 + c <= (row0 + r) / group;
        const float p = weight_of(s[i][j], seen, a.scale, slse[r]);
        sp[c * S::LP + r] = p;
        sd[c * S::LP + r] = score_gradient(p, dp[i][j], seen, row0 + r < group, sdelta[r]);
      }
    __syncwarp();  // a row's weights are written and read by the same half warp
    dv.add(sp, sg);
    if (!kApart<DP>) {
      __syncthreads();
      load_rows<T, DP, BT>(sq, D, [&](int r) { return row_of(a.q[rank], a.q_stride, a.q_head, r); });
      __syncthreads();
    }
    dk.add(sd, sq);
  }
#pragma unroll
  for (int i = 0; i < S::MT; i++) {
    const int r = ty + 16 * i;
    if (r >= keys) continue;
    const int64_t token = seq.first + j0 + r;
    if (split.parts > 1) {
      const int64_t each = key_part_floats(a.nranks, a.tokens, a.kv_heads, D);
      float* const to = split.sums + 2 * part * each + (((int64_t)rank * a.tokens + token) * a.kv_heads + head) * D;
      dk.store_row(i, to, D, a.scale);
      dv.store_row(i, to + each, D, 1.f);
      continue;
    }
    dk.store_row(i, (T*)a.dk[rank] + token * a.dk_stride + head * a.dk_head, D, a.scale);
    dv.store_row(i, (T*)a.dv[rank] + token * a.dv_stride + head * a.dv_head, D, 1.f);
  }
}

// dk and dv of eight elements a thread, from the parts' sums.
template <typename T>
__global__ void __launch_bounds__(256) prompt_key_parts_kernel(const __grid_constant__ PromptBwdArgs a,
                                                               const __grid_constant__ KeyParts split) {
  const uint32_t magic = op_start(a.ws);
  if (!op_ready(a.ws, magic)) return;
  const int width = a.kv_heads * a.head_dim, rank = blockIdx.y;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, token = at / width;
  // tokens in no sequence have no sums
  if (token < a.starts[0] || token >= a.starts[a.sequences] || token >= a.tokens) return;
  const int64_t each = key_part_floats(a.nranks, a.tokens, a.kv_heads, a.head_dim);
#pragma unroll
  for (int which = 0; which < 2; which++) {
    float sum[8] = {}, v[8];
    const float* from = split.sums + which * each + (int64_t)rank * a.tokens * width + at;
#pragma unroll 4
    for (int k = 0; k < split.parts; k++) {
      Pack8<float> x;
      x.load_stream(from + 2 * k * each);
      x.widen(v);
#pragma unroll
      for (int i = 0; i < 8; i++) sum[i] += v[i];
    }
    Pack8<T> y;
    y.narrow(sum);
    const int head = (int)(at % width) / a.head_dim, d = (int)(at % width) % a.head_dim;
    y.store(which == 0 ? (T*)a.dk[rank] + token * a.dk_stride + head * a.dk_head + d
                       : (T*)a.dv[rank] + token * a.dv_stride + head * a.dv_head + d);
  }
}

template <int DP, int BT>
constexpr int shared_bytes(int rows, int scores) {
  return (rows * Shape<DP, BT>::kRows + scores * Shape<DP, BT>::kScores) * 4;
}

int64_t delta_bytes(int nranks, int64_t tokens, int q_heads) { return align_up((int64_t)nranks * tokens * q_heads * 4, 256); }

cudaError_t launch(const void* fn, dim3 grid, int shared, cudaStream_t stream, void** params) {
  int blocks = 0;
  const cudaError_t e = resident_blocks(fn, kThreads, shared, &blocks);  // lets the kernel have its shared memory
  return e != cudaSuccess ? e : launch_op(fn, grid, kThreads, shared, stream, params);
}

// Few items' keys are split so that every block of two an SM has some, two tiles at least.
template <typename T, int DP, int BT>
cudaError_t forward(const PromptArgs& a, cudaStream_t stream) {
  int64_t slots = prompt_slots(a.tokens, a.sequences, a.q_heads / a.kv_heads, BT);
  const int64_t items = slots * a.kv_heads * a.nranks;
  Split split = {1, (float*)(a.ws + kOpScratchOffset)};
  if (items * 2 <= kPromptParts) {
    const int64_t most = a.table != nullptr ? (int64_t)a.max_blocks << a.page_shift : likely_keys(a.tokens, a.sequences);
    const int64_t room = kPromptParts / items, wanted = div_up(most, 2 * BT);
    split.parts = (int)(room < wanted ? room : wanted);
  }
  PromptArgs copy = a;
  void* params[] = {&copy, &split, &slots};
  const cudaError_t e = launch((const void*)prompt_kernel<T, DP, BT>,
                               dim3((unsigned)(items * split.parts)),
                               shared_bytes<DP, BT>(2, 1), stream, params);
  if (e != cudaSuccess || split.parts == 1) return e;
  if (split.parts <= kFewParts)
    return launch_prompt_join_few(a, {split.sums, split.parts, BT, DP, 0, kPartFloats<DP, BT>, slots}, stream);
  return launch_op((const void*)prompt_join_rows_kernel<T, DP, BT>, dim3((unsigned)(items * BT)), 128, 0, stream, params);
}

template <typename T, int DP, int BT>
cudaError_t backward(const PromptBwdArgs& a, cudaStream_t stream) {
  PromptBwdArgs copy = a;
  void* params[] = {&copy};
  const int64_t lanes = (int64_t)a.kv_heads * a.nranks;
  cudaError_t e = launch((const void*)prompt_bwd_rows_kernel<T, DP, BT>,
                               dim3((unsigned)(prompt_slots(a.tokens, a.sequences, a.q_heads / a.kv_heads, BT) * lanes)),
                               shared_bytes<DP, BT>(kApart<DP> ? 4 : 3, 1), stream, params);
  if (e != cudaSuccess) return e;
  const int64_t slots = prompt_slots(a.tokens, a.sequences, 1, BT);
  KeyParts split;
  split.parts = key_parts(slots * lanes, kPromptParts, likely_keys(a.tokens, a.sequences) * (a.q_heads / a.kv_heads) / (2 * BT),
                          kLeastPlainRowTilesFew, kLeastPlainRowTiles);
  split.sums = (float*)(a.ws + kOpScratchOffset + delta_bytes(a.nranks, a.tokens, a.q_heads));
  void* key_params[] = {&copy, &split};
  e = launch((const void*)prompt_bwd_keys_kernel<T, DP, BT>, dim3((unsigned)(slots * lanes * split.parts)),
             shared_bytes<DP, BT>(kApart<DP> ? 4 : 3, 2), stream, key_params);
  return e != cudaSuccess || split.parts == 1 ? e : launch_prompt_key_parts(a, split, stream);
}

// Whether the tensor core form takes the call: a group of heads fills no more than the
// 128 rows of a tile, sums of 128 elements a row fit tensor memory beside the scores,
// and strides are what a TMA map can say.
bool tensor_cores(int dtype, int head_dim, int group, std::initializer_list<int64_t> strides) {
  for (const int64_t s : strides)
    if (s >= (int64_t)1 << 38) return false;
  return dtype != 0 && head_dim <= 128 && group <= 128;
}

}  // namespace

// By head size, padded to 64, 96, 128 or 256.
template <typename T>
cudaError_t by_size(const PromptArgs& a, cudaStream_t stream) {
  if (a.head_dim <= 64) return forward<T, 64, 64>(a, stream);
  if (a.head_dim <= 96) return forward<T, 96, 64>(a, stream);
  if (a.head_dim <= 128) return forward<T, 128, 64>(a, stream);
  return forward<T, 256, 32>(a, stream);
}
template <typename T>
cudaError_t by_size(const PromptBwdArgs& a, cudaStream_t stream) {
  if (a.head_dim <= 64) return backward<T, 64, 64>(a, stream);
  if (a.head_dim <= 96) return backward<T, 96, 64>(a, stream);
  if (a.head_dim <= 128) return backward<T, 128, 64>(a, stream);
  return backward<T, 256, 32>(a, stream);
}

cudaError_t launch_prompt_join_few(const PromptArgs& a, const FewParts& parts, cudaStream_t stream) {
  PromptArgs copy = a;
  FewParts few = parts;
  void* params[] = {&copy, &few};
  const void* fn = a.dtype == 0 ? (const void*)prompt_join_few_kernel<float> : (const void*)prompt_join_few_kernel<uint16_t>;
  return launch_op(fn, dim3((unsigned)div_up((int64_t)a.nranks * a.tokens * a.q_heads, 4)), 128, 0, stream, params);
}

cudaError_t launch_prompt_key_parts(const PromptBwdArgs& a, const KeyParts& parts, cudaStream_t stream) {
  PromptBwdArgs copy = a;
  KeyParts split = parts;
  void* params[] = {&copy, &split};
  const void* fn = a.dtype == 0 ? (const void*)prompt_key_parts_kernel<float> : (const void*)prompt_key_parts_kernel<uint16_t>;
  const int64_t pieces = (int64_t)a.tokens * a.kv_heads * a.head_dim / 8;
  return launch_op(fn, dim3((unsigned)div_up(pieces, 256), (unsigned)a.nranks), 256, 0, stream, params);
}

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream) {
  if (a.dtype == 0) return by_size<float>(a, stream);
  if (tensor_cores(a.dtype, a.head_dim, a.q_heads / a.kv_heads,
                   {a.q_stride, a.k_stride, a.v_stride, a.out_stride, a.q_head, a.k_head, a.v_head, a.out_head}))
    return launch_prompt_attention_tc(a, stream);
  return by_size<uint16_t>(a, stream);
}

cudaError_t launch_prompt_attention_bwd(const PromptBwdArgs& a, cudaStream_t stream) {
  if (a.dtype == 0) return by_size<float>(a, stream);
  if (tensor_cores(a.dtype, a.head_dim, a.q_heads / a.kv_heads,
                   {a.q_stride, a.k_stride, a.v_stride, a.dout_stride, a.q_head, a.k_head, a.v_head, a.dout_head}))
    return launch_prompt_attention_bwd_tc(a, stream);
  return by_size<uint16_t>(a, stream);
}

// The most tokens times parts that a gradient of `tokens` or fewer leaves sums of, 0 if none is split: for each number of
// parts the most tokens that still have so many. More sequences than one never have more parts.
template <typename Tiles>
int64_t most_key_parts(int64_t tokens, int64_t lanes, int64_t unit, int64_t blocks, int64_t least_few, int64_t least, Tiles row_tiles) {
  int64_t most = 0;
  for (int parts = 2; parts <= kMostKeyParts; parts++)
    for (const int64_t waves : {1, 2, 8}) {
      const int64_t fit = waves * blocks / parts / lanes * unit - 1, t = tokens < fit ? tokens : fit;  // items * parts <= waves * blocks
      if (t > 0 && key_parts((t / unit + 1) * lanes, blocks, row_tiles(t), least_few, least) >= parts && t * parts > most)
        most = t * parts;
    }
  return most;
}

// Enough for every call of so many tokens or fewer.
int64_t prompt_attention_scratch_bytes(int nranks, int64_t tokens, int q_heads, int kv_heads, int head_dim) {
  const int64_t delta = delta_bytes(nranks, tokens, q_heads);
  // the parts of few items' keys, where they may be split: rows of O, m and l, in either form
  const int group = q_heads / kv_heads, rows = head_dim <= 128 ? 64 : 32;
  const int64_t lanes = (int64_t)kv_heads * nranks, padded = head_dim <= 64 ? 64 : head_dim <= 96 ? 96 : head_dim <= 128 ? 128 : 256;
  const bool tensor = group <= 128 && head_dim <= 128;
  int64_t parts = 0;
  if ((group / rows + 1) * lanes * 2 <= kPromptParts) parts = kPromptParts * rows * (padded + 2) * 4;
  if (tensor && lanes * 2 <= kPromptSplitBlocks) {
    const int64_t more = (int64_t)kPromptSplitBlocks * 256 * ((head_dim <= 64 ? 64 : 128) + 2) * 4;
    parts = more > parts ? more : parts;
  }
  // what parts of the rows leave of dk and dv
  int64_t split = most_key_parts(tokens, lanes, rows, kPromptParts, kLeastPlainRowTilesFew, kLeastPlainRowTiles,
                                 [&](int64_t t) { return t * group / (2 * rows); });
  if (tensor) {
    const int64_t most = most_key_parts(tokens, lanes, 128, kPromptSplitBlocks, kLeastRowTilesFew, kLeastRowTiles,
                                        [&](int64_t t) { return t / (2 * (128 / group)); });
    split = most > split ? most : split;
  }
  const int64_t gradient = delta + 2 * key_part_floats(nranks, split, kv_heads, head_dim) * 4;
  return gradient > parts ? gradient : parts;
}

}  // namespace rar
