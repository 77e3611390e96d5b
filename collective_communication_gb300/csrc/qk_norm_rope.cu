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
// eight consecutive elements a lane it took eight shuffles a row: 108 us for
// 8192 tokens of 10 heads of 128 on 8 ranks where this takes 63); the group's
// loads still cover whole lines. A group takes a strip of a few heads of one
// token, all loaded before the first is used; weights and angles are read once
// a strip. Arithmetic is two binary32 values an instruction.
//
// Bound by memory, with instruction issue close: the case above moves 340 MB in
// 62.9 us, 5.4 TB/s (0.81 of the measured copy); four strips of rows a thread and
// 60 registers keep 27 warps an SM, more rows a thread were slower (75 us with
// eight, at 78 registers).
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kNrThreads = 256;
template <typename T>
constexpr int kStrip = 4;                 // rows of a forward strip
constexpr int kBwdThreads = 128;
constexpr int kBwdStages = 4;             // rows of x and dy of a group in shared memory
constexpr int kBwdJoin = 32;              // partial weight sums that one block joins
constexpr int kNormRopeBwdBlocks = 1216;  // most blocks of a backward launch, all ranks together
constexpr int kBwdCounters = 48;          // arrival counters of a rank: two kinds, then runs of blocks
static_assert(kBwdCounters * kMaxRanks <= kOpCounters && kNormRopeBwdBlocks / kBwdJoin + 4 <= kBwdCounters, "counters");

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

// A lane's eight elements in binary32, so that elements p[j] and p[j + 2] make
// two pairs of the rotation in either layout.
struct Row8 {
  F2 p[4];
};
__device__ __forceinline__ Row8 operator*(const Row8& a, const Row8& b) {
  Row8 r;
#pragma unroll
  for (int j = 0; j < 4; j++) r.p[j] = mul2(a.p[j], b.p[j]);
  return r;
}
__device__ __forceinline__ Row8 operator*(const Row8& a, float f) {
  const F2 ff = f2(f, f);
  Row8 r;
#pragma unroll
  for (int j = 0; j < 4; j++) r.p[j] = mul2(a.p[j], ff);
  return r;
}
__device__ __forceinline__ Row8 fma_row(const Row8& a, const Row8& b, const Row8& c) {
  Row8 r;
#pragma unroll
  for (int j = 0; j < 4; j++) r.p[j] = fma2(a.p[j], b.p[j], c.p[j]);
  return r;
}
__device__ __forceinline__ float dot8(const Row8& a, const Row8& b) {
  F2 s = mul2(a.p[0], b.p[0]);
#pragma unroll
  for (int j = 1; j < 4; j++) s = fma2(a.p[j], b.p[j], s);
  const float2 x = unpack(s);
  return x.x + x.y;
}

// Two chunks of four elements as they are in memory. INTER: the even elements
// of the eight make p[0], p[1], the odd ones p[2], p[3].
template <typename T, bool INTER>
struct Chunks;
template <bool INTER>
struct Chunks<uint16_t, INTER> {
  uint2 a, b;
  __device__ __forceinline__ void load(const uint16_t* row, const Lane& n) {
    a = *reinterpret_cast<const uint2*>(row + n.o0);
    b = *reinterpret_cast<const uint2*>(row + n.o1);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0, 0); }
  __device__ __forceinline__ Row8 widen() const {
    if (INTER)
      return Row8{{f2(bf16_lo(a.x), bf16_lo(a.y)), f2(bf16_lo(b.x), bf16_lo(b.y)), f2(bf16_hi(a.x), bf16_hi(a.y)),
                   f2(bf16_hi(b.x), bf16_hi(b.y))}};
    return Row8{{f2(bf16_lo(a.x), bf16_hi(a.x)), f2(bf16_lo(a.y), bf16_hi(a.y)), f2(bf16_lo(b.x), bf16_hi(b.x)),
                 f2(bf16_lo(b.y), bf16_hi(b.y))}};
  }
  __device__ __forceinline__ void narrow(const Row8& r) {
    const float2 p = unpack(r.p[0]), q = unpack(r.p[1]), s = unpack(r.p[2]), t = unpack(r.p[3]);
    if (INTER) {
      a = make_uint2(bf16_pair(p.x, s.x), bf16_pair(p.y, s.y));
      b = make_uint2(bf16_pair(q.x, t.x), bf16_pair(q.y, t.y));
    } else {
      a = make_uint2(bf16_pair(p.x, p.y), bf16_pair(q.x, q.y));
      b = make_uint2(bf16_pair(s.x, s.y), bf16_pair(t.x, t.y));
    }
  }
  __device__ __forceinline__ void store(uint16_t* row, const Lane& n) const {
    *reinterpret_cast<uint2*>(row + n.o0) = a;
    *reinterpret_cast<uint2*>(row + n.o1) = b;
  }
};
template <bool INTER>
struct Chunks<float, INTER> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, const Lane& n) {
    a = *reinterpret_cast<const float4*>(row + n.o0);
    b = *reinterpret_cast<const float4*>(row + n.o1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ Row8 widen() const {
    if (INTER) return Row8{{f2(a.x, a.z), f2(b.x, b.z), f2(a.y, a.w), f2(b.y, b.w)}};
    return Row8{{f2(a.x, a.y), f2(a.z, a.w), f2(b.x, b.y), f2(b.z, b.w)}};
  }
  __device__ __forceinline__ void narrow(const Row8& r) {
    const float2 p = unpack(r.p[0]), q = unpack(r.p[1]), s = unpack(r.p[2]), t = unpack(r.p[3]);
    a = INTER ? make_float4(p.x, s.x, p.y, s.y) : make_float4(p.x, p.y, q.x, q.y);
    b = INTER ? make_float4(q.x, t.x, q.y, t.y) : make_float4(s.x, s.y, t.x, t.y);
  }
  __device__ __forceinline__ void store(float* row, const Lane& n) const {
    *reinterpret_cast<float4*>(row + n.o0) = a;
    *reinterpret_cast<float4*>(row + n.o1) = b;
  }
};

// A lane's four angles (1, 0 where nothing turns): cosines, sines, negative sines.
struct Turn {
  F2 c[2], s[2], n[2];
};
__device__ __forceinline__ Turn load_turn(const float* row, int rot, const Lane& n) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n.turn) {
    c = *reinterpret_cast<const float4*>(row + n.angle);
    s = *reinterpret_cast<const float4*>(row + (rot >> 1) + n.angle);
  }
  return Turn{{f2(c.x, c.y), f2(c.z, c.w)}, {f2(s.x, s.y), f2(s.z, s.w)}, {f2(-s.x, -s.y), f2(-s.z, -s.w)}};
}

// R v, or R^T v with BACK.
template <bool BACK>
__device__ __forceinline__ Row8 rotate(const Row8& v, const Turn& t) {
  Row8 r;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    r.p[j] = fma2(v.p[j + 2], BACK ? t.s[j] : t.n[j], mul2(v.p[j], t.c[j]));
    r.p[j + 2] = fma2(v.p[j], BACK ? t.n[j] : t.s[j], mul2(v.p[j + 2], t.c[j]));
  }
  return r;
}

// Sum over a group; all lanes of the warp call it.
template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d, L);
  return x;
}
template <int L>
__device__ __forceinline__ float2 group_sum2(float x, float y) {  // two sums side by side
  F2 s = f2(x, y);
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) {
    const float2 p = unpack(s);
    s = add2(s, f2(__shfl_xor_sync(~0u, p.x, d, L), __shfl_xor_sync(~0u, p.y, d, L)));
  }
  return unpack(s);
}
// Subnormal x counts as it is, so that a row of zeros with such an eps has a norm
// (flushed to zero: 62.2 us for the 8192 tokens above instead of 62.9).
__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The lane's weights of a head's kind.
template <typename T, bool INTER>
__device__ __forceinline__ Row8 load_weight(const void* p, const Lane& n) {
  Chunks<T, INTER> c;
  c.zero();
  if (n.in) c.load(reinterpret_cast<const T*>(p), n);
  return c.widen();
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
  const uint32_t magic = op_start(a.ws);
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
  const int heads = in ? min(is_q ? per_q : per_kv, (is_q ? a.q_heads : a.kv_heads) - h0) : 0;
  // rows of the strip: its heads, and with CACHE from row per_kv the same heads' values (a shorter strip leaves gaps)
  const int rows = is_q ? per_q : CACHE ? 2 * per_kv : per_kv, values = CACHE && !is_q ? per_kv : kRows;

  int pos = live ? a.positions[token] : 0;
  int64_t slot = CACHE && live ? a.slots[token] : -1;  // below zero: a padding token, no cache row
  const T* x0 = reinterpret_cast<const T*>(a.qkv[rank]) + (int64_t)token * a.qkv_stride + (h0 + (is_q ? 0 : a.q_heads)) * D;
  Chunks<T, INTER> x[kRows];
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    x[i].zero();
    if (i < values) {
      if (i < heads) x[i].load(x0 + i * D, n);
    } else if (i - values < heads) {
      x[i].load(x0 + (a.kv_heads + i - values) * D, n);
    }
  }
  bool bad = false;
  if (pos < 0 || pos >= a.max_pos) { bad = true; pos = 0; }
  if (CACHE && slot >= a.num_slots) { bad = true; slot = -1; }
  const Turn turn = load_turn(a.cos_sin + (int64_t)pos * a.rot, a.rot, n);
  const Row8 w = load_weight<T, INTER>(is_q ? a.q_weight : a.k_weight, n);
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
  const int stores = kept ? heads : 0;
#pragma unroll
  for (int i = 0; i < kRows; i++) {
    if (i >= rows) break;
    if (i < values) {
      const Row8 v = x[i].widen();
      const float r = rsqrt_fast(fmaf(group_sum<L>(dot8(v, v)), inv, a.eps));
      x[i].narrow(rotate<false>(v * r * w, turn));
      if (i < stores) x[i].store(out, n);
      out += apart;
    } else {
      if (i - values < stores) x[i].store(out_v, n);
      out_v += apart;
    }
  }
  if (bad) op_report(a.ws, kErrCapacity);
}

// The gradient. z = R^T dy, dw = sum z x r, u = z w,
// dx = r u - r^3 mean(u x) x; dv is copied. A rank's blocks are of three kinds,
// for query heads, key heads and values, so one set of weights and weight sums
// stays in registers. A group walks over tokens, head by head; rows of x and dy
// come through a ring of kBwdStages rows in shared memory (16-byte asynchronous
// copies of consecutive elements, read back as the lane's two chunks), so three
// rows a group are in flight whatever the registers hold.
//
// 4097 tokens of 16 heads of 96 on 4 ranks, interleaved: 42.5 us, 4.2 TB/s (0.62 of
// the measured copy). No unit is full (0.6 instructions a scheduler and cycle, DRAM
// at 0.39): the chain of a row's loads and its two sums over the lanes bounds it,
// then instructions (12 of a group's 16 lanes work at 96 elements), then the start
// and the two joins, about 7 us together.
//
// Weight sums are added over the block's groups in group order, then over runs
// of kBwdJoin blocks and over the runs in block order, each time by the block
// that arrives last: the same bits every time.
namespace {

__device__ __forceinline__ void copy_async16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void store_zero16(uint32_t smem) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(smem), "r"(0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace

// SPLIT: few tokens, whose heads go to several groups (tested as it runs, it costs many tokens 2 to 9 %).
template <typename T, int L, bool INTER, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdArgs a,
                                                                    int q_blocks, int k_blocks, int q_split,
                                                                    int k_split) {
  constexpr int kGroups = kBwdThreads / L, kRow = L * 8, kCopies = (int)sizeof(T) / 2;
  __shared__ __align__(16) T ring[kGroups][kBwdStages][2][kRow];
  __shared__ float s_dw[kBwdThreads][9];
  __shared__ bool s_last;
  const uint32_t magic = op_start(a.ws);
  const int rank = blockIdx.y, group = threadIdx.x / L, l = threadIdx.x & (L - 1), D = a.head_dim;
  const Lane n = lane_of<INTER>(l, D, a.rot);
  const T* xs = reinterpret_cast<const T*>(a.qkv[rank]);
  T* ds = reinterpret_cast<T*>(a.dqkv[rank]);

  if (blockIdx.x >= q_blocks + k_blocks) {  // values
    const int block = blockIdx.x - q_blocks - k_blocks, blocks = gridDim.x - q_blocks - k_blocks;
    const int place = (a.q_heads + a.kv_heads) * D, packs = a.kv_heads * D / 8;
    const int64_t all = (int64_t)a.tokens * packs, step = (int64_t)blocks * kBwdThreads;
    if (!op_ready(a.ws, magic)) return;
    for (int64_t i = (int64_t)block * kBwdThreads + threadIdx.x; i < all; i += 4 * step) {
      Pack8<T> u[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int64_t e = i + j * step, token = e / packs;
        if (e < all) u[j].load(reinterpret_cast<const T*>(a.dv[rank]) + token * a.dv_stride + (e - token * packs) * 8);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int64_t e = i + j * step, token = e / packs;
        if (e < all) u[j].store(ds + token * a.dqkv_stride + place + (e - token * packs) * 8);
      }
    }
    return;
  }

  const bool is_q = blockIdx.x < q_blocks;
  // a unit is a token's heads, or where there are few tokens the `split`-th part of them
  const int split = !SPLIT ? 1 : is_q ? q_split : k_split, units = a.tokens * split;
  const int walkers = (is_q ? q_blocks : k_blocks) * kGroups;  // groups that share the units
  const int walker = (is_q ? blockIdx.x : blockIdx.x - q_blocks) * kGroups + group;
  const int heads = (is_q ? a.q_heads : a.kv_heads) / split, place = is_q ? 0 : a.q_heads * D;
  auto token_of = [&](int unit) { return SPLIT ? unit / split : unit; };
  auto part_of = [&](int unit, int token) { return SPLIT ? (unit - token * split) * heads * D : 0; };
  const int64_t g_stride = is_q ? a.dq_stride : a.dk_stride;
  const T* gs = reinterpret_cast<const T*>(is_q ? a.dq[rank] : a.dk[rank]);
  const Row8 w = load_weight<T, INTER>(is_q ? a.q_weight : a.k_weight, n);
  const F2 zero = f2(0.f, 0.f);
  Row8 dw = {{zero, zero, zero, zero}};
  const float inv = 1.f / (float)D;
  bool bad = false;
  // the warp's first group has the most units; the others run as long, with rows of zeros at the end
  const int first_walker = walker - (threadIdx.x & 31) / L;
  const int rows = first_walker < units ? ((units - 1 - first_walker) / walkers + 1) * heads : 0;
  const int mine = walker < units ? ((units - 1 - walker) / walkers + 1) * heads : 0;

  // Pointers go one head on within a unit, and are set anew at the group's next one.
  const T* fx = xs + place + l * 8;  // of the next row to ask for
  const T* fg = gs + l * 8;
  int f_unit = walker < units ? walker : 0;
  {
    const int f_token = token_of(f_unit), part = part_of(f_unit, f_token);
    fx += f_token * a.qkv_stride + part;
    fg += f_token * g_stride + part;
  }
  constexpr uint32_t kCell = kRow * sizeof(T), kSlot = 2 * kCell;  // bytes of a row of x or dy, of both
  const uint32_t cell = smem_addr(&ring[group][0][0][l * 8]);
  int f_left = mine, f_head = 0;
  uint32_t f_cell = cell;
  // the next row into the next slot; zeros after the group's last row, and always where a lane is past the head
  auto fetch = [&]() {
    if (n.in && f_left > 0) {
#pragma unroll
      for (int c = 0; c < kCopies; c++) {
        copy_async16(f_cell + 16 * c, fx + c * (16 / (int)sizeof(T)));
        copy_async16(f_cell + kCell + 16 * c, fg + c * (16 / (int)sizeof(T)));
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCopies; c++) {
        store_zero16(f_cell + 16 * c);
        store_zero16(f_cell + kCell + 16 * c);
      }
    }
    copy_async_commit();
    f_cell = f_cell == cell + (kBwdStages - 1) * kSlot ? cell : f_cell + kSlot;
    f_left--;
    fx += D;
    fg += D;
    if (++f_head == heads) {
      f_head = 0;
      f_unit += walkers;
      const int f_token = token_of(f_unit), part = part_of(f_unit, f_token);
      fx = xs + f_token * a.qkv_stride + place + part + l * 8;
      fg = gs + f_token * g_stride + part + l * 8;
    }
  };
  auto position = [&](int unit) {
    const int pos = unit < units ? a.positions[token_of(unit)] : 0;
    if (pos >= 0 && pos < a.max_pos) return pos;
    bad = true;
    return 0;
  };
#pragma unroll
  for (int s = 0; s < kBwdStages - 1; s++) fetch();
  int unit = walker, head = 0, slot = 0;
  Turn turn = load_turn(a.cos_sin + (int64_t)position(unit) * a.rot, a.rot, n);
  int pos_next = position(unit + walkers);
  auto out_of = [&](int unit) {
    const int token = token_of(unit);
    return ds + token * a.dqkv_stride + place + part_of(unit, token);
  };
  T* out = out_of(walker < units ? walker : 0);
  const int stores = n.in ? mine : 0;
  if (!op_ready(a.ws, magic)) {
    copy_async_wait<0>();
    return;
  }
  for (int r = 0; r < rows; r++) {
    copy_async_wait<kBwdStages - 2>();
    __syncwarp();  // every lane's copies of this row are there, and every lane is past the last row's slot
    Chunks<T, INTER> x, dy;
    x.load(ring[group][slot][0], n);
    dy.load(ring[group][slot][1], n);
    fetch();
    // with u = z w: dw += z x r, dx = r u - (r^3 mean(u x)) x; both sums at once
    const Row8 v = x.widen(), z = rotate<true>(dy.widen(), turn), u = z * w;
    const float2 sums = group_sum2<L>(dot8(v, v), dot8(u, v));
    // a row of zeros at a group's end must not reach dw: with eps 0 its root would be infinite
    const float root = r < mine ? rsqrt_fast(fmaf(sums.x, inv, a.eps)) : 0.f;
    dw = fma_row(z * root, v, dw);
    const float down = -inv * sums.y * root * root * root;
    const F2 down2 = f2(down, down);
    dy.narrow(fma_row(v, Row8{{down2, down2, down2, down2}}, u * root));
    if (r < stores) dy.store(out, n);
    slot = slot + 1 == kBwdStages ? 0 : slot + 1;
    out += D;
    if (++head == heads) {
      head = 0;
      unit += walkers;
      out = out_of(unit);
      turn = load_turn(a.cos_sin + (int64_t)pos_next * a.rot, a.rot, n);
      pos_next = position(unit + walkers);
    }
  }
  copy_async_wait<0>();
  if (bad) op_report(a.ws, kErrCapacity);

  // partial sums of the rank's blocks: [block][D], the query blocks first
  float* parts = reinterpret_cast<float*>(a.ws + kOpScratchOffset) + (int64_t)rank * gridDim.x * D;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    s_dw[threadIdx.x][2 * j] = unpack(dw.p[j]).x;
    s_dw[threadIdx.x][2 * j + 1] = unpack(dw.p[j]).y;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kBwdThreads) {
    // the lane and chunk that hold element e
    const int half = a.rot >> 1;
    const bool turned = !INTER && e < a.rot;
    const int from = turned ? (e < half ? e : e - half) >> 2 : e >> 3;
    const int j = turned ? (e & 3) + (e < half ? 0 : 4) : INTER ? (e & 1) * 4 + ((e & 7) >> 1) : e & 7;
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; g++) s += s_dw[g * L + from][j];
    parts[(int64_t)blockIdx.x * D + e] = s;
  }
  // join: runs of kBwdJoin blocks of one kind, then the kind's runs
  const int k0 = is_q ? 0 : q_blocks, kind_blocks = is_q ? q_blocks : k_blocks;
  const int quads = D >> 2, many = kBwdThreads / quads, quad = threadIdx.x % quads, turn_of = threadIdx.x / quads;
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes) + rank * kBwdCounters;
  int from = k0 + ((int)blockIdx.x - k0) / kBwdJoin * kBwdJoin, apart = 1;
  int count = min(kBwdJoin, k0 + kind_blocks - from);
  uint32_t* counter = counters + 2 + from / kBwdJoin + (is_q ? 0 : 1);  // runs of the two kinds do not share one
  for (;;) {
    __syncthreads();
    if (threadIdx.x == 0) {
      // releases the block's sums, and acquires the others' if it is the last
      s_last = atom_add_acq_rel_u32(counter, 1u) == (uint32_t)(count - 1);
      if (s_last) *counter = 0;
    }
    __syncthreads();
    if (!s_last) return;
    // four elements a thread; the threads that share them take every `many`-th partial, eight loads at a time whatever
    // is left (loops over the rest cost up to 3 us), then join in that order
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turn_of < many) {
      for (int i0 = turn_of; i0 < count; i0 += 8 * many) {
        float4 y[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const int i = i0 + j * many;
          y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < count)
            y[j] = __ldcg(reinterpret_cast<const float4*>(parts + (int64_t)(from + i * apart) * D + quad * 4));
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
          s.x += y[j].x; s.y += y[j].y; s.z += y[j].z; s.w += y[j].w;
        }
      }
    }
    s_dw[threadIdx.x][0] = s.x;
    s_dw[threadIdx.x][1] = s.y;
    s_dw[threadIdx.x][2] = s.z;
    s_dw[threadIdx.x][3] = s.w;
    __syncthreads();
    const bool whole = apart > 1 || count == kind_blocks;
    float* out = whole ? (is_q ? a.dq_weight[rank] : a.dk_weight[rank]) : parts + (int64_t)from * D;
    for (int e = threadIdx.x; e < D; e += kBwdThreads) {
      float t = 0.f;
      for (int k = 0; k < many && k < count; k++) t += s_dw[k * quads + (e >> 2)][e & 3];
      out[e] = t;
    }
    if (whole) return;
    from = k0;
    apart = kBwdJoin;
    count = (kind_blocks + kBwdJoin - 1) / kBwdJoin;
    counter = counters + (is_q ? 0 : 1);
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
const void* backward_of(bool inter, bool split) {
  return inter ? (split ? (const void*)norm_rope_bwd_kernel<T, L, true, true> : (const void*)norm_rope_bwd_kernel<T, L, true, false>)
               : (split ? (const void*)norm_rope_bwd_kernel<T, L, false, true>
                        : (const void*)norm_rope_bwd_kernel<T, L, false, false>);
}
template <typename T>
const void* backward_of(int lanes, bool inter, bool split) {
  return lanes == 8 ? backward_of<T, 8>(inter, split) : lanes == 16 ? backward_of<T, 16>(inter, split)
                                                                    : backward_of<T, 32>(inter, split);
}

}  // namespace

int64_t norm_rope_scratch_bytes(int nranks, int head_dim) {
  return (kNormRopeBwdBlocks + 3ll * nranks) * head_dim * (int64_t)sizeof(float);
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
  return launch_op(fn, grid, kNrThreads, 0, stream, params);
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, cudaStream_t stream) {
  const int lanes = lanes_of(a.head_dim), groups = kBwdThreads / lanes;
  auto kernel = [&](bool split) {
    return a.dtype == kF32 ? backward_of<float>(lanes, a.interleaved != 0, split)
                           : backward_of<uint16_t>(lanes, a.interleaved != 0, split);
  };
  int resident = 0;
  const cudaError_t e = resident_blocks(kernel(false), kBwdThreads, 0, &resident);
  if (e != cudaSuccess) return e;
  // one resident wave, shared out in proportion to the kinds' bytes: x, dy and dx of query and key heads, dv twice
  const int64_t most = imin(kNormRopeBwdBlocks, (int64_t)resident) / a.nranks;
  const int64_t q = 3ll * a.q_heads, k = 3ll * a.kv_heads, v = 2ll * a.kv_heads;
  auto share = [&](int64_t weight) { return imax(1, most * weight / (q + k + v)); };
  auto blocks_of = [&](int64_t weight, int64_t units) { return (int)imax(1, imin(div_up(units, groups), share(weight))); };
  // Fewer tokens than groups: a token's heads go to several groups in equal parts, of 2 heads or more while the blocks join
  // in one level, else of 8 or more (3 tokens of 32 and 4 heads of 192: 5 us against 14; 2048 of 32 and 8 heads of 128
  // 17.5 against 21.8; 235 of 16 and 2 heads of 256 in f32 11.8 with 8 heads a part, 13.2 with 4, 13.6 undivided).
  auto split_of = [&](int64_t weight, int heads) {
    int split = 1;
    for (int s = 2; s <= heads; s++) {
      const int64_t units = (int64_t)a.tokens * s;
      if (heads % s == 0 && units <= share(weight) * groups && heads / s >= (units <= kBwdJoin * groups ? 2 : 8)) split = s;
    }
    return split;
  };
  int q_split = split_of(q, a.q_heads), k_split = split_of(k, a.kv_heads);
  int q_blocks = blocks_of(q, (int64_t)a.tokens * q_split), k_blocks = blocks_of(k, (int64_t)a.tokens * k_split);
  const int v_blocks = blocks_of(v, a.tokens);
  dim3 grid((unsigned)(q_blocks + k_blocks + v_blocks), (unsigned)a.nranks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: qk_norm_rope_backward nranks=%d tokens=%d heads=%d/%d dim=%d rot=%d grid=%ux%u\n",
                 a.nranks, a.tokens, a.q_heads, a.kv_heads, a.head_dim, a.rot, grid.x, grid.y);
  void* params[] = {const_cast<NormRopeBwdArgs*>(&a), &q_blocks, &k_blocks, &q_split, &k_split};
  return launch_op(kernel(q_split * k_split > 1), grid, kBwdThreads, 0, stream, params);
}

}  // namespace rar
