// Rotary positions with three axes, and the per-head norm of queries and keys
// with that rotation in the same pass, on the way into (or out of) block order.
//
// Mathematics, per row x of d elements (one token of one head):
//   norm      r = 1 / sqrt(mean(x^2) + eps),  n = x r,  u = n w
//   rotation  the pair p of the first rd = dt + dh + dw elements turns by the
//             angle of its axis: (a, b) -> (a c - b s, a s + b c); pairs
//             [0, dt/2) follow the token's time, then dh/2 its height, dw/2 its
//             width.  A rotation's gradient is the rotation by -angle.
//   gradient  du = R^T dy,  dw += du n,  dn = du w,
//             dx = r (dn - n mean(dn n)); r and n are computed again from x.
// The angles come from a table of (cos, sin) per axis and position, a few KB
// that stays in L1: a token costs no angle traffic, where an [N, rd / 2] table
// would add as many bytes as a head of bf16 rows.
//
// What bounds it: memory.  Every element is read once and written once
// (backward: x and dy read, dx written).  A row is held by d / 8 lanes, eight
// elements each, so the row sums are three or four shuffles.  A block walks
// token tiles of one unit (up to kMaxHeads heads of one tensor and batch
// element): a token's position, perm entry and (cos, sin) are looked up once
// for its heads, the weight once for the block, and the next rows' loads are in
// flight while a batch of rows is worked on.  Rotation alone runs at the copy
// rate (q and k of 32,760 tokens, 12 heads of 128: 403 MB in 62 us); with the
// norm's row sums 604 MB take 96 us, 96 % of it.
#include "lbsa_train_device.cuh"

namespace lbsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeads = 16;    // heads of a unit

struct RopeArgs {
  RopeItem it[3];
  int count;
  int chunk_end[3];              // running number of (batch, head chunk) units per item
  int heads[3];                  // heads of a unit (1 .. kMaxHeads)
  int N, d;
  RopePos pos;
  const int32_t* perm;
  float eps;
  int inverse;                   // rotation by -angle, scatter
  int32_t* status;
  float* partial;                // backward: [weight rows of a unit][gridDim.y][gridDim.x][d], a block's weight gradients
};

// The elements of a row that a lane holds.
// interleaved: eight in a row, pairs 4 l .. 4 l + 3.
// half-split: element e of the first half pairs with e + rd / 2, so a lane
// holds four of each half, 4 l .. and rd / 2 + 4 l ..: its pairs are the same
// ones, and no element comes from another lane: a layer's norm and rotation
// (21 x 30 x 52 tokens, q, k, v of 12 heads of 128) 108 us, 130 us with eight
// shuffles a row.  Past rd eight in a row.
struct Place {
  int at, gap;                   // the first four; from there to the second four
  __device__ __forceinline__ Place(bool half, const RopePos& pos, int lane) {
    const int rd = pos.dt + pos.dh + pos.dw;
    const bool split = half && lane * 8 < rd;
    at = split ? lane * 4 : lane * 8;
    gap = split ? rd / 2 : 4;
  }
};

template <typename T, bool HALF>
struct Eight;
template <bool HALF>
struct Eight<__nv_bfloat16, HALF> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int gap) {
    if (HALF) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p)), b = __ldg(reinterpret_cast<const uint2*>(p + gap));
      v = make_uint4(a.x, a.y, b.x, b.y);
    } else {
      v = __ldg(reinterpret_cast<const uint4*>(p));
    }
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void copy_to(__nv_bfloat16* p, int gap) const {
    if (HALF) {
      *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(p + gap) = make_uint2(v.z, v.w);
    } else {
      *reinterpret_cast<uint4*>(p) = v;
    }
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, int gap, const float (&f)[8]) {
    Eight e;
    e.v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    e.copy_to(p, gap);
  }
};
template <bool HALF>
struct Eight<float, HALF> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int gap) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p + (HALF ? gap : 4)));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void copy_to(float* p, int gap) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + (HALF ? gap : 4)) = b;
  }
  __device__ __forceinline__ static void store(float* p, int gap, const float (&f)[8]) {
    Eight e;
    e.a = make_float4(f[0], f[1], f[2], f[3]);
    e.b = make_float4(f[4], f[5], f[6], f[7]);
    e.copy_to(p, gap);
  }
};

// A lane's share of the rotation: pairs 4 l .. 4 l + 3.
template <bool HALF>
struct Turn {
  float c[4], s[4];
  bool on[4];                    // tokens past the grid and pairs past rd / 2 keep their place
  // token: source (raster) index
  __device__ __forceinline__ void look(const RopePos& pos, int lane, int token, float sign) {
    const int ht = pos.dt >> 1, hh = pos.dh >> 1, hw = pos.dw >> 1, half = ht + hh + hw;
    const bool in = token < pos.tokens;
    const uint32_t area = static_cast<uint32_t>(pos.Hg) * pos.Wg;
    const uint32_t tok = static_cast<uint32_t>(in ? token : 0);
    const uint32_t t = tok / area, r = tok - t * area, h = r / pos.Wg, w = r - h * pos.Wg;
    // pair p of an axis: its table row's start plus p's place in the axis
    const int row_t = static_cast<int>(t) * ht;
    const int row_h = pos.T * ht + static_cast<int>(h) * hh - ht;
    const int row_w = pos.T * ht + pos.Hg * hh + static_cast<int>(w) * hw - ht - hh;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = lane * 4 + j;
      float2 cs = make_float2(1.f, 0.f);
      on[j] = in && p < half;
      if (on[j]) cs = __ldg(pos.table + (p + (p < ht ? row_t : p < ht + hh ? row_h : row_w)));
      c[j] = cs.x;
      s[j] = cs.y * sign;
    }
  }
  __device__ __forceinline__ void apply(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float &a = f[HALF ? j : 2 * j], &b = f[HALF ? j + 4 : 2 * j + 1];
      const float x = a * c[j] - b * s[j], y = a * s[j] + b * c[j];
      a = on[j] ? x : a;         // not x: an infinity beside it would make it NaN
      b = on[j] ? y : b;
    }
  }
};

// sums of the lanes of each row, n of them side by side
template <int LANES, int n>
__device__ __forceinline__ void row_sums(float (&v)[n]) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

template <bool HALF>
__device__ __forceinline__ void load_weight(const RopeItem& it, int head, Place l, int d, float (&w)[8]) {
  const long long at = static_cast<long long>(it.weight_heads > 1 ? head : 0) * d + l.at;
  if (it.weight_dtype == LBSA_F32) {
    Eight<float, HALF> v;
    v.load(static_cast<const float*>(it.weight) + at, l.gap);
    v.get(w);
  } else {
    Eight<__nv_bfloat16, HALF> v;
    v.load(static_cast<const __nv_bfloat16*>(it.weight) + at, l.gap);
    v.get(w);
  }
}

// The source token of a slot: -1 past the last slot, or for a bad perm entry
// (reported by one lane).
__device__ __forceinline__ int token_of(const RopeArgs& a, int slot, bool report) {
  if (slot >= a.N) return -1;
  const int tok = a.perm ? __ldg(a.perm + slot) : slot;
  if (tok >= 0 && tok < a.N) return tok;
  if (report) raise_status(a.status, LBSA_ERR_BAD_INDEX);
  return -1;
}

struct Unit {
  int item, b, h0, nh;
};
__device__ __forceinline__ Unit unit_of(const RopeArgs& a, int y) {
  Unit u;
  u.item = y < a.chunk_end[0] ? 0 : y < a.chunk_end[1] ? 1 : 2;
  const int at = y - (u.item ? a.chunk_end[u.item - 1] : 0);
  const int per = (a.it[u.item].H + a.heads[u.item] - 1) / a.heads[u.item];   // chunks of one batch element
  u.b = at / per;
  u.h0 = (at - u.b * per) * a.heads[u.item];
  u.nh = min(a.heads[u.item], a.it[u.item].H - u.h0);
  return u;
}

// What a unit's rows need is known to the compiler, so that a batch's rows are
// worked on side by side, without a branch between them: for a layer's q, k, v
// (21 x 30 x 52 tokens, 12 heads of 128, bf16) the call takes 99 to 102 us, 105
// where the kernel asks row by row.  A weight row for each head is read again
// for each row (122 us), as eight more registers a head would not fit.
template <typename T, int D, bool HALF, bool NORM, bool ROTATE, bool PER_HEAD>
__device__ __forceinline__ void rope_rows(const RopeArgs& a, const RopeItem& it, const Unit& u) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  constexpr int kBatch = 8 / sizeof(T);          // heads of a token that a thread loads together: 64 bytes
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Place pl(HALF, a.pos, lane);
  const T* x = static_cast<const T*>(it.x) + u.b * it.xs[0] + u.h0 * it.xs[1] + pl.at;
  T* y = static_cast<T*>(it.y) + u.b * it.ys[0] + u.h0 * it.ys[1] + pl.at;
  const int64_t x_head = it.xs[1], y_head = it.ys[1];
  Turn<HALF> turn;
  float w[8];
  if (NORM && !PER_HEAD) load_weight<HALF>(it, 0, pl, D, w);
  const float sign = a.inverse ? -1.f : 1.f;
  const int tiles = (a.N + GROUPS - 1) / GROUPS, batches = (u.nh + kBatch - 1) / kBatch;

  auto load = [&](Eight<T, HALF> (&v)[kBatch], int slot, int tok, int h) {
    const T* row = x + static_cast<long long>(a.inverse ? slot : tok) * it.xs[2] + h * x_head;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      v[i].zero();
      if (tok >= 0 && h + i < u.nh) v[i].load(row + i * x_head, pl.gap);
    }
  };
  int slot = blockIdx.x * GROUPS + group, tok = token_of(a, slot, lane == 0);
  Eight<T, HALF> cur[kBatch], nxt[kBatch];
  load(cur, slot, tok, 0);
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int next_slot = slot + gridDim.x * GROUPS;
    const int next_tok = tile + gridDim.x < tiles ? token_of(a, next_slot, lane == 0) : -1;
    if (ROTATE) turn.look(a.pos, lane, max(tok, 0), sign);
    T* out = y + static_cast<long long>(a.inverse ? tok : slot) * it.ys[2];
    for (int b = 0; b < batches; ++b) {
      const bool last = b + 1 == batches;
      load(nxt, last ? next_slot : slot, last ? next_tok : tok, last ? 0 : (b + 1) * kBatch);
      // the batch's row sums first, so that their shuffles overlap
      float r[kBatch];
      if (NORM) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          float f[8];
          cur[i].get(f);
          r[i] = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i] = fmaf(f[j], f[j], r[i]);
        }
        row_sums<LANES>(r);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) r[i] = rsqrtf(r[i] * (1.f / D) + a.eps);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = b * kBatch + i;
        T* dst = out + h * y_head;
        if (NORM || ROTATE) {
          float f[8];
          cur[i].get(f);
          if (NORM) {
            if (PER_HEAD) load_weight<HALF>(it, u.h0 + min(h, u.nh - 1), pl, D, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * r[i] * w[j];
          }
          if (ROTATE) turn.apply(f);
          if (tok >= 0 && h < u.nh) Eight<T, HALF>::store(dst, pl.gap, f);
        } else if (tok >= 0 && h < u.nh) {
          cur[i].copy_to(dst, pl.gap);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) cur[i] = nxt[i];
    }
    slot = next_slot;
    tok = next_tok;
  }
}

// grid (blocks along the tokens, units): a block takes kThreads / LANES tokens
// at a time, token tiles blockIdx.x, blockIdx.x + gridDim.x, ... of one unit.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ RopeArgs a) {
  const Unit u = unit_of(a, blockIdx.y);
  const RopeItem& it = a.it[u.item];
  if (it.weight && it.weight_heads > 1) {
    if (it.rotate) rope_rows<T, D, HALF, true, true, true>(a, it, u);
    else rope_rows<T, D, HALF, true, false, true>(a, it, u);
  } else if (it.weight) {
    if (it.rotate) rope_rows<T, D, HALF, true, true, false>(a, it, u);
    else rope_rows<T, D, HALF, true, false, false>(a, it, u);
  } else {
    if (it.rotate) rope_rows<T, D, HALF, false, true, false>(a, it, u);
    else rope_rows<T, D, HALF, false, false, false>(a, it, u);
  }
}

// A lane's elements of a row from global to its slots of shared memory (16
// bytes each, kThreads slots apart), zeros where !on.
__device__ __forceinline__ void async_16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <typename T>
__device__ __forceinline__ void async_row(uint32_t dst, const T* src, int gap, bool on) {
  async_16(dst, src, on);
  if (sizeof(T) == 4) async_16(dst + kThreads * 16, src + gap, on);
}

// Same tiling; x is read in source order, dy in block order, dx written in
// source order.  A thread's rows come through its own slots of shared memory,
// kStages - 1 batches ahead (another's slots are read within a half-split row
// only).  For a layer's q, k, v (21 x 30 x 52 tokens, 12 heads of 128, bf16), for
// which memory needs 123 us, the kernel takes 133 us and the call 142 to 153 us.
// (Side by side, each from one run: 139 us, 151 where the kernel asks row by row
// what a unit needs, 168 with the next batch in registers; half-split rows 143 us,
// 172 with pairs that are exchanged between lanes, 171 with copies of 8 bytes.)
// fp32 rows need 246 us: half-split 257 us, interleaved 394, where each of a lane's
// two 16-byte copies takes every second half of a 32-byte sector (no counters).
// A thread adds its columns' du n over all its rows; the block adds its groups'
// sums in a fixed order and writes one partial row, so the weight gradient does
// not depend on the order in which blocks run.  With a weight row for each head
// a unit is one batch of heads, with a sum each: 216 us (one head: 305), half-split
// 236, fp32 364 and interleaved 690; a token's place and angles are looked up
// again for every batch.
constexpr int kStages = 4;
constexpr int kStageVecs = 4;                    // 16-byte slots of a thread in a stage: 64 bytes of x and dy
// heads of a token that a thread works on together
template <typename T>
__host__ __device__ constexpr int batch_heads() { return kStageVecs * 16 / (2 * 8 * sizeof(T)); }
constexpr int kBackwardSmem = kStages * kStageVecs * kThreads * 16 + kThreads * 8 * 4;

template <typename T, int D, bool HALF, bool NORM, bool ROTATE, bool PER_HEAD>
__device__ __forceinline__ void backward_rows(uint8_t* smem, const RopeArgs& a, const RopeItem& it, const Unit& u) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  constexpr int VECS = sizeof(T) / 2;            // slots of a row's eight elements
  constexpr int kBatch = batch_heads<T>(), ROWS = PER_HEAD ? kBatch : 1;   // weight rows of the unit
  uint4* slots = reinterpret_cast<uint4*>(smem) + threadIdx.x;       // [stage][vec][thread]
  float* sum = reinterpret_cast<float*>(smem + kStages * kStageVecs * kThreads * 16);   // [GROUPS][D]
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Place pl(HALF, a.pos, lane);
  // Half-split bf16 rows are fetched 16 bytes a lane like the others and each
  // lane takes its two times four elements from the row's slots: 8-byte copies
  // of its own would be twice as many.
  constexpr bool SHARED = HALF && sizeof(T) == 2;
  const int from = SHARED ? lane * 8 : pl.at;
  // without a norm x is not read (it may be NULL)
  const T* x = NORM ? static_cast<const T*>(it.x) + u.b * it.xs[0] + u.h0 * it.xs[1] + from : nullptr;
  const T* dy = static_cast<const T*>(it.dy) + u.b * it.ds[0] + u.h0 * it.ds[1] + from;
  T* dx = static_cast<T*>(it.y) + u.b * it.ys[0] + u.h0 * it.ys[1] + pl.at;
  Turn<HALF> turn;
  float w[ROWS][8], acc[ROWS][8] = {};
  if (NORM) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) load_weight<HALF>(it, PER_HEAD ? u.h0 + min(i, u.nh - 1) : 0, pl, D, w[i]);
  }
  const int tiles = (a.N + GROUPS - 1) / GROUPS, batches = PER_HEAD ? 1 : (u.nh + kBatch - 1) / kBatch;
  const int stride = gridDim.x;

  // the batch to be fetched next: its tile, slot, token and head
  int f_tile = blockIdx.x, f_slot = f_tile * GROUPS + group, f_tok = token_of(a, f_slot, lane == 0), f_h = 0, f_stage = 0;
  int f_next = f_tile + stride < tiles ? token_of(a, f_slot + stride * GROUPS, false) : -1;
  auto fetch = [&] {
    const uint32_t dst = smem_u32(slots + f_stage * kStageVecs * kThreads);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const bool on = f_tok >= 0 && f_h + i < u.nh;
      const T* rd = dy + (on ? f_slot * it.ds[2] + (f_h + i) * it.ds[1] : 0);
      const T* rx = NORM ? x + (on ? f_tok * it.xs[2] + (f_h + i) * it.xs[1] : 0) : rd;
      async_row(dst + i * 2 * VECS * kThreads * 16, rd, pl.gap, on);
      if (NORM) async_row(dst + (i * 2 + 1) * VECS * kThreads * 16, rx, pl.gap, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++f_stage == kStages) f_stage = 0;
    f_h += kBatch;
    if (f_h >= u.nh) {
      f_h = 0;
      f_tile += stride;
      f_slot += stride * GROUPS;
      f_tok = f_next;
      f_next = f_tile + stride < tiles ? token_of(a, f_slot + stride * GROUPS, false) : -1;
    }
  };
  auto take = [&](Eight<T, HALF>& v, int stage, int vec) {
    uint4* to = reinterpret_cast<uint4*>(&v);
    const uint4* own = slots + (stage * kStageVecs + vec) * kThreads;
    if (SHARED) {
      const T* row = reinterpret_cast<const T*>(own - lane) + pl.at;
      const uint2 lo = *reinterpret_cast<const uint2*>(row), hi = *reinterpret_cast<const uint2*>(row + pl.gap);
      to[0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
#pragma unroll
      for (int i = 0; i < VECS; ++i) to[i] = own[i * kThreads];
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  int slot = blockIdx.x * GROUPS + group, tok = token_of(a, slot, false), stage = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += stride) {
    const int next_tok = tile + stride < tiles ? token_of(a, slot + stride * GROUPS, lane == 0) : -1;
    if (ROTATE) turn.look(a.pos, lane, max(tok, 0), -1.f);
    T* out = dx + static_cast<long long>(tok) * it.ys[2];
    for (int b = 0; b < batches; ++b) {
      if (SHARED) __syncwarp();                                // the slots refilled next are read by the row's lanes
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      if (SHARED) __syncwarp();
      Eight<T, HALF> cd[kBatch];
      float g[kBatch][8], sums[2 * kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        take(cd[i], stage, i * 2 * VECS);
        cd[i].get(g[i]);
        if (ROTATE) turn.apply(g[i]);
      }
      if (NORM) {
        // sum x^2 and sum dn x of the batch together: mean(dn n) = r mean(dn x)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          Eight<T, HALF> cx;
          float n[8];
          take(cx, stage, i * 2 * VECS + VECS);
          cx.get(n);
          sums[2 * i] = sums[2 * i + 1] = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sums[2 * i] = fmaf(n[j], n[j], sums[2 * i]);
            sums[2 * i + 1] = fmaf(g[i][j] * w[i % ROWS][j], n[j], sums[2 * i + 1]);
          }
        }
        row_sums<LANES>(sums);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = b * kBatch + i;
        if (NORM) {
          Eight<T, HALF> cx;
          float n[8];
          take(cx, stage, i * 2 * VECS + VECS);
          cx.get(n);
          // a row that is not there adds nothing, with eps = 0 (1 / 0) too
          const float r = tok >= 0 && h < u.nh ? rsqrtf(sums[2 * i] * (1.f / D) + a.eps) : 0.f;
          const float k = sums[2 * i + 1] * (1.f / D) * r * r;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            acc[i % ROWS][j] = fmaf(g[i][j], n[j] * r, acc[i % ROWS][j]);   // rows that are not there are 0
            g[i][j] = r * fmaf(-n[j], k, g[i][j] * w[i % ROWS][j]);
          }
        }
        if (tok >= 0 && h < u.nh) {
          if (NORM || ROTATE) Eight<T, HALF>::store(out + h * it.ys[1], pl.gap, g[i]);
          else cd[i].copy_to(out + h * it.ys[1], pl.gap);
        }
      }
      if (++stage == kStages) stage = 0;
    }
    slot += stride * GROUPS;
    tok = next_tok;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  grid_launch_dependents();
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (i) __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[group * D + pl.at + (j < 4 ? j : pl.gap + j - 4)] = acc[i][j];
      __syncthreads();
      for (int e = threadIdx.x; e < D; e += kThreads) {
        float t = 0.f;
        for (int g = 0; g < GROUPS; ++g) t += sum[g * D + e];
        a.partial[(static_cast<long long>(i * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * D + e] = t;
      }
    }
  }
}

template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_backward_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Unit u = unit_of(a, blockIdx.y);
  const RopeItem& it = a.it[u.item];
  if (it.weight && it.weight_heads > 1) {
    if (it.rotate) backward_rows<T, D, HALF, true, true, true>(smem, a, it, u);
    else backward_rows<T, D, HALF, true, false, true>(smem, a, it, u);
  } else if (it.weight) {
    if (it.rotate) backward_rows<T, D, HALF, true, true, false>(smem, a, it, u);
    else backward_rows<T, D, HALF, true, false, false>(smem, a, it, u);
  } else {
    if (it.rotate) backward_rows<T, D, HALF, false, true, false>(smem, a, it, u);
    else backward_rows<T, D, HALF, false, false, false>(smem, a, it, u);
  }
}

// dweight[row][e] = sum of the partial rows of the units that share the weight
// row, in 64 bits, in a fixed order.  grid (d / 32, weight rows of all items), 32 x 32 threads.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const __grid_constant__ RopeArgs a, int gx, int B) {
  __shared__ double sum[32][33];
  const int e = blockIdx.x * 32 + threadIdx.x;
  int item = 0, row = blockIdx.y;
  while (item < a.count - 1 && row >= (a.it[item].weight ? a.it[item].weight_heads : 0)) {
    row -= a.it[item].weight ? a.it[item].weight_heads : 0;
    ++item;
  }
  const RopeItem& it = a.it[item];
  const int first = item ? a.chunk_end[item - 1] : 0;
  const bool shared = it.weight_heads == 1;
  // the units' partial rows lie together: all of the item's, or (a weight row
  // for each head: plane row % heads) one run a batch element
  const long long run = shared ? static_cast<long long>(a.chunk_end[item] - first) * gx : gx;
  const int heads = a.heads[item], chunks = (it.H + heads - 1) / heads;
  double t = 0.0;
  grid_wait();
  for (int b = 0; b < (shared ? 1 : B); ++b) {
    const long long at = shared ? first : static_cast<long long>(row % heads) * a.chunk_end[2] + first + b * chunks + row / heads;
    const float* p = a.partial + at * gx * a.d + e;
#pragma unroll 8
    for (long long i = threadIdx.y; i < run; i += 32) t += p[i * a.d];
  }
  sum[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0) {
    for (int i = 1; i < 32; ++i) t += sum[i][threadIdx.x];
    it.dweight[static_cast<long long>(row) * a.d + e] = static_cast<float>(t);
  }
}

// Angles in 64 bits (far positions: an fp32 product would be off by position * 2^-24).
__global__ void rope_table_kernel(RopePos p, double theta, double st, double sh, double sw, float2* table) {
  const int ht = p.dt / 2, hh = p.dh / 2, hw = p.dw / 2;
  const long long nt = static_cast<long long>(p.T) * ht, nh = static_cast<long long>(p.Hg) * hh;
  const long long n = nt + nh + static_cast<long long>(p.Wg) * hw;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int axis = i < nt ? 0 : i < nt + nh ? 1 : 2;
    const long long r = axis == 0 ? i : axis == 1 ? i - nt : i - nt - nh;
    const int half = axis == 0 ? ht : axis == 1 ? hh : hw;
    const long long at = r / half;
    const double pos = static_cast<double>(at) + (axis == 0 ? st : axis == 1 ? sh : sw);
    double s, c;
    sincos(pos * pow(theta, -static_cast<double>(r - at * half) / half), &s, &c);
    table[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
  }
}

int token_tiles(int N, int d) { return (N + kThreads / (d / 8) - 1) / (kThreads / (d / 8)); }

int unit_rows(int dtype) { return dtype == LBSA_BF16 ? batch_heads<__nv_bfloat16>() : batch_heads<float>(); }

// Units: (batch, up to `heads` heads) of each item; with a weight row for each
// head up to `rows` of them.  With few tokens the heads
// are spread over more units, down to one head, until every SM has a block: a
// single token's 24 heads of 128 take 4.4 us so, 5.4 us as two units.  More
// blocks than that cost more than they give: 924 tokens with 10 heads of 128,
// half-split, take 6.7 us in 232 blocks and 11.4 us in 580.
int plan_units(RopeArgs& a, const RopeItem* items, int count, int B, int N, int d, int rows) {
  a.count = count;
  int total = 0;
  for (int most = kMaxHeads; most >= 1; most /= 2) {
    total = 0;
    for (int i = 0; i < 3; ++i) {
      if (i < count) {
        a.it[i] = items[i];
        const bool per_head = items[i].weight && items[i].weight_heads > 1;
        a.heads[i] = std::min(items[i].H, per_head ? std::min(rows, most) : most);
        total += B * ((items[i].H + a.heads[i] - 1) / a.heads[i]);
      } else {
        a.heads[i] = 1;
      }
      a.chunk_end[i] = total;
    }
    if (static_cast<long long>(total) * token_tiles(N, d) >= 148) break;
  }
  return total;
}

// Blocks along the tokens: about kBlocksPerSm an SM in all (three waves of the
// three that fit), so that a block walks several tiles and the backward pass
// has few partial rows; 8 against 6 for a layer's q, k, v (norm_rope, 21 x 30 x
// 52 tokens, 12 heads of 128), when they were compared: 104 and 107 us.
constexpr int kBlocksPerSm = 9;
int token_blocks(int N, int d, int units) {
  return std::max(1, std::min(token_tiles(N, d), (148 * kBlocksPerSm + units - 1) / units));
}

template <bool BWD>
cudaError_t launch(const RopeArgs& a, int dtype, dim3 grid, cudaStream_t s) {
  const int smem = BWD ? kBackwardSmem : 0;
  auto go = [&](auto kern) {
    if (BWD) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
    kern<<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
  };
#define LBSA_ROPE(T, D)                                                                          \
  (a.pos.half ? (BWD ? go(norm_rope_backward_kernel<T, D, true>) : go(rope_kernel<T, D, true>))  \
              : (BWD ? go(norm_rope_backward_kernel<T, D, false>) : go(rope_kernel<T, D, false>)))
  if (dtype == LBSA_BF16) return a.d == 128 ? LBSA_ROPE(__nv_bfloat16, 128) : LBSA_ROPE(__nv_bfloat16, 64);
  return a.d == 128 ? LBSA_ROPE(float, 128) : LBSA_ROPE(float, 64);
#undef LBSA_ROPE
}

}  // namespace

cudaError_t launch_rope(const RopeItem* items, int count, int B, int N, int d, int dtype, const RopePos& pos,
                        const int32_t* perm, float eps, int inverse, int32_t* status, cudaStream_t s) {
  RopeArgs a{};
  a.N = N;
  a.d = d;
  a.pos = pos;
  a.perm = perm;
  a.eps = eps;
  a.inverse = inverse;
  a.status = status;
  const int units = plan_units(a, items, count, B, N, d, kMaxHeads);
  return launch<false>(a, dtype, dim3(token_blocks(N, d, units), units), s);
}

size_t norm_rope_backward_workspace_bytes(const RopeItem* items, int count, int B, int N, int d, int dtype) {
  RopeArgs a{};
  const int rows = unit_rows(dtype), units = plan_units(a, items, count, B, N, d, rows);
  return static_cast<size_t>(rows) * units * token_blocks(N, d, units) * d * sizeof(float);
}

cudaError_t launch_norm_rope_backward(const RopeItem* items, int count, int B, int N, int d, int dtype,
                                      const RopePos& pos, const int32_t* perm, float eps, void* workspace,
                                      int32_t* status, cudaStream_t s) {
  RopeArgs a{};
  a.N = N;
  a.d = d;
  a.pos = pos;
  a.perm = perm;
  a.eps = eps;
  a.status = status;
  a.partial = static_cast<float*>(workspace);
  const int units = plan_units(a, items, count, B, N, d, unit_rows(dtype));
  const int gx = token_blocks(N, d, units);
  cudaError_t e = launch<true>(a, dtype, dim3(gx, units), s);
  int rows = 0;
  for (int i = 0; i < count; ++i) rows += items[i].weight ? items[i].weight_heads : 0;
  if (e != cudaSuccess || rows == 0) return e;
  return launch_dependent(weight_grad_kernel, dim3(d / 32, rows), dim3(32, 32), 0, s, a, gx, B);
}

cudaError_t launch_rope_table(const RopePos& pos, double theta, const double* start, float* table, cudaStream_t s) {
  const long long n = static_cast<long long>(pos.T) * (pos.dt / 2) + static_cast<long long>(pos.Hg) * (pos.dh / 2) +
                      static_cast<long long>(pos.Wg) * (pos.dw / 2);
  const int blocks = static_cast<int>(std::min<long long>((n + 255) / 256, 148 * 8));
  rope_table_kernel<<<blocks, 256, 0, s>>>(pos, theta, start[0], start[1], start[2], reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

}  // namespace lbsa
