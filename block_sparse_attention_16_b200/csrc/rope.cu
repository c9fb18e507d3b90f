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
// elements each, so the row sums are three or four shuffles; a thread takes
// kHeads heads of one token, so their loads are in flight together and the
// token's position, perm entry and (cos, sin) are looked up once for them.
#include "lbsa_device.cuh"

namespace lbsa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;        // heads of one token that a thread has in flight

struct RopeArgs {
  RopeItem it[3];
  int count;
  int chunk_end[3];              // running number of (batch, head chunk) units per item
  int heads[3];                  // heads of a unit (1 .. kHeads)
  int N, d;
  RopePos pos;
  const int32_t* perm;
  float eps;
  int inverse;                   // rotation by -angle, scatter
  int32_t* status;
  float* partial;                // backward: [gridDim.y][gridDim.x][d] weight gradients of a block
};

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static void store(void* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
  __device__ __forceinline__ void copy_to(void* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ static void store(void* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void copy_to(void* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

// A lane's share of the rotation: which table entries its pairs take.
// interleaved: pairs 4 l .. 4 l + 3 lie in the lane's own eight elements.
// half-split: element e of the first half pairs with e + rd / 2, which a lane
// rd / 16 further holds; both lanes look the pair's eight entries up.
template <bool HALF>
struct Turn {
  static constexpr int P = HALF ? 8 : 4;
  float c[P], s[P];
  int entry[P];       // table entry at position 0 of the pair's axis; -1: not rotated
  int step[P];        // entries from one position to the next, axis in the low two bits
  __device__ __forceinline__ void plan(const RopePos& pos, int lane, bool rotate) {
    const int ht = pos.dt >> 1, hh = pos.dh >> 1, hw = pos.dw >> 1;
    const int half = ht + hh + hw;
    const int first = HALF ? (lane * 8 < half ? lane * 8 : lane * 8 - half) : lane * 4;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int p = first + j;
      if (!rotate || p >= half) {
        entry[j] = -1;
        step[j] = 0;
      } else if (p < ht) {
        entry[j] = p;
        step[j] = ht << 2;
      } else if (p < ht + hh) {
        entry[j] = pos.T * ht + p - ht;
        step[j] = (hh << 2) | 1;
      } else {
        entry[j] = pos.T * ht + pos.Hg * hh + p - ht - hh;
        step[j] = (hw << 2) | 2;
      }
    }
  }
  // token: source (raster) index; tokens past the grid keep their place
  __device__ __forceinline__ void look(const RopePos& pos, int token, float sign) {
    const bool in = token < pos.tokens;
    const uint32_t area = static_cast<uint32_t>(pos.Hg) * pos.Wg;
    const uint32_t tt = static_cast<uint32_t>(in ? token : 0);
    const uint32_t t = tt / area, r = tt - t * area, h = r / pos.Wg, w = r - h * pos.Wg;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint32_t at = (step[j] & 3) == 0 ? t : (step[j] & 3) == 1 ? h : w;
      float2 cs = make_float2(1.f, 0.f);
      if (in && entry[j] >= 0) cs = __ldg(pos.table + entry[j] + static_cast<int>(at) * (step[j] >> 2));
      c[j] = cs.x;
      s[j] = cs.y * sign;
    }
  }
  // every lane of the warp takes part (half-split exchanges elements)
  __device__ __forceinline__ void apply(float (&f)[8], const RopePos& pos, int lane, int lanes) const {
    if (!HALF) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = f[2 * j], b = f[2 * j + 1];
        f[2 * j] = a * c[j & (P - 1)] - b * s[j & (P - 1)];
        f[2 * j + 1] = a * s[j & (P - 1)] + b * c[j & (P - 1)];
      }
    } else {
      const int hl = (pos.dt + pos.dh + pos.dw) >> 4;       // lanes of a half
      const bool lo = lane < hl, rot = lane < 2 * hl;
      const int other = rot ? (lo ? lane + hl : lane - hl) : lane;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float o = __shfl_sync(0xffffffffu, f[j], other, lanes);
        const float cj = c[j & (P - 1)], sj = s[j & (P - 1)];
        // lo: a c - b s;  hi: a s + b c with a the other lane's element
        f[j] = rot ? (lo ? f[j] * cj - o * sj : o * sj + f[j] * cj) : f[j];
      }
    }
  }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void load_weight(const RopeItem& it, int head, int lane, int d, float (&w)[8]) {
  const long long at = static_cast<long long>(it.weight_heads > 1 ? head : 0) * d + lane * 8;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j] = it.weight_dtype == LBSA_F32 ? __ldg(static_cast<const float*>(it.weight) + at + j)
                                       : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(it.weight) + at + j));
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

// grid (token tiles, units): a block takes kThreads / LANES tokens at a time,
// token tiles blockIdx.x, blockIdx.x + gridDim.x, ... of one unit.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Unit u = unit_of(a, blockIdx.y);
  const RopeItem& it = a.it[u.item];
  const T* x = static_cast<const T*>(it.x) + u.b * it.xs[0] + u.h0 * it.xs[1] + lane * 8;
  T* y = static_cast<T*>(it.y) + u.b * it.ys[0] + u.h0 * it.ys[1] + lane * 8;
  Turn<HALF> turn;
  turn.plan(a.pos, lane, it.rotate);
  const float sign = a.inverse ? -1.f : 1.f;
  const int tiles = (a.N + GROUPS - 1) / GROUPS;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int slot = tile * GROUPS + group;
    int tok = slot < a.N ? (a.perm ? __ldg(a.perm + slot) : slot) : -1;
    if (tok >= a.N || (tok < 0 && slot < a.N)) {
      if (lane == 0) raise_status(a.status, LBSA_ERR_BAD_INDEX);
      tok = -1;
    }
    const bool ok = tok >= 0;
    const long long from = a.inverse ? slot : tok, to = a.inverse ? tok : slot;
    Eight<T> v[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (ok && i < u.nh) v[i].load(x + from * it.xs[2] + i * it.xs[1]);
      else v[i].zero();
    }
    if (it.rotate) turn.look(a.pos, max(tok, 0), sign);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (i >= u.nh) break;                                    // the same for the whole block
      float f[8];
      v[i].get(f);
      if (it.weight) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
        const float r = rsqrtf(row_sum<LANES>(ss) * (1.f / D) + a.eps);
        float w[8];
        load_weight(it, u.h0 + i, lane, D, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * r * w[j];
      }
      if (it.rotate) turn.apply(f, a.pos, lane, LANES);
      if (ok) {
        T* dst = y + to * it.ys[2] + i * it.ys[1];
        if (it.weight || it.rotate) Eight<T>::store(dst, f);
        else v[i].copy_to(dst);
      }
    }
  }
}

// Same tiling; x is read in source order, dy in block order, dx written in
// source order.  A thread adds its columns' du n over all its rows; the block
// adds its groups' sums in a fixed order and writes one partial row, so the
// weight gradient does not depend on the order in which blocks run.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads) norm_rope_backward_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  __shared__ float sum[GROUPS][D];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Unit u = unit_of(a, blockIdx.y);
  const RopeItem& it = a.it[u.item];
  const T* x = static_cast<const T*>(it.x) + u.b * it.xs[0] + u.h0 * it.xs[1] + lane * 8;
  const T* dy = static_cast<const T*>(it.dy) + u.b * it.ds[0] + u.h0 * it.ds[1] + lane * 8;
  T* dx = static_cast<T*>(it.y) + u.b * it.ys[0] + u.h0 * it.ys[1] + lane * 8;
  Turn<HALF> turn;
  turn.plan(a.pos, lane, it.rotate);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int tiles = (a.N + GROUPS - 1) / GROUPS;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int slot = tile * GROUPS + group;
    int tok = slot < a.N ? (a.perm ? __ldg(a.perm + slot) : slot) : -1;
    if (tok >= a.N || (tok < 0 && slot < a.N)) {
      if (lane == 0) raise_status(a.status, LBSA_ERR_BAD_INDEX);
      tok = -1;
    }
    const bool ok = tok >= 0;
    Eight<T> vx[kHeads], vd[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (ok && i < u.nh) vd[i].load(dy + static_cast<long long>(slot) * it.ds[2] + i * it.ds[1]);
      else vd[i].zero();
      if (ok && i < u.nh && it.weight) vx[i].load(x + static_cast<long long>(tok) * it.xs[2] + i * it.xs[1]);
      else vx[i].zero();
    }
    if (it.rotate) turn.look(a.pos, max(tok, 0), -1.f);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (i >= u.nh) break;
      float g[8];
      vd[i].get(g);
      if (it.rotate) turn.apply(g, a.pos, lane, LANES);
      if (it.weight) {
        float n[8], w[8], ss = 0.f;
        vx[i].get(n);
        load_weight(it, u.h0 + i, lane, D, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(n[j], n[j], ss);
        const float r = rsqrtf(row_sum<LANES>(ss) * (1.f / D) + a.eps);
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n[j] *= r;
          acc[j] = fmaf(g[j], n[j], acc[j]);
          g[j] *= w[j];
          dot = fmaf(g[j], n[j], dot);
        }
        dot = row_sum<LANES>(dot) * (1.f / D);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = r * (g[j] - n[j] * dot);
      }
      if (ok) {
        T* dst = dx + static_cast<long long>(tok) * it.ys[2] + i * it.ys[1];
        if (it.weight || it.rotate) Eight<T>::store(dst, g);
        else vd[i].copy_to(dst);
      }
    }
  }
  if (!it.weight) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[group][lane * 8 + j] = acc[j];
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kThreads) {
    float t = 0.f;
    for (int g = 0; g < GROUPS; ++g) t += sum[g][e];
    a.partial[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * D + e] = t;
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
  const int per = (it.H + a.heads[item] - 1) / a.heads[item];
  const bool shared = it.weight_heads == 1;
  const long long n = static_cast<long long>(shared ? a.chunk_end[item] - first : B) * gx;   // partial rows to add
  double t = 0.0;
  for (long long i = threadIdx.y; i < n; i += 32) {
    const long long unit = shared ? first + i / gx : first + (i / gx) * per + row;           // one head a unit there
    t += a.partial[(unit * gx + i % gx) * a.d + e];
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

// Units: (batch, up to `heads` heads) of each item.  Few tokens: one head a
// unit, so that a single token's heads run side by side.
int plan_units(RopeArgs& a, const RopeItem* items, int count, int B, bool backward) {
  int total = 0;
  a.count = count;
  for (int i = 0; i < 3; ++i) {
    if (i < count) {
      a.it[i] = items[i];
      const bool own_rows = backward && items[i].weight && items[i].weight_heads > 1;
      a.heads[i] = own_rows || static_cast<long long>(a.N) * B * items[i].H < 148ll * 64 ? 1 : std::min(items[i].H, kHeads);
      total += B * ((items[i].H + a.heads[i] - 1) / a.heads[i]);
    } else {
      a.heads[i] = 1;
    }
    a.chunk_end[i] = total;
  }
  return total;
}

template <bool BWD>
cudaError_t launch(const RopeArgs& a, int dtype, dim3 grid, cudaStream_t s) {
  auto go = [&](auto kern) {
    kern<<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  };
#define LBSA_ROPE(T, D)                                                                          \
  (a.pos.half ? (BWD ? go(norm_rope_backward_kernel<T, D, true>) : go(rope_kernel<T, D, true>))  \
              : (BWD ? go(norm_rope_backward_kernel<T, D, false>) : go(rope_kernel<T, D, false>)))
  if (dtype == LBSA_BF16) return a.d == 128 ? LBSA_ROPE(__nv_bfloat16, 128) : LBSA_ROPE(__nv_bfloat16, 64);
  return a.d == 128 ? LBSA_ROPE(float, 128) : LBSA_ROPE(float, 64);
#undef LBSA_ROPE
}

int token_tiles(int N, int d) { return (N + kThreads / (d / 8) - 1) / (kThreads / (d / 8)); }

// Blocks along the tokens in the backward pass: about eight blocks an SM in
// all, so that the partial rows stay few.
int backward_blocks(int N, int d, int units) {
  return std::max(1, std::min(token_tiles(N, d), (148 * 8 + units - 1) / units));
}

}  // namespace

int rope_units(const RopeItem* items, int count, int B, int N, bool backward) {
  RopeArgs a{};
  a.N = N;
  return plan_units(a, items, count, B, backward);
}

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
  const int units = plan_units(a, items, count, B, false);
  return launch<false>(a, dtype, dim3(token_tiles(N, d), units), s);
}

size_t norm_rope_backward_workspace_bytes(const RopeItem* items, int count, int B, int N, int d) {
  const int units = rope_units(items, count, B, N, true);
  return static_cast<size_t>(units) * backward_blocks(N, d, units) * d * sizeof(float);
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
  const int units = plan_units(a, items, count, B, true);
  const int gx = backward_blocks(N, d, units);
  cudaError_t e = launch<true>(a, dtype, dim3(gx, units), s);
  int rows = 0;
  for (int i = 0; i < count; ++i) rows += items[i].weight ? items[i].weight_heads : 0;
  if (e != cudaSuccess || rows == 0) return e;
  weight_grad_kernel<<<dim3(d / 32, rows), dim3(32, 32), 0, s>>>(a, gx, B);
  return cudaGetLastError();
}

cudaError_t launch_rope_table(const RopePos& pos, double theta, const double* start, float* table, cudaStream_t s) {
  const long long n = static_cast<long long>(pos.T) * (pos.dt / 2) + static_cast<long long>(pos.Hg) * (pos.dh / 2) +
                      static_cast<long long>(pos.Wg) * (pos.dw / 2);
  const int blocks = static_cast<int>(std::min<long long>((n + 255) / 256, 148 * 8));
  rope_table_kernel<<<blocks, 256, 0, s>>>(pos, theta, start[0], start[1], start[2], reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

}  // namespace lbsa
