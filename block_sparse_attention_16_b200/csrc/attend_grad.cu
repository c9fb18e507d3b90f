// Gradients of block-sparse attention: the per-call tables both kernels read,
// and the fp32 kernel on CUDA cores.
//
// Mathematics.  For a query row r with kept keys K_r and the forward's lse_r:
//   P_rc = exp(q_r . k_c / sqrt(d) - lse_r) on kept pairs, else 0
//   D_r  = sum_e dout_re out_re             (= sum_c P_rc dP_rc)
//   dP_rc = dout_r . v_c,   dS_rc = P_rc (dP_rc - D_r)
//   dv_c = sum_r P_rc dout_r,  dk_c = sum_r dS_rc q_r / sqrt(d),
//   dq_r = sum_c dS_rc k_c / sqrt(d)
// dv and dk sum over the query blocks that keep a key block, dq over the key
// blocks that a query block keeps.  Each of the two sums is walked by the CTAs
// that own its rows, which compute S and dP twice over but need no atomics, no
// fp32 gradient buffer in memory and no order between CTAs: the same inputs
// give the same bits.
//
// Tables (scratch of the call): -lse in log2 units and -D, padded to whole
// 128-row tiles (a row that keeps nothing, or does not exist, gets -inf and 0:
// its P is 0, or 2^-125 where the bf16 kernel takes the exponential on the FMA
// pipe, for which masks and the zeros read past the last row leave nothing), and
// the kept pairs as bits in both directions; the per-token sets go to [key
// block][query block].
#include "lbsa_train_device.cuh"

namespace lbsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPrepThreads = 256;

__device__ __forceinline__ long long offset(const GradStride& s, int b, int h, int n) {
  return b * s.b + h * s.h + n * s.n;
}

// sum of the products of 16 bytes of two rows
__device__ __forceinline__ float dot16(uint4 x, uint4 y, float) {
  float s = __uint_as_float(x.x) * __uint_as_float(y.x);
  s = fmaf(__uint_as_float(x.y), __uint_as_float(y.y), s);
  s = fmaf(__uint_as_float(x.z), __uint_as_float(y.z), s);
  return fmaf(__uint_as_float(x.w), __uint_as_float(y.w), s);
}
__device__ __forceinline__ float dot16(uint4 x, uint4 y, __nv_bfloat16) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
    s = fmaf(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), s);
  }
  return s;
}

constexpr int kRowsPerBlock = 64;        // query rows of a block of the second kind; divides 128

// Blocks [0, index_blocks): 32 query blocks of one (batch, head) each, whose
// lists become bit rows and, transposed in shared memory, one word of every
// key block's bits.  The others: 64 rows each, D = dout . out and, bf16, the
// mean of the key rows if they have much in common: 0 unless |mean|^2 is more
// than a quarter of what they vary by, so that a few keys far from the others
// (fewer than a fifth of the 64), or infinite ones, are not taken for all of
// them.  Bound by reading out, dout and k once.
template <typename T, int D>
__global__ void __launch_bounds__(kPrepThreads)
attend_grad_prep_kernel(const T* __restrict__ out, const T* __restrict__ dout, const float* __restrict__ lse,
                        AttendGradArgs a, int index_blocks) {
  extern __shared__ uint32_t bm[];                     // [32][W], or the threads' key sums
  grid_launch_dependents();
  const int W = (a.nB + 31) >> 5;
  if (blockIdx.x < index_blocks) {
    const int w = blockIdx.x % W;
    const long long bh = blockIdx.x / W;
    for (int i = threadIdx.x; i < 32 * W; i += kPrepThreads) bm[i] = 0u;
    __syncthreads();
    // four rows a warp, their lists' loads in flight together
    constexpr int ROWS = 32 / (kPrepThreads / 32);
    const int lane = threadIdx.x & 31, i0 = w * 32 + (threadIdx.x >> 5) * ROWS;
    const long long row = bh * a.nB + i0;
    int cnt[ROWS], most = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      cnt[r] = i0 + r < a.nB ? a.counts[row + r] : 0;
      most = max(most, cnt[r]);
    }
    for (int t = lane; t < most; t += 32) {
      int j[ROWS];
      uint64_t set[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        j[r] = t < cnt[r] ? a.cols[(row + r) * a.nB + t] : 0;
        set[r] = a.masks && t < cnt[r] ? a.masks[(row + r) * a.nB + t] : 0ull;
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (t >= cnt[r]) continue;
        if (j[r] < 0 || j[r] >= a.nB) {
          raise_status(a.status, LBSA_ERR_BAD_INDEX);
          continue;
        }
        const uint32_t bit = 1u << (j[r] & 31);
        if (atomicOr(&bm[(i0 + r - w * 32) * W + (j[r] >> 5)], bit) & bit) raise_status(a.status, LBSA_ERR_BAD_INDEX);   // named twice
        if (a.masks) a.masks_t[(bh * a.nB + j[r]) * a.nB + i0 + r] = set[r];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * W; i += kPrepThreads) {
      const int r = i / W, q = w * 32 + r;
      if (q < a.nB) a.bits[(bh * a.nB + q) * W + i - r * W] = bm[i];
    }
    for (int j = threadIdx.x; j < a.nB; j += kPrepThreads) {
      uint32_t v = 0u;
#pragma unroll
      for (int r = 0; r < 32; ++r) v |= ((bm[r * W + (j >> 5)] >> (j & 31)) & 1u) << r;
      a.bits_t[(bh * a.nB + j) * W + w] = v;
    }
    return;
  }
  // a row is held by LANES lanes, 16 bytes each
  constexpr int LANES = D * sizeof(T) / 16, GROUPS = kPrepThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const long long row0 = static_cast<long long>(blockIdx.x - index_blocks) * kRowsPerBlock;   // of one (batch, head)
  const long long bh = row0 / a.Npad;
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh - static_cast<long long>(b) * a.H);
#pragma unroll
  for (int i = 0; i < kRowsPerBlock / GROUPS; ++i) {
    const long long row = row0 + i * GROUPS + threadIdx.x / LANES;
    const int n = static_cast<int>(row - bh * a.Npad);
    float sum = 0.f, l = -INFINITY;
    if (n < a.N_valid) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(out + offset(a.st[kOut], b, h, n)) + lane);
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(dout + offset(a.st[kDout], b, h, n)) + lane);
      sum = dot16(x, y, T());
      l = __ldg(lse + bh * a.N_valid + n);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const bool none = l == -INFINITY;
      a.neg_lse2[row] = none ? -INFINITY : -l * kLog2e;
      a.neg_delta[row] = none ? 0.f : -sum;
    }
  }
  if constexpr (sizeof(T) == 2) {
    float* part = reinterpret_cast<float*>(bm);        // [GROUPS][D]
    __shared__ float squares[kPrepThreads / 32], mean_squares[D / 32];
    float s[8] = {}, sq = 0.f;
#pragma unroll
    for (int i = 0; i < kRowsPerBlock / GROUPS; ++i) {
      const int n = static_cast<int>(row0 + i * GROUPS + threadIdx.x / LANES - bh * a.Npad);
      if (n >= a.N_valid) continue;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + offset(a.st[kK], b, h, n)) + lane);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xFFFF0000u);
        s[2 * e] += lo;
        s[2 * e + 1] += hi;
        sq = fmaf(lo, lo, fmaf(hi, hi, sq));
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[threadIdx.x / LANES * D + lane * 8 + e] = s[e];
    auto warp_sum = [](float v) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    sq = warp_sum(sq);
    if ((threadIdx.x & 31) == 0) squares[threadIdx.x >> 5] = sq;
    __syncthreads();
    constexpr float R = 1.f / kRowsPerBlock;           // a ragged piece's mean is not used
    float mean = 0.f;
    if (threadIdx.x < D) {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) mean += part[g * D + threadIdx.x];
      mean *= R;
      const float m2 = warp_sum(mean * mean);
      if ((threadIdx.x & 31) == 0) mean_squares[threadIdx.x >> 5] = m2;
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float m2 = 0.f, all = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) m2 += mean_squares[i];
#pragma unroll
      for (int i = 0; i < kPrepThreads / 32; ++i) all += squares[i];
      // false where a sum is not finite, too
      a.k_means[row0 / kRowsPerBlock * D + threadIdx.x] = 4.f * m2 > all * R - m2 ? mean : 0.f;
    }
  }
}

// ------------------------------------------------------------------ CUDA cores
// A CTA owns R rows (keys, or queries) and walks the 64-row pieces of the
// other side that its block is kept with.  Two groups of 128 threads: the first
// computes S and P, the second dP and dS; then the first adds to dv, the second
// to dk (or, for dq, each over half of the piece's rows).  A group's threads
// stand R / 8 x 16 x 64 / R: thread (ty, tx, kz) takes rows ty + R / 8 i and
// columns tx + 16 j over its share of the elements (the 64 / R threads of a
// share sum by shuffles).
// No pipe is full: 8 x 4 results take 12 shared-memory vectors for 128 FMAs, where
// FMA issue would cover 8, and 8 warps an SM leave gaps: with 24 heads of 128,
// 2,600 tokens, half of the blocks, FMA 57 %, shared memory 53 %, issue 66 %, and
// 3.9 ms, 38 TFLOP/s of the seven products, half of what the FMA pipes can do.
// (With one group of 256 threads, 4 x 4 results took 8 vectors for 64 FMAs: 4 such
// heads 0.89 ms against 0.82.)
// R = 64 wherever that fills the SMs; with fewer rows R = 32 or 16 spreads them
// over more CTAs.  A call with R = 64 / 32 / 16: 41 / 31 / 27 us for 256 tokens,
// 2 heads of 64 (16 CTAs with R = 64), 200 / 151 / 191 us for 1,000 tokens,
// 3 heads of 128 (96), 277 / 333 / 518 us for 1,500 tokens, 8 heads of 64 (384).
constexpr int kPitch = 68;        // floats a row of P and dS: 16-byte rows, no bank conflicts

// Rows r0 .. of a tensor into shared memory, zeros past N; cp.async, not waited for.
template <int D>
__device__ __forceinline__ void load_rows(float* s, const float* g, long long stride, int r0, int rows, int N) {
  for (int i = threadIdx.x; i < rows * (D / 4); i += 256) {
    const int r = i / (D / 4), e = (i - r * (D / 4)) * 4;
    const bool in = r0 + r < N;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(s + r * (D + 4) + e)),
                 "l"(g + (in ? r0 + r : 0) * stride + e), "r"(in ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void loads_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void loads_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The 64-row pieces that a block is kept with, ascending.
struct Pieces {
  const uint32_t* list;
  int W, N, shift, w, sub;
  uint32_t word;
  int other, c0;                // the piece's block and first row
  __device__ __forceinline__ bool next() {
    if (sub > 0 && sub <= shift && (other << shift) * 64 + sub * 64 < N) {      // the block's other half
      c0 = (other << shift) * 64 + sub * 64;
      ++sub;
      return true;
    }
    while (word == 0u) {
      if (++w >= W) return false;
      word = list[w];
    }
    other = w * 32 + __ffs(word) - 1;
    word &= word - 1u;
    c0 = (other << shift) * 64;
    sub = 1;
    return true;
  }
};

template <int KS>
__device__ __forceinline__ float sum_shares(float v) {
#pragma unroll
  for (int o = 1; o < KS; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// acc[i][j] = row ty + R / 8 i of x  .  row tx + 16 j of y
template <int D, int R>
__device__ __forceinline__ void dots(float (&acc)[8][4], const float* x, const float* y, int ty, int tx, int kz) {
  constexpr int KS = 64 / R;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
  for (int e = 4 * kz; e < D; e += 4 * KS) {
    float4 yr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) yr[j] = *reinterpret_cast<const float4*>(y + (tx + 16 * j) * (D + 4) + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 xr = *reinterpret_cast<const float4*>(x + (ty + R / 8 * i) * (D + 4) + e);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(xr.x, yr[j].x, fmaf(xr.y, yr[j].y, fmaf(xr.z, yr[j].z, fmaf(xr.w, yr[j].w, acc[i][j]))));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = sum_shares<KS>(acc[i][j]);
}

// acc[i][.] += sum of w[ty + R / 8 i][c] y[c][columns of tx] over the thread's share of c0 <= c < c1
template <int D, int R>
__device__ __forceinline__ void weighted(float (&acc)[8][D / 16], const float* w, const float* y, int c0, int c1, int ty,
                                         int tx, int kz) {
#pragma unroll 1
  for (int c = c0 + 4 * kz; c < c1; c += 4 * (64 / R)) {
    float4 wr[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wr[i] = *reinterpret_cast<const float4*>(w + (ty + R / 8 * i) * kPitch + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        const float4 v = *reinterpret_cast<const float4*>(y + (c + k) * (D + 4) + g * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = k == 0 ? wr[i].x : k == 1 ? wr[i].y : k == 2 ? wr[i].z : wr[i].w;
          acc[i][g * 4 + 0] = fmaf(p, v.x, acc[i][g * 4 + 0]);
          acc[i][g * 4 + 1] = fmaf(p, v.y, acc[i][g * 4 + 1]);
          acc[i][g * 4 + 2] = fmaf(p, v.z, acc[i][g * 4 + 2]);
          acc[i][g * 4 + 3] = fmaf(p, v.w, acc[i][g * 4 + 3]);
        }
      }
    }
  }
}

// The shares' sums, plus the other group's where `more` holds them; each of a
// share's threads stores some of the rows.
template <int D, int R>
__device__ __forceinline__ void store_rows(float* g, long long stride, int r0, int N, const float (&acc)[8][D / 16], float f,
                                           const float* more, int ty, int tx, int kz) {
  constexpr int KS = 64 / R;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = ty + R / 8 * i, r = r0 + row;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float4 v;
      v.x = sum_shares<KS>(acc[i][c * 4]);
      v.y = sum_shares<KS>(acc[i][c * 4 + 1]);
      v.z = sum_shares<KS>(acc[i][c * 4 + 2]);
      v.w = sum_shares<KS>(acc[i][c * 4 + 3]);
      if (more) {
        const float4 m = *reinterpret_cast<const float4*>(more + row * (D + 4) + c * 64 + tx * 4);
        v = make_float4(v.x + m.x, v.y + m.y, v.z + m.z, v.w + m.w);
      }
      if (r < N && i / (8 / KS) == kz)
        *reinterpret_cast<float4*>(g + r * stride + c * 64 + tx * 4) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    }
  }
}

// The next piece's rows are on their way while one is worked on, wherever two
// buffers fit (all but d = 128, R = 64).
template <int D, int R>
constexpr int kF32Buffers = D == 128 && R == 64 ? 1 : 2;
template <int D, int R>
constexpr int f32_smem() { return ((2 * R + kF32Buffers<D, R> * 2 * 64) * (D + 4) + 2 * R * kPitch) * 4; }

template <int D, int R, bool keys>
__device__ __forceinline__ void f32_tile(float* sm, const float* q, const float* k, const float* v, const float* dout,
                                         const AttendGradArgs& a, int tile) {
  constexpr int KS = 64 / R, NB = kF32Buffers<D, R>, PIECE = 64 * (D + 4);
  float *r1 = sm, *r2 = r1 + R * (D + 4), *cs = r2 + R * (D + 4), *sp = cs + NB * 2 * PIECE, *sd = sp + R * kPitch;
  const int h = blockIdx.y, b = keys ? blockIdx.z : blockIdx.z - a.B;
  const int group = threadIdx.x >> 7, lane = threadIdx.x & 127;
  const int kz = lane % KS, tx = lane / KS % 16, ty = lane / (KS * 16);
  const int N = a.N_valid, shift = a.block == 128 ? 1 : 0, W = (a.nB + 31) >> 5;
  const long long bh = static_cast<long long>(b) * a.H + h;
  const GradStride &s_r1 = a.st[keys ? kK : kQ], &s_r2 = a.st[keys ? kV : kDout];
  const GradStride &s_c1 = a.st[keys ? kQ : kK], &s_c2 = a.st[keys ? kDout : kV];
  const float* g1 = (keys ? q : k) + offset(s_c1, b, h, 0);
  const float* g2 = (keys ? dout : v) + offset(s_c2, b, h, 0);
  const int r0 = tile * R, mine = r0 / a.block;
  const float scale = 1.0f / sqrtf(static_cast<float>(D)), scale2 = scale * kLog2e;
  load_rows<D>(r1, (keys ? k : q) + offset(s_r1, b, h, 0), s_r1.n, r0, R, N);
  load_rows<D>(r2, (keys ? v : dout) + offset(s_r2, b, h, 0), s_r2.n, r0, R, N);
  float acc[8][D / 16];             // dv or dk by the group, or the group's share of dq
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
  grid_wait();
  auto load = [&](int buf, int c0) {
    load_rows<D>(cs + buf * 2 * PIECE, g1, s_c1.n, c0, 64, N);
    load_rows<D>(cs + buf * 2 * PIECE + PIECE, g2, s_c2.n, c0, 64, N);
    loads_commit();
  };
  Pieces it{(keys ? a.bits_t : a.bits) + (bh * a.nB + mine) * W, W, N, shift, -1, 0, 0u, 0, 0};
  bool more = it.next();
  if (more) load(0, it.c0);
  const float* column = (group ? a.neg_delta : a.neg_lse2) + bh * a.Npad;      // rows < Npad: the tables are padded
  float nv[keys ? 4 : 8];           // -lse or -D of the thread's columns (keys) or rows (queries)
  if (!keys) {
#pragma unroll
    for (int i = 0; i < 8; ++i) nv[i] = column[r0 + ty + R / 8 * i];
  }
  for (int buf = 0; more; buf ^= NB - 1) {
    const int c0 = it.c0;
    uint64_t set = ~0ull;           // per-token lists: the query tokens that keep the key block
    if (a.masks) set = a.masks_t[(bh * a.nB + (keys ? mine : it.other)) * a.nB + (keys ? it.other : mine)];
    if (keys) {
#pragma unroll
      for (int j = 0; j < 4; ++j) nv[j] = column[c0 + tx + 16 * j];
    }
    more = it.next();
    if (NB == 2 && more) load(buf ^ 1, it.c0);
    else loads_commit();
    loads_wait<NB - 1>();
    __syncthreads();
    const float *c1 = cs + buf * 2 * PIECE, *c2 = c1 + PIECE;
    float p[8][4];
    dots<D, R>(p, group ? r2 : r1, group ? c2 : c1, ty, tx, kz);
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i / (8 / KS) != kz) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = ty + R / 8 * i, col = tx + 16 * j;
          const int qn = keys ? c0 + col : r0 + row, kn = keys ? r0 + row : c0 + col;
          const bool on = kn < N && ((set >> (qn & 63)) & 1ull);
          sp[row * kPitch + col] = on ? exp2f(fmaf(p[i][j], scale2, nv[keys ? j : i])) : 0.f;
        }
      }
    }
    __syncthreads();
    if (group == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i / (8 / KS) != kz) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = (ty + R / 8 * i) * kPitch + tx + 16 * j;
          sd[at] = sp[at] * (p[i][j] + nv[keys ? j : i]);
        }
      }
    }
    if (keys) {
      if (group == 1) named_bar_sync(1, 128);
      weighted<D, R>(acc, group ? sd : sp, group ? c1 : c2, 0, 64, ty, tx, kz);
    } else {
      __syncthreads();
      weighted<D, R>(acc, sd, c1, 32 * group, 32 * group + 32, ty, tx, kz);
    }
    __syncthreads();                // the piece's rows, P and dS may be overwritten
    if (NB == 1 && more) load(0, it.c0);
  }
  loads_wait<0>();
  if (keys) {
    const GradStride& st = a.st[group ? kDk : kDv];
    store_rows<D, R>(static_cast<float*>(group ? a.dk : a.dv) + offset(st, b, h, 0), st.n, r0, N, acc, group ? scale : 1.f,
                     nullptr, ty, tx, kz);
  } else {
    // the second group's share through shared memory (the loop is over)
    if (group == 1) store_rows<D, R>(cs, D + 4, 0, R, acc, 1.f, nullptr, ty, tx, kz);
    __syncthreads();
    if (group == 0)
      store_rows<D, R>(static_cast<float*>(a.dq) + offset(a.st[kDq], b, h, 0), a.st[kDq].n, r0, N, acc, scale, cs, ty, tx, kz);
  }
}

// blockIdx.z: batch elements of keys (dk, dv), then of queries (dq): the shorter tiles fill the last wave.
template <int D, int R>
__global__ void __launch_bounds__(256) attend_grad_f32_kernel(const float* __restrict__ q, const float* __restrict__ k,
                                                             const float* __restrict__ v, const float* __restrict__ dout,
                                                             const __grid_constant__ AttendGradArgs a) {
  extern __shared__ __align__(16) float sm[];
  if (static_cast<int>(blockIdx.z) < a.B) f32_tile<D, R, true>(sm, q, k, v, dout, a, blockIdx.x);
  else f32_tile<D, R, false>(sm, q, k, v, dout, a, blockIdx.x);
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

template <typename T, int D>
cudaError_t prep(const void* out, const void* dout, const float* lse, const AttendGradArgs& a, cudaStream_t s) {
  const long long W = (a.nB + 31) / 32, bh = static_cast<long long>(a.B) * a.H;
  const long long index_blocks = bh * W, row_blocks = bh * a.Npad / kRowsPerBlock;
  if (index_blocks + row_blocks > 2147483647ll) return cudaErrorInvalidValue;
  const size_t sums = sizeof(T) == 2 ? kPrepThreads * 8 * sizeof(float) : 0;
  const size_t smem = std::max<size_t>(32 * W * 4, sums);
  attend_grad_prep_kernel<T, D><<<static_cast<unsigned>(index_blocks + row_blocks), kPrepThreads, smem, s>>>(
      static_cast<const T*>(out), static_cast<const T*>(dout), lse, a, static_cast<int>(index_blocks));
  return cudaGetLastError();
}

template <int D, int R>
cudaError_t f32(const float* q, const float* k, const float* v, const float* dout, const AttendGradArgs& a, cudaStream_t s) {
  constexpr int smem = f32_smem<D, R>();
  cudaError_t e = cudaFuncSetAttribute(attend_grad_f32_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.N_valid + R - 1) / R;
  return launch_dependent(attend_grad_f32_kernel<D, R>, dim3(tiles, a.H, 2 * a.B), dim3(256), smem, s, q, k, v, dout, a);
}

template <int D>
cudaError_t f32_rows(const float* q, const float* k, const float* v, const float* dout, const AttendGradArgs& a,
                     cudaStream_t s) {
  const long long ctas = 2ll * a.B * a.H * ((a.N_valid + 63) / 64);      // with R = 64
  if (ctas >= 148) return f32<D, 64>(q, k, v, dout, a, s);
  return ctas >= 74 ? f32<D, 32>(q, k, v, dout, a, s) : f32<D, 16>(q, k, v, dout, a, s);
}

}  // namespace

size_t attend_grad_workspace(AttendGradArgs* a, int dtype, void* base) {
  const size_t bh = static_cast<size_t>(a->B) * a->H, W = (a->nB + 31) / 32;
  a->Npad = (a->N_valid + 127) / 128 * 128;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return static_cast<char*>(base) + here;
  };
  char* p[6];
  p[0] = take(bh * a->Npad * sizeof(float));
  p[1] = take(bh * a->Npad * sizeof(float));
  p[2] = take(bh * a->nB * W * sizeof(uint32_t));
  p[3] = take(bh * a->nB * W * sizeof(uint32_t));
  p[4] = a->masks ? take(bh * a->nB * a->nB * sizeof(uint64_t)) : nullptr;
  p[5] = dtype == LBSA_BF16 ? take(bh * (a->Npad / kRowsPerBlock) * a->d * sizeof(float)) : nullptr;
  if (base) {
    a->k_means = reinterpret_cast<float*>(p[5]);
    a->neg_lse2 = reinterpret_cast<float*>(p[0]);
    a->neg_delta = reinterpret_cast<float*>(p[1]);
    a->bits = reinterpret_cast<uint32_t*>(p[2]);
    a->bits_t = reinterpret_cast<uint32_t*>(p[3]);
    a->masks_t = reinterpret_cast<uint64_t*>(p[4]);
  }
  return at;
}

cudaError_t launch_attend_grad_prep(const void* out, const void* dout, const float* lse, int dtype,
                                    const AttendGradArgs& a, cudaStream_t s) {
  if (dtype == LBSA_BF16)
    return a.d == 128 ? prep<__nv_bfloat16, 128>(out, dout, lse, a, s) : prep<__nv_bfloat16, 64>(out, dout, lse, a, s);
  return a.d == 128 ? prep<float, 128>(out, dout, lse, a, s) : prep<float, 64>(out, dout, lse, a, s);
}

cudaError_t launch_attend_grad_f32(const float* q, const float* k, const float* v, const float* dout,
                                   const AttendGradArgs& a, cudaStream_t s) {
  return a.d == 128 ? f32_rows<128>(q, k, v, dout, a, s) : f32_rows<64>(q, k, v, dout, a, s);
}

}  // namespace lbsa
