// Gradients of block-sparse attention on sm_100a tensor cores (bf16 in, fp32
// accumulate).  The mathematics and the tables are attend_grad.cu's.
//
// Two kinds of CTA in one launch, each owning 128 rows and walking the union of
// its two 64-row blocks' lists in steps of 128 columns (two 64-row pieces of the
// other side, which need not be neighbours):
//   keys      S^T = K Q^T, dP^T = V dO^T (rows are keys, columns queries), then
//             dV += P^T dO and dK += dS^T Q: four products a step
//   queries   S = Q K^T, dP = dO V^T, then dQ += dS K: three products a step
// Seven products in place of the formula's five, for which no gradient is
// added across CTAs: no atomics, no fp32 dQ in memory (a read-modify-write of
// 64 KB a step) and the same bits on every call.
//
// Warp roles (18 warps, one CTA an SM):
//   softmax   four warpgroups; thread t of each owns row t = TMEM lane
//             and 32 of the step's columns.  P = 2^(S scale - lse), packed to
//             bf16 over the S columns just read (keys); dS = P (dP - D), over
//             the dP columns; at the end the rows' sums.
//   producer  TMA: walks the two bit rows, loads the CTA's own tiles once, then
//             the first operand's pieces through a 3-stage and the second's
//             through a 2-stage ring, each refilled when its own last product
//             is done (keys: with lse and D of the columns).
//   issuer    UMMAs.
// TMEM columns: S, dP, dK or dQ, dV.  A query tile has no dV: its q and dout
// rows take those columns, so that all three of its products read their A
// operand from TMEM.  With both operands in shared memory a 128 x 128 x 16
// product reads 8 KB in the 64 cycles that the tensor core needs for it, the
// whole bandwidth, and took 90 to 100 cycles.
//
// Roundings: P and dS become bf16 once, as operands (2^-8 relative at most); all
// else is fp32.  D is taken from the rounded out.  sum_c dS_rc = 0 takes out of dq
// what the keys have in common, but rounded dS sum to some e_r, which would bring
// it back.  So dq_r = scale sum_c dS_rc (k_c - m_r), the same number for any m_r,
// and e_r m_r is taken off at the end.  What is best taken off is the row's own
// mean key, sum_c P_rc k_c, a fourth product; m_r stands near it and is read from
// a table: the mean of the 64 keys among which the row's largest P is, 0 where
// those have little in common (attend_grad_prep_kernel), or that P's own key where
// it takes half of the row or its piece is ragged.  Keys that the row does not
// keep, or gives no P, have no part in it, whatever their size.  dq off by
// (Frobenius; 4,096 tokens, d = 128, half of the blocks; rounding the exact result
// costs 1.7e-3): keys of unit noise 2.4e-3, about a common vector of 1 or of 20
// times that size 2.4e-3 (without m_r 3.2e-3 and 4.5e-2), about one that changes
// along the clip 2.5e-3, about a vector for each block of 1 to 20 times that size
// 2.9e-3 to 3.4e-3 (without 2.7e-3 to 1.3e-2; with the nearest kept piece's mean
// 3.3e-3 to 1.9e-2), logits of deviation 12 2.9e-3.  e_r takes a mixed fp32 + bf16
// addition an element, the largest P half a three-way maximum: 0.5 % of the
// time below.
//
// What bounds it: 21 x 30 x 52 tokens, 12 heads of 128, 0.90 of the blocks kept
// (0.97 of them in a tile's union): 16.1 ms from idle, 18.3 ms back to back, where
// the card sits at its power limit (1.55 GHz); 810 TFLOP/s of the formula's
// five products, 1,220 of the products done, 0.88 of what cuBLAS sustains.  A
// keys step is a chain of P, then dV and the next S: 2,650 cycles for 2,048 of
// products; a queries step one of dS, then dQ and the next dP: 2,050 for 1,536.
#include "lbsa_train_device.cuh"

namespace lbsa {
namespace {

constexpr int BM = 128;             // rows of a tile
constexpr int kCols = 32;           // columns of a step that a softmax warpgroup takes
constexpr int N1 = 3, N2 = 2;       // ring depths of the two operands
// Of every 8 groups of four logits kPoly8 take two of their exponentials on the
// FMA pipe (a cubic, relative error 7.5e-5, far below the rounding of P and dS
// to bf16, 2^-8), which unloads the MUFU: with 4 (a quarter of them) 8,192
// dense tokens of 8 heads of 64 took 0.59 ms, with none 0.61.
constexpr int kPoly8 = 4;
constexpr int BN = 128;             // columns of a step, two 64-row pieces
constexpr int kGroups = BN / kCols; // softmax warpgroups
constexpr int kProducer = kGroups * 4, kIssuer = kProducer + 1;      // their warps
constexpr int kThreads = (kIssuer + 1) * 32;
constexpr uint32_t kTmemCols = 512;

template <int D, bool KEYS>
struct Layout {
  // S buffers: where the sums leave room for a second (keys, d = 64), S of the
  // step after next is issued as soon as P has been read, instead of one later
  // (8,192 dense tokens, 8 heads: 0.59 -> 0.58 ms)
  static constexpr int SB = KEYS && D == 64 ? 2 : 1;
  // TMEM columns
  static constexpr uint32_t S = 0, DP = SB * BN, ACC1 = DP + BN, ACC2 = ACC1 + D;
  static constexpr uint32_t ROWS1 = ACC2, ROWS2 = ACC2 + D / 2;      // queries: the tile's q and dout, two bf16 a column
  // shared memory
  static constexpr int TILE = BM * D * 2;                    // also a step's rows of one operand
  static constexpr int OFF_R1 = 0, OFF_R2 = TILE;            // queries: RowParts
  static constexpr int OFF_C1 = 2 * TILE, OFF_C2 = OFF_C1 + N1 * TILE;
  static constexpr int OFF_COL = OFF_C2 + N2 * TILE;         // per stage: BN lse, BN D
  static constexpr int OFF_BAR = OFF_COL + N2 * 2 * BN * 4;
  static constexpr int OFF_SETS = OFF_BAR + 20 * 8;          // per step of four: token sets [half][piece]
  static constexpr int OFF_MISC = OFF_SETS + 4 * 4 * 8;      // tmem, abort, count, pad, entries[4][2]
};
template <int D>
constexpr int kSmemBytes = Layout<D, true>::OFF_MISC + 48;
static_assert(kSmemBytes<128> <= 227 * 1024, "shared memory of a CTA");

// What a step's columns are: the piece of each 64 | kWhole where all its rows
// exist | the halves of the tile that keep it << 30.
constexpr uint32_t kPiece = 0x0FFFFFFFu, kWhole = 1u << 29;

// c_empty: a step's last product is done (first operand's stage, columns' lse
// and D); c2_empty: the second operand's last product is done.  s_full has two
// arrivals, the UMMAs' completion and the issuer's own, which passes on what it
// has waited for: the step's entry and (with one S buffer) its columns' values,
// for which the softmax warps then need no wait of their own.  With two S
// buffers the issuer may not wait for those: they come when step j - 2 is over,
// which takes a product that it issues later.
struct Bars {
  uint64_t *r_full, *c1_full, *c2_full, *col_full, *c_empty, *c2_empty, *s_full, *dp_full, *drain, *s_done, *ds_full;
};
constexpr int kBars = 20, kSFull = 13, kWarpBars = 17;      // from kWarpBars on every softmax warp arrives
__device__ __forceinline__ Bars make_bars(uint8_t* base) {
  uint64_t* b = reinterpret_cast<uint64_t*>(base);
  return Bars{b, b + 1, b + 4, b + 6, b + 8, b + 11, b + kSFull, b + 15, b + 16, b + kWarpBars, b + 19};
}

// Bulk copy of `bytes` (a multiple of 16) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

struct Tile {
  int tile, h, b, n_steps;
  long long bh;
};

// The walk over a tile's kept pieces: the set bits of its two bit rows.
struct Walk {
  const uint32_t *r0, *r1;          // r1: NULL for 128-row blocks and a missing second block
  int W, w, shift, sub, N;
  uint32_t a, b, rest;              // words and their union's bits still to come
  __device__ __forceinline__ void init(const uint32_t* x, const uint32_t* y, int words, int sh, int n) {
    N = n;
    r0 = x;
    r1 = y;
    W = words;
    shift = sh;
    w = -1;
    sub = 0;
    rest = 0u;
  }
  // the next piece's entry; 0 at the end (a piece that is walked is kept by a half)
  __device__ __forceinline__ uint32_t next() {
    while (rest == 0u) {
      if (++w >= W) return 0u;
      a = r0[w];
      b = r1 ? r1[w] : (shift ? a : 0u);
      rest = a | b;
    }
    const int bit = __ffs(rest) - 1;
    const uint32_t halves = ((a >> bit) & 1u) | (((b >> bit) & 1u) << 1);
    const uint32_t piece = ((static_cast<uint32_t>(w * 32 + bit)) << shift) + sub;
    if (sub == shift) {
      rest &= rest - 1u;
      sub = 0;
    } else {
      sub = 1;
    }
    return piece | ((piece + 1) * 64 <= static_cast<uint32_t>(N) ? kWhole : 0u) | (halves << 30);
  }
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long wl, int32_t* status,
                                          volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, wl, status, abort_flag));
}
// Every lane's TMEM accesses are done: one arrival for the warp.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// 64 rows into the `half` of a 128-row buffer
template <int D>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int half, int piece, const Tile& t) {
  for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * BM * 128 + half * 64 * 128, m, bar, c * 64, piece * 64, t.h, t.b);
}

template <int D, bool KEYS, bool MASKED>
__device__ __forceinline__ void produce(uint8_t* smem, const Bars& bars, const CUtensorMap* c1, const CUtensorMap* c2,
                                        const AttendGradArgs& a, const Tile& t, Walk walk, uint32_t* entries,
                                        volatile int* abort_flag) {
  using L = Layout<D, KEYS>;
  uint32_t e[2], ahead[2];          // entries of this step, of the next one
  int done1 = 0, done2 = 0, done_col = 0;
  // step j's first operand into the stage that step j - 3 had, its entries into
  // the slots that step j - 4 had; false past the last step
  auto first = [&](int j, int stage) {
    ahead[0] = walk.next();
    if (ahead[0] == 0u) return false;
    ahead[1] = walk.next();
    if (ahead[1] == 0u) ahead[1] = ahead[0] & kPiece;       // an odd tail: the piece again, kept by nobody
    entries[(j & 3) * 2] = ahead[0];
    entries[(j & 3) * 2 + 1] = ahead[1];
    if (MASKED) {
      // per-token lists: the query tokens of each (half, piece) pair that keep its key block
      uint64_t* sets = reinterpret_cast<uint64_t*>(smem + L::OFF_SETS) + (j & 3) * 4;
      uint64_t v[4];
      for (int i = 0; i < 4; ++i) {
        const long long mine = t.tile * 2 + (i >> 1), piece = ahead[i & 1] & kPiece;
        v[i] = (ahead[i & 1] >> (30 + (i >> 1))) & 1u
                   ? a.masks_t[(t.bh * a.nB + (KEYS ? mine : piece)) * a.nB + (KEYS ? piece : mine)]
                   : 0ull;
      }
      for (int i = 0; i < 4; ++i) sets[i] = v[i];
    }
    mbar_arrive_expect_tx(bars.c1_full + stage, L::TILE);
    for (int p = 0; p < 2; ++p) load_rows<D>(smem + L::OFF_C1 + stage * L::TILE, c1, bars.c1_full + stage, p, ahead[p] & kPiece, t);
    done1 = j + 1;
    return true;
  };
  if (!first(0, 0)) {
    if (KEYS) mbar_wait(bars.r_full, 0, a.wait_limit, a.status, nullptr);      // the own rows land before the CTA exits
    return;
  }
  int stage = 1;                    // of step j + 1
  for (int j = 0;; ++j) {
    e[0] = ahead[0];
    e[1] = ahead[1];
    if (j >= N2 && !mbar_wait(bars.c2_empty + (j & 1), ((j >> 1) & 1) ^ 1, a.wait_limit, a.status, abort_flag)) break;
    uint64_t* f2 = bars.c2_full + (j & 1);
    mbar_arrive_expect_tx(f2, L::TILE);
    for (int p = 0; p < 2; ++p) load_rows<D>(smem + L::OFF_C2 + (j & 1) * L::TILE, c2, f2, p, e[p] & kPiece, t);
    done2 = j + 1;
    // step j - 2 is over: its columns' values and the stage that step j + 1 takes are free
    if (j >= 2 && !mbar_wait(bars.c_empty + stage, (((j - 2) / N1) & 1), a.wait_limit, a.status, abort_flag)) break;
    if (KEYS) {
      uint64_t* fc = bars.col_full + (j & 1);
      mbar_arrive_expect_tx(fc, 2 * BN * 4);
      for (int p = 0; p < 2; ++p) {
        const int piece = e[p] & kPiece;
        float* col = reinterpret_cast<float*>(smem + L::OFF_COL) + (j & 1) * 2 * BN + p * 64;
        bulk_load(col, a.neg_lse2 + t.bh * a.Npad + piece * 64, 256, fc);
        bulk_load(col + BN, a.neg_delta + t.bh * a.Npad + piece * 64, 256, fc);
      }
      done_col = j + 1;
    }
    if (!first(j + 1, stage)) break;
    if (++stage == N1) stage = 0;
  }
  if (*abort_flag) {
    // copies still in flight land before the CTA can exit
    if (KEYS) mbar_wait(bars.r_full, 0, a.wait_limit, a.status, nullptr);
    for (int s = max(done1 - N1, 0); s < done1; ++s)
      mbar_wait(bars.c1_full + s % N1, (s / N1) & 1, a.wait_limit, a.status, nullptr);
    for (int s = max(done2 - N2, 0); s < done2; ++s)
      mbar_wait(bars.c2_full + s % N2, (s / N2) & 1, a.wait_limit, a.status, nullptr);
    for (int s = max(done_col - N2, 0); s < done_col; ++s)
      mbar_wait(bars.col_full + s % N2, (s / N2) & 1, a.wait_limit, a.status, nullptr);
  }
}

// d[128 x BN] = x y^T over d; x, y: descriptors of K-major rows in shared memory
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d, uint64_t x, uint64_t y) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    umma_ss(d, x + (((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4), y + (((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4),
            idesc_bf16_f32(BM, BN, 0), kk > 0 ? 1u : 0u);
}
// the same with x's rows packed in TMEM
template <int D>
__device__ __forceinline__ void mma_rows_ts(uint32_t d, uint32_t x, uint64_t y) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    umma_ts(d, x + kk * 8, y + (((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4), idesc_bf16_f32(BM, BN, 0), kk > 0 ? 1u : 0u);
}
// d[128 x D] += p y; p packed in TMEM (each warpgroup's columns start kCols further), y: MN-major rows
template <int D>
__device__ __forceinline__ void mma_sum(uint32_t d, uint32_t p, uint64_t y, bool first) {
  constexpr int PER = kCols / 16;
#pragma unroll
  for (int kk = 0; kk < BN / 16; ++kk)
    umma_ts(d, p + (kk / PER) * kCols + (kk % PER) * 8, y + kk * (2048 >> 4), idesc_bf16_f32(BM, D, 1),
            (!first || kk > 0) ? 1u : 0u);
}

// The whole warp walks the steps, so that addresses and descriptors stay
// warp-uniform, and one elected lane issues: with a single lane in the loop the
// operands went through per-thread registers and an instruction took about 100
// cycles to issue, where the tensor core needs 64 for it.
// Rings are as long as a barrier's phase could be missed otherwise.  c_empty is
// three: the producer loads step j's second operand before it waits for the end
// of step j - 2, so that on a pair step j's end could come first.  With two S
// buffers S of step j + 1 is issued before P of step j is waited for: s_full and
// s_done are pairs.  Every other barrier's next phase needs an instruction that
// follows the wait for the last one.
// tcgen05.mma instructions of one thread complete in the order of their issue:
// S of step j + 1 may follow the product that reads P of step j from the same
// columns, and dP the one that reads dS.
template <int D, bool KEYS>
__device__ __forceinline__ void issue(uint8_t* smem, const Bars& bars, uint32_t tmem, const AttendGradArgs& a,
                                      int n_steps, volatile int* abort_flag) {
  using L = Layout<D, KEYS>;
  const uint64_t r1 = smem_desc_sw128(smem_u32(smem + L::OFF_R1), 16, 1024), r2 = r1 + ((L::OFF_R2 - L::OFF_R1) >> 4);
  const uint64_t c1 = r1 + ((L::OFF_C1 - L::OFF_R1) >> 4), c2 = r1 + ((L::OFF_C2 - L::OFF_R1) >> 4);
  const uint64_t m1 = smem_desc_sw128(smem_u32(smem + L::OFF_C1), BN * 128, 1024), m2 = m1 + ((L::OFF_C2 - L::OFF_C1) >> 4);
  constexpr uint64_t STAGE = L::TILE >> 4;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = warp_wait(bar, parity, a.wait_limit, a.status, abort_flag);
    tc_fence_after();
    return ok;
  };
  int st_next = 0, ph_next = 0;                 // the first operand's ring: stage and phase of the next S
  auto s_of = [&](int j) {
    const int buf = j & (L::SB - 1);
    if (!wait(bars.c1_full + st_next, ph_next)) return false;
    if (elect_one()) {
      if (KEYS) mma_rows<D>(tmem + L::S + buf * BN, r1, c1 + st_next * STAGE);
      else mma_rows_ts<D>(tmem + L::S, tmem + L::ROWS1, c1 + st_next * STAGE);
      umma_commit(bars.s_full + buf);
    }
    __syncwarp();
    if (KEYS && L::SB == 1 && !wait(bars.col_full + (j & 1), (j >> 1) & 1)) return false;
    if (elect_one()) mbar_arrive(bars.s_full + buf);
    __syncwarp();
    if (++st_next == N1) {
      st_next = 0;
      ph_next ^= 1;
    }
    return true;
  };
  auto dp_of = [&](int j) {
    if (!wait(bars.c2_full + (j & 1), (j >> 1) & 1)) return false;
    if (elect_one()) {
      if (KEYS) mma_rows<D>(tmem + L::DP, r2, c2 + (j & 1) * STAGE);
      else mma_rows_ts<D>(tmem + L::DP, tmem + L::ROWS2, c2 + (j & 1) * STAGE);
      umma_commit(bars.dp_full);
      if (!KEYS) umma_commit(bars.c2_empty + (j & 1));
    }
    __syncwarp();
    return true;
  };
  bool ok = n_steps > 0 && wait(bars.r_full, 0) && s_of(0) && dp_of(0) && (L::SB == 1 || n_steps == 1 || s_of(1));
  int st = 0;                                   // step j's stage of the first operand
  for (int j = 0; ok && j < n_steps; ++j) {
    const int buf = j & (L::SB - 1);
    if (!wait(bars.s_done + buf, (j / L::SB) & 1)) break;
    if (KEYS) {
      if (elect_one()) {
        mma_sum<D>(tmem + L::ACC2, tmem + L::S + buf * BN, m2 + (j & 1) * STAGE, j == 0);
        umma_commit(bars.c2_empty + (j & 1));
      }
      __syncwarp();
    }
    if (j + L::SB < n_steps && !s_of(j + L::SB)) break;
    if (!wait(bars.ds_full, j & 1)) break;
    if (elect_one()) {
      mma_sum<D>(tmem + L::ACC1, tmem + L::DP, m1 + st * STAGE, j == 0);
      umma_commit(bars.c_empty + st);
    }
    __syncwarp();
    if (++st == N1) st = 0;
    if (j + 1 < n_steps && !dp_of(j + 1)) break;
  }
  // every UMMA has completed before the sums are read and TMEM is released
  if (elect_one()) umma_commit(bars.drain);
  __syncwarp();
  mbar_wait(bars.drain, 0, a.wait_limit, a.status, nullptr);
}

// P of a thread's columns in place of their logits (r), then dS = P (dP - D) in place
// of dP.  neg_lse / neg_delta: of the columns (keys) or of the row (queries).
template <bool KEYS>
__device__ __forceinline__ void probabilities(uint32_t (&r)[kCols], const float* neg_lse, float row_neg_lse, float scale_log2) {
  const unsigned long long sc2 = f2_as_u64(scale_log2, scale_log2);
#pragma unroll
  for (int c = 0; c < kCols; c += 4) {
    ulonglong2 l = make_ulonglong2(f2_as_u64(row_neg_lse, row_neg_lse), f2_as_u64(row_neg_lse, row_neg_lse));
    if (KEYS) l = *reinterpret_cast<const ulonglong2*>(neg_lse + c);
    float v[4];
    u64_as_f2(ffma2(f2_as_u64(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, l.x), v[0], v[1]);
    u64_as_f2(ffma2(f2_as_u64(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), sc2, l.y), v[2], v[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[c + i] = __float_as_uint((c / 4 * kPoly8) % 8 < kPoly8 && i < 2 ? exp2_poly3(v[i]) : ex2(v[i]));
  }
}
template <bool KEYS>
__device__ __forceinline__ void score_gradients(uint32_t (&g)[kCols], const uint32_t (&p)[kCols], const float* neg_delta,
                                                float row_neg_delta) {
#pragma unroll
  for (int c = 0; c < kCols; c += 4) {
    ulonglong2 d = make_ulonglong2(f2_as_u64(row_neg_delta, row_neg_delta), f2_as_u64(row_neg_delta, row_neg_delta));
    if (KEYS) d = *reinterpret_cast<const ulonglong2*>(neg_delta + c);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const unsigned long long x =
          fmul2(fadd2(f2_as_u64(__uint_as_float(g[c + i]), __uint_as_float(g[c + i + 1])), i ? d.y : d.x),
                f2_as_u64(__uint_as_float(p[c + i]), __uint_as_float(p[c + i + 1])));
      g[c + i] = static_cast<uint32_t>(x);
      g[c + i + 1] = static_cast<uint32_t>(x >> 32);
    }
  }
}

// 0 in the columns that do not count.  ROWS: `on` is all or nothing (a query row
// keeps a whole piece or none of it) unless the piece is ragged.
template <bool ROWS>
__device__ __forceinline__ void keep_columns(uint32_t (&r)[kCols], uint32_t on, uint32_t whole) {
  if (ROWS && whole) {
#pragma unroll
    for (int c = 0; c < kCols; ++c) r[c] &= on;
  } else {
#pragma unroll
    for (int c = 0; c < kCols; ++c) r[c] = ((on >> c) & 1u) ? r[c] : 0u;
  }
}
// rounded to bf16, two a column
__device__ __forceinline__ void store_packed(uint32_t taddr, const uint32_t (&r)[kCols], uint32_t (&pk)[kCols / 2]) {
#pragma unroll
  for (int c = 0; c < kCols / 2; ++c) pk[c] = pack_bf16x2(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]));
  tmem_st16(taddr, pk);
  tmem_wait_st();
}

// A query tile's own rows into TMEM: each warpgroup a part of q's or dout's row.
template <int D>
__device__ __forceinline__ void own_rows(const Bars& bars, uint32_t tmem, const AttendGradArgs& a, const Tile& t) {
  using L = Layout<D, false>;
  constexpr int PART = D / kGroups;              // 32-bit words: D / 2 a row, two warpgroups a tensor
  const int wg = threadIdx.x >> 7, row = threadIdx.x & 127, grow = t.tile * BM + row;
  const GradStride& st = a.st[wg & 1 ? kDout : kQ];
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(wg & 1 ? a.dout : a.q) + t.b * st.b +
                                                    t.h * st.h + grow * st.n) + (wg >> 1) * (PART / 4);
  const uint32_t dst = tmem + (static_cast<uint32_t>(row & ~31) << 16) + (wg & 1 ? L::ROWS2 : L::ROWS1) + (wg >> 1) * PART;
  uint32_t v[PART / 16][16];                     // every load in flight before the first store
#pragma unroll
  for (int c = 0; c < PART / 16; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = grow < a.N_valid ? __ldg(src + c * 4 + i) : make_uint4(0u, 0u, 0u, 0u);
      v[c][4 * i] = x.x;
      v[c][4 * i + 1] = x.y;
      v[c][4 * i + 2] = x.z;
      v[c][4 * i + 3] = x.w;
    }
#pragma unroll
  for (int c = 0; c < PART / 16; ++c) tmem_st16(dst + c * 16, v[c]);
  tmem_wait_st();
  warp_arrive(bars.r_full, threadIdx.x & 31);
}

// What the four warpgroups know of a query row, each from its columns.
struct RowParts {
  float sum[kGroups][BM];           // of dS, as rounded
  float top[kGroups][BM];           // the largest P
  int at[kGroups][BM];              // its piece; ~its key where P is half of the row's or more, or the piece ragged
};
static_assert(sizeof(RowParts) <= Layout<64, false>::TILE, "in an operand's tile");

template <int D, bool KEYS, bool MASKED>
__device__ __forceinline__ void softmax(uint8_t* smem, const Bars& bars, uint32_t tmem, const AttendGradArgs& a,
                                        const Tile& t, const uint32_t* entries, const CUtensorMap* out1,
                                        const CUtensorMap* out2, float scale_log2, float scale, volatile int* abort_flag) {
  using L = Layout<D, KEYS>;
  const int lane = threadIdx.x & 31, wg = threadIdx.x >> 7, row = threadIdx.x & 127;
  const int half = row >> 6, grow = t.tile * BM + row;
  const int c0 = wg * kCols, p = c0 >> 6, in_piece = c0 & 63;          // the thread's columns, their piece of the step
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(row & ~31) << 16);
  const uint32_t s_col = t_lane + L::S + c0, dp_col = t_lane + L::DP + c0;
  const long long wl = a.wait_limit;
  float neg_lse = 0.f, neg_delta = 0.f;
  if (!KEYS) {
    neg_lse = a.neg_lse2[t.bh * a.Npad + grow];
    neg_delta = a.neg_delta[t.bh * a.Npad + grow];
  }
  const uint64_t* sets = reinterpret_cast<const uint64_t*>(smem + L::OFF_SETS);
  bool alive = true;
  float ds_sum[2] = {0.f, 0.f};       // queries: the row's rounded dS, two sums
  float top = 0.f;                    // queries: RowParts::top, at
  int top_at = 0;
  for (int j = 0; j < t.n_steps; ++j) {
    const int buf = j & (L::SB - 1);
    if (KEYS && L::SB == 2) {
      alive = warp_wait(bars.col_full + (j & 1), (j >> 1) & 1, wl, a.status, abort_flag);
      if (!alive) break;
    }
    alive = warp_wait(bars.s_full + buf, (j / L::SB) & 1, wl, a.status, abort_flag);
    if (!alive) break;
    tc_fence_after();
    uint32_t r[kCols], g[kCols];
    tmem_ld32(s_col + buf * BN, r);
    const float* col = reinterpret_cast<const float*>(smem + L::OFF_COL) + (j & 1) * 2 * BN + c0;
    const uint32_t e = entries[(j & 3) * 2 + p];
    // every column counts (the same for the warp); otherwise those of `on`, from bit 0
    const bool all = !MASKED && ((e >> (30 + half)) & 1u) && (KEYS || (e & kWhole));
    uint32_t on = 0u;
    if (!all) {
      const int valid = a.N_valid - static_cast<int>(e & kPiece) * 64 - in_piece;
      if (MASKED) {
        const uint64_t set = sets[(j & 3) * 4 + half * 2 + p];
        on = KEYS ? static_cast<uint32_t>(set >> in_piece) : ((set >> (row & 63)) & 1ull) ? 0xFFFFFFFFu : 0u;
      } else if ((e >> (30 + half)) & 1u) {
        on = 0xFFFFFFFFu;
      }
      if (!KEYS && valid < kCols) on &= valid > 0 ? (1u << valid) - 1u : 0u;
    }
    tmem_wait_ld_dep(r);
    if (!KEYS) warp_arrive(bars.s_done, lane);                       // the S columns are free
    probabilities<KEYS>(r, col, neg_lse, scale_log2);
    if (!all) {
      keep_columns<MASKED && !KEYS>(r, on, e & kWhole);
    }
    if (KEYS) {
      uint32_t pk[kCols / 2];
      store_packed(s_col + buf * BN, r, pk);
      warp_arrive(bars.s_done + buf, lane);
    } else {
      float most[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        most[0] = fmax3(most[0], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
        most[1] = fmax3(most[1], __uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
      }
      most[0] = fmaxf(most[0], most[1]);
      if (most[0] > top) {
        top = most[0];
        top_at = static_cast<int>(e & kPiece);
        if (top >= 0.5f || !(e & kWhole)) {
          const int key0 = top_at * 64 + in_piece;
#pragma unroll
          for (int c = kCols - 1; c >= 0; --c)
            if (__uint_as_float(r[c]) == top) top_at = ~(key0 + c);
        }
      }
    }
    alive = warp_wait(bars.dp_full, j & 1, wl, a.status, abort_flag);
    if (!alive) break;
    tc_fence_after();
    tmem_ld32(dp_col, g);
    tmem_wait_ld_dep(g);
    score_gradients<KEYS>(g, r, col + BN, neg_delta);                // 0 where P is
    uint32_t pk[kCols / 2];
    store_packed(dp_col, g, pk);
    warp_arrive(bars.ds_full, lane);
    if (!KEYS) {
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c)
        asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\nadd.rn.f32.bf16 %0, l, %0;\nadd.rn.f32.bf16 %1, h, %1;\n}"
            : "+f"(ds_sum[0]), "+f"(ds_sum[1])
            : "r"(pk[c]));
    }
  }
  // ---- the rows' sums
  // Two warpgroups take a panel of 64 columns at a time: 32 columns a thread,
  // rounded, into the first operand's ring (every product is done) in the
  // swizzle of its tensor map, then one TMA store, which leaves out rows past
  // N_valid.  (16-byte stores from the threads' rows took 5,200 cycles for dk and
  // dv of d = 128.)
  constexpr int PANELS = (KEYS ? 2 : 1) * (D / 64);
  const int pr = wg >> 1;
  float off_zero = 0.f, mean[32];
  if (!KEYS) {
    RowParts* m = reinterpret_cast<RowParts*>(smem + L::OFF_R1);
    m->sum[wg][row] = ds_sum[0] + ds_sum[1];
    m->top[wg][row] = top;
    m->at[wg][row] = top_at;
    named_bar_sync(4, kGroups * 128);
    top = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      off_zero += m->sum[i][row];
      if (m->top[i][row] > top) {
        top = m->top[i][row];
        top_at = m->at[i][row];
      }
    }
    // on their way while the last products run
    if (pr < PANELS) {
      const int at = pr * 64 + (wg & 1) * 32;
      if (top_at >= 0) {
        const float4* src = reinterpret_cast<const float4*>(a.k_means + (t.bh * (a.Npad / 64) + top_at) * D + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 x = src[j];
          mean[4 * j] = x.x;
          mean[4 * j + 1] = x.y;
          mean[4 * j + 2] = x.z;
          mean[4 * j + 3] = x.w;
        }
      } else {
        const GradStride& st = a.st[kK];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + t.b * st.b + t.h * st.h +
                                                          ~top_at * st.n + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 x = __ldg(src + j);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mean[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
            mean[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        }
      }
    }
  }
  bool sums = alive && t.n_steps > 0;
  if (sums) {
    sums = warp_wait(bars.drain, 0, wl, a.status, abort_flag);
    tc_fence_after();
  }
  for (int i = pr; i < PANELS; i += 2) {
    const int acc = i / (D / 64), c64 = (i % (D / 64)) * 64;
    const float f = KEYS && acc == 1 ? 1.f : scale;
    uint32_t o[32];
    if (sums) {
      tmem_ld32(t_lane + (acc == 1 ? L::ACC2 : L::ACC1) + c64 + (wg & 1) * 32, o);
      tmem_wait_ld_dep(o);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = 0u;
    }
    if (!KEYS && sums) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(fmaf(-off_zero, mean[j], __uint_as_float(o[j])));
    }
    uint8_t* panel = smem + L::OFF_C1 + i * BM * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t pk[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        pk[e] = pack_bf16x2(__uint_as_float(o[8 * j + 2 * e]) * f, __uint_as_float(o[8 * j + 2 * e + 1]) * f);
      *reinterpret_cast<uint4*>(panel + row * 128 + ((((wg & 1) * 4 + j) ^ (row & 7)) << 4)) =
          make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    fence_proxy_async_smem();
    named_bar_sync(2 + pr, 256);
    if ((threadIdx.x & 255) == 0) {
      tma_store_4d(acc == 1 ? out2 : out1, panel, c64, t.tile * BM, t.h, t.b);
      tma_store_commit();
    }
  }
  if ((threadIdx.x & 255) == 0) tma_store_wait_read<0>();
}

template <int D, bool KEYS, bool MASKED>
__device__ __forceinline__ void run_tile(uint8_t* smem, const CUtensorMap* tq, const CUtensorMap* tk,
                                         const CUtensorMap* tv, const CUtensorMap* tdo, const CUtensorMap* out1,
                                         const CUtensorMap* out2, const AttendGradArgs& a, int tile, float scale_log2,
                                         float scale) {
  using L = Layout<D, KEYS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Bars bars = make_bars(smem + L::OFF_BAR);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  uint32_t* entries = misc + 4;
  if (threadIdx.x == 0) {
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    for (int i = 0; i < kBars; ++i) mbar_init(b + i, i >= kWarpBars || (i == 0 && !KEYS) ? kGroups * 4 : (i == kSFull || i == kSFull + 1) ? 2 : 1);   // 0: r_full
    misc[1] = 0;
    misc[2] = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(misc, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  Tile t;
  t.tile = tile;
  t.h = blockIdx.y;
  t.b = KEYS ? blockIdx.z : blockIdx.z - a.B;
  t.n_steps = 0;
  t.bh = static_cast<long long>(t.b) * a.H + t.h;
  // the tile's own rows do not depend on the tables: they are on their way while
  // the tables are waited for and the lists counted
  if (KEYS) {
    if (threadIdx.x == kProducer * 32) {
      mbar_arrive_expect_tx(bars.r_full, 2 * L::TILE);
      for (int p = 0; p < 2; ++p) {
        load_rows<D>(smem + L::OFF_R1, tk, bars.r_full, p, tile * 2 + p, t);
        load_rows<D>(smem + L::OFF_R2, tv, bars.r_full, p, tile * 2 + p, t);
      }
    }
  } else if (warp < kProducer) {
    own_rows<D>(bars, tmem, a, t);
  }
  grid_wait();
  // the tile's kept pieces: the set bits of its blocks' rows, one row for 128-token blocks
  const int shift = a.block == 128 ? 1 : 0, W = (a.nB + 31) >> 5;
  const uint32_t* rows = KEYS ? a.bits_t : a.bits;
  const int first = shift ? tile : 2 * tile;
  const uint32_t* row0 = rows + (t.bh * a.nB + first) * W;
  const uint32_t* row1 = !shift && first + 1 < a.nB ? row0 + W : nullptr;
  if (warp == kProducer) {
    // finds the end of the list itself: the first copies start while the others count
    if (lane == 0) {
      Walk walk;
      walk.init(row0, row1, W, shift, a.N_valid);
      if (KEYS) produce<D, KEYS, MASKED>(smem, bars, tq, tdo, a, t, walk, entries, abort_flag);
      else produce<D, KEYS, MASKED>(smem, bars, tk, tv, a, t, walk, entries, abort_flag);
    }
  } else {
    if (threadIdx.x < 128) {
      int n = 0;
      for (int w = threadIdx.x; w < W; w += 128) n += __popc(row0[w] | (row1 ? row1[w] : 0u));
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0 && n) atomicAdd(misc + 2, static_cast<uint32_t>(n));
    }
    named_bar_sync(1, kThreads - 32);
    t.n_steps = ((static_cast<int>(misc[2]) << shift) + 1) >> 1;
    if (warp == kIssuer) issue<D, KEYS>(smem, bars, tmem, a, t.n_steps, abort_flag);
    else softmax<D, KEYS, MASKED>(smem, bars, tmem, a, t, entries, out1, out2, scale_log2, scale, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool MASKED>
__global__ void __launch_bounds__(kThreads, 1)
attend_grad_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                      const __grid_constant__ CUtensorMap tdq, const __grid_constant__ CUtensorMap tdk,
                      const __grid_constant__ CUtensorMap tdv, const __grid_constant__ AttendGradArgs a, float scale_log2,
                      float scale) {
  extern __shared__ __align__(1024) uint8_t smem[];
  // a CTA already gave up on a wait: skip the work, the call has failed
  if (*reinterpret_cast<volatile int32_t*>(a.status) == LBSA_ERR_TIMEOUT) return;
  // keys first, all heads: the shorter tiles of the queries fill the last wave
  if (static_cast<int>(blockIdx.z) < a.B) run_tile<D, true, MASKED>(smem, &tq, &tk, &tv, &tdo, &tdk, &tdv, a, blockIdx.x, scale_log2, scale);
  else run_tile<D, false, MASKED>(smem, &tq, &tk, &tv, &tdo, &tdq, nullptr, a, blockIdx.x, scale_log2, scale);
}

}  // namespace

cudaError_t launch_attend_grad_tc(const CUtensorMap* in, const CUtensorMap* out, const AttendGradArgs& a, cudaStream_t s) {
  const int tiles = (a.N_valid + BM - 1) / BM;
  const double scale = 1.0 / std::sqrt(static_cast<double>(a.d));
  auto go = [&](auto kern, int smem) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(tiles, a.H, 2 * a.B), dim3(kThreads), smem, s, in[0], in[1], in[2], in[3], out[0], out[1], out[2], a,
                            static_cast<float>(1.4426950408889634 * scale), static_cast<float>(scale));
  };
  if (a.d == 128)
    return a.masks ? go(attend_grad_tc_kernel<128, true>, kSmemBytes<128>)
                   : go(attend_grad_tc_kernel<128, false>, kSmemBytes<128>);
  return a.masks ? go(attend_grad_tc_kernel<64, true>, kSmemBytes<64>)
                 : go(attend_grad_tc_kernel<64, false>, kSmemBytes<64>);
}

}  // namespace lbsa
