// Gradient of the PR-Sink attention with respect to its raw queries, raw keys and values.
//
//   P = exp(s - lse),  delta_i = sum_c d_out_ic out_ic,  dP = d_out V^T,
//   dS = P o (dP - delta) / sqrt(d),  dV = P^T d_out,  dK = R^T (dS^T q~),  dQ = R^T (dS k~)
//
// with q~, k~ the rotated queries and keys and R^T the inverse rotation of the row's position.
//
// What is held in bf16, and why: the operands of the tensor core, which have one type (V and d_out
// come in bf16): q~ and k~ (once, as the forward's), P for dV, dS for dK and dQ; `out` inside delta, as
// the forward stored it.  Scores, P and dP - delta before those roundings, delta and every sum are
// f32.  The roundings are independent and average out: dq and dk are off by 3.8-4.4e-3 in the 2-norm,
// dv by 3.5e-3, of which the rounding of the results is 1.7e-3.  Wider operands (tf32) would double
// every tile in shared memory and halve the tensor rate, and both bound the pass.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "prsink_internal.cuh"

namespace prsink {
namespace bwd {

constexpr int kMaxSlots = 3 + PRSINK_MAX_RING;
constexpr int BM = 128;                    // rows of a tile (= TMEM lanes); statistics are padded
constexpr int kMaxTiles = 1024;            // key tiles per call, as in the forward

struct Params {
  int H, L_blk, L_pad, T, L_f, grid_w;
  int n_slots;
  int slot_start[kMaxSlots + 1];
  int slot_frame[kMaxSlots];
  unsigned valid_mask, grad_mask;
  int prep_heads;                          // heads of a CTA of the preparation
  int q_row;                               // first row of the current block's ring slot
  int rope_mode;
  int rd[3];                               // rotated pairs per axis
  double inv_pi_freq[64];                  // base^(-2j/d_axis) / pi of every pair
  float scale, scale_log2;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* out;
  const __nv_bfloat16* d_out;
  const float* lse;
  const long long* dyn_src;
  int* status;
  unsigned long long timeout_ns;
  int debug_stall;                         // self-test: withhold the first commit of S
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  // scratch
  __nv_bfloat16* k_rot;                    // [H][T][d], rows of empty slots zero
  __nv_bfloat16* q_rot;                    // [H][L_blk][d]
  float2* tab;                             // [T][d/2] (cos, sin) of every key row's position
  float* nlse;                             // [H][L_pad] -lse in log2 units; -inf: no probability
  float* ndelta;                           // [H][L_pad] -delta
};

__device__ __forceinline__ int slot_of(int row, const Params& p) {
  int s = 0;
  while (s + 1 < p.n_slots && row >= p.slot_start[s + 1]) ++s;
  return s;
}
__device__ __forceinline__ unsigned live_mask(const Params& p) {
  unsigned m = p.valid_mask;
  if (p.dyn_src && *p.dyn_src < 0) m &= ~(1u << PRSINK_SLOT_DYNAMIC);
  return m;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Rotate (dir = 1) or rotate back (dir = -1) the pair (x0, x1).
__device__ __forceinline__ float2 turn(float x0, float x1, float2 cs, float dir) {
  const float s = cs.y * dir;
  return make_float2(x0 * cs.x - x1 * s, x0 * s + x1 * cs.x);
}

// Keys rotated into k_rot (rows of empty slots zeroed: dS is 0 there, but 0 * NaN is not), the
// table of their cos / sin, queries rotated into q_rot (head-major) and the queries' statistics.
// HBM-bound.  A CTA takes 256 / C rows and prep_heads heads, a thread one 16-byte chunk of a row,
// whose four f64 angles serve all of them.
template <int D>
__global__ void __launch_bounds__(256) prep_kernel(const __grid_constant__ Params p) {
  constexpr int C = D / 8, R = 256 / C;
  const int c = threadIdx.x % C;
  const int key_blocks = (p.T + R - 1) / R;
  const bool keys = static_cast<int>(blockIdx.x) < key_blocks;
  const int i = (keys ? blockIdx.x : blockIdx.x - key_blocks) * R + threadIdx.x / C;
  const int h0 = blockIdx.y * p.prep_heads, h1 = min(p.H, h0 + p.prep_heads);
  const int row = keys ? i : p.q_row + i;    // the queries sit on the current block's positions
  const bool in = keys ? i < p.T : i < p.L_blk;
  grid_dependency_wait();
  grid_launch_dependents();
  bool live = false;
  float2 cs[4];
  if (in) {
    const int s = slot_of(row, p), u = row - p.slot_start[s];
    live = !keys || ((live_mask(p) >> s) & 1u);
    const int frame = p.slot_frame[s] + u / p.L_f, tok = u % p.L_f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = 4 * c + e;
      int x;
      if (p.rope_mode == 3)
        x = j < p.rd[0] ? frame : (j < p.rd[0] + p.rd[1] ? tok / p.grid_w : tok % p.grid_w);
      else
        x = frame * p.L_f + tok;
      double sn, co;
      sincospi(static_cast<double>(x) * p.inv_pi_freq[j], &sn, &co);
      cs[e] = make_float2(static_cast<float>(co), static_cast<float>(sn));
      if (keys && blockIdx.y == 0) p.tab[static_cast<size_t>(row) * (D / 2) + j] = cs[e];
    }
  }
  auto rotate = [&](uint4& x) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = turn(lo16(w[e]), hi16(w[e]), cs[e], 1.f);
      w[e] = pack2(y.x, y.y);
    }
  };
  if (keys) {
    if (!in) return;
    const size_t step = static_cast<size_t>(p.T) * C;
    const size_t at = static_cast<size_t>(row) * C + c;
#pragma unroll 5
    for (int h = h0; h < h1; ++h) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (live) {
        x = __ldcs(reinterpret_cast<const uint4*>(p.k) + at + h * step);
        rotate(x);
      }
      reinterpret_cast<uint4*>(p.k_rot)[at + h * step] = x;
    }
    return;
  }
#pragma unroll 2
  for (int h = h0; h < h1; ++h) {
    float dot = 0.f;
    if (in) {
      const size_t at = (static_cast<size_t>(i) * p.H + h) * C + c;
      uint4 x = reinterpret_cast<const uint4*>(p.q)[at];
      const uint4 o = reinterpret_cast<const uint4*>(p.out)[at];
      const uint4 g = reinterpret_cast<const uint4*>(p.d_out)[at];
      const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) dot += lo16(ow[e]) * lo16(gw[e]) + hi16(ow[e]) * hi16(gw[e]);
      rotate(x);
      reinterpret_cast<uint4*>(p.q_rot)[(static_cast<size_t>(h) * p.L_blk + i) * C + c] = x;
    }
#pragma unroll
    for (int o = C / 2; o; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
    if (c == 0 && i < p.L_pad) {
      float l = -INFINITY;                             // padding, or a row without keys
      if (in) {
        l = p.lse[static_cast<size_t>(h) * p.L_blk + i] * -1.4426950408889634f;
        if (l == INFINITY) l = -INFINITY;
      }
      p.nlse[static_cast<size_t>(h) * p.L_pad + i] = l;
      p.ndelta[static_cast<size_t>(h) * p.L_pad + i] = -dot;
    }
  }
}

// -------------------------------------------------------------------------------- the products
// One kernel for both sides.  A CTA owns 128 rows (its two operand tiles A1, A2 stay in shared
// memory, its sums in tensor memory) and streams the other side's tiles Y1, Y2 past them:
//                rows     A1  A2     Y1  Y2     S = A1 Y1^T   dP = A2 Y2^T   sums
//   kKeys        keys     k~  v      q~  d_out  S^T           dP^T           dV += P Y2, dK += dS Y1
//   otherwise    queries  q~  d_out  k~  v      S             dP                         dQ += dS Y1
// so that P and dS come out as [own rows][streamed rows], which is what the A operand of the sums
// wants: they go back to tensor memory as bf16 in the place of the scores they came from and
// never touch shared memory.  Seven products of 128 x 128 x d per pair of tiles instead of the
// five that one pass would need, but no sum crosses a CTA: a fused pass would have to add 64 KB
// of float32 dQ to global memory per pair, in an order that changes from run to run.
//
// Warps 0-7 turn S into P and dP into dS (row = lane, a half of the streamed rows each: 32 of
// every 64 on the keys' side, 64 in one piece on the queries', see `col`), warp 8
// sends the tiles (Y1 through three stages, since both S and the sum read it; Y2 through two),
// warp 9 issues the MMAs:
//   kKeys      dV(j) in two halves, S(j+1)  |  dK(j)  dP(j+1)
//   otherwise  S(j+1)  dP(j+1)              |  dQ(j)              (two buffers of dP)
// Every wait or commit of the issuing thread costs the tensor pipe about 100 cycles (it runs only
// a few MMAs ahead), so there are few of them: a gate opens when the warps have done their part
// (P(j) written, S(j) read, dS(j) written) AND the tiles that the next products read have landed
// (the warps' arrivals and the TMA's bytes count on one barrier), and the stages are given back
// by commits that are there anyway.
//
// Measured on a B200 at 480x480 (40 heads, 128-wide, 2700 x 14400): keys' side 3150 cycles per pair
// of tiles (2048 of MMAs at 64 each): the products from shared memory run at about 85 cycles per
// MMA beside the TMA writes (they take all of its 128 B per cycle), and the issuing thread's waits
// add 350; queries' side 2280 (1536), bound by the conversion warps (1140 cycles of exponentials
// at 16 per cycle, 640 for dS).  2.3 ms the first time, 2.7 ms in a loop at the 1 kW cap.  Slower
// or not worth it, measured: two issuing threads (+15 %), a quarter to three quarters of the
// exponentials as polynomials (+1 to +5 %), dS written out and dQ as a plain product of it (-6 %
// at this size for 3.3 GB of scratch, +15 % at 13x17).
constexpr int kThreads = 320;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
constexpr int kY1 = 3, kY2 = 2;            // stages

// GATE1[tile % 3]  Y1 of the tile has landed; the warps have written all of P of the tile before
//                  it (keys) / read its S, and Y2 has landed as well (queries)
// PHALF            the warps have written the first half of P (keys)
// GATE2[tile % 2]  Y2 of the tile has landed (keys); dS of the tile before it is written
// SFULL, DPFULL[tile % 2]  the product is done (keys: SFULL[0] alone)
enum Bar {
  B_A = 0, B_GATE1 = 1, B_GATE2 = B_GATE1 + kY1, B_PHALF = B_GATE2 + kY2, B_SFULL,
  B_DPFULL = B_SFULL + 2, B_SUM = B_DPFULL + 2, B_TAB, B_FINAL, B_COUNT
};

template <int D>
struct Smem {
  static constexpr int kTile = (D / 64) * 16384;         // 128 rows in 128-byte swizzled panels
  static constexpr int kA1 = 0, kA2 = kTile;
  static constexpr int kStage1 = 2 * kTile, kStage2 = kStage1 + kY1 * kTile;
  // statistics of the streamed queries (kKeys: lse per Y1 stage, delta per Y2 stage), or the list
  // of live key tiles (otherwise)
  static constexpr int kStat = kStage2 + kY2 * kTile;
  static constexpr int kStatBytes = (kY1 + kY2) * BM * 4;
  static constexpr int kBars = kStat + kStatBytes;
  static constexpr int kTail = kBars + B_COUNT * 8;
  // what becomes of the tile's rows at the end: memory of its own, since copies of the statistics
  // may still be on their way when a wait has given up, and a row's fate decides whether it is
  // written (rows past the end among them)
  static constexpr int kFate = kTail + 32;
  static constexpr int kBytes = kFate + BM;
  static constexpr uint32_t kIdescSum = idesc_bf16_f32(128, D, false, true);
  static_assert(kMaxTiles * 2 <= kStatBytes, "tile list");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct Tail {                              // what follows the barriers in shared memory
  uint32_t tmem;
  AbortState ab;
  int n_live, y1, y2, tab;                 // live tiles; tiles sent (for the drain)
};

// D (+)= A B over 64 streamed rows: A as bf16 pairs in tensor memory (8 columns per 16 rows), B
// MN-major in shared memory (2 KB per 16 rows).
__device__ __forceinline__ void umma_sum64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "setp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 p1, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p1;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p1;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p1;\n\t}"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// D = A B^T over the head dimension, both K-major.
template <int D>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
  if constexpr (D == 128) umma_ss_k128(d, a, b, idesc);
  else umma_ss_k64(d, a, b, idesc);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ float4 lds4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;"
               :: "r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 lds4u(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
               :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t dl = globaltimer() + 5000000ull;
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() > dl) break;
}

// Bits 0 / 1 of a key tile: it holds a row of a live slot / also rows that are not live.
__device__ __forceinline__ int tile_flags(int n, unsigned vm, const Params& p) {
  const int lo = n * BM, hi = lo + BM, end = min(hi, p.T);
  bool live = false, full = hi <= p.T;
  for (int s = 0; s < p.n_slots; ++s) {
    const bool in = p.slot_start[s] < end && p.slot_start[s + 1] > lo;
    if ((vm >> s) & 1u) live |= in;
    else full &= !in;
  }
  return (live ? 1 : 0) | (full ? 0 : 2);
}

// W finished sums of this thread's row (tensor memory) -> bf16 in a staged tile (row t, elements
// from e0 on, 128-byte swizzle), rotated back by the row's cos / sin in `tab` (a tile of 2 D-byte
// rows in 128-byte panels of two halves; 0: as they are).
template <int D>
__device__ __forceinline__ void stage_row(uint32_t taddr, uint32_t dst, int t, int e0,
                                          uint32_t tab0, uint32_t tab1, float scale) {
  constexpr int W = D / 2;
#pragma unroll 1
  for (int c = 0; c < W; c += 32) {
    uint32_t a[32];
    tmem_ld32(taddr + c, a);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int pair = (e0 + c + i) / 2 + e;           // even: 16 bytes hold this pair and the next
        float4 cs = make_float4(1.f, 0.f, 1.f, 0.f);
        if (tab0) {
          // panel of 16 pairs; the first half of the panels is in tab0, the other in tab1
          const int panel = pair >> 4, half = panel / (D / 64), chunk = (pair & 15) >> 1;
          cs = lds4((half ? tab1 : tab0) + (panel % (D / 64)) * 16384 + t * 128 +
                    ((chunk ^ (t & 7)) << 4));
        }
        const float x0 = __uint_as_float(a[i + 2 * e]) * scale;
        const float x1 = __uint_as_float(a[i + 2 * e + 1]) * scale;
        const float x2 = __uint_as_float(a[i + 2 * e + 2]) * scale;
        const float x3 = __uint_as_float(a[i + 2 * e + 3]) * scale;
        const float2 y0 = turn(x0, x1, make_float2(cs.x, cs.y), -1.f);
        const float2 y1 = turn(x2, x3, make_float2(cs.z, cs.w), -1.f);
        w[e] = tab0 ? pack2(y0.x, y0.y) : pack2(x0, x1);
        w[e + 1] = tab0 ? pack2(y1.x, y1.y) : pack2(x2, x3);
      }
      const int k = (e0 + c + i) >> 3;                   // 16-byte chunk of the row
      sts4(dst + (k >> 3) * 16384 + t * 128 + (((k & 7) ^ (t & 7)) << 4),
           make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

// One CTA's rows: tile `tile` of head h.
template <int D, bool kKeys>
__device__ __forceinline__ void run_rows(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                         const CUtensorMap& tm_v, const CUtensorMap& tm_g,
                                         const CUtensorMap& tm_t, const Params& p, int h,
                                         int tile, uint8_t* smem) {
  using SM = Smem<D>;
  constexpr uint32_t kColS = 0, kColDP = 128;
  constexpr uint32_t kColDV = 256, kColSum = kKeys ? 256 + D : 384;
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = tile * BM;
  auto bar = [&](int i) { return sb + SM::kBars + i * 8; };
  auto tab_stage = [&](int j) { return sb + SM::kStage1 + (j % kY1) * SM::kTile; };
  Tail* tail = reinterpret_cast<Tail*>(smem + SM::kTail);
  static_assert(sizeof(Tail) <= SM::kFate - SM::kTail, "tail");
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + SM::kStat);      // (queries only)
  const unsigned vm = live_mask(p);
  if (sb & 1023u) {                                  // (the swizzle needs 1 KB atoms; no static
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);    // memory moves the base)
    return;
  }

  if (kKeys) {
    // key rows that need no gradient, or get zeros
    if (!(tile_flags(tile, p.grad_mask, p) & 1)) return;
    if (!(tile_flags(tile, vm, p) & 1)) {
      for (int i = threadIdx.x; i < BM * (D / 8); i += kThreads) {
        const int r = row0 + i / (D / 8);
        if (r >= p.T || !((p.grad_mask >> slot_of(r, p)) & 1u)) continue;
        const size_t at = (static_cast<size_t>(h) * p.T + r) * (D / 8) + i % (D / 8);
        reinterpret_cast<uint4*>(p.dk)[at] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(p.dv)[at] = make_uint4(0, 0, 0, 0);
      }
      return;
    }
  }
  // rows r.. of the rotated queries, the keys, the values (head-major) or d_out (token-major)
  auto load = [&](int which, uint32_t dst, uint32_t b, int r) {
    const CUtensorMap* tm = which == 0 ? &tm_q : which == 1 ? &tm_k : which == 2 ? &tm_v : &tm_g;
    for (int pp = 0; pp < D / 64; ++pp)
      tma_load_3d(dst + pp * 16384, tm, b, pp * 64, which == 3 ? h : r, which == 3 ? r : h);
  };
  if (threadIdx.x == kProducerWarp * 32) {
    mbar_init(bar(B_A), 1);
    for (int i = 0; i < kY1; ++i) mbar_init(bar(B_GATE1 + i), 257);
    for (int i = 0; i < kY2; ++i) {
      mbar_init(bar(B_GATE2 + i), kKeys ? 257 : 256);
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_DPFULL + i), 1);
    }
    mbar_init(bar(B_PHALF), 256);
    mbar_init(bar(B_SUM), 1);
    mbar_init(bar(B_TAB), 1);
    mbar_init(bar(B_FINAL), 1);
    tail->ab.flag = 0;
    tail->y1 = tail->y2 = tail->tab = 0;
    fence_barrier_init();
    // the CTA's own rows need nothing else
    mbar_arrive_expect_tx(bar(B_A), 2 * SM::kTile);
    load(kKeys ? 1 : 0, sb + SM::kA1, bar(B_A), row0);
    load(kKeys ? 2 : 3, sb + SM::kA2, bar(B_A), row0);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&tail->tmem), 512);
    tmem_relinquish();
  }
  if (!kKeys && warp == 0) {
    // the key tiles that hold a live row, in order; bit 15: some of their rows are not live
    const int n_tiles = (p.T + BM - 1) / BM;
    int base = 0;
    for (int n0 = 0; n0 < n_tiles; n0 += 32) {
      const int f = n0 + lane < n_tiles ? tile_flags(n0 + lane, vm, p) : 0;
      const uint32_t bal = __ballot_sync(~0u, f & 1);
      if (f & 1)
        list[base + __popc(bal & ((1u << lane) - 1u))] =
            static_cast<uint16_t>((n0 + lane) | ((f & 2) ? 0x8000 : 0));
      base += __popc(bal);
    }
    if (lane == 0) tail->n_live = base;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail->tmem;
  AbortState* ab = &tail->ab;
  const int n = kKeys ? p.L_pad / BM : tail->n_live;     // streamed tiles
  const uint64_t deadline = globaltimer() + p.timeout_ns;

  if (warp == kProducerWarp) {
    if (lane == 0 && n == 0) mbar_wait(bar(B_A), 0, ab, deadline, p.status);   // (no reader)
    if (lane == 0 && n > 0) {
      constexpr uint32_t stat = kKeys ? BM * 4 : 0;
      const float* nlse = p.nlse + static_cast<size_t>(h) * p.L_pad;
      const float* ndelta = p.ndelta + static_cast<size_t>(h) * p.L_pad;
      // Stages: Y1(j) takes the one of tile j - 3, Y2(j) that of tile j - 2.
      //   keys     dP(j - 1) is issued after dK(j - 2) and dV(j - 2), and frees both; Y1 a step
      //            ahead.  One step past the last tile opens the gates behind it without a copy.
      //   queries  dP(j - 2) frees Y2's, S(j - 1), issued after dQ(j - 3), frees Y1's.
      // (A parity wait is only sound for a barrier's next phase: with one barrier for the even and
      // one for the odd tiles, the phase after the one waited for needs a tile not yet sent.)
      bool ok = true;
      auto dp_done = [&](int j) {
        return mbar_wait(bar(B_DPFULL + (j & 1)), (j >> 1) & 1, ab, deadline, p.status);
      };
      for (int j = 0; j <= n; ++j) {
        const int r = j == n ? 0 : (kKeys ? j : list[j] & 0x7FFF) * BM;
        const uint32_t g1 = bar(B_GATE1 + j % kY1), g2 = bar(B_GATE2 + j % kY2);
        const uint32_t to1 = sb + SM::kStage1 + (j % kY1) * SM::kTile;
        const uint32_t to2 = sb + SM::kStage2 + (j % kY2) * SM::kTile;
        if (kKeys) {
          if (j == n) {
            mbar_arrive(g1);
          } else {
            mbar_arrive_expect_tx(g1, SM::kTile + stat);
            load(0, to1, g1, r);
            bulk_load(sb + SM::kStat + (j % kY1) * stat, nlse + r, stat, g1);
            tail->y1 = j + 1;
          }
          if (j >= kY2) ok = dp_done(j - 1);
          if (!ok) break;
          if (j == n) {
            mbar_arrive(g2);
          } else {
            mbar_arrive_expect_tx(g2, SM::kTile + stat);
            load(3, to2, g2, r);
            bulk_load(sb + SM::kStat + (kY1 + j % kY2) * stat, ndelta + r, stat, g2);
            tail->y2 = j + 1;
          }
        } else if (j < n) {
          if (j >= kY2) ok = dp_done(j - 2);
          if (!ok) break;
          mbar_expect_tx(g1, SM::kTile);
          load(2, to2, g1, r);
          tail->y2 = j + 1;
          if (j >= kY1)
            ok = mbar_wait(bar(B_SFULL + ((j - 1) & 1)), ((j - 1) >> 1) & 1, ab, deadline,
                           p.status);
          if (!ok) break;
          mbar_arrive_expect_tx(g1, SM::kTile);
          load(1, to1, g1, r);
          tail->y1 = j + 1;
        }
      }
      if (ok) {
        // the rows' cos / sin, for the end, into the two Y1 stages that the last tile does not
        // use (the sum of the tile before it, which read the younger of them, is done: keys when
        // dP(n - 1) is, queries at the end)
        if (kKeys) ok = n >= kY2 || dp_done(0);
        else ok = mbar_wait(bar(B_SUM), 0, ab, deadline, p.status);
        if (ok) {
          const int r = kKeys ? row0 : p.q_row + row0;
          mbar_arrive_expect_tx(bar(B_TAB), 2 * SM::kTile);
          for (int pp = 0; pp < D / 32; ++pp)
            tma_load_3d(tab_stage(n + pp / (D / 64)) + (pp % (D / 64)) * 16384, &tm_t, bar(B_TAB),
                        pp * 64, r, 0);
          tail->tab = 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0 && n > 0) {
      bool ok = mbar_wait(bar(B_A), 0, ab, deadline, p.status);
      constexpr uint32_t step = SM::kTile >> 4;        // of a stage, in descriptor units
      const uint64_t a1 = sdesc_sw128(sb + SM::kA1, 16, 1024), a2 = sdesc_sw128(sb + SM::kA2, 16, 1024);
      const uint64_t k1 = sdesc_sw128(sb + SM::kStage1, 16, 1024);       // K-major: S, dP
      const uint64_t k2 = sdesc_sw128(sb + SM::kStage2, 16, 1024);
      const uint64_t m1 = sdesc_sw128(sb + SM::kStage1, 16384, 1024);    // MN-major: the sums
      const uint64_t m2 = sdesc_sw128(sb + SM::kStage2, 16384, 1024);
      // Y1 stage and its gate's parity of tile j + 1, Y1 stage of tile j
      int s1 = 0, c1 = 0;
      uint32_t par = 0;
      auto gate1 = [&]() { return mbar_wait(bar(B_GATE1 + s1), par, ab, deadline, p.status); };
      auto next = [&]() {
        c1 = s1;
        if (++s1 == kY1) {
          s1 = 0;
          par ^= 1;
        }
      };
      auto score = [&](int j) {
        product<D>(tmem + kColS, a1, k1 + s1 * step);
        if (!(p.debug_stall && j == 0)) umma_commit(bar(B_SFULL + (kKeys ? 0 : j & 1)));
      };
      auto dprob = [&](int j) {
        product<D>(tmem + kColDP + (kKeys ? 0 : (j & 1) * 128), a2, k2 + (j & 1) * step);
        umma_commit(bar(B_DPFULL + (j & 1)));
      };
      ok = ok && gate1();
      if (ok) {
        tc_fence_after();
        score(0);
        next();
        if (kKeys) {
          ok = mbar_wait(bar(B_GATE2), 0, ab, deadline, p.status);
          tc_fence_after();
        }
        if (ok) dprob(0);
      }
      for (int j = 0; ok && j < n; ++j) {
        const int cur = c1;                            // Y1 stage of tile j
        if (kKeys) {
          const uint64_t y2 = m2 + (j & 1) * step;
          ok = mbar_wait(bar(B_PHALF), j & 1, ab, deadline, p.status);
          if (!ok) break;
          tc_fence_after();
          umma_sum64(tmem + kColDV, tmem + kColS, y2, SM::kIdescSum, j > 0);
          ok = gate1();
          if (!ok) break;
          tc_fence_after();
          umma_sum64(tmem + kColDV, tmem + kColS + 64, y2 + 512, SM::kIdescSum, 1);
          if (j + 1 < n) score(j + 1);
          next();
          ok = mbar_wait(bar(B_GATE2 + ((j + 1) & 1)), ((j + 1) >> 1) & 1, ab, deadline, p.status);
        } else {
          if (j + 1 < n) {
            ok = gate1();
            if (!ok) break;
            tc_fence_after();
            score(j + 1);
            next();
            dprob(j + 1);
          }
          ok = mbar_wait(bar(B_GATE2 + (j & 1)), (j >> 1) & 1, ab, deadline, p.status);
        }
        if (!ok) break;
        tc_fence_after();
        const uint32_t ds = tmem + kColDP + (kKeys ? 0 : (j & 1) * 128);
        umma_sum64(tmem + kColSum, ds, m1 + cur * step, SM::kIdescSum, j > 0);
        umma_sum64(tmem + kColSum, ds + 64, m1 + cur * step + 512, SM::kIdescSum, 1);
        if (kKeys && j + 1 < n) dprob(j + 1);
      }
      if (ok) umma_commit(bar(B_SUM));
    }
    __syncwarp();
  } else {
    // Columns of a thread, in two parts of 32.  Keys: one of the streamed rows 0-63 and one of
    // 64-127, so that the first half of P is ready early; P and dS go, as bf16 pairs, into the
    // first 32 columns of each 64, and the two warps that share the lanes meet before that, since
    // each writes where the other has read.  Queries: 64 columns of its own.
    const int half = warp >> 2;
    const int row = row0 + (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + kColS;
    const uint32_t col[2] = {kKeys ? half * 32u : half * 64u, kKeys ? 64u + half * 32u : half * 64u + 32u};
    const uint32_t packed[2] = {kKeys ? half * 16u : half * 64u, kKeys ? 64u + half * 16u : half * 64u + 16u};
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    float2 nlse = make_float2(0.f, 0.f), ndelta = nlse;    // queries: this row's
    if (!kKeys) {
      const size_t at = static_cast<size_t>(h) * p.L_pad + row;
      nlse.x = nlse.y = __ldcg(p.nlse + at);
      ndelta.x = ndelta.y = __ldcg(p.ndelta + at);
    }
    bool ok = true;
    if (n > 0) {                                     // nothing comes before the first tile
      mbar_arrive(bar(B_GATE1));
      if (kKeys) mbar_arrive(bar(B_GATE2));
    }
    int s1 = 0;                                      // j % 3
    uint32_t par1 = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t gate1 = bar(B_GATE1 + s1), stat1 = sb + SM::kStat + s1 * (BM * 4) + half * 128;
      const uint32_t gate1_par = par1;
      if (++s1 == kY1) {
        s1 = 0;
        par1 ^= 1;
      }
      const uint32_t next1 = bar(B_GATE1 + s1);
      const uint32_t done2 = bar(B_GATE2 + ((kKeys ? j + 1 : j) & 1));
      ok = mbar_wait(bar(B_SFULL + (kKeys ? 0 : j & 1)), (kKeys ? j : j >> 1) & 1, ab, deadline,
                     p.status);
      if (kKeys)                                     // (open: it let S(j) start; for lse)
        ok = ok && mbar_wait(gate1, gate1_par, ab, deadline, p.status);
      __syncwarp();
      tc_fence_after();
      uint32_t s[64];
      tmem_ld32(t_s + col[0], *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
      tmem_ld32(t_s + col[1], *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
      tmem_wait_ld();
      if (!kKeys) {
        tc_fence_before();
        mbar_arrive(next1);
      }
      // (a wait that gave up in one of the two warps ends the loop for both)
      ok = kKeys ? named_bar_and(2 + (warp & 3), 64, ok) : __all_sync(~0u, ok);
      if (!ok) break;
      float2 pr[32];
#pragma unroll
      for (int part = 0; part < 2; ++part) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const int c = part * 32 + i;
          float2 l0 = nlse, l1 = nlse;
          if (kKeys) {
            const float4 l = lds4(stat1 + part * 256 + i * 4);
            l0 = make_float2(l.x, l.y);
            l1 = make_float2(l.z, l.w);
          }
          const float2 e0 = ffma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                  scale2, l0);
          const float2 e1 = ffma2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                                  scale2, l1);
          pr[c / 2] = make_float2(ex2(e0.x), ex2(e0.y));
          pr[c / 2 + 1] = make_float2(ex2(e1.x), ex2(e1.y));
        }
        if (kKeys) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack2(pr[part * 16 + i].x, pr[part * 16 + i].y);
          tmem_st16(t_s + packed[part], pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(part == 0 ? bar(B_PHALF) : next1);
        }
      }
      ok = mbar_wait(bar(B_DPFULL + (j & 1)), (j >> 1) & 1, ab, deadline,
                     p.status);
      if (kKeys)                                     // (open likewise; for delta)
        ok = ok && mbar_wait(bar(B_GATE2 + (j & 1)), (j >> 1) & 1, ab, deadline, p.status);
      __syncwarp();
      tc_fence_after();
      const uint32_t t_dp = tmem + lane_off + kColDP + (kKeys ? 0 : (j & 1) * 128);
      tmem_ld32(t_dp + col[0], *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
      tmem_ld32(t_dp + col[1], *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
      tmem_wait_ld();
      // rows of the streamed tile that are not live (queries side): their keys' columns
      uint32_t mask[2] = {~0u, ~0u};
      if (!kKeys && (list[j] & 0x8000)) {
        const int lo = (list[j] & 0x7FFF) * BM + half * 64;
        for (int s2 = 0; s2 <= p.n_slots; ++s2) {
          if (s2 < p.n_slots && ((vm >> s2) & 1u)) continue;
          const int a = (s2 < p.n_slots ? p.slot_start[s2] : p.T) - lo;
          const int e = s2 < p.n_slots ? p.slot_start[s2 + 1] - lo : 64;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int cl = max(a, w * 32), ch = min(e, w * 32 + 32);
            if (cl < ch)
              mask[w] &= ~((ch - cl == 32 ? ~0u : ((1u << (ch - cl)) - 1u)) << (cl - w * 32));
          }
        }
      }
      const uint32_t stat2 = sb + SM::kStat + (kY1 + (j & 1)) * (BM * 4) + half * 128;
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        float2 d0 = ndelta, d1 = ndelta;
        if (kKeys) {
          const float4 d = lds4(stat2 + (c >> 5) * 256 + (c & 31) * 4);
          d0 = make_float2(d.x, d.y);
          d1 = make_float2(d.z, d.w);
        }
        const float2 x0 = fmul2(pr[c / 2], fadd2(make_float2(__uint_as_float(s[c]),
                                                             __uint_as_float(s[c + 1])), d0));
        const float2 x1 = fmul2(pr[c / 2 + 1], fadd2(make_float2(__uint_as_float(s[c + 2]),
                                                                 __uint_as_float(s[c + 3])), d1));
        pk[c / 2] = pack2(x0.x, x0.y);
        pk[c / 2 + 1] = pack2(x1.x, x1.y);
      }
      // (keys side: a row that is not live may hold anything, and spoils only its own sums)
      if (!kKeys && (mask[0] & mask[1]) != ~0u) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const uint32_t b = mask[c >> 4] >> (2 * (c & 15));
          pk[c] &= ((b & 1u) ? 0xFFFFu : 0u) | ((b & 2u) ? 0xFFFF0000u : 0u);
        }
      }
      ok = kKeys ? named_bar_and(2 + (warp & 3), 64, ok) : __all_sync(~0u, ok);
      if (!ok) break;
      tmem_st16(t_dp + packed[0], *reinterpret_cast<uint32_t(*)[16]>(&pk[0]));
      tmem_st16(t_dp + packed[1], *reinterpret_cast<uint32_t(*)[16]>(&pk[16]));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(done2);
    }
    // the rows' gradients: each half of the warps writes its half of the elements
    bool have = false;
    if (__all_sync(~0u, ok) && n > 0) {
      have = __all_sync(~0u, mbar_wait(bar(B_SUM), 0, ab, deadline, p.status));
      tc_fence_after();
    }
    // the sums rotated back (but for dV), rounded and staged in the Y2 stages, which are free now;
    // then whole rows leave, 2 D bytes at a time, where they are wanted
    const int t = (warp & 3) * 32 + lane;
    const uint32_t stage[2] = {sb + SM::kStage2, sb + SM::kStage2 + SM::kTile};
    if (have) {
      const bool tab = mbar_wait(bar(B_TAB), 0, ab, deadline, p.status);
      have = __all_sync(~0u, tab);
      stage_row<D>(tmem + lane_off + kColSum + half * (D / 2), stage[0], t, half * (D / 2),
                   tab_stage(n), tab_stage(n + 1), p.scale);
      if (kKeys)
        stage_row<D>(tmem + lane_off + kColDV + half * (D / 2), stage[1], t, half * (D / 2), 0, 0,
                     1.f);
    }
    // what becomes of the tile's rows: 0 nothing, 1 zeros, 2 the staged row
    uint8_t* fate = smem + SM::kFate;
    if (threadIdx.x < BM) {
      int f = row < p.L_blk ? 2 : 0;
      if (kKeys) {
        f = 0;
        if (row < p.T) {
          const int slot = slot_of(row, p);
          if ((p.grad_mask >> slot) & 1u) f = (vm >> slot) & 1u ? 2 : 1;
        }
      }
      fate[t] = static_cast<uint8_t>(f);
    }
    have = named_bar_and(1, 256, have);
    constexpr int C = D / 8, kPasses = BM * C / 256;
    const int k = threadIdx.x % C, r0 = threadIdx.x / C;
    const uint32_t off0 = (k >> 3) * 16384 + ((k & 7) << 4);
    uint4* d1 = reinterpret_cast<uint4*>(kKeys ? p.dk : p.dq) +
                (kKeys ? static_cast<size_t>(h) * p.T + row0
                       : static_cast<size_t>(row0) * p.H + h) * C + k;
    uint4* d2 = reinterpret_cast<uint4*>(p.dv) + (static_cast<size_t>(h) * p.T + row0) * C + k;
    const size_t pitch = static_cast<size_t>(kKeys ? 1 : p.H) * C;
#pragma unroll 4
    for (int i = 0; i < kPasses; ++i) {
      const int r = r0 + i * (256 / C);
      const int f = fate[r];
      if (f == 0) continue;
      const bool keep = have && f == 2;
      const uint32_t off = (off0 ^ ((r & 7) << 4)) + r * 128;
      const uint4 none = make_uint4(0, 0, 0, 0);
      d1[r * pitch] = keep ? lds4u(stage[0] + off) : none;
      if (kKeys) d2[r * pitch] = keep ? lds4u(stage[1] + off) : none;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (ab->flag) {
    // a wait gave up: copies and MMAs in flight end before their memory is released
    if (warp == kProducerWarp && lane == 0) {
      drain_wait(bar(B_A), 0);
      if (tail->tab) drain_wait(bar(B_TAB), 0);
      // (arrivals may be missing once every role has given up: these then run their time, which is
      // far more than a copy takes)
      const int sent = kKeys ? tail->y1 : tail->y2;  // (queries: Y2 goes first, on the same gate)
      for (int i = max(0, sent - kY1); i < sent; ++i)
        drain_wait(bar(B_GATE1 + i % kY1), (i / kY1) & 1);
      for (int i = max(0, tail->y2 - kY2); kKeys && i < tail->y2; ++i)
        drain_wait(bar(B_GATE2 + i % kY2), (i / kY2) & 1);
    }
    if (warp == kMmaWarp && lane == 0) {
      umma_commit(bar(B_FINAL));
      drain_wait(bar(B_FINAL), 0);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Both sides in one grid: the queries' CTAs, which run longest, first, the keys' behind them, so
// that neither side leaves SMs idle while the other could run.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
products_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_g,
                const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int q_tiles = p.L_pad / BM, n_q = q_tiles * p.H, b = blockIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  if (b < n_q) {
    run_rows<D, false>(tm_q, tm_k, tm_v, tm_g, tm_t, p, b / q_tiles, b % q_tiles, smem);
  } else {
    const int k_tiles = (p.T + BM - 1) / BM;
    run_rows<D, true>(tm_q, tm_k, tm_v, tm_g, tm_t, p, (b - n_q) / k_tiles, (b - n_q) % k_tiles,
                      smem);
  }
}

// ---------------------------------------------------------------------------------- host side
struct Plan {                              // scratch regions, each 256-byte aligned
  size_t k_rot, q_rot, tab, nlse, ndelta, total;
};

static Plan plan(const Geometry& g, int H, int D) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t pad = (g.L_blk + BM - 1) / BM * BM;
  Plan p{};
  p.k_rot = 0;
  p.q_rot = p.k_rot + up(static_cast<size_t>(H) * g.T * D * 2);
  p.tab = p.q_rot + up(static_cast<size_t>(H) * g.L_blk * D * 2);
  p.nlse = p.tab + up(static_cast<size_t>(g.T) * (D / 2) * 8);
  p.ndelta = p.nlse + up(H * pad * 4);
  p.total = p.ndelta + up(H * pad * 4);
  return p;
}

static void fill(const prsink_layout* L, const Geometry& g, Params& p) {
  const int D = L->head_dim, R = L->ring_slots, Bf = L->frames_per_block;
  p.H = L->n_heads;
  p.L_blk = static_cast<int>(g.L_blk);
  p.L_pad = (p.L_blk + BM - 1) / BM * BM;
  p.T = static_cast<int>(g.T);
  p.L_f = static_cast<int>(g.L_f);
  p.grid_w = L->grid_w;
  p.n_slots = g.n_slots;
  for (int s = 0; s <= g.n_slots; ++s) p.slot_start[s] = static_cast<int>(g.slot_start[s]);
  p.slot_frame[PRSINK_SLOT_REF] = 0;
  p.slot_frame[PRSINK_SLOT_STATIC] = L->ref_frames;
  p.slot_frame[PRSINK_SLOT_DYNAMIC] = L->ref_frames + Bf;
  const long long oldest = L->block_index - R + 1;     // ring slot s: block s (mod R), by age
  for (int s = 0; s < R; ++s)
    p.slot_frame[PRSINK_SLOT_RING0 + s] =
        L->ref_frames + (2 + static_cast<int>((((s - oldest) % R) + R) % R)) * Bf;
  // the queries sit on the current block's positions: those of its ring slot's rows
  p.q_row = p.slot_start[PRSINK_SLOT_RING0 + static_cast<int>(L->block_index % R)];
  p.valid_mask = L->valid_mask & ((1u << g.n_slots) - 1u);
  p.rope_mode = L->rope_mode;
  const int one[3] = {D, 0, 0};
  const int* split = L->rope_mode == 3 ? L->rope_split : one;
  int at = 0;
  for (int ax = 0; ax < 3; ++ax) {
    p.rd[ax] = split[ax] / 2;
    rope_frequencies(L->rope_base, split[ax], p.inv_pi_freq + at);
    at += p.rd[ax];
  }
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
}

template <int D>
static int launch(Params& p, cudaStream_t st) {
  constexpr int R = 256 / (D / 8);
  const char* what = "prsink_attention_backward";
  CUtensorMap mq, mk, mv, mg, mt;
  const uint64_t row = 2ull * D, H = p.H;
  int rc = make_map(&mq, p.q_rot, D, p.L_blk, H, row, row * p.L_blk, BM, 1);
  if (!rc) rc = make_map(&mk, p.k_rot, D, p.T, H, row, row * p.T, BM, 1);
  if (!rc) rc = make_map(&mv, p.v, D, p.T, H, row, row * p.T, BM, 1);
  if (!rc) rc = make_map(&mg, p.d_out, D, H, p.L_blk, row, row * H, 1, BM);
  // the table of cos / sin as rows of 4 D bytes
  if (!rc) rc = make_map(&mt, p.tab, 2 * D, p.T, 1, 2 * row, 2 * row * p.T, BM, 1);
  if (rc) return rc;
  static std::atomic<bool> allowed[64];      // (host threads may call at once)
  int n_sm = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    if (cudaFuncSetAttribute(products_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem<D>::kBytes) != cudaSuccess)
      return check_launch(what);
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  // as many heads per CTA (the angles are computed once for them) as leave eight CTAs per SM
  const int row_ctas = (p.T + R - 1) / R + p.L_pad / R;
  const long long most = static_cast<long long>(row_ctas) * p.H / (8 * n_sm);
  const int groups = most < 1 ? p.H : (p.H + static_cast<int>(most) - 1) / static_cast<int>(most);
  p.prep_heads = (p.H + groups - 1) / groups;
  launch_dependent(prep_kernel<D>, dim3(row_ctas, groups), 256, 0, st, p);
  const int tiles = p.L_pad / BM + (p.grad_mask ? (p.T + BM - 1) / BM : 0);
  launch_dependent(products_kernel<D>, dim3(tiles * p.H), kThreads, Smem<D>::kBytes, st, mq, mk,
                   mv, mg, mt, p);
  count_launch(2);
  return check_launch(what);
}

}  // namespace bwd
}  // namespace prsink

using namespace prsink;

extern "C" long long prsink_attention_backward_scratch_bytes(const prsink_layout* layout) {
  Geometry g;
  if (geometry(layout, &g)) return -1;
  return static_cast<long long>(bwd::plan(g, layout->n_heads, layout->head_dim).total);
}

extern "C" int prsink_attention_backward(const prsink_layout* layout, const void* q,
                                         const void* k_cache, const void* v_cache,
                                         const void* out, const float* lse, const void* d_out,
                                         void* dq, void* dk, void* dv, unsigned grad_mask,
                                         const long long* dyn_src, void* scratch,
                                         long long scratch_bytes, void* stream) {
  using namespace prsink::bwd;
  const char* what = "prsink_attention_backward";
  Geometry g;
  int rc = geometry(layout, &g);
  if (rc) return rc;
  grad_mask &= (1u << g.n_slots) - 1u;
  const void* bufs[] = {q, k_cache, v_cache, out, d_out, dq, dk, dv};
  const int n_bufs = grad_mask ? 8 : 6;
  for (int i = 0; i < n_bufs; ++i)
    if (!bufs[i] || !lse) {
      set_error("%s: null pointer", what);
      return PRSINK_ERR_ARG;
    }
  const int D = layout->head_dim;
  if (D != 64 && D != 128) {
    set_error("%s: head_dim %d not supported (64 or 128)", what, D);
    return PRSINK_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < n_bufs; ++i)
    if (!aligned16(bufs[i]) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
        (reinterpret_cast<uintptr_t>(dyn_src) & 7u)) {
      set_error("%s: every K/V/Q/out/gradient buffer must be 16-byte aligned, lse 4-byte, "
                "dyn_src 8-byte aligned", what);
      return PRSINK_ERR_ALIGN;
    }
  if ((g.T + BM - 1) / BM > kMaxTiles) {
    set_error("%s: %lld keys exceed the %d-tile limit", what, g.T, kMaxTiles);
    return PRSINK_ERR_UNSUPPORTED;
  }
  if (layout->n_heads > 65535) {
    set_error("%s: %d heads exceed the limit of 65535", what, layout->n_heads);
    return PRSINK_ERR_UNSUPPORTED;
  }
  const Plan pl = plan(g, layout->n_heads, D);
  if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) ||
      scratch_bytes < static_cast<long long>(pl.total)) {
    set_error("%s: scratch must be 256-byte aligned and hold %zu bytes (got %lld)", what, pl.total,
              scratch_bytes);
    return PRSINK_ERR_ARG;
  }
  const long long row = 2ll * layout->n_heads * D, nq = row * g.L_blk, nk = row * g.T;
  const Span span[] = {{q, nq}, {k_cache, nk}, {v_cache, nk}, {out, nq},
                       {lse, 4ll * layout->n_heads * g.L_blk}, {d_out, nq}, {dyn_src, 8},
                       {dq, nq}, {scratch, static_cast<long long>(pl.total)},
                       {grad_mask ? dk : nullptr, nk}, {grad_mask ? dv : nullptr, nk}};
  for (int i = 7; i < 11; ++i)             // in the place of an input or of one another
    for (int j = 0; j < i; ++j)
      if (overlap(span[i], span[j])) {
        set_error("%s: dq, dk, dv and scratch must be buffers of their own", what);
        return PRSINK_ERR_ARG;
      }
  Params p{};
  fill(layout, g, p);
  p.grad_mask = grad_mask;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k_cache);
  p.v = static_cast<const __nv_bfloat16*>(v_cache);
  p.out = static_cast<const __nv_bfloat16*>(out);
  p.d_out = static_cast<const __nv_bfloat16*>(d_out);
  p.lse = lse;
  p.dyn_src = dyn_src;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  char* base = static_cast<char*>(scratch);
  p.k_rot = reinterpret_cast<__nv_bfloat16*>(base + pl.k_rot);
  p.q_rot = reinterpret_cast<__nv_bfloat16*>(base + pl.q_rot);
  p.tab = reinterpret_cast<float2*>(base + pl.tab);
  p.status = status_word_ptr();
  if (!p.status) return PRSINK_ERR_LAUNCH;
  p.timeout_ns = 2000000000ull;
  if (const long long ns = take_debug_stall()) {
    p.debug_stall = 1;
    p.timeout_ns = static_cast<unsigned long long>(ns);
  }
  p.nlse = reinterpret_cast<float*>(base + pl.nlse);
  p.ndelta = reinterpret_cast<float*>(base + pl.ndelta);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch<128>(p, st) : launch<64>(p, st);
}
