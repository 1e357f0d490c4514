// Paged K/V cache: the append of new tokens with the rotary embedding applied on the way, and
// the attention of one new token per sequence over the pages.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <initializer_list>

#include "prsink_internal.cuh"

namespace prsink {
namespace paged {

constexpr int kMaxPairs = 64;              // head_dim / 2

// Geometry of the paged cache as the kernels use it.
struct Cache {
  int n_seqs, H, Hkv, page_size, n_pages, max_pages;
  int capacity;                            // max_pages * page_size
  int n_sink, window;
  const int* table;
  const int* lens;
  int* status;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// Length of sequence s, clamped to the table's capacity (out of range: recorded).
__device__ __forceinline__ int seq_len(const Cache& c, int s) {
  const int n = __ldcg(c.lens + s);
  if (n >= 0 && n <= c.capacity) return n;
  atomicOr(c.status, kStatusPage);
  return n < 0 ? 0 : c.capacity;
}

// ------------------------------------------------------------------------------------ append
// HBM-bound copy of n * (H + 2 Hkv) rows of d bf16, K and q rotated on the way.  A CTA takes one
// token, a share of its rows or four tokens; a thread owns one 16-byte chunk of a row, the same
// chunk of every row it moves.  The loads of the first kBatch rows, which depend on nothing, are sent
// before the token's place is looked up and the cos / sin of its position (f64 angles, shared by
// every head) are computed.
constexpr int kAppendThreads = 256;
constexpr int kBatch = 8;

struct AppendParams {
  Cache c;
  int n_tokens;
  const int* cu;                           // nullable: one token per sequence
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;                  // nullable
  long long k_stride, v_stride, q_stride;
  __nv_bfloat16* k_pages;
  __nv_bfloat16* v_pages;
  __nv_bfloat16* q_rot;
  int rope_mode, grid_w, L_f;
  int rd[3];                               // rotated pairs per axis
  double inv_pi_freq[kMaxPairs];           // base^(-2j/d_axis) / pi of every pair
};

// Rotate the four pairs of a 16-byte chunk: y0 = x0 cos - x1 sin, y1 = x0 sin + x1 cos.
__device__ __forceinline__ uint4 rotate_chunk(uint4 v, const float2 (&cs)[4]) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xFFFF0000u);
    w[i] = pack2(x0 * cs[i].x - x1 * cs[i].y, x0 * cs[i].y + x1 * cs[i].x);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Position of token i, or -1 (nothing to do), and its row in the pages, or -1 (no page).  One
// warp; the sequence is found by a 32-way search.
__device__ __forceinline__ void place_token(const AppendParams& p, int i, int lane, int& pos,
                                            long long& row) {
  pos = -1;
  row = -1;
  int s = i, back = 1;                     // the token is the back-th last of sequence s
  if (p.cu) {
    // the last s with cu[s] <= i, of cu[0 .. n_seqs]
    int lo = 0, n = p.c.n_seqs + 1;
    while (n > 1) {
      const int step = (n + 31) / 32, at = lo + lane * step;
      const bool below = lane * step < n && p.cu[at] <= i;
      const int last = 31 - __clz(__ballot_sync(~0u, below) | 1u);
      n = min(step, n - last * step);
      lo += last * step;
    }
    s = lo;
    if (s == p.c.n_seqs) return;           // behind the last sequence
    const int a = p.cu[s], b = p.cu[s + 1];
    if (i < a || i >= b) {
      if (lane == 0) atomicOr(p.c.status, kStatusPage);
      return;
    }
    back = b - i;
  }
  const int n = p.c.lens[s];
  if (n < back || n > p.c.capacity) {
    if ((n != 0 || p.cu) && lane == 0) atomicOr(p.c.status, kStatusPage);     // (0: an idle row)
    return;
  }
  pos = n - back;
  const int at = pos / p.c.page_size;
  const int page = p.c.table[static_cast<long long>(s) * p.c.max_pages + at];
  if (page >= 0 && page < p.c.n_pages)
    row = static_cast<long long>(page) * p.c.Hkv * p.c.page_size + (pos - at * p.c.page_size);
  else if (lane == 0)
    atomicOr(p.c.status, kStatusPage);
}

template <int D, int kTok>
__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int C = D / 8;                 // 16-byte chunks of a row
  constexpr int R = kAppendThreads / C;    // rows per pass
  __shared__ int pos_s[kTok];
  __shared__ long long row_s[kTok];
  __shared__ __align__(16) float2 tab[kTok][D / 2];
  const int i0 = blockIdx.x * kTok, n_tok = min(kTok, p.n_tokens - i0);
  const int c = threadIdx.x % C, r0 = threadIdx.x / C, warp = threadIdx.x >> 5;
  const int Hq = p.q ? p.c.H : 0, Hkv = p.c.Hkv;
  // rows of this CTA: an equal share of every token's rows per blockIdx.y
  const int rows = Hq + 2 * Hkv;
  const int per = (rows + gridDim.y - 1) / gridDim.y;
  const int ra = blockIdx.y * per, mine = min(rows, ra + per) - ra;
  const int items = mine > 0 ? mine * n_tok : 0;           // (token, row) pairs, token-major
  // this thread's items, R apart: token and row of the next one to load and of the next to store
  struct Item {
    int k, tok, r;
  };
  auto wrap = [&](Item& it) {
    if (kTok > 1)
      while (it.r >= mine) {
        it.r -= mine;
        ++it.tok;
      }
  };
  auto next = [&](Item& it) {
    it.k += R;
    it.r += R;
    wrap(it);
  };
  Item ld{r0, 0, r0}, st;
  if (mine > 0) wrap(ld);
  st = ld;
  auto load = [&](const Item& it) {
    const long long i = i0 + (kTok > 1 ? it.tok : 0);
    const int r = ra + it.r;
    const __nv_bfloat16* src =
        r < Hq ? p.q + i * p.q_stride + r * D
               : (r < Hq + Hkv ? p.k + i * p.k_stride + (r - Hq) * D
                               : p.v + i * p.v_stride + (r - Hq - Hkv) * D);
    return __ldcs(reinterpret_cast<const uint4*>(src) + c);
  };
  grid_dependency_wait();
  grid_launch_dependents();
  uint4 x[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u)
    if (ld.k < items) {
      x[u] = load(ld);
      next(ld);
    }
  if (warp < n_tok) {
    int pos;
    long long row;
    place_token(p, i0 + warp, threadIdx.x & 31, pos, row);
    if ((threadIdx.x & 31) == 0) {
      pos_s[warp] = pos;
      row_s[warp] = row;
    }
  }
  __syncthreads();
  if (p.rope_mode) {
    for (int e = threadIdx.x; e < n_tok * (D / 2); e += kAppendThreads) {
      const int t = e / (D / 2), j = e % (D / 2);
      int at = pos_s[t];
      if (at < 0) continue;
      if (p.rope_mode == 3) {
        const int f = at / p.L_f, in = at - f * p.L_f, y = in / p.grid_w;
        at = j < p.rd[0] ? f : (j < p.rd[0] + p.rd[1] ? y : in - y * p.grid_w);
      }
      double sn, co;
      sincospi(static_cast<double>(at) * p.inv_pi_freq[j], &sn, &co);   // exact reduction
      tab[t][j] = make_float2(static_cast<float>(co), static_cast<float>(sn));
    }
    __syncthreads();
  }
  const long long head = static_cast<long long>(p.c.page_size) * D;    // a page's next head
  while (st.k < items) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (st.k >= items) break;
      const int r = ra + st.r, tok = kTok > 1 ? st.tok : 0;
      const long long row = row_s[tok];
      if (p.rope_mode && r < Hq + Hkv) {
        const float4* tp = reinterpret_cast<const float4*>(&tab[tok][4 * c]);
        const float4 a = tp[0], b = tp[1];
        const float2 cs[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w),
                              make_float2(b.x, b.y), make_float2(b.z, b.w)};
        x[u] = rotate_chunk(x[u], cs);
      }
      __nv_bfloat16* dst =
          r < Hq ? p.q_rot + (static_cast<long long>(i0 + tok) * Hq + r) * D
                 : (r < Hq + Hkv ? p.k_pages + row * D + (r - Hq) * head
                                 : p.v_pages + row * D + (r - Hq - Hkv) * head);
      if (pos_s[tok] >= 0 && (r < Hq || row >= 0)) reinterpret_cast<uint4*>(dst)[c] = x[u];
      next(st);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (ld.k < items) {
        x[u] = load(ld);
        next(ld);
      }
  }
}

// --------------------------------------------------------------------------------- attention
// One new token per sequence: HBM-bound, every K and V byte is read once for 64 query heads of its
// key head (more heads are taken 64 at a time, each with a pass of its own).  The tensor core takes
// the products with the KEYS as the 128 rows of its tile and the query heads that share a key
// head as its N columns, so K and V go from TMA straight to the MMA and no thread touches them:
//   S^T [128 keys][N heads] = K Q^T        (A = K tile, K-major;  B = Q, N rows)
//   O^T [d][N heads]       += V^T P^T      (A = V tile, MN-major; B = P, N rows of 128 keys)
// The softmax between them has one key per thread.  Its running maximum m is only an offset: any
// m within 2^8 of the true one keeps every probability in range, so a tile whose scores stay
// below m + 8 (log2 units) needs no reduction at all, just one vote; the sums stay per thread
// until the row ends.  A tile that exceeds it (and the first one of a row) takes the maximum
// across the threads, and O and the sums are rescaled.
//
// P is rounded to bf16: both operands of an MMA have one type, and V's is bf16.  A probability is
// off by 2^-8 of itself at most, independently of the others; the sums and lse take it unrounded.
// The output's error in the 2-norm is 2.1-2.4e-3, of which 1.7e-3 is its own rounding.  A second
// product with what the rounding leaves would remove the rest, for twice the stores of the softmax
// (which with 32 and more heads is what bounds the kernel, see below).
//
// Work is cut into units of one key tile of one (sequence, key head) row, in row order; every
// CTA (one per SM) takes an equal, contiguous share, so ragged lengths balance and one long
// sequence spreads over the device.  A row shared by several CTAs leaves one partial result
// (O, m, l) each in scratch; a second kernel, launched early and waiting for the first, joins
// them in CTA order (no counters to clear, no order that depends on timing).
//
// Where the table (or the sinks and the window) leaves no room for a row longer than kWholeRow tiles,
// a row belongs to the CTA that holds its first unit and nothing is left to join: a tile more costs
// less than the second kernel.  The lengths themselves are on the device, so a short sequence in a
// wide table takes both kernels: 256 tokens, one head, 6.6 us on the device with a table of 256 tokens,
// 8.2 with one of 1024 or 65536; about 2 us more on the host.
//
// A tile holds whole pages up to 128 tokens, or up to 128 tokens of one page; one TMA box per
// page.  Warps: 0-3 softmax, 4 and 7 send K and V, 5 issues the S products, 6 the O products (one
// thread issues an MMA in about 45 cycles whatever its size, one warp a box in about 100: with one
// sending warp, pages of 8 took 402 us where two take 319, 64 sequences x 8000 tokens).
//
// Measured on a B200 (6551 GB/s copy), the same inputs each time: 64 sequences x 8000 tokens x 8 key
// heads of 128, 64 query heads, 316 us (6.6 TB/s) at pages of 16 and more; 48 ragged sequences of up
// to 16001 tokens, 40 heads on 8, pages of 16, 239 us (6.6 TB/s; 242-249 with inputs that change);
// one sequence of 14400 tokens, 40 heads, 52.5 us (5.6 TB/s: the start, about 5 us to the first
// landed tile, and the join are 7 us of it; 53-54 with inputs that change).
//
// Heads on a key head, one key head, 16000 tokens, pages of 16 (64 sequences of width 128 / 128 of 64):
//   1         98 us (5.4 TB/s) / 115 us (4.6)        33   117 us (4.5) / 180 us (2.9)
//   16, 17   102, 105 (5.2, 5.0) / 123, 137          64   150 us (3.5) / 234 us (2.2)
//   32       109 us (4.8) / 155 us (3.4)            128   244 us: two passes / 426 us
// A tile takes the softmax warps about 0.5 us at N = 16 where HBM needs 1.45 (width 128) or 0.73 (64),
// and about four times that at N = 64, where they are the bound (255 registers and 204 bytes spilled).
constexpr int kTile = 128;                 // key rows of a tile = TMEM lanes
constexpr int kAttThreads = 256;
constexpr int kKeyWarp = 4, kScoreWarp = 5, kOutWarp = 6, kValueWarp = 7;
constexpr int kMaxStages = 6;
constexpr int kWholeRow = 4;
constexpr int kMetaRing = 16;              // tiles whose bad-page bits are kept
constexpr float kRescale = 8.0f;           // log2 units: O is rescaled when a maximum grows > 2^8
// Offset of a head whose scores so far are all -inf.  Finite: a score of -inf stays -inf beside it
// (it weighs nothing; -inf minus -inf would be NaN), a finite one exceeds it by far more than 2^8.
constexpr float kNoOffset = -3.402823466e38f;

// Quotient by a constant of the call: q = (n + hi(n m)) >> s for 0 <= n < 2^31, with 2^s the next
// power of two >= d and m = floor(2^32 (2^s - d) / d) + 1.
struct Divisor {
  uint32_t m, s;
  void set(uint32_t d) {
    s = 0;
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>((((1ull << s) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((static_cast<uint32_t>(n) + __umulhi(static_cast<uint32_t>(n), m)) >> s);
  }
};

struct AttParams {
  Cache c;
  Divisor by_tile;                         // tokens of a tile (small pages) or of a page
  Divisor by_tiles_per_page, by_chunks;
  bool whole_rows;                         // rows are not shared (see above)
  int group, chunks;                       // query heads per key head, N-column chunks of them
  int tile_tokens, pages_per_tile;         // of a tile when pages are smaller than a tile
  int tiles_per_page;                      // tiles of a page when pages are larger (else 0)
  int box_rows;                            // rows of one TMA box (a page, or a tile)
  // K / V tiles in shared memory, in 1 KB swizzle atoms of 8 rows x 64 elements: bytes between
  // row groups and between the two 64-element panels of a row
  int group_bytes, panel_bytes;
  bool one_box;                            // a box lands both panels (5-D map)
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;                           // [CTAs][2][N][D] unnormalised partial results
  float2* part_ml;                         // [CTAs][2][N] their maximum (log2 units) and sum
  unsigned long long timeout_ns;
  int debug_stall;                         // self-test: withhold the first commit of S
};

template <int D, int N>
struct Smem {
  static constexpr int kTileBytes = kTile * D * 2;
  // K and V stages: as many as fit beside Q, P and the scores
  static constexpr int kKS = D == 128 ? (N == 64 ? 2 : 3) : (N == 16 ? 6 : (N == 32 ? 5 : 4));
  static constexpr int kVS = D == 128 ? (N == 16 ? 3 : 2) : kKS;
  // V first: the second 64-row panel that the MMA reads past a 64-wide V tile (rows of O^T that
  // nobody uses) then stays inside the allocation
  static constexpr int kV = 0;
  static constexpr int kK = kV + kVS * kTileBytes;
  static constexpr int kQ = kK + kKS * kTileBytes;      // 2 buffers
  static constexpr int kP = kQ + 2 * N * D * 2;
  static constexpr int kPBytes = N * kTile * 2;         // 2 buffers
  static constexpr int kBytes = kP + 2 * kPBytes;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, N, false, false);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(128, N, true, false);
  static constexpr uint32_t kColO = 2 * N;              // TMEM: S0, S1, O
  static constexpr uint32_t kTmemCols = N == 16 ? 64 : (N == 32 ? 128 : 256);
  static_assert(kKS <= kMaxStages && kKS + 2 < kMetaRing, "stages");
  static_assert(kBytes + 1024 <= 227 * 1024, "shared memory");
};

// The attended tokens of a sequence and their tiles: tokens [0, sink) and [win0, len); tiles
// [0, n_a) and [first_b, first_b + count - n_a).
struct Row {
  int len, sink, win0, n_a, first_b, count;
  __device__ __forceinline__ static int tile_of(const AttParams& p, int token) {
    const int x = p.by_tile(token);
    return p.tiles_per_page ? x * p.tiles_per_page + (token - x * p.c.page_size) / kTile : x;
  }
  __device__ __forceinline__ Row(const AttParams& p, int n) {
    len = n;
    win0 = p.c.window > 0 ? max(0, len - p.c.window) : 0;
    sink = min(p.c.n_sink, win0);
    n_a = sink > 0 ? tile_of(p, sink - 1) + 1 : 0;
    first_b = 0;
    count = 0;
    if (len > 0) {
      first_b = max(tile_of(p, win0), n_a);
      count = n_a + max(0, tile_of(p, len - 1) + 1 - first_b);
    }
  }
  __device__ __forceinline__ bool attended(int token) const {
    return token < sink || (token >= win0 && token < len);
  }
  // every token of a tile is attended
  __device__ __forceinline__ bool whole(int start, int cnt) const {
    return start + cnt <= sink || (start >= win0 && start + cnt <= len);
  }
};

// The attended tiles of a row from the i-th on: first token, tokens, first page and the token's
// row in it.
struct Tile {
  int i, start, cnt, page, sub;
  __device__ __forceinline__ Tile(const AttParams& p, const Row& row, int i_) : i(i_) {
    seek(p, i < row.n_a ? i : row.first_b + (i - row.n_a));
  }
  __device__ __forceinline__ void seek(const AttParams& p, int t) {
    if (!p.tiles_per_page) {
      page = t * p.pages_per_tile;
      sub = 0;
      cnt = p.tile_tokens;
    } else {
      page = p.by_tiles_per_page(t);
      sub = (t - page * p.tiles_per_page) * kTile;
      cnt = min(kTile, p.c.page_size - sub);
    }
    start = page * p.c.page_size + sub;
  }
  __device__ __forceinline__ void next(const AttParams& p, const Row& row) {
    if (++i == row.n_a) {
      seek(p, row.first_b);
    } else if (!p.tiles_per_page) {
      start += cnt;
      page += p.pages_per_tile;
    } else {
      start += cnt;
      sub += kTile;
      if (sub >= p.c.page_size) {
        sub = 0;
        ++page;
      }
      cnt = min(kTile, p.c.page_size - sub);
    }
  }
};

// Stage of a ring and the parity of its current phase, advanced tile by tile.
template <int kStages>
struct Ring {
  int st = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++st == kStages) {
      st = 0;
      parity ^= 1;
    }
  }
};

// 64-bit quotient, by the 32-bit division where both fit.
__device__ __forceinline__ long long quot(long long a, long long b) {
  if (((a | b) >> 31) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// A CTA's share of the units, row by row; every role walks it on its own.
struct Start {
  int s, hc, i0, len;                      // sequence, head chunk, tile, the sequence's length
};

struct Walk {
  long long left;                          // units left, this segment's included
  int s, hc, i0, n;                        // sequence, head chunk, first tile, tiles here
  Row row;
  bool first;                              // the CTA's first segment
  __device__ __forceinline__ Walk(const AttParams& p, const Start& at, long long units)
      : left(units), s(at.s), hc(at.hc), i0(at.i0), n(0), row(p, at.len), first(true) {
    if (p.whole_rows && i0 > 0) {          // this row is the CTA's before
      n = row.count - i0;
      next(p);
    } else {
      take(p);
    }
  }
  __device__ __forceinline__ void take(const AttParams& p) {
    n = row.count - i0;
    if (!p.whole_rows) n = static_cast<int>(min(left, static_cast<long long>(n)));
  }
  __device__ __forceinline__ void next(const AttParams& p) {
    left -= n;
    first = false;
    if (left <= 0) return;
    i0 = 0;
    if (++hc == p.c.Hkv * p.chunks) {
      hc = 0;
      do {
        if (++s >= p.c.n_seqs) { left = 0; return; }       // (lengths changed under the call)
        row = Row(p, seq_len(p.c, s));
      } while (row.count == 0);
    }
    take(p);
  }
};

__device__ __forceinline__ float warp_max(float x) {
  float y;
  // volatile: all 32 lanes have to get here, also where one lane alone uses the result
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void sts_bf16(uint32_t addr, float x) {
  asm volatile("st.shared.b16 [%0], %1;"
               :: "r"(addr), "h"(__bfloat16_as_ushort(__float2bfloat16_rn(x))) : "memory");
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
}

// KFULL / VFULL: a stage has landed.  SDONE: the S product of the tile in K stage i is done (its
// scores may be read, the stage refilled); ODONE: likewise the O product of V stage i (O holds
// the tile, P and the stage are free).  SFREE: the scores of a buffer have been read.
enum Bar {
  B_KFULL = 0, B_SDONE = B_KFULL + kMaxStages, B_VFULL = B_SDONE + kMaxStages,
  B_ODONE = B_VFULL + kMaxStages, B_SFREE = B_ODONE + kMaxStages, B_PFULL = B_SFREE + 2,
  B_QFULL = B_PFULL + 2, B_QFREE = B_QFULL + 2, B_FINAL = B_QFREE + 2, B_COUNT = B_FINAL + 2
};

// Bounded wait that ignores the abort flag (used while draining after an abort).
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t dl = globaltimer() + 100000000ull;
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() > dl) break;
}

// Units of a call and a CTA's share of them: the first total % G CTAs take one more than the
// others, and no CTA that takes part is without work.
struct Share {
  long long total, each, extra;
  int G;
  __device__ __forceinline__ Share(long long total_, int ctas) : total(total_) {
    G = static_cast<int>(min(static_cast<long long>(ctas), max(total, 1ll)));
    each = quot(total, G);
    extra = total - each * G;
  }
  __device__ __forceinline__ long long begin(int cta) const {
    return cta < G ? each * cta + min(static_cast<long long>(cta), extra) : total;
  }
  __device__ __forceinline__ int cta_of(long long u) const {
    const long long split = extra * (each + 1);
    return static_cast<int>(u < split ? quot(u, each + 1) : extra + quot(u - split, each));
  }
};

// Where unit `begin(cta)` lies, by a block-wide scan over the lengths (consecutive sequences per
// thread).  Two barriers; `warp_s` one word per warp.
template <int kThreads>
__device__ __forceinline__ Share find_share(const AttParams& p, int cta, long long* warp_s,
                                            Start* at_s) {
  const int hcs = p.c.Hkv * p.chunks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.c.n_seqs + kThreads - 1) / kThreads;
  const int sa = min(p.c.n_seqs, static_cast<int>(threadIdx.x) * per);
  const int se = min(p.c.n_seqs, sa + per);
  long long mine = 0;
  int len = 0;
  for (int s = sa; s < se; ++s) {
    len = seq_len(p.c, s);
    mine += Row(p, len).count;
  }
  mine *= hcs;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_s[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_s[w];
    total += warp_s[w];
  }
  const Share sh(total, gridDim.x);
  const long long u0 = sh.begin(cta);
  if (u0 >= before && u0 < before + mine) {
    long long off = u0 - before;
    int s = sa;
    int count = Row(p, len).count;
    if (per > 1)
      for (;; ++s) {
        len = seq_len(p.c, s);
        count = Row(p, len).count;
        const long long n = static_cast<long long>(count) * hcs;
        if (off < n || s + 1 >= se) break;
        off -= n;
      }
    count = max(count, 1);
    const int hc = static_cast<int>(quot(off, count));
    *at_s = Start{s, hc, static_cast<int>(off - static_cast<long long>(hc) * count), len};
  }
  __syncthreads();
  return sh;
}

template <int D, int N>
__global__ void __launch_bounds__(kAttThreads, 1)
paged_attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ AttParams p) {
  using SM = Smem<D, N>;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t bars[B_COUNT];
  __shared__ uint32_t tmem_base_s;
  __shared__ AbortState ab;
  __shared__ uint16_t bad_pages[kMetaRing];
  __shared__ __align__(16) float m_s[N];           // the heads' running offsets (log2 units)
  __shared__ __align__(16) float alpha_s[N];       // what a new offset rescales by
  __shared__ __align__(16) float red_s[4][N];      // per warp: tile maxima, then sums
  __shared__ long long scan_s[kAttThreads / 32];
  __shared__ Start start_s;
  __shared__ int loads_s[3];                       // Q, K and V loads sent (for the drain)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(dsmem);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* gb = dsmem + (sb - raw);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(bar(B_KFULL + i), 1);
      mbar_init(bar(B_SDONE + i), 1);
      mbar_init(bar(B_VFULL + i), 1);
      mbar_init(bar(B_ODONE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_SFREE + i), 128);
      mbar_init(bar(B_PFULL + i), 128);
      mbar_init(bar(B_QFULL + i), 1);
      mbar_init(bar(B_QFREE + i), 1);
      mbar_init(bar(B_FINAL + i), 1);
    }
    ab.flag = 0;
    start_s = Start{};
    loads_s[0] = loads_s[1] = loads_s[2] = 0;
    fence_barrier_init();
  }
  if (warp == kKeyWarp && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == kScoreWarp) {
    tmem_alloc(smem_u32(&tmem_base_s), SM::kTmemCols);
    tmem_relinquish();
  }
  // V rows that no box fills (pages that do not divide a tile) must be finite: P is 0 there, but
  // 0 * NaN is not.  (Columns of P that no head fills may hold anything: they reach only columns of O
  // that nobody reads.)
  if (!p.tiles_per_page && p.tile_tokens < kTile)
    for (int i = threadIdx.x; i < SM::kVS * SM::kTileBytes / 16; i += kAttThreads)
      reinterpret_cast<uint4*>(gb + SM::kV)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  grid_dependency_wait();
  grid_launch_dependents();
  const int cta = blockIdx.x;
  const Share sh = find_share<kAttThreads>(p, cta, scan_s, &start_s);
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  // (a CTA's share of the call may take any time, so each wait has a limit of its own)
  auto wait = [&](int i, uint32_t parity) {
    return mbar_wait_limit(bar(i), parity, &ab, p.timeout_ns, p.c.status);
  };
  const long long u1 = sh.begin(cta + 1);
  Walk w(p, start_s, u1 - sh.begin(cta));

  if (warp == kKeyWarp || warp == kValueWarp) {
    // ------------------------------------------------------------------- TMA producers
    // Lane i loads page i of the tile; pages without an attended token are left alone (their
    // rows are masked).
    const bool keys = warp == kKeyWarp;
    const int stages = keys ? SM::kKS : SM::kVS;
    const int b_full = keys ? B_KFULL : B_VFULL, b_done = keys ? B_SDONE : B_ODONE;
    const CUtensorMap* tm = keys ? &tm_k : &tm_v;
    const uint32_t ring = sb + (keys ? SM::kK : SM::kV);
    int j = 0, seg = 0, st = 0;
    uint32_t parity = 1;                           // of the phase that frees the stage
    bool ok = true;
    for (; ok && w.left > 0; w.next(p), ++seg) {
      const int* table = p.c.table + static_cast<long long>(w.s) * p.c.max_pages;
      const int kvh = p.by_chunks(w.hc), chunk = w.hc - kvh * p.chunks;
      // Table entries are read 32 at a time, a batch ahead of their use: lane l holds page
      // l % pages_per_tile of tile base + l / pages_per_tile.
      const int ppt = p.pages_per_tile, batch = 32 / ppt;
      const int my_tile = lane / ppt, my_page = lane - my_tile * ppt;
      int page = 0, row = 0, base = 0;
      bool need = false;
      auto fetch = [&](int from, int& e_page, int& e_row, bool& e_need) {
        e_need = my_tile < batch && from + my_tile < w.n;
        if (e_need) {
          const Tile tile(p, w.row, w.i0 + from + my_tile);
          const int first = tile.start + my_page * p.c.page_size;
          e_need = first < w.row.sink ||
                   (first + p.c.page_size > w.row.win0 && first < w.row.len);
          e_row = tile.sub;
          if (e_need) e_page = __ldg(table + tile.page + my_page);
        }
      };
      int n_page = 0, n_row = 0;
      bool n_need = false;
      fetch(0, n_page, n_row, n_need);
      if (keys) {
        if (seg >= 2)
          ok = wait(B_QFREE + (seg & 1), ((seg >> 1) - 1) & 1);
        if (!__all_sync(~0u, ok)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_QFULL + (seg & 1)), N * D * 2);
          for (int pp = 0; pp < D / 64; ++pp)
            tma_load_3d(sb + SM::kQ + (seg & 1) * N * D * 2 + pp * N * 128, &tm_q,
                        bar(B_QFULL + (seg & 1)), pp * 64, chunk * N, w.s * p.c.Hkv + kvh);
          loads_s[0] = seg + 1;
        }
      }
      for (int i = 0; i < w.n; ++i, ++j) {
        if (i == 0 || i == base + batch) {
          base = i;
          page = n_page;
          row = n_row;
          need = n_need;
          fetch(base + batch, n_page, n_row, n_need);
        }
        const int src = (i - base) * ppt + lane;
        const int t_page = __shfl_sync(~0u, page, src & 31);
        const int t_row = __shfl_sync(~0u, row, src & 31);
        const bool t_need = __shfl_sync(~0u, static_cast<int>(need), src & 31) && lane < ppt;
        const bool bad = t_need && (t_page < 0 || t_page >= p.c.n_pages);
        const int np = __popc(__ballot_sync(~0u, t_need));
        const uint32_t bad_mask = __ballot_sync(~0u, bad);
        if (j >= stages) ok = wait(b_done + st, parity);
        if (!__all_sync(~0u, ok)) { ok = false; break; }
        if (lane == 0) {
          if (keys) {
            bad_pages[j & (kMetaRing - 1)] = static_cast<uint16_t>(bad_mask);
            if (bad_mask) atomicOr(p.c.status, kStatusPage);
          }
          mbar_arrive_expect_tx(bar(b_full + st), np * p.box_rows * D * 2);
          loads_s[keys ? 1 : 2] = j + 1;
        }
        __syncwarp();
        if (t_need) {
          // (a bad page: a box past the pool, which is filled with zeros)
          const int c2 = bad ? p.c.n_pages * p.c.Hkv : t_page * p.c.Hkv + kvh;
          const uint32_t dst = ring + st * SM::kTileBytes;
          if (p.one_box) {
            tma_load_5d(dst + lane * p.box_rows * D * 2, tm, bar(b_full + st), 0, 0, 0,
                        t_row >> 3, c2);
          } else {                                 // a large page whose rows end inside a group
            for (int pp = 0; pp < D / 64; ++pp)
              tma_load_3d(dst + pp * (kTile * 128), tm, bar(b_full + st), pp * 64, t_row, c2);
          }
        }
        if (++st == stages) {
          st = 0;
          parity ^= 1;
        }
      }
    }
  } else if (warp == kScoreWarp) {
    // ------------------------------------------------------------------- S = K Q^T
    if (lane == 0) {
      int j = 0, seg = 0;
      Ring<SM::kKS> rk;
      bool ok = true;
      const uint32_t panel = static_cast<uint32_t>(p.panel_bytes) >> 4;    // descriptor units
      for (; ok && w.left > 0; w.next(p), ++seg) {
        ok = wait(B_QFULL + (seg & 1), (seg >> 1) & 1);
        const uint64_t b = sdesc_sw128(sb + SM::kQ + (seg & 1) * N * D * 2, 16, 1024);
        for (int i = 0; ok && i < w.n; ++i, ++j, rk.next()) {
          const int st = rk.st, sbuf = j & 1;
          ok = (j < 2 || wait(B_SFREE + sbuf, ((j >> 1) - 1) & 1)) &&
               wait(B_KFULL + st, rk.parity);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = sdesc_sw128(sb + SM::kK + st * SM::kTileBytes, 16, p.group_bytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_ss(tmem + sbuf * N, a + (kk >> 2) * panel + (kk & 3) * 2,
                    b + (kk >> 2) * (N * 8) + (kk & 3) * 2, SM::kIdescS, kk != 0);
          if (!(p.debug_stall && j == 0)) umma_commit(bar(B_SDONE + st));
          if (i + 1 == w.n) umma_commit(bar(B_QFREE + (seg & 1)));
        }
      }
    }
    __syncwarp();
  } else if (warp == kOutWarp) {
    // ------------------------------------------------------------------- O += V^T P^T
    if (lane == 0) {
      int j = 0;
      Ring<SM::kVS> rv;
      bool ok = true;
      const uint32_t keys16 = static_cast<uint32_t>(p.group_bytes) >> 3;   // two row groups
      for (; ok && w.left > 0; w.next(p)) {
        for (int i = 0; i < w.n; ++i, ++j, rv.next()) {
          const int st = rv.st;
          ok = wait(B_VFULL + st, rv.parity) &&
               wait(B_PFULL + (j & 1), (j >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = sdesc_sw128(sb + SM::kV + st * SM::kTileBytes, p.panel_bytes,
                                         p.group_bytes);
          const uint64_t b = sdesc_sw128(sb + SM::kP + (j & 1) * SM::kPBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ss(tmem + SM::kColO, a + kk * keys16, b + (kk >> 2) * (N * 8) + (kk & 3) * 2,
                    SM::kIdescO, !(i == 0 && kk == 0));
          umma_commit(bar(B_ODONE + st));
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------- softmax (warps 0-3)
    const int t = threadIdx.x;                     // key row = TMEM lane; O^T: element of d
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    constexpr int CH = N < 32 ? 16 : 32;           // columns of one TMEM access
    auto ld_cols = [&](uint32_t at, uint32_t (&r)[CH]) {
      if constexpr (CH == 16) tmem_ld16(at, r); else tmem_ld32(at, r);
    };
    // sequences with nothing to attend
    for (int s = cta; s < p.c.n_seqs; s += gridDim.x) {
      if (Row(p, seq_len(p.c, s)).count) continue;
      uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<long long>(s) * p.c.H * D);
      for (int i = t; i < p.c.H * D / 8; i += 128) o[i] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int i = t; i < p.c.H; i += 128)
          p.lse[static_cast<long long>(s) * p.c.H + i] = -INFINITY;
    }
    // this key's place in P: row g (head), column t, 128-byte swizzle
    const uint32_t p_col0 = sb + SM::kP + (t >> 6) * (N * 128) + (t & 7) * 2;
    const int chunk16 = (t & 63) >> 3;
    int j = 0;
    Ring<SM::kKS> rk;
    Ring<SM::kVS> rv, rv1, rv2;                    // V stages of tiles j, j - 1, j - 2
    bool ok = true;
    auto o_done = [&](const Ring<SM::kVS>& r) {    // the O product of the tile is complete
      return wait(B_ODONE + r.st, r.parity);
    };
    for (; ok && w.left > 0; w.next(p)) {
      const int kvh = p.by_chunks(w.hc), chunk = w.hc - kvh * p.chunks;
      const int nh = min(N, p.group - chunk * N);  // heads of this chunk
      float l[N];                                  // this key's share of the heads' sums
#pragma unroll
      for (int g = 0; g < N; ++g) l[g] = 0.f;
      Tile tile(p, w.row, w.i0);
      for (int i = 0; i < w.n; ++i, ++j, tile.next(p, w.row)) {
        const bool whole = w.row.whole(tile.start, tile.cnt);
        bool live = t < tile.cnt && (whole || w.row.attended(tile.start + t));
        ok = ok && wait(B_SDONE + rk.st, rk.parity);
        rk.next();
        __syncwarp();
        tc_fence_after();
        uint32_t s[N];
#pragma unroll
        for (int c = 0; c < N; c += CH)
          ld_cols(tmem + lane_off + (j & 1) * N + c, *reinterpret_cast<uint32_t(*)[CH]>(&s[c]));
        const uint32_t bad = bad_pages[j & (kMetaRing - 1)];
        if (bad) live = live && !((bad >> (p.tiles_per_page ? 0 : t / p.c.page_size)) & 1u);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(bar(B_SFREE + (j & 1)));
        // scores in log2 units relative to the running offsets: does any exceed them by > 2^8?
        // (Heads are taken four at a time; those past nh have zero queries and offset 0.)
        float z[N];
        bool over = i == 0;
        if (i > 0) {
          float top = -INFINITY;
#pragma unroll
          for (int g = 0; g < N; g += 4) {
            if (g >= nh) break;
            const float4 m4 = *reinterpret_cast<const float4*>(&m_s[g]);
            const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[g + e] = fmaf(__uint_as_float(s[g + e]), p.scale_log2, -m[e]);
              top = fmaxf(top, z[g + e]);
            }
          }
          over = live && top > kRescale;
        }
        if (!named_bar_and(1, 128, ok && !over)) {
          // new offsets: the tile's maxima where they exceed the old ones by more than 2^8
          if (!named_bar_and(1, 128, ok)) { ok = false; break; }
#pragma unroll
          for (int g = 0; g < N; g += 4) {
            if (g >= nh) break;
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = warp_max(live ? __uint_as_float(s[g + e]) : -INFINITY);
            if (lane == 0)
              *reinterpret_cast<float4*>(&red_s[warp][g]) = make_float4(x[0], x[1], x[2], x[3]);
          }
          if (j > 0) ok = o_done(rv1);             // O may be rescaled
          named_bar_sync(1, 128);
          if (t < N) {
            float m = 0.f, alpha = 1.f;
            if (t < nh) {
              const float mt = fmaxf(fmaxf(red_s[0][t], red_s[1][t]),
                                     fmaxf(red_s[2][t], red_s[3][t])) * p.scale_log2;
              m = i > 0 ? m_s[t] : kNoOffset;
              if (mt > m + kRescale) {
                if (m > kNoOffset) alpha = ex2(m - mt);
                m = mt;
              }
            }
            m_s[t] = m;
            alpha_s[t] = alpha;
          }
          named_bar_sync(1, 128);
          if (i > 0) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < N; c += CH) {
              if (c >= nh) break;
              uint32_t o[CH];
              ld_cols(tmem + lane_off + SM::kColO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < CH; e += 4) {
                const float4 a4 = *reinterpret_cast<const float4*>(&alpha_s[c + e]);
                const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                  l[c + e + f] *= a[f];
                  o[e + f] = __float_as_uint(__uint_as_float(o[e + f]) * a[f]);
                }
              }
              if constexpr (CH == 16) tmem_st16(tmem + lane_off + SM::kColO + c, o);
              else tmem_st32(tmem + lane_off + SM::kColO + c, o);
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int g = 0; g < N; g += 4) {
            if (g >= nh) break;
            const float4 m4 = *reinterpret_cast<const float4*>(&m_s[g]);
            const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              z[g + e] = fmaf(__uint_as_float(s[g + e]), p.scale_log2, -m[e]);
          }
        } else if (j > 1) {
          ok = o_done(rv2);                        // its P buffer may be overwritten
        }
        rv2 = rv1;
        rv1 = rv;
        const uint32_t p_col = p_col0 + (j & 1) * SM::kPBytes;
#pragma unroll
        for (int g = 0; g < N; g += 4) {
          if (g >= nh) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = live ? ex2(z[g + e]) : 0.f;
            l[g + e] += x;
            sts_bf16(p_col + (g + e) * 128 + ((chunk16 ^ ((g + e) & 7)) << 4), x);
          }
        }
        if (!whole) {
          // rows without an attended token may hold anything
          ok = ok && wait(B_VFULL + rv.st, rv.parity);
          if (!live && t < tile.cnt)
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(gb + SM::kV + rv.st * SM::kTileBytes +
                                        (t >> 3) * p.group_bytes + (c >> 3) * p.panel_bytes +
                                        (t & 7) * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
        rv.next();
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(B_PFULL + (j & 1)));
      }
      // the row's result, or this CTA's part of it
      if (ok) ok = o_done(rv1);
      if (!named_bar_and(1, 128, ok)) { ok = false; break; }
      tc_fence_after();
      // sums: each key's shares through the P buffers (free now), a head per warp pass
      float* part = reinterpret_cast<float*>(gb + SM::kP);
#pragma unroll
      for (int g = 0; g < N; g += 4) {
        if (g >= nh) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) part[(g + e) * kTile + t] = l[g + e];
      }
      named_bar_sync(1, 128);
      const long long head0 = static_cast<long long>(w.s) * p.c.H + kvh * p.group + chunk * N;
      const long long slot = (static_cast<long long>(cta) * 2 + (w.first ? 0 : 1)) * N;
      const bool complete = w.n == w.row.count;
#pragma unroll 1
      for (int g = warp; g < nh; g += 4) {
        const float4 x = *reinterpret_cast<const float4*>(part + g * kTile + 4 * lane);
        float lg = (x.x + x.y) + (x.z + x.w);
#pragma unroll
        for (int k = 16; k; k >>= 1) lg += __shfl_xor_sync(~0u, lg, k);
        if (lane == 0) {
          alpha_s[g] = lg == 0.f ? 0.f : 1.f / lg;
          if (!complete)
            p.part_ml[slot + g] = make_float2(m_s[g], lg);
          else if (p.lse)
            p.lse[head0 + g] =
                lg == 0.f ? -INFINITY : (m_s[g] + log2f(lg)) * 0.69314718055994530942f;
        }
      }
      named_bar_sync(1, 128);
#pragma unroll 1
      for (int g = 0; g < nh; g += 4) {
        uint32_t o[4];
        tmem_ld4(tmem + lane_off + SM::kColO + g, o);
        tmem_wait_ld();
        if (t < D) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (g + e >= nh) break;
            const float og = __uint_as_float(o[e]);
            if (complete)
              p.out[(head0 + g + e) * D + t] =
                  __float2bfloat16_rn(alpha_s[g + e] == 0.f ? 0.f : og * alpha_s[g + e]);
            else
              p.part_o[(slot + g + e) * D + t] = og;
          }
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (ab.flag) {
    // something gave up: the copies and MMAs in flight end before their memory is released
    if ((warp == kScoreWarp || warp == kOutWarp) && lane == 0) {
      umma_commit(bar(B_FINAL + (warp == kOutWarp)));
      drain_wait(bar(B_FINAL + (warp == kOutWarp)), 0);
    }
    if (warp == kKeyWarp && lane == 0) {
      for (int i = max(0, loads_s[0] - 2); i < loads_s[0]; ++i)
        drain_wait(bar(B_QFULL + (i & 1)), (i >> 1) & 1);
      for (int i = max(0, loads_s[1] - SM::kKS); i < loads_s[1]; ++i)
        drain_wait(bar(B_KFULL + i % SM::kKS), (i / SM::kKS) & 1);
      for (int i = max(0, loads_s[2] - SM::kVS); i < loads_s[2]; ++i)
        drain_wait(bar(B_VFULL + i % SM::kVS), (i / SM::kVS) & 1);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmemCols);
  }
}

// Block b joins the row that ends in CTA b's share and began in an earlier one's, if there is
// one:  M = max m,  L = sum l 2^(m - M),  O = sum O 2^(m - M) / L  over its CTAs, in order.  The
// row is found while the attention kernel still runs.  One head per warp, D / 32 elements a lane.
constexpr int kJoinThreads = 256;

template <int D, int N>
__global__ void __launch_bounds__(kJoinThreads)
paged_join_kernel(const __grid_constant__ AttParams p) {
  constexpr int E = D / 32;
  __shared__ long long scan_s[kJoinThreads / 32];
  __shared__ Start start_s;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  // (the lengths were there before the attention kernel began)
  const Share sh = find_share<kJoinThreads>(p, b, scan_s, &start_s);
  bool shared = false, aligned = false;
  int c0 = 0, n = 0, nh = 0;
  long long head0 = 0;
  if (b > 0 && b < sh.G) {
    const Start at = start_s;
    const Row row(p, at.len);
    const long long u0 = sh.begin(b), a = u0 - at.i0;        // the row's first unit
    shared = at.i0 > 0 && a + row.count <= sh.begin(b + 1);
    if (shared) {
      c0 = sh.cta_of(a);
      n = b - c0 + 1;
      aligned = sh.begin(c0) == a;                           // c0's share starts with the row
      const int kvh = p.by_chunks(at.hc), chunk = at.hc - kvh * p.chunks;
      nh = min(N, p.group - chunk * N);
      head0 = static_cast<long long>(at.s) * p.c.H + kvh * p.group + chunk * N;
    }
  }
  grid_dependency_wait();
  grid_launch_dependents();
  for (int g = threadIdx.x >> 5; g < nh; g += kJoinThreads / 32) {
    auto part = [&](int i) {
      return (static_cast<long long>(c0 + i) * 2 + (i > 0 || aligned ? 0 : 1)) * N + g;
    };
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (i0 + lane < n) ml = __ldcg(&p.part_ml[part(i0 + lane)]);
      const float top = fmaxf(M, warp_max(ml.x));
      // (the first batch: nothing to rescale; a part without a finite score has the offset
      // kNoOffset and sums of 0)
      const float scale = M > -INFINITY ? ex2(M - top) : 0.f;
      const float wt = ml.x > -INFINITY ? ex2(ml.x - top) : 0.f;
      M = top;
      L = L * scale + wt * ml.y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= scale;
      const int k = min(32, n - i0);
#pragma unroll 4
      for (int i = 0; i < k; ++i) {
        const float w = __shfl_sync(~0u, wt, i);
        const float* src = p.part_o + part(i0 + i) * D + lane * E;
        if constexpr (E == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          acc[0] += w * x.x; acc[1] += w * x.y; acc[2] += w * x.z; acc[3] += w * x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          acc[0] += w * x.x; acc[1] += w * x.y;
        }
      }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(~0u, L, x);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (head0 + g) * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2)
      dst[e / 2] = L == 0.f ? 0u : pack2(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0)
      p.lse[head0 + g] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
  }
}

// ---------------------------------------------------------------------------------- host side
// Checks the description; fills the kernel's view of it.
static int check(const prsink_paged* g, const char* what, Cache* c) {
  if (!g) { set_error("%s: paged is NULL", what); return PRSINK_ERR_ARG; }
  if (g->n_seqs < 0 || g->n_seqs > 65535 || g->n_heads < 1 || g->n_kv_heads < 1 ||
      g->n_heads > 65535 || g->n_heads % g->n_kv_heads || g->head_dim < 2 || g->page_size < 1 ||
      g->n_pages < 1 || g->max_pages < 1 || g->n_sink < 0 || g->window < 0) {
    set_error("%s: invalid paged cache (%d sequences, heads %d / %d, head_dim %d, %d pages of %d, "
              "%d per sequence, sink %d, window %d)", what, g->n_seqs, g->n_heads, g->n_kv_heads,
              g->head_dim, g->n_pages, g->page_size, g->max_pages, g->n_sink, g->window);
    return PRSINK_ERR_ARG;
  }
  if (static_cast<long long>(g->max_pages) * g->page_size > (1ll << 30) ||
      static_cast<long long>(g->n_pages) * g->n_kv_heads > (1ll << 30) ||
      static_cast<long long>(g->n_seqs) * g->n_heads > (1ll << 30)) {
    set_error("%s: paged cache too large (%d sequences x %d heads of %d x %d tokens, %d pages x %d "
              "heads)", what, g->n_seqs, g->n_heads, g->max_pages, g->page_size, g->n_pages,
              g->n_kv_heads);
    return PRSINK_ERR_ARG;
  }
  if (g->rope_mode != 0 && g->rope_mode != 1 && g->rope_mode != 3) {
    set_error("%s: rope_mode must be 0, 1 or 3 (got %d)", what, g->rope_mode);
    return PRSINK_ERR_ARG;
  }
  if (g->rope_mode && !(g->rope_base > 0.f)) {
    set_error("%s: rope_base must be positive", what);
    return PRSINK_ERR_ARG;
  }
  if (g->rope_mode == 3) {
    const int* s = g->rope_split;
    if (s[0] < 0 || s[1] < 0 || s[2] < 0 || (s[0] | s[1] | s[2]) & 1 ||
        s[0] + s[1] + s[2] != g->head_dim || g->grid_h < 1 || g->grid_w < 1 ||
        static_cast<long long>(g->grid_h) * g->grid_w > (1ll << 30)) {
      set_error("%s: rope_split (%d,%d,%d) must be even and sum to head_dim %d, the grid (%dx%d) "
                "positive", what, s[0], s[1], s[2], g->head_dim, g->grid_h, g->grid_w);
      return PRSINK_ERR_ARG;
    }
  }
  if (g->head_dim != 64 && g->head_dim != 128) {
    set_error("%s: head_dim %d not supported (64 or 128)", what, g->head_dim);
    return PRSINK_ERR_UNSUPPORTED;
  }
  if (g->page_size < 128 && g->page_size % 8) {
    set_error("%s: page_size %d not supported (a multiple of 8 below 128, any size from 128 on)",
              what, g->page_size);
    return PRSINK_ERR_UNSUPPORTED;
  }
  *c = Cache{};
  c->n_seqs = g->n_seqs;
  c->H = g->n_heads;
  c->Hkv = g->n_kv_heads;
  c->page_size = g->page_size;
  c->n_pages = g->n_pages;
  c->max_pages = g->max_pages;
  c->capacity = g->max_pages * g->page_size;
  c->n_sink = g->n_sink;
  c->window = g->window;
  return PRSINK_OK;
}

static int check_ptrs(const char* what, std::initializer_list<const void*> bufs,
                      std::initializer_list<const void*> words) {
  for (auto list : {bufs, words})
    for (const void* p : list)
      if (!p) { set_error("%s: null pointer", what); return PRSINK_ERR_ARG; }
  for (const void* p : bufs)
    if (!aligned16(p)) {
      set_error("%s: every K/V/Q/out buffer must be 16-byte aligned", what);
      return PRSINK_ERR_ALIGN;
    }
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) & 3u) {
      set_error("%s: tables and lengths must be 4-byte aligned", what);
      return PRSINK_ERR_ALIGN;
    }
  return PRSINK_OK;
}

// Tokens per CTA and CTAs per token, measured on a B200 (one token per CTA / four):
//   16384 tokens x 56 rows of 256 B (470 MB)   91.9 us / 81.5 us (5.8 TB/s; 84-87 when inputs change)
//   2700 tokens x 120 rows (166 MB)            29.8 us (5.6 TB/s) / 38.1 us
//   64 tokens x 56 rows                         3.7 us / 6.8 us; one token split over 4: 3.3 us
// Short tokens share a CTA (and the latency of looking up their place) while the grid still fills
// the device four times over; where there are few tokens, each is split down to one pass of rows.
template <int D>
static void launch_append(const AppendParams& p, cudaStream_t st) {
  constexpr int R = kAppendThreads / (D / 8);
  const int rows = (p.q ? p.c.H : 0) + 2 * p.c.Hkv;
  int n_sm = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (2 * rows <= 7 * R && p.n_tokens >= 16 * n_sm) {
    launch_dependent(paged_append_kernel<D, 4>, dim3((p.n_tokens + 3) / 4), kAppendThreads, 0, st,
                     p);
    return;
  }
  int split = 2 * n_sm / p.n_tokens;
  split = split < 1 ? 1 : (split > (rows + R - 1) / R ? (rows + R - 1) / R : split);
  launch_dependent(paged_append_kernel<D, 1>, dim3(p.n_tokens, split), kAppendThreads, 0, st, p);
}

// Columns of the score tile (query heads of a key head, in chunks of at most 64), CTAs and
// scratch of an attention call.
struct AttPlan {
  int N, grid;
  size_t o, total;                         // byte offset of the partial O behind m and l
};

static AttPlan att_plan(const Cache& c, int D) {
  AttPlan a{};
  const int group = c.H / c.Hkv;
  a.N = group <= 16 ? 16 : (group <= 32 ? 32 : 64);
  int n_sm = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  a.grid = n_sm;
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t parts = static_cast<size_t>(a.grid) * 2 * a.N;
  a.o = up(parts * sizeof(float2));
  a.total = a.o + up(parts * D * sizeof(float));
  return a;
}

template <int D_, int N_>
struct Shape {
  static constexpr int d = D_, n = N_;
};

template <int D, int N>
static int launch_attention(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                            const AttParams& p, int grid, cudaStream_t st) {
  const int smem = Smem<D, N>::kBytes + 1024;
  static std::atomic<bool> allowed[64];      // (host threads may call at once)
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !allowed[dev]) {
    if (cudaFuncSetAttribute(paged_attention_kernel<D, N>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return check_launch("prsink_paged_attention");
    if (dev >= 0 && dev < 64) allowed[dev] = true;
  }
  launch_dependent(paged_attention_kernel<D, N>, grid, kAttThreads, smem, st, mq, mk, mv, p);
  count_launch();
  if (!p.whole_rows) {
    launch_dependent(paged_join_kernel<D, N>, grid, kJoinThreads, 0, st, p);
    count_launch();
  }
  return check_launch("prsink_paged_attention");
}

}  // namespace paged
}  // namespace prsink

using namespace prsink;

extern "C" int prsink_paged_append(const prsink_paged* paged, const void* k_new,
                                   const void* v_new, long long k_stride, long long v_stride,
                                   void* k_pages, void* v_pages, const int* page_table,
                                   const int* seq_lens, int n_tokens, const int* cu_new,
                                   const void* q, long long q_stride, void* q_rot,
                                   void* stream) {
  using namespace prsink::paged;
  const char* what = "prsink_paged_append";
  AppendParams p{};
  int rc = check(paged, what, &p.c);
  if (rc) return rc;
  const int D = paged->head_dim;
  if (n_tokens < 0 || (!cu_new && n_tokens != paged->n_seqs)) {
    set_error("%s: n_tokens %d (without cu_new it is n_seqs = %d)", what, n_tokens,
              paged->n_seqs);
    return PRSINK_ERR_ARG;
  }
  if (n_tokens == 0 || paged->n_seqs == 0) return PRSINK_OK;
  rc = check_ptrs(what, {k_new, v_new, k_pages, v_pages}, {page_table, seq_lens});
  if (rc) return rc;
  if (!q != !q_rot) {
    set_error("%s: q and q_rot go together", what);
    return PRSINK_ERR_ARG;
  }
  if (!aligned16(q) || !aligned16(q_rot) || (reinterpret_cast<uintptr_t>(cu_new) & 3u)) {
    set_error("%s: q and q_rot must be 16-byte aligned, cu_new 4-byte aligned", what);
    return PRSINK_ERR_ALIGN;
  }
  const long long kv_row = static_cast<long long>(paged->n_kv_heads) * D;
  const long long q_row = static_cast<long long>(paged->n_heads) * D;
  if (k_stride < kv_row || v_stride < kv_row || (k_stride | v_stride) % 8 ||
      (q && (q_stride < q_row || q_stride % 8)) || (q == q_rot && q && q_stride != q_row)) {
    set_error("%s: token strides %lld, %lld, %lld must be multiples of 8, at least one token "
              "long (in place, q is contiguous)", what, k_stride, v_stride, q_stride);
    return PRSINK_ERR_ARG;
  }
  const long long pool = 2ll * paged->n_pages * paged->n_kv_heads * paged->page_size * D;
  const Span table{page_table, 4ll * paged->n_seqs * paged->max_pages};
  const Span lens{seq_lens, 4ll * paged->n_seqs}, cu{cu_new, 4ll * (paged->n_seqs + 1)};
  const Span kp{k_pages, pool}, vp{v_pages, pool}, rot{q_rot, 2 * q_row * n_tokens};
  // (new rows may lie in the pages themselves: a row that is written must not be one that is read)
  if (overlap_any(kp, {vp, table, lens, cu}) || overlap_any(vp, {table, lens, cu}) ||
      overlap_any(rot, {kp, vp, table, lens, cu, {k_new, 2 * kv_row, n_tokens, 2 * k_stride},
                        {v_new, 2 * kv_row, n_tokens, 2 * v_stride}}) ||
      (q != q_rot && overlap(rot, {q, 2 * q_row, n_tokens, 2 * q_stride}))) {
    set_error("%s: k_pages, v_pages and q_rot must be buffers of their own (q_rot may be q itself)",
              what);
    return PRSINK_ERR_ARG;
  }
  p.c.table = page_table;
  p.c.lens = seq_lens;
  p.c.status = status_word_ptr();
  if (!p.c.status) return PRSINK_ERR_LAUNCH;
  p.n_tokens = n_tokens;
  p.cu = cu_new;
  p.k = static_cast<const __nv_bfloat16*>(k_new);
  p.v = static_cast<const __nv_bfloat16*>(v_new);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  p.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  p.q_rot = static_cast<__nv_bfloat16*>(q_rot);
  p.rope_mode = paged->rope_mode;
  if (p.rope_mode) {
    const int one[3] = {D, 0, 0};
    const int* split = p.rope_mode == 3 ? paged->rope_split : one;
    int at = 0;
    for (int ax = 0; ax < 3; ++ax) {
      p.rd[ax] = split[ax] / 2;
      rope_frequencies(paged->rope_base, split[ax], p.inv_pi_freq + at);
      at += p.rd[ax];
    }
    if (p.rope_mode == 3) {
      p.grid_w = paged->grid_w;
      p.L_f = paged->grid_h * paged->grid_w;
    }
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D == 128) launch_append<128>(p, st);
  else launch_append<64>(p, st);
  count_launch();
  return check_launch(what);
}

extern "C" long long prsink_paged_attention_scratch_bytes(const prsink_paged* paged) {
  using namespace prsink::paged;
  Cache c;
  if (check(paged, "prsink_paged_attention_scratch_bytes", &c)) return -1;
  return static_cast<long long>(att_plan(c, paged->head_dim).total);
}

extern "C" int prsink_paged_attention(const prsink_paged* paged, const void* q,
                                      const void* k_pages, const void* v_pages,
                                      const int* page_table, const int* seq_lens, void* out,
                                      float* lse, void* scratch, long long scratch_bytes,
                                      void* stream) {
  using namespace prsink::paged;
  const char* what = "prsink_paged_attention";
  AttParams p{};
  int rc = check(paged, what, &p.c);
  if (rc) return rc;
  if (p.c.n_seqs == 0) return PRSINK_OK;
  rc = check_ptrs(what, {q, k_pages, v_pages, out}, {page_table, seq_lens});
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) {
    set_error("%s: lse must be 4-byte aligned", what);
    return PRSINK_ERR_ALIGN;
  }
  const int D = paged->head_dim;
  const AttPlan pl = att_plan(p.c, D);
  if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) ||
      scratch_bytes < static_cast<long long>(pl.total)) {
    set_error("%s: scratch must be 256-byte aligned and hold %zu bytes (got %lld)", what, pl.total,
              scratch_bytes);
    return PRSINK_ERR_ARG;
  }
  // CTAs that share a row read its queries and write its results at different times
  const long long pool = 2ll * p.c.n_pages * p.c.Hkv * p.c.page_size * D;
  const long long heads = static_cast<long long>(p.c.n_seqs) * p.c.H;
  const Span in[] = {{q, 2 * heads * D}, {k_pages, pool}, {v_pages, pool},
                     {page_table, 4ll * p.c.n_seqs * p.c.max_pages}, {seq_lens, 4ll * p.c.n_seqs}};
  const Span o{out, 2 * heads * D}, l{lse, 4 * heads};
  const Span sc{scratch, static_cast<long long>(pl.total)};
  bool own = !overlap_any(o, {l, sc}) && !overlap(l, sc);
  for (const Span& x : in) own = own && !overlap(o, x) && !overlap(l, x) && !overlap(sc, x);
  if (!own) {
    set_error("%s: out, lse and scratch must be buffers of their own", what);
    return PRSINK_ERR_ARG;
  }
  p.c.table = page_table;
  p.c.lens = seq_lens;
  p.c.status = status_word_ptr();
  if (!p.c.status) return PRSINK_ERR_LAUNCH;
  p.group = p.c.H / p.c.Hkv;
  p.chunks = (p.group + pl.N - 1) / pl.N;
  const int ps = p.c.page_size;
  p.tiles_per_page = ps < kTile ? 0 : (ps + kTile - 1) / kTile;
  p.pages_per_tile = ps < kTile ? kTile / ps : 1;
  p.tile_tokens = ps < kTile ? p.pages_per_tile * ps : kTile;
  p.box_rows = ps < kTile ? ps : kTile;
  // tiles of the longest row: the table's capacity, or the sinks and the window with the tiles
  // that they begin and end in
  auto tiles_of = [&](long long tokens) {
    const long long in_pages = (tokens + ps - 1) / ps;
    return p.tiles_per_page ? in_pages * p.tiles_per_page
                            : (in_pages + p.pages_per_tile - 1) / p.pages_per_tile;
  };
  long long longest = tiles_of(p.c.capacity);
  if (p.c.window > 0) {
    const long long bounded = tiles_of(p.c.n_sink) + tiles_of(p.c.window) + 1;
    if (bounded < longest) longest = bounded;
  }
  p.whole_rows = longest <= kWholeRow;
  p.by_tile.set(ps < kTile ? p.tile_tokens : ps);
  p.by_tiles_per_page.set(p.tiles_per_page ? p.tiles_per_page : 1);
  p.by_chunks.set(p.chunks);
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.timeout_ns = 2000000000ull;
  if (const long long ns = take_debug_stall()) {
    p.debug_stall = 1;
    p.timeout_ns = static_cast<unsigned long long>(ns);
  }
  char* base = static_cast<char*>(scratch);
  p.part_ml = reinterpret_cast<float2*>(base);
  p.part_o = reinterpret_cast<float*>(base + pl.o);
  CUtensorMap mq, mk, mv;
  const uint64_t rows = static_cast<uint64_t>(p.c.n_pages) * p.c.Hkv;
  rc = make_map(&mq, q, D, p.group, static_cast<uint64_t>(p.c.n_seqs) * p.c.Hkv, 2ull * D,
                2ull * D * p.group, pl.N, 1);
  p.one_box = ps % 8 == 0;
  p.group_bytes = p.one_box ? D / 64 * 1024 : 1024;
  p.panel_bytes = p.one_box && D > 64 ? 1024 : kTile * 128;
  auto map = [&](CUtensorMap* m, const void* pages) {
    return p.one_box ? make_map_rows(m, pages, D, ps, rows, p.box_rows / 8)
                     : make_map(m, pages, D, ps, rows, 2ull * D, 2ull * D * ps, p.box_rows, 1);
  };
  if (!rc) rc = map(&mk, k_pages);
  if (!rc) rc = map(&mv, v_pages);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto tag) { return launch_attention<decltype(tag)::d, decltype(tag)::n>(
      mq, mk, mv, p, pl.grid, st); };
  if (D == 128)
    return pl.N == 16 ? go(Shape<128, 16>{}) : pl.N == 32 ? go(Shape<128, 32>{})
                                                          : go(Shape<128, 64>{});
  return pl.N == 16 ? go(Shape<64, 16>{}) : pl.N == 32 ? go(Shape<64, 32>{})
                                                       : go(Shape<64, 64>{});
}
