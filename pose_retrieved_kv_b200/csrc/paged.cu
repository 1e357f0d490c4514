// Paged K/V cache: the append of new tokens with the rotary embedding applied on the way, and
// the attention of one new token per sequence over the pages.
#include <cuda_bf16.h>

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
  const int n = c.lens[s];
  if (n >= 0 && n <= c.capacity) return n;
  atomicOr(c.status, kStatusPage);
  return n < 0 ? 0 : c.capacity;
}

// ------------------------------------------------------------------------------------ append
// HBM-bound copy of n * (H + 2 Hkv) rows of d bf16, K and q rotated on the way.  A CTA takes
// kTok tokens: their places and the cos / sin of their positions (f64 angles, shared by every
// head) go to shared memory once, then each thread owns one 16-byte chunk of a row (four pairs,
// their cos / sin in registers per token) and walks the rows of the token.
constexpr int kAppendThreads = 256;

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

template <int D, int kTok>
__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int C = D / 8;                 // 16-byte chunks of a row
  constexpr int R = kAppendThreads / C;    // rows per pass
  __shared__ int tok_pos[kTok];            // position, or -1: nothing to do
  __shared__ long long tok_row[kTok];      // (page * Hkv) * page_size + offset, or -1: no page
  __shared__ __align__(16) float2 tab[kTok][D / 2];
  const int t0 = blockIdx.x * kTok;
  if (threadIdx.x < kTok) {
    const int i = t0 + threadIdx.x;
    int pos = -1;
    long long row = -1;
    if (i < p.n_tokens) {
      int s = -1, back = 1;                // the token is the back-th last of sequence s
      if (!p.cu) {
        s = i;
      } else if (i < p.cu[p.c.n_seqs]) {
        int lo = 0, hi = p.c.n_seqs;       // the last s with cu[s] <= i
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (p.cu[mid] <= i) lo = mid; else hi = mid;
        }
        if (p.cu[lo] <= i && i < p.cu[lo + 1]) {
          s = lo;
          back = p.cu[lo + 1] - i;
        } else {
          atomicOr(p.c.status, kStatusPage);
        }
      }
      if (s >= 0) {
        const int n = p.c.lens[s];
        pos = n - back;
        if (n < 0 || n > p.c.capacity || pos < 0) {
          if (!(n == 0 && !p.cu)) atomicOr(p.c.status, kStatusPage);
          pos = -1;
        } else {
          const int page = p.c.table[static_cast<long long>(s) * p.c.max_pages +
                                     pos / p.c.page_size];
          if (page >= 0 && page < p.c.n_pages)
            row = static_cast<long long>(page) * p.c.Hkv * p.c.page_size + pos % p.c.page_size;
          else
            atomicOr(p.c.status, kStatusPage);
        }
      }
    }
    tok_pos[threadIdx.x] = pos;
    tok_row[threadIdx.x] = row;
  }
  __syncthreads();
  if (p.rope_mode) {
    for (int e = threadIdx.x; e < kTok * (D / 2); e += kAppendThreads) {
      const int t = e / (D / 2), j = e % (D / 2);
      int x = tok_pos[t];
      if (x < 0) continue;
      if (p.rope_mode == 3) {
        const int f = x / p.L_f, in = x - f * p.L_f, y = in / p.grid_w;
        x = j < p.rd[0] ? f : (j < p.rd[0] + p.rd[1] ? y : in - y * p.grid_w);
      }
      double sn, cs;
      sincospi(static_cast<double>(x) * p.inv_pi_freq[j], &sn, &cs);   // exact reduction
      tab[t][j] = make_float2(static_cast<float>(cs), static_cast<float>(sn));
    }
    __syncthreads();
  }
  const int c = threadIdx.x % C, r0 = threadIdx.x / C;
  const int Hq = p.q ? p.c.H : 0, Hkv = p.c.Hkv;
  const int rows = Hq + 2 * Hkv;
  // rows of this CTA: an equal share of the token's rows per blockIdx.y
  const int per = (rows + gridDim.y - 1) / gridDim.y;
  const int ra = blockIdx.y * per, rb = min(rows, ra + per);
#pragma unroll 1
  for (int t = 0; t < kTok; ++t) {
    if (tok_pos[t] < 0) continue;
    const long long i = t0 + t, row = tok_row[t];
    float2 cs[4];
    if (p.rope_mode) {
      const float4* tp = reinterpret_cast<const float4*>(&tab[t][4 * c]);
      const float4 a = tp[0], b = tp[1];
      cs[0] = make_float2(a.x, a.y); cs[1] = make_float2(a.z, a.w);
      cs[2] = make_float2(b.x, b.y); cs[3] = make_float2(b.z, b.w);
    }
#pragma unroll 4
    for (int r = ra + r0; r < rb; r += R) {
      const __nv_bfloat16* src;
      __nv_bfloat16* dst = nullptr;
      if (r < Hq) {
        src = p.q + i * p.q_stride + static_cast<long long>(r) * D;
        dst = p.q_rot + (i * Hq + r) * D;
      } else if (r < Hq + Hkv) {
        src = p.k + i * p.k_stride + static_cast<long long>(r - Hq) * D;
        if (row >= 0) dst = p.k_pages + (row + static_cast<long long>(r - Hq) * p.c.page_size) * D;
      } else {
        src = p.v + i * p.v_stride + static_cast<long long>(r - Hq - Hkv) * D;
        if (row >= 0)
          dst = p.v_pages + (row + static_cast<long long>(r - Hq - Hkv) * p.c.page_size) * D;
      }
      if (!dst) continue;
      uint4 x = reinterpret_cast<const uint4*>(src)[c];
      if (p.rope_mode && r < Hq + Hkv) x = rotate_chunk(x, cs);
      reinterpret_cast<uint4*>(dst)[c] = x;
    }
  }
}

// --------------------------------------------------------------------------------- attention
// One CTA per (sequence, query head); each warp walks every fourth key with a running maximum
// and sum, lanes across the head dimension; the four warps are joined in shared memory.
template <int D>
__global__ void __launch_bounds__(128)
paged_attention_kernel(const Cache cc, const __nv_bfloat16* q, const __nv_bfloat16* k_pages,
                       const __nv_bfloat16* v_pages, __nv_bfloat16* out, float* lse,
                       float scale_log2) {
  constexpr int E = D / 32;
  const int s = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = h / (cc.H / cc.Hkv);
  const int len = seq_len(cc, s);
  const int win0 = cc.window > 0 ? max(0, len - cc.window) : 0;
  const long long qrow = (static_cast<long long>(s) * cc.H + h) * D;
  float qv[E], acc[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(q[qrow + lane * E + e]) * scale_log2;
    acc[e] = 0.f;
  }
  for (int t = warp; t < len; t += 4) {
    if (t >= cc.n_sink && t < win0) continue;
    const int page = cc.table[static_cast<long long>(s) * cc.max_pages + t / cc.page_size];
    if (page < 0 || page >= cc.n_pages) {
      if (lane == 0) atomicOr(cc.status, kStatusPage);
      continue;
    }
    const long long row = ((static_cast<long long>(page) * cc.Hkv + kvh) * cc.page_size +
                           t % cc.page_size) * D + lane * E;
    float x = 0.f;
    for (int e = 0; e < E; ++e) x += qv[e] * __bfloat162float(k_pages[row + e]);
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    const float mn = fmaxf(m, x), a = exp2f(m - mn), w = exp2f(x - mn);
    l = l * a + w;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * __bfloat162float(v_pages[row + e]);
    m = mn;
  }
  __shared__ float sm[4], sl[4], so[4][D];
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
  __syncthreads();
  const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float L = 0.f, w[4];
  for (int i = 0; i < 4; ++i) {
    w[i] = sm[i] > -INFINITY ? exp2f(sm[i] - M) : 0.f;
    L += w[i] * sl[i];
  }
  if (threadIdx.x < D) {
    float o = 0.f;
    for (int i = 0; i < 4; ++i) o += w[i] * so[i][threadIdx.x];
    out[qrow + threadIdx.x] = __float2bfloat16_rn(L > 0.f ? o / L : 0.f);
  }
  if (lse && threadIdx.x == 0)
    lse[static_cast<long long>(s) * cc.H + h] =
        L > 0.f ? (M + log2f(L)) * 0.69314718055994530942f : -INFINITY;
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
      static_cast<long long>(g->n_pages) * g->n_kv_heads > (1ll << 30)) {
    set_error("%s: paged cache too large (%d x %d tokens per sequence, %d pages x %d heads)", what,
              g->max_pages, g->page_size, g->n_pages, g->n_kv_heads);
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

template <int D>
static void launch_append(const AppendParams& p, cudaStream_t st) {
  paged_append_kernel<D, 1><<<dim3(p.n_tokens, 1), kAppendThreads, 0, st>>>(p);
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
    const double log2_base = std::log2(static_cast<double>(paged->rope_base));
    int at = 0;
    for (int ax = 0; ax < 3; ++ax) {
      p.rd[ax] = split[ax] / 2;
      for (int j = 0; j < p.rd[ax]; ++j)
        p.inv_pi_freq[at++] = std::exp2(-(2.0 * j / split[ax]) * log2_base) *
                              0.31830988618379067154;
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
  return 0;
}

extern "C" int prsink_paged_attention(const prsink_paged* paged, const void* q,
                                      const void* k_pages, const void* v_pages,
                                      const int* page_table, const int* seq_lens, void* out,
                                      float* lse, void* scratch, long long scratch_bytes,
                                      void* stream) {
  using namespace prsink::paged;
  const char* what = "prsink_paged_attention";
  Cache c;
  int rc = check(paged, what, &c);
  if (rc) return rc;
  if (c.n_seqs == 0) return PRSINK_OK;
  rc = check_ptrs(what, {q, k_pages, v_pages, out}, {page_table, seq_lens});
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) {
    set_error("%s: lse must be 4-byte aligned", what);
    return PRSINK_ERR_ALIGN;
  }
  c.table = page_table;
  c.lens = seq_lens;
  c.status = status_word_ptr();
  if (!c.status) return PRSINK_ERR_LAUNCH;
  const float scale_log2 =
      static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(paged->head_dim)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(c.n_seqs, c.H);
  auto launch = [&](auto kernel) {
    kernel<<<grid, 128, 0, st>>>(c, static_cast<const __nv_bfloat16*>(q),
                                 static_cast<const __nv_bfloat16*>(k_pages),
                                 static_cast<const __nv_bfloat16*>(v_pages),
                                 static_cast<__nv_bfloat16*>(out), lse, scale_log2);
  };
  if (paged->head_dim == 128) launch(paged_attention_kernel<128>);
  else launch(paged_attention_kernel<64>);
  count_launch();
  return check_launch(what);
}
