// Gradient of the PR-Sink attention with respect to its raw queries, raw keys and values.
//
//   P = exp(s - lse),  delta_i = sum_c d_out_ic out_ic,  dP = d_out V^T,
//   dS = P o (dP - delta) / sqrt(d),  dV = P^T d_out,  dK = R^T (dS^T q~),  dQ = R^T (dS k~)
//
// with q~, k~ the rotated queries and keys and R^T the inverse rotation of the row's position.
#include <cuda_bf16.h>

#include <cmath>

#include "prsink_internal.cuh"

namespace prsink {
namespace bwd {

constexpr int kMaxSlots = 3 + PRSINK_MAX_RING;
constexpr int BM = 128;                    // rows of the statistics are padded to this

struct Params {
  int H, L_blk, L_pad, T, L_f, grid_w;
  int n_slots;
  int slot_start[kMaxSlots + 1];
  int slot_frame[kMaxSlots];
  unsigned valid_mask, grad_mask;
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
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  // scratch
  __nv_bfloat16* k_rot;                    // [H][T][d], rows of empty slots zero
  __nv_bfloat16* q_rot;                    // [H][L_blk][d]
  float2* tab;                             // [T][d/2] (cos, sin) of every key row's position
  float* lse2;                             // [H][L_pad] lse in log2 units; +inf: no probability
  float* delta;                            // [H][L_pad]
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

// Keys rotated into k_rot (rows of empty slots zeroed: dS is 0 there, but 0 * NaN is not) and
// the table of the rows' cos / sin.  A CTA takes 256 / C rows, a thread one 16-byte chunk of a
// row, whose four f64 angles serve every head.
template <int D>
__global__ void __launch_bounds__(256) prep_keys_kernel(const __grid_constant__ Params p) {
  constexpr int C = D / 8, R = 256 / C;
  const int c = threadIdx.x % C, row = blockIdx.x * R + threadIdx.x / C;
  if (row >= p.T) return;
  const int s = slot_of(row, p), u = row - p.slot_start[s];
  const bool live = (live_mask(p) >> s) & 1u;
  const int frame = p.slot_frame[s] + u / p.L_f, tok = u % p.L_f;
  float2 cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * c + i;
    int x;
    if (p.rope_mode == 3)
      x = j < p.rd[0] ? frame : (j < p.rd[0] + p.rd[1] ? tok / p.grid_w : tok % p.grid_w);
    else
      x = frame * p.L_f + tok;
    double sn, co;
    sincospi(static_cast<double>(x) * p.inv_pi_freq[j], &sn, &co);
    cs[i] = make_float2(static_cast<float>(co), static_cast<float>(sn));
    p.tab[static_cast<size_t>(row) * (D / 2) + j] = cs[i];
  }
  const size_t step = static_cast<size_t>(p.T) * C;
  const size_t at = static_cast<size_t>(row) * C + c;
#pragma unroll 4
  for (int h = 0; h < p.H; ++h) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live) {
      x = reinterpret_cast<const uint4*>(p.k)[at + h * step];
      uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = turn(lo16(w[i]), hi16(w[i]), cs[i], 1.f);
        w[i] = pack2(y.x, y.y);
      }
    }
    reinterpret_cast<uint4*>(p.k_rot)[at + h * step] = x;
  }
}

// Queries rotated into q_rot (head-major) and the rows' statistics.  C threads per row.
template <int D>
__global__ void __launch_bounds__(256) prep_queries_kernel(const __grid_constant__ Params p) {
  constexpr int C = D / 8, R = 256 / C;
  const int c = threadIdx.x % C, i = blockIdx.x * R + threadIdx.x / C, h = blockIdx.y;
  float dot = 0.f;
  if (i < p.L_blk) {
    const size_t at = (static_cast<size_t>(i) * p.H + h) * C + c;
    uint4 x = reinterpret_cast<const uint4*>(p.q)[at];
    const uint4 o = reinterpret_cast<const uint4*>(p.out)[at];
    const uint4 g = reinterpret_cast<const uint4*>(p.d_out)[at];
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
    const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
    const float2* cs = p.tab + static_cast<size_t>(p.q_row + i) * (D / 2) + 4 * c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = turn(lo16(w[e]), hi16(w[e]), cs[e], 1.f);
      w[e] = pack2(y.x, y.y);
      dot += lo16(ow[e]) * lo16(gw[e]) + hi16(ow[e]) * hi16(gw[e]);
    }
    reinterpret_cast<uint4*>(p.q_rot)[(static_cast<size_t>(h) * p.L_blk + i) * C + c] = x;
  }
#pragma unroll
  for (int o = C / 2; o; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
  if (c == 0 && i < p.L_pad) {
    float l = INFINITY;
    if (i < p.L_blk) {
      l = p.lse[static_cast<size_t>(h) * p.L_blk + i] * 1.4426950408889634f;
      if (!(l > -INFINITY)) l = INFINITY;            // a row without keys
    }
    p.lse2[static_cast<size_t>(h) * p.L_pad + i] = l;
    p.delta[static_cast<size_t>(h) * p.L_pad + i] = dot;
  }
}

template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* src, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = __bfloat162float(src[e]);
}
template <int E>
__device__ __forceinline__ float dot_row(const float (&a)[E], const float (&b)[E]) {
  float x = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) x += a[e] * b[e];
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// One warp per query row: dQ.
template <int D>
__global__ void __launch_bounds__(256) dq_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y;
  if (i >= p.L_blk) return;
  const unsigned vm = live_mask(p);
  float q[E], g[E], k[E], v[E], acc[E] = {};
  load_row<E>(p.q_rot + (static_cast<size_t>(h) * p.L_blk + i) * D + lane * E, q);
  load_row<E>(p.d_out + (static_cast<size_t>(i) * p.H + h) * D + lane * E, g);
  const float l2 = p.lse2[static_cast<size_t>(h) * p.L_pad + i];
  const float dl = p.delta[static_cast<size_t>(h) * p.L_pad + i];
  for (int s = 0; s < p.n_slots; ++s) {
    if (!((vm >> s) & 1u)) continue;
    for (int r = p.slot_start[s]; r < p.slot_start[s + 1]; ++r) {
      const size_t at = (static_cast<size_t>(h) * p.T + r) * D + lane * E;
      load_row<E>(p.k_rot + at, k);
      load_row<E>(p.v + at, v);
      const float pr = exp2f(dot_row<E>(q, k) * p.scale_log2 - l2);
      const float ds = pr * (dot_row<E>(g, v) - dl) * p.scale;
      for (int e = 0; e < E; ++e) acc[e] += ds * k[e];
    }
  }
  const float2* cs = p.tab + static_cast<size_t>(p.q_row + i) * (D / 2) + lane * (E / 2);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.dq + (static_cast<size_t>(i) * p.H + h) * D) +
                  lane * (E / 2);
  for (int e = 0; e < E / 2; ++e) {
    const float2 y = turn(acc[2 * e], acc[2 * e + 1], cs[e], -1.f);
    dst[e] = pack2(y.x, y.y);
  }
}

// One warp per key row: dK and dV.
template <int D>
__global__ void __launch_bounds__(256) dkv_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, r = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y;
  if (r >= p.T) return;
  const int s = slot_of(r, p);
  if (!((p.grad_mask >> s) & 1u)) return;
  float q[E], g[E], k[E], v[E], ak[E] = {}, av[E] = {};
  const size_t at = (static_cast<size_t>(h) * p.T + r) * D + lane * E;
  if ((live_mask(p) >> s) & 1u) {
    load_row<E>(p.k_rot + at, k);
    load_row<E>(p.v + at, v);
    for (int i = 0; i < p.L_blk; ++i) {
      load_row<E>(p.q_rot + (static_cast<size_t>(h) * p.L_blk + i) * D + lane * E, q);
      load_row<E>(p.d_out + (static_cast<size_t>(i) * p.H + h) * D + lane * E, g);
      const float l2 = p.lse2[static_cast<size_t>(h) * p.L_pad + i];
      const float dl = p.delta[static_cast<size_t>(h) * p.L_pad + i];
      const float pr = exp2f(dot_row<E>(q, k) * p.scale_log2 - l2);
      const float ds = pr * (dot_row<E>(g, v) - dl) * p.scale;
      for (int e = 0; e < E; ++e) {
        av[e] += pr * g[e];
        ak[e] += ds * q[e];
      }
    }
  }
  const float2* cs = p.tab + static_cast<size_t>(r) * (D / 2) + lane * (E / 2);
  for (int e = 0; e < E / 2; ++e) {
    const float2 y = turn(ak[2 * e], ak[2 * e + 1], cs[e], -1.f);
    reinterpret_cast<uint32_t*>(p.dk + at)[e] = pack2(y.x, y.y);
    reinterpret_cast<uint32_t*>(p.dv + at)[e] = pack2(av[2 * e], av[2 * e + 1]);
  }
}

// ---------------------------------------------------------------------------------- host side
struct Plan {                              // scratch regions, each 256-byte aligned
  size_t k_rot, q_rot, tab, lse2, delta, total;
};

static Plan plan(const Geometry& g, int H, int D) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t pad = (g.L_blk + BM - 1) / BM * BM;
  Plan p{};
  p.k_rot = 0;
  p.q_rot = p.k_rot + up(static_cast<size_t>(H) * g.T * D * 2);
  p.tab = p.q_rot + up(static_cast<size_t>(H) * g.L_blk * D * 2);
  p.lse2 = p.tab + up(static_cast<size_t>(g.T) * (D / 2) * 8);
  p.delta = p.lse2 + up(H * pad * 4);
  p.total = p.delta + up(H * pad * 4);
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
  const double log2_base = std::log2(static_cast<double>(L->rope_base));
  int at = 0;
  for (int ax = 0; ax < 3; ++ax) {
    p.rd[ax] = split[ax] / 2;
    for (int j = 0; j < p.rd[ax]; ++j)
      p.inv_pi_freq[at++] = std::exp2(-(2.0 * j / split[ax]) * log2_base) *
                            0.31830988618379067154;
  }
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
}

template <int D>
static int launch(const Params& p, cudaStream_t st) {
  constexpr int R = 256 / (D / 8);
  const char* what = "prsink_attention_backward";
  prep_keys_kernel<D><<<(p.T + R - 1) / R, 256, 0, st>>>(p);
  prep_queries_kernel<D><<<dim3(p.L_pad / R, p.H), 256, 0, st>>>(p);
  dq_kernel<D><<<dim3((p.L_blk + 7) / 8, p.H), 256, 0, st>>>(p);
  count_launch(3);
  if (p.grad_mask) {
    dkv_kernel<D><<<dim3((p.T + 7) / 8, p.H), 256, 0, st>>>(p);
    count_launch();
  }
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
  p.lse2 = reinterpret_cast<float*>(base + pl.lse2);
  p.delta = reinterpret_cast<float*>(base + pl.delta);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return D == 128 ? launch<128>(p, st) : launch<64>(p, st);
}
