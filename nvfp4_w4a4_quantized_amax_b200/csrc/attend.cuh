// attend.cuh — what the attention kernels over the NVFP4 cache share: their parameters, the
// visibility rule, the form of the scores and the partial results of split keys.
//
// For a query row (one query of one head) and the keys j of a window
//   x_j = scale * sum_d q_d K^_jd,            K^ = e2m1 * s * g_K + mu   (not rounded)
//   s_j = cap * tanh(x_j / cap) - slope * |q_pos - k_pos|       (cap, slope optional)
//   O   = sum_j p_j V^_j,  p = softmax over the visible keys,    V^ = e2m1 * s * g_V
// e2m1 * s is exact in binary16, so the matrix products run on it: K's mean is one constant
// per (row, slot), added to the scores as q . mu, and g_K is a factor of the scores.  The
// queries enter as binary16 after a power-of-two scaling of each row that puts its largest
// element in [2^14, 2^15): exact for elements down to 2^-29 of it and within 2^-40 of it
// below.  The weights enter as binary16 with a row's largest between 2^10 and 2^14: rounded by
// 2^-11 of their value at most (bf16: 2^-8), or by 2^-35 of the largest where they are small.  g_V
// differs from slot to slot: relative to the window's largest it goes into the exponent of the
// weights (see SlotView::lg; these bounds are for the weights so scaled), and O is multiplied by
// the largest at the end.  Scores, softmax
// statistics and sums are FP32.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace attend {

constexpr int kD = 128;
constexpr int kMaxFoldedDrafts = 4;  // more are taken as the parts are joined
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// The running maximum follows the true one only when that grew by more than 2^kLazy, so O is
// rarely rescaled; a row's largest weight is then between 2^kUp and 2^(kUp + kLazy) = 2^14.
constexpr float kLazy = 4.0f, kUp = 10.0f;

struct Params {
  const uint8_t* base;
  int64_t off_k_codes, off_v_codes, off_k_scales, off_v_scales, off_mu, off_gscale, off_tokens;
  int64_t chunk;  // tokens of a slot
  int32_t heads, group;  // cache heads, query heads of each
  FastDiv by_group;
  int32_t n_slots;
  int32_t slots[kMaxWindowSlots];
  int32_t tokens[kMaxWindowSlots];
  int32_t pos[kMaxWindowSlots];       // position of the slot's first token
  int32_t step_end[kMaxWindowSlots];  // key steps (kernel's own size) up to and with the slot
  int32_t steps, splits;              // steps in all, and CTAs that share them
  const uint8_t* q;                   // bf16 [tq][heads * group][128]
  int64_t q_pitch;                    // bytes
  int64_t rows;                       // tq * group rows of each cache head, query by query
  float scale, cap;
  const float* slopes;
  int32_t causal, window, prefix;     // window: 0 none
  int32_t q_pos0;
  const int32_t* q_pos;
  const int32_t* q_doc;
  const int32_t* k_doc;
  // a tree of drafted tokens (parents == nullptr: none)
  const int32_t* parents;
  const uint8_t* k_new;
  const uint8_t* v_new;
  int64_t new_pitch;  // bytes
  int32_t drafts;
  uint8_t* o;         // bf16 [tq][heads * group][128]
  int64_t o_pitch;    // bytes
  float* lse;         // [heads * group][tq], nullable
  int64_t tq;
  // partial results of `parts` sets of keys: O (normalised) [part][cache head][row][128] and
  // log2 of the sum [part][cache head][row].  The drafts come in as the parts are joined; where one
  // CTA has the whole window and there are few of them (fold), it takes them itself and keeps
  // their result as the one part until it joins it
  int32_t parts;
  bool fold;
  float* part_o;
  float* part_l;
  unsigned* status;
};

// Constants of one listed slot.
struct SlotView {
  float gk;    // g_K
  float lg;    // log2(g_V / largest g_V): p 2^lg goes to the product, p to the sum
  float inv;   // 2^-lg
  int16_t ok;     // the slot holds the stated number of tokens
  int16_t vzero;  // its values count as zero: g_V is 0 or under 2^-60 of the largest
};

// Reads the listed slots' scales, one warp; *top_out = the largest g_V, 1 where all are 0.  The
// caller synchronises before it uses either.
__device__ __forceinline__ void load_slots(const Params& p, SlotView* view, float* top_out, bool report) {
  const int lane = threadIdx.x & 31;
  const int32_t* tokens = reinterpret_cast<const int32_t*>(p.base + p.off_tokens);
  const float2* gs = reinterpret_cast<const float2*>(p.base + p.off_gscale);
  static_assert(kMaxWindowSlots <= 64, "two slots a lane");
  int32_t held[2] = {0, 0};
  float2 g[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (lane + 32 * u < p.n_slots) {
      held[u] = tokens[p.slots[lane + 32 * u]];
      g[u] = gs[p.slots[lane + 32 * u]];
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (lane + 32 * u < p.n_slots && held[u] == p.tokens[lane + 32 * u]) top = fmaxf(top, g[u].y);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
  if (!(top > 0.0f)) top = 1.0f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    if (i >= p.n_slots) continue;
    const bool ok = held[u] == p.tokens[i];
    const float r = g[u].y / top;
    const bool zero = !(r > 8.6736173798840355e-19f);  // 2^-60
    view[i].ok = ok;
    view[i].gk = g[u].x;
    view[i].vzero = zero;
    view[i].lg = zero ? 0.0f : log2f(r);
    view[i].inv = zero ? 1.0f : 1.0f / r;
    if (!ok && report) set_status(p.status, kStatusShape);
  }
  if (lane == 0) *top_out = top;
}

// Exponent of the power of two that takes a row of queries with largest magnitude `top` (bf16 bits)
// to [2^14, 2^15); 0 for a row of zeros, or with a NaN or Inf: the whole row (or the factor of its
// scores) is then NaN, and with it the result wherever it sees a key.  Infinities as they are could give
// scores of -Inf alone, which look like masked ones, or finite ones under a cap.
__device__ __forceinline__ int query_exponent(unsigned top) {
  if (top == 0 || top >= 0x7F80u) return 0;
  const int e = 141 - (int)(top >> 7);
  return e > 120 ? 120 : e;  // 2^e and 2^-e stay FP32 numbers
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// tanh z for |z| <= kTanhNear: z times a polynomial in z^2, interpolated at the Chebyshev nodes of
// [0, kTanhNear^2] (the series' nearest singularity, z = i pi / 2, is far: five terms are within
// 2^-23 of tanh).  Scores are mostly well inside their cap, and this runs on the FMA units, two
// lanes at a time, where the form for larger z takes two of the sixteen special-function results a
// cycle that the softmax's own exponentials need.
constexpr float kTanhNear = 0.625f;
__device__ __forceinline__ void tanh_near2(float& a, float& b) {
  float ua, ub, pa = 0.015043356455862522f, pb = pa;
  mul2(ua, ub, a, b, a, b);
  fma2(pa, pb, pa, pb, ua, ub, -0.05181591212749481f, -0.05181591212749481f);
  fma2(pa, pb, pa, pb, ua, ub, 0.1330437958240509f, 0.1330437958240509f);
  fma2(pa, pb, pa, pb, ua, ub, -0.33331942558288574f, -0.33331942558288574f);
  fma2(pa, pb, pa, pb, ua, ub, 0.9999998807907104f, 0.9999998807907104f);
  mul2(a, b, a, b, pa, pb);
}

// tanh z = 1 - 2 / (1 + 2^(2 z log2 e)) beyond kTanhNear, the polynomial inside it: relative error
// about 2^-21 everywhere.  The first form alone is off by 2^-22 of the cap however small the score,
// which under a wide cap is more than the score's other roundings.
__device__ __forceinline__ void tanh2(float& a, float& b) {
  const float fa = 1.0f - 2.0f * rcp_approx(1.0f + ex2(a * (2.0f * kLog2e)));
  const float fb = 1.0f - 2.0f * rcp_approx(1.0f + ex2(b * (2.0f * kLog2e)));
  const bool na = fabsf(a) <= kTanhNear, nb = fabsf(b) <= kTanhNear;
  tanh_near2(a, b);
  a = na ? a : fa;
  b = nb ? b : fb;
}

// The visibility of keys [k0, k1] (positions) to queries [q0, q1]: 0 none, 1 some, 2 all.
__device__ __forceinline__ int visibility(const Params& p, int k0, int k1, int q0, int q1) {
  if (p.prefix > 0 && k0 < p.prefix) {
    if (k1 < p.prefix) return 2;
    return 1;
  }
  int v = 2;
  if (p.causal) {
    if (k0 > q1) return 0;
    if (k1 > q0) v = 1;
  }
  if (p.window) {
    if ((int64_t)q0 - k1 >= p.window) return 0;
    if ((int64_t)q1 - k0 >= p.window) v = 1;
  }
  return v;
}

__device__ __forceinline__ bool visible(const Params& p, int k, int q) {
  if (k < p.prefix) return true;
  return (!p.causal || k <= q) && (!p.window || q - k < p.window);
}

// Drafts' depth below the window, following the parents (at most `drafts` steps: a parent comes
// before its child).  A parent that does not is refused: it counts as none and sets SHAPE.
__device__ __forceinline__ int parent_of(const Params& p, const int32_t* parents, int i) {
  const int j = parents[i];
  if (j < -1 || j >= i) {
    set_status(p.status, kStatusShape);
    return -1;
  }
  return j;
}

// Four dims from d on of row r's result among `part`, normalised; log2l: log2 of its sum of weights.
__device__ __forceinline__ void store_partial(const Params& p, int part, int h, int64_t r, int d, float4 o,
                                              float log2l, bool with_l) {
  const int64_t at = ((int64_t)part * p.heads + h) * p.rows + r;
  *reinterpret_cast<float4*>(p.part_o + at * kD + d) = o;
  if (with_l) p.part_l[at] = log2l;
}

// A window's result of row r: a partial where it is joined with others, else the output, with what
// the drafts gave (kept by this CTA as the one partial) joined in.
__device__ __forceinline__ void store_row(const Params& p, int part, int h, int64_t r, int d, float4 o, float log2l,
                                          bool with_l) {
  if (p.parts > 1 || (p.parents && !p.fold)) return store_partial(p, part, h, r, d, o, log2l, with_l);
  if (p.fold) {
    const int64_t at = (int64_t)h * p.rows + r;
    const float lt = *(volatile float*)(p.part_l + at);
    const float4 t = *reinterpret_cast<const float4*>(p.part_o + at * kD + d);
    const float top = lt == -INFINITY && log2l == -INFINITY ? 0.0f : fmaxf(lt, log2l);
    const float a = ex2(log2l - top), b = ex2(lt - top), inv = 1.0f / (a + b);
    if (a + b != 0.0f) {  // a NaN of either goes on
      o.x = (a * o.x + b * t.x) * inv;
      o.y = (a * o.y + b * t.y) * inv;
      o.z = (a * o.z + b * t.z) * inv;
      o.w = (a * o.w + b * t.w) * inv;
      log2l = top + log2f(a + b);
    }
  }
  const int64_t i = p.by_group.div((uint32_t)r);
  const int head = h * p.group + (int)(r - i * p.group);
  stg_v2(p.o + i * p.o_pitch + ((int64_t)head * kD + d) * 2, make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w)));
  if (with_l && p.lse) p.lse[(int64_t)head * p.tq + i] = log2l * kLn2;
}

// Position of row r's query.
__device__ __forceinline__ int row_position(const Params& p, const int32_t* parents, int64_t r) {
  const int64_t i = p.by_group.div((uint32_t)r);
  if (!p.parents) return p.q_pos ? p.q_pos[i] : p.q_pos0 + (int)i;
  int pos = p.q_pos0;
  for (int j = parent_of(p, parents, (int)i); j >= 0; j = parent_of(p, parents, j)) ++pos;
  return pos;
}

// Running softmax of one row, four dims a lane: maximum and sum in log2 units, O not normalised.
struct RowSum {
  float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  // Makes `top` (not -inf) the maximum; a NaN of either stays.
  __device__ __forceinline__ void raise(float top) {
    top = top != top || m != m ? NAN : fmaxf(m, top);
    const float a = ex2(m - top);
    l *= a;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] *= a;
    m = top;
  }
  __device__ __forceinline__ void add(float w, float4 v) {
    l += w;
    o[0] = fmaf(w, v.x, o[0]);
    o[1] = fmaf(w, v.y, o[1]);
    o[2] = fmaf(w, v.z, o[2]);
    o[3] = fmaf(w, v.w, o[3]);
  }
};

// A draft and its ancestors, one thread: list[0] = i, list[1] its parent, ...; returns their number.
__device__ __forceinline__ int ancestors_of(const Params& p, const int32_t* parents, int i, int16_t* list) {
  int n = 0;
  for (int j = i; j >= 0; j = parent_of(p, parents, j)) list[n++] = (int16_t)j;
  return n;
}

// Entries first, first + step, ... of a draft's list (itself and its ancestors) into its row's sum:
// one warp, a lane holding 4 dims, in FP32.  A draft that a row does not see is never read for it,
// so whatever it holds (NaN, Inf) cannot reach the row.
__device__ __forceinline__ void tree_row(const Params& p, const int16_t* list, int n, int first, int step, int i,
                                         int h, int head, RowSum& row) {
  constexpr int kBatch = 4;  // reads of this many drafts together
  const int lane = threadIdx.x & 31;
  const uint2 qw = *reinterpret_cast<const uint2*>(p.q + (int64_t)i * p.q_pitch + ((int64_t)head * kD + 4 * lane) * 2);
  const float q[4] = {bf16_lo(qw.x), bf16_hi(qw.x), bf16_lo(qw.y), bf16_hi(qw.y)};
  const float slope = p.slopes ? p.slopes[head] : 0.0f;
  const unsigned top_q = __vmaxu2(qw.x & 0x7FFF7FFFu, qw.y & 0x7FFF7FFFu);
  const bool odd_q = max(top_q >> 16, top_q & 0xFFFFu) >= 0x7F80u;
  const float scale = __any_sync(0xFFFFFFFFu, odd_q) ? NAN : p.scale;  // as in the window (query_exponent)
  for (int e0 = first; e0 < n; e0 += kBatch * step) {
    uint2 kw[kBatch], vw[kBatch];
    float s[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int at = e0 + e * step < n ? e0 + e * step : e0;
      const int64_t off = (int64_t)list[at] * p.new_pitch + ((int64_t)h * kD + 4 * lane) * 2;
      kw[e] = *reinterpret_cast<const uint2*>(p.k_new + off);
      vw[e] = *reinterpret_cast<const uint2*>(p.v_new + off);
    }
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      s[e] = fmaf(q[0], bf16_lo(kw[e].x), fmaf(q[1], bf16_hi(kw[e].x), fmaf(q[2], bf16_lo(kw[e].y), q[3] * bf16_hi(kw[e].y))));
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s[e] += __shfl_xor_sync(0xFFFFFFFFu, s[e], x);
      s[e] *= scale;
    }
    if (p.cap > 0.0f) {
#pragma unroll
      for (int e = 0; e < kBatch; e += 2) {
        s[e] /= p.cap, s[e + 1] /= p.cap;
        tanh2(s[e], s[e + 1]);
        s[e] *= p.cap, s[e + 1] *= p.cap;
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      // the list holds draft i, its parent, ...: an entry is its number of positions before i
      const int back = e0 + e * step;
      s[e] = (s[e] - slope * (float)back) * kLog2e;
      if (back >= n || (p.window && back >= p.window)) s[e] = -INFINITY;
      top = s[e] != s[e] || top != top ? NAN : fmaxf(top, s[e]);
    }
    if (top == -INFINITY) continue;
    row.raise(top);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (s[e] == -INFINITY) continue;
      row.add(ex2(s[e] - row.m), make_float4(bf16_lo(vw[e].x), bf16_hi(vw[e].x), bf16_lo(vw[e].y), bf16_hi(vw[e].y)));
    }
  }
}

// The drafts that rows first, first + stride, ... below r1 of cache head h see, for this warp, as
// partial results.  list: kMaxFoldedDrafts entries of this warp.
__device__ __forceinline__ void tree_rows(const Params& p, const int32_t* parents, int16_t* list, int h,
                                          int64_t first, int64_t r1, int stride) {
  const int lane = threadIdx.x & 31;
  for (int64_t r = first; r < r1 && r < p.rows; r += stride) {
    const int i = (int)p.by_group.div((uint32_t)r);
    const int head = h * p.group + (int)(r - (int64_t)i * p.group);
    int n = 0;
    if (lane == 0) n = ancestors_of(p, parents, i, list);
    n = __shfl_sync(0xFFFFFFFFu, n, 0);
    __syncwarp();
    RowSum row;
    tree_row(p, list, n, 0, 1, i, h, head, row);
    const float inv = row.l > 0.0f ? 1.0f / row.l : (row.l == 0.0f ? 0.0f : row.l);
    store_partial(p, 0, h, r, 4 * lane, make_float4(row.o[0] * inv, row.o[1] * inv, row.o[2] * inv, row.o[3] * inv),
                  row.l == 0.0f ? -INFINITY : row.m + log2f(row.l), lane == 0);
    __syncwarp();
  }
}

// Tensor-core form for many rows (attend_tiles.cu): key steps of kTileKeys, at most kMaxListed of
// them a CTA.
constexpr int kTileKeys = 64;
constexpr int kMaxListed = 2048;
constexpr int64_t kTileRows = 128;
cudaError_t launch_attend_tiles(const Params& p, cudaStream_t s);

}  // namespace attend
}  // namespace nvfp4
