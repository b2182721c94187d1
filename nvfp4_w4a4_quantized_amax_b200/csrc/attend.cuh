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
// below.  The weights enter as binary16 with their maximum near 2^14 (relative rounding
// 2^-12, as against 2^-9 for bf16).  g_V differs from slot to slot: relative to the window's
// largest it goes into the exponent of the weights (see SlotView::lg), and O is multiplied by
// the largest at the end.  Scores, softmax statistics and sums are FP32.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace attend {

constexpr int kD = 128;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kShift = 14.0f;  // weights are scaled by 2^kShift

struct Params {
  const uint8_t* base;
  int64_t off_k_codes, off_v_codes, off_k_scales, off_v_scales, off_mu, off_gscale, off_tokens;
  int64_t slot_codes, slot_scales;
  int32_t heads, group;  // cache heads, query heads of each
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
  // log2 of the sum [part][cache head][row]
  int32_t parts;
  float* part_o;
  float* part_l;
  unsigned* status;
};

// Constants of one listed slot.
struct SlotView {
  float gk;    // g_K
  float lg;    // log2(g_V / largest g_V): p 2^lg goes to the product, p to the sum
  float inv;   // 2^-lg
  int ok;      // the slot holds the stated number of tokens
  int vzero;   // its values count as zero: g_V is 0 or under 2^-60 of the largest
};

// Reads the listed slots' scales (whole CTA); returns the largest g_V, 1 where all are 0.
__device__ __forceinline__ float load_slots(const Params& p, SlotView* view, bool report) {
  const float* gs = reinterpret_cast<const float*>(p.base + p.off_gscale);
  for (int i = threadIdx.x; i < p.n_slots; i += blockDim.x) {
    const bool ok = reinterpret_cast<const int32_t*>(p.base + p.off_tokens)[p.slots[i]] == p.tokens[i];
    view[i].ok = ok;
    view[i].gk = gs[2 * p.slots[i]];
    view[i].lg = gs[2 * p.slots[i] + 1];  // g_V for now
    if (!ok && report) set_status(p.status, kStatusShape);
  }
  __syncthreads();
  float top = 0.0f;
  for (int i = 0; i < p.n_slots; ++i)
    if (view[i].ok) top = fmaxf(top, view[i].lg);
  if (!(top > 0.0f)) top = 1.0f;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n_slots; i += blockDim.x) {
    const float r = view[i].lg / top;
    const bool zero = !(r > 8.6736173798840355e-19f);  // 2^-60
    view[i].vzero = zero;
    view[i].lg = zero ? 0.0f : log2f(r);
    view[i].inv = zero ? 1.0f : 1.0f / r;
  }
  __syncthreads();
  return top;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x -> cap tanh(x / cap), through tanh z = 1 - 2 / (1 + 2^(2 z log2 e)): absolute error about
// cap 2^-22 from ex2.approx and rcp.approx, saturating at both ends.
__device__ __forceinline__ float softcap(float x, float cap, float two_log2e_over_cap) {
  return cap - 2.0f * cap * rcp_approx(1.0f + ex2(x * two_log2e_over_cap));
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

}  // namespace attend
}  // namespace nvfp4
