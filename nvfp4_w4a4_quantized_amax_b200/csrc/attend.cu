// attend.cu — softmax attention of few query rows over a window of the NVFP4 cache, the
// drafted tokens of a tree, and the joining of partial results (attend.cuh gives the formulas).
#include <algorithm>
#include <atomic>

#include "attend.cuh"
#include "tc.cuh"

namespace nvfp4 {
namespace attend {
namespace {

using tc::smem_u32;

constexpr int kRows = 16;       // query rows of a CTA: the M of one mma.sync
constexpr int kStep = 32;       // keys a warp takes at a time
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
}

// A warp's ring of key steps on their way from the cache: codes, scales and what the step is.
constexpr int kRing = 4;
struct Stage {
  uint8_t k_codes[kStep * 64], v_codes[kStep * 64];
  uint8_t k_scales[kStep * 8], v_scales[kStep * 8];
};
struct StepInfo {
  int32_t seg, t0, n, vis;  // n == 0: no more steps
};

struct Shared {
  union {
    Stage ring[kWarps][kRing];
    float o[kWarps][kRows][kD];
    struct {
      int32_t parents[kMaxTreeDrafts];
      int16_t list[kWarps][kMaxTreeDrafts];
    } tree;
  };
  StepInfo info[kWarps][kRing];
  SlotView view[kMaxWindowSlots];
  float m[kWarps][kRows], l[kWarps][kRows];
  int32_t row_pos[kRows], row_doc[kRows];
  float gv_top;
};

__device__ __forceinline__ void copy_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Within an 8-key tile the product's column 2 c + e is key c + 4 e: the lanes of one read of V then
// take neighbouring keys.
__device__ __forceinline__ int tile_key(int n) { return (n >> 1) + 4 * (n & 1); }

// One CTA: 16 query rows of one cache head against a range of the window's 32-key steps, the
// steps dealt out to four warps.  mma.sync and not tcgen05: with at most 16 rows the kernel
// waits for the cache's bytes and for their decoding, and mma.sync takes the decoded codes from
// registers, where tcgen05 would have them stored to shared memory first.
// Each warp copies its steps' codes and scales into its own ring three steps ahead (cp.async: no
// registers, and no barrier but the warp's own).
// Lane (g, c) = (lane / 4, lane % 4).  Scores: the contraction runs over dims in an order in
// which lane c owns dims 32 c .. 32 c + 31 (16 bytes of codes, two scale bytes) of key g of an
// 8-key tile.  Values: lane (g, c) owns dims 16 g .. 16 g + 15 (8 bytes, one scale) of keys
// c, c + 4 of a tile; nibbles of the two keys are interleaved before the conversion, which
// then yields the pairs of columns the product wants.
template <bool kExtras>  // a cap, a bias or documents
__global__ void __launch_bounds__(kThreads, 3) attend_rows_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int part = blockIdx.x, h = blockIdx.y;
  constexpr int64_t r0 = 0;
  const bool tree_part = p.parents && part == p.parts - 1;
  const bool positions = p.causal || p.window || p.prefix || p.slopes;
  if (p.parents && (tree_part || positions)) {
    for (int i = threadIdx.x; i < p.drafts; i += kThreads) sh.tree.parents[i] = p.parents[i];
    __syncthreads();
  }
  if (tree_part) {
    tree_rows(p, sh.tree.parents, sh.tree.list[warp], h, r0 + warp, r0 + kRows, kWarps);
    return;
  }
  if (threadIdx.x < kRows) {
    const int64_t r = r0 + threadIdx.x < p.rows ? r0 + threadIdx.x : p.rows - 1;
    const int64_t i = p.by_group.div((uint32_t)r);
    sh.row_pos[threadIdx.x] = positions ? row_position(p, sh.tree.parents, r) : 0;
    if (kExtras) sh.row_doc[threadIdx.x] = p.q_doc ? p.q_doc[i] : 0;
  }
  if (warp == kWarps - 1) load_slots(p, sh.view, &sh.gv_top, part == 0 && h == 0 && r0 == 0);
  __syncthreads();
  const float gv_top = sh.gv_top;
  int q_first = sh.row_pos[0], q_last = q_first;
#pragma unroll
  for (int i = 1; i < kRows; ++i) {
    q_first = min(q_first, sh.row_pos[i]);
    q_last = max(q_last, sh.row_pos[i]);
  }

  // this lane's rows: g and g + 8; queries as binary16 A fragments and each row's factor
  uint32_t qa[8][4];
  float fac[2];
  int qpos[2], qdoc[2] = {0, 0};
  float slope[2] = {0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t r = r0 + g + 8 * u;
    const int64_t rr = r < p.rows ? r : p.rows - 1;
    const int64_t i = p.by_group.div((uint32_t)rr);
    const int head = h * p.group + (int)(rr - i * p.group);
    const uint8_t* src = p.q + i * p.q_pitch + ((int64_t)head * kD + 32 * c) * 2;
    uint32_t w[16];
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 v = ldg_nc_v4(src + 16 * k);
      w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
    top = max(top >> 16, top & 0xFFFFu);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int e = query_exponent(top);
    const float up = exp2i(e);
    fac[u] = p.scale * exp2i(-e);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qa[ks][u] = pack_f16x2(bf16_lo(w[2 * ks]) * up, bf16_hi(w[2 * ks]) * up);
      qa[ks][2 + u] = pack_f16x2(bf16_lo(w[2 * ks + 1]) * up, bf16_hi(w[2 * ks + 1]) * up);
    }
    qpos[u] = sh.row_pos[g + 8 * u];
    if (kExtras) {
      qdoc[u] = sh.row_doc[g + 8 * u];
      if (p.slopes) slope[u] = p.slopes[head] * kLog2e;
    }
  }

  float o[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[j][k] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

  const int first = (int)((int64_t)p.steps * part / p.splits), last = (int)((int64_t)p.steps * (part + 1) / p.splits);
  const int64_t code_step = (int64_t)p.heads * (kD / 2), scale_step = (int64_t)p.heads * (kD / 16);
  // next step that some row sees, into ring place `to`
  int next = first + warp, next_seg = 0;
  auto issue = [&](int to) {
    StepInfo si = {0, 0, 0, 0};
    for (; next < last; next += kWarps) {
      while (next >= p.step_end[next_seg]) ++next_seg;
      if (!sh.view[next_seg].ok) continue;
      const int t0 = (next - (next_seg ? p.step_end[next_seg - 1] : 0)) * kStep;
      const int n = min(kStep, p.tokens[next_seg] - t0);
      const int kp0 = p.pos[next_seg] + t0;
      const int vis = visibility(p, kp0, kp0 + n - 1, q_first, q_last);
      if (vis == 0) continue;
      si = {next_seg, t0, n, n < kStep || (kExtras && p.k_doc) ? 1 : vis};
      next += kWarps;
      break;
    }
    if (si.n > 0) {
      Stage& st = sh.ring[warp][to];
      const int64_t slot = p.slots[si.seg], row0 = (int64_t)si.t0 * p.heads + h;
      const uint8_t* kc = p.base + p.off_k_codes + slot * p.slot_codes + row0 * (kD / 2) + 16 * c;
      const uint8_t* vc = p.base + p.off_v_codes + slot * p.slot_codes + row0 * (kD / 2) + 16 * c;
      const uint8_t* ks = p.base + p.off_k_scales + slot * p.slot_scales + row0 * (kD / 16);
      const uint8_t* vs = p.base + p.off_v_scales + slot * p.slot_scales + row0 * (kD / 16);
      const uint32_t kd = smem_u32(st.k_codes), vd = smem_u32(st.v_codes);
#pragma unroll
      for (int t = 0; t < 4; ++t) {  // keys behind the step's last repeat it and are masked
        copy_16(kd + (32 * t + lane) * 16, kc + min(8 * t + tile_key(g), si.n - 1) * code_step);
        const int key = 8 * t + g;
        copy_16(vd + key * 64 + ((c ^ (key & 2)) << 4), vc + min(key, si.n - 1) * code_step);
      }
      copy_8(smem_u32(st.k_scales) + lane * 8, ks + min((lane & ~7) + tile_key(lane & 7), si.n - 1) * scale_step);
      copy_8(smem_u32(st.v_scales) + lane * 8, vs + min(lane, si.n - 1) * scale_step);
    }
    if (lane == 0) sh.info[warp][to] = si;
    copy_commit();
  };
  int seg_at = -1, key_seg = 0;
  float bias[2] = {0.0f, 0.0f}, mul[2] = {0.0f, 0.0f}, lg = 0.0f, inv = 1.0f;
  int64_t key_base = 0;  // keys listed before slot key_seg
  bool vzero = false;
  const float rcap = p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(i);
  for (int at = 0;; at = (at + 1) % kRing) {
    copy_wait<kRing - 2>();
    __syncwarp();
    const StepInfo si = sh.info[warp][at];
    if (si.n == 0) break;
    const int seg = si.seg, t0 = si.t0, n = si.n, vis = si.vis;
    const int kp0 = p.pos[seg] + t0;
    if (kExtras && p.k_doc)
      for (; key_seg < seg; ++key_seg) key_base += p.tokens[key_seg];
    const Stage& stage = sh.ring[warp][at];
    if (seg != seg_at) {  // the slot's scales and q . mu of this lane's rows
      seg_at = seg;
      const SlotView sv = sh.view[seg];
      lg = sv.lg, inv = sv.inv, vzero = sv.vzero;
      const float4* mu = reinterpret_cast<const float4*>(
          p.base + p.off_mu + (((int64_t)p.slots[seg] * p.heads + h) * kD + 32 * c) * 4);
      float acc[2] = {0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const float4 v = __ldg(mu + ks);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x, y;
          f16x2_to_f32x2(qa[ks][u], x, y);
          acc[u] = fmaf(x, v.x, fmaf(y, v.y, acc[u]));
          f16x2_to_f32x2(qa[ks][2 + u], x, y);
          acc[u] = fmaf(x, v.z, fmaf(y, v.w, acc[u]));
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float f = kExtras && p.cap > 0.0f ? fac[u] : fac[u] * kLog2e;  // log2 units without a cap
        bias[u] = quad_sum(acc[u]) * f;
        mul[u] = f * sv.gk;
      }
    }
    // scores of 4 tiles of 8 keys
    float s[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[t][k] = 0.0f;
      const uint4 kw = *reinterpret_cast<const uint4*>(stage.k_codes + (32 * t + lane) * 16);
      const uint32_t kb = *reinterpret_cast<const uint16_t*>(stage.k_scales + (8 * t + g) * 8 + 2 * c);
      const uint32_t words[4] = {kw.x, kw.y, kw.z, kw.w};
      const uint32_t s2[2] = {e4m3_to_f16x2_bcast(kb & 0xFFu), e4m3_to_f16x2_bcast(kb >> 8)};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t b[4];
        e2m1x8_times_scale(words[w], s2[w >> 1], b);
        mma_f16(s[t], qa[2 * w][0], qa[2 * w][1], qa[2 * w][2], qa[2 * w][3], b[0], b[1]);
        mma_f16(s[t], qa[2 * w + 1][0], qa[2 * w + 1][1], qa[2 * w + 1][2], qa[2 * w + 1][3], b[2], b[3]);
      }
    }
    // element k of a tile: row g + 8 (k / 2), key c + 4 (k % 2)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = k >> 1, key = 8 * t + c + 4 * (k & 1);
        float x = fmaf(s[t][k], mul[u], bias[u]);
        if (kExtras) {
          if (p.cap > 0.0f) x = softcap(x, p.cap, rcap) * kLog2e;
          if (p.slopes) x = fmaf(-slope[u], fabsf((float)(qpos[u] - (kp0 + key))), x);
        }
        if (vis == 1) {
          bool see = key < n && visible(p, kp0 + key, qpos[u]);
          if (kExtras && p.k_doc) see = see && p.k_doc[key_base + t0 + min(key, n - 1)] == qdoc[u];
          if (!see) x = -INFINITY;
        }
        s[t][k] = x;
      }
    }
    float alpha[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t) top = fmaxf(top, fmaxf(s[t][2 * u], s[t][2 * u + 1]));
      top = quad_max(top);
      const float mn = fmaxf(m[u], top + lg);
      alpha[u] = mn == -INFINITY ? 1.0f : ex2(m[u] - mn);
      m[u] = mn;
      const float ref = mn == -INFINITY ? 0.0f : mn - lg - kShift;  // a row that has seen nothing: weights 0
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int k = 2 * u; k < 2 * u + 2; ++k) {
          s[t][k] = ex2(s[t][k] - ref);
          sum += s[t][k];
        }
      }
      l[u] = fmaf(sum, inv, l[u] * alpha[u]);
    }
    if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][0] *= alpha[0];
        o[j][1] *= alpha[0];
        o[j][2] *= alpha[1];
        o[j][3] *= alpha[1];
      }
    }
    if (!vzero) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {  // 16 keys: tiles 2 ks and 2 ks + 1
      const uint32_t a0 = pack_f16x2(s[2 * ks][0], s[2 * ks][1]), a1 = pack_f16x2(s[2 * ks][2], s[2 * ks][3]);
      const uint32_t a2 = pack_f16x2(s[2 * ks + 1][0], s[2 * ks + 1][1]);
      const uint32_t a3 = pack_f16x2(s[2 * ks + 1][2], s[2 * ks + 1][3]);
      uint2 wa[2], wb[2];
      uint32_t s2[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = 16 * ks + 8 * t + c;  // and key + 4
        const int off = (((g >> 1) ^ (c & 2)) << 4) + 8 * (g & 1);
        wa[t] = *reinterpret_cast<const uint2*>(stage.v_codes + key * 64 + off);
        wb[t] = *reinterpret_cast<const uint2*>(stage.v_codes + (key + 4) * 64 + off);
        const uint32_t pair = stage.v_scales[key * 8 + g] | ((uint32_t)stage.v_scales[(key + 4) * 8 + g] << 8);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2[t]) : "h"((uint16_t)pair));
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {  // 8 dims of the lane's block at a time
        uint32_t even[2][4], odd[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t xa = w ? wa[t].y : wa[t].x, xb = w ? wb[t].y : wb[t].x;
          e2m1x8_times_scale((xa & 0x0F0F0F0Fu) | ((xb << 4) & 0xF0F0F0F0u), s2[t], even[t]);
          e2m1x8_times_scale(((xa >> 4) & 0x0F0F0F0Fu) | (xb & 0xF0F0F0F0u), s2[t], odd[t]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mma_f16(o[8 * w + 2 * k], a0, a1, a2, a3, even[0][k], even[1][k]);
          mma_f16(o[8 * w + 2 * k + 1], a0, a1, a2, a3, odd[0][k], odd[1][k]);
        }
      }
    }
    }
    __syncwarp();
    issue((at + kRing - 1) % kRing);
  }
  copy_wait<0>();

  // join the warps: element k of o[j]: row g + 8 (k / 2), dim 32 c + 16 (k % 2) + j
  __syncthreads();  // the rings share this memory
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float ls = quad_sum(l[u]);
    if (c == 0) {
      sh.m[warp][g + 8 * u] = m[u];
      sh.l[warp][g + 8 * u] = ls;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int j = 0; j < 16; j += 4)
      *reinterpret_cast<float4*>(&sh.o[warp][g + 8 * (k >> 1)][32 * c + 16 * (k & 1) + j]) =
          make_float4(o[j][k], o[j + 1][k], o[j + 2][k], o[j + 3][k]);
  __syncthreads();
  for (int r = warp; r < kRows && r0 + r < p.rows; r += kWarps) {
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.m[w][r]);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (sh.l[w][r] == 0.0f) continue;  // saw nothing
      const float f = ex2(sh.m[w][r] - top);
      sum = fmaf(f, sh.l[w][r], sum);
      const float4 v = *reinterpret_cast<const float4*>(&sh.o[w][r][4 * lane]);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum * gv_top;
    store_row(p, part, h, r0 + r, 4 * lane, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f),
              sum == 0.0f ? -INFINITY : top + log2f(sum) - kShift, lane == 0);
  }
}

// Joins the partial results: O = sum_i 2^(L_i - L) O_i, L = log2 sum_i 2^L_i.  kSplit warps of a CTA
// of eight share a row's parts (each taking every kSplit-th, eight reads in flight) and add their
// sums in a fixed order.
template <int kSplit>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ Params p) {
  constexpr int kJoin = 8;
  __shared__ float4 part[kSplit > 1 ? 8 : 1][32];
  __shared__ float part_sum[8];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)p.heads * p.rows;
  const int h = blockIdx.y;
  const int64_t r = (int64_t)blockIdx.x * (8 / kSplit) + warp / kSplit;
  const int w = warp % kSplit;
  const bool live = r < p.rows;
  const int64_t rr = h * p.rows + (live ? r : p.rows - 1);
  float top = -INFINITY;
  for (int i = lane; i < p.parts; i += 32) {
    const float l = p.part_l[i * n + rr];
    top = l != l || top != top ? NAN : fmaxf(top, l);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) {
    const float v = __shfl_xor_sync(0xFFFFFFFFu, top, x);
    top = v != v || top != top ? NAN : fmaxf(top, v);
  }
  const float ref = top == -INFINITY ? 0.0f : top;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f;
  for (int i0 = w; i0 < p.parts; i0 += kSplit * kJoin) {
    float f[kJoin];
    float4 v[kJoin];
#pragma unroll
    for (int e = 0; e < kJoin; ++e) {
      const int i = i0 + e * kSplit < p.parts ? i0 + e * kSplit : i0;
      f[e] = p.part_l[i * n + rr];
      v[e] = *reinterpret_cast<const float4*>(p.part_o + (i * n + rr) * kD + 4 * lane);
    }
#pragma unroll
    for (int e = 0; e < kJoin; ++e) {
      if (i0 + e * kSplit >= p.parts) break;
      f[e] = ex2(f[e] - ref);  // 0 for a part that saw nothing, whose O is 0 as well
      sum += f[e];
      acc.x = fmaf(f[e], v[e].x, acc.x);
      acc.y = fmaf(f[e], v[e].y, acc.y);
      acc.z = fmaf(f[e], v[e].z, acc.z);
      acc.w = fmaf(f[e], v[e].w, acc.w);
    }
  }
  if (kSplit > 1) {
    part[warp][lane] = acc;
    if (lane == 0) part_sum[warp] = sum;
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int e = 1; e < kSplit; ++e) {
      const float4 v = part[warp + e][lane];
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      sum += part_sum[warp + e];
    }
  }
  if (!live) return;
  const float f = top == -INFINITY ? 0.0f : 1.0f / sum;
  const int64_t i = p.by_group.div((uint32_t)r);
  const int head = h * p.group + (int)(r - i * p.group);
  stg_v2(p.o + i * p.o_pitch + ((int64_t)head * kD + 4 * lane) * 2,
         make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f)));
  if (lane == 0 && p.lse) p.lse[(int64_t)head * p.tq + i] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------------------- host

constexpr int kSms = 148;

struct Plan {
  bool tiles;           // tensor-core form for many rows, else 16-row CTAs
  int32_t step, steps;  // keys a step, steps in the window (none straddles two slots)
  int32_t splits;       // CTAs that share a window
};

// Up to 16 rows a cache head: 16-row CTAs, about three an SM, each with two steps a warp at least.
// More: tiles of 128 rows; the keys are split where rows and heads do not fill the SMs evenly, by
// the least of waves * (steps a CTA + a CTA's own cost), with the partial results' traffic.
Plan make_plan(const int32_t* tokens, int n_slots, int heads, int64_t rows) {
  Plan plan;
  plan.tiles = rows > kRows;
  plan.step = plan.tiles ? kTileKeys : kStep;
  int64_t steps = 0;
  for (int i = 0; i < n_slots; ++i) steps += (tokens[i] + plan.step - 1) / plan.step;
  plan.steps = (int32_t)steps;
  int64_t splits = 1;
  if (!plan.tiles) {
    splits = std::min<int64_t>(heads > 0 ? 3 * kSms / heads : 1, steps / (2 * kWarps));
  } else {
    const bool pair = rows > kTileRows;
    const int64_t base = heads * ((rows + (pair ? 2 : 1) * kTileRows - 1) / ((pair ? 2 : 1) * kTileRows));
    const double step_us = pair ? 0.8 : 0.4, cta_us = 6.0;
    double best = 0.0;
    const int64_t least = (steps + kMaxListed - 1) / kMaxListed;
    for (int64_t n = std::max<int64_t>(least, 1); n <= std::max<int64_t>(least, std::min<int64_t>(steps / 8, kSms)); ++n) {
      const int64_t waves = (base * n + kSms - 1) / kSms;
      const double join_us = n > 1 ? 4.0 + 2.0 * n * heads * rows * 516 / 5e6 : 0.0;
      const double us = waves * ((steps + n - 1) / n * step_us + cta_us) + join_us;
      if (best == 0.0 || us < best) {
        best = us;
        splits = n;
      }
    }
  }
  plan.splits = (int32_t)std::max<int64_t>(splits, 1);
  return plan;
}

template <bool kExtras>
cudaError_t launch_rows(const Params& p, dim3 grid, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {  // doing it twice is harmless
    e = cudaFuncSetAttribute(attend_rows_kernel<kExtras>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  return launch_pdl(attend_rows_kernel<kExtras>, grid, kThreads, sizeof(Shared), s, p);
}

}  // namespace
}  // namespace attend

size_t attention_workspace_bytes(const int32_t* tokens, int n_slots, int heads, int64_t rows) {
  const attend::Plan plan = attend::make_plan(tokens, n_slots, heads, rows);
  return (size_t)(plan.splits + 1) * heads * rows * (attend::kD + 1) * sizeof(float);
}

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t s) {
  using namespace attend;
  if (a.tq == 0) return cudaSuccess;
  const KVLayout& c = *a.cache;
  Params p = {};
  p.base = c.base;
  p.off_k_codes = c.off_k_codes;
  p.off_v_codes = c.off_v_codes;
  p.off_k_scales = c.off_k_scales;
  p.off_v_scales = c.off_v_scales;
  p.off_mu = c.off_mu;
  p.off_gscale = c.off_gscale;
  p.off_tokens = c.off_tokens;
  p.slot_codes = c.slot_codes_bytes;
  p.slot_scales = c.slot_scales_bytes;
  p.chunk = c.chunk_tokens;
  p.heads = c.heads;
  p.group = a.q_heads / c.heads;
  p.by_group = FastDiv((uint32_t)p.group);
  p.n_slots = a.n_slots;
  p.rows = a.tq * p.group;
  const Plan plan = make_plan(a.tokens, a.n_slots, c.heads, p.rows);
  int32_t steps = 0;
  for (int i = 0; i < a.n_slots; ++i) {
    p.slots[i] = a.slots[i];
    p.tokens[i] = a.tokens[i];
    p.pos[i] = (int32_t)a.slot_pos[i];
    steps += (a.tokens[i] + plan.step - 1) / plan.step;
    p.step_end[i] = steps;
  }
  p.steps = plan.steps;
  p.splits = plan.splits;
  p.q = (const uint8_t*)a.q;
  p.q_pitch = a.ldq * 2;
  p.scale = a.scale;
  p.cap = a.cap;
  p.slopes = a.slopes;
  p.causal = a.causal;
  p.window = (int32_t)a.window;
  p.prefix = (int32_t)a.prefix;
  p.q_pos0 = (int32_t)a.q_pos0;
  p.q_pos = a.q_pos;
  p.q_doc = a.q_doc;
  p.k_doc = a.k_doc;
  p.parents = a.parents;
  p.k_new = (const uint8_t*)a.k_new;
  p.v_new = (const uint8_t*)a.v_new;
  p.new_pitch = a.ld_new * 2;
  p.drafts = a.parents ? (int32_t)a.tq : 0;
  p.o = (uint8_t*)a.o;
  p.o_pitch = a.ldo * 2;
  p.lse = a.lse;
  p.tq = a.tq;
  p.status = a.status;
  p.parts = plan.splits + (a.parents ? 1 : 0);
  if (p.parts > 1) {
    p.part_o = a.workspace;
    p.part_l = a.workspace + (int64_t)p.parts * p.heads * p.rows * kD;
  }
  const dim3 grid(p.parts, p.heads);
  cudaError_t e;
  if (plan.tiles) e = launch_attend_tiles(p, s);
  else if (p.cap > 0.0f || p.slopes || p.k_doc) e = launch_rows<true>(p, grid, s);
  else e = launch_rows<false>(p, grid, s);
  if (e != cudaSuccess || p.parts == 1) return e;
  // few parts: a warp a row; more: eight warps share a row's
  if (p.parts <= 8) return launch_pdl(attend_join_kernel<1>, dim3((unsigned)((p.rows + 7) / 8), p.heads), 256, 0, s, p);
  return launch_pdl(attend_join_kernel<8>, dim3((unsigned)p.rows, p.heads), 256, 0, s, p);
}

}  // namespace nvfp4
