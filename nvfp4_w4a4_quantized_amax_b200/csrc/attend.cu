// attend.cu — softmax attention of few query rows over a window of the NVFP4 cache, the
// drafted tokens of a tree, and the joining of partial results (attend.cuh gives the formulas).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attend.cuh"
#include "tc.cuh"

namespace nvfp4 {
namespace attend {
namespace {

using tc::smem_u32;

constexpr int kRows = 16;       // most query rows of a cache head that a CTA takes
constexpr int64_t kMostRows = 64;  // and that are dealt out to such CTAs
constexpr int kStep = 32;       // keys a warp takes at a time
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of the 8 x 8 matrix of 16-bit values that a warp holds, row lane / 4, columns
// 2 (lane % 4) and + 1.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// A warp's ring of key steps on their way from the cache: codes, scales and what the step is.
constexpr int kRing = 3;
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
    struct {
      float o[kWarps][kRows][kD], m[kWarps][kRows], l[kWarps][kRows];
    } join;
    struct {
      int32_t parents[kMaxTreeDrafts];
      int16_t list[kWarps][kMaxFoldedDrafts];
    } tree;
  };
  StepInfo info[kWarps][kRing];
  SlotView view[kMaxWindowSlots];
  int32_t row_pos[kRows], row_doc[kRows];
  float row_fac[kRows];
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

// Key of the product's index n within 8: index 2 c + e is key c + 4 e, so that the lanes of one read
// of V take neighbouring keys.
__device__ __forceinline__ int tile_key(int n) { return (n >> 1) + 4 * (n & 1); }

// One CTA: up to 8 kTiles query rows of one cache head against a range of the window's 32-key
// steps, the steps dealt out to four warps.  mma.sync and not tcgen05: with so few rows the kernel
// waits for the cache's bytes and for their decoding, and mma.sync takes the decoded codes from
// registers, where tcgen05 would have them stored to shared memory first.  Keys and dims are the
// product's 16 rows and queries its 8 columns, S^T = K~ Q^T and O^T = V~^T P^T: a row of queries
// alone then wastes 7 of 8 columns and not 15 of 16 rows, and O takes 32 registers a tile.
// Each warp copies its steps' codes and scales into its own ring two steps ahead (cp.async: no
// registers, and no barrier but the warp's own).
// Lane (g, c) = (lane / 4, lane % 4).  K~: the contraction runs over dims in an order in which lane
// c owns dims 32 c .. 32 c + 31 (16 bytes of codes, two scale bytes) of keys g and g + 8 of 16.
// V~^T: lane (g, c) owns dims 16 g .. 16 g + 15 (8 bytes, one scale) of the keys of columns 2 c,
// 2 c + 1 (and + 8); nibbles of two keys are interleaved before the conversion, which then yields
// the pairs the product wants.  P^T comes from S^T by one 8 x 8 transpose a tile.
// A loop step takes the scores of one step of keys and the output of the step before: one alone
// leaves a scheduler's few warps waiting for their own latencies.  That takes registers, so three CTAs
// an SM (168) and not four: 1 query x 24 heads x 32768 keys 44 us with the join, 51 with one step at a
// time and four CTAs, 51 with both in 128 registers.  16 rows take two CTAs (255) and not three: 16 x 8
// heads x 16384 keys 22.4 us against 25.5, 32 x 8 x 4096 16.7 against 19.7, but 12 x 24 x 32768 65 against
// 61.5, and 104 against 86 with a cap.  Bound by the copies and the decoding together: the copies
// alone take 31 to 35, half as much again as their codes without the 8-byte pieces of scales.
template <bool kExtras, int kTiles>  // kExtras: a cap, a bias or documents
__global__ void __launch_bounds__(kThreads, kTiles == 1 ? 3 : 2) attend_rows_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int part = blockIdx.x, h = blockIdx.y;
  const int64_t r0 = (int64_t)blockIdx.z * kRows, last_row = p.rows - 1;
  const bool positions = p.causal || p.window || p.prefix || p.slopes;
  if (p.parents && (p.fold || positions)) {
    for (int i = threadIdx.x; i < p.drafts; i += kThreads) sh.tree.parents[i] = p.parents[i];
    __syncthreads();
  }
  // a warp's rows, lane by lane, are those that it stores at the end: each thread then reads back
  // what it wrote itself
  if (p.fold) tree_rows(p, sh.tree.parents, sh.tree.list[warp], h, warp, kRows, kWarps);
  int q_first = 0, q_last = 0;
  if (positions || p.parents || (kExtras && p.q_doc)) {
    if (threadIdx.x < kRows) {
      const int64_t r = min(r0 + threadIdx.x, last_row);
      sh.row_pos[threadIdx.x] = positions ? row_position(p, sh.tree.parents, r) : 0;
      if (kExtras) sh.row_doc[threadIdx.x] = p.q_doc ? p.q_doc[p.by_group.div((uint32_t)r)] : 0;
    }
    __syncthreads();  // and the ring's memory is free of the drafts' parents
    q_first = q_last = sh.row_pos[0];
#pragma unroll
    for (int i = 1; i < kRows; ++i) {
      q_first = min(q_first, sh.row_pos[i]);
      q_last = max(q_last, sh.row_pos[i]);
    }
  }

  const int first = (int)((int64_t)p.steps * part / p.splits), last = (int)((int64_t)p.steps * (part + 1) / p.splits);
  const uint32_t code_step = (uint32_t)p.heads * (kD / 2), scale_step = (uint32_t)p.heads * (kD / 16);
  // next step that some row sees, into ring place `to`
  int next = first + warp, next_seg = 0;
  auto issue = [&](int to) {
    StepInfo si = {0, 0, 0, 0};
    for (; next < last; next += kWarps) {
      while (next >= p.step_end[next_seg]) ++next_seg;
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
      const uint32_t row0 = (uint32_t)((int64_t)p.slots[si.seg] * p.chunk + si.t0);
      const uint8_t* kc = p.base + p.off_k_codes + (int64_t)h * (kD / 2) + 16 * c;
      const uint8_t* vc = p.base + p.off_v_codes + (int64_t)h * (kD / 2) + 16 * c;
      const uint8_t* ks = p.base + p.off_k_scales + (int64_t)h * (kD / 16);
      const uint8_t* vs = p.base + p.off_v_scales + (int64_t)h * (kD / 16);
      const uint32_t kd = smem_u32(st.k_codes), vd = smem_u32(st.v_codes);
      auto row = [&](int key) { return (uint64_t)(row0 + (uint32_t)min(key, si.n - 1)); };
#pragma unroll
      for (int t = 0; t < 4; ++t) {  // keys behind the step's last repeat it and are masked
        copy_16(kd + (32 * t + lane) * 16, kc + row(8 * t + tile_key(g)) * code_step);
        const int key = 8 * t + g;
        copy_16(vd + key * 64 + ((c ^ (key & 2)) << 4), vc + row(key) * code_step);
      }
      copy_8(smem_u32(st.k_scales) + lane * 8, ks + row((lane & ~7) + tile_key(lane & 7)) * scale_step);
      copy_8(smem_u32(st.v_scales) + lane * 8, vs + row(lane) * scale_step);
    }
    if (lane == 0) sh.info[warp][to] = si;
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(i);
  if (warp == kWarps - 1) load_slots(p, sh.view, &sh.gv_top, part == 0 && h == 0 && r0 == 0);

  // queries as binary16 B fragments: lane (g, c) holds dims 32 c .. of row 8 tile + g
  uint32_t qb[kTiles][8][2];
#pragma unroll
  for (int u = 0; u < kTiles; ++u) {
    const uint32_t r = (uint32_t)min(r0 + 8 * u + g, last_row);
    const int i = (int)p.by_group.div(r);
    const int head = h * p.group + (int)(r - (uint32_t)i * p.group);
    const uint8_t* src = p.q + (int64_t)i * p.q_pitch + ((int64_t)head * kD + 32 * c) * 2;
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
    if (warp == 0 && c == 0) sh.row_fac[8 * u + g] = top >= 0x7F80u ? NAN : p.scale * exp2i(-e);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qb[u][ks][0] = pack_f16x2(bf16_lo(w[2 * ks]) * up, bf16_hi(w[2 * ks]) * up);
      qb[u][ks][1] = pack_f16x2(bf16_lo(w[2 * ks + 1]) * up, bf16_hi(w[2 * ks + 1]) * up);
    }
  }
  __syncthreads();

  // statistics of this lane's rows: row 8 u + 2 c + e is [u][e]
  float o[kTiles][8][4], m[kTiles][2], l[kTiles][2], bias[kTiles][2], mul[kTiles][2];
#pragma unroll
  for (int u = 0; u < kTiles; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[u][j][k] = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) m[u][e] = -INFINITY, l[u][e] = 0.0f, bias[u][e] = mul[u][e] = 0.0f;
  }
  int qpos[kTiles][2];
  float slope[kTiles][2];
  const float cap = kExtras ? p.cap * kLog2e : 0.0f;
#pragma unroll
  for (int u = 0; u < kTiles; ++u) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t r = (uint32_t)min(r0 + 8 * u + 2 * c + e, last_row);
      qpos[u][e] = positions ? sh.row_pos[8 * u + 2 * c + e] : 0;
      slope[u][e] = 0.0f;
      if (kExtras && p.slopes)
        slope[u][e] = kLog2e * p.slopes[h * p.group + (int)(r - p.by_group.div(r) * p.group)];
    }
  }
  int seg_at = -1;
  float lg = 0.0f, inv = 1.0f;
  // S^T of a step: element k of [tile t][u] is key 16 t + 8 (k / 2) + tile_key(g), row 8 u + 2 c + k % 2
  float s[2][kTiles][4];
  // weights of the step before, and whether its values count.  A step of a refused slot leaves them as
  // they are with its values masked to 0, so they are numbers from the start: 0 times an unset
  // register could be a NaN
  uint32_t pb[2][kTiles][2] = {};
  uint32_t keep = 0;
  // The scores of one step and the output of the step before it: two independent chains, which hide
  // each other's latencies (a scheduler has three warps, with 16 rows two).
  auto products = [&](const Stage& now, const Stage& before, auto scores, auto output) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint4 kw[2];
      uint32_t ks2[2][2];
      if constexpr (decltype(scores)::value) {
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[t][u][k] = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // keys g and g + 8
          kw[e] = *reinterpret_cast<const uint4*>(now.k_codes + (64 * t + 32 * e + lane) * 16);
          const uint32_t kb = *reinterpret_cast<const uint16_t*>(now.k_scales + (16 * t + 8 * e + g) * 8 + 2 * c);
          ks2[e][0] = e4m3_to_f16x2_bcast(kb & 0xFFu);
          ks2[e][1] = e4m3_to_f16x2_bcast(kb >> 8);
        }
      }
      uint2 wa[2], wb[2];
      uint32_t vs2[2];
      if constexpr (decltype(output)::value) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // keys of columns 2 c, 2 c + 1, and of 8 further
          const int key = 16 * t + 8 * e + c;  // and key + 4
          const int off = (((g >> 1) ^ (c & 2)) << 4) + 8 * (g & 1);
          wa[e] = *reinterpret_cast<const uint2*>(before.v_codes + key * 64 + off);
          wb[e] = *reinterpret_cast<const uint2*>(before.v_codes + (key + 4) * 64 + off);
          const uint32_t pair = (before.v_scales[key * 8 + g] | ((uint32_t)before.v_scales[(key + 4) * 8 + g] << 8)) & keep;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(vs2[e]) : "h"((uint16_t)pair));
        }
      }
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        if constexpr (decltype(scores)::value) {
#pragma unroll
          for (int w = 2 * odd; w < 2 * odd + 2; ++w) {
            uint32_t a[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              e2m1x8_times_scale(w == 0 ? kw[e].x : w == 1 ? kw[e].y : w == 2 ? kw[e].z : kw[e].w, ks2[e][w >> 1], a[e]);
#pragma unroll
            for (int u = 0; u < kTiles; ++u) {
              mma_f16(s[t][u], a[0][0], a[1][0], a[0][1], a[1][1], qb[u][2 * w][0], qb[u][2 * w][1]);
              mma_f16(s[t][u], a[0][2], a[1][2], a[0][3], a[1][3], qb[u][2 * w + 1][0], qb[u][2 * w + 1][1]);
            }
          }
        }
        if constexpr (decltype(output)::value) {  // even, then odd dims of the lane's block
          uint32_t a[2][2][4];  // [column pair][8 dims of the block][dim / 2]
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t xa = w ? wa[e].y : wa[e].x, xb = w ? wb[e].y : wb[e].x;
              const uint32_t both = odd ? ((xa >> 4) & 0x0F0F0F0Fu) | (xb & 0xF0F0F0F0u)
                                        : (xa & 0x0F0F0F0Fu) | ((xb << 4) & 0xF0F0F0F0u);
              e2m1x8_times_scale(both, vs2[e], a[e][w]);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < kTiles; ++u)
              mma_f16(o[u][2 * k + odd], a[0][0][k], a[0][1][k], a[1][0][k], a[1][1][k], pb[t][u][0], pb[t][u][1]);
        }
      }
    }
  };
  using Yes = std::true_type;
  using No = std::false_type;
  bool begun = false;
  for (int at = 0;; at = at + 1 == kRing ? 0 : at + 1) {
    copy_wait<kRing - 2>();
    __syncwarp();
    const StepInfo si = sh.info[warp][at];
    const int free = at == 0 ? kRing - 1 : at - 1;  // the step before's place
    const Stage &now = sh.ring[warp][at], &before = sh.ring[warp][free];
    if (si.n == 0) {
      if (begun) products(now, before, No{}, Yes{});
      break;
    }
    if (begun) products(now, before, Yes{}, Yes{});
    else products(now, before, Yes{}, No{});
    begun = true;
    __syncwarp();
    issue(free);
    if (si.seg != seg_at) {  // the slot's scales, and q . mu of this lane's rows
      seg_at = si.seg;
      const SlotView sv = sh.view[seg_at];
      lg = sv.lg, inv = sv.inv;
      const float4* mu = reinterpret_cast<const float4*>(
          p.base + p.off_mu + (((int64_t)p.slots[seg_at] * p.heads + h) * kD + 32 * c) * 4);
      float acc[kTiles];
#pragma unroll
      for (int u = 0; u < kTiles; ++u) acc[u] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const float4 v = __ldg(mu + ks);
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
          float x, y;
          f16x2_to_f32x2(qb[u][ks][0], x, y);
          acc[u] = fmaf(x, v.x, fmaf(y, v.y, acc[u]));
          f16x2_to_f32x2(qb[u][ks][1], x, y);
          acc[u] = fmaf(x, v.z, fmaf(y, v.w, acc[u]));
        }
      }
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        acc[u] += __shfl_xor_sync(0xFFFFFFFFu, acc[u], 1);
        acc[u] += __shfl_xor_sync(0xFFFFFFFFu, acc[u], 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float fac = sh.row_fac[8 * u + 2 * c + e];
          // log2 units, or shares of the cap
          const float f = kExtras && p.cap > 0.0f ? fac / p.cap : fac * kLog2e;
          bias[u][e] = __shfl_sync(0xFFFFFFFFu, acc[u], 4 * (2 * c + e)) * f;
          mul[u][e] = f * sv.gk;
        }
      }
    }
    keep = 0;
    if (sh.view[seg_at].ok) {
      const int kp0 = p.pos[seg_at] + si.t0;
      const int32_t* docs = p.k_doc;
      if (kExtras && docs) {
        docs += si.t0;
        for (int i = 0; i < seg_at; ++i) docs += p.tokens[i];
      }
      bool grow = false;
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = k & 1;
#pragma unroll
          for (int t = 0; t < 2; ++t) s[t][u][k] = fmaf(s[t][u][k], mul[u][e], bias[u][e]);
          if (kExtras && p.cap > 0.0f) {
            tanh2(s[0][u][k], s[1][u][k]);
            mul2(s[0][u][k], s[1][u][k], s[0][u][k], s[1][u][k], cap, cap);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float x = s[t][u][k];
            if (kExtras || si.vis == 1) {
              const int key = 16 * t + 8 * (k >> 1) + tile_key(g);
              if (kExtras && p.slopes) x = fmaf(-slope[u][e], fabsf((float)(qpos[u][e] - (kp0 + key))), x);
              if (si.vis == 1) {
                bool see = key < si.n && visible(p, kp0 + key, qpos[u][e]);
                if (kExtras && p.k_doc) see = see && docs[min(key, si.n - 1)] == sh.row_doc[8 * u + 2 * c + e];
                if (!see) x = -INFINITY;
              }
            }
            s[t][u][k] = x;
            grow |= x + lg > m[u][e] + kLazy || (m[u][e] == -INFINITY && x > -INFINITY);
          }
        }
      }
      if (__any_sync(0xFFFFFFFFu, grow)) {  // new maxima: the same in every lane of a row
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(fmaxf(s[0][u][e], s[0][u][2 + e]), fmaxf(s[1][u][e], s[1][u][2 + e]));
#pragma unroll
            for (int x = 16; x > 2; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            const float mn = fmaxf(m[u][e], top + lg);
            const float alpha = mn == -INFINITY ? 1.0f : ex2(m[u][e] - mn);
            m[u][e] = mn;
            l[u][e] *= alpha;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[u][j][e] *= alpha;
              o[u][j][2 + e] *= alpha;
            }
          }
        }
      }
      // weights, transposed: columns 2 c, 2 c + 1 of 16 keys of row g
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        float ref[2], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 2; ++e) ref[e] = m[u][e] == -INFINITY ? 0.0f : m[u][e] - lg - kUp;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float w0 = ex2(s[t][u][2 * half] - ref[0]), w1 = ex2(s[t][u][2 * half + 1] - ref[1]);
            sum[0] += w0;
            sum[1] += w1;
            pb[t][u][half] = transpose_8x8(pack_f16x2(w0, w1));
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) l[u][e] = fmaf(sum[e], inv, l[u][e]);
      }
      if (!sh.view[seg_at].vzero) keep = 0xFFFFu;
    }
  }
  copy_wait<0>();

  // join the warps: element k of o[u][j] is dim 16 g + 8 (k / 2) + j of row 8 u + 2 c + k % 2
  __syncthreads();  // the rings share this memory
#pragma unroll
  for (int u = 0; u < kTiles; ++u) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 16; x > 2; x >>= 1) l[u][e] += __shfl_xor_sync(0xFFFFFFFFu, l[u][e], x);
      if (g == 0) {
        sh.join.m[warp][8 * u + 2 * c + e] = m[u][e];
        sh.join.l[warp][8 * u + 2 * c + e] = l[u][e];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        *reinterpret_cast<float4*>(&sh.join.o[warp][8 * u + 2 * c + (k & 1)][16 * g + 8 * (k >> 1) + j]) =
            make_float4(o[u][j][k], o[u][j + 1][k], o[u][j + 2][k], o[u][j + 3][k]);
  }
  __syncthreads();
  for (int r = warp; r < 8 * kTiles && r0 + r < p.rows; r += kWarps) {
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.join.m[w][r]);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (sh.join.l[w][r] == 0.0f) continue;  // saw nothing
      const float f = ex2(sh.join.m[w][r] - top);
      sum = fmaf(f, sh.join.l[w][r], sum);
      const float4 v = *reinterpret_cast<const float4*>(&sh.join.o[w][r][4 * lane]);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    // g_V last: the quotient alone is in range, its product with a small g_V need not be
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum, gv = sh.gv_top;
    store_row(p, part, h, r0 + r, 4 * lane, make_float4(acc.x * f * gv, acc.y * f * gv, acc.z * f * gv, acc.w * f * gv),
              sum == 0.0f ? -INFINITY : top + log2f(sum) - kUp, lane == 0);
  }
}

// Joins the partial results (bound by the latency of reading them; 4 us for 24 rows of 24 parts):
// O = sum_i 2^(L_i - L) O_i, L = log2 sum_i 2^L_i.  kSplit warps of a CTA
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

// The same with a tree's drafts (64 drafts x 24 heads over 32768 keys: 81 us against 72
// for the window alone): kShare warps of a CTA of eight take a row, and deal out the drafts
// that it sees and the window's parts.
template <int kShare>
__global__ void __launch_bounds__(256) attend_join_tree_kernel(const __grid_constant__ Params p) {
  constexpr int kWide = 8, kJoin = 4, kAtOnce = kWide / kShare;
  __shared__ int32_t parents[kMaxTreeDrafts];
  __shared__ int16_t lists[kAtOnce][kMaxTreeDrafts];
  __shared__ float part[kShare > 1 ? kWide : 1][kD], part_m[kWide], part_l[kWide];
  __shared__ int listed[kAtOnce];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, turn = w % kShare;
  const int h = blockIdx.y;
  const int64_t n = (int64_t)p.heads * p.rows;
  const int64_t r = (int64_t)blockIdx.x * kAtOnce + w / kShare;
  const bool live = r < p.rows;
  const int64_t rr = h * p.rows + (live ? r : 0);
  const int i = (int)p.by_group.div((uint32_t)(live ? r : 0));
  const int head = h * p.group + (int)((live ? r : 0) - (int64_t)i * p.group);
  for (int j = threadIdx.x; j < p.drafts; j += 256) parents[j] = p.parents[j];
  __syncthreads();
  int16_t* list = lists[w / kShare];
  if (turn == 0 && lane == 0) listed[w / kShare] = live ? ancestors_of(p, parents, i, list) : 0;
  if (kShare > 1) __syncthreads();
  else __syncwarp();
  {
    RowSum row;
    if (live) {
      tree_row(p, list, listed[w / kShare], turn, kShare, i, h, head, row);
      for (int i0 = turn; i0 < p.parts; i0 += kShare * kJoin) {
        float l[kJoin], top = -INFINITY;
        float4 v[kJoin];
#pragma unroll
        for (int e = 0; e < kJoin; ++e) {
          const int at = i0 + e * kShare < p.parts ? i0 + e * kShare : i0;
          l[e] = p.part_l[at * n + rr];
          v[e] = *reinterpret_cast<const float4*>(p.part_o + (at * n + rr) * kD + 4 * lane);
          if (i0 + e * kShare >= p.parts) l[e] = -INFINITY;
          top = l[e] != l[e] || top != top ? NAN : fmaxf(top, l[e]);
        }
        if (top == -INFINITY) continue;
        row.raise(top);
#pragma unroll
        for (int e = 0; e < kJoin; ++e)
          if (l[e] != -INFINITY) row.add(ex2(l[e] - row.m), v[e]);
      }
    }
    if (kShare > 1) {
      *reinterpret_cast<float4*>(&part[w][4 * lane]) = make_float4(row.o[0], row.o[1], row.o[2], row.o[3]);
      if (lane == 0) part_m[w] = row.m, part_l[w] = row.l;
      __syncthreads();
    }
    if (live && turn == 0) {
      RowSum all = row;
      for (int e = w + 1; e < w + kShare; ++e) {
        if (part_m[e] == -INFINITY) continue;
        all.raise(part_m[e]);
        const float f = ex2(part_m[e] - all.m);
        all.l = fmaf(f, part_l[e], all.l);
#pragma unroll
        for (int d = 0; d < 4; ++d) all.o[d] = fmaf(f, part[e][4 * lane + d], all.o[d]);
      }
      const float inv = all.l == 0.0f ? 0.0f : 1.0f / all.l;
      stg_v2(p.o + (int64_t)i * p.o_pitch + ((int64_t)head * kD + 4 * lane) * 2,
             make_uint2(pack_bf16x2(all.o[0] * inv, all.o[1] * inv), pack_bf16x2(all.o[2] * inv, all.o[3] * inv)));
      if (lane == 0 && p.lse)
        p.lse[(int64_t)head * p.tq + i] = all.l == 0.0f ? -INFINITY : (all.m + log2f(all.l)) * kLn2;
    }
  }
}

// ------------------------------------------------------------------------------- host

constexpr int kSms = 148;

// Up to kRows rows a cache head take CTAs of few rows, above kMostRows tiles of 128; in between, where
// CTAs of few rows decode the window more than once but start sooner, and for the number of CTAs
// that share a window, the least of a model of the time decides, with constants from B200 (us, high for
// few rows, which no choice depends on: 0.7 of them moved no case by 10 %): a step of 32 keys takes a
// warp 1.8 (2.2 with 16 rows) and 0.12 (0.18) for each warp on its SM, a CTA 5 besides; a step of 64
// keys takes a tile's CTA 1.2 (two tiles) or 0.65, a CTA 14 besides; joining is another launch, 5, the
// partial results' traffic and 0.04 a part.
AttentionPlan make_plan(const int32_t* tokens, int n_slots, int heads, int64_t rows) {
  AttentionPlan best = {};
  double best_us = 0.0;
  for (int tiles = rows > kMostRows; tiles <= (rows > kRows ? 1 : 0); ++tiles) {
    AttentionPlan plan = {};
    plan.tiles = tiles != 0;
    plan.step = plan.tiles ? kTileKeys : kStep;
    int64_t steps = 0;
    for (int i = 0; i < n_slots; ++i) steps += (tokens[i] + plan.step - 1) / plan.step;
    plan.steps = (int32_t)steps;
    const bool pair = rows > kTileRows;
    const int64_t at_once = !plan.tiles ? kRows : pair ? 2 * kTileRows : kTileRows;
    const int64_t base = heads * ((rows + at_once - 1) / at_once);
    int64_t least = 1, most;
    if (plan.tiles) {
      least = std::max<int64_t>((steps + kMaxListed - 1) / kMaxListed, 1);
      most = std::min<int64_t>(steps / 4, kSms);
    } else {
      most = std::min<int64_t>((rows <= 8 ? 3 : 2) * kSms / base, steps / kWarps);
    }
    most = std::max(least, most);
    // every number of CTAs up to 32, then an eighth more at a time
    for (int64_t n = least; n <= most; n = n == most ? n + 1 : std::min(n + 1 + (n > 32 ? n / 8 : 0), most)) {
      double us;
      if (plan.tiles) {
        us = (double)((base * n + kSms - 1) / kSms) * ((double)((steps + n - 1) / n) * (pair ? 1.2 : 0.65) + 14.0);
      } else {
        const double warps = (double)(kWarps * n * base) / kSms;  // on an SM
        us = (double)((steps + n * kWarps - 1) / (n * kWarps)) * (rows <= 8 ? 1.8 + 0.12 * warps : 2.2 + 0.18 * warps) + 5.0;
      }
      if (n > 1) us += 5.0 + 0.04 * n + 2.0 * n * heads * rows * 516 / 5e6;
      if (best_us == 0.0 || us < best_us) {
        best_us = us;
        best = plan;
        best.splits = (int32_t)n;
      }
    }
  }
  return best;
}

template <bool kExtras, int kTiles>
cudaError_t launch_rows(const Params& p, dim3 grid, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {  // doing it twice is harmless
    e = cudaFuncSetAttribute(attend_rows_kernel<kExtras, kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  return launch_pdl(attend_rows_kernel<kExtras, kTiles>, grid, kThreads, sizeof(Shared), s, p);
}

}  // namespace
}  // namespace attend

AttentionPlan plan_attention(const int32_t* tokens, int n_slots, int heads, int64_t tq, int64_t group) {
  const int64_t rows = tq * group;
  AttentionPlan plan = attend::make_plan(tokens, n_slots, heads, std::max<int64_t>(rows, 1));
  // a window that is not shared out writes its results at once, unless drafts may have to be joined
  if (plan.splits > 1 || tq <= kMaxTreeDrafts)
    plan.workspace_bytes = (size_t)plan.splits * heads * rows * (attend::kD + 1) * sizeof(float);
  return plan;
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
  p.chunk = c.chunk_tokens;
  p.heads = c.heads;
  p.group = a.q_heads / c.heads;
  p.by_group = FastDiv((uint32_t)p.group);
  p.n_slots = a.n_slots;
  p.rows = a.tq * p.group;
  const AttentionPlan& plan = a.plan;
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
  p.parts = plan.splits;
  p.fold = a.parents && plan.splits == 1 && p.drafts <= kMaxFoldedDrafts && p.rows <= 8;
  if (p.parts > 1 || a.parents) {
    p.part_o = a.workspace;
    p.part_l = a.workspace + (int64_t)p.parts * p.heads * p.rows * kD;
  }
  const dim3 grid(p.parts, p.heads, (unsigned)((p.rows + kRows - 1) / kRows));  // of CTAs of few rows
  cudaError_t e;
  if (plan.tiles) e = launch_attend_tiles(p, s);
  else if (p.cap > 0.0f || p.slopes || p.k_doc)
    e = p.rows <= 8 ? launch_rows<true, 1>(p, grid, s) : launch_rows<true, 2>(p, grid, s);
  else
    e = p.rows <= 8 ? launch_rows<false, 1>(p, grid, s) : launch_rows<false, 2>(p, grid, s);
  if (e != cudaSuccess) return e;
  if (p.parents && !p.fold) {  // many drafts may be a long chain: two warps a row
    if (p.drafts <= 64)
      return launch_pdl(attend_join_tree_kernel<1>, dim3((unsigned)((p.rows + 7) / 8), p.heads), 256, 0, s, p);
    return launch_pdl(attend_join_tree_kernel<2>, dim3((unsigned)((p.rows + 3) / 4), p.heads), 256, 0, s, p);
  }
  if (p.parts == 1) return e;
  // few parts: a warp a row; more: eight warps share a row's
  if (p.parts <= 8) return launch_pdl(attend_join_kernel<1>, dim3((unsigned)((p.rows + 7) / 8), p.heads), 256, 0, s, p);
  return launch_pdl(attend_join_kernel<8>, dim3((unsigned)p.rows, p.heads), 256, 0, s, p);
}

}  // namespace nvfp4
