// layer.cu — what a transformer layer does between the GEMMs and the KV cache: RMS norm
// with the residual's addition and NVFP4 output, and rotary positions.  Both move each
// element once or twice and are bound by HBM.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kCached = 4;  // 16-value blocks of a row that a thread keeps in registers

__device__ __forceinline__ uint4 ldg_v4(const void* p) {  // plain load: the output may be the input's buffer
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// ------------------------------------------------------------------------ RMS norm
//   h = RN_t(x + residual)          (t: bf16 or FP32; the residual stream, stored)
//   r = RN(1 / sqrt(sum(h^2) / cols + eps)),  the sum, the division and the root in binary64
//   y = RN(RN(h * r) * w)
//   codes, scales, g = the NVFP4 quantization of y (FP32)
// The sum is binary64 because the codes are a step function of y: with an FP32 sum the
// last bits of r would depend on the order of the adds and elements next to an E2M1 border
// would change code with the launch shape.

enum NormMode {
  kGiven,   // g supplied: one pass over x (and residual)
  kAmax,    // first of two passes: h, max|y|
  kEncode,  // second of two passes: h read again (mostly L2), r recomputed, y encoded
};

struct NormParams {
  const uint8_t* x;
  const uint8_t* res;  // nullable
  uint8_t* h;          // nullable
  const uint8_t* w;    // nullable
  int64_t x_pitch, res_pitch, h_pitch;  // bytes
  bool w_bf16, h_wide;  // h_wide: rows of h are 32-byte aligned
  int64_t rows, vrows;  // vrows: rows rounded up to the scale layout's tile
  int32_t nb, vnb;      // blocks a row, and with the scale layout's padding
  double inv_cols, eps;
  uint8_t* codes;
  int64_t ld_codes;
  uint8_t* scales;
  int64_t ld_scales, groups;
  const float* gscale_in;
  float* gscale_out;
  unsigned* amax;  // nullable with a supplied scale
  int32_t stages;   // rows on their way to shared memory (kPipe)
  bool amax_store;  // CTA 0 sees every row: it stores the maximum instead of accumulating it
  unsigned* status;
};
constexpr int kSms = 148;
constexpr size_t kRowRingBytes = 220 * 1024;  // of an SM's shared memory, for rows on their way

// 16 values as loaded: 8 words of bf16 pairs or 16 FP32 words.
template <bool kBf16>
struct Block {
  uint32_t w[kBf16 ? 8 : 16];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int k = 0; k < (kBf16 ? 2 : 4); ++k) {
      const uint4 v = ldg_v4(p + 16 * k);
      w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
    }
  }
  __device__ __forceinline__ void load_shared(const uint8_t* p) {
#pragma unroll
    for (int k = 0; k < (kBf16 ? 2 : 4); ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * k);
      w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
    }
  }
  // wide: p is 32-byte aligned.  A thread's 32 bytes in one access fill whole sectors; two halves
  // cost the kernel 5 %.
  __device__ __forceinline__ void store(uint8_t* p, bool wide) const {
    if (wide) {
#pragma unroll
      for (int k = 0; k < (kBf16 ? 8 : 16); k += 8)
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + 4 * k), "r"(w[k]), "r"(w[k + 1]),
                     "r"(w[k + 2]), "r"(w[k + 3]), "r"(w[k + 4]), "r"(w[k + 5]), "r"(w[k + 6]), "r"(w[k + 7])
                     : "memory");
      return;
    }
#pragma unroll
    for (int k = 0; k < (kBf16 ? 2 : 4); ++k)
      stg_v4(p + 16 * k, make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
  }
  __device__ __forceinline__ float get(int k) const {
    if (!kBf16) return __uint_as_float(w[k % (kBf16 ? 8 : 16)]);
    return (k & 1) ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
  }
  __device__ __forceinline__ void add(const Block& o) {  // FP32 sum, rounded to the stream's type
    if (kBf16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float a, b;
        add2(a, b, get(2 * k), get(2 * k + 1), o.get(2 * k), o.get(2 * k + 1));
        w[k] = pack_bf16x2(a, b);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(get(k) + o.get(k));
    }
  }
};

template <bool kBf16, int kMode>
__device__ __forceinline__ Block<kBf16> norm_input(const NormParams& p, int64_t row, int32_t j) {
  const int64_t off = (int64_t)j * (kBf16 ? 32 : 64);
  Block<kBf16> b;
  if (kMode == kEncode && p.h) {  // written by the first pass (and it may be x or residual itself)
    b.load(p.h + row * p.h_pitch + off);
    return b;
  }
  b.load(p.x + row * p.x_pitch + off);
  if (p.res) {
    Block<kBf16> r;
    r.load(p.res + row * p.res_pitch + off);
    b.add(r);
  }
  return b;
}

template <bool kBf16>
__device__ __forceinline__ double block_squares(const Block<kBf16>& b) {
  double s0 = 0.0, s1 = 0.0;
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    const double u = b.get(k), v = b.get(k + 1);
    s0 = fma(u, u, s0);
    s1 = fma(v, v, s1);
  }
  return s0 + s1;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN of either stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// y of one block, and its largest magnitude's bits (a NaN or Inf gives bits >= 0x7F800000).
template <bool kBf16>
__device__ __forceinline__ unsigned norm_values(const NormParams& p, const Block<kBf16>& b, int32_t j, float r,
                                                float (&y)[16]) {
#pragma unroll
  for (int k = 0; k < 16; k += 2) mul2(y[k], y[k + 1], b.get(k), b.get(k + 1), r, r);
  if (p.w) {
    if (p.w_bf16) {
      const uint8_t* src = p.w + (int64_t)j * 32;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint4 v = ldg_nc_v4_l1(src + 16 * q);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float* v = y + 8 * q + 2 * k;
          mul2(v[0], v[1], v[0], v[1], bf16_lo(w[k]), bf16_hi(w[k]));
        }
      }
    } else {
      const uint8_t* src = p.w + (int64_t)j * 64;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 v = ldg_nc_v4_l1(src + 16 * q);
        float* u = y + 4 * q;
        mul2(u[0], u[1], u[0], u[1], __uint_as_float(v.x), __uint_as_float(v.y));
        mul2(u[2], u[3], u[2], u[3], __uint_as_float(v.z), __uint_as_float(v.w));
      }
    }
  }
  float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    m0 = max_nan(m0, fabsf(y[k]));
    m1 = max_nan(m1, fabsf(y[k + 1]));
  }
  return __float_as_uint(max_nan(m0, m1)) & 0x7FFFFFFFu;
}

template <bool kMma>
__device__ __forceinline__ void norm_encode(const NormParams& p, int64_t row, int32_t j, const float (&y)[16],
                                            unsigned amax_bits, float g, float d6, float r6) {
  const uint32_t s = block_scale_fast(__uint_as_float(amax_bits), d6, r6);
  const BlockEncoder enc(e4m3_to_float(s) * g);
  float v0[8], v1[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v0[k] = y[k];
    v1[k] = y[8 + k];
  }
  uint2 out;
  out.x = enc.encode8s(v0);
  out.y = enc.encode8s(v1);
  stg_v2(p.codes + row * p.ld_codes + (int64_t)j * 8, out);
  p.scales[kMma ? sf_mma_offset(row, j, p.groups) : row * p.ld_scales + j] = (uint8_t)s;
}

// Rows of x and residual on their way to shared memory, one bulk copy each.
constexpr unsigned long long kRowWaitNs = 2000000000ull;
constexpr int kMaxStages = 3;
struct RowRing {
  uint64_t full[kMaxStages];
  int abort;
};
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void fetch_row(const NormParams& p, int64_t row, uint32_t bytes, uint8_t* to,
                                          uint64_t* bar) {
  const uint32_t b = tc::smem_u32(bar), dst = tc::smem_u32(to);
  tc::mbar_arrive_expect_tx(b, 2 * bytes);
  bulk_load(dst, p.x + row * p.x_pitch, bytes, b);
  bulk_load(dst + bytes, p.res + row * p.res_pitch, bytes, b);
}

// 1 / sqrt of a row's mean square, from each thread's part of its sum.  kLanes threads a row: 8 (rows
// up to 8 blocks), 32 (up to 128 blocks), or the whole CTA, whose first warp then takes the root and
// the quotient for all (both are long in binary64: every warp taking them cost the kernel 1 %).
template <int kLanes>
__device__ __forceinline__ float row_factor(const NormParams& p, double v, double* red, float* shared_r) {
#pragma unroll
  for (int o = (kLanes == 8 ? 4 : 16); o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (kLanes <= 32) return (float)(1.0 / sqrt(v * p.inv_cols + p.eps));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    double s = red[0];
    for (int w = 1; w < (int)blockDim.x / 32; ++w) s += red[w];  // the same order in every pass
    const float r = (float)(1.0 / sqrt(s * p.inv_cols + p.eps));
    if (threadIdx.x == 0) *shared_r = r;
  }
  __syncthreads();
  return *shared_r;
}

// Registers for three CTAs of 256 threads an SM (80; two for FP32, whose rows take twice as many): a
// row's reads, reduction and encoding follow one another within a CTA, so others have to fill in.
// 9216 columns take CTAs of 192 threads, four of which fit; with the plain loads, 8192 x 9216 with
// residual took 122 us in registers for two CTAs of 256 threads, 107 for three, 117 for four, 135 for
// five.  Bound by HBM with the encoding's instructions close behind: 91 us for 495 MB (5.4 TB/s; without
// the encoding 78).  FP32 206 us for 949 MB; 8192 x 3072 45 us for 165 MB in bf16, 85 for 316 in FP32.
template <bool kBf16, bool kMma, int kMode, int kLanes, bool kPipe>
__global__ void __launch_bounds__(kThreads, kBf16 ? 3 : 2) norm_kernel(NormParams p) {
  extern __shared__ __align__(128) uint8_t rows_smem[];
  __shared__ RowRing ring;
  __shared__ double red[kThreads / 32];
  __shared__ float shared_r;
  __shared__ unsigned redm[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int lanes = kLanes > 32 ? (int)blockDim.x : kLanes;
  const int per_cta = (int)blockDim.x / lanes, warps = (int)blockDim.x / 32;
  const int lane = (int)threadIdx.x % lanes;
  float g = 0.0f;
  if (kMode == kGiven) {
    g = *p.gscale_in;
    if (!(g >= 0.0f) || !(g <= 3.402823466e38f)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, kStatusNonfinite);
      return;
    }
  } else if (kMode == kEncode) {
    const unsigned ab = *p.amax;
    if (ab >= 0x7F800000u) {
      if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, kStatusNonfinite);
      return;
    }
    g = __uint_as_float(ab) / 2688.0f;
  }
  if (kMode != kAmax && blockIdx.x == 0 && threadIdx.x == 0) *p.gscale_out = g;
  const float d6 = 6.0f * g, r6 = 1.0f / d6;
  const bool encodes = kMode != kAmax;
  const int64_t row_end = kMma && encodes ? p.vrows : p.rows;
  unsigned local_max = 0;
  const uint32_t block_bytes = kBf16 ? 32 : 64, row_bytes = (uint32_t)p.nb * block_bytes;
  const uint32_t stage_bytes = 2 * row_bytes;
  auto row_at = [&](int64_t base) { return kMode == kEncode ? row_end - 1 - base : base; };
  int stage = 0;
  uint32_t phases = 0;  // bit i: parity of ring place i's next phase
  if (kPipe) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < p.stages; ++i) tc::mbar_init(tc::smem_u32(&ring.full[i]), 1);
      ring.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      for (int i = 0; i < p.stages; ++i) {
        const int64_t row = row_at(blockIdx.x + (int64_t)i * gridDim.x);
        if (row >= 0 && row < p.rows) fetch_row(p, row, row_bytes, rows_smem + i * stage_bytes, &ring.full[i]);
      }
    }
    __syncthreads();
  }
  // every thread of the CTA takes the same number of steps: the reductions are collective
  for (int64_t base = (int64_t)blockIdx.x * per_cta; base < row_end; base += (int64_t)gridDim.x * per_cta) {
    // the second pass goes backwards: the first one's latest rows are the most likely still in L2
    const int64_t at = base + threadIdx.x / lanes, row = kMode == kEncode ? row_end - 1 - at : at;
    const bool live = row >= 0 && row < p.rows;
    Block<kBf16> kept[kCached];
    double ss = 0.0;
    if (kPipe) {
      if (live) {
        const uint8_t* src = rows_smem + stage * stage_bytes;
        const uint32_t bar = tc::smem_u32(&ring.full[stage]);
        if (!__syncthreads_and(tc::mbar_wait(bar, phases >> stage & 1u, &ring.abort, kRowWaitNs))) {
          if (threadIdx.x == 0) {
            set_status(p.status, kStatusTimeout);
            for (int i = 0; i < p.stages; ++i)  // copies still on their way
              tc::mbar_wait_drain(tc::smem_u32(&ring.full[i]), phases >> i & 1u, kRowWaitNs);
          }
          break;
        }
        phases ^= 1u << stage;
#pragma unroll
        for (int i = 0; i < kCached; ++i) {
          const int32_t j = lane + i * lanes;
          if (j < p.nb) {
            Block<kBf16> r;
            kept[i].load_shared(src + j * block_bytes);
            r.load_shared(src + row_bytes + j * block_bytes);
            kept[i].add(r);
          }
        }
        __syncthreads();  // the row is in registers: its place takes another
      }
      if (threadIdx.x == 0) {
        const int64_t next = row_at(base + (int64_t)p.stages * gridDim.x);
        if (next >= 0 && next < p.rows)
          fetch_row(p, next, row_bytes, rows_smem + stage * stage_bytes, &ring.full[stage]);
      }
      stage = stage + 1 == p.stages ? 0 : stage + 1;
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < kCached; ++i) {
        const int32_t j = lane + i * lanes;
        if (!kPipe && j < p.nb) kept[i] = norm_input<kBf16, kMode>(p, row, j);
      }
#pragma unroll
      for (int i = 0; i < kCached; ++i) {
        const int32_t j = lane + i * lanes;
        if (j < p.nb) {
          if (kMode != kEncode && p.h) kept[i].store(p.h + row * p.h_pitch + (int64_t)j * (kBf16 ? 32 : 64), p.h_wide);
          ss += block_squares(kept[i]);
        }
      }
      for (int32_t j = lane + kCached * lanes; j < p.nb; j += lanes) {  // rows too wide for the registers
        const Block<kBf16> b = norm_input<kBf16, kMode>(p, row, j);
        if (kMode != kEncode && p.h) b.store(p.h + row * p.h_pitch + (int64_t)j * (kBf16 ? 32 : 64), p.h_wide);
        ss += block_squares(b);
      }
    }
    const float r = row_factor<kLanes>(p, ss, red, &shared_r);
    if (live) {
#pragma unroll
      for (int i = 0; i < kCached; ++i) {
        const int32_t j = lane + i * lanes;
        if (j < p.nb) {
          float y[16];
          const unsigned m = norm_values(p, kept[i], j, r, y);
          local_max = max(local_max, m);
          if (encodes) norm_encode<kMma>(p, row, j, y, m, g, d6, r6);
        }
      }
      for (int32_t j = lane + kCached * lanes; j < p.nb; j += lanes) {
        // h_out when there is one: it may be x's or residual's buffer, which is gone by now
        const Block<kBf16> b = norm_input<kBf16, kEncode>(p, row, j);
        float y[16];
        const unsigned m = norm_values(p, b, j, r, y);
        local_max = max(local_max, m);
        if (encodes) norm_encode<kMma>(p, row, j, y, m, g, d6, r6);
      }
    }
    if (kMma && encodes && row >= 0 && row < p.vrows)  // padding of the tensor-core scale layout
      for (int32_t j = live ? p.nb + lane : lane; j < p.vnb; j += lanes) p.scales[sf_mma_offset(row, j, p.groups)] = 0;
  }
  if (kMode == kEncode) return;
  if (local_max >= 0x7F800000u) set_status(p.status, kStatusNonfinite);
  if (!p.amax) return;
  local_max = warp_max_u32(local_max);
  if ((threadIdx.x & 31) == 0) redm[threadIdx.x >> 5] = local_max;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < warps; ++w) local_max = max(local_max, redm[w]);
    if (p.amax_store && blockIdx.x == 0) *p.amax = local_max;
    else if (local_max != 0u) atomicMax(p.amax, local_max);
  }
}

template <bool kBf16, bool kMma, int kMode, int kLanes, bool kPipe>
cudaError_t launch_norm_kernel(NormParams p, int threads, cudaStream_t s) {
  const int per_cta = kLanes > 32 ? 1 : threads / kLanes;
  p.amax_store = p.rows <= per_cta;
  if (kMode != kEncode && p.amax && !p.amax_store) {
    const cudaError_t e = launch_zero_words(p.amax, 1, s);
    if (e != cudaSuccess) return e;
  }
  const int64_t rows = kMma && kMode != kAmax ? p.vrows : p.rows;
  // one wave of CTAs; a row a CTA (or 8 or 32 of them) at a time
  static std::atomic<int> resident[64][kThreads / 32 + 1];  // an SM's, per device and CTA size; racing writers agree
  int dev = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* known = dev >= 0 && dev < 64 ? &resident[dev][threads / 32] : nullptr;
  if (known) per_sm = known->load(std::memory_order_relaxed);
  auto kernel = norm_kernel<kBf16, kMma, kMode, kLanes, kPipe>;
  if (per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
    if (e == cudaSuccess && kPipe)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowRingBytes);
    if (e != cudaSuccess) return e;
    if (known) known->store(per_sm, std::memory_order_relaxed);
  }
  size_t smem = 0;
  if (kPipe) {
    const size_t stage = (size_t)p.nb * (kBf16 ? 32 : 64) * 2;
    const size_t fit = kRowRingBytes / per_sm / stage;  // rows, with as many CTAs as registers allow
    p.stages = (int32_t)std::max<size_t>(std::min<size_t>(fit, kMaxStages), 1);
    smem = p.stages * stage;
    per_sm = std::min<int>(per_sm, (int)(kRowRingBytes / smem));
  }
  const int64_t want = (rows + per_cta - 1) / per_cta, wave = (int64_t)per_sm * kSms;
  const int grid = (int)(want < wave ? want : wave);
  return launch_pdl(kernel, grid, threads, smem, s, p);
}

template <bool kBf16, bool kMma, int kMode>
cudaError_t launch_norm_mode(const NormParams& p, cudaStream_t s) {
  if (p.nb <= 8) return launch_norm_kernel<kBf16, kMma, kMode, 8, false>(p, kThreads, s);
  if (p.nb <= 32 * kCached) return launch_norm_kernel<kBf16, kMma, kMode, 32, false>(p, kThreads, s);
  // as many threads as share the row's blocks evenly
  const int rounds = (p.nb + kThreads - 1) / kThreads;
  const int threads = ((p.nb + rounds - 1) / rounds + 31) / 32 * 32;
  // x and residual through shared memory, the next row's on their way while this one's is encoded:
  // 8192 x 9216 takes 90 us so and 103 with plain loads, 8192 x 14336 151 and 167.  With x alone the
  // plain loads keep up (76 and 70), as they do for few rows a CTA (592 x 9216: 11.9 and 11.0) and one
  // block a thread (2368 x 4096: 20.3 and 20.1).
  const bool both = p.res && !(kMode == kEncode && p.h);
  if (both && rounds > 1 && rounds <= kCached && p.rows >= 8 * kSms)
    return launch_norm_kernel<kBf16, kMma, kMode, kThreads, true>(p, threads, s);
  return launch_norm_kernel<kBf16, kMma, kMode, kThreads, false>(p, threads, s);
}

template <bool kBf16, bool kMma>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.gscale_in) return launch_norm_mode<kBf16, kMma, kGiven>(p, s);
  const cudaError_t e = launch_norm_mode<kBf16, kMma, kAmax>(p, s);
  if (e != cudaSuccess) return e;
  return launch_norm_mode<kBf16, kMma, kEncode>(p, s);
}

// ---------------------------------------------------------------- rotary positions
//   (a, b) -> (a cos - b sin, a sin + b cos),  angle = position * frequency
// The angle is formed in binary64 as a number of turns, so that only its fraction is left
// for the FP32 sine and cosine (at position 10^6 an FP32 angle would be off by 2^-5).  A CTA
// takes a few tokens, computes their cosines and sines once into shared memory and applies
// them to its heads.  Bound by HBM: 32768 tokens x 24 heads x 128 in bf16 65 us (6.2 TB/s), 8191 x 23
// x 128 in FP32 with 72 interleaved 35 us (5.5 TB/s).

struct RopeParams {
  const uint8_t* x;
  uint8_t* y;
  int64_t x_pitch, y_pitch;  // bytes a token
  int64_t tokens;
  int32_t heads, head_bytes;
  int32_t half;       // rot_dim / 2
  int32_t tile;       // tokens a CTA
  int32_t head_split; // heads a CTA
  int32_t units;      // work items a (token, head): rotated ones first, then copied ones
  int32_t turned;     // of these, rotated
  FastDiv by_units, by_heads, by_last_heads;  // by_last_heads: the last CTA column may hold fewer heads
  const double* freq;
  float mscale;
  const int32_t* pos;  // nullable
  int64_t pos0;
};

// kVec elements (16 bytes) of a and of b an item, or single pairs where alignment or the
// number of rotated elements does not allow it.
template <bool kBf16, bool kInterleaved, bool kVector>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeParams p) {
  constexpr int kEsz = kBf16 ? 2 : 4;
  constexpr int kVec = kVector ? 16 / kEsz : 1;          // elements of one 16-byte access
  // items a thread reads at a time: 64 bytes on their way where an item is one 16-byte read
  constexpr int kRopeBatch = kInterleaved ? 4 : 2;
  constexpr int kPairs = kVector ? (kInterleaved ? kVec / 2 : kVec) : 1;  // pairs an item
  extern __shared__ float2 trig[];  // [token][pair group of 2][item] (two pairs = one 16-byte read)
  pdl_trigger();
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * p.tile;
  const int nt = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile);
  const int h0 = blockIdx.y * p.head_split;
  const int nh = p.heads - h0 < p.head_split ? p.heads - h0 : p.head_split;
  for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
    const int t = i / p.half, k = i - t * p.half;
    const int64_t pos = p.pos ? (int64_t)p.pos[t0 + t] : p.pos0 + t0 + t;
    double turns = (double)pos * (p.freq[k] * 0.15915494309189533577);  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif((float)(2.0 * turns), &s, &c);
    const int item = k / kPairs, e = k - item * kPairs;
    const int at = kVector ? t * p.half + (e / 2) * (2 * p.turned) + item * 2 + (e & 1) : i;
    trig[at] = make_float2(c * p.mscale, s * p.mscale);
  }
  __syncthreads();
  const int n = nt * nh * p.units;
  for (int i0 = threadIdx.x; i0 < n; i0 += kRopeBatch * kThreads) {
    // kRopeBatch items' reads on their way before the first is used
    const uint8_t* src[kRopeBatch];
    uint8_t* dst[kRopeBatch];
    int item[kRopeBatch], token[kRopeBatch];
    int64_t oa[kRopeBatch], ob[kRopeBatch];
    uint4 va[kRopeBatch], vb[kRopeBatch];
#pragma unroll
    for (int x = 0; x < kRopeBatch; ++x) {
      const int i = i0 + x * kThreads;
      if (i >= n) break;
      const uint32_t q = p.by_units.div((uint32_t)i);
      item[x] = i - (int)q * p.units;
      token[x] = (int)(nh == p.head_split ? p.by_heads.div(q) : p.by_last_heads.div(q));
      const int h = h0 + (int)q - token[x] * nh;
      src[x] = p.x + (t0 + token[x]) * p.x_pitch + (int64_t)h * p.head_bytes;
      dst[x] = p.y + (t0 + token[x]) * p.y_pitch + (int64_t)h * p.head_bytes;
      // a rotated item's a (and b); one behind them copies what follows the rotated elements
      const bool turned = item[x] < p.turned;
      oa[x] = turned ? (int64_t)item[x] * kPairs * (kInterleaved ? 2 : 1) * kEsz
                     : (int64_t)2 * p.half * kEsz + (int64_t)(item[x] - p.turned) * kVec * kEsz;
      ob[x] = kInterleaved ? oa[x] + kEsz : oa[x] + (int64_t)p.half * kEsz;
      if (kVector) {
        va[x] = ldg_v4(src[x] + oa[x]);
        if (!kInterleaved && turned) vb[x] = ldg_v4(src[x] + ob[x]);
      } else if (kBf16) {
        va[x].x = (uint32_t)*reinterpret_cast<const uint16_t*>(src[x] + oa[x]) << 16;
        if (turned) vb[x].x = (uint32_t)*reinterpret_cast<const uint16_t*>(src[x] + ob[x]) << 16;
      } else {
        va[x].x = *reinterpret_cast<const uint32_t*>(src[x] + oa[x]);
        if (turned) vb[x].x = *reinterpret_cast<const uint32_t*>(src[x] + ob[x]);
      }
    }
#pragma unroll
    for (int x = 0; x < kRopeBatch; ++x) {
      if (i0 + x * kThreads >= n) break;
      if (item[x] >= p.turned) {
        if (kVector) stg_v4(dst[x] + oa[x], va[x]);
        else if (kBf16) *reinterpret_cast<uint16_t*>(dst[x] + oa[x]) = (uint16_t)(va[x].x >> 16);
        else *reinterpret_cast<uint32_t*>(dst[x] + oa[x]) = va[x].x;
        continue;
      }
      float a[kPairs], b[kPairs];
      const uint32_t wa[4] = {va[x].x, va[x].y, va[x].z, va[x].w}, wb[4] = {vb[x].x, vb[x].y, vb[x].z, vb[x].w};
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        if (!kVector) {
          a[k] = __uint_as_float(wa[0]);
          b[k] = __uint_as_float(wb[0]);
        } else if (kInterleaved) {
          a[k] = kBf16 ? bf16_lo(wa[k & 3]) : __uint_as_float(wa[(2 * k) & 3]);
          b[k] = kBf16 ? bf16_hi(wa[k & 3]) : __uint_as_float(wa[(2 * k + 1) & 3]);
        } else {
          a[k] = !kBf16 ? __uint_as_float(wa[k & 3]) : (k & 1) ? bf16_hi(wa[(k / 2) & 3]) : bf16_lo(wa[(k / 2) & 3]);
          b[k] = !kBf16 ? __uint_as_float(wb[k & 3]) : (k & 1) ? bf16_hi(wb[(k / 2) & 3]) : bf16_lo(wb[(k / 2) & 3]);
        }
      }
      float ra[kPairs], rb[kPairs];
#pragma unroll
      for (int k = 0; k < kPairs; k += 2) {
        float2 cs[2];
        if (kVector) {
          const float4 v =
              *reinterpret_cast<const float4*>(&trig[token[x] * p.half + (k / 2) * (2 * p.turned) + item[x] * 2]);
          cs[0] = make_float2(v.x, v.y);
          cs[1] = make_float2(v.z, v.w);
        } else {
          cs[0] = trig[token[x] * p.half + item[x]];
        }
#pragma unroll
        for (int e = 0; e < 2 && k + e < kPairs; ++e) {
          ra[k + e] = fmaf(a[k + e], cs[e].x, -(b[k + e] * cs[e].y));
          rb[k + e] = fmaf(a[k + e], cs[e].y, b[k + e] * cs[e].x);
        }
      }
      if (kVector) {
        uint32_t sa[4], sb[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (kInterleaved) {
            sa[k] = kBf16 ? pack_bf16x2(ra[k % kPairs], rb[k % kPairs])
                          : __float_as_uint((k & 1) ? rb[(k / 2) % kPairs] : ra[(k / 2) % kPairs]);
          } else {
            sa[k] = kBf16 ? pack_bf16x2(ra[(2 * k) % kPairs], ra[(2 * k + 1) % kPairs]) : __float_as_uint(ra[k % kPairs]);
            sb[k] = kBf16 ? pack_bf16x2(rb[(2 * k) % kPairs], rb[(2 * k + 1) % kPairs]) : __float_as_uint(rb[k % kPairs]);
          }
        }
        stg_v4(dst[x] + oa[x], make_uint4(sa[0], sa[1], sa[2], sa[3]));
        if (!kInterleaved) stg_v4(dst[x] + ob[x], make_uint4(sb[0], sb[1], sb[2], sb[3]));
      } else if (kBf16) {
        const uint32_t v = pack_bf16x2(ra[0], rb[0]);
        *reinterpret_cast<uint16_t*>(dst[x] + oa[x]) = (uint16_t)(v & 0xFFFFu);
        *reinterpret_cast<uint16_t*>(dst[x] + ob[x]) = (uint16_t)(v >> 16);
      } else {
        *reinterpret_cast<float*>(dst[x] + oa[x]) = ra[0];
        *reinterpret_cast<float*>(dst[x] + ob[x]) = rb[0];
      }
    }
  }
}

template <bool kBf16, bool kInterleaved, bool kVector>
cudaError_t launch_rope_kernel(RopeParams& p, dim3 grid, size_t smem, cudaStream_t s) {
  return launch_pdl(rope_kernel<kBf16, kInterleaved, kVector>, grid, kThreads, smem, s, p);
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(const RmsnormArgs& a, cudaStream_t s) {
  const int64_t esz = a.x_bf16 ? 2 : 4;
  if (a.rows == 0) {  // an empty tensor: g as supplied or 0, max|y| = 0
    if (a.amax_out) {
      cudaError_t e = launch_zero_words(a.amax_out, 1, s);
      if (e != cudaSuccess) return e;
    }
    if (!a.gscale_in) return launch_zero_words(a.gscale_out, 1, s);
    return cudaMemcpyAsync(a.gscale_out, a.gscale_in, sizeof(float), cudaMemcpyDeviceToDevice, s);
  }
  NormParams p;
  p.x = (const uint8_t*)a.x;
  p.res = (const uint8_t*)a.residual;
  p.h = (uint8_t*)a.h_out;
  p.w = (const uint8_t*)a.weight;
  p.x_pitch = a.ldx * esz;
  p.res_pitch = a.ldr * esz;
  p.h_pitch = a.ldh * esz;
  p.h_wide = ((reinterpret_cast<uintptr_t>(a.h_out) | (uintptr_t)p.h_pitch) & 31u) == 0;
  p.w_bf16 = a.w_bf16;
  p.rows = a.rows;
  p.nb = (int32_t)(a.cols / 16);
  p.groups = (p.nb + 3) / 4;
  p.vnb = a.sf_mma ? (int32_t)p.groups * 4 : p.nb;
  p.vrows = a.sf_mma ? (a.rows + 127) / 128 * 128 : a.rows;
  p.inv_cols = 1.0 / (double)a.cols;
  p.eps = (double)a.eps;
  p.codes = a.codes;
  p.ld_codes = a.ld_codes;
  p.scales = a.scales;
  p.ld_scales = a.ld_scales;
  p.gscale_in = a.gscale_in;
  p.gscale_out = a.gscale_out;
  p.amax = reinterpret_cast<unsigned*>(a.amax_out);
  p.amax_store = false;
  p.status = a.status;
  if (a.x_bf16) return a.sf_mma ? launch_norm<true, true>(p, s) : launch_norm<true, false>(p, s);
  return a.sf_mma ? launch_norm<false, true>(p, s) : launch_norm<false, false>(p, s);
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  if (a.tokens == 0 || a.heads == 0) return cudaSuccess;
  const int esz = a.x_bf16 ? 2 : 4, vec = 16 / esz;
  const int half = a.rot_dim / 2, tail = a.head_dim - a.rot_dim;
  const bool inplace = a.x == a.y;
  auto multiple = [&](int64_t elements) { return elements % vec == 0; };
  const bool vector = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15u) == 0 &&
                      multiple(a.ldx) && multiple(a.ldy) && multiple(a.head_dim) && multiple(a.rot_dim) &&
                      (a.interleaved || multiple(half));
  RopeParams p;
  p.x = (const uint8_t*)a.x;
  p.y = (uint8_t*)a.y;
  p.x_pitch = a.ldx * esz;
  p.y_pitch = a.ldy * esz;
  p.tokens = a.tokens;
  p.heads = a.heads;
  p.head_bytes = a.head_dim * esz;
  p.half = half;
  const int pairs = !vector ? 1 : a.interleaved ? vec / 2 : vec;
  p.turned = half / pairs;
  p.units = p.turned + (inplace ? 0 : tail / (vector ? vec : 1));
  p.freq = a.freq;
  p.mscale = a.mscale;
  p.pos = a.positions;
  p.pos0 = a.pos0;
  // about 512 angles a CTA; fewer tokens, then fewer heads, until the grid has two CTAs an SM
  int sms = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int64_t tile = 512 / half > 0 ? 512 / half : 1;
  while (tile > 1 && (a.tokens + tile - 1) / tile < 2 * sms) tile = (tile + 1) / 2;
  int split = a.heads;
  while (split > 1 && (a.tokens + tile - 1) / tile * ((a.heads + split - 1) / split) < 2 * sms &&
         (int64_t)tile * split * p.units > kThreads)
    split = (split + 1) / 2;
  p.tile = (int32_t)tile;
  p.head_split = split;
  p.by_units = FastDiv((uint32_t)p.units);
  const dim3 grid((unsigned)((a.tokens + tile - 1) / tile), (unsigned)((a.heads + split - 1) / split));
  p.by_heads = FastDiv((uint32_t)split);
  p.by_last_heads = FastDiv((uint32_t)(a.heads - (a.heads - 1) / split * split));
  const size_t smem = (size_t)tile * half * sizeof(float2);
  if (a.x_bf16) {
    if (a.interleaved)
      return vector ? launch_rope_kernel<true, true, true>(p, grid, smem, s) : launch_rope_kernel<true, true, false>(p, grid, smem, s);
    return vector ? launch_rope_kernel<true, false, true>(p, grid, smem, s) : launch_rope_kernel<true, false, false>(p, grid, smem, s);
  }
  if (a.interleaved)
    return vector ? launch_rope_kernel<false, true, true>(p, grid, smem, s) : launch_rope_kernel<false, true, false>(p, grid, smem, s);
  return vector ? launch_rope_kernel<false, false, true>(p, grid, smem, s) : launch_rope_kernel<false, false, false>(p, grid, smem, s);
}

}  // namespace nvfp4
