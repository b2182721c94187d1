// attend_tiles.cu — softmax attention of many query rows over a window of the NVFP4 cache, on the
// fifth-generation tensor cores (attend.cuh gives the formulas).
#include <stddef.h>

#include <atomic>

#include "attend.cuh"
#include "tc.cuh"

namespace nvfp4 {
namespace attend {
namespace {

using namespace tc;

// One CTA of five warpgroups, one CTA an SM, in steps of 64 keys:
//   warps 0..3, 4..7  softmax of two tiles of 128 rows: thread = row
//   warps 8..11       decode the window's K to binary16 e2m1 * s in shared memory, 12..15 its V
//                     (one group doing both in turn was the slowest part of a step)
//   warps 16, 17      issue the tensor core's work of a tile each: S = Q K~^T and O += P V~
// Tensor memory holds, for each tile, two score buffers of 64 columns and the output (128).  The
// weights P (binary16) take the place of the scores they come from and are the A operand of the
// second product straight from there.  With two buffers the scores of the next step are ready
// when a softmax warpgroup has finished one: with one buffer of 128 keys a tile the chain scores,
// softmax, output ran in turn and the tensor core idled two thirds of the time.
//   kPair:  256 rows; both tiles take every step, so a decoded step feeds 256 rows.
//   !kPair: up to 128 rows; tile t takes the steps t, t + 2, ... and the two results are joined at
//           the end.
// 1024 queries x 24 heads x 32768 keys: 447 us, 920 TFLOP/s; no unit is above 47 % busy, and a
// step takes what a tile's chain takes (softmax about 1600 cycles for 64 keys, 550 from its weights
// to the next scores).  With a bias 744; with a cap 720 where scores stay within 0.625 of it, 1020
// where each warp's steps hold one beyond (tanh2's second form, 16 scores at a time); up to 128
// queries about 75.
// Both operands of both products are in the 128-byte swizzle: K~ as rows of keys (K-major), V~
// the same way, which for O += P V~ is the MN-major B operand, so one decoder writes both.
constexpr int kThreads = 640;
constexpr int kIssueWarp = 16;
constexpr int kQBytes = 128 * kD * 2;        // 32 KB: two 128-row x 128-byte blocks
constexpr int kQBlock = 128 * 128;
constexpr int kKvBytes = kTileKeys * kD * 2;  // 16 KB: two 64-row x 128-byte blocks
constexpr int kKvBlock = kTileKeys * 128;
constexpr int kStages = 4;
constexpr int kTmemCols = 512;
constexpr unsigned long long kWaitNs = 2000000000ull;

// Registers: the launch's 96 a thread (20 warps, five on each of the SM's four files) are moved
// between the warpgroups.
constexpr int kRegsLaunch = 96, kRegsSoftmax = 136, kRegsDecode = 64, kRegsIssue = 80;
static_assert(2 * kRegsSoftmax + 2 * kRegsDecode + kRegsIssue == 5 * kRegsLaunch, "the register split must balance");

struct Control {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2][2], p_ready[2][2], o_done[2], done[2];  // [tile][buffer]
  uint32_t tmem;
  volatile int abort;
  int32_t listed;
  int32_t q_first, q_last;
  float gv_top;
  int32_t row_pos[256], row_doc[256];
  float row_fac[256];  // factor of a row's products: scale and the power of two of its queries
  SlotView view[kMaxWindowSlots];
  float m[128], l[128];  // of tile 1, when the two are joined
};
constexpr int kControlBytes = (sizeof(Control) + 127) / 128 * 128;

constexpr int smem_bytes(bool pair) {
  return 1024 + (pair ? 2 : 1) * kQBytes + 2 * kStages * kKvBytes + kControlBytes + kMaxListed * 8 + kMaxTreeDrafts * 4;
}

// Instruction descriptor: D FP32 (bits 4..5 = 1), A and B binary16 (0), N >> 3, M >> 4; bit 16: B
// is MN-major.
constexpr uint32_t kIdescScores = (1u << 4) | ((uint32_t)(kTileKeys >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescOutput = (1u << 4) | (1u << 16) | ((uint32_t)(kD >> 3) << 17) | ((128u >> 4) << 24);

// Operand descriptors as two words, so that stepping through a tile is one 32-bit addition (the
// address field is the low word's): one thread issues every instruction of its tile.
__device__ __forceinline__ uint64_t descriptor(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

// accumulate == false: D = A B, else D += A B
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kIdescScores), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kIdescOutput), "r"((uint32_t)accumulate)
      : "memory");
}

// 32 columns of this thread's lane; the values may be used after ld_wait and ld_tie.
__device__ __forceinline__ void ld_x32(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Orders the uses of r behind the wait that was issued before this.
__device__ __forceinline__ void ld_tie(float* r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+f"(r[i]), "+f"(r[i + 1]), "+f"(r[i + 2]), "+f"(r[i + 3]), "+f"(r[i + 4]), "+f"(r[i + 5]),
                      "+f"(r[i + 6]), "+f"(r[i + 7]));
}
__device__ __forceinline__ void ld_x16(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void ld_tie16(float* r) {
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    asm volatile("" : "+f"(r[i]), "+f"(r[i + 1]), "+f"(r[i + 2]), "+f"(r[i + 3]), "+f"(r[i + 4]), "+f"(r[i + 5]),
                      "+f"(r[i + 6]), "+f"(r[i + 7]));
}
__device__ __forceinline__ void st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A listed key step: the cache row (slot * chunk_tokens + token) of its first key; its number of
// keys (bits 0..7), list entry of its slot (8..15) and whether every row sees all of it (16).
__device__ __forceinline__ uint2 listed_step(uint32_t row, int n, int seg, bool full) {
  return make_uint2(row, (uint32_t)n | ((uint32_t)seg << 8) | (full ? 1u << 16 : 0u));
}

template <bool kExtras, bool kPair>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(const __grid_constant__ Params p) {
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = smem;
  uint8_t* kbuf = qbuf + (kPair ? 2 : 1) * kQBytes;
  uint8_t* vbuf = kbuf + kStages * kKvBytes;
  Control& ct = *reinterpret_cast<Control*>(vbuf + kStages * kKvBytes);
  uint2* list = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(&ct) + kControlBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x, h = blockIdx.y;
  const int64_t r0 = (int64_t)blockIdx.z * (kPair ? 256 : 128);
  const int64_t r_end = min(r0 + (kPair ? 256 : 128), p.rows);
  const bool positions = p.causal || p.window || p.prefix || p.slopes;

  pdl_wait();
  int32_t* parents = reinterpret_cast<int32_t*>(list + kMaxListed);
  if (p.parents && positions) {
    for (int i = threadIdx.x; i < p.drafts; i += kThreads) parents[i] = p.parents[i];
    __syncthreads();
  }

  const bool two = kPair && r_end - r0 > 128;  // the second tile of a pair has rows
  if (threadIdx.x == 0) {
    for (int b = 0; b < kStages; ++b) {
      mbar_init(smem_u32(&ct.k_full[b]), 2);
      mbar_init(smem_u32(&ct.k_empty[b]), two ? 2 : 1);  // tiles that take a step
      mbar_init(smem_u32(&ct.v_full[b]), 2);
      mbar_init(smem_u32(&ct.v_empty[b]), two ? 2 : 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&ct.s_full[t][0]), 1);
      mbar_init(smem_u32(&ct.s_full[t][1]), 1);
      mbar_init(smem_u32(&ct.o_done[t]), 1);
      mbar_init(smem_u32(&ct.p_ready[t][0]), 4);
      mbar_init(smem_u32(&ct.p_ready[t][1]), 4);
      mbar_init(smem_u32(&ct.done[t]), 1);
    }
    ct.abort = 0;
    ct.q_first = 0x7FFFFFFF;
    ct.q_last = -0x7FFFFFFF - 1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ct.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();
  // the rows' positions and documents (the last row's for those behind the end), a thread a row
  if (warp < (kPair ? 8 : 4)) {
    const int64_t rr = r0 + threadIdx.x < r_end ? r0 + threadIdx.x : r_end - 1;
    const int qpos = positions ? row_position(p, parents, rr) : 0;
    const int lo = __reduce_min_sync(0xFFFFFFFFu, qpos), hi = __reduce_max_sync(0xFFFFFFFFu, qpos);
    if (lane == 0) {
      atomicMin(&ct.q_first, lo);
      atomicMax(&ct.q_last, hi);
    }
    ct.row_pos[threadIdx.x] = qpos;
    if (kExtras) ct.row_doc[threadIdx.x] = p.q_doc ? p.q_doc[p.by_group.div((uint32_t)rr)] : 0;
  }
  // the slots' scales by one warp, the queries by the others: half a warp a row, to binary16 scaled
  // by a power of two, into the swizzled operand tiles (zeros behind the last row)
  if (warp == kThreads / 32 - 1) {
    load_slots(p, ct.view, &ct.gv_top, part == 0 && h == 0 && blockIdx.z == 0);
  } else {
    constexpr int kQWarps = kThreads / 32 - 1, kRounds = ((kPair ? 128 : 64) + kQWarps - 1) / kQWarps;
    const int k = lane & 15;
    uint4 v[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {  // every read on its way before the first is used
      const int r = 2 * (warp + u * kQWarps) + (lane >> 4);
      const int64_t rr = r0 + r < r_end ? r0 + r : r_end - 1;
      const int64_t i = p.by_group.div((uint32_t)rr);
      const int head = h * p.group + (int)(rr - i * p.group);
      v[u] = ldg_nc_v4(p.q + i * p.q_pitch + (int64_t)head * kD * 2 + 16 * k);
    }
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      const int r = 2 * (warp + u * kQWarps) + (lane >> 4);
      unsigned top = __vmaxu2(__vmaxu2(v[u].x & 0x7FFF7FFFu, v[u].y & 0x7FFF7FFFu),
                              __vmaxu2(v[u].z & 0x7FFF7FFFu, v[u].w & 0x7FFF7FFFu));
      top = max(top >> 16, top & 0xFFFFu);
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
      if (r >= (kPair ? 256 : 128)) continue;
      const int e = query_exponent(top);
      const bool some = r0 + r < r_end;
      // a negative scale goes into the queries, so that larger products are larger scores
      const float up = copysignf(top >= 0x7F80u ? NAN : exp2i(e), p.scale);
      const uint4 w = make_uint4(pack_f16x2(bf16_lo(v[u].x) * up, bf16_hi(v[u].x) * up),
                                 pack_f16x2(bf16_lo(v[u].y) * up, bf16_hi(v[u].y) * up),
                                 pack_f16x2(bf16_lo(v[u].z) * up, bf16_hi(v[u].z) * up),
                                 pack_f16x2(bf16_lo(v[u].w) * up, bf16_hi(v[u].w) * up));
      *reinterpret_cast<uint4*>(qbuf + (r >> 7) * kQBytes + (k >> 3) * kQBlock + (r & 127) * 128 +
                                (((k & 7) ^ (r & 7)) << 4)) = some ? w : make_uint4(0, 0, 0, 0);
      if (k == 0) ct.row_fac[r] = fabsf(p.scale) * exp2i(-e);
    }
    fence_proxy_async_smem();
  }
  __syncthreads();
  // the key steps of this CTA's range that some row sees, in order
  const int first = (int)((int64_t)p.steps * part / p.splits), last = (int)((int64_t)p.steps * (part + 1) / p.splits);
  const int n_range = last - first;  // at most kMaxListed
  uint8_t* flags = kbuf;             // 0 unseen, 1 partly, 2 wholly seen; the slot's entry behind
  uint8_t* segs = kbuf + kMaxListed;
  for (int rel = threadIdx.x; rel < n_range; rel += kThreads) {
    const int st = first + rel;
    int seg = 0;
    while (st >= p.step_end[seg]) ++seg;
    const int t0 = (st - (seg ? p.step_end[seg - 1] : 0)) * kTileKeys;
    const int n = min(kTileKeys, p.tokens[seg] - t0);
    int vis = ct.view[seg].ok ? visibility(p, p.pos[seg] + t0, p.pos[seg] + t0 + n - 1, ct.q_first, ct.q_last) : 0;
    if (vis == 2 && n < kTileKeys) vis = 1;
    flags[rel] = (uint8_t)vis;
    segs[rel] = (uint8_t)seg;
  }
  __syncthreads();
  if (kExtras && p.k_doc) {  // one warp a step: the range of its keys' documents
    for (int rel = warp; rel < n_range; rel += kThreads / 32) {
      if (flags[rel] == 0) continue;
      const int seg = segs[rel];
      int64_t base = 0;
      for (int i = 0; i < seg; ++i) base += p.tokens[i];
      const int t0 = (first + rel - (seg ? p.step_end[seg - 1] : 0)) * kTileKeys;
      const int n = min(kTileKeys, p.tokens[seg] - t0);
      int lo = 0x7FFFFFFF, hi = -0x7FFFFFFF - 1;
      for (int k = lane; k < n; k += 32) {
        const int d = p.k_doc[base + t0 + k];
        lo = min(lo, d);
        hi = max(hi, d);
      }
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      __syncwarp();
      bool some = false, every = lo == hi;  // rows with a document among them; rows of just that one
      for (int r = lane; r < (kPair ? 256 : 128); r += 32) {
        const int d = ct.row_doc[r];
        some |= d >= lo && d <= hi;
        every &= d == lo;
      }
      some = __any_sync(0xFFFFFFFFu, some);
      every = __all_sync(0xFFFFFFFFu, every);
      if (lane == 0) flags[rel] = !some ? 0 : every ? flags[rel] : 1;
    }
    __syncthreads();
  }
  if (warp == 0) {
    int n = 0;
    for (int b = 0; b < n_range; b += 32) {
      const int rel = b + lane;
      const int vis = rel < n_range ? flags[rel] : 0;
      const unsigned seen = __ballot_sync(0xFFFFFFFFu, vis != 0);
      if (vis) {
        const int seg = segs[rel];
        const int t0 = (first + rel - (seg ? p.step_end[seg - 1] : 0)) * kTileKeys;
        list[n + __popc(seen & ((1u << lane) - 1u))] =
            listed_step((uint32_t)((int64_t)p.slots[seg] * p.chunk + t0), min(kTileKeys, p.tokens[seg] - t0), seg, vis == 2);
      }
      n += __popc(seen);
    }
    if (lane == 0) ct.listed = n;
  }
  fence_before();
  __syncthreads();  // the flags' memory belongs to the decoders from here on
  fence_after();
  const uint32_t tmem = ct.tmem;
  const int n = ct.listed;
  volatile int* abort_flag = &ct.abort;

  if (warp >= kIssueWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    const int t = warp - kIssueWarp;
    if (t < (two || !kPair ? 2 : 1) && lane == 0) {
      // ---------------------------------------------------- tensor core, tile t
      // Few instructions between a wait and what it lets go: the other warps leave this one few issue
      // slots.  The loop is unrolled over the ring, so buffers and barriers are constants.
      const uint32_t hi = (uint32_t)(smem_desc(0, 0, 1024, 2) >> 32);
      const uint32_t q_lo = (uint32_t)smem_desc(smem_u32(qbuf + (kPair ? t : 0) * kQBytes), 16, 1024, 2);
      // a pair's tiles both take every step; else tile t takes steps t, t + 2, ...: buffers t, t + 2
      const uint32_t k_lo = (uint32_t)smem_desc(smem_u32(kbuf) + (kPair ? 0 : t * kKvBytes), 16, 1024, 2);
      const uint32_t v_lo = (uint32_t)smem_desc(smem_u32(vbuf) + (kPair ? 0 : t * kKvBytes), kKvBlock, 1024, 2);
      const uint32_t ts = tmem + t * 128, to = tmem + 256 + t * 128;
      const uint32_t bars = smem_u32(&ct) + (kPair ? 0 : 8 * t), tbars = smem_u32(&ct) + 16 * t;
      constexpr uint32_t kKFull = offsetof(Control, k_full), kKEmpty = offsetof(Control, k_empty);
      constexpr uint32_t kVFull = offsetof(Control, v_full), kVEmpty = offsetof(Control, v_empty);
      constexpr uint32_t kSFull = offsetof(Control, s_full), kPReady = offsetof(Control, p_ready);
      constexpr int kMine = kPair ? kStages : kStages / 2, kStride = kPair ? 1 : 2;  // ring buffers of a tile
      const uint32_t o_done = smem_u32(&ct.o_done[t]);
      const int n_mine = kPair ? n : (n + 1 - t) / 2;
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok && !mbar_wait(bar, parity, abort_flag, kWaitNs)) ok = false;
      };
      auto scores = [&](int e, uint32_t parity) {  // S_t = Q_t K~^T from this tile's ring buffer e
        wait(bars + kKFull + 8 * kStride * e, parity);
        fence_after();
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk)
          mma_ss(ts + (e & 1) * kTileKeys, descriptor(q_lo + (((kk >> 2) * kQBlock + (kk & 3) * 32) >> 4), hi),
                 descriptor(k_lo + ((kStride * e * kKvBytes + (kk >> 2) * kKvBlock + (kk & 3) * 32) >> 4), hi), kk > 0);
        commit(tbars + kSFull + 8 * (e & 1));
        commit(bars + kKEmpty + 8 * kStride * e);
      };
      if (n_mine > 0) scores(0, 0);
      if (n_mine > 1) scores(1 % kMine, (uint32_t)(1 / kMine) & 1u);
      uint32_t ring = 0;  // parity of the ring's round
      for (int i0 = 0; i0 < n_mine && ok; i0 += kMine, ring ^= 1u) {
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
          const int i = i0 + e;
          if (i >= n_mine || !ok) break;
          // O_t += P_t V~, 16 keys an instruction
          const uint32_t half = kMine == 4 ? (uint32_t)(e >> 1) : ring;  // parity of score buffer e & 1
          wait(bars + kVFull + 8 * kStride * e, ring);
          wait(tbars + kPReady + 8 * (e & 1), half);
          fence_after();
#pragma unroll
          for (int kk = 0; kk < kTileKeys / 16; ++kk)
            mma_ts(to, ts + (e & 1) * kTileKeys + kk * 8,
                   descriptor(v_lo + ((kStride * e * kKvBytes + kk * 2048) >> 4), hi), i > 0 || kk > 0);
          commit(o_done);
          commit(bars + kVEmpty + 8 * kStride * e);
          // the scores of step i + 2 take the buffer whose weights this reads; the two products differ
          // in shape, so only completion orders them (those of step i + 1 are there already)
          if (i + 2 < n_mine) {
            wait(o_done, (uint32_t)e & 1u);
            scores((e + 2) % kMine, ring ^ (uint32_t)((e + 2) / kMine & 1));
          }
        }
      }
      if (!ok) {
        set_status(p.status, kStatusTimeout);
        *abort_flag = 1;
      }
      commit(smem_u32(&ct.done[t]));
      mbar_wait_drain(smem_u32(&ct.done[t]), 0, kWaitNs);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ decoders
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
    // Two warps take every other step: a step's fixed costs (its barriers, and the proxy fence, which
    // waits for the stores) are then paid once per 32 keys of a warp, and two steps overlap.
    // thread: dims 32 c .. 32 c + 31 (16 bytes of codes, two scale bytes) of keys key0 + 16 u; the
    // lanes of a quarter warp store to 8 different 16-byte banks (4 keys x 2 chunks of one block)
    const int c = (lane & 1) | (((lane >> 3) & 1) << 1);
    const int key0 = ((lane >> 1) & 3) | ((lane >> 4) << 2) | ((warp & 1) << 3);
    const uint32_t code_step = (uint32_t)p.heads * (kD / 2), scale_step = (uint32_t)p.heads * (kD / 16);
    struct Raw {
      uint4 w[4];
      uint32_t s[4];
    };
    const bool is_v = warp >= 12;
    const uint32_t dst0 = smem_u32(is_v ? vbuf : kbuf) + (c >> 1) * kKvBlock + key0 * 128;
    const uint32_t full = smem_u32(is_v ? ct.v_full : ct.k_full), empty = smem_u32(is_v ? ct.v_empty : ct.k_empty);
    const uint8_t* codes0 = p.base + (is_v ? p.off_v_codes : p.off_k_codes) + (int64_t)h * (kD / 2) + 16 * c;
    const uint8_t* scales0 = p.base + (is_v ? p.off_v_scales : p.off_k_scales) + (int64_t)h * (kD / 16) + 2 * c;
    auto fetch = [&](Raw& r, const uint2 st) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {  // keys behind the step's last repeat it; their weights are 0
        const uint32_t row = st.x + (uint32_t)min(key0 + 16 * u, (int)(st.y & 0xFFu) - 1);
        r.w[u] = ldg_nc_v4(codes0 + (uint64_t)row * code_step);
        r.s[u] = ldg_nc_u16(scales0 + (uint64_t)row * scale_step);
      }
    };
    Raw raw;  // the next step of this pair, on its way since the last one was decoded
    int j = (warp >> 1) & 1;
    if (j < n) fetch(raw, list[j]);
    bool ok = true;
    for (; j < n; j += 2) {
      const int b = j % kStages;
      const uint2 next = list[min(j + 2, n - 1)];
      ok = __all_sync(0xFFFFFFFFu,
                      mbar_wait(empty + 8 * b, ((uint32_t)(j / kStages) & 1u) ^ 1u, abort_flag, kWaitNs));
      if (!ok) break;
      const uint32_t dst = dst0 + b * kKvBytes;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t words[4] = {raw.w[u].x, raw.w[u].y, raw.w[u].z, raw.w[u].w};
        const uint32_t s2[2] = {e4m3_to_f16x2_bcast(raw.s[u] & 0xFFu), e4m3_to_f16x2_bcast(raw.s[u] >> 8)};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t v[4];
          e2m1x8_times_scale(words[w], s2[w >> 1], v);
          st_shared_v4(dst + u * (16 * 128) + (((4 * (c & 1) + w) ^ (key0 & 7)) << 4),
                       make_uint4(v[0], v[1], v[2], v[3]));
        }
      }
      fetch(raw, next);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * b);
    }
    if (!ok) {
      if (lane == 0) set_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
  } else {
    // ------------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int tile = warp >> 2, slot_row = (kPair ? tile * 128 : 0) + (threadIdx.x & 127);
    const int64_t row = r0 + slot_row;
    const bool live = row < r_end;
    const int qpos = ct.row_pos[slot_row], qdoc = kExtras ? ct.row_doc[slot_row] : 0;
    const float fac = ct.row_fac[slot_row];
    float slope = 0.0f;
    if (kExtras && p.slopes) {
      const int64_t rr = live ? row : r_end - 1;
      slope = p.slopes[h * p.group + (int)(rr - (int64_t)p.by_group.div((uint32_t)rr) * p.group)] * kLog2e;
    }
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + tile * 128, to = tmem + lanes + 256 + tile * 128;
    const uint8_t* qrow = qbuf + (kPair ? tile : 0) * kQBytes + (threadIdx.x & 127) * 128;
    const int n_mine = kPair ? (tile == 0 || two ? n : 0) : (n + 1 - tile) / 2;
    float m = -INFINITY, l = 0.0f;
    float mul = 0.0f, bias = 0.0f, lg = 0.0f, inv = 1.0f;
    bool vzero = false, ok = true;
    int seg_at = -1;
    const bool idle = __all_sync(0xFFFFFFFFu, !live);  // no row of this warp's: its lanes of P and O are left as they are
    for (int i = 0; i < n_mine; ++i) {
      if (idle) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ct.s_full[tile][i & 1]), (uint32_t)(i >> 1) & 1u, abort_flag,
                                               kWaitNs))) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive(smem_u32(&ct.p_ready[tile][i & 1]));
        continue;
      }
      const uint2 st = list[kPair ? i : 2 * i + tile];
      const int st_n = (int)(st.y & 0xFFu);
      const bool full = st.y >> 16;
      if ((int)(st.y >> 8 & 0xFFu) != seg_at) {  // the slot's scales, and q . mu of this row
        seg_at = (int)(st.y >> 8 & 0xFFu);
        const SlotView sv = ct.view[seg_at];
        lg = sv.lg, inv = sv.inv, vzero = sv.vzero;
        const float4* mu = reinterpret_cast<const float4*>(
            p.base + p.off_mu + ((int64_t)p.slots[seg_at] * p.heads + h) * kD * 4);
        float acc0 = 0.0f, acc1 = 0.0f;
#pragma unroll 4
        for (int k = 0; k < 16; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(qrow + (k >> 3) * kQBlock +
                                                          (((k & 7) ^ (threadIdx.x & 7)) << 4));
          const float4 m0 = __ldg(mu + 2 * k), m1 = __ldg(mu + 2 * k + 1);
          float x, y;
          f16x2_to_f32x2(v.x, x, y);
          acc0 = fmaf(x, m0.x, acc0), acc1 = fmaf(y, m0.y, acc1);
          f16x2_to_f32x2(v.y, x, y);
          acc0 = fmaf(x, m0.z, acc0), acc1 = fmaf(y, m0.w, acc1);
          f16x2_to_f32x2(v.z, x, y);
          acc0 = fmaf(x, m1.x, acc0), acc1 = fmaf(y, m1.y, acc1);
          f16x2_to_f32x2(v.w, x, y);
          acc0 = fmaf(x, m1.z, acc0), acc1 = fmaf(y, m1.w, acc1);
        }
        // log2 units, or shares of the cap
        const float f = kExtras && p.cap > 0.0f ? fac / p.cap : fac * kLog2e;
        bias = (acc0 + acc1) * f;
        mul = f * sv.gk;
      }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ct.s_full[tile][i & 1]), (uint32_t)(i >> 1) & 1u, abort_flag,
                                             kWaitNs))) {
        ok = false;
        break;
      }
      fence_after();
      const uint32_t si = ts + (i & 1) * kTileKeys;
      float s[kTileKeys];
      ld_x32(si, s);
      ld_x32(si + 32, s + 32);
      ld_wait();
      ld_tie(s);
      ld_tie(s + 32);
      float top, scale = mul, shift = bias;
      if (full && !kExtras) {
        float t0 = s[0], t1 = s[1];
#pragma unroll
        for (int e = 2; e + 3 < kTileKeys; e += 4) {
          t0 = fmaxf(t0, fmaxf(s[e], s[e + 1]));
          t1 = fmaxf(t1, fmaxf(s[e + 2], s[e + 3]));
        }
        top = fmaf(fmaxf(fmaxf(t0, t1), fmaxf(s[kTileKeys - 2], s[kTileKeys - 1])), mul, bias);
      } else {
        // cap, bias and mask: raw products to log2 units, with -inf where the row does not see the key
        const int t0 = (int)(st.x - (uint32_t)((int64_t)p.slots[seg_at] * p.chunk));
        const int kp0 = p.pos[seg_at] + t0;
#pragma unroll
        for (int e = 0; e < kTileKeys; e += 2) fma2(s[e], s[e + 1], s[e], s[e + 1], mul, mul, bias, bias);
        if (kExtras && p.cap > 0.0f) {
          const float cap = p.cap * kLog2e;
          float far = 0.0f;
#pragma unroll
          for (int e = 0; e < kTileKeys; e += 2) far = fmaxf(far, fmaxf(fabsf(s[e]), fabsf(s[e + 1])));
          if (__all_sync(0xFFFFFFFFu, far <= kTanhNear)) {
#pragma unroll
            for (int e = 0; e < kTileKeys; e += 2) {
              tanh_near2(s[e], s[e + 1]);
              mul2(s[e], s[e + 1], s[e], s[e + 1], cap, cap);
            }
          } else {
            // the rarer form 16 scores at a time through their tensor memory: unrolled over all 64 its
            // code and registers slowed the other paths as well (a bias without a cap by 7 %)
#pragma unroll 1
            for (int k = 0; k < kTileKeys; k += 16) {
              float x[16];
              uint32_t w[16];
              ld_x16(si + k, x);
              ld_wait();
              ld_tie16(x);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                x[e] = fmaf(x[e], mul, bias), x[e + 1] = fmaf(x[e + 1], mul, bias);
                tanh2(x[e], x[e + 1]);
                w[e] = __float_as_uint(x[e] * cap), w[e + 1] = __float_as_uint(x[e + 1] * cap);
              }
              st_x16(si + k, w);
            }
            st_wait();
            ld_x32(si, s);
            ld_x32(si + 32, s + 32);
            ld_wait();
            ld_tie(s);
            ld_tie(s + 32);
          }
        }
        if (kExtras && p.slopes) {
          const float d0 = (float)(qpos - kp0);
#pragma unroll
          for (int e = 0; e < kTileKeys; ++e) s[e] = fmaf(-slope, fabsf(d0 - (float)e), s[e]);
        }
        if (!full) {
          // visible: keys [lo, hi) of the step, and those below pre
          int lo = 0, hi = st_n, pre = 0;
          if (p.causal) hi = (int)min((int64_t)hi, max((int64_t)0, (int64_t)qpos - kp0 + 1));
          if (p.window) lo = (int)max((int64_t)0, (int64_t)qpos - kp0 - p.window + 1);
          if (p.prefix > kp0) pre = min(p.prefix - kp0, st_n);
          const int32_t* docs = p.k_doc;
          if (kExtras && docs) {
            for (int e = 0; e < seg_at; ++e) docs += p.tokens[e];
            docs += t0;
          }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            auto below = [&](int c) { c -= 32 * w; return c >= 32 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << c) - 1u; };
            uint32_t see = (below(hi) & ~below(lo)) | below(pre);
            if (kExtras && docs) {
              const int doc = docs[min(32 * w + lane, st_n - 1)];
              const int row0 = __shfl_sync(0xFFFFFFFFu, qdoc, 0);
              if (__all_sync(0xFFFFFFFFu, qdoc == row0)) {  // the warp's rows are of one document
                see &= __ballot_sync(0xFFFFFFFFu, doc == row0);
              } else {
                uint32_t same = 0;
#pragma unroll 4
                for (int e = 0; e < 32; ++e) same |= (uint32_t)(__shfl_sync(0xFFFFFFFFu, doc, e) == qdoc) << e;
                see &= same;
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) s[32 * w + e] = (see >> e) & 1u ? s[32 * w + e] : -INFINITY;
          }
        }
        top = -INFINITY;
#pragma unroll
        for (int e = 0; e < kTileKeys; e += 2) top = fmaxf(top, fmaxf(s[e], s[e + 1]));
        scale = 1.0f;
        shift = 0.0f;
      }
      const float need = top + lg;
      const bool grow = need > m + kLazy || (m == -INFINITY && need > -INFINITY);
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float alpha = grow ? ex2(m - need) : 1.0f;
        if (grow) m = need;
        l *= alpha;
        if (i > 0) {  // the output of the step before has to be complete
          if (!__all_sync(0xFFFFFFFFu,
                          mbar_wait(smem_u32(&ct.o_done[tile]), (uint32_t)(i - 1) & 1u, abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          fence_after();
#pragma unroll 1
          for (int k = 0; k < kD; k += 16) {
            float o[16];
            ld_x16(to + k, o);
            ld_wait();
            ld_tie16(o);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
            st_x16(to + k, w);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m - lg - kUp;
      const float c0 = shift - ref;
      float sum0 = 0.0f, sum1 = 0.0f, sum2 = 0.0f, sum3 = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float* x = s + 32 * k + e;
          fma2(x[0], x[1], x[0], x[1], scale, scale, c0, c0);
          fma2(x[2], x[3], x[2], x[3], scale, scale, c0, c0);
          x[0] = ex2(x[0]), x[1] = ex2(x[1]), x[2] = ex2(x[2]), x[3] = ex2(x[3]);
          add2(sum0, sum1, sum0, sum1, x[0], x[1]);
          add2(sum2, sum3, sum2, sum3, x[2], x[3]);
          w[e / 2] = pack_f16x2(x[0], x[1]);
          w[e / 2 + 1] = pack_f16x2(x[2], x[3]);
        }
        if (vzero) {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0;
        }
        st_x16(si + 16 * k, w);
      }
      l = fmaf((sum0 + sum1) + (sum2 + sum3), inv, l);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ct.p_ready[tile][i & 1]));
    }
    // a tile's own work; where the two are joined through the key buffers, the other's too
    for (int t = 0; t < 2 && ok; ++t) {
      if (kPair && (t != tile || (t == 1 && !two))) continue;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&ct.done[t]), 0, abort_flag, kWaitNs));
    }
    if (!ok) {
      if (lane == 0) set_status(p.status, kStatusTimeout);
      *abort_flag = 1;
    }
    fence_after();
    {  // after a wait that gave up as well: every softmax warp meets at the barrier below
      float other = 0.0f;  // factor of tile 1's output, when the two are joined
      float mine = 1.0f;
      if (!kPair) {
        // tile 1 hands over through the decoders' buffers, 16 bytes of a row side by side with the
        // next row's
        float4* hand = reinterpret_cast<float4*>(kbuf);
        if (tile == 1) {
          ct.m[threadIdx.x & 127] = m;
          ct.l[threadIdx.x & 127] = l;
          if (n_mine > 0) {
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              float o[32];
              ld_x32(to + 32 * k, o);
              ld_wait();
              ld_tie(o);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                hand[(8 * k + e) * 128 + (threadIdx.x & 127)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tile == 0) {
          const float m1 = ct.m[threadIdx.x & 127], l1 = ct.l[threadIdx.x & 127];
          const float mt = fmaxf(m, m1);
          if (l1 != 0.0f) {
            other = ex2(m1 - mt);
            mine = l != 0.0f ? ex2(m - mt) : 0.0f;
            l = l * mine + l1 * other;
            m = mt;
          }
        }
      }
      if (kPair || tile == 0) {
        // g_V last: the quotient alone is in range, its product with a small g_V need not be
        const float f = l == 0.0f ? 0.0f : 1.0f / l, gv = ct.gv_top;
        mine *= f;
        other *= f;
        const float log2l = l == 0.0f ? -INFINITY : m + log2f(l) - kUp;
        const float4* hand = reinterpret_cast<const float4*>(kbuf);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          float o[32];
          if (n_mine > 0) {  // warp-uniform
            ld_x32(to + 32 * k, o);
            ld_wait();
            ld_tie(o);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (l != 0.0f && n_mine > 0 && mine != 0.0f)
              v = make_float4(o[4 * e] * mine, o[4 * e + 1] * mine, o[4 * e + 2] * mine, o[4 * e + 3] * mine);
            if (!kPair && other != 0.0f) {
              const float4 u = hand[(8 * k + e) * 128 + (threadIdx.x & 127)];
              v.x = fmaf(u.x, other, v.x);
              v.y = fmaf(u.y, other, v.y);
              v.z = fmaf(u.z, other, v.z);
              v.w = fmaf(u.w, other, v.w);
            }
            v.x *= gv, v.y *= gv, v.z *= gv, v.w *= gv;
            if (live) store_row(p, part, h, row, 32 * k + 4 * e, v, log2l, k == 0 && e == 0);
          }
        }
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kIssueWarp) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

template <bool kExtras, bool kPair>
cudaError_t launch(const Params& p, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {  // doing it twice is harmless
    // the register split balances only for this launch count: with fewer the softmax warps would
    // wait for registers that nobody releases
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, attend_tiles_kernel<kExtras, kPair>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;
    e = cudaFuncSetAttribute(attend_tiles_kernel<kExtras, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes(kPair));
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  const int64_t group = (kPair ? 2 : 1) * kTileRows;
  return launch_pdl(attend_tiles_kernel<kExtras, kPair>, dim3(p.splits, p.heads, (unsigned)((p.rows + group - 1) / group)),
                    kThreads, smem_bytes(kPair), s, p);
}

}  // namespace

cudaError_t launch_attend_tiles(const Params& p, cudaStream_t s) {
  const bool extras = p.cap > 0.0f || p.slopes || p.k_doc;
  if (p.rows > kTileRows) return extras ? launch<true, true>(p, s) : launch<false, true>(p, s);
  return extras ? launch<true, false>(p, s) : launch<false, false>(p, s);
}

}  // namespace attend
}  // namespace nvfp4
