// decode_int4.cu -- split-KV attention over 4-bit pools: single-token decode
// and steps of 1..16 query tokens per sequence, causal inside the step
// (TileInfer.jl "Performance" page, "INT8 KV cache": dequantisation inside
// attention; "Attention for verify steps").  The combine kernels are those of
// the other pools.
//
// A 4-bit page of a head is 2 x 1,152 bytes, so HBM leaves an SM ~51 ns, some
// 100 cycles, per page (6.8 TB/s over 152 SMs): the kernel is bound by the
// instructions per page unless codes reach the tensor cores almost as they
// lie in memory.  They do, as f16 subnormals: a 16-bit half whose low four
// bits are u = code + 8 and whose other bits are 0 is exactly u 2^-24, and one
// with u in bits 4-7 is u 2^-20, so one AND per register turns two codes of a
// 32-bit word into two f16 MMA operands; nothing is converted and no exponent
// bias has to be taken off.  The products are exact in the tensor core's fp32.
// What is left of the encoding is put right outside the loop over the page:
//   2^-20 against 2^-24: the query channels that meet bits 4-7 are divided by
//     16 beforehand (QK), the output rows afterwards (PV);
//   the 8 in u = code + 8: QK starts its accumulators at -8 sum(q) of the
//     group; PV counts sum(P') in one extra MMA per group and takes 8 sum(P')
//     off at the end.
//
// One CTA per (split, KV head x row group, sequence), mma.sync m16n8k16, f16
// in, fp32 out.  A warp takes whole pages of its split, round-robin, from a
// private ring of shared-memory buffers filled by two bulk copies a page.
// Per page and 8 query rows (n-tile; row = token * G + head):
//   S^T = K Q^T: A = the page's 16 keys by ldmatrix, one group of 32 channels
//     per two MMAs, because the group's scale of a key multiplies its partial
//     score (fp32);
//   O^T += V^T P'^T: A = V^T by ldmatrix.trans, whose 16-bit elements are four
//     channels of one key, so that a register pairs the keys the MMA wants;
//     B = P' = p * scale of the group, rounded to f16 (half a step is 2^-12 of
//     the value, against 2^-9 for the bf16 P of the bf16 kernel) and moved to
//     the B layout by movmatrix.
// f16 reaches from 2^-24 to 65504, so p is taken against the running maximum
// of score + log2(the key's largest V scale, rounded up to a power of two):
// P' <= 2^15 for any V, and the sum of p stays in fp32.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace {

using namespace pkv;

__device__ uint32_t g_err_int4;

constexpr int W = 4;                                // warps per CTA
constexpr int kPageBytes = 2 * kInt4Slab;           // K slab, then V slab
constexpr float kNoKey = -1.0e30f;                  // running max before any visible key
constexpr float kShift = 7.f;                       // p carries 2^7: P' <= 2^(8 + 7)

// Page buffers per warp: at least what the parked results of 8 NT rows need.
constexpr int bufs_of(int nt) { return nt == 1 ? 4 : (8 * nt * (kHeadDim + 2) * 4 + kPageBytes - 1) / kPageBytes; }
// The query fragments of all n-tiles wait in shared memory when there are
// several (NT x 8 k-steps x 32 lanes x 8 bytes, twice with a low part).
constexpr int qfrag_bytes(int nt, bool smooth) { return nt == 1 ? 0 : nt * 2048 * (smooth ? 2 : 1); }
constexpr int smem_of(int nt, bool smooth) {
  return 1024 + qfrag_bytes(nt, smooth) + W * bufs_of(nt) * kPageBytes;
}

struct Launch {
  const uint8_t* k;
  const uint8_t* v;
  int num_pages, num_kv_heads;
  const __nv_bfloat16* q;
  const int32_t* cu_q;     // null: one row per sequence
  int num_q_heads, group;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seq_lens;
  int max_q;
  float softmax_scale;
  const float* k_smooth;
  int splits, pages_per_split, row_groups;
  uint32_t* ws_ctr;        // fused merge, as DecodeLaunch
  float* ws_o;
  float* ws_lse;
  __nv_bfloat16* out;
  float* lse;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B + (c0, c1) in both row halves.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                             float c1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %10, %11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float2 halves(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Upper bound of log2 of the largest of a key's four V scales (fp16, >= 0),
// from the exponent field E: scale < 2^(E - 14).
__device__ __forceinline__ float scale_exponent(uint2 s) {
  const uint32_t m = __vmaxu2(s.x, s.y);
  const uint32_t e = max(m & 0xffffu, m >> 16) >> 10;
  return __uint_as_float(0x4B000000u | e) - (8388608.f + 14.f);
}

// This lane's part of query row q0 (128 channels; null: zeros) as B fragments
// of the 8 k-steps: hi[2 g + s] = channels (0, 4) + 2s and (1, 5) + 2s of the
// lane's eight channels 32 g + 8 qd .. of group g, the latter divided by 16,
// all times the power of two that puts the row's largest magnitude into
// [2^13, 2^14).  With SMOOTH the channels are multiplied by the key weight and
// lo holds what f16 leaves of them (hi + lo is good to 2^-22).  Without it a
// bf16 query is exact in f16 down to 2^-30 of the row's maximum.  Returns the
// power of two that undoes the scaling.
template <bool SMOOTH>
__device__ __forceinline__ float query_frags(const __nv_bfloat16* q0, const float* w, int qd,
                                             uint32_t (&hi)[8][2], uint32_t (&lo)[SMOOTH ? 8 : 1][2]) {
  float x[4][8];
  float top = 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (q0) raw = __ldg(reinterpret_cast<const uint4*>(q0 + 32 * g + 8 * qd));
    const uint32_t r4[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[g][2 * e] = bf16lo(r4[e]);
      x[g][2 * e + 1] = bf16hi(r4[e]);
    }
    if constexpr (SMOOTH) {
      const float4* ws = reinterpret_cast<const float4*>(w + 32 * g + 8 * qd);
      const float4 w0 = __ldg(ws), w1 = __ldg(ws + 1);
      x[g][0] *= w0.x, x[g][1] *= w0.y, x[g][2] *= w0.z, x[g][3] *= w0.w;
      x[g][4] *= w1.x, x[g][5] *= w1.y, x[g][6] *= w1.z, x[g][7] *= w1.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[g][e]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 2^(13 - floor(log2 top)), within 2^+-100
  const int sh = max(-100, min(100, 13 + 127 - (__float_as_int(top) >> 23)));
  const float f = __int_as_float((127 + sh) << 23);
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float fj = j ? f * 0.0625f : f;
        const float y0 = x[g][2 * s + j] * fj, y1 = x[g][2 * s + j + 4] * fj;
        const uint32_t h2 = pack_f16x2(y0, y1);
        hi[2 * g + s][j] = h2;
        if constexpr (SMOOTH) {
          const float2 h = halves(h2);
          lo[2 * g + s][j] = pack_f16x2(y0 - h.x, y1 - h.y);
        }
      }
  return __int_as_float((127 - sh) << 23);
}

template <int NT, bool SMOOTH>
__global__ void __launch_bounds__(W * 32, NT == 1 ? 4 : (NT == 2 ? 3 : 2))
    decode_int4_kernel(const __grid_constant__ Launch a) {
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr int NB = bufs_of(NT);
  constexpr uint32_t NIB0 = 0x000F000Fu, NIB1 = 0x00F000F0u;
  pdl_trigger();                                    // the combine may be placed now
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  uint8_t* bufs = smem + 1024 + qfrag_bytes(NT, SMOOTH);
  static_assert(W * NB * 8 <= 1016, "barriers fit the header");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, qd = lane & 3;
  const int split = blockIdx.x, b = blockIdx.z;
  const int h = blockIdx.y / a.row_groups, rg = blockIdx.y % a.row_groups;
  const int Hq = a.num_q_heads, G = a.group;

  // the length, this warp's first 32 page ids and the rows' offsets go out first
  const int32_t* bt_row = a.block_table + (size_t)b * a.max_pages;
  const int p_begin = split * a.pages_per_split;
  int L = a.seq_lens[b];
  const int lp0 = p_begin + warp + lane * W;
  const int bt_first = lp0 < a.max_pages ? __ldg(bt_row + lp0) : 0;
  int q0 = b, qn = 1;
  if (a.cu_q) {
    q0 = a.cu_q[b];
    qn = a.cu_q[b + 1] - q0;
    if (qn < 0 || qn > a.max_q || L < qn || L > a.max_pages * kPageSize) {
      if (threadIdx.x == 0 && (qn != 0 || L < 0 || L > a.max_pages * kPageSize))
        atomicOr(&g_err_int4, kErrBadIndex);
      return;
    }
  } else if (L < 0 || L > a.max_pages * kPageSize) {
    if (threadIdx.x == 0) atomicOr(&g_err_int4, kErrBadIndex);
    L = 0;
  }
  const int R = qn * G, row0 = rg * 8 * NT;         // rows of (b, h); the CTA's first
  if (row0 >= R) return;
  const int npages = (L + kPageSize - 1) / kPageSize;
  if (split > 0 && p_begin >= npages) return;       // empty split: the merge skips it
  const int nv = max(1, (npages + a.pages_per_split - 1) / a.pages_per_split);
  const bool direct = a.splits == 1 || nv == 1;
  const int p_end = min(npages, p_begin + a.pages_per_split);
  const int n_w = max(0, (p_end - p_begin - warp + W - 1) / W);   // pages of this warp

  const uint32_t bar0 = smem_u32(bars + warp * NB);
  uint8_t* wbuf = bufs + (size_t)warp * NB * kPageBytes;
  const uint32_t wbuf_s = smem_u32(wbuf);
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NB; ++k) mbar_init(bar0 + 8 * k, 1);
    fence_mbar_init();
  }
  __syncwarp();

  const uint64_t policy = l2_policy_evict_first();
  int bt_cache = 0;
  auto page_id = [&](int i) -> int {                // ids of this warp's pages, 32 at a time
    if ((i & 31) == 0) {
      const int lp = p_begin + warp + (i + lane) * W;
      bt_cache = (i + lane < n_w) ? (i == 0 ? bt_first : __ldg(bt_row + lp)) : 0;
    }
    int pg = __shfl_sync(FULL, bt_cache, i & 31);
    if (pg < 0 || pg >= a.num_pages) {
      if (lane == 0) atomicOr(&g_err_int4, kErrBadIndex);
      pg = 0;
    }
    return pg;
  };
  auto issue = [&](int i, int pg) {
    if (lane == 0) {
      const int k = i % NB;
      const uint32_t bar = bar0 + 8 * k, dst = wbuf_s + k * kPageBytes;
      const size_t at = ((size_t)pg * a.num_kv_heads + h) * kInt4Slab;
      // the warp's reads of this buffer are done (__syncwarp); order them
      // before the async-proxy refill
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive_expect_tx(bar, kPageBytes);
      bulk_g2s_hint(dst, a.k + at, kInt4Slab, bar, policy);
      bulk_g2s_hint(dst + kInt4Slab, a.v + at, kInt4Slab, bar, policy);
    }
  };
  const int pro = min(NB, n_w);
  for (int i = 0; i < pro; ++i) issue(i, page_id(i));
  int issued = pro;

  // Query fragments (column r of n-tile nt = row row0 + 8 nt + r) and, for
  // this lane's accumulator columns 2 qd + e, the factor from raw scores to
  // the log2 domain and the last position the row sees.
  uint32_t qh[NT == 1 ? 8 : 1][2], ql[NT == 1 && SMOOTH ? 8 : 1][2];
  uint2* qs = reinterpret_cast<uint2*>(smem + 1024);      // [hi | lo][nt][k-step][lane]
  float sl2[NT][2];
  int lim[NT][2];
  auto row_ptr = [&](int n) -> const __nv_bfloat16* {     // null for padding rows
    const int rho = row0 + n;
    return rho < R ? a.q + ((size_t)(q0 + rho / G) * Hq + h * G + rho % G) * kHeadDim : nullptr;
  };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t hi[8][2], lo[SMOOTH ? 8 : 1][2];
    const float back = query_frags<SMOOTH>(row_ptr(8 * nt + r), a.k_smooth, qd, hi, lo);
    if constexpr (NT == 1) {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qh[ks][0] = hi[ks][0];
        qh[ks][1] = hi[ks][1];
        if constexpr (SMOOTH) {
          ql[ks][0] = lo[ks][0];
          ql[ks][1] = lo[ks][1];
        }
      }
    } else if (nt % W == warp) {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qs[(nt * 8 + ks) * 32 + lane] = make_uint2(hi[ks][0], hi[ks][1]);
        if constexpr (SMOOTH)
          qs[((NT + nt) * 8 + ks) * 32 + lane] = make_uint2(lo[ks][0], lo[ks][1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rho = row0 + 8 * nt + 2 * qd + e;
      // raw scores are in units of 2^-24
      sl2[nt][e] = a.softmax_scale * kLog2e * 16777216.f * __shfl_sync(FULL, back, (2 * qd + e) * 4);
      lim[nt][e] = rho < R ? L - qn + rho / G : L - 1;
    }
  }
  if constexpr (NT > 1) __syncthreads();
  int lim_min = L - 1;                              // pages up to it need no mask
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) lim_min = min(lim_min, min(lim[nt][0], lim[nt][1]));
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) lim_min = min(lim_min, __shfl_xor_sync(FULL, lim_min, x));

  auto q_frag = [&](int nt, int ks, bool low) -> uint2 {
    if constexpr (NT == 1) {
      if constexpr (SMOOTH)
        return low ? make_uint2(ql[ks][0], ql[ks][1]) : make_uint2(qh[ks][0], qh[ks][1]);
      else
        return make_uint2(qh[ks][0], qh[ks][1]);
    } else {
      return qs[(((low ? NT : 0) + nt) * 8 + ks) * 32 + lane];
    }
  };
  // -8 sum(q) of each group, by the MMA itself: A = -8 in every code
  float c0[NT][4], c1[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint2 f = q_frag(nt, 2 * g + s, false);
        mma_f16(d, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, f.x, f.y);
        if constexpr (SMOOTH) {
          const uint2 fl = q_frag(nt, 2 * g + s, true);
          mma_f16(d, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, fl.x, fl.y);
        }
      }
      c0[nt][g] = d[0];
      c1[nt][g] = d[1];
    }

  // O^T of n-tile nt, group g, half t: channels 32 g + 4 r + 2 t (o[..][0..1])
  // and + 1 (o[..][2..3], times 16) of columns 2 qd, 2 qd + 1, in units of
  // 2^-24 and with the codes' offset of 8; cs: 8 sum(P') of group r / 2
  float o[NT][8][4], cs[NT][4];
  float mu[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][t][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) cs[nt][j] = 0.f;
    mu[nt][0] = mu[nt][1] = kNoKey;
    l[nt][0] = l[nt][1] = 0.f;
  }

  bool failed = false;
  int i_fail = 0;
  for (int i = 0; i < n_w; ++i) {
    const int k = i % NB;
    if (!__all_sync(FULL, mbar_wait(bar0 + 8 * k, (uint32_t)(i / NB) & 1u))) {
      failed = true;
      i_fail = i;
      break;
    }
    const int key0 = (p_begin + warp + i * W) * kPageSize;
    const bool masked = key0 + kPageSize - 1 > lim_min;           // warp-uniform
    const uint32_t kst = wbuf_s + k * kPageBytes, vst = kst + kInt4Slab;
    const uint8_t* kb = wbuf + k * kPageBytes;

    // scales of keys r and r + 8
    const uint2 ks0 = *reinterpret_cast<const uint2*>(kb + kInt4Codes + r * 8);
    const uint2 ks1 = *reinterpret_cast<const uint2*>(kb + kInt4Codes + r * 8 + 64);
    uint2 vs0 = *reinterpret_cast<const uint2*>(kb + kInt4Slab + kInt4Codes + r * 8);
    uint2 vs1 = *reinterpret_cast<const uint2*>(kb + kInt4Slab + kInt4Codes + r * 8 + 64);
    if (masked) {                    // slots past the sequence may hold anything
      if (key0 + r >= L) vs0 = make_uint2(0u, 0u);
      if (key0 + r + 8 >= L) vs1 = make_uint2(0u, 0u);
    }

    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[nt][j] = 0.f;
#pragma unroll
    for (int g2 = 0; g2 < 2; ++g2) {
      uint32_t kw[4];                // group 2 g2: keys r, r + 8; group 2 g2 + 1: the same
      ldsm_x4(kst + g2 * 512 + lane * 16, kw);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int g = 2 * g2 + u;
        const uint32_t w0 = kw[2 * u], w1 = kw[2 * u + 1];
        const uint32_t x0 = w0 >> 8, x1 = w1 >> 8;
        const uint32_t sa = g < 2 ? ks0.x : ks0.y, sb = g < 2 ? ks1.x : ks1.y;
        const float f0 = (g & 1) ? halves(sa).y : halves(sa).x;
        const float f1 = (g & 1) ? halves(sb).y : halves(sb).x;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4];
          const uint2 fa = q_frag(nt, 2 * g, false), fb = q_frag(nt, 2 * g + 1, false);
          mma_f16_from(d, w0 & NIB0, w1 & NIB0, w0 & NIB1, w1 & NIB1, fa.x, fa.y, c0[nt][g],
                       c1[nt][g]);
          mma_f16(d, x0 & NIB0, x1 & NIB0, x0 & NIB1, x1 & NIB1, fb.x, fb.y);
          if constexpr (SMOOTH) {
            const uint2 la = q_frag(nt, 2 * g, true), lb = q_frag(nt, 2 * g + 1, true);
            mma_f16(d, w0 & NIB0, w1 & NIB0, w0 & NIB1, w1 & NIB1, la.x, la.y);
            mma_f16(d, x0 & NIB0, x1 & NIB0, x0 & NIB1, x1 & NIB1, lb.x, lb.y);
          }
          s[nt][0] = fmaf(f0, d[0], s[nt][0]);
          s[nt][1] = fmaf(f0, d[1], s[nt][1]);
          s[nt][2] = fmaf(f1, d[2], s[nt][2]);
          s[nt][3] = fmaf(f1, d[3], s[nt][3]);
        }
      }
    }

    // softmax: the running max (of score + the key's V exponent) moves only
    // when a page passes it by more than 8
    const float e0 = scale_exponent(vs0), e1 = scale_exponent(vs1);
    float p[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      bool on[4] = {true, true, true, true};
      float t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = fmaf(s[nt][j], sl2[nt][j & 1], j < 2 ? e0 : e1);
      if (masked) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          on[j] = key0 + r + (j < 2 ? 0 : 8) <= lim[nt][j & 1];
          if (!on[j]) t[j] = -INFINITY;
        }
      }
      float pm[2] = {fmaxf(t[0], t[2]), fmaxf(t[1], t[3])};
#pragma unroll
      for (int x = 4; x <= 16; x <<= 1) {
        pm[0] = fmaxf(pm[0], __shfl_xor_sync(FULL, pm[0], x));
        pm[1] = fmaxf(pm[1], __shfl_xor_sync(FULL, pm[1], x));
      }
      float alpha[2] = {1.f, 1.f};
      bool grow = false;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (pm[e] > mu[nt][e] + 8.f) {
          alpha[e] = fast_exp2(mu[nt][e] - pm[e]);
          mu[nt][e] = pm[e];
          l[nt][e] *= alpha[e];
          grow = true;
        }
      if (__any_sync(FULL, grow)) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          o[nt][q][0] *= alpha[0];
          o[nt][q][2] *= alpha[0];
          o[nt][q][1] *= alpha[1];
          o[nt][q][3] *= alpha[1];
        }
        cs[nt][0] *= alpha[0];
        cs[nt][1] *= alpha[1];
      }
      const float sub0 = kShift - mu[nt][0], sub1 = kShift - mu[nt][1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[nt][j] = fast_exp2(fmaf(s[nt][j], sl2[nt][j & 1], (j & 1) ? sub1 : sub0));
        if (masked && !on[j]) p[nt][j] = 0.f;
      }
      l[nt][0] += p[nt][0] + p[nt][2];
      l[nt][1] += p[nt][1] + p[nt][3];
    }

    // O += V P', group by group
#pragma unroll
    for (int g2 = 0; g2 < 2; ++g2) {
      uint32_t vw[4];
      ldsm_x4_t(vst + g2 * 512 + lane * 16, vw);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int g = 2 * g2 + u;
        const uint32_t w0 = vw[2 * u], w1 = vw[2 * u + 1];
        const uint32_t x0 = w0 >> 8, x1 = w1 >> 8;
        const uint32_t sa = g < 2 ? vs0.x : vs0.y, sb = g < 2 ? vs1.x : vs1.y;
        const float f0 = (g & 1) ? halves(sa).y : halves(sa).x;
        const float f1 = (g & 1) ? halves(sb).y : halves(sb).x;
        const uint32_t eight = (r >> 1) == g ? 0x00080008u : 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t pb0 = movm_t(pack_f16x2(p[nt][0] * f0, p[nt][1] * f0));
          const uint32_t pb1 = movm_t(pack_f16x2(p[nt][2] * f1, p[nt][3] * f1));
          mma_f16(o[nt][2 * g], w0 & NIB0, w0 & NIB1, w1 & NIB0, w1 & NIB1, pb0, pb1);
          mma_f16(o[nt][2 * g + 1], x0 & NIB0, x0 & NIB1, x1 & NIB0, x1 & NIB1, pb0, pb1);
          mma_f16(cs[nt], eight, 0u, eight, 0u, pb0, pb1);
        }
      }
    }
    __syncwarp();
    if (issued < n_w) {
      issue(issued, page_id(issued));
      ++issued;
    }
  }
  if (failed) {
    if (lane == 0) atomicOr(&g_err_int4, kErrTimeout);
    // let every copy this warp issued land (bounded) before the buffers are
    // reused or the CTA exits
    for (int i = i_fail; i < issued; ++i)
      (void)mbar_wait(bar0 + 8 * (i % NB), (uint32_t)(i / NB) & 1u);
  }
  __syncwarp();

  // Park (O unnormalised, m, l) of the warp's rows in its buffers (all of its
  // copies have landed): O [8 NT][128], m [8 NT], l [8 NT].
  float* wo = reinterpret_cast<float*>(wbuf);
  float* wm = wo + 8 * NT * kHeadDim;
  float* wl = wm + 8 * NT;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int x = 4; x <= 16; x <<= 1) {
      l[nt][0] += __shfl_xor_sync(FULL, l[nt][0], x);
      l[nt][1] += __shfl_xor_sync(FULL, l[nt][1], x);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float k0 = __shfl_sync(FULL, cs[nt][0], 8 * g + qd);
      const float k1 = __shfl_sync(FULL, cs[nt][1], 8 * g + qd);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* row = wo + (8 * nt + 2 * qd + e) * kHeadDim + 32 * g + 4 * r;
        const float kk = e ? k1 : k0;
        float4 v = make_float4((o[nt][2 * g][e] - kk) * 16777216.f,
                               (o[nt][2 * g][2 + e] * 0.0625f - kk) * 16777216.f,
                               (o[nt][2 * g + 1][e] - kk) * 16777216.f,
                               (o[nt][2 * g + 1][2 + e] * 0.0625f - kk) * 16777216.f);
        if (failed) v = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(row) = v;
      }
    }
    if (r == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        wm[8 * nt + 2 * qd + e] = failed ? kNoKey : mu[nt][e];
        wl[8 * nt + 2 * qd + e] = failed ? 0.f : l[nt][e];
      }
    }
  }
  __syncthreads();

  // Merge the warps (log-sum-exp rule); write the bf16 output (one split) or
  // the split's partial.
  constexpr size_t kStride = (size_t)NB * kPageBytes;
  const int rows = min(8 * NT, R - row0);
  for (int t = threadIdx.x; t < rows * kHeadDim; t += W * 32) {
    const int n = t / kHeadDim, d = t % kHeadDim;
    float M = kNoKey;
#pragma unroll
    for (int w = 0; w < W; ++w)
      M = fmaxf(M, reinterpret_cast<const float*>(bufs + w * kStride)[8 * NT * kHeadDim + n]);
    float Ls = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float* x = reinterpret_cast<const float*>(bufs + w * kStride);
      const float f = fast_exp2(x[8 * NT * kHeadDim + n] - M);
      Ls += f * x[8 * NT * (kHeadDim + 1) + n];
      O += f * x[n * kHeadDim + d];
    }
    const bool none = Ls == 0.f;                    // no key seen
    O = none ? 0.f : O / Ls;
    const float lse2 = none ? -INFINITY : M - kShift + fast_log2(Ls);
    const int rho = row0 + n;
    const size_t bh = (size_t)(q0 + rho / G) * Hq + h * G + rho % G;
    if (direct) {
      a.out[bh * kHeadDim + d] = __float2bfloat16_rn(O);
      if (a.lse && d == 0) a.lse[bh] = lse2 * kLn2;
    } else {
      const size_t slot = bh * a.splits + split;
      a.ws_o[slot * kHeadDim + d] = O;
      if (d == 0) a.ws_lse[slot] = lse2;
    }
  }
  if (direct || !a.ws_ctr) return;                  // separate combine kernel

  // Fused merge (decode): the part that completes the count of (b, KV head)
  // merges the nv splits of its rows and resets the count.
  volatile uint32_t& s_last = *reinterpret_cast<volatile uint32_t*>(smem + 1020);
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t* ctr = a.ws_ctr + (size_t)b * a.num_kv_heads + h;
    uint32_t old;
    asm volatile("fence.acq_rel.gpu;\n\tatom.relaxed.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(old) : "l"(ctr) : "memory");
    const bool last = old == (uint32_t)nv * ((R + 8 * NT - 1) / (8 * NT)) - 1u;
    if (last) {
      asm volatile("fence.acq_rel.gpu;" ::: "memory");
      *ctr = 0u;
    }
    s_last = last ? 1u : 0u;
  }
  __syncthreads();
  if (!s_last) return;
  float* wsm = reinterpret_cast<float*>(bufs);      // the buffers are free now
  float* red = wsm + 128;
  for (int rho = 0; rho < R; ++rho) {
    const size_t bh = (size_t)(q0 + rho / G) * Hq + h * G + rho % G;
    const float2 res = merge_splits(a.ws_lse + bh * a.splits, a.ws_o + bh * a.splits * kHeadDim,
                                    nv, wsm, red);
    const int d = threadIdx.x;
    if (d < kHeadDim) {
      a.out[bh * kHeadDim + d] = __float2bfloat16_rn(res.x);
      if (a.lse && d == 0) a.lse[bh] = res.y * kLn2;
    }
  }
}

template <int NT, bool SMOOTH>
cudaError_t launch_as(const Launch& a, int batch, cudaStream_t s) {
  const int smem = smem_of(NT, SMOOTH);
  cudaError_t e = pkv_host::set_max_dynamic_smem(
      reinterpret_cast<const void*>(decode_int4_kernel<NT, SMOOTH>), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.splits, a.num_kv_heads * a.row_groups, batch);
  decode_int4_kernel<NT, SMOOTH><<<grid, W * 32, smem, s>>>(a);
  return cudaGetLastError();
}

template <int NT>
cudaError_t launch_nt(const Launch& a, int batch, cudaStream_t s) {
  return a.k_smooth ? launch_as<NT, true>(a, batch, s) : launch_as<NT, false>(a, batch, s);
}

// The n-tiles of 8 rows that cover `rows` in as few CTAs as hold them.
cudaError_t launch_rows(Launch& a, int rows, int batch, cudaStream_t s) {
  const int tiles = (rows + 7) / 8;
  a.row_groups = (tiles + 3) / 4;
  switch ((tiles + a.row_groups - 1) / a.row_groups) {
    case 1: return launch_nt<1>(a, batch, s);
    case 2: return launch_nt<2>(a, batch, s);
    case 3: return launch_nt<3>(a, batch, s);
    default: return launch_nt<4>(a, batch, s);
  }
}

}  // namespace

namespace pkv_host {

cudaError_t launch_split_int4(const DecodeLaunch& d, cudaStream_t s) {
  Launch a{};
  a.k = static_cast<const uint8_t*>(d.k);
  a.v = static_cast<const uint8_t*>(d.v);
  a.num_pages = d.num_pages;
  a.num_kv_heads = d.num_kv_heads;
  a.q = static_cast<const __nv_bfloat16*>(d.q);
  a.num_q_heads = d.num_q_heads;
  a.group = d.num_q_heads / d.num_kv_heads;
  a.block_table = d.block_table;
  a.max_pages = d.max_pages;
  a.seq_lens = d.seq_lens;
  a.max_q = 1;
  a.softmax_scale = d.softmax_scale;
  a.k_smooth = d.k_smooth;
  a.splits = d.splits;
  a.pages_per_split = d.pages_per_split;
  a.ws_ctr = d.ws_ctr;
  a.ws_o = d.ws_o;
  a.ws_lse = d.ws_lse;
  a.out = static_cast<__nv_bfloat16*>(d.out);
  a.lse = d.lse;
  return launch_rows(a, a.group, d.batch, s);
}

cudaError_t launch_multi_int4(const MultiLaunch& m, cudaStream_t s) {
  Launch a{};
  a.k = static_cast<const uint8_t*>(m.k);
  a.v = static_cast<const uint8_t*>(m.v);
  a.num_pages = m.num_pages;
  a.num_kv_heads = m.num_kv_heads;
  a.q = static_cast<const __nv_bfloat16*>(m.q);
  a.cu_q = m.cu_q;
  a.num_q_heads = m.num_q_heads;
  a.group = m.num_q_heads / m.num_kv_heads;
  a.block_table = m.block_table;
  a.max_pages = m.max_pages;
  a.seq_lens = m.seq_lens;
  a.max_q = m.max_q;
  a.softmax_scale = m.softmax_scale;
  a.k_smooth = m.k_smooth;
  a.splits = m.splits;
  a.pages_per_split = m.pages_per_split;
  a.ws_o = m.ws_o;
  a.ws_lse = m.ws_lse;
  a.out = static_cast<__nv_bfloat16*>(m.out);
  a.lse = m.lse;
  return launch_rows(a, m.max_q * a.group, m.batch, s);
}

uint32_t take_int4_error(cudaStream_t s) { return take_error_word(&g_err_int4, s); }

}  // namespace pkv_host
