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
#include <type_traits>

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

// Pages that a warp takes at a time: two where the registers allow (the wait,
// the maximum's shuffles and votes are per step), and buffers per warp: at
// least what the parked results of 8 NT rows need.
constexpr int pages_of_step(int nt) { return nt <= 2 ? 2 : 1; }
constexpr int bufs_of(int nt) {
  return nt <= 2 ? 2 : (8 * nt * (kHeadDim + 2) * 4 + kPageBytes - 1) / kPageBytes;
}
// The query fragments of all n-tiles wait in shared memory when there are
// several (NT x 8 k-steps x 32 lanes x 8 bytes, twice with a low part).
constexpr int qfrag_bytes(int nt, bool smooth) { return nt == 1 ? 0 : nt * 2048 * (smooth ? 2 : 1); }
constexpr int warp_bytes(int nt) { return bufs_of(nt) * pages_of_step(nt) * kPageBytes; }
constexpr int smem_of(int nt, bool smooth) {
  return 1024 + qfrag_bytes(nt, smooth) + W * warp_bytes(nt);
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

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&x),
                            *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}

// This lane's part of query row q0 (128 channels; null: zeros) as B fragments
// of the 8 k-steps: hi[2 g + s] = channels (0, 4) + 2s and (1, 5) + 2s of the
// lane's eight channels 32 g + 8 qd .. of group g, the latter divided by 16,
// all times `sign` and the power of two that puts the row's largest magnitude
// into [2^13, 2^14).  With SMOOTH the channels are multiplied by the key weight
// and lo holds what f16 leaves of them (hi + lo is good to 2^-22).  Without it a
// bf16 query is exact in f16 down to 2^-30 of the row's maximum.  off: the B
// fragment of -8 sum(q) of the four groups, f16 high parts in rows 0-3 and low
// parts in rows 4-7 (good to 2^-22).  Returns the power of two that undoes the
// scaling.
template <bool SMOOTH>
__device__ __forceinline__ float query_frags(const __nv_bfloat16* q0, const float* w, float sign,
                                             int qd, uint32_t (&hi)[8][2],
                                             uint32_t (&lo)[SMOOTH ? 8 : 1][2], uint32_t& off) {
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
  const float f = sign * __int_as_float((127 + sh) << 23);
  float sum[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    sum[g] = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float fj = j ? f * 0.0625f : f;
        const float y0 = x[g][2 * s + j] * fj, y1 = x[g][2 * s + j + 4] * fj;
        const uint32_t h2 = pack_f16x2(y0, y1);
        const float2 h = halves(h2);
        float both = h.x + h.y;
        hi[2 * g + s][j] = h2;
        if constexpr (SMOOTH) {
          const uint32_t l2 = pack_f16x2(y0 - h.x, y1 - h.y);
          const float2 l = halves(l2);
          lo[2 * g + s][j] = l2;
          both += l.x + l.y;
        }
        sum[g] += j ? 16.f * both : both;
      }
    sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
    sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
    sum[g] *= -8.f / 16777216.f;
  }
  const float c0 = (qd & 1) ? sum[2] : sum[0], c1 = (qd & 1) ? sum[3] : sum[1];
  const uint32_t ch = pack_f16x2(c0, c1);
  const float2 cf = halves(ch);
  off = qd < 2 ? ch : pack_f16x2(c0 - cf.x, c1 - cf.y);
  return __int_as_float((127 - sh) << 23);
}

template <int NT, bool SMOOTH>
__global__ void __launch_bounds__(W * 32, NT == 1 ? 4 : (NT == 2 ? 3 : 2))
    decode_int4_kernel(const __grid_constant__ Launch a) {
  constexpr uint32_t FULL = 0xffffffffu;
  constexpr int NB = bufs_of(NT), NP = pages_of_step(NT);
  constexpr uint32_t NIB0 = 0x000F000Fu, NIB1 = 0x00F000F0u;
  pdl_trigger();                                    // the combine may be placed now
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  uint8_t* bufs = smem + 1024 + qfrag_bytes(NT, SMOOTH);
  static_assert(W * NB * 8 <= 1016, "barriers fit the header");
  static_assert(8 * NT * (kHeadDim + 2) * 4 <= warp_bytes(NT), "a warp's results fit its ring");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, qd = lane & 3;
  const int split = blockIdx.x, b = blockIdx.z;
  const int h = blockIdx.y / a.row_groups, rg = blockIdx.y % a.row_groups;
  const int Hq = a.num_q_heads, G = a.group;

  // The length, this warp's first 32 page ids and the rows' offsets go out
  // first.  Step j of the warp is pages p_begin + NP (warp + j W) + 0 .. NP - 1;
  // lane l of an id word holds page l % NP of step l / NP.
  const int32_t* bt_row = a.block_table + (size_t)b * a.max_pages;
  const int p_begin = split * a.pages_per_split;
  auto id_page = [&](int j) { return p_begin + NP * (warp + (j + lane / NP) * W) + lane % NP; };
  int L = a.seq_lens[b];
  const int bt_first = id_page(0) < a.max_pages ? __ldg(bt_row + id_page(0)) : 0;
  int q0 = b, qn = 1;
  if (a.cu_q) {
    q0 = a.cu_q[b];
    qn = a.cu_q[b + 1] - q0;
    if (qn < 0 || qn > a.max_q || L < qn || L > a.max_pages * kPageSize) {
      if (threadIdx.x == 0 && (qn != 0 || L < 0 || L > a.max_pages * kPageSize))
        atomicOr(&g_err_int4, kErrBadIndex);
      return;
    }
    if (qn == 0) return;                            // no token in this step
  } else if (L < 0 || L > a.max_pages * kPageSize) {
    if (threadIdx.x == 0) atomicOr(&g_err_int4, kErrBadIndex);
    L = 0;
  }
  // the rows of (b, h), their n-tiles shared evenly by as many CTAs as need be
  const int R = qn * G, tiles = (R + 7) >> 3;
  const int per = NT == 1 ? 1 : (tiles + (tiles + NT - 1) / NT - 1) / max(1, (tiles + NT - 1) / NT);
  const int row0 = rg * 8 * per;
  if (row0 >= R) return;
  const int nt_used = NT == 1 ? 1 : min(per, tiles - rg * per);
  const int npages = (L + kPageSize - 1) / kPageSize;
  if (split > 0 && p_begin >= npages) return;       // empty split: the merge skips it
  const int nv = max(1, (npages + a.pages_per_split - 1) / a.pages_per_split);
  const bool direct = a.splits == 1 || nv == 1;
  const int p_end = min(npages, p_begin + a.pages_per_split);
  const int L_end = min(L, p_end * kPageSize);      // a step may reach past the split
  const int n_w = max(0, (p_end - p_begin - NP * warp + NP * W - 1) / (NP * W));   // steps

  const uint32_t bar0 = smem_u32(bars + warp * NB);
  uint8_t* wbuf = bufs + (size_t)warp * warp_bytes(NT);
  const uint32_t wbuf_s = smem_u32(wbuf);
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NB; ++k) mbar_init(bar0 + 8 * k, 1);
    fence_mbar_init();
  }
  __syncwarp();

  const uint64_t policy = l2_policy_evict_first();
  int ids = 0;
  auto checked = [&](int id, int page) {            // 0 for what is not to be read
    if (page >= p_end) return 0;
    if (id < 0 || id >= a.num_pages) {
      atomicOr(&g_err_int4, kErrBadIndex);
      return 0;
    }
    return id;
  };
  const uint8_t* k_head = a.k + (size_t)h * kInt4Slab;
  const uint8_t* v_head = a.v + (size_t)h * kInt4Slab;
  const size_t page_stride = (size_t)a.num_kv_heads * kInt4Slab;
  auto issue = [&](int j) {
    constexpr int kSteps = 32 / NP;                 // steps of an id word
    if (j % kSteps == 0) {
      const int pg = id_page(j);
      ids = checked(j == 0 ? bt_first : (pg < p_end ? __ldg(bt_row + pg) : 0), pg);
    }
    int id[NP];
#pragma unroll
    for (int u = 0; u < NP; ++u) id[u] = __shfl_sync(FULL, ids, (j % kSteps) * NP + u);
    if (lane == 0) {
      const int k = j % NB;
      const uint32_t bar = bar0 + 8 * k, dst = wbuf_s + k * (NP * kPageBytes);
      const int n = min(NP, p_end - (p_begin + NP * (warp + j * W)));
      // the warp's reads of this buffer are done (__syncwarp); order them
      // before the async-proxy refill
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive_expect_tx(bar, n * kPageBytes);
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        if (u >= n) break;
        bulk_g2s_hint(dst + u * kPageBytes, k_head + id[u] * page_stride, kInt4Slab, bar, policy);
        bulk_g2s_hint(dst + u * kPageBytes + kInt4Slab, v_head + id[u] * page_stride, kInt4Slab,
                      bar, policy);
      }
    }
  };
  const int pro = min(NB, n_w);
  for (int j = 0; j < pro; ++j) issue(j);
  int issued = pro;

  // Query fragments (column r of n-tile nt = row row0 + 8 nt + r) and, for
  // this lane's accumulator columns 2 qd + e, the factor from raw scores to
  // the log2 domain (never negative: the scale's sign is in the query) and the
  // last position the row sees.
  uint32_t qh[NT == 1 ? 8 : 1][2], ql[NT == 1 && SMOOTH ? 8 : 1][2], off[NT];
  uint2* qs = reinterpret_cast<uint2*>(smem + 1024);      // [hi | lo][nt][k-step][lane]
  float sl2[NT][2];
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t hi[8][2], lo[SMOOTH ? 8 : 1][2];
    const int rq = row0 + 8 * nt + r;
    const __nv_bfloat16* q =
        rq < R ? a.q + ((size_t)(q0 + rq / G) * Hq + h * G + rq % G) * kHeadDim : nullptr;
    const float back =
        query_frags<SMOOTH>(q, a.k_smooth, a.softmax_scale < 0.f ? -1.f : 1.f, qd, hi, lo, off[nt]);
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
      sl2[nt][e] = fabsf(a.softmax_scale) * (kLog2e * 16777216.f) *
                   __shfl_sync(FULL, back, (2 * qd + e) * 4);
      lim[nt][e] = min(L_end - 1, rho < R ? L - qn + rho / G : L - 1);
    }
  }
  if constexpr (NT > 1) __syncthreads();
  int lim_min = L_end - 1;                          // steps up to it need no mask
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) lim_min = min(lim_min, min(lim[nt][0], lim[nt][1]));
  lim_min = __reduce_min_sync(FULL, lim_min);

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

  // O^T of n-tile nt, group g, half t: channels 32 g + 4 r + 2 t (o[..][0..1])
  // and + 1 (o[..][2..3], times 16) of columns 2 qd, 2 qd + 1, in units of
  // 2^-24 and with the codes' offset of 8; cs: 8 sum(P') of group r / 2.
  // mu: the maximum the exponentials are taken against; p carries 2^(kShift -
  // vexp), where every V scale so far is below 2^vexp.
  float o[NT][8][4], cs[NT][4];
  float mu[NT][2], l[NT][2];
  int vexp = 0;
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
  auto rescale = [&](int nt, float a0, float a1) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      o[nt][q][0] *= a0;
      o[nt][q][2] *= a0;
      o[nt][q][1] *= a1;
      o[nt][q][3] *= a1;
    }
    cs[nt][0] *= a0;
    cs[nt][1] *= a1;
    l[nt][0] *= a0;
    l[nt][1] *= a1;
  };

  // One step: the NP pages in the buffer at kb, whose first key is key0.
  // MASKED: it holds the causal edge or the end of the sequence or the split.
  auto step = [&](const uint8_t* kb, uint32_t kst, int key0, auto masked_tag) {
    constexpr bool MASKED = decltype(masked_tag)::value;
    // V scales of keys 2 qd, 2 qd + 1 (a) and + 8 (b): words (g0 g1, g2 g3) of
    // each; slots past the sequence may hold anything
    uint4 va[NP], vb[NP];
    uint32_t vm = 0;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const uint8_t* sc = kb + u * kPageBytes + kInt4Slab + kInt4Codes;
      va[u] = *reinterpret_cast<const uint4*>(sc + qd * 16);
      vb[u] = *reinterpret_cast<const uint4*>(sc + 64 + qd * 16);
      if constexpr (MASKED) {
        const int left = L_end - (key0 + u * kPageSize + 2 * qd);     // valid from this lane's first key on
        if (left <= 0) va[u].x = va[u].y = 0u;
        if (left <= 1) va[u].z = va[u].w = 0u;
        if (left <= 8) vb[u].x = vb[u].y = 0u;
        if (left <= 9) vb[u].z = vb[u].w = 0u;
      }
      vm = __vmaxu2(vm, __vmaxu2(__vmaxu2(va[u].x, va[u].y), __vmaxu2(va[u].z, va[u].w)));
      vm = __vmaxu2(vm, __vmaxu2(__vmaxu2(vb[u].x, vb[u].y), __vmaxu2(vb[u].z, vb[u].w)));
    }
    // a scale of 2^vexp or more (its fp16 exponent field E: scale < 2^(E - 14))
    const int ve = (int)(max(vm & 0xffffu, vm >> 16) >> 10) - 14;
    if (__any_sync(FULL, ve > vexp)) {
      const int now = __reduce_max_sync(FULL, ve);
      const float f = __int_as_float((127 + vexp - now) << 23);
      vexp = now;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) rescale(nt, f, f);
    }

    // raw scores s = sum_g scale (sum u q - 8 sum q) of keys r and r + 8
    float s[NP][NT][4];
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const uint8_t* kc = kb + u * kPageBytes;
      const uint32_t kcs = kst + u * kPageBytes;
      const uint2 ks0 = *reinterpret_cast<const uint2*>(kc + kInt4Codes + r * 8);
      const uint2 ks1 = *reinterpret_cast<const uint2*>(kc + kInt4Codes + r * 8 + 64);
      const uint32_t t0 = (qd & 1) ? ks0.y : ks0.x, t1 = (qd & 1) ? ks1.y : ks1.x;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.f;
        mma_f16(s[u][nt], t0, t1, 0u, 0u, off[nt], 0u);
      }
#pragma unroll
      for (int g2 = 0; g2 < 2; ++g2) {
        uint32_t kw[4];              // group 2 g2: keys r, r + 8; group 2 g2 + 1: the same
        ldsm_x4(kcs + g2 * 512 + lane * 16, kw);
        const float2 fa = halves(g2 ? ks0.y : ks0.x), fb = halves(g2 ? ks1.y : ks1.x);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int g = 2 * g2 + w;
          const uint32_t w0 = kw[2 * w], w1 = kw[2 * w + 1];
          const uint32_t x0 = w0 >> 8, x1 = w1 >> 8;
          const float f0 = w ? fa.y : fa.x, f1 = w ? fb.y : fb.x;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && nt >= nt_used) break;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            const uint2 qa = q_frag(nt, 2 * g, false), qb = q_frag(nt, 2 * g + 1, false);
            mma_f16(d, w0 & NIB0, w1 & NIB0, w0 & NIB1, w1 & NIB1, qa.x, qa.y);
            mma_f16(d, x0 & NIB0, x1 & NIB0, x0 & NIB1, x1 & NIB1, qb.x, qb.y);
            if constexpr (SMOOTH) {
              const uint2 la = q_frag(nt, 2 * g, true), lb = q_frag(nt, 2 * g + 1, true);
              mma_f16(d, w0 & NIB0, w1 & NIB0, w0 & NIB1, w1 & NIB1, la.x, la.y);
              mma_f16(d, x0 & NIB0, x1 & NIB0, x0 & NIB1, x1 & NIB1, lb.x, lb.y);
            }
            s[u][nt][0] = fmaf(f0, d[0], s[u][nt][0]);
            s[u][nt][1] = fmaf(f0, d[1], s[u][nt][1]);
            s[u][nt][2] = fmaf(f1, d[2], s[u][nt][2]);
            s[u][nt][3] = fmaf(f1, d[3], s[u][nt][3]);
          }
        }
      }
    }

    // softmax; P of a page as the B fragment's two words (keys 2 qd, 2 qd + 1
    // and + 8 of head r), in f16
    uint32_t pw[NP][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (NT > 1 && nt >= nt_used) break;
      auto sees = [&](int u, int j) {
        return key0 + u * kPageSize + r + (j < 2 ? 0 : 8) <= lim[nt][j & 1];
      };
      float pm[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int u = 0; u < NP; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (MASKED) {
            if (sees(u, j)) pm[j & 1] = fmaxf(pm[j & 1], s[u][nt][j]);
          } else {
            pm[j & 1] = fmaxf(pm[j & 1], s[u][nt][j]);
          }
        }
#pragma unroll
      for (int x = 4; x <= 16; x <<= 1) {
        pm[0] = fmaxf(pm[0], __shfl_xor_sync(FULL, pm[0], x));
        pm[1] = fmaxf(pm[1], __shfl_xor_sync(FULL, pm[1], x));
      }
      // the maximum moves only when a step passes it by more than 8
      pm[0] *= sl2[nt][0];
      pm[1] *= sl2[nt][1];
      const bool g0 = pm[0] > mu[nt][0] + 8.f, g1 = pm[1] > mu[nt][1] + 8.f;
      if (__any_sync(FULL, g0 || g1)) {
        const float a0 = g0 ? fast_exp2(mu[nt][0] - pm[0]) : 1.f;
        const float a1 = g1 ? fast_exp2(mu[nt][1] - pm[1]) : 1.f;
        if (g0) mu[nt][0] = pm[0];
        if (g1) mu[nt][1] = pm[1];
        rescale(nt, a0, a1);
      }
      const float sub0 = kShift - (float)vexp - mu[nt][0], sub1 = kShift - (float)vexp - mu[nt][1];
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[j] = fast_exp2(fmaf(s[u][nt][j], sl2[nt][j & 1], (j & 1) ? sub1 : sub0));
          if constexpr (MASKED) {
            if (!sees(u, j)) p[j] = 0.f;
          }
        }
        l[nt][0] += p[0] + p[2];
        l[nt][1] += p[1] + p[3];
        pw[u][nt][0] = movm_t(pack_f16x2(p[0], p[1]));
        pw[u][nt][1] = movm_t(pack_f16x2(p[2], p[3]));
      }
    }

    // O += V P', group by group
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const uint32_t vcs = kst + u * kPageBytes + kInt4Slab;
#pragma unroll
      for (int g2 = 0; g2 < 2; ++g2) {
        uint32_t vw[4];
        ldsm_x4_t(vcs + g2 * 512 + lane * 16, vw);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int g = 2 * g2 + w;
          const uint32_t w0 = vw[2 * w], w1 = vw[2 * w + 1];
          const uint32_t x0 = w0 >> 8, x1 = w1 >> 8;
          const uint32_t sel = w ? 0x7632u : 0x5410u;    // group g of two keys' words
          const uint32_t sa = __byte_perm(g2 ? va[u].y : va[u].x, g2 ? va[u].w : va[u].z, sel);
          const uint32_t sb = __byte_perm(g2 ? vb[u].y : vb[u].x, g2 ? vb[u].w : vb[u].z, sel);
          const uint32_t eight = (r >> 1) == g ? 0x00080008u : 0u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && nt >= nt_used) break;
            const uint32_t pb0 = mul_f16x2(pw[u][nt][0], sa), pb1 = mul_f16x2(pw[u][nt][1], sb);
            mma_f16(o[nt][2 * g], w0 & NIB0, w0 & NIB1, w1 & NIB0, w1 & NIB1, pb0, pb1);
            mma_f16(o[nt][2 * g + 1], x0 & NIB0, x0 & NIB1, x1 & NIB0, x1 & NIB1, pb0, pb1);
            mma_f16(cs[nt], eight, 0u, eight, 0u, pb0, pb1);
          }
        }
      }
    }
  };

  bool failed = false;
  int j_fail = 0;
  for (int j = 0; j < n_w; ++j) {
    const int k = j % NB;
    if (!__all_sync(FULL, mbar_wait(bar0 + 8 * k, (uint32_t)(j / NB) & 1u))) {
      failed = true;
      j_fail = j;
      break;
    }
    const int key0 = (p_begin + NP * (warp + j * W)) * kPageSize;
    const int at = k * (NP * kPageBytes);
    if (key0 + NP * kPageSize - 1 <= lim_min)
      step(wbuf + at, wbuf_s + at, key0, std::false_type{});
    else
      step(wbuf + at, wbuf_s + at, key0, std::true_type{});
    __syncwarp();
    if (issued < n_w) issue(issued++);
  }
  if (failed) {
    if (lane == 0) atomicOr(&g_err_int4, kErrTimeout);
    // let every copy this warp issued land (bounded) before the buffers are
    // reused or the CTA exits
    for (int j = j_fail; j < issued; ++j)
      (void)mbar_wait(bar0 + 8 * (j % NB), (uint32_t)(j / NB) & 1u);
  }
  __syncwarp();

  // Park (O unnormalised, m, l) of the warp's rows in its buffers (all of its
  // copies have landed): O [8 NT][128], m [8 NT], l [8 NT]; m is where p = 1.
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
        const bool none = failed || mu[nt][e] == kNoKey;
        wm[8 * nt + 2 * qd + e] = none ? kNoKey : mu[nt][e] + (float)vexp;
        wl[8 * nt + 2 * qd + e] = failed ? 0.f : l[nt][e];
      }
    }
  }
  __syncthreads();

  // Merge the warps (log-sum-exp rule); write the bf16 output (one split) or
  // the split's partial.
  constexpr size_t kStride = warp_bytes(NT);
  const int rows = min(8 * nt_used, R - row0);
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
    const bool last = old == (uint32_t)(nv * ((tiles + per - 1) / per)) - 1u;
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
