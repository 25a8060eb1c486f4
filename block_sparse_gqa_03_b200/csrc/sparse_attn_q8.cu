// Sparse attention over an 8-bit KV cache (e4m3 codes, a scale per (block, KV head)):
// with x_j = scale * s^K_beta(j) <q, k_j> over the selected blocks' visible tokens,
//   out = sum_j e^(x_j - m) s^V_beta(j) v_j / sum_j e^(x_j - m),  lse = m + log(...).
//
// The structure is that of sparse_attn.cu: a producer warp streams each selected
// block's K and V tiles by TMA (rows of d codes, swizzled by the row size) into a ring
// of stages, consumer warps hold a running softmax each, and the warps' states are
// merged through shared memory; few rows run on persistent CTAs that split the
// flattened (row, slot) list evenly, many rows on one CTA each.
//
// What is different.  Half the bytes arrive in half the time, so what the bf16 kernel
// hides behind its copies shows here:
//  * a warp takes a whole stage (64 tokens of one block and head): one maximum, one
//    rescaling of O and one barrier wait serve them all, and the 16-token score
//    chains are independent.  With four warps on one block, as for bf16, a decode step
//    at 128K took 79 us, with a stage per warp 54 us;
//  * a row that ends inside a CTA's range is merged and published by a warp of its own
//    while the consumers go on with the next row (they stopped for 3 to 6 us each time);
//  * the merge buffer's rows are padded by 16 bytes (unpadded, four lanes met on one
//    bank at every store).
// Bound: HBM, 2 d bytes per selected visible token and group.  16 x 128K tokens, 64
// heads in 8 groups of 128 dims, 128 of 2048 blocks each: 52.1 to 52.8 us against 41.4 us of
// HBM time (268 MB at the measured copy rate; the bf16 cache: 93 us); of the rest about
// 4 us pass before the first block arrives, the others in the merges behind the last one.
// A block's K scale joins the softmax scale of its scores and its V scale the fp32
// accumulation of its product, so that neither is rounded to 16 bits.
// A NaN among a row's visible scores makes its maximum, and with it its output and
// log-sum-exp, NaN (a maximum that left NaN out would make a row of NaN scores look empty).
#include <math.h>

#include <type_traits>

#include "attn_common.cuh"
#include "q8.cuh"

namespace msa {
namespace {

// Zeroes V rows [r0, r1) (codes that may be uninitialised memory: a NaN code must not
// meet a zero probability); the swizzle stays inside a row of D bytes.
template <int D>
__device__ __forceinline__ void zero_v_rows(uint8_t* vtile, int r0, int r1, int lane) {
  for (int x = lane; x < (r1 - r0) * (D / 16); x += 32)
    reinterpret_cast<uint4*>(vtile + r0 * D)[x] = make_uint4(0, 0, 0, 0);
}

// Four transposed codes (two tokens x two neighbouring dims, as ldmatrix.trans
// leaves them) regrouped by dim: low half the even dim's two tokens.
__device__ __forceinline__ uint32_t by_dim(uint32_t v) { return __byte_perm(v, 0, 0x3120); }

// WarpStateT over an 8-bit cache: groups of at most 8 heads, operands swapped.  A
// K register holds four consecutive dims of a token, so k-step c takes its 16 dims
// in the order 4j, 4j + 1, 4j + 2, 4j + 3 per lane quad j and the query fragments
// follow it; a transposed V register holds two dims of two tokens, so output row r
// of tile mt is dim 16mt + 2r and row r + 8 dim 16mt + 2r + 1.
template <int D, int NS_>
struct WarpStateTQ {
  static constexpr int kD = D, NS = NS_;
  static constexpr int kLd = D + 4;  // floats between O rows of the merge buffer
  uint32_t qlo[D / 16], qhi[D / 16];
  float o[D / 16][4];
  float m0, m1, l0, l1;
  float f0, f1;  // softmax scale (log2) with the query scaling undone, heads 2q4, 2q4 + 1

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = neg_inf();
    l0 = l1 = 0.f;
  }

  __device__ __forceinline__ void load_q(const AttnArgs& a, const RowGeo& rg, int lane) {
    const int r = lane >> 2, q4 = lane & 3;
    const float inv = q8::load_row_f16<D / 16>(a.q + rg.b * a.q_s0 + (int64_t)rg.t * a.q_s1 +
                                                   (int64_t)(rg.g * a.G + r) * a.q_s2 + 4 * q4,
                                               r < a.G, qlo, qhi) *
                      a.scale_log2;
    f0 = __shfl_sync(0xffffffffu, inv, 8 * q4);
    f1 = __shfl_sync(0xffffffffu, inv, 8 * q4 + 4);
  }

  // 16 NS tokens: rows `tok`.. of the tiles, absolute first token j0 < lim.
  __device__ __forceinline__ void attend(uint8_t* smem, uint32_t sbase, uint32_t kbase,
                                         uint32_t vbase, int tok, int j0, int lim, int lane,
                                         float ks, float vs, bool& wrote_smem) {
    const int r = lane >> 2;
    const float ninf = neg_inf();
    const bool cut = j0 + 16 * NS > lim;
    if (cut) {
      zero_v_rows<D>(smem + (vbase - sbase), tok + lim - j0, tok + 16 * NS, lane);
      wrote_smem = true;
      __syncwarp();
    }
    // tokens tok + 16u + lane % 16, chunks c (lanes 0-15) and c + 1
    const uint32_t row = tok + (lane & 15);
    // S^T of slice u: tokens 16u + r (s[0], s[1]) and 16u + r + 8 (s[2], s[3]), heads
    // 2q4, 2q4 + 1
    float s[NS][4];
#pragma unroll
    for (int u = 0; u < NS; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        uint32_t k0, k1, k2, k3;  // tokens 0-7, 8-15 of step c, then of step c + 1
        ldmatrix_x4(kbase + q8::swz<D>(row + 16 * u, c + (lane >> 4)), k0, k1, k2, k3);
        q8::mma_f16(s[u], q8::lo_f16x2(k0), q8::lo_f16x2(k1), q8::hi_f16x2(k0), q8::hi_f16x2(k1),
                    qlo[c], qhi[c]);
        q8::mma_f16(s[u], q8::lo_f16x2(k2), q8::lo_f16x2(k3), q8::hi_f16x2(k2), q8::hi_f16x2(k3),
                    qlo[c + 1], qhi[c + 1]);
      }
    }
    const float g0 = f0 * ks, g1 = f1 * ks;
    float mx0 = ninf, mx1 = ninf;
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      mul2(s[u][0], s[u][1], s[u][0], s[u][1], g0, g1);
      mul2(s[u][2], s[u][3], s[u][2], s[u][3], g0, g1);
      if (cut) {
        const int j = j0 + 16 * u + r;
        s[u][0] = j < lim ? s[u][0] : ninf;
        s[u][1] = j < lim ? s[u][1] : ninf;
        s[u][2] = j + 8 < lim ? s[u][2] : ninf;
        s[u][3] = j + 8 < lim ? s[u][3] : ninf;
      }
      mx0 = fmax3_nan(mx0, s[u][0], s[u][2]);
      mx1 = fmax3_nan(mx1, s[u][1], s[u][3]);
    }
    mx0 = warp_max_xor_nan(warp_max_xor_nan(warp_max_xor_nan(mx0, 4), 8), 16);
    mx1 = warp_max_xor_nan(warp_max_xor_nan(warp_max_xor_nan(mx1, 4), 8), 16);
    const float mn0 = fmax_nan(m0, mx0), mn1 = fmax_nan(m1, mx1);
    const float c0 = exp2_approx(m0 - mn0), c1 = exp2_approx(m1 - mn1);
    m0 = mn0;
    m1 = mn1;
    mul2(l0, l1, l0, l1, c0, c1);
    // probabilities in [0, 1] as f16 (relative error 2^-11, absolute 2^-25 below 2^-14)
    uint32_t pb[NS][2];
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      add2(s[u][0], s[u][1], s[u][0], s[u][1], -mn0, -mn1);
      add2(s[u][2], s[u][3], s[u][2], s[u][3], -mn0, -mn1);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[u][e] = exp2_approx(s[u][e]);
      add2(l0, l1, l0, l1, s[u][0], s[u][1]);
      add2(l0, l1, l0, l1, s[u][2], s[u][3]);
      pb[u][0] = movmatrix_trans(q8::pack_f16(s[u][0], s[u][1]));
      pb[u][1] = movmatrix_trans(q8::pack_f16(s[u][2], s[u][3]));
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; mt += 2) {
      float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        uint32_t v0, v1, v2, v3;  // tokens 0-7, 8-15 of dims 16mt.., then of the next 16
        ldmatrix_x4_trans(vbase + q8::swz<D>(row + 16 * u, mt + (lane >> 4)), v0, v1, v2, v3);
        v0 = by_dim(v0);
        v1 = by_dim(v1);
        v2 = by_dim(v2);
        v3 = by_dim(v3);
        q8::mma_f16(x, q8::lo_f16x2(v0), q8::hi_f16x2(v0), q8::lo_f16x2(v1), q8::hi_f16x2(v1),
                    pb[u][0], pb[u][1]);
        q8::mma_f16(y, q8::lo_f16x2(v2), q8::hi_f16x2(v2), q8::lo_f16x2(v3), q8::hi_f16x2(v3),
                    pb[u][0], pb[u][1]);
      }
      // o = o c + vs x
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float* p = &o[mt][e];
        mul2(p[0], p[1], p[0], p[1], c0, c1);
        fma2(p[0], p[1], x[e], x[e + 1], vs, vs, p[0], p[1]);
        p = &o[mt + 1][e];
        mul2(p[0], p[1], p[0], p[1], c0, c1);
        fma2(p[0], p[1], y[e], y[e + 1], vs, vs, p[0], p[1]);
      }
    }
  }

  __device__ __forceinline__ void stash(float* mo, float* mm, float* ml, int warp, int lane,
                                        int gr) {
    const int r = lane >> 2, h0 = 2 * (lane & 3), h1 = h0 + 1;
    float s0 = l0, s1 = l1;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, x);
      s1 += __shfl_xor_sync(0xffffffffu, s1, x);
    }
    float* mw = mo + warp * gr * kLd;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const int dd = mt * 16 + 2 * r;
      if (h0 < gr) *reinterpret_cast<float2*>(mw + h0 * kLd + dd) = make_float2(o[mt][0], o[mt][2]);
      if (h1 < gr) *reinterpret_cast<float2*>(mw + h1 * kLd + dd) = make_float2(o[mt][1], o[mt][3]);
    }
    if (r == 0) {
      mm[warp * 16 + h0] = m0;
      mm[warp * 16 + h1] = m1;
      ml[warp * 16 + h0] = s0;
      ml[warp * 16 + h1] = s1;
    }
  }
};

// WarpState over an 8-bit cache (up to 16 heads on the MMA rows).  Output tile
// columns: for dims 16c .. 16c + 15, o[2c] holds the even dims and o[2c + 1] the odd
// ones (column n is dim 16c + 2n (+ 1)).
template <int D, int NS_>
struct WarpStateQ {
  static constexpr int kD = D, NS = NS_;
  static constexpr int kLd = D + 4;  // floats between O rows of the merge buffer
  uint32_t qlo[2][D / 16], qhi[2][D / 16];  // head rows r and r + 8
  float o[D / 8][4];
  float m_a, m_b, l_a, l_b;
  float f_a, f_b;  // softmax scale (log2) with the query scaling undone

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m_a = m_b = neg_inf();
    l_a = l_b = 0.f;
  }

  __device__ __forceinline__ void load_q(const AttnArgs& a, const RowGeo& rg, int lane) {
    const int r = lane >> 2, q4 = lane & 3;
    const uint16_t* qb = a.q + rg.b * a.q_s0 + (int64_t)rg.t * a.q_s1 +
                         (int64_t)(rg.g * a.G) * a.q_s2 + 4 * q4;
    f_a = a.scale_log2 *
          q8::load_row_f16<D / 16>(qb + (int64_t)r * a.q_s2, r < a.G, qlo[0], qhi[0]);
    f_b = a.scale_log2 *
          q8::load_row_f16<D / 16>(qb + (int64_t)(r + 8) * a.q_s2, r + 8 < a.G, qlo[1], qhi[1]);
  }

  __device__ __forceinline__ void attend(uint8_t* smem, uint32_t sbase, uint32_t kbase,
                                         uint32_t vbase, int tok, int j0, int lim, int lane,
                                         float ks, float vs, bool& wrote_smem) {
    const int q4 = lane & 3;
    const float ninf = neg_inf();
    const bool cut = j0 + 16 * NS > lim;
    if (cut) {
      zero_v_rows<D>(smem + (vbase - sbase), tok + lim - j0, tok + 16 * NS, lane);
      wrote_smem = true;
      __syncwarp();
    }
    const uint32_t row = tok + (lane & 15);
    float sc[2 * NS][4];  // 8-token columns
#pragma unroll
    for (int nt = 0; nt < 2 * NS; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        uint32_t k0, k1, k2, k3;  // tokens 0-7, 8-15 of step c, then of step c + 1
        ldmatrix_x4(kbase + q8::swz<D>(row + 16 * u, c + (lane >> 4)), k0, k1, k2, k3);
        q8::mma_f16(sc[2 * u], qlo[0][c], qlo[1][c], qhi[0][c], qhi[1][c], q8::lo_f16x2(k0),
                    q8::hi_f16x2(k0));
        q8::mma_f16(sc[2 * u + 1], qlo[0][c], qlo[1][c], qhi[0][c], qhi[1][c], q8::lo_f16x2(k1),
                    q8::hi_f16x2(k1));
        q8::mma_f16(sc[2 * u], qlo[0][c + 1], qlo[1][c + 1], qhi[0][c + 1], qhi[1][c + 1],
                    q8::lo_f16x2(k2), q8::hi_f16x2(k2));
        q8::mma_f16(sc[2 * u + 1], qlo[0][c + 1], qlo[1][c + 1], qhi[0][c + 1], qhi[1][c + 1],
                    q8::lo_f16x2(k3), q8::hi_f16x2(k3));
      }
    }
    const float g_a = f_a * ks, g_b = f_b * ks;
    float mx_a = ninf, mx_b = ninf;
#pragma unroll
    for (int nt = 0; nt < 2 * NS; ++nt) {
      mul2(sc[nt][0], sc[nt][1], sc[nt][0], sc[nt][1], g_a, g_a);
      mul2(sc[nt][2], sc[nt][3], sc[nt][2], sc[nt][3], g_b, g_b);
      if (cut) {
        const int j = j0 + nt * 8 + 2 * q4;
        sc[nt][0] = j < lim ? sc[nt][0] : ninf;
        sc[nt][1] = j + 1 < lim ? sc[nt][1] : ninf;
        sc[nt][2] = j < lim ? sc[nt][2] : ninf;
        sc[nt][3] = j + 1 < lim ? sc[nt][3] : ninf;
      }
      mx_a = fmax3_nan(mx_a, sc[nt][0], sc[nt][1]);
      mx_b = fmax3_nan(mx_b, sc[nt][2], sc[nt][3]);
    }
    mx_a = warp_max_xor_nan(warp_max_xor_nan(mx_a, 1), 2);
    mx_b = warp_max_xor_nan(warp_max_xor_nan(mx_b, 1), 2);
    const float mn_a = fmax_nan(m_a, mx_a), mn_b = fmax_nan(m_b, mx_b);
    const float c_a = exp2_approx(m_a - mn_a), c_b = exp2_approx(m_b - mn_b);
    m_a = mn_a;
    m_b = mn_b;
    float ps_a = 0.f, ps_b = 0.f;
    uint32_t pa[NS][4];
#pragma unroll
    for (int nt = 0; nt < 2 * NS; ++nt) {
      const float p0 = exp2_approx(sc[nt][0] - mn_a), p1 = exp2_approx(sc[nt][1] - mn_a);
      const float p2 = exp2_approx(sc[nt][2] - mn_b), p3 = exp2_approx(sc[nt][3] - mn_b);
      ps_a += p0 + p1;
      ps_b += p2 + p3;
      pa[nt / 2][(nt & 1) * 2] = q8::pack_f16(p0, p1);
      pa[nt / 2][(nt & 1) * 2 + 1] = q8::pack_f16(p2, p3);
    }
    l_a = l_a * c_a + ps_a;
    l_b = l_b * c_b + ps_b;
    auto add = [&](float (&acc)[4], const float (&x)[4]) {
      mul2(acc[0], acc[1], acc[0], acc[1], c_a, c_a);
      fma2(acc[0], acc[1], x[0], x[1], vs, vs, acc[0], acc[1]);
      mul2(acc[2], acc[3], acc[2], acc[3], c_b, c_b);
      fma2(acc[2], acc[3], x[2], x[3], vs, vs, acc[2], acc[3]);
    };
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {
      float x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        uint32_t v0, v1, v2, v3;  // tokens 0-7, 8-15 of dims 16c.., then of the next 16
        ldmatrix_x4_trans(vbase + q8::swz<D>(row + 16 * u, c + (lane >> 4)), v0, v1, v2, v3);
        v0 = by_dim(v0);
        v1 = by_dim(v1);
        v2 = by_dim(v2);
        v3 = by_dim(v3);
        const uint32_t(&p)[4] = pa[u];
        q8::mma_f16(x[0], p[0], p[1], p[2], p[3], q8::lo_f16x2(v0), q8::lo_f16x2(v1));
        q8::mma_f16(x[1], p[0], p[1], p[2], p[3], q8::hi_f16x2(v0), q8::hi_f16x2(v1));
        q8::mma_f16(x[2], p[0], p[1], p[2], p[3], q8::lo_f16x2(v2), q8::lo_f16x2(v3));
        q8::mma_f16(x[3], p[0], p[1], p[2], p[3], q8::hi_f16x2(v2), q8::hi_f16x2(v3));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) add(o[2 * c + i], x[i]);
    }
  }

  __device__ __forceinline__ void stash(float* mo, float* mm, float* ml, int warp, int lane,
                                        int gr) {
    const int r = lane >> 2, q4 = lane & 3;
    float la = l_a, lb = l_b;
    la += __shfl_xor_sync(0xffffffffu, la, 1);
    la += __shfl_xor_sync(0xffffffffu, la, 2);
    lb += __shfl_xor_sync(0xffffffffu, lb, 1);
    lb += __shfl_xor_sync(0xffffffffu, lb, 2);
    float* mw = mo + warp * gr * kLd;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const int dd = c * 16 + 4 * q4;
      const float(&ev)[4] = o[2 * c];
      const float(&od)[4] = o[2 * c + 1];
      if (r < gr)
        *reinterpret_cast<float4*>(mw + r * kLd + dd) = make_float4(ev[0], od[0], ev[1], od[1]);
      if (r + 8 < gr)
        *reinterpret_cast<float4*>(mw + (r + 8) * kLd + dd) = make_float4(ev[2], od[2], ev[3], od[3]);
    }
    if (q4 == 0) {
      mm[warp * 16 + r] = m_a;
      mm[warp * 16 + r + 8] = m_b;
      ml[warp * 16 + r] = la;
      ml[warp * 16 + r + 8] = lb;
    }
  }
};

// Scales of list entry i (block id, plane and KV head resolved by compact_ids); a
// page outside the pool reads as zeros.
__device__ __forceinline__ void entry_scales(const AttnArgs& a, int beta, int plane, int g,
                                             float& ks, float& vs) {
  const int64_t at =
      (a.pg.table == nullptr ? (int64_t)plane * a.nblk + beta : (int64_t)plane) * a.h + g;
  ks = plane < 0 ? 1.f : __ldg(a.ks + at);
  vs = plane < 0 ? 1.f : __ldg(a.vs + at);
}

// A consumer warp's way through the items of an 8-bit cache (item = `unit` tokens of a
// list entry): items warp, warp + nw, ..., item i in stage i % stages, nw = min(NC,
// stages).  A stage's successive fills belong to different warps, so a warp first
// makes sure that the fill before its own has been consumed: the parity test of the
// full barrier could otherwise meet the fill before that one.  (The test of the empty
// barrier cannot be that far off: the warp's previous item was only issued after the
// fill two before this one had been consumed, since stages >= nw.)
template <int NC>
struct Q8Walk {
  int i, s, fill;  // item, stage, how often the stage was filled before
  int nw, n;       // stride, items
  int shift;       // log2 of the items per entry
  float ks, vs, ks_n, vs_n;

  __device__ __forceinline__ void start(const AttnArgs& a, int warp, int entries,
                                        const int32_t* list, const int32_t* plist,
                                        const int32_t* glist) {
    nw = min(NC, a.stages);
    shift = a.unit < a.block ? 1 : 0;
    n = warp < nw ? entries << shift : 0;
    i = s = warp;
    fill = 0;
    ks_n = vs_n = 1.f;
    fetch(a, i, list, plist, glist);
  }
  __device__ __forceinline__ void fetch(const AttnArgs& a, int item, const int32_t* list,
                                        const int32_t* plist, const int32_t* glist) {
    const int e = item >> shift;
    if (item < n) entry_scales(a, list[e] & 0xffff, plist[e], glist[e], ks_n, vs_n);
  }
  // Waits for item i (false: a wait ran out) and requests the next one's scales.
  __device__ __forceinline__ bool wait(const AttnArgs& a, uint32_t full0, uint32_t empty0,
                                       const int32_t* list, const int32_t* plist,
                                       const int32_t* glist) {
    ks = ks_n;
    vs = vs_n;
    fetch(a, i + nw, list, plist, glist);
    if (fill > 0 && !mbar_wait_warp(empty0 + 8 * s, (fill - 1) & 1, a.st, 4u, a.wait_ns))
      return false;
    return mbar_wait_warp(full0 + 8 * s, fill & 1, a.st, 3u, a.wait_ns);
  }
  // Attends to item i (list entry e) and releases its stage.
  template <class WS>
  __device__ __forceinline__ void attend(const AttnArgs& a, WS& ws, uint8_t* smem, uint32_t sbase,
                                         uint32_t empty0, int e, int lim, int lane) {
    const uint32_t kbase = sbase + (uint32_t)s * a.stage_bytes;
    const int j0 = (e & 0xffff) * a.block + (i & ((1 << shift) - 1)) * a.unit;
    bool wrote = false;
    for (int t = 0; t < a.unit && j0 + t < lim; t += 16 * WS::NS)
      ws.attend(smem, sbase, kbase, kbase + WS::kD * a.unit, t, j0 + t, lim, lane, ks, vs, wrote);
    if (wrote) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * s);
  }
  __device__ __forceinline__ void next(int stages) {
    i += nw;
    s += nw;
    if (s >= stages) {
      s -= stages;
      ++fill;
    }
  }
};

// Producer: streams the K and V tiles of list entries [0, n) into the stage ring, in
// items of `unit` tokens, one box for K and one for V.  Waits are bounded; before
// leaving, the producer waits for its copies still in flight.
template <int D>
__device__ __forceinline__ void produce_q8(const AttnArgs& a, const CUtensorMap* tmk,
                                           const CUtensorMap* tmv, const int32_t* list,
                                           const int32_t* plist, const int32_t* glist, int n,
                                           uint32_t sbase, uint32_t full0, uint32_t empty0) {
  int s = 0, fill = 0, issued = 0;
  bool ok = true;
  for (int i = 0; i < n && ok; ++i) {
    const int g = glist[i], p = plist[i];
    const bool paged = a.pg.table != nullptr;
    const int plane = paged && p < 0 ? (int)a.pg.pages : p;
    const int tok = paged ? 0 : (list[i] & 0xffff) * a.block;
    for (int t = 0; t < a.block; t += a.unit) {
      if (fill > 0 &&
          !mbar_wait_bounded(empty0 + 8 * s, (fill - 1) & 1, a.st, 1u, a.wait_ns)) {
        ok = false;
        break;
      }
      const uint32_t full = full0 + 8 * s;
      mbar_arrive_expect_tx(full, a.stage_bytes);
      const uint32_t kdst = sbase + (uint32_t)s * a.stage_bytes;
      tma_load_4d(kdst, tmk, full, 0, g, tok + t, plane);
      tma_load_4d(kdst + D * a.unit, tmv, full, 0, g, tok + t, plane);
      ++issued;
      if (++s == a.stages) {
        s = 0;
        ++fill;
      }
    }
  }
  for (int i = max(0, issued - a.stages); i < issued; ++i)
    mbar_wait_bounded(full0 + 8 * (i % a.stages), (i / a.stages) & 1, a.st, 2u, a.wait_ns);
}


// ----------------------------------------------------- merging a row's segment
__device__ __forceinline__ int atom_add_acq_rel(int* p, int v) {
  int r;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}

// Ends the segment of row `rg` (row number `cur`) that CTA `c` holds, from the stashed
// warp states: the output (row entirely in this CTA), or a partial, merged with the
// row's other partials by the last of its CTAs to publish.  Run by NT threads with
// `sync` as their barrier.  A row's first CTA reaches it at the end of its range and
// usually finds the other segments published: it then merges them straight into its own
// without writing it (no other CTA can then be the last, since the count never reaches
// nseg).  Segments are added in their order on either way.
//
// This code runs once or twice per CTA, so it is kept short: fetched cold, unrolled
// over items it took one warp 15 us.  The weights are computed once per head row.
template <int D, int NC, int LD, int NT, class Sync>
__device__ __forceinline__ void finish_row(const AttnArgs& a, int c, int cur, const RowGeo& rg,
                                        float* mo, float* mm, float* ml, int* flag, int tid,
                                        Sync sync) {
  // items per thread, and segments of each, whose loads are under way together.  K sets the
  // order of the roundings, so it is the same whoever merges: with 2 here and 4 there, a row
  // of four segments and more changed its last bits with the CTA that came last.
  constexpr int U = NT == 32 ? 4 : 2, K = 4;
  const int c_first = cur * a.topk / a.per;
  const int nseg = ((cur + 1) * a.topk - 1) / a.per - c_first + 1;
  const int seg = c - c_first;
  const float ninf = neg_inf();
  const int64_t pr_g = ((int64_t)rg.bt * a.H + rg.g * a.G) * a.smax;
  const int total = a.G * (D / 4);
  if (nseg > 1 && seg == 0 && tid == 0) *flag = ld_acquire_gpu(a.counters + cur);
  // per head row: the warps' weights (over their maxima), 1 / sum (over the sums of warp
  // 0), log-sum-exp (warp 1)
  if (tid < a.G) {
    float M = ninf;
#pragma unroll
    for (int w = 0; w < NC; ++w) M = fmax_nan(M, mm[w * 16 + tid]);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < NC; ++w) {
      const float f = M != ninf ? exp2f(mm[w * 16 + tid] - M) : 0.f;
      sum += f * ml[w * 16 + tid];
      mm[w * 16 + tid] = f;
    }
    ml[tid] = M != ninf ? 1.f / sum : 0.f;
    ml[16 + tid] = M != ninf ? (M + log2f(sum)) * kLn2 : ninf;
  }
  sync();
  const bool fast = nseg > 1 && seg == 0 && *flag == nseg - 1;
  // the warps' states merged: four dims of a head row
  auto stashed = [&](int row, int dim) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NC; ++w) {
      const float f = mm[w * 16 + row];
      const float4 o = *reinterpret_cast<const float4*>(mo + (w * a.G + row) * LD + dim);
      v.x += f * o.x;
      v.y += f * o.y;
      v.z += f * o.z;
      v.w += f * o.w;
    }
    const float inv = ml[row];
    return make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  };
  const int64_t orow = rg.b * a.o_s0 + (int64_t)rg.t * a.o_s1 + (int64_t)(rg.g * a.G) * a.o_s2;
  auto put = [&](int row, int dim, const float4& v, float l) {
    *reinterpret_cast<uint2*>(a.out + orow + row * a.o_s2 + dim) =
        make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    if (dim == 0 && a.lse) a.lse[(int64_t)rg.bt * a.H + rg.g * a.G + row] = l;
  };
  // The row's output from its segments, four dims per thread: segment 0 (this CTA's, from
  // the stash, when `own`; else its partial) and then the others in their order, K at a
  // time: a row of up to K + 1 segments takes one round trip to L2.
  auto merge_segments = [&](bool own) {
#pragma unroll 1
    for (int x0 = tid; x0 < total; x0 += U * NT) {
      float M[U], den[U];
      float4 acc[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int x = min(x0 + i * NT, total - 1), row = x / (D / 4), dim = (x % (D / 4)) * 4;
        const int64_t pr = pr_g + (int64_t)row * a.smax;
        acc[i] = own ? stashed(row, dim)
                     : __ldcg(reinterpret_cast<const float4*>(a.part_o + pr * D + dim));
        M[i] = own ? ml[16 + row] : __ldcg(a.part_lse + pr);
        den[i] = M[i] != ninf ? 1.f : 0.f;  // a segment without a key holds zeros
      }
#pragma unroll 1
      for (int sp = 1; sp < nseg; sp += K) {
        float l[U][K];
        float4 o[U][K];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int x = min(x0 + i * NT, total - 1), row = x / (D / 4), dim = (x % (D / 4)) * 4;
            const int64_t pr = pr_g + (int64_t)row * a.smax + min(sp + k, nseg - 1);
            l[i][k] = __ldcg(a.part_lse + pr);
            o[i][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + pr * D + dim));
            if (sp + k >= nseg) l[i][k] = ninf;
          }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float Mn = M[i];
#pragma unroll
          for (int k = 0; k < K; ++k) Mn = fmax_nan(Mn, l[i][k]);
          if (Mn == ninf) continue;
          const float c = exp2f((M[i] - Mn) * kLog2e);
          M[i] = Mn;
          den[i] *= c;
          acc[i].x *= c;
          acc[i].y *= c;
          acc[i].z *= c;
          acc[i].w *= c;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float w = exp2f((l[i][k] - Mn) * kLog2e);
            den[i] += w;
            acc[i].x += w * o[i][k].x;
            acc[i].y += w * o[i][k].y;
            acc[i].z += w * o[i][k].z;
            acc[i].w += w * o[i][k].w;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int x = x0 + i * NT;
        const float inv = M[i] != ninf ? 1.f / den[i] : 0.f;
        if (x < total)
          put(x / (D / 4), (x % (D / 4)) * 4,
              make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv),
              M[i] != ninf ? M[i] + log2f(den[i]) * kLn2 : ninf);
      }
    }
  };
  // (the row's counter goes back to zero, for the next call, with the merge)
  if (fast) {
    if (tid == 0) a.counters[cur] = 0;
    merge_segments(true);
    return;
  }
  // this CTA's segment: the output, or a partial
#pragma unroll 1
  for (int x = tid; x < total; x += NT) {
    const int row = x / (D / 4), dim = (x % (D / 4)) * 4;
    const float4 v = stashed(row, dim);
    if (nseg == 1) {
      put(row, dim, v, ml[16 + row]);
    } else {
      const int64_t pr = pr_g + (int64_t)row * a.smax + seg;
      *reinterpret_cast<float4*>(a.part_o + pr * D + dim) = v;
      if (dim == 0) a.part_lse[pr] = ml[16 + row];
    }
  }
  if (nseg == 1) return;
  // One thread publishes the partial (the other threads' stores ordered before its
  // atomic by the barrier) and learns whether it is the row's last; the atomic also
  // orders the other CTAs' partials before the loads above.
  sync();
  if (tid == 0) {
    const int f = atom_add_acq_rel(a.counters + cur, 1);
    *flag = f;
    if (f == nseg - 1) a.counters[cur] = 0;
  }
  sync();
  if (*flag == nseg - 1) merge_segments(false);
}

// ------------------------------------------------------- one CTA per row
// Rows of fewer than 1024 listed tokens take two consumer warps and up to five CTAs per
// SM (the many rows of a prompt with small blocks: what counts is how many of them are
// under way), longer ones four warps and two CTAs (decode of many sequences: deeper
// buffers).  1998 rows of 8 x 32 tokens 23.5 us with two warps, 39.4 us with four; 768
// rows of 64 x 64 tokens 128 us with four, 175 us with two.
constexpr int kShortRow = 1024;

template <int NC, class WS>
__global__ void __launch_bounds__((NC + 1) * 32, NC == 2 ? 5 : 2)
    sparse_attn_rows_q8_kernel(const __grid_constant__ CUtensorMap tmk,
                               const __grid_constant__ CUtensorMap tmv, AttnArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int D = WS::kD, LD = WS::kLd;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.region_bytes);
  int32_t* list = reinterpret_cast<int32_t*>(bars + 2 * a.stages);
  int32_t* n_list = list + a.list_cap;
  int32_t* plist = n_list + 1;          // [list_cap] sequence or page of each entry
  int32_t* glist = plist + a.list_cap;  // [list_cap] KV head of each entry
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + a.stages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rowg = blockIdx.x;

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    fence_mbar_init();
  }
  // the consumers load their queries while the list is built
  WS ws;
  const RowGeo rg = row_geo(a, rowg);
  if (warp == NC) {
    if (lane == 0) {
      prefetch_tensormap(&tmk);
      prefetch_tensormap(&tmv);
    }
    const bool skip = status_failed(a.st);
    const int n =
        compact_ids(a, rowg * a.topk, (rowg + 1) * a.topk, rowg, rowg, list, plist, glist, lane);
    if (lane == 0) *n_list = skip ? -1 : n;
  } else {
    ws.reset();
    ws.load_q(a, rg, lane);
  }
  __syncthreads();
  const int n = *n_list;
  if (n < 0) return;
  if (warp == NC) {
    if (lane == 0 && n > 0)
      produce_q8<D>(a, &tmk, &tmv, list, plist, glist, n, sbase, full0, empty0);
    return;
  }
  Q8Walk<NC> w;
  for (w.start(a, warp, n, list, plist, glist); w.i < w.n; w.next(a.stages)) {
    if (!w.wait(a, full0, empty0, list, plist, glist)) break;
    w.attend(a, ws, smem, sbase, empty0, list[w.i >> w.shift], rg.lim, lane);
  }
  // Merge the warps' states (the stages are free: every load was consumed).
  consumer_sync(NC * 32);
  float* mo = reinterpret_cast<float*>(smem);
  float* mm = mo + NC * a.G * LD;
  float* ml = mm + NC * 16;
  ws.stash(mo, mm, ml, warp, lane, a.G);
  consumer_sync(NC * 32);
  for (int x = tid; x < a.G * (D / 4); x += NC * 32) {
    const int row = x / (D / 4), dim = (x % (D / 4)) * 4;
    float4 val;
    float lsev;
    merge_warps4<D, NC, LD, true>(mo, mm, ml, a.G, row, dim, val, lsev);
    const int hq = rg.g * a.G + row;
    store_out4(a, rg, hq, dim, val);
    if (dim == 0 && a.lse) a.lse[(int64_t)rg.bt * a.H + hq] = lsev;
  }
}

// ----------------------------------------- persistent, balanced streaming
// Warps 0 .. NC - 1 consume, warp NC produces, warp NC + 1 finishes the rows that end
// before the CTA's last one.
//
// Barriers: 1 the consumers; 2 list published; 3 a row's states stashed (consumers
// arrive, the finishing warp waits); 4 the merge buffer is free again (it arrives, the
// consumers wait before their next stash there).
template <int NC, class WS>
__global__ void __launch_bounds__((NC + 2) * 32, 1)
    sparse_attn_stream_q8_kernel(const __grid_constant__ CUtensorMap tmk,
                                 const __grid_constant__ CUtensorMap tmv, AttnArgs a) {
  constexpr int D = WS::kD, LD = WS::kLd;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* mo = reinterpret_cast<float*>(smem + a.merge_off);  // [NC][G][LD]
  float* mm = mo + NC * a.G * LD;                             // [NC][16]
  float* ml = mm + NC * 16;                                   // [NC][16]
  int* flag = reinterpret_cast<int*>(ml + NC * 16);           // [2]: consumers, finishing warp
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.region_bytes);
  int32_t* list = reinterpret_cast<int32_t*>(bars + 2 * a.stages);
  int32_t* n_list = list + a.list_cap;
  int32_t* plist = n_list + 1;          // [list_cap] sequence or page of each entry
  int32_t* glist = plist + a.list_cap;  // [list_cap] KV head of each entry
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + a.stages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // rows and slots of a streamed shape fit 32 bits (fewer than 4 rows per SM)
  const int c = blockIdx.x;
  const int s0 = c * a.per;
  const int s1 = min(s0 + a.per, (int)a.total_slots);
  if (s0 >= s1) return;
  const int r0 = s0 / a.topk, r1 = (s1 - 1) / a.topk;
  if (warp == NC && lane == 0) {
    // needs nothing of the kernels before this one
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    fence_mbar_init();
  }
  grid_dep_wait();
  grid_dep_launch();

  if (warp == NC) {
    // Builds the list and starts streaming at once; the arrive on barrier 2 publishes
    // it and the stage barriers.  After an earlier timeout the kernel does nothing.
    const bool skip = status_failed(a.st);
    const int n = compact_ids(a, s0, s1, r0, r1, list, plist, glist, lane);
    if (lane == 0) *n_list = skip ? -1 : n;
    __syncwarp();
    named_arrive(2, (NC + 2) * 32);
    if (lane == 0 && !skip && n > 0)
      produce_q8<D>(a, &tmk, &tmv, list, plist, glist, n, sbase, full0, empty0);
    return;
  }
  if (warp == NC + 1) {
    named_sync(2, (NC + 2) * 32);
    if (*n_list < 0) return;
    for (int cur = r0; cur < r1; ++cur) {
      const RowGeo rg = row_geo(a, cur);
      named_sync(3, (NC + 1) * 32);
      finish_row<D, NC, LD, 32>(a, c, cur, rg, mo, mm, ml, flag + 1, lane, [] { __syncwarp(); });
      __syncwarp();
      if (cur + 1 < r1) named_arrive(4, (NC + 1) * 32);
    }
    return;
  }
  // the consumers load their first row's queries while the list is built
  WS ws;
  int cur = r0;
  RowGeo rg = row_geo(a, cur);
  ws.reset();
  ws.load_q(a, rg, lane);
  named_sync(2, (NC + 2) * 32);
  const int n = *n_list;
  if (n < 0) return;
  bool failed = false;
  // Hands the state of row `cur` over and moves to the next row.
  auto leave_row = [&]() {
    if (cur > r0) named_sync(4, (NC + 1) * 32);
    ws.stash(mo, mm, ml, warp, lane, a.G);
    named_arrive(3, (NC + 1) * 32);
    ++cur;
    ws.reset();
  };
  Q8Walk<NC> w;
  for (w.start(a, warp, n, list, plist, glist); w.i < w.n; w.next(a.stages)) {
    const int e = list[w.i >> w.shift];
    const int row = r0 + (e >> 16);
    if (cur < row) {
      while (cur < row) leave_row();
      rg = row_geo(a, cur);
      ws.load_q(a, rg, lane);
    }
    // After a wait runs out the warp computes no more but keeps walking the list, so
    // that every consumer warp still reaches the same row-boundary barriers.
    if (failed || !w.wait(a, full0, empty0, list, plist, glist)) {
      failed = true;
      continue;
    }
    w.attend(a, ws, smem, sbase, empty0, e, rg.lim, lane);
  }
  while (cur < r1) leave_row();
  // The last row: its states go where the stages were (every load has been consumed),
  // not to the merge buffer, which the finishing warp may still be reading.
  rg = row_geo(a, cur);
  float* so = reinterpret_cast<float*>(smem);
  float* sm = so + NC * a.G * LD;
  consumer_sync(NC * 32);
  ws.stash(so, sm, sm + NC * 16, warp, lane, a.G);
  consumer_sync(NC * 32);
  finish_row<D, NC, LD, NC * 32>(a, c, cur, rg, so, sm, sm + NC * 16, flag, tid,
                                 [] { consumer_sync(NC * 32); });
}

// ------------------------------------------------------------ host helpers
// Tokens per stage: 16 KB at most, so that there are more stages than consumer warps.
int stage_tokens(const Shape& s) { return s.block < 64 ? s.block : 64; }

// Consumer warps of the one-CTA-per-row kernel.
int rows_warps(const Shape& s) { return (int64_t)s.topk * s.block < kShortRow ? 2 : 4; }

constexpr int kStreamNC = 6;    // consumer warps of the streaming kernel
constexpr int kMaxList = 4096;  // entries a streaming CTA compacts up front

// Calls f with a warp state for the shape's head dim, group size and block: 64 tokens
// at a time, or the block when it is smaller; groups of more than 8 heads hold twice
// as many scores and outputs per thread and take 32.
template <class F>
cudaError_t with_state(const Shape& s, F f) {
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (s.G <= 8)
      return s.block >= 64   ? f(WarpStateTQ<D, 4>())
             : s.block == 32 ? f(WarpStateTQ<D, 2>())
                             : f(WarpStateTQ<D, 1>());
    return s.block >= 32 ? f(WarpStateQ<D, 2>()) : f(WarpStateQ<D, 1>());
  };
  return s.d == 128 ? pick(std::integral_constant<int, 128>())
                    : pick(std::integral_constant<int, 64>());
}

}  // namespace

// L2 fills are kept to 128 bytes, one row of a head: with the heads of a token side by
// side, a wider fill would bring rows that no selected block needs.
bool make_codes_map(CUtensorMap* map, const void* base, const Shape& s, const int64_t* str,
                    int dims, int tokens, bool swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const bool paged = s.pages.table != nullptr;
  cuuint64_t size[4] = {(cuuint64_t)s.d, (cuuint64_t)s.h,
                        (cuuint64_t)(paged ? s.block : s.max_kv),
                        (cuuint64_t)(paged ? s.pages.pages : s.batch)};
  cuuint64_t strides[3] = {(cuuint64_t)str[2], (cuuint64_t)str[1], (cuuint64_t)str[0]};
  cuuint32_t box[4] = {(cuuint32_t)dims, 1, (cuuint32_t)tokens, 1};
  cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = !swizzle      ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : dims == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                              : CU_TENSOR_MAP_SWIZZLE_64B;
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), size, strides, box,
             ones, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

AttnPlan plan_attn_q8(const Shape& s) {
  AttnPlan pl;
  pl.stage_bytes = 2u * s.d * stage_tokens(s);  // K and V tiles of one stage
  const int64_t rows_g = (int64_t)s.batch * s.n_q * s.h;
  pl.total = rows_g * s.topk;
  // merge buffer: O [warps][G][d + 4], max and sum [warps][16], two flag words
  auto merge_bytes = [&](int nc) { return (uint32_t)nc * (s.G * (s.d + 4) + 32) * 4 + 16; };
  const size_t cap = (size_t)max_smem_optin();
  pl.stream = rows_g < 4LL * num_sms();
  if (pl.stream) {
    pl.ctas = num_sms();
    // an even share, but a block for each consumer warp: in a small problem, finer shares
    // only add partials to merge
    pl.per = max((int)((pl.total + pl.ctas - 1) / pl.ctas), min(kStreamNC, s.topk));
    // A longer share also means fewer segments for a row's last CTA to merge, one after
    // the other: per * t + topk / per * 0.18 us is least at sqrt(topk * 0.18 / t), t the
    // time a block takes its SM (its bytes at 44 GB/s, 0.1 us at least).
    const double t = fmax(0.1, 2.0 * s.d * s.block / 44000.0);
    pl.per = max(pl.per, (int)ceil(sqrt(s.topk * 0.18 / t)));
    // Whole rows where that adds at most a block per warp (2 us): a split row's partials
    // are published and merged in 3 to 4 us.  (128 rows of 16 blocks: 14.7 us
    // with split rows, 12.1 us with whole ones.)
    const int whole = (pl.per + s.topk - 1) / s.topk * s.topk;
    if (whole - pl.per <= kStreamNC) pl.per = whole;
    pl.per = min(pl.per, kMaxList);
    pl.ctas = (int)((pl.total + pl.per - 1) / pl.per);
    pl.smax = (s.topk - 1) / pl.per + 2;
    pl.list_cap = pl.per;
    // as many stages as the shared memory holds: the bytes in flight per SM set the
    // streaming rate
    const size_t merge_r = (merge_bytes(kStreamNC) + 1023) & ~1023u;
    const size_t fixed = 1024 + merge_r + 4 * (3 * (size_t)pl.list_cap + 1);
    pl.stages = min(32, (int)((cap - fixed) / (pl.stage_bytes + 16)));
    pl.merge_off = pl.stages * pl.stage_bytes;
    pl.region_bytes = pl.merge_off + merge_r;
  } else {
    const int nc = rows_warps(s);
    pl.stages = nc == 2 ? max(2, min(4, (int)((40u * 1024u) / pl.stage_bytes)))
                        : min(8, (int)((100u * 1024u) / pl.stage_bytes));
    pl.region_bytes = max(pl.stages * pl.stage_bytes, merge_bytes(nc));
    pl.region_bytes = (pl.region_bytes + 15) & ~15u;
    pl.merge_off = 0;
    pl.ctas = (int)rows_g;
    pl.per = s.topk;
    pl.smax = 1;
    pl.list_cap = s.topk;
  }
  pl.smem_bytes = 1024 + pl.region_bytes + 16 * pl.stages + 4 * (3 * (size_t)pl.list_cap + 1);
  return pl;
}

cudaError_t run_attn_q8(const Shape& s, const AttnPlan& pl, const void* k, const void* v,
                        const AttnArgs& args, cudaStream_t stream) {
  CUtensorMap tmk, tmv;
  if (!make_codes_map(&tmk, k, s, s.k_s, s.d, stage_tokens(s), true) ||
      !make_codes_map(&tmv, v, s, s.v_s, s.d, stage_tokens(s), true))
    return cudaErrorInvalidValue;
  AttnArgs a = args;
  a.unit = stage_tokens(s);
  auto launch = [&](auto kernel, int threads) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)pl.smem_bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)pl.ctas), dim3(threads), pl.smem_bytes, stream, tmk,
                      tmv, a);
  };
  if (pl.stream)
    return with_state(s, [&](auto ws) {
      return launch(sparse_attn_stream_q8_kernel<kStreamNC, decltype(ws)>, (kStreamNC + 2) * 32);
    });
  if (rows_warps(s) == 2)
    return with_state(
        s, [&](auto ws) { return launch(sparse_attn_rows_q8_kernel<2, decltype(ws)>, 3 * 32); });
  return with_state(
      s, [&](auto ws) { return launch(sparse_attn_rows_q8_kernel<4, decltype(ws)>, 5 * 32); });
}

}  // namespace msa
