// Sparse branch: exact softmax attention over the selected KV blocks.
//
// "MiniMax goes sparse" (atlascloud.ai), section 1, step 2: with the block ids of
// step 1, the matching block subsets are taken from the raw K/V and ordinary
// softmax attention runs over them; all query heads of a GQA group share the
// group's top-k selection, so one load of a block serves the whole group
// ("MiniMax M3 的 MSA ...", second layer).
//
// A "row" is one (sequence, query, group); its G query heads are the 16 rows of
// a bf16 m16n8k16 tensor-core tile (rows >= G are zero), or, in the streaming
// kernel for G <= 8, the 8 columns of the tile with the operands swapped
// (WarpStateT).  Both kernels below share the same engine:
//  * one producer warp streams each selected block's K and V tiles into a ring of
//    shared-memory stages with TMA (4-D tensor maps over [batch, token, kv head,
//    dim], 128-byte swizzle), completion tracked by mbarriers whose waits are
//    bounded (a wait that runs out records an error; nothing hangs);
//  * consumer warps take 16-token slices of the blocks in turn: S = Q K^T and
//    O += P V on MMAs fed by ldmatrix from the swizzled tiles, with an fp32
//    online softmax in the exp2 domain; each warp keeps its own running max, sum
//    and output, and the warps' states are merged through shared memory.
//
// sparse_attn_rows_kernel: one CTA per row (prefill: many rows, each with a
// modest block list).  Writes bf16 output and the log-sum-exp directly.
//
// sparse_attn_stream_kernel: decode-style work, few rows with long block lists.
// A persistent grid of one CTA per SM splits the flattened (row, slot) list into
// equal contiguous ranges, so every SM streams the same number of blocks through
// one pipeline that never drains.  At each row boundary the consumers merge their
// states; a row covered by several CTAs gets one fp32 partial per CTA, and the
// last CTA to finish the row (a per-row counter, zero before the launch and put
// back to zero by the merging CTA) merges them by log-sum-exp weights.  The row's first CTA, which reaches the
// row at the end of its range, usually finds the others' partials already
// published and merges them into its own state without writing its own.
//
// 8-bit cache (e4m3 codes, a scale per (block, KV head)): the same two kernels with
// the Q8 warp states below.  A stage holds half the bytes (rows of d bytes, one TMA
// box per tile), codes are widened to f16 between ldmatrix and the MMA, a block's K
// scale joins the softmax scale of its scores and its V scale the fp32 accumulation
// of its product, so that neither is ever rounded to 16 bits.
#include <type_traits>

#include "kernels.h"
#include "q8.cuh"

namespace msa {
namespace {

struct AttnArgs {
  const uint16_t* q;
  int64_t q_s0, q_s1, q_s2;
  const int32_t* ids;
  const int32_t* seq_lens;
  int n_q, max_kv, H, h, G, topk, block, nblk, causal;
  float scale_log2;
  int stages;
  uint32_t stage_bytes, region_bytes, merge_off;
  int list_cap;
  // stream kernel only
  int64_t total_slots;
  int per, smax;
  float* part_o;
  float* part_lse;
  int* counters;
  uint16_t* out;
  int64_t o_s0, o_s1, o_s2;
  float* lse;
  DeviceStatus* st;
  uint64_t wait_ns;
  KvPages pg;  // table == nullptr: contiguous K/V
  // 8-bit cache: scales per (block, KV head); a stage holds `unit` tokens of a block,
  // which is all of it or (block 128) half
  const float *ks, *vs;
  int unit;
};

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t ld_b32(const uint16_t* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }

// Geometry of one row: sequence b, query t, group g, and the visible-token bound.
struct RowGeo {
  int b, t, g, bt, lim;
};

__device__ __forceinline__ RowGeo row_geo(const AttnArgs& a, int64_t rowg) {
  RowGeo r;
  r.g = (int)(rowg % a.h);
  r.bt = (int)(rowg / a.h);
  r.t = r.bt % a.n_q;
  r.b = r.bt / a.n_q;
  const int L = kv_length(a.seq_lens, r.b, a.max_kv, a.st);
  const int p = L - a.n_q + r.t;
  r.lim = a.causal ? min(L, p + 1) : L;  // visible tokens: j < lim
  return r;
}

// Running softmax state of one warp: rows r and r + 8 of the 16-row tile.
template <int D>
struct WarpState {
  static constexpr bool kQ8 = false;
  uint32_t qa[D / 16][4];
  float o[D / 8][4];
  float m_a, m_b, l_a, l_b;

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m_a = m_b = neg_inf();
    l_a = l_b = 0.f;
  }

  // A-operand fragments of the group's G query heads (rows >= G are zero).
  __device__ __forceinline__ void load_q(const AttnArgs& a, const RowGeo& rg, int lane) {
    const int r = lane >> 2, q4 = lane & 3;
    const bool vlo = r < a.G, vhi = r + 8 < a.G;
    const uint16_t* qb = a.q + rg.b * a.q_s0 + (int64_t)rg.t * a.q_s1 +
                         (int64_t)(rg.g * a.G) * a.q_s2 + 2 * q4;
    const uint16_t* qlo = qb + (int64_t)r * a.q_s2;
    const uint16_t* qhi = qb + (int64_t)(r + 8) * a.q_s2;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][0] = vlo ? ld_b32(qlo + 16 * kk) : 0u;
      qa[kk][1] = vhi ? ld_b32(qhi + 16 * kk) : 0u;
      qa[kk][2] = vlo ? ld_b32(qlo + 16 * kk + 8) : 0u;
      qa[kk][3] = vhi ? ld_b32(qhi + 16 * kk + 8) : 0u;
    }
  }

  // One 16-token slice (rows `tok`.. of the stage tiles, absolute first token j0).
  __device__ __forceinline__ void attend(const AttnArgs& a, uint8_t* smem, uint32_t sbase,
                                         uint32_t kbase, uint32_t vbase, uint32_t half_bytes,
                                         int tok, int j0, int lim, int lane, bool& wrote_smem) {
    constexpr int NH = D / 64;
    const int q4 = lane & 3;
    const float ninf = neg_inf();
    if (j0 + 16 > lim) {
      // Tokens j >= lim of this slice may be uninitialised memory: zero their V rows
      // so that a zero probability never meets a non-finite value.
      const int r0 = lim - j0;
      const int per_h = (16 - r0) * 8;
      uint8_t* vrow = smem + (vbase - sbase);
      for (int x = lane; x < per_h * NH; x += 32) {
        const int hh = x / per_h, rem = x % per_h;
        const int row = tok + r0 + rem / 8;
        *reinterpret_cast<uint4*>(vrow + hh * half_bytes + row * 128 + (rem % 8) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      wrote_smem = true;
      __syncwarp();
    }
    float sc[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
    {
      const int mi = lane >> 3, rr = lane & 7;
      const uint32_t row = tok + (mi >> 1) * 8 + rr;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t chunk = (kk & 3) * 2 + (mi & 1);
        uint32_t k0, k1, k2, k3;
        ldmatrix_x4(kbase + (kk >> 2) * half_bytes + swz128(row, chunk), k0, k1, k2, k3);
        mma_bf16_16816(sc[0], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], k0, k1);
        mma_bf16_16816(sc[1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], k2, k3);
      }
    }
    float mx_a = ninf, mx_b = ninf;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool ok = j0 + nt * 8 + 2 * q4 + e < lim;
        sc[nt][e] = ok ? sc[nt][e] * a.scale_log2 : ninf;
        sc[nt][2 + e] = ok ? sc[nt][2 + e] * a.scale_log2 : ninf;
        mx_a = fmaxf(mx_a, sc[nt][e]);
        mx_b = fmaxf(mx_b, sc[nt][2 + e]);
      }
    mx_a = warp_max_xor(warp_max_xor(mx_a, 1), 2);
    mx_b = warp_max_xor(warp_max_xor(mx_b, 1), 2);
    const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
    const float c_a = exp2f(m_a - mn_a), c_b = exp2f(m_b - mn_b);
    m_a = mn_a;
    m_b = mn_b;
    float ps_a = 0.f, ps_b = 0.f;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sc[nt][e] = exp2f(sc[nt][e] - mn_a);
        sc[nt][2 + e] = exp2f(sc[nt][2 + e] - mn_b);
        ps_a += sc[nt][e];
        ps_b += sc[nt][2 + e];
      }
    l_a = l_a * c_a + ps_a;
    l_b = l_b * c_b + ps_b;
#pragma unroll
    for (int i2 = 0; i2 < D / 8; ++i2) {
      o[i2][0] *= c_a;
      o[i2][1] *= c_a;
      o[i2][2] *= c_b;
      o[i2][3] *= c_b;
    }
    const uint32_t pa0 = pack_bf16(sc[0][0], sc[0][1]);
    const uint32_t pa1 = pack_bf16(sc[0][2], sc[0][3]);
    const uint32_t pa2 = pack_bf16(sc[1][0], sc[1][1]);
    const uint32_t pa3 = pack_bf16(sc[1][2], sc[1][3]);
    const int mi = lane >> 3, rr = lane & 7;
    const uint32_t row = tok + (mi & 1) * 8 + rr;
#pragma unroll
    for (int c2 = 0; c2 < D / 16; ++c2) {
      const uint32_t chunk = (c2 & 3) * 2 + (mi >> 1);
      uint32_t v0, v1, v2, v3;
      ldmatrix_x4_trans(vbase + (c2 >> 2) * half_bytes + swz128(row, chunk), v0, v1, v2, v3);
      mma_bf16_16816(o[2 * c2], pa0, pa1, pa2, pa3, v0, v1);
      mma_bf16_16816(o[2 * c2 + 1], pa0, pa1, pa2, pa3, v2, v3);
    }
  }

  // Stores this warp's state in the merge buffer: o [16][D], m [16], l [16].
  // Writes this warp's state for the merge: O rows [warp][gr][D] (only the gr
  // head rows in use), running max and sum [warp][16].
  __device__ __forceinline__ void stash(float* mo, float* mm, float* ml, int warp, int lane,
                                        int gr) {
    const int r = lane >> 2, q4 = lane & 3;
    float la = l_a, lb = l_b;
    la += __shfl_xor_sync(0xffffffffu, la, 1);
    la += __shfl_xor_sync(0xffffffffu, la, 2);
    lb += __shfl_xor_sync(0xffffffffu, lb, 1);
    lb += __shfl_xor_sync(0xffffffffu, lb, 2);
    float* mw = mo + warp * gr * D;
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt) {
      const int c = nt * 8 + 2 * q4;
      if (r < gr) *reinterpret_cast<float2*>(mw + r * D + c) = make_float2(o[nt][0], o[nt][1]);
      if (r + 8 < gr)
        *reinterpret_cast<float2*>(mw + (r + 8) * D + c) = make_float2(o[nt][2], o[nt][3]);
    }
    if (q4 == 0) {
      mm[warp * 16 + r] = m_a;
      mm[warp * 16 + r + 8] = m_b;
      ml[warp * 16 + r] = la;
      ml[warp * 16 + r + 8] = lb;
    }
  }
};

// The same state for groups of at most 8 heads with the MMA operands swapped:
// S^T = K Q^T puts a slice's 16 tokens on the MMA rows and the G heads on the
// n8 columns, and O^T = V^T P^T puts 16 output dims on the rows, so no MMA row
// is spent on padding (half as many MMAs and exponentials as the layout above
// at G = 8).  The K and V tiles feed the A operands through the same ldmatrix
// loads (K as stored, V transposed); P^T reaches the B layout of the second MMA
// through an in-register 8x8 transpose.  Each thread keeps heads 2 (lane % 4)
// and 2 (lane % 4) + 1: running max (shared by the 8 lanes of those heads) and
// its own part of the running sum.
template <int D>
struct WarpStateT {
  static constexpr bool kQ8 = false;
  uint32_t qb[D / 16][2];  // B fragments of Q^T: dims 16kk + 2 (lane % 4) (+8), head lane / 4
  float o[D / 16][4];      // O^T tile mt: dims 16mt + lane / 4 (+8), heads 2 (lane % 4) (+1)
  float m0, m1, l0, l1;

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = neg_inf();
    l0 = l1 = 0.f;
  }

  __device__ __forceinline__ void load_q(const AttnArgs& a, const RowGeo& rg, int lane) {
    const int r = lane >> 2, q4 = lane & 3;
    const bool valid = r < a.G;
    const uint16_t* qh = a.q + rg.b * a.q_s0 + (int64_t)rg.t * a.q_s1 +
                         (int64_t)(rg.g * a.G + r) * a.q_s2 + 2 * q4;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qb[kk][0] = valid ? ld_b32(qh + 16 * kk) : 0u;
      qb[kk][1] = valid ? ld_b32(qh + 16 * kk + 8) : 0u;
    }
  }

  __device__ __forceinline__ void attend(const AttnArgs& a, uint8_t* smem, uint32_t sbase,
                                         uint32_t kbase, uint32_t vbase, uint32_t half_bytes,
                                         int tok, int j0, int lim, int lane, bool& wrote_smem) {
    constexpr int NH = D / 64;
    const int r = lane >> 2;
    const float ninf = neg_inf();
    if (j0 + 16 > lim) {
      // Tokens j >= lim of this slice may be uninitialised memory: zero their V rows
      // so that a zero probability never meets a non-finite value.
      const int r0 = lim - j0;
      const int per_h = (16 - r0) * 8;
      uint8_t* vrow = smem + (vbase - sbase);
      for (int x = lane; x < per_h * NH; x += 32) {
        const int hh = x / per_h, rem = x % per_h;
        const int row = tok + r0 + rem / 8;
        *reinterpret_cast<uint4*>(vrow + hh * half_bytes + row * 128 + (rem % 8) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      wrote_smem = true;
      __syncwarp();
    }
    // S^T: tokens tok + r (s[0], s[1]) and tok + r + 8 (s[2], s[3]), heads 2q4, 2q4 + 1
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const int mi = lane >> 3, rr = lane & 7;
      const uint32_t row = tok + (mi >> 1) * 8 + rr;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t chunk = (kk & 3) * 2 + (mi & 1);
        uint32_t k0, k1, k2, k3;  // tokens 0-7 / 8-15 x dims low / high of the k-step
        ldmatrix_x4(kbase + (kk >> 2) * half_bytes + swz128(row, chunk), k0, k1, k2, k3);
        mma_bf16_16816(s, k0, k2, k1, k3, qb[kk][0], qb[kk][1]);
      }
    }
    const bool ok_lo = j0 + r < lim, ok_hi = j0 + r + 8 < lim;
    s[0] = ok_lo ? s[0] * a.scale_log2 : ninf;
    s[1] = ok_lo ? s[1] * a.scale_log2 : ninf;
    s[2] = ok_hi ? s[2] * a.scale_log2 : ninf;
    s[3] = ok_hi ? s[3] * a.scale_log2 : ninf;
    float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
    mx0 = warp_max_xor(warp_max_xor(warp_max_xor(mx0, 4), 8), 16);
    mx1 = warp_max_xor(warp_max_xor(warp_max_xor(mx1, 4), 8), 16);
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
    const float c0 = exp2f(m0 - mn0), c1 = exp2f(m1 - mn1);
    m0 = mn0;
    m1 = mn1;
    s[0] = exp2f(s[0] - mn0);
    s[1] = exp2f(s[1] - mn1);
    s[2] = exp2f(s[2] - mn0);
    s[3] = exp2f(s[3] - mn1);
    l0 = l0 * c0 + (s[0] + s[2]);
    l1 = l1 * c1 + (s[1] + s[3]);
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      o[mt][0] *= c0;
      o[mt][1] *= c1;
      o[mt][2] *= c0;
      o[mt][3] *= c1;
    }
    // P^T as the B operand: tokens 2q4 (+1) (+8), head r
    const uint32_t pb0 = movmatrix_trans(pack_bf16(s[0], s[1]));
    const uint32_t pb1 = movmatrix_trans(pack_bf16(s[2], s[3]));
    const int mi = lane >> 3, rr = lane & 7;
    const uint32_t row = tok + (mi & 1) * 8 + rr;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const uint32_t chunk = (mt & 3) * 2 + (mi >> 1);
      uint32_t v0, v1, v2, v3;  // dims low / high x tokens 0-7 / 8-15, transposed
      ldmatrix_x4_trans(vbase + (mt >> 2) * half_bytes + swz128(row, chunk), v0, v1, v2, v3);
      mma_bf16_16816(o[mt], v0, v2, v1, v3, pb0, pb1);
    }
  }

  // Same merge-buffer layout as WarpState::stash: O rows [warp][gr][D], running
  // max and sum [warp][16].
  __device__ __forceinline__ void stash(float* mo, float* mm, float* ml, int warp, int lane,
                                        int gr) {
    const int r = lane >> 2, h0 = 2 * (lane & 3), h1 = h0 + 1;
    float s0 = l0, s1 = l1;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, x);
      s1 += __shfl_xor_sync(0xffffffffu, s1, x);
    }
    float* mw = mo + warp * gr * D;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const int dd = mt * 16 + r;
      if (h0 < gr) {
        mw[h0 * D + dd] = o[mt][0];
        mw[h0 * D + dd + 8] = o[mt][2];
      }
      if (h1 < gr) {
        mw[h1 * D + dd] = o[mt][1];
        mw[h1 * D + dd + 8] = o[mt][3];
      }
    }
    if (r == 0) {
      mm[warp * 16 + h0] = m0;
      mm[warp * 16 + h1] = m1;
      ml[warp * 16 + h0] = s0;
      ml[warp * 16 + h1] = s1;
    }
  }
};

// ------------------------------------------------------------- 8-bit cache
// A warp takes whole list entries (a block of one head), NS 16-token slices at a time
// (64 tokens, fewer when the block is smaller): one running-maximum step, one
// rescaling of O and one barrier wait serve all of them, and the slices' score
// chains are independent.  With four warps on the slices of one entry, as for bf16,
// the per-entry bookkeeping and the rescaling of O came to about 775 instructions
// per slice, and the 128K decode attention took 79 us against 42 us of HBM time.

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
  static constexpr bool kQ8 = true;
  static constexpr int kD = D, NS = NS_;
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
      mx0 = fmax3(mx0, s[u][0], s[u][2]);
      mx1 = fmax3(mx1, s[u][1], s[u][3]);
    }
    mx0 = warp_max_xor(warp_max_xor(warp_max_xor(mx0, 4), 8), 16);
    mx1 = warp_max_xor(warp_max_xor(warp_max_xor(mx1, 4), 8), 16);
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
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
    float* mw = mo + warp * gr * D;
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const int dd = mt * 16 + 2 * r;
      if (h0 < gr) *reinterpret_cast<float2*>(mw + h0 * D + dd) = make_float2(o[mt][0], o[mt][2]);
      if (h1 < gr) *reinterpret_cast<float2*>(mw + h1 * D + dd) = make_float2(o[mt][1], o[mt][3]);
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
  static constexpr bool kQ8 = true;
  static constexpr int kD = D, NS = NS_;
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
      mx_a = fmax3(mx_a, sc[nt][0], sc[nt][1]);
      mx_b = fmax3(mx_b, sc[nt][2], sc[nt][3]);
    }
    mx_a = warp_max_xor(warp_max_xor(mx_a, 1), 2);
    mx_b = warp_max_xor(warp_max_xor(mx_b, 1), 2);
    const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
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
    float* mw = mo + warp * gr * D;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const int dd = c * 16 + 4 * q4;
      const float(&ev)[4] = o[2 * c];
      const float(&od)[4] = o[2 * c + 1];
      if (r < gr)
        *reinterpret_cast<float4*>(mw + r * D + dd) = make_float4(ev[0], od[0], ev[1], od[1]);
      if (r + 8 < gr)
        *reinterpret_cast<float4*>(mw + (r + 8) * D + dd) = make_float4(ev[2], od[2], ev[3], od[3]);
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

// Merge of NC warp states for tile row `row`, dims [dim, dim + 4) (dim a
// multiple of 4): normalised output and natural-log LSE (-inf and 0 when no key
// was seen).  The warps' weights are computed once for the four dims.
template <int D, int NC>
__device__ __forceinline__ void merge_warps4(const float* mo, const float* mm, const float* ml,
                                             int gr, int row, int dim, float4& val, float& lsev) {
  const float ninf = neg_inf();
  float M = ninf;
#pragma unroll
  for (int w = 0; w < NC; ++w) M = fmaxf(M, mm[w * 16 + row]);
  val = make_float4(0.f, 0.f, 0.f, 0.f);
  lsev = ninf;
  if (M == ninf) return;
  float wsum = 0.f;
  float4 acc = val;
#pragma unroll
  for (int w = 0; w < NC; ++w) {
    const float f = exp2f(mm[w * 16 + row] - M);
    wsum += f * ml[w * 16 + row];
    const float4 o = *reinterpret_cast<const float4*>(mo + (w * gr + row) * D + dim);
    acc.x += f * o.x;
    acc.y += f * o.y;
    acc.z += f * o.z;
    acc.w += f * o.w;
  }
  val = make_float4(acc.x / wsum, acc.y / wsum, acc.z / wsum, acc.w / wsum);
  lsev = (M + log2f(wsum)) * kLn2;
}

// Four consecutive bf16 outputs of head hq (one 8-byte store when aligned).
__device__ __forceinline__ void store_out4(const AttnArgs& a, const RowGeo& rg, int hq, int dim,
                                           const float4& v) {
  uint16_t* p = a.out + rg.b * a.o_s0 + (int64_t)rg.t * a.o_s1 + (int64_t)hq * a.o_s2 + dim;
  const uint32_t lo = pack_bf16(v.x, v.y), hi = pack_bf16(v.z, v.w);
  if ((reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
  } else {
    p[0] = (uint16_t)lo;
    p[1] = (uint16_t)(lo >> 16);
    p[2] = (uint16_t)hi;
    p[3] = (uint16_t)(hi >> 16);
  }
}

__device__ __forceinline__ void consumer_sync(int nthreads) {
  asm volatile("bar.sync 1, %0;" ::"r"(nthreads) : "memory");
}

// Producer: streams the K and V tiles of list entries [0, n) into the stage ring.
// Each entry is (block id in the low 16 bits, row offset in the high bits); the
// row supplies the sequence and the KV head.  Waits are bounded; before leaving,
// the producer waits for its copies still in flight.
template <int D>
__device__ __forceinline__ void produce(const AttnArgs& a, const CUtensorMap* tmk,
                                        const CUtensorMap* tmv, const int32_t* list,
                                        const int32_t* plist, const int32_t* glist, int n,
                                        uint32_t sbase, uint32_t full0, uint32_t empty0) {
  constexpr int NH = D / 64;
  const uint32_t half_bytes = (uint32_t)a.block * 128u;
  prefetch_tensormap(tmk);
  prefetch_tensormap(tmv);
  // (head, token, plane) of entry i: the head and the plane (sequence, or page of
  // a paged cache, -1 for a page outside the pool) were resolved when the list
  // was built
  auto coords = [&](int i, int& g, int& tok, int& plane) {
    const int e = list[i];
    g = glist[i];
    if (a.pg.table == nullptr) {
      tok = (e & 0xffff) * a.block;
      plane = plist[i];
    } else {
      tok = 0;
      plane = plist[i] < 0 ? (int)a.pg.pages : plist[i];
    }
  };
  int g_n = 0, tok_n = 0, plane_n = 0;
  if (n > 0) coords(0, g_n, tok_n, plane_n);
  int issued = 0;
  for (int i = 0; i < n; ++i) {
    const int g = g_n, tok = tok_n, plane = plane_n;
    if (i + 1 < n) coords(i + 1, g_n, tok_n, plane_n);
    const int s = i % a.stages;
    if (i >= a.stages &&
        !mbar_wait_bounded(empty0 + 8 * s, ((i / a.stages) - 1) & 1, a.st, 1u, a.wait_ns))
      break;
    const uint32_t full = full0 + 8 * s;
    mbar_arrive_expect_tx(full, a.stage_bytes);
    const uint32_t kdst = sbase + (uint32_t)s * a.stage_bytes;
    const uint32_t vdst = kdst + NH * half_bytes;
#pragma unroll
    for (int hh = 0; hh < NH; ++hh) {
      tma_load_4d(kdst + hh * half_bytes, tmk, full, hh * 64, g, tok, plane);
      tma_load_4d(vdst + hh * half_bytes, tmv, full, hh * 64, g, tok, plane);
    }
    ++issued;
  }
  for (int i = max(0, issued - a.stages); i < issued; ++i)
    mbar_wait_bounded(full0 + 8 * (i % a.stages), (i / a.stages) & 1, a.st, 2u, a.wait_ns);
}

// The same for an 8-bit cache: items of `unit` tokens, one box for K and one for V.
template <int D>
__device__ __forceinline__ void produce_q8(const AttnArgs& a, const CUtensorMap* tmk,
                                           const CUtensorMap* tmv, const int32_t* list,
                                           const int32_t* plist, const int32_t* glist, int n,
                                           uint32_t sbase, uint32_t full0, uint32_t empty0) {
  prefetch_tensormap(tmk);
  prefetch_tensormap(tmv);
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

// Compacts slots [s0, s1) of the flattened id array into the entry list: only
// blocks holding a visible token are kept.  For each kept block, glist gets its
// KV head and plist its sequence (with a paged cache: its page, looked up by the
// lanes in parallel), so that the producer's loop does no index arithmetic.  Run
// by one full warp; returns the count.
__device__ __forceinline__ int compact_ids(const AttnArgs& a, int64_t s0, int64_t s1,
                                           int64_t row0, int32_t* list, int32_t* plist,
                                           int32_t* glist, int lane) {
  constexpr int PF = 8;  // 32-slot groups whose ids are loaded together
  const unsigned lt = (1u << lane) - 1u;
  // Slot i belongs to row row0 + (i - first) / topk; the range is one CTA's
  // list (at most list_cap slots), so the offsets fit 32 bits.
  const int64_t first = row0 * a.topk;
  int ids[PF];
  auto load_ids = [&](int64_t base) {
#pragma unroll
    for (int k = 0; k < PF; ++k) {
      const int64_t i = base + k * 32 + lane;
      ids[k] = i < s1 ? __ldg(a.ids + i) : -1;
    }
  };
  load_ids(s0);  // issued before the row geometry: the two loads overlap
  const int64_t span = (s1 - 1) / a.topk - row0 + 1;
  const int nrows = span < 32 ? (int)span : 32;
  // visible-token limit, head and sequence of rows row0 .. row0 + 31, one per lane
  RowGeo geo_l;
  geo_l.lim = geo_l.g = geo_l.b = 0;
  if (lane < nrows) geo_l = row_geo(a, row0 + lane);
  int n = 0;
  for (int64_t base = s0; base < s1; base += 32 * PF) {
    if (base != s0) load_ids(base);
#pragma unroll
    for (int k = 0; k < PF; ++k) {
      if (base + k * 32 >= s1) break;
      const int64_t i = base + k * 32 + lane;
      const int beta = ids[k];
      const int rr = i < s1 ? (int)(i - first) / a.topk : 0;
      const int64_t rowg = row0 + rr;
      const int src = rr < 31 ? rr : 31;
      int lim = __shfl_sync(0xffffffffu, geo_l.lim, src);
      int g = __shfl_sync(0xffffffffu, geo_l.g, src);
      int b = __shfl_sync(0xffffffffu, geo_l.b, src);
      if (rr >= 32) {
        const RowGeo gr = row_geo(a, rowg);
        lim = gr.lim;
        g = gr.g;
        b = gr.b;
      }
      const bool bad = beta >= a.nblk;
      if (bad) record_error(a.st, kErrDeviceAssert, (uint32_t)rowg);
      const bool keep = beta >= 0 && !bad && (int64_t)beta * a.block < lim;
      const unsigned msk = __ballot_sync(0xffffffffu, keep);
      if (keep) {
        const int at = n + __popc(msk & lt);
        list[at] = beta | (rr << 16);
        glist[at] = g;
        plist[at] = a.pg.table != nullptr ? (int)kv_page(a.pg, b, beta, a.st) : b;
      }
      n += __popc(msk);
    }
  }
  return n;
}

// ------------------------------------------------------- one CTA per row
template <int D, class WS>
__global__ void __launch_bounds__(5 * 32, 1)
    sparse_attn_rows_kernel(const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv, AttnArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int NC = 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.region_bytes);
  int32_t* list = reinterpret_cast<int32_t*>(bars + 2 * a.stages);
  int32_t* n_list = list + a.list_cap;
  int32_t* plist = n_list + 1;       // [list_cap] sequence or page of each entry
  int32_t* glist = plist + a.list_cap;  // [list_cap] KV head of each entry
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + a.stages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rowg = blockIdx.x;
  const int nsub = a.block / 16;
  const uint32_t half_bytes = (uint32_t)a.block * 128u;

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, WS::kQ8 ? 1 : min(NC, nsub));
    }
    fence_mbar_init();
  }
  // the consumers load their queries while the list is built
  WS ws;
  const RowGeo rg = row_geo(a, rowg);
  if (warp == NC) {
    // after an earlier timeout the kernel does nothing (status read first: its
    // latency overlaps the compaction)
    const bool skip = status_failed(a.st);
    const int n = compact_ids(a, rowg * a.topk, (rowg + 1) * a.topk, rowg, list, plist, glist, lane);
    if (lane == 0) *n_list = skip ? -1 : n;
  } else {
    ws.reset();
    ws.load_q(a, rg, lane);
  }
  __syncthreads();
  const int n = *n_list;
  if (n < 0) return;
  if (warp == NC) {
    if (lane == 0 && n > 0) {
      if constexpr (WS::kQ8)
        produce_q8<D>(a, &tmk, &tmv, list, plist, glist, n, sbase, full0, empty0);
      else
        produce<D>(a, &tmk, &tmv, list, plist, glist, n, sbase, full0, empty0);
    }
    return;
  }
  if constexpr (WS::kQ8) {
    Q8Walk<NC> w;
    for (w.start(a, warp, n, list, plist, glist); w.i < w.n; w.next(a.stages)) {
      if (!w.wait(a, full0, empty0, list, plist, glist)) break;
      w.attend(a, ws, smem, sbase, empty0, list[w.i >> w.shift], rg.lim, lane);
    }
  } else {
    for (int i = 0; i < n; ++i) {
      const int u0 = i * nsub;
      const int st0 = (warp - (u0 % NC) + NC) % NC;  // first slice of block i owned by this warp
      if (st0 >= nsub) continue;
      const int s = i % a.stages;
      if (!mbar_wait_warp(full0 + 8 * s, (i / a.stages) & 1, a.st, 3u, a.wait_ns)) break;
      const uint32_t kbase = sbase + (uint32_t)s * a.stage_bytes;
      const uint32_t vbase = kbase + (D / 64) * half_bytes;
      const int beta = list[i] & 0xffff;
      bool wrote = false;
      for (int st = st0; st < nsub; st += NC) {
        const int j0 = beta * a.block + st * 16;
        if (j0 < rg.lim)
          ws.attend(a, smem, sbase, kbase, vbase, half_bytes, st * 16, j0, rg.lim, lane, wrote);
      }
      if (wrote) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * s);
    }
  }
  // Merge the warps' states (the stages are free: every load was consumed).
  consumer_sync(NC * 32);
  float* mo = reinterpret_cast<float*>(smem);
  float* mm = mo + NC * a.G * D;
  float* ml = mm + NC * 16;
  ws.stash(mo, mm, ml, warp, lane, a.G);
  consumer_sync(NC * 32);
  for (int x = tid; x < a.G * (D / 4); x += NC * 32) {
    const int row = x / (D / 4), dim = (x % (D / 4)) * 4;
    float4 val;
    float lsev;
    merge_warps4<D, NC>(mo, mm, ml, a.G, row, dim, val, lsev);
    const int hq = rg.g * a.G + row;
    store_out4(a, rg, hq, dim, val);
    if (dim == 0 && a.lse) a.lse[(int64_t)rg.bt * a.H + hq] = lsev;
  }
}

// ----------------------------------------- persistent, balanced streaming
template <int D, int NC, class WS>
__global__ void __launch_bounds__((NC + 1) * 32, 1)
    sparse_attn_stream_kernel(const __grid_constant__ CUtensorMap tmk,
                              const __grid_constant__ CUtensorMap tmv, AttnArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  float* mo = reinterpret_cast<float*>(smem + a.merge_off);  // [NC][G][D]
  float* mm = mo + NC * a.G * D;                              // [NC][16]
  float* ml = mm + NC * 16;                                   // [NC][16]
  int* flag = reinterpret_cast<int*>(ml + NC * 16);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.region_bytes);
  int32_t* list = reinterpret_cast<int32_t*>(bars + 2 * a.stages);
  int32_t* n_list = list + a.list_cap;
  int32_t* plist = n_list + 1;       // [list_cap] sequence or page of each entry
  int32_t* glist = plist + a.list_cap;  // [list_cap] KV head of each entry
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + a.stages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nsub = a.block / 16;
  const uint32_t half_bytes = (uint32_t)a.block * 128u;
  const int64_t c = blockIdx.x;
  const int64_t s0 = c * a.per;
  const int64_t s1 = min(s0 + a.per, a.total_slots);
  if (s0 >= s1) return;
  const int64_t r0 = s0 / a.topk, r1 = (s1 - 1) / a.topk;

  if (warp == NC) {
    // The producer warp sets up the stage barriers, builds the list and starts
    // streaming at once; the arrive on barrier 2 publishes both to the consumers.
    // After an earlier timeout the kernel does nothing; the status load is issued
    // first so that its latency overlaps the compaction.
    if (lane == 0) {
      for (int s = 0; s < a.stages; ++s) {
        mbar_init(full0 + 8 * s, 1);
        mbar_init(empty0 + 8 * s, WS::kQ8 ? 1 : min(NC, nsub));
      }
      fence_mbar_init();
    }
    const bool skip = status_failed(a.st);
    const int n = compact_ids(a, s0, s1, r0, list, plist, glist, lane);
    if (lane == 0) *n_list = skip ? -1 : n;
    __syncwarp();
    named_arrive(2, (NC + 1) * 32);
    if (lane == 0 && !skip && n > 0) {
      if constexpr (WS::kQ8)
        produce_q8<D>(a, &tmk, &tmv, list, plist, glist, n, sbase, full0, empty0);
      else
        produce<D>(a, &tmk, &tmv, list, plist, glist, n, sbase, full0, empty0);
    }
    return;
  }
  // the consumers load their first row's queries while the list is built
  WS ws;
  int64_t cur = r0;
  RowGeo rg = row_geo(a, cur);
  ws.reset();
  ws.load_q(a, rg, lane);
  named_sync(2, (NC + 1) * 32);
  const int n = *n_list;
  if (n < 0) return;
  bool failed = false;

  // Ends the segment of row `cur` held by this CTA: merge the warps, then write
  // the output (row entirely in this CTA) or a partial (and merge the row's
  // partials if this CTA is the last of the row to finish).
  //
  // A row's first CTA reaches it at the end of its range, while the row's other
  // CTAs start their ranges with it, so their partials are usually published
  // long before.  The first CTA reads the row's counter as it arrives: if every
  // other segment is in, it merges them straight into its own state (its own
  // partial is never written, and no atomic is taken; no other CTA can then be
  // the last, since the count never reaches nseg).  Otherwise it publishes like
  // the others.
  auto flush = [&]() {
    const int64_t c_first = (cur * a.topk) / a.per;
    const int64_t c_last = ((cur + 1) * a.topk - 1) / a.per;
    const int nseg = (int)(c_last - c_first + 1);
    const int seg = (int)(c - c_first);
    const bool first = nseg > 1 && seg == 0;
    if (first && tid == 0) {
      *flag = ld_acquire_gpu(a.counters + cur);
      __threadfence();
    }
    ws.stash(mo, mm, ml, warp, lane, a.G);
    consumer_sync(NC * 32);
    const bool fast = first && *flag == nseg - 1;
    for (int x = tid; x < a.G * (D / 4); x += NC * 32) {
      const int row = x / (D / 4), dim = (x % (D / 4)) * 4;
      const int hq = rg.g * a.G + row;
      const int64_t pr0 = ((int64_t)rg.bt * a.H + hq) * a.smax;
      // the second segment's partial, loaded before the warps' merge
      float l1 = neg_inf();
      float4 o1 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (fast) {
        l1 = __ldcg(a.part_lse + pr0 + 1);
        o1 = __ldcg(reinterpret_cast<const float4*>(a.part_o + (pr0 + 1) * D + dim));
      }
      float4 val;
      float lsev;
      merge_warps4<D, NC>(mo, mm, ml, a.G, row, dim, val, lsev);
      if (fast) {
        // the same operations in the same order as the last CTA's merge below,
        // so that the result does not depend on which of the two ran
        const float ninf = neg_inf();
        float M = fmaxf(fmaxf(ninf, lsev), l1);
        for (int sp = 2; sp < nseg; ++sp) M = fmaxf(M, __ldcg(a.part_lse + pr0 + sp));
        float4 res = make_float4(0.f, 0.f, 0.f, 0.f);
        float lres = ninf;
        if (M != ninf) {
          float den = 0.f;
          float4 acc = res;
          auto add = [&](float l, const float4& o) {
            const float w = exp2f((l - M) * kLog2e);
            den += w;
            acc.x += w * o.x;
            acc.y += w * o.y;
            acc.z += w * o.z;
            acc.w += w * o.w;
          };
          add(lsev, val);
          add(l1, o1);
          for (int sp = 2; sp < nseg; ++sp)
            add(__ldcg(a.part_lse + pr0 + sp),
                __ldcg(reinterpret_cast<const float4*>(a.part_o + (pr0 + sp) * D + dim)));
          res = make_float4(acc.x / den, acc.y / den, acc.z / den, acc.w / den);
          lres = M + log2f(den) * kLn2;
        }
        val = res;
        lsev = lres;
      }
      if (nseg == 1 || fast) {
        store_out4(a, rg, hq, dim, val);
        if (dim == 0 && a.lse) a.lse[(int64_t)rg.bt * a.H + hq] = lsev;
      } else {
        const int64_t pr = pr0 + seg;
        *reinterpret_cast<float4*>(a.part_o + pr * D + dim) = val;
        if (dim == 0) a.part_lse[pr] = lsev;
      }
    }
    if (nseg > 1 && !fast) {
      // One thread publishes the CTA's partial (its stores ordered before the
      // fence by the barrier) and learns whether it is the row's last; its
      // second fence orders the other CTAs' partials before the loads below.
      consumer_sync(NC * 32);
      if (tid == 0) {
        __threadfence();
        const int f = atomicAdd(&a.counters[cur], 1);
        __threadfence();
        *flag = f;
      }
      consumer_sync(NC * 32);
      if (*flag == nseg - 1 && nseg <= NC) {
        // Last CTA of the row: stage the row's partials in the (now free) merge
        // buffer with independent loads, then merge them from shared memory.
        float* so = mo;              // [G][nseg][D]
        float* sl = mo + NC * a.G * D;  // [G][nseg], over the free max/sum arrays
        const int64_t pr_g = ((int64_t)rg.bt * a.H + rg.g * a.G) * a.smax;
        const int q4n = nseg * (D / 4);
#pragma unroll 4
        for (int y = tid; y < a.G * q4n; y += NC * 32) {
          const int row = y / q4n, sp = (y % q4n) / (D / 4), c4 = y % (D / 4);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(
                                      a.part_o + (pr_g + (int64_t)row * a.smax + sp) * D) +
                                  c4);
          reinterpret_cast<float4*>(so)[(row * nseg + sp) * (D / 4) + c4] = v;
        }
        for (int y = tid; y < a.G * nseg; y += NC * 32)
          sl[y] = __ldcg(a.part_lse + pr_g + (int64_t)(y / nseg) * a.smax + y % nseg);
        consumer_sync(NC * 32);
        for (int x = tid; x < a.G * (D / 4); x += NC * 32) {
          const int row = x / (D / 4), dim = (x % (D / 4)) * 4;
          const int hq = rg.g * a.G + row;
          const float ninf = neg_inf();
          float M = ninf;
          for (int sp = 0; sp < nseg; ++sp) M = fmaxf(M, sl[row * nseg + sp]);
          float4 val = make_float4(0.f, 0.f, 0.f, 0.f);
          float lsev = ninf;
          if (M != ninf) {
            float den = 0.f;
            float4 acc = val;
            for (int sp = 0; sp < nseg; ++sp) {
              const float w = exp2f((sl[row * nseg + sp] - M) * kLog2e);
              den += w;
              const float4 o = *reinterpret_cast<const float4*>(so + (row * nseg + sp) * D + dim);
              acc.x += w * o.x;
              acc.y += w * o.y;
              acc.z += w * o.z;
              acc.w += w * o.w;
            }
            val = make_float4(acc.x / den, acc.y / den, acc.z / den, acc.w / den);
            lsev = M + log2f(den) * kLn2;
          }
          store_out4(a, rg, hq, dim, val);
          if (dim == 0 && a.lse) a.lse[(int64_t)rg.bt * a.H + hq] = lsev;
        }
      } else if (*flag == nseg - 1) {
        // more segments than the merge buffer holds: merge from global memory
        for (int x = tid; x < a.G * D; x += NC * 32) {
          const int row = x / D, dim = x % D;
          const int hq = rg.g * a.G + row;
          const int64_t pr0 = ((int64_t)rg.bt * a.H + hq) * a.smax;
          const float ninf = neg_inf();
          float M = ninf;
          for (int sp = 0; sp < nseg; ++sp) M = fmaxf(M, __ldcg(a.part_lse + pr0 + sp));
          float val = 0.f, lsev = ninf;
          if (M != ninf) {
            float den = 0.f, acc = 0.f;
            for (int sp = 0; sp < nseg; ++sp) {
              const float w = exp2f((__ldcg(a.part_lse + pr0 + sp) - M) * kLog2e);
              den += w;
              acc += w * __ldcg(a.part_o + (pr0 + sp) * D + dim);
            }
            val = acc / den;
            lsev = M + log2f(den) * kLn2;
          }
          a.out[rg.b * a.o_s0 + (int64_t)rg.t * a.o_s1 + (int64_t)hq * a.o_s2 + dim] =
              __bfloat16_as_ushort(__float2bfloat16_rn(val));
          if (dim == 0 && a.lse) a.lse[(int64_t)rg.bt * a.H + hq] = lsev;
        }
      }
    }
    // the row's merge is done: its counter goes back to zero for the next call
    if (nseg > 1 && tid == 0 && *flag == nseg - 1) a.counters[cur] = 0;
    consumer_sync(NC * 32);  // the merge buffer is free again
  };

  // Moves on to `row`: ends the rows before it.
  auto go_to = [&](int64_t row) {
    while (cur < row) {
      flush();
      ++cur;
      rg = row_geo(a, cur);
      ws.reset();
      ws.load_q(a, rg, lane);
    }
  };
  if constexpr (WS::kQ8) {
    Q8Walk<NC> w;
    for (w.start(a, warp, n, list, plist, glist); w.i < w.n; w.next(a.stages)) {
      const int e = list[w.i >> w.shift];
      go_to(r0 + (e >> 16));
      // after a wait runs out the warp computes no more but keeps walking (see below)
      if (failed || !w.wait(a, full0, empty0, list, plist, glist)) {
        failed = true;
        continue;
      }
      w.attend(a, ws, smem, sbase, empty0, e, rg.lim, lane);
    }
  } else {
    for (int i = 0; i < n; ++i) {
      const int e = list[i];
      go_to(r0 + (e >> 16));
      const int u0 = i * nsub;
      const int st0 = (warp - (u0 % NC) + NC) % NC;
      if (st0 >= nsub || failed) continue;
      const int s = i % a.stages;
      // After a wait runs out this warp stops computing but keeps walking the list,
      // so that every consumer warp still reaches the same row-boundary barriers.
      if (!mbar_wait_warp(full0 + 8 * s, (i / a.stages) & 1, a.st, 3u, a.wait_ns)) {
        failed = true;
        continue;
      }
      const uint32_t kbase = sbase + (uint32_t)s * a.stage_bytes;
      const uint32_t vbase = kbase + (D / 64) * half_bytes;
      const int beta = e & 0xffff;
      bool wrote = false;
      for (int st = st0; st < nsub; st += NC) {
        const int j0 = beta * a.block + st * 16;
        if (j0 < rg.lim)
          ws.attend(a, smem, sbase, kbase, vbase, half_bytes, st * 16, j0, rg.lim, lane, wrote);
      }
      if (wrote) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * s);
    }
  }
  while (true) {
    flush();
    if (cur >= r1) break;
    ++cur;
    rg = row_geo(a, cur);
    ws.reset();
  }
}

// ------------------------------------------------------------ host helpers
// Tokens per stage of an 8-bit cache: 16 KB at most, so that there are more stages
// than consumer warps.
int q8_unit(const Shape& s) { return s.block < 64 ? s.block : 64; }

// K or V as a 4-D tensor [batch][token][kv head][dim], or for a paged cache
// [page][token in page][kv head][dim]; one box is 64 dims x 1 head x `block`
// tokens (128 bytes per row, 128-byte swizzle).
bool make_kv_map(CUtensorMap* map, const void* base, const Shape& s, const int64_t* str) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const bool paged = s.pages.table != nullptr;
  if (s.kv8) {
    // e4m3 codes: one box is a whole row of d bytes x 1 head x a stage's tokens.  L2
    // fills are kept to the row's 128 bytes: with the heads of a token side by side,
    // a wider fill would bring rows that no selected block needs.
    cuuint64_t dims8[4] = {(cuuint64_t)s.d, (cuuint64_t)s.h,
                           (cuuint64_t)(paged ? s.block : s.max_kv),
                           (cuuint64_t)(paged ? s.pages.pages : s.batch)};
    cuuint64_t strides8[3] = {(cuuint64_t)str[2], (cuuint64_t)str[1], (cuuint64_t)str[0]};
    cuuint32_t box8[4] = {(cuuint32_t)s.d, 1, (cuuint32_t)q8_unit(s), 1};
    cuuint32_t ones[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims8, strides8,
               box8, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               s.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
  }
  cuuint64_t dims[4] = {(cuuint64_t)s.d, (cuuint64_t)s.h,
                        (cuuint64_t)(paged ? s.block : s.max_kv),
                        (cuuint64_t)(paged ? s.pages.pages : s.batch)};
  cuuint64_t strides[3] = {(cuuint64_t)str[2] * 2, (cuuint64_t)str[1] * 2,
                           (cuuint64_t)str[0] * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)s.block, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// Q as a 4-D tensor [batch][token][head][dim]; one box is 64 dims x the G heads
// of a group x 1 token, i.e. G rows of 128 bytes (128-byte swizzle).
bool make_q_group_map(CUtensorMap* map, const uint16_t* base, const Shape& s) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)s.d, (cuuint64_t)s.H, (cuuint64_t)s.n_q, (cuuint64_t)s.batch};
  cuuint64_t strides[3] = {(cuuint64_t)s.q_s[2] * 2, (cuuint64_t)s.q_s[1] * 2,
                           (cuuint64_t)s.q_s[0] * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)s.G, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

constexpr int kStreamNC = 8;       // consumer warps of the streaming kernel
constexpr int kMaxList = 4096;     // entries a streaming CTA compacts up front
constexpr uint32_t kSmemCap = 227u * 1024u;

struct AttnPlan {
  bool stream;
  int stages, ctas, per, smax, list_cap;
  int64_t total;
  uint32_t stage_bytes, region_bytes, merge_off;
  size_t smem_bytes;
};

// Stage count that keeps every block of a stage on the same warps (a warp waits
// only on the stages of blocks it processes): with fewer 16-token slices per
// block than consumer warps, a multiple of the warp cycle.
int stage_count(int want, int nsub, int nc) {
  const int cycle = nsub >= nc ? 1 : nc / nsub;
  want = max(2, min(8, want));
  return max(cycle, want - want % cycle);
}

AttnPlan plan_attn(const Shape& s) {
  AttnPlan pl;
  const bool kv8 = s.kv8;
  // K and V tiles: of one block, or one stage's share of it
  pl.stage_bytes = kv8 ? 2u * s.d * q8_unit(s) : 4u * s.d * s.block;
  const int nsub = s.block / 16;
  const int64_t rows_g = (int64_t)s.batch * s.n_q * s.h;
  pl.total = rows_g * s.topk;
  // merge buffer: O [warps][G][d], max and sum [warps][16], one flag word
  const uint32_t merge_bytes =
      (uint32_t)kStreamNC * s.G * s.d * 4 + (uint32_t)kStreamNC * 16 * 2 * 4 + 16;
  // Few rows with many blocks (decode): the persistent streaming kernel.
  pl.stream = rows_g < 4LL * num_sms();
  if (pl.stream) {
    pl.ctas = num_sms();
    pl.per = (int)((pl.total + pl.ctas - 1) / pl.ctas);
    if (pl.per > kMaxList) {
      pl.per = kMaxList;
      pl.ctas = (int)((pl.total + kMaxList - 1) / kMaxList);
    }
    pl.ctas = (int)((pl.total + pl.per - 1) / pl.per);
    pl.smax = (s.topk - 1) / pl.per + 2;
    pl.list_cap = pl.per;
    // as many stages as the shared memory holds: the bytes in flight per SM set
    // the streaming rate
    const size_t merge_r = (merge_bytes + 1023) & ~1023u;
    const size_t fixed = 1024 + merge_r + 4 * (3 * (size_t)pl.list_cap + 1);
    const size_t cap = (size_t)max_smem_optin();
    const int fit = cap > fixed ? (int)((cap - fixed) / (pl.stage_bytes + 16)) : 0;
    // bf16: fit >= 3 for every supported shape
    pl.stages = kv8 ? min(32, fit) : stage_count(fit, nsub, kStreamNC);
    pl.region_bytes = pl.stages * pl.stage_bytes + merge_r;
    pl.merge_off = pl.stages * pl.stage_bytes;
  } else {
    // Two CTAs per SM when the stages allow it, else one with deeper buffering.
    int want = (int)((100u * 1024u) / pl.stage_bytes);
    if (want < 2) want = min(4, (int)((200u * 1024u) / pl.stage_bytes));
    pl.stages = kv8 ? max(4, min(8, want)) : stage_count(want, nsub, 4);
    pl.region_bytes = max(pl.stages * pl.stage_bytes, merge_bytes);
    pl.merge_off = 0;
    pl.ctas = (int)rows_g;
    pl.per = s.topk;
    pl.smax = 1;
    pl.list_cap = s.topk;
  }
  pl.smem_bytes = 1024 + pl.region_bytes + 16 * pl.stages + 4 * (3 * (size_t)pl.list_cap + 1);
  return pl;
}

// Calls f with a warp state for the shape's head dim, group size and block: 64 tokens
// at a time, or the block when it is smaller; groups of more than 8 heads hold twice
// as many scores and outputs per thread and take 32.
template <class F>
cudaError_t with_q8_state(const Shape& s, F f) {
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (s.G <= 8)
      return s.block >= 64 ? f(WarpStateTQ<D, 4>()) : s.block == 32 ? f(WarpStateTQ<D, 2>())
                                                                    : f(WarpStateTQ<D, 1>());
    return s.block >= 32 ? f(WarpStateQ<D, 2>()) : f(WarpStateQ<D, 1>());
  };
  return s.d == 128 ? pick(std::integral_constant<int, 128>()) : pick(std::integral_constant<int, 64>());
}

}  // namespace

bool make_rows_map(CUtensorMap* map, uint16_t* base, int64_t rows, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, 32};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t attn_partial_bytes(const Shape& s) {
  const AttnPlan pl = plan_attn(s);
  if (!pl.stream) return !s.kv8 && kv_attn_supported(s) ? kv_workspace_bytes(s) : 0;
  const size_t n = (size_t)s.batch * s.n_q * s.H * pl.smax;
  const size_t rows_g = (size_t)s.batch * s.n_q * s.h;
  return n * (size_t)(s.d + 1) * sizeof(float) + rows_g * sizeof(int) + 512;
}

int attn_launches(const Shape& s) {
  const AttnPlan pl = plan_attn(s);
  return !pl.stream && !s.kv8 && kv_attn_supported(s) ? kv_launches(s) : 1;
}

int* attn_merge_counters(const Shape& s, void* partials, int* count) {
  const AttnPlan pl = plan_attn(s);
  *count = 0;
  if (!pl.stream || partials == nullptr) return nullptr;
  const size_t nrow_h = (size_t)s.batch * s.n_q * s.H;
  const float* part_lse = reinterpret_cast<float*>(partials) + nrow_h * pl.smax * s.d;
  *count = s.batch * s.n_q * s.h;
  return reinterpret_cast<int*>(
      (reinterpret_cast<uintptr_t>(part_lse + nrow_h * pl.smax) + 255) & ~uintptr_t(255));
}

cudaError_t launch_sparse_attn(const Shape& s, const uint16_t* q, const void* k,
                               const void* v, const int32_t* ids, uint16_t* out, float* lse,
                               void* partials, size_t partial_bytes, DeviceStatus* st,
                               cudaStream_t stream, bool counters_zeroed, int* fixed_counters) {
  const AttnPlan pl = plan_attn(s);
  if (pl.smem_bytes > kSmemCap) return cudaErrorInvalidValue;
  CUtensorMap tmk, tmv;
  if (!make_kv_map(&tmk, k, s, s.k_s) || !make_kv_map(&tmv, v, s, s.v_s))
    return cudaErrorInvalidValue;
  AttnArgs a;
  a.q = q;
  a.q_s0 = s.q_s[0];
  a.q_s1 = s.q_s[1];
  a.q_s2 = s.q_s[2];
  a.ids = ids;
  a.seq_lens = s.seq_lens;
  a.n_q = s.n_q;
  a.max_kv = s.max_kv;
  a.H = s.H;
  a.h = s.h;
  a.G = s.G;
  a.topk = s.topk;
  a.block = s.block;
  a.nblk = s.nblk;
  a.causal = s.causal;
  a.scale_log2 = s.scale * kLog2e;
  a.stages = pl.stages;
  a.stage_bytes = pl.stage_bytes;
  a.region_bytes = pl.region_bytes;
  a.merge_off = pl.merge_off;
  a.list_cap = pl.list_cap;
  a.total_slots = pl.total;
  a.per = pl.per;
  a.smax = pl.smax;
  a.part_o = nullptr;
  a.part_lse = nullptr;
  a.counters = nullptr;
  a.out = out;
  a.o_s0 = s.o_s[0];
  a.o_s1 = s.o_s[1];
  a.o_s2 = s.o_s[2];
  a.lse = lse;
  a.st = st;
  a.wait_ns = 4000000000ull;  // 4 s: far above any healthy wait, even under a profiler
  a.pg = s.pages;
  a.ks = s.ks;
  a.vs = s.vs;
  a.unit = q8_unit(s);
  cudaError_t err;
  if (!pl.stream && !s.kv8 && kv_attn_supported(s)) {
    CUtensorMap tmq;
    if (!make_q_group_map(&tmq, q, s)) return cudaErrorInvalidValue;
    return launch_kv_attn(s, tmq, tmk, tmv, q, ids, out, lse, partials, partial_bytes, st, stream);
  }
  const bool kv8 = s.kv8;
  auto launch = [&](auto kernel, int threads) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)pl.smem_bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)pl.ctas), dim3(threads), pl.smem_bytes, stream, tmk,
                      tmv, a);
  };
  if (!pl.stream) {
    constexpr int NT = 5 * 32;
    if (kv8)
      return with_q8_state(
          s, [&](auto ws) { return launch(sparse_attn_rows_kernel<decltype(ws)::kD, decltype(ws)>, NT); });
    return s.d == 128 ? launch(sparse_attn_rows_kernel<128, WarpState<128>>, NT)
                      : launch(sparse_attn_rows_kernel<64, WarpState<64>>, NT);
  }
  const size_t nrow_h = (size_t)s.batch * s.n_q * s.H;
  if (partials == nullptr || partial_bytes < attn_partial_bytes(s)) return cudaErrorInvalidValue;
  a.part_o = reinterpret_cast<float*>(partials);
  a.part_lse = a.part_o + nrow_h * pl.smax * s.d;
  int ncounters = 0;
  a.counters = attn_merge_counters(s, partials, &ncounters);
  if (fixed_counters != nullptr && ncounters <= kFixedCounters) {
    a.counters = fixed_counters;  // zero already, and left at zero
  } else if (!counters_zeroed) {
    err = cudaMemsetAsync(a.counters, 0, (size_t)ncounters * sizeof(int), stream);
    if (err != cudaSuccess) return err;
  }
  constexpr int NT = (kStreamNC + 1) * 32;
  // groups of up to 8 heads take the swapped MMA operands
  if (kv8)
    return with_q8_state(s, [&](auto ws) {
      using WS = decltype(ws);
      return launch(sparse_attn_stream_kernel<WS::kD, kStreamNC, WS>, NT);
    });
  if (s.d == 128)
    return s.G <= 8 ? launch(sparse_attn_stream_kernel<128, kStreamNC, WarpStateT<128>>, NT)
                    : launch(sparse_attn_stream_kernel<128, kStreamNC, WarpState<128>>, NT);
  return s.G <= 8 ? launch(sparse_attn_stream_kernel<64, kStreamNC, WarpStateT<64>>, NT)
                  : launch(sparse_attn_stream_kernel<64, kStreamNC, WarpState<64>>, NT);
}

}  // namespace msa
