// Shared by the sparse attention kernels that walk (row, slot) lists: their arguments,
// row geometry, the compaction of a range of slots into a list of blocks, and the merge
// of the consumer warps' states.  A "row" is one (sequence, query, group).
#pragma once

#include "kernels.h"

namespace msa {

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

namespace {

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

// Rows number batch * n_q * h, which fits 32 bits.
__device__ __forceinline__ RowGeo row_geo(const AttnArgs& a, int64_t row) {
  RowGeo r;
  const int rowg = (int)row;
  r.bt = rowg / a.h;
  r.g = rowg - r.bt * a.h;
  r.b = r.bt / a.n_q;
  r.t = r.bt - r.b * a.n_q;
  const int L = kv_length(a.seq_lens, r.b, a.max_kv, a.st);
  const int p = L - a.n_q + r.t;
  r.lim = a.causal ? min(L, p + 1) : L;  // visible tokens: j < lim
  return r;
}

// Merge of NC warp states for tile row `row`, dims [dim, dim + 4) (dim a
// multiple of 4): normalised output and natural-log LSE (-inf and 0 when no key
// was seen).  The warps' weights are computed once for the four dims.  LD: floats from
// one O row to the next.  NANS: a NaN maximum of a warp makes the row NaN.
template <int D, int NC, int LD = D, bool NANS = false>
__device__ __forceinline__ void merge_warps4(const float* mo, const float* mm, const float* ml,
                                             int gr, int row, int dim, float4& val, float& lsev) {
  const float ninf = neg_inf();
  float M = ninf;
#pragma unroll
  for (int w = 0; w < NC; ++w) M = NANS ? fmax_nan(M, mm[w * 16 + row]) : fmaxf(M, mm[w * 16 + row]);
  val = make_float4(0.f, 0.f, 0.f, 0.f);
  lsev = ninf;
  if (M == ninf) return;
  float wsum = 0.f;
  float4 acc = val;
#pragma unroll
  for (int w = 0; w < NC; ++w) {
    const float f = exp2f(mm[w * 16 + row] - M);
    wsum += f * ml[w * 16 + row];
    const float4 o = *reinterpret_cast<const float4*>(mo + (w * gr + row) * LD + dim);
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

// Compacts slots [s0, s1) of the flattened id array into the entry list: only
// blocks holding a visible token are kept.  For each kept block, glist gets its
// KV head and plist its sequence (with a paged cache: its page, looked up by the
// lanes in parallel), so that the producer's loop does no index arithmetic.  row0 and
// row1: the rows of the first and the last slot.  Run by one full warp; returns the
// count.
__device__ __forceinline__ int compact_ids(const AttnArgs& a, int64_t s0, int64_t s1,
                                           int64_t row0, int64_t row1, int32_t* list, int32_t* plist,
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
  const int64_t span = row1 - row0 + 1;
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

}  // namespace

// How launch_sparse_attn runs a shape.
struct AttnPlan {
  bool stream;  // persistent streaming kernel (few rows), else one CTA per row
  int stages, ctas, per, smax, list_cap;
  int64_t total;
  uint32_t stage_bytes, region_bytes, merge_off;
  size_t smem_bytes;
};

// 8-bit cache (sparse_attn_q8.cu).
AttnPlan plan_attn_q8(const Shape& s);
// K or V codes as a 4-D tensor [batch][token][kv head][dim], or for a paged cache
// [page][token in page][kv head][dim]; one box is `dims` codes x 1 head x `tokens`,
// swizzled by its row size when `swizzle`.
bool make_codes_map(CUtensorMap* map, const void* base, const Shape& s, const int64_t* str,
                    int dims, int tokens, bool swizzle);
cudaError_t run_attn_q8(const Shape& s, const AttnPlan& pl, const void* k, const void* v,
                        const AttnArgs& a, cudaStream_t stream);

}  // namespace msa
