// Index scores of a decode step over an 8-bit index key (e4m3 codes, one scale per
// block):  S[b, g, beta] = s_beta * max over visible j in beta of <q_idx, code_j>.
// The scale is positive, so it moves out of the maximum and multiplies one number
// per (group, block).
//
// What bounds it: L_b * d_idx bytes of HBM per sequence, half of the bf16 scan's.
// Persistent, one CTA per SM, each an equal contiguous share of the flattened items (a
// block of a sequence, or 64 tokens of smaller blocks: a block of 16 at a time took 29 us
// for 9 x 60K tokens, four of them 13.5 us); the CTA's warps take its items in turn.  Each
// warp streams its own
// items: it resolves 32 of them at a time (one per lane: sequence, block, page,
// scale), its lane 0 issues the TMA loads (rows of d_idx bytes, swizzled by the row
// size) into the warp's private ring of stages and refills a stage as soon as the
// warp has read it.  One producer warp for all of them, as in the bf16 scan, issues an
// 8 KB block every 250 ns at best: 61.7 us against 52.3 us for 16 x 128K tokens of 128
// dims (41.7 us of HBM time).
//
// A code row is read by ldmatrix as pairs of bytes: a lane's 32-bit register holds
// four consecutive codes of one token, which two hardware conversions widen to f16
// pairs, i.e. to the two halves of an A fragment whose 16 dims are taken in that order
// (the query's fragments are laid out alike).
#include <type_traits>

#include "kernels.h"
#include "q8.cuh"
#include "sm100.cuh"

namespace msa {
namespace {

struct ScanQ8Args {
  const uint16_t* q_idx;
  int64_t qi_s0, qi_s2;
  const float* scale;
  const int32_t* seq_lens;
  int batch, max_kv, h, block, nblk;
  int depth;  // stages per warp, 64 tokens each
  uint32_t stage_bytes;
  float* scores;
  int fill_tail;
  DeviceStatus* st;
  uint64_t wait_ns;
  KvPages pg;
};

constexpr int kWarps = 12;  // 8: 53.4 us for the scan above, 12: 52.3, 16: 53.9
constexpr int kMaxDepth = 16;  // stages of a warp

__device__ __forceinline__ int seq_blocks(const ScanQ8Args& a, int b) {
  return (kv_length(a.seq_lens, b, a.max_kv, a.st) + a.block - 1) / a.block;
}
// Items of a sequence: a block, or the 64 tokens of several smaller ones.
__device__ __forceinline__ int seq_items(const ScanQ8Args& a, int b) {
  const int per = a.block < 64 ? 64 : a.block;
  return (kv_length(a.seq_lens, b, a.max_kv, a.st) + per - 1) / per;
}

// NB: blocks of an item (block 16: 4, 32: 2, else 1).
template <int DI, int NT, int NB>
__global__ void __launch_bounds__(kWarps * 32, 1)
    index_scan_q8_kernel(const __grid_constant__ CUtensorMap tmk, ScanQ8Args a) {
  constexpr int NW = kWarps;
  constexpr int NC = DI / 16;   // 16-dim steps
  constexpr int MT = 4;         // 16-token tiles of a stage
  constexpr int TPB = MT / NB;  // of them, a block's
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int depth = a.depth;
  // this warp's ring: stages, barriers, and each stage's (sequence, first block) and
  // block scales
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * depth) * a.stage_bytes;
  uint8_t* tail = smem + (size_t)(NW * depth) * a.stage_bytes;
  float4* iscale = reinterpret_cast<float4*>(tail) + warp * depth;
  int2* info = reinterpret_cast<int2*>(tail + (size_t)(NW * depth) * 16) + warp * depth;
  const uint32_t bars =
      smem_u32(reinterpret_cast<uint64_t*>(tail + (size_t)(NW * depth) * 24) + warp * depth);
  if (lane == 0) {
    for (int s = 0; s < depth; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
    if (warp == 0) prefetch_tensormap(&tmk);
  }
  grid_dep_wait();  // nothing above needs the kernels before this one
  grid_dep_launch();
  const bool skip = status_failed(a.st);
  // this CTA's share of the items, counted over the sequences
  int total = 0;
  for (int b = lane; b < a.batch; b += 32) total += seq_items(a, b);
  total = (int)__reduce_add_sync(0xffffffffu, (unsigned)total);
  const int per = (total + (int)gridDim.x - 1) / (int)gridDim.x;
  const int i0 = (int)min((int64_t)blockIdx.x * per, (int64_t)total);
  const int n = skip ? 0 : min(total - i0, per);
  int b0 = 0, beta0 = 0, carry = 0;
  bool found = false;
  for (int base = 0; base < a.batch && !found; base += 32) {
    const int b = base + lane;
    const int nb = b < a.batch ? seq_items(a, b) : 0;
    int inc = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const int excl = carry + inc - nb;
    const unsigned hit = __ballot_sync(0xffffffffu, nb > 0 && i0 >= excl && i0 < excl + nb);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b0 = base + src;
      beta0 = i0 - __shfl_sync(0xffffffffu, excl, src);
      found = true;
    }
    carry += __shfl_sync(0xffffffffu, inc, 31);
  }

  // the warp's items j = 0, 1, ...: item warp + j NW of the share
  const int items = n > warp ? (n - warp + NW - 1) / NW : 0;
  const int subs = a.block > 64 ? a.block / 64 : 1;  // stages per item (1 or 2)
  const int loads = items * subs;
  int bb = b0, bt = beta0 + warp + lane * NW;
  int plane[NB];
  float scale[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    plane[k] = 0;
    scale[k] = 1.f;
  }
  const bool paged = a.pg.table != nullptr;
  auto resolve = [&](int j) {  // this lane's item j
    if (j >= items) return;
    for (int nbb; bt >= (nbb = seq_items(a, bb)); ++bb) bt -= nbb;
    const int nblk_b = seq_blocks(a, bb);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int beta = bt * NB + k;
      plane[k] = bb;
      if (paged) {
        // a block past the sequence's end, or a page outside the pool, reads as zeros
        const int64_t page = beta < nblk_b ? kv_page(a.pg, bb, beta, a.st) : -1;
        plane[k] = page < 0 ? (int)a.pg.pages : (int)page;
      }
      scale[k] = 1.f;
      if (beta < nblk_b && (!paged || plane[k] < a.pg.pages))
        scale[k] = __ldg(a.scale + (paged ? (int64_t)plane[k] : (int64_t)bb * a.nblk + beta));
    }
  };
  resolve(lane);
  int is = 0;  // stage of the next load
  auto issue = [&](int l) {
    const int j = l / subs, sub = l - j * subs;
    if (sub == 0 && j > 0 && (j & 31) == 0) {
      bt += 32 * NW;
      resolve(j + lane);
    }
    const int src = j & 31;
    const int bj = __shfl_sync(0xffffffffu, bb, src), ej = __shfl_sync(0xffffffffu, bt, src) * NB;
    int pj[NB];
    float sj[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      pj[k] = __shfl_sync(0xffffffffu, plane[k], src);
      sj[k] = __shfl_sync(0xffffffffu, scale[k], src);
    }
    if (lane == 0) {
      info[is] = make_int2(bj, ej);
      iscale[is] = make_float4(sj[0], sj[1], sj[2], sj[3]);
      const uint32_t dst = ring + (uint32_t)is * a.stage_bytes, bar = bars + 8 * is;
      mbar_arrive_expect_tx(bar, a.stage_bytes);
      if (!paged) {
        tma_load_3d(dst, &tmk, bar, 0, ej * a.block + sub * 64, bj);
      } else {
#pragma unroll
        for (int k = 0; k < NB; ++k)
          tma_load_3d(dst + (uint32_t)(k * (64 / NB) * DI), &tmk, bar, 0, sub * 64, pj[k]);
      }
    }
    __syncwarp();
    if (++is == depth) is = 0;
  };
  int issued = 0;
  for (; issued < min(depth, loads); ++issued) issue(issued);

  const int r = lane >> 2, q = lane & 3;
  const float ninf = -__int_as_float(0x7f800000);
  uint32_t blo[NT][NC], bhi[NT][NC];
  float inv[NT][2];  // the query scaling of columns 2q and 2q + 1 undone
  float cm[NB][NT][2];
  int cur_b = -1, L = 0;
  int s = 0, sub = 0;
  uint32_t par = 0;
  for (int l = 0; l < loads; ++l) {
    if (!mbar_wait_warp(bars + 8 * s, par, a.st, 0x402u, a.wait_ns)) {
      // before leaving, wait (bounded) for the copies still in flight
      for (++l; l < issued; ++l) {
        if (++s == depth) {
          s = 0;
          par ^= 1u;
        }
        mbar_wait_warp(bars + 8 * s, par, a.st, 0x403u, a.wait_ns);
      }
      break;
    }
    const int2 it = info[s];
    const float4 sc4 = iscale[s];
    if (it.x != cur_b) {
      cur_b = it.x;
      L = kv_length(a.seq_lens, cur_b, a.max_kv, a.st);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int g = nt * 8 + r;
        const float f = q8::load_row_f16<NC>(
            a.q_idx + cur_b * a.qi_s0 + (int64_t)g * a.qi_s2 + 4 * q, g < a.h, blo[nt], bhi[nt]);
        inv[nt][0] = __shfl_sync(0xffffffffu, f, 8 * q);
        inv[nt][1] = __shfl_sync(0xffffffffu, f, 8 * q + 4);
      }
    }
    const uint32_t base = ring + (uint32_t)s * a.stage_bytes;
    if (sub == 0) {
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) cm[k][nt][0] = cm[k][nt][1] = ninf;
    }
    // the stage's 16-token tiles together: their MMA chains are independent
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        acc[m][nt][0] = acc[m][nt][1] = acc[m][nt][2] = acc[m][nt][3] = 0.f;
    const uint32_t row = (uint32_t)(lane & 15);
#pragma unroll
    for (int c = 0; c < NC; c += 2) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t x0, x1, x2, x3;  // tokens 0-7, 8-15 of step c, then of step c + 1
        ldmatrix_x4(base + q8::swz<DI>(row + 16 * m, (uint32_t)(c + (lane >> 4))), x0, x1, x2, x3);
        const uint32_t a0 = q8::lo_f16x2(x0), a1 = q8::lo_f16x2(x1);
        const uint32_t a2 = q8::hi_f16x2(x0), a3 = q8::hi_f16x2(x1);
        const uint32_t b0 = q8::lo_f16x2(x2), b1 = q8::lo_f16x2(x3);
        const uint32_t b2 = q8::hi_f16x2(x2), b3 = q8::hi_f16x2(x3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          q8::mma_f16(acc[m][nt], a0, a1, a2, a3, blo[nt][c], bhi[nt][c]);
          q8::mma_f16(acc[m][nt], b0, b1, b2, b3, blo[nt][c + 1], bhi[nt][c + 1]);
        }
      }
    }
    const int j0 = it.y * a.block + sub * 64;
    const bool whole = j0 + 16 * MT <= L;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int jl = j0 + 16 * m + r, jh = jl + 8;
      const bool okl = whole || jl < L, okh = whole || jh < L;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = cm[m / TPB][nt][e];
          x = fmax3(x, okl ? acc[m][nt][e] : ninf, okh ? acc[m][nt][2 + e] : ninf);
        }
    }
    __syncwarp();  // every lane has read the stage: it may be refilled
    if (issued < loads) issue(issued++);
    if (++s == depth) {
      s = 0;
      par ^= 1u;
    }
    if (++sub < subs) continue;
    sub = 0;
    const float scs[4] = {sc4.x, sc4.y, sc4.z, sc4.w};
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (NB > 1 && (it.y + k) * a.block >= L) break;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = cm[k][nt][e];
          v = warp_max_xor(v, 4);
          v = warp_max_xor(v, 8);
          v = warp_max_xor(v, 16);
          const int g = nt * 8 + 2 * q + e;
          if (r == 0 && g < a.h)
            a.scores[((int64_t)it.x * a.h + g) * a.nblk + it.y + k] = v * (inv[nt][e] * scs[k]);
        }
    }
  }
  if (a.fill_tail) {
    // blocks past each sequence's end: -inf, spread over every thread
    const int nthr = (int)gridDim.x * NW * 32;
    const int gt = (int)blockIdx.x * NW * 32 + (int)threadIdx.x;
    for (int b = 0; b < a.batch; ++b)
      for (int beta = seq_blocks(a, b) + gt; beta < a.nblk; beta += nthr)
        for (int g = 0; g < a.h; ++g) a.scores[((int64_t)b * a.h + g) * a.nblk + beta] = ninf;
  }
}

template <int DI, int NT, int NB>
cudaError_t run_scan(const Shape& s, const uint8_t* k_idx, ScanQ8Args& a, cudaStream_t stream) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const bool paged = s.pages.table != nullptr;
  cuuint64_t dims[3] = {(cuuint64_t)DI, (cuuint64_t)(paged ? s.block : s.max_kv),
                        (cuuint64_t)(paged ? s.pages.pages : s.batch)};
  cuuint64_t str[2] = {(cuuint64_t)s.ki_s[1], (cuuint64_t)s.ki_s[0]};
  // a stage's 64 tokens, or the pages of its blocks one by one
  cuuint32_t box[3] = {DI, (cuuint32_t)(paged && s.block < 64 ? s.block : 64), 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUtensorMap tmk;
  const CUtensorMapSwizzle sw = DI == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : DI == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_32B;
  if (enc(&tmk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(k_idx), dims, str, box, es,
          CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  a.stage_bytes = (uint32_t)DI * 64u;
  const size_t fixed = 1024, per_stage = a.stage_bytes + 32;
  a.depth = min(kMaxDepth, (int)(((size_t)max_smem_optin() - fixed) / (per_stage * kWarps)));
  if (a.depth < 1) return cudaErrorInvalidValue;  // 8 KB stages at most: 2 fit
  const size_t smem = fixed + (size_t)(a.depth * kWarps) * per_stage;
  cudaError_t err = cudaFuncSetAttribute(index_scan_q8_kernel<DI, NT, NB>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(index_scan_q8_kernel<DI, NT, NB>, dim3(num_sms()), dim3(kWarps * 32), smem,
                    stream, tmk, a);
}

}  // namespace

cudaError_t launch_index_scan_q8(const Shape& s, const uint16_t* q_idx, const uint8_t* k_idx,
                                 const float* k_idx_scale, float* scores, bool fill_tail,
                                 DeviceStatus* st, cudaStream_t stream) {
  if (s.n_q != 1 || (int64_t)s.batch * s.nblk > INT32_MAX - 4096) return cudaErrorInvalidValue;
  ScanQ8Args a = {};
  a.q_idx = q_idx;
  a.qi_s0 = s.qi_s[0];
  a.qi_s2 = s.qi_s[2];
  a.scale = k_idx_scale;
  a.seq_lens = s.seq_lens;
  a.batch = s.batch;
  a.max_kv = s.max_kv;
  a.h = s.h;
  a.block = s.block;
  a.nblk = s.nblk;
  a.scores = scores;
  a.fill_tail = fill_tail ? 1 : 0;
  a.st = st;
  a.wait_ns = 4000000000ull;
  a.pg = s.pages;
  auto run = [&](auto di, auto nt) {
    constexpr int DI = decltype(di)::value, NT = decltype(nt)::value;
    return s.block >= 64   ? run_scan<DI, NT, 1>(s, k_idx, a, stream)
           : s.block == 32 ? run_scan<DI, NT, 2>(s, k_idx, a, stream)
                           : run_scan<DI, NT, 4>(s, k_idx, a, stream);
  };
  auto with_di = [&](auto di) {
    return s.h > 8 ? run(di, std::integral_constant<int, 2>())
                   : run(di, std::integral_constant<int, 1>());
  };
  if (s.d_idx == 128) return with_di(std::integral_constant<int, 128>());
  if (s.d_idx == 64) return with_di(std::integral_constant<int, 64>());
  if (s.d_idx == 32) return with_di(std::integral_constant<int, 32>());
  return cudaErrorInvalidValue;
}

}  // namespace msa
