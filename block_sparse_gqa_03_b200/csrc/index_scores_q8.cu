// Index scores of a decode step over an 8-bit index key (e4m3 codes, one scale per
// block):  S[b, g, beta] = s_beta * max over visible j in beta of <q_idx, code_j>.
// The scale is positive, so it moves out of the maximum and multiplies one number
// per (group, block).
//
// What bounds it: L_b * d_idx bytes of HBM per sequence, half of the bf16 scan's.
// Persistent, one CTA per SM, each an equal contiguous share of the flattened
// (sequence, block) items.  A producer lane streams each block's codes by TMA (rows
// of d_idx bytes, swizzled by the row size) into a ring of stages; consumer warp w
// takes items w, w + 8, ...  A code row is read by ldmatrix as pairs of bytes: a
// lane's 32-bit register holds four consecutive codes of one token, which two
// hardware conversions widen to f16 pairs, i.e. to the two halves of an A fragment
// whose 16 dims are taken in that order (the query's fragments are laid out alike).
#include "kernels.h"
#include "q8.cuh"

namespace msa {
namespace {

struct ScanQ8Args {
  const uint16_t* q_idx;
  int64_t qi_s0, qi_s2;
  const float* scale;
  const int32_t* seq_lens;
  int batch, max_kv, h, block, nblk, stages;
  uint32_t stage_bytes;
  float* scores;
  int fill_tail;
  DeviceStatus* st;
  uint64_t wait_ns;
  KvPages pg;
};

constexpr int kWarps = 8;      // consumer warps; one more warp produces
constexpr int kMaxStages = 64;

__device__ __forceinline__ int seq_blocks(const ScanQ8Args& a, int b) {
  return (kv_length(a.seq_lens, b, a.max_kv, a.st) + a.block - 1) / a.block;
}

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                              int tok, int plane) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(tok), "r"(plane), "r"(bar)
      : "memory");
}

template <int DI, int NT>
__global__ void __launch_bounds__((kWarps + 1) * 32, 1)
    index_scan_q8_kernel(const __grid_constant__ CUtensorMap tmk, ScanQ8Args a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int NW = kWarps;
  constexpr int NC = DI / 16;  // 16-dim steps
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int S = a.stages;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)S * a.stage_bytes);
  int4* info = reinterpret_cast<int4*>(bars + 2 * S);  // [S] (sequence, block, scale index)
  int* n_items = reinterpret_cast<int*>(info + S);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == NW) {
    // Producer warp: barriers, this CTA's share of the items (counted over the
    // sequences' block counts), then groups of 32 items: every lane resolves one
    // item's sequence, block and page, and lane 0 streams the group.
    if (lane == 0) {
      for (int s = 0; s < S; ++s) {
        mbar_init(full0 + 8 * s, 1);
        mbar_init(empty0 + 8 * s, 1);
      }
      fence_mbar_init();
      prefetch_tensormap(&tmk);
    }
    const bool skip = status_failed(a.st);
    int total = 0;
    for (int b = lane; b < a.batch; b += 32) total += seq_blocks(a, b);
    total = (int)__reduce_add_sync(0xffffffffu, (unsigned)total);
    const int per = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const int i0 = (int)min((int64_t)blockIdx.x * per, (int64_t)total);
    const int n = min(total - i0, per);
    int b0 = 0, beta0 = 0, carry = 0;
    bool found = false;
    for (int base = 0; base < a.batch && !found; base += 32) {
      const int b = base + lane;
      const int nb = b < a.batch ? seq_blocks(a, b) : 0;
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
    if (lane == 0) *n_items = skip ? -1 : n;
    __syncwarp();
    named_arrive(2, (NW + 1) * 32);
    if (skip || n == 0) return;
    int b = b0, beta = beta0, issued = 0;
    bool failed = false;
    for (int k0 = 0; k0 < n && !failed; k0 += 32) {
      int bb = b, bt = beta, tok = 0, plane = 0, sidx = 0;
      if (k0 + lane < n) {
        bt += lane;
        int nbb = seq_blocks(a, bb);
        while (bt >= nbb) {  // the item exists, so bb stays below the batch
          bt -= nbb;
          nbb = seq_blocks(a, ++bb);
        }
        kv_block_coords(a.pg, bb, bt, a.block, a.st, tok, plane);
        sidx = a.pg.table == nullptr ? bb * a.nblk + bt : plane < a.pg.pages ? plane : -1;
      }
      const int cnt = min(32, n - k0);
      for (int j = 0; j < cnt; ++j) {
        const int tj = __shfl_sync(0xffffffffu, tok, j), pj = __shfl_sync(0xffffffffu, plane, j);
        const int bj = __shfl_sync(0xffffffffu, bb, j), ej = __shfl_sync(0xffffffffu, bt, j);
        const int sj = __shfl_sync(0xffffffffu, sidx, j);
        const int k = k0 + j, s = k % S;
        if (lane == 0 && !failed) {
          if (k >= S &&
              !mbar_wait_bounded(empty0 + 8 * s, ((k / S) - 1) & 1, a.st, 0x401u, a.wait_ns)) {
            failed = true;
          } else {
            info[s] = make_int4(bj, ej, sj, 0);
            const uint32_t full = full0 + 8 * s;
            mbar_arrive_expect_tx(full, a.stage_bytes);
            tma_load_rows(sbase + (uint32_t)s * a.stage_bytes, &tmk, full, tj, pj);
            issued = k + 1;
          }
        }
        __syncwarp();
      }
      failed = __shfl_sync(0xffffffffu, failed, 0);
      b = __shfl_sync(0xffffffffu, bb, 31);  // the next group starts after this group's last item
      beta = __shfl_sync(0xffffffffu, bt, 31) + 1;
    }
    if (lane != 0) return;
    // before leaving, wait (bounded) for the copies still in flight
    for (int k = max(0, issued - S); k < issued; ++k)
      mbar_wait_bounded(full0 + 8 * (k % S), (k / S) & 1, a.st, 0x403u, a.wait_ns);
    return;
  }

  named_sync(2, (NW + 1) * 32);
  const int n = *n_items;
  if (n < 0) return;
  const int r = lane >> 2, q = lane & 3;
  const float ninf = -__int_as_float(0x7f800000);
  uint32_t blo[NT][NC], bhi[NT][NC];
  float inv[NT][2];  // the query scaling of columns 2q and 2q + 1 undone
  int cur_b = -1, L = 0;
  for (int k = warp; k < n; k += NW) {
    const int s = k % S;
    if (!mbar_wait_warp(full0 + 8 * s, (k / S) & 1, a.st, 0x402u, a.wait_ns)) break;
    const int4 it = info[s];
    const float sc = it.z >= 0 ? __ldg(a.scale + it.z) : 1.f;  // a bad page reads as zeros
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
    const uint32_t base = sbase + (uint32_t)s * a.stage_bytes;
    float cm[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) cm[nt][0] = cm[nt][1] = ninf;
    for (int mt = 0; mt < a.block / 16; ++mt) {
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
      const uint32_t row = (uint32_t)(mt * 16 + (lane & 15));
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        uint32_t x0, x1, x2, x3;  // tokens 0-7, 8-15 of step c, then of step c + 1
        ldmatrix_x4(base + q8::swz<DI>(row, (uint32_t)(c + (lane >> 4))), x0, x1, x2, x3);
        const uint32_t a0 = q8::lo_f16x2(x0), a1 = q8::lo_f16x2(x1);
        const uint32_t a2 = q8::hi_f16x2(x0), a3 = q8::hi_f16x2(x1);
        const uint32_t b0 = q8::lo_f16x2(x2), b1 = q8::lo_f16x2(x3);
        const uint32_t b2 = q8::hi_f16x2(x2), b3 = q8::hi_f16x2(x3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          q8::mma_f16(acc[nt], a0, a1, a2, a3, blo[nt][c], bhi[nt][c]);
          q8::mma_f16(acc[nt], b0, b1, b2, b3, blo[nt][c + 1], bhi[nt][c + 1]);
        }
      }
      const int jl = it.y * a.block + mt * 16 + r, jh = jl + 8;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          cm[nt][e] = fmaxf(cm[nt][e], jl < L ? acc[nt][e] : ninf);
          cm[nt][e] = fmaxf(cm[nt][e], jh < L ? acc[nt][2 + e] : ninf);
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * s);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = cm[nt][e];
        v = warp_max_xor(v, 4);
        v = warp_max_xor(v, 8);
        v = warp_max_xor(v, 16);
        const int g = nt * 8 + 2 * q + e;
        if (r == 0 && g < a.h)
          a.scores[((int64_t)it.x * a.h + g) * a.nblk + it.y] = v * (inv[nt][e] * sc);
      }
  }
  if (a.fill_tail) {
    // blocks past each sequence's end: -inf, spread over every consumer thread
    const int nthr = (int)gridDim.x * NW * 32;
    const int gt = (int)blockIdx.x * NW * 32 + (int)threadIdx.x;
    for (int b = 0; b < a.batch; ++b)
      for (int beta = seq_blocks(a, b) + gt; beta < a.nblk; beta += nthr)
        for (int g = 0; g < a.h; ++g) a.scores[((int64_t)b * a.h + g) * a.nblk + beta] = ninf;
  }
}

template <int DI, int NT>
cudaError_t run_scan(const Shape& s, const uint8_t* k_idx, ScanQ8Args& a, cudaStream_t stream) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const bool paged = s.pages.table != nullptr;
  cuuint64_t dims[3] = {(cuuint64_t)DI, (cuuint64_t)(paged ? s.block : s.max_kv),
                        (cuuint64_t)(paged ? s.pages.pages : s.batch)};
  cuuint64_t str[2] = {(cuuint64_t)s.ki_s[1], (cuuint64_t)s.ki_s[0]};
  cuuint32_t box[3] = {DI, (cuuint32_t)s.block, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUtensorMap tmk;
  const CUtensorMapSwizzle sw = DI == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : DI == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_32B;
  if (enc(&tmk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(k_idx), dims, str, box, es,
          CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  a.stage_bytes = (uint32_t)DI * (uint32_t)s.block;
  // A stage count that is a multiple of the warps keeps each stage on one consumer
  // warp, so a parity wait never meets a phase two fills behind.
  const size_t fixed = 1024 + 16, per_stage = a.stage_bytes + 32;
  const int fit = (int)(((size_t)max_smem_optin() - fixed) / per_stage);
  a.stages = min(kMaxStages, fit - fit % kWarps);
  if (a.stages < kWarps) return cudaErrorInvalidValue;  // 16 KB stages: 8 always fit
  const size_t smem = fixed + (size_t)a.stages * per_stage;
  cudaError_t err = cudaFuncSetAttribute(index_scan_q8_kernel<DI, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(index_scan_q8_kernel<DI, NT>, dim3(num_sms()), dim3((kWarps + 1) * 32), smem,
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
  const bool two = s.h > 8;
  switch (s.d_idx) {
    case 128:
      return two ? run_scan<128, 2>(s, k_idx, a, stream) : run_scan<128, 1>(s, k_idx, a, stream);
    case 64:
      return two ? run_scan<64, 2>(s, k_idx, a, stream) : run_scan<64, 1>(s, k_idx, a, stream);
    case 32:
      return two ? run_scan<32, 2>(s, k_idx, a, stream) : run_scan<32, 1>(s, k_idx, a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace msa
