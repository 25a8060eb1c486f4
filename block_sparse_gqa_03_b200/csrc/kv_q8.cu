// The 8-bit KV cache's write and read-back.
//
// Write (append_kv_q8_kernel).  New bf16 rows x of sequence b go to positions
// L_b - n .. L_b - 1.  For each (block, head) that receives rows:
//   need = smallest 2^e >= 2^-100 with max |x| <= 448 * 2^e  (largest finite |x|)
//   s'   = max(s, need) when the block holds older rows, else need
//   older rows: code' = e4m3(code * s / s');  new rows: code = e4m3(x / s')
// (round to nearest even; infinities saturate, NaN stays NaN).  s and s' are powers
// of two, so both quotients are exact before the one rounding.  A larger s' leaves
// a code that stays normal as it is, so a block filled row by row drifts from one
// filled at once only in values below 2^-6 of the scale.
// A block's first row starts it afresh: what a recycled page held before does not
// count.  One CTA per (sequence, touched block, K head | V head | index key): it
// holds the block's new rows in registers between the maximum and the rounding, so
// each new element is read once, and no other CTA touches the scale it replaces.
// Bound: HBM, 3 bytes per element.  2 x 32K rows of 4 heads of 128 dims (213 MB): 35.3
// us with CTAs of 128 threads, 40.1 us of 256 (fewer CTAs per SM cover the wait for the
// maximum); 32.6 us at the measured copy rate.
//
// Read (read_kv_q8_kernel).  out = bf16(code * s), exact for power-of-two scales.
// One CTA per 32 (or block, when smaller) tokens of a sequence: one page lookup and
// one set of scales serve all its rows.  Bound: 3 bytes of HBM per element (2 of them
// written) and, above that, the latency of its loads.  The rows above (213 MB): 43 us, and
// the same within 3% for pieces of 8 codes, other orders of heads and rows and other CTA
// sizes; a plain copy of as many bytes takes 36.3 us, DRAM runs at 45% of its peak and 41%
// of the warps are resident (2048 CTAs, 1.7 rounds).
#include "kernels.h"
#include "q8.cuh"

namespace msa {
namespace {

struct Q8Args {
  int n, max_kv, h, d, d_idx, block, nblk;
  const int32_t* seq_lens;
  const uint16_t *k_new, *v_new, *ki_new;  // dense rows to write
  uint16_t *k_out, *v_out, *ki_out;        // dense rows to read into
  uint8_t *k, *v, *ki;
  float *ks, *vs, *kis;
  int64_t k_s[3], v_s[3], ki_s[2];
  KvPages pg;
  DeviceStatus* st;
  int per_seq;      // write: block slots of a sequence; read: token groups
  int64_t base;     // read: first position
  int group;        // read: tokens per CTA
  float* block_scales;  // read: the index key comes out as codes, its scales here
};

constexpr int kThreads = 128;

// The K head, V head or index key that CTA unit `u` of a token row stands for.
struct Unit {
  const uint16_t* src;
  int64_t src_s;  // elements between two tokens of the dense rows
  uint8_t* codes;
  int64_t plane_s, row_s;
  float* scale;
  int heads, g, d;
};

__device__ __forceinline__ Unit unit_of(const Q8Args& a, int u) {
  Unit r;
  if (u < a.h) {
    r = {a.k_new == nullptr ? nullptr : a.k_new + u * a.d, (int64_t)a.h * a.d,
         a.k + u * a.k_s[2], a.k_s[0], a.k_s[1], a.ks, a.h, u, a.d};
  } else if (u < 2 * a.h) {
    const int g = u - a.h;
    r = {a.v_new == nullptr ? nullptr : a.v_new + g * a.d, (int64_t)a.h * a.d,
         a.v + g * a.v_s[2], a.v_s[0], a.v_s[1], a.vs, a.h, g, a.d};
  } else {
    r = {a.ki_new, a.d_idx, a.ki, a.ki_s[0], a.ki_s[1], a.kis, 1, 0, a.d_idx};
  }
  return r;
}

// Largest finite magnitude (bf16 bits) of 16 elements.
__device__ __forceinline__ uint32_t finite_max(const uint4& x, const uint4& y, uint32_t m) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t p = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) p = q8::abs_max2(p, w[i]);
  uint32_t r = max(p & 0xffffu, p >> 16);
  if (r >= 0x7f80u) {  // an infinity or NaN among them
    r = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
      r = max(r, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
  }
  return max(m, r);
}

__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float f) {
  return q8::to_e4m3x4(__uint_as_float(a << 16) * f, __uint_as_float(a & 0xffff0000u) * f,
                       __uint_as_float(b << 16) * f, __uint_as_float(b & 0xffff0000u) * f);
}

// Four codes times a power of two f <= 1 (0 when it underflows), rounded to codes.
__device__ __forceinline__ uint32_t requant4(uint32_t c, float f) {
  const float2 x = q8::f16x2_floats(q8::lo_f16x2(c)), y = q8::f16x2_floats(q8::hi_f16x2(c));
  return q8::to_e4m3x4(x.x * f, x.y * f, y.x * f, y.y * f);
}

// NU: 16-element pieces of a block's new rows per thread.
template <int NU>
__global__ void __launch_bounds__(kThreads) append_kv_q8_kernel(Q8Args a) {
  grid_dep_wait();
  grid_dep_launch();
  const int units = 2 * a.h + 1;
  const int u = blockIdx.x % units;
  const int slot = (blockIdx.x / units) % a.per_seq, b = blockIdx.x / units / a.per_seq;
  const Unit w = unit_of(a, u);
  if (w.src == nullptr) return;
  const int L = kv_length(a.seq_lens, b, a.max_kv, a.st);
  // a length out of range (recorded by kv_length) has no place for the rows: at the end of
  // the cache they would replace the last ones
  if (a.seq_lens != nullptr && a.seq_lens[b] != L) return;
  const int start = L - a.n;  // position of the first new row
  if (start < 0 && slot == 0 && threadIdx.x == 0)
    record_error(a.st, kErrDeviceAssert, 0x30000u | (uint32_t)b);
  const int beta = max(start, 0) / a.block + slot;
  const int tok0 = beta * a.block;  // the block's first position
  if (tok0 >= L) return;
  int64_t plane = b, row0 = tok0, scale_at = ((int64_t)b * a.nblk + beta) * w.heads + w.g;
  if (a.pg.table != nullptr) {
    plane = kv_page(a.pg, b, beta, a.st);
    if (plane < 0) return;  // recorded by kv_page
    row0 = 0;
    scale_at = plane * w.heads + w.g;
  }
  const int r0 = max(start - tok0, 0), r1 = min(L - tok0, a.block);  // the block's new rows
  const float s_old = r0 > 0 ? w.scale[scale_at] : 0.f;
  const int cpr = w.d / 16, shift = __ffs(cpr) - 1;  // 16-element pieces per row (a power of two)
  const int pieces = (r1 - r0) * cpr;
  const uint16_t* src = w.src + ((int64_t)b * a.n + (tok0 + r0 - start)) * w.src_s;
  uint4 x[NU][2];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int p = i * kThreads + threadIdx.x;
    if (p < pieces) {
      const uint16_t* q = src + (int64_t)(p >> shift) * w.src_s + (p & (cpr - 1)) * 16;
      x[i][0] = ld_stream_u4(q);
      x[i][1] = ld_stream_u4(q + 8);
    }
  }
#pragma unroll
  for (int i = 0; i < NU; ++i)
    if (i * kThreads + threadIdx.x < pieces) m = finite_max(x[i][0], x[i][1], m);
  __shared__ uint32_t wmax[kThreads / 32];
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = max(m, wmax[i]);
  int e = q8::scale_exp(m);
  uint8_t* dst = w.codes + plane * w.plane_s + row0 * w.row_s;
  if (r0 > 0) {
    const int e_old = q8::stored_exp(s_old);
    if (e_old == INT_MIN) {  // not a scale of this cache: the block is left as it is
      if (threadIdx.x == 0) record_error(a.st, kErrDeviceAssert, 0x40000u | (uint32_t)b);
      return;
    }
    if (e > e_old) {
      const float f = e_old - e < -60 ? 0.f : q8::pow2f(e_old - e);
      for (int p = threadIdx.x; p < r0 * cpr; p += kThreads) {
        uint4* at = reinterpret_cast<uint4*>(dst + (p >> shift) * w.row_s + (p & (cpr - 1)) * 16);
        const uint4 c = *at;
        *at = make_uint4(requant4(c.x, f), requant4(c.y, f), requant4(c.z, f), requant4(c.w, f));
      }
    } else {
      e = e_old;
    }
  }
  const float inv = q8::pow2f(-e);
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int p = i * kThreads + threadIdx.x;
    if (p < pieces)
      *reinterpret_cast<uint4*>(dst + (r0 + (p >> shift)) * w.row_s + (p & (cpr - 1)) * 16) =
          make_uint4(codes4(x[i][0].x, x[i][0].y, inv), codes4(x[i][0].z, x[i][0].w, inv),
                     codes4(x[i][1].x, x[i][1].y, inv), codes4(x[i][1].z, x[i][1].w, inv));
  }
  if (threadIdx.x == 0) w.scale[scale_at] = q8::pow2f(e);
}

// Two codes times a scale as bf16x2.
__device__ __forceinline__ uint32_t value2(uint32_t f16x2, float s) {
  const float2 v = q8::f16x2_floats(f16x2);
  return pack_bf16(v.x * s, v.y * s);
}

// CODES: the index key comes out as codes, with the scales of its blocks (a form of its own:
// in one with the values, those took 47 us instead of 43 for the rows above).
template <bool CODES>
__global__ void __launch_bounds__(kThreads) read_kv_q8_kernel(Q8Args a) {
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x / a.per_seq, gi = blockIdx.x % a.per_seq;
  const int L = kv_length(a.seq_lens, b, a.max_kv, a.st);
  // positions [p0, p1): one group of the sequence, cut to the rows asked for
  const int64_t g0 = (a.base / a.group + gi) * a.group;
  const int64_t p0 = g0 > a.base ? g0 : a.base;
  int64_t p1 = g0 + a.group;
  if (p1 > a.base + a.n) p1 = a.base + a.n;
  if (p1 > L) p1 = L;
  if (p0 >= p1) return;
  const int beta = (int)(p0 / a.block);
  int64_t plane = b, row0 = p0, scale_at = (int64_t)b * a.nblk + beta;
  if (a.pg.table != nullptr) {
    plane = kv_page(a.pg, b, beta, a.st);
    row0 = p0 - (int64_t)beta * a.block;
    scale_at = plane;
  }
  const bool bad = plane < 0;  // recorded by kv_page; the rows read as zeros
  // (loaded here and stored at the end, so that the codes' loads do not wait for it)
  const bool first = CODES && threadIdx.x == 0 && p0 == (int64_t)beta * a.block;
  float block_scale = 1.f;
  if (first && !bad) block_scale = __ldg(a.kis + scale_at);
  const int rows = (int)(p1 - p0);
  const int64_t out0 = (int64_t)b * a.n + (p0 - a.base);
  // K and V: piece = (head, row, 16 codes), a head's rows together
  auto plane_of = [&](const uint8_t* codes, const int64_t* st, const float* scales, int heads,
                      int d, uint16_t* out) {
    if (out == nullptr) return;
    const int cpr = d / 16, shift = __ffs(cpr) - 1;
    const int per_head = rows << shift;
    const int total = heads * per_head;
    constexpr int U = 4;  // pieces per thread whose loads are under way together
    for (int p0 = threadIdx.x; p0 < total; p0 += U * kThreads) {
      uint4 x[U];
      float s[U];
      uint16_t* o[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = min(p0 + i * kThreads, total - 1);
        const int g = p / per_head, rem = p - g * per_head;
        const int r = rem >> shift, c = rem & (cpr - 1);
        x[i] = make_uint4(0, 0, 0, 0);
        s[i] = 1.f;
        if (!bad) {
          x[i] = ld_stream_u4(codes + plane * st[0] + (row0 + r) * st[1] +
                              (heads > 1 ? g * st[2] : 0) + c * 16);
          if (!CODES) s[i] = __ldg(scales + scale_at * heads + g);
        }
        o[i] = out + ((out0 + r) * heads + g) * d + c * 16;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (p0 + i * kThreads >= total) break;
        *reinterpret_cast<uint4*>(o[i]) =
            make_uint4(value2(q8::lo_f16x2(x[i].x), s[i]), value2(q8::hi_f16x2(x[i].x), s[i]),
                       value2(q8::lo_f16x2(x[i].y), s[i]), value2(q8::hi_f16x2(x[i].y), s[i]));
        *reinterpret_cast<uint4*>(o[i] + 8) =
            make_uint4(value2(q8::lo_f16x2(x[i].z), s[i]), value2(q8::hi_f16x2(x[i].z), s[i]),
                       value2(q8::lo_f16x2(x[i].w), s[i]), value2(q8::hi_f16x2(x[i].w), s[i]));
      }
    }
  };
  if constexpr (!CODES) {
    plane_of(a.k, a.k_s, a.ks, a.h, a.d, a.k_out);
    plane_of(a.v, a.v_s, a.vs, a.h, a.d, a.v_out);
  }
  plane_of(a.ki, a.ki_s, a.kis, 1, a.d_idx, a.ki_out);
  if (first) a.block_scales[(int64_t)b * kis_stride(a.nblk) + beta] = block_scale;
}

Q8Args base_args(const Shape& s, const Q8Cache& c, DeviceStatus* st) {
  Q8Args a = {};
  a.n = s.n_q;
  a.max_kv = s.max_kv;
  a.h = s.h;
  a.d = s.d;
  a.d_idx = s.d_idx;
  a.block = s.block;
  a.nblk = s.nblk;
  a.seq_lens = s.seq_lens;
  a.k = c.k;
  a.v = c.v;
  a.ki = c.ki;
  a.ks = c.ks;
  a.vs = c.vs;
  a.kis = c.kis;
  for (int i = 0; i < 3; ++i) {
    a.k_s[i] = s.k_s[i];
    a.v_s[i] = s.v_s[i];
  }
  a.ki_s[0] = s.ki_s[0];
  a.ki_s[1] = s.ki_s[1];
  a.pg = s.pages;
  a.st = st;
  return a;
}

}  // namespace

cudaError_t launch_append_kv_q8(const Shape& s, const uint16_t* k_new, const uint16_t* v_new,
                                const uint16_t* ki_new, const Q8Cache& c, DeviceStatus* st,
                                cudaStream_t stream) {
  Q8Args a = base_args(s, c, st);
  a.k_new = k_new;
  a.v_new = v_new;
  a.ki_new = ki_new;
  // n consecutive rows touch at most this many blocks
  a.per_seq = (int)(((int64_t)s.n_q + s.block - 2) / s.block + 1);
  const int64_t grid = (int64_t)s.batch * a.per_seq * (2 * s.h + 1);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int d = s.d > s.d_idx ? s.d : s.d_idx;
  const int rows = s.n_q < s.block ? s.n_q : s.block;
  const int pieces = (rows * d / 16 + kThreads - 1) / kThreads;
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
  };
  if (pieces <= 1) return run(append_kv_q8_kernel<1>);
  if (pieces <= 2) return run(append_kv_q8_kernel<2>);
  if (pieces <= 4) return run(append_kv_q8_kernel<4>);
  return run(append_kv_q8_kernel<8>);  // block 128, 128 dims: 1024 pieces
}

cudaError_t launch_read_kv_q8(const Shape& s, const Q8Cache& c, int64_t base, int64_t n,
                              uint16_t* k_out, uint16_t* v_out, uint16_t* ki_out, DeviceStatus* st,
                              cudaStream_t stream, float* block_scales) {
  Q8Args a = base_args(s, c, st);
  a.n = (int)n;
  a.k_out = k_out;
  a.v_out = v_out;
  a.ki_out = ki_out;
  a.base = base;
  a.block_scales = block_scales;
  a.group = s.block < 32 ? s.block : 32;
  a.per_seq = (int)((base + n - 1) / a.group - base / a.group + 1);
  const int64_t grid = (int64_t)s.batch * a.per_seq;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(block_scales == nullptr ? read_kv_q8_kernel<false> : read_kv_q8_kernel<true>,
                    dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
}

}  // namespace msa
