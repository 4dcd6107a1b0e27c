// kv_cache.cu -- the FP8 key/value cache: quantizing new rows as they are written to their
// pages, and reading rows back as bf16.
//
// A row is one token of one head, D channels.  Its rule is the library's (qat_quant.cuh) with
// one scale per row: amax = max |x|, code = E4M3_RNE_SATFINITE(fl32(x fl32(448 / amax))),
// scale = fl32(amax / 448).  Two cases are put apart so that every stored code is finite, and a
// masked key can be multiplied by zero wherever it is read:
//   amax < 2^-110 (448 / amax nears the fp32 range's end)  ->  codes 0, scale 0
//   a NaN or an infinity in the row                        ->  codes 0, scale NaN (reads as NaN)
//
// Layout: codes [page][head][slot][D] bytes, scales [page][head][slot] fp32; position i of
// sequence b is slot i % page_size of page table[b][i / page_size].
//
// Both kernels move every byte once: D / 16 lanes hold one row, 16 channels each (32 bytes of
// bf16, 16 bytes of codes), so a warp covers 4 (D = 128) or 8 (D = 64) rows, consecutive tokens
// of one head, which are consecutive in a page.  Keys and values of a row are handled by the same
// lanes, which keeps four 16-byte loads in flight each.
#include "qat_internal.h"
#include "qat_quant.cuh"
#include "sm100.cuh"

#include <cuda_bf16.h>

namespace qat {
namespace {

constexpr int kThreads = 256;
constexpr float kTinyRow = 7.703719777548943e-34f;  // 2^-110

// The page of a position and its place in it; false when the table's entry lies outside the
// cache (reported in the device error word).
__device__ __forceinline__ bool find_slot(const KvCacheArgs& p, int b, int pos, int& page, int& slot) {
  page = __ldg(p.table + static_cast<long long>(b) * p.max_pages + (pos >> p.page_shift));
  slot = pos & ((1 << p.page_shift) - 1);
  if (page >= 0 && page < p.num_pages) return true;
  atomicOr(p.err, kErrBadPage);
  return false;
}

// A sequence's length as the table can hold it.
__device__ __forceinline__ int seq_len(const KvCacheArgs& p, int b) {
  const int len = __ldg(p.seq_lens + b);
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  if (len <= cap) return max(len, 0);
  atomicOr(p.err, kErrBadPage);
  return static_cast<int>(cap);
}

// max(|a|, |b|) of two bf16 pairs, NaN if either is.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
  return r;
}

// amax is the largest magnitude itself, so it is taken on the bf16 bits; a NaN stays one, and an
// infinity is one's own.
template <int D>
__device__ __forceinline__ void quant_store(const uint4 (&raw)[2], uint8_t* code, float* scale,
                                            size_t row, int j, bool in) {
  constexpr int L = D / 16;
  const uint32_t x[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  uint32_t mx = absmax_bf16x2(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) mx = absmax_bf16x2(mx, x[i]);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) mx = absmax_bf16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  mx = absmax_bf16x2(mx, mx >> 16);
  const float amax = __uint_as_float(mx << 16);
  const bool bad = !(amax <= 3.4028234663852886e38f);
  const TileScale ts = tile_scale(bad || amax < kTinyRow ? 0.f : amax);
  if (!in) return;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = x[2 * i], v = x[2 * i + 1];
    const float2 p = mul_rn_f32x2(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)),
                                  make_float2(ts.inv, ts.inv));
    const float2 q = mul_rn_f32x2(make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)),
                                  make_float2(ts.inv, ts.inv));
    w[i] = e4m3x2_rn_satfinite(p.x, p.y) | static_cast<uint32_t>(e4m3x2_rn_satfinite(q.x, q.y)) << 16;
  }
  *reinterpret_cast<uint4*>(code + row * D + 16 * j) =
      bad ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(w[0], w[1], w[2], w[3]);
  if (j == 0) scale[row] = bad ? __int_as_float(0x7fc00000) : ts.scale;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvCacheArgs p) {
  constexpr int L = D / 16;
  const int j = threadIdx.x % L;
  // at most 2^31 rows: 32-bit divisions
  const unsigned row = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  bool in = row < static_cast<unsigned long long>(p.B) * p.H * p.N;
  const unsigned bh = row / static_cast<unsigned>(p.N);
  const int n = static_cast<int>(row - bh * p.N), b = static_cast<int>(bh / static_cast<unsigned>(p.H));
  const int h = static_cast<int>(bh - static_cast<unsigned>(b) * p.H);
  uint4 rk[2], rv[2];
  rk[0] = rk[1] = rv[0] = rv[1] = make_uint4(0u, 0u, 0u, 0u);
  size_t at = 0;
  if (in) {
    const int count = p.new_lens != nullptr ? min(__ldg(p.new_lens + b), p.N) : p.N;
    in = n < count;
    if (in) {
      const uint4* k = reinterpret_cast<const uint4*>(p.k + b * p.k_sb + h * p.k_sh + n * p.k_sn);
      const uint4* v = reinterpret_cast<const uint4*>(p.v + b * p.v_sb + h * p.v_sh + n * p.v_sn);
      rk[0] = __ldg(k + 2 * j);
      rk[1] = __ldg(k + 2 * j + 1);
      rv[0] = __ldg(v + 2 * j);
      rv[1] = __ldg(v + 2 * j + 1);
      // the count's tokens are the sequence's last
      const int len = __ldg(p.seq_lens + b);
      const long long pos = static_cast<long long>(len) - count + n;
      const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
      if (pos < 0 || pos >= cap) {
        if (pos >= cap) atomicOr(p.err, kErrBadPage);
        in = false;
      } else {
        int page, slot;
        in = find_slot(p, b, static_cast<int>(pos), page, slot);
        at = ((static_cast<size_t>(page) * p.H + h) << p.page_shift) + slot;
      }
    }
  }
  if (!__any_sync(0xffffffffu, in)) return;  // padding
  quant_store<D>(rk, p.k_codes, p.k_scales, at, j, in);
  quant_store<D>(rv, p.v_codes, p.v_scales, at, j, in);
}

__device__ __forceinline__ void dequant_store(const uint4& codes, float scale, uint16_t* dst) {
  const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = mul_rn_f32x2(e4m3x2_decode(static_cast<uint16_t>(c[i])), make_float2(scale, scale));
    const float2 hi = mul_rn_f32x2(e4m3x2_decode(static_cast<uint16_t>(c[i] >> 16)), make_float2(scale, scale));
    const __nv_bfloat162 a = __floats2bfloat162_rn(lo.x, lo.y), b = __floats2bfloat162_rn(hi.x, hi.y);
    w[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
    w[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvCacheArgs p) {
  constexpr int L = D / 16;
  const int j = threadIdx.x % L;
  const unsigned row = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  if (row >= static_cast<unsigned long long>(p.B) * p.H * p.N) return;
  const unsigned bh = row / static_cast<unsigned>(p.N);
  const int n = static_cast<int>(row - bh * p.N), b = static_cast<int>(bh / static_cast<unsigned>(p.H));
  const int h = static_cast<int>(bh - static_cast<unsigned>(b) * p.H);
  const long long pos = static_cast<long long>(p.begin) + n;
  uint4 ck = make_uint4(0u, 0u, 0u, 0u), cv = ck;
  float sk = 0.f, sv = 0.f;
  if (pos < seq_len(p, b)) {
    int page, slot;
    if (find_slot(p, b, static_cast<int>(pos), page, slot)) {
      const size_t at = ((static_cast<size_t>(page) * p.H + h) << p.page_shift) + slot;
      ck = __ldg(reinterpret_cast<const uint4*>(p.k_codes + at * D) + j);
      cv = __ldg(reinterpret_cast<const uint4*>(p.v_codes + at * D) + j);
      sk = __ldg(p.k_scales + at);
      sv = __ldg(p.v_scales + at);
    } else {
      sk = sv = __int_as_float(0x7fc00000);  // no page: the row reads as NaN
    }
  }
  dequant_store(ck, sk, p.k_out + static_cast<size_t>(row) * D + 16 * j);
  dequant_store(cv, sv, p.v_out + static_cast<size_t>(row) * D + 16 * j);
}

inline unsigned blocks_of(const KvCacheArgs& a, int D) {
  const long long lanes = static_cast<long long>(a.B) * a.H * a.N * (D / 16);
  return static_cast<unsigned>((lanes + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_kv_append(const KvCacheArgs& a, int D, cudaStream_t s) {
  if (D == 64)
    kv_append_kernel<64><<<blocks_of(a, D), kThreads, 0, s>>>(a);
  else
    kv_append_kernel<128><<<blocks_of(a, D), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvCacheArgs& a, int D, cudaStream_t s) {
  if (D == 64)
    kv_read_kernel<64><<<blocks_of(a, D), kThreads, 0, s>>>(a);
  else
    kv_read_kernel<128><<<blocks_of(a, D), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace qat
