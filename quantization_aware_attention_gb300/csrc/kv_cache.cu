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
// Both kernels move every byte once: D / 16 lanes hold one row, so a warp covers 4 (D = 128) or 8
// (D = 64) rows, consecutive tokens of one head, which are consecutive in a page.  Lane j takes
// channels 8 j .. 8 j + 7 and the same of the row's second half, so that every load and store of a row
// is one run of whole sectors: 16 bytes a lane of bf16, 8 bytes of codes.  Keys and values of a row are
// handled by the same lanes, which keeps four loads in flight each.  HBM bounds both.  Measured, D = 128:
//   append  8 sequences' prompts of 1000 to 8192 tokens, 8 heads   36.3 us, 6.3 TB/s
//   read    6 sequences' prefixes of 9000 to 32768 tokens, 8 heads  158 us, 6.8 TB/s
//   append of one token to each of 64 sequences                     2.1 us: a launch and its chain of loads
// (Tiles of 8 tokens by 4 or 8 heads, which read a token's heads as one run, made append 5 percent slower.)
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
  page = p.table[static_cast<long long>(b) * p.max_pages + (pos >> p.page_shift)];
  slot = pos & ((1 << p.page_shift) - 1);
  if (page >= 0 && page < p.num_pages) return true;
  atomicOr(p.err, kErrBadPage);
  return false;
}

// A sequence's length as the table can hold it.
__device__ __forceinline__ int seq_len(const KvCacheArgs& p, int b) {
  const int len = p.seq_lens[b];
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  if (len <= cap) return max(len, 0);
  atomicOr(p.err, kErrBadPage);
  return static_cast<int>(cap);
}

// max(|a|, |b|) of two bf16 pairs up to the signs, NaN if either is.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The row's largest magnitude: it is a bf16 value itself, so it is taken on the bits.  A NaN stays one.
template <int L>
__device__ __forceinline__ float row_amax(const uint4 (&raw)[2]) {
  const uint32_t x[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  uint32_t mx = absmax_bf16x2(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) mx = absmax_bf16x2(mx, x[i]);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) mx = absmax_bf16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  return __uint_as_float((absmax_bf16x2(mx, mx >> 16) & 0x7fffu) << 16);
}

__device__ __forceinline__ uint2 quant8(const uint4& raw, float inv) {
  const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = mul_rn_f32x2(make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)),
                                  make_float2(inv, inv));
    c[i] = e4m3x2_rn_satfinite(y.x, y.y);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

template <int D>
__device__ __forceinline__ void store_codes(uint8_t* code, size_t row, int j, const uint4 (&raw)[2],
                                            float inv, bool bad) {
  const uint2 lo = quant8(raw[0], inv), hi = quant8(raw[1], inv), none = make_uint2(0u, 0u);
  uint2* dst = reinterpret_cast<uint2*>(code + row * D);
  dst[j] = bad ? none : lo;
  dst[j + D / 16] = bad ? none : hi;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8) kv_append_kernel(const KvCacheArgs p) {
  constexpr int L = D / 16;
  const int j = threadIdx.x % L;
  const unsigned row = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  after_previous();
  bool in = row < static_cast<unsigned long long>(p.B) * p.H * p.N;
  const unsigned bh = p.by_n(row);
  const int n = static_cast<int>(row - bh * p.N), b = static_cast<int>(p.by_h(bh));
  const int h = static_cast<int>(bh - static_cast<unsigned>(b) * p.H);
  uint4 rk[2], rv[2];
  rk[0] = rk[1] = rv[0] = rv[1] = make_uint4(0u, 0u, 0u, 0u);
  size_t at = 0;
  if (in) {
    const int count = p.new_lens != nullptr ? min(p.new_lens[b], p.N) : p.N;
    in = n < count;
    if (in) {
      const uint4* k = reinterpret_cast<const uint4*>(p.k + b * p.k_sb + h * p.k_sh + n * p.k_sn);
      const uint4* v = reinterpret_cast<const uint4*>(p.v + b * p.v_sb + h * p.v_sh + n * p.v_sn);
      rk[0] = k[j];
      rk[1] = k[L + j];
      rv[0] = v[j];
      rv[1] = v[L + j];
      // the count's tokens are the sequence's last
      const int len = p.seq_lens[b];
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
  const float ak = row_amax<L>(rk), av = row_amax<L>(rv);
  const bool bad_k = !(ak <= 3.4028234663852886e38f), bad_v = !(av <= 3.4028234663852886e38f);
  // the row's four divisions, 448 / amax and amax / 448 of K and V, one to a lane
  const float am = (j & 2) ? av : ak;
  const bool zero = !(am >= kTinyRow) || ((j & 2) ? bad_v : bad_k);
  const float q = zero ? 0.f : ((j & 1) ? __fdiv_rn(am, kE4M3Max) : __fdiv_rn(kE4M3Max, am));
  const int first = (threadIdx.x & 31) - j;
  const float inv_k = __shfl_sync(0xffffffffu, q, first), inv_v = __shfl_sync(0xffffffffu, q, first + 2);
  if (!in) return;
  store_codes<D>(p.k_codes, at, j, rk, inv_k, bad_k);
  store_codes<D>(p.v_codes, at, j, rv, inv_v, bad_v);
  const float nan = __int_as_float(0x7fc00000);
  if (j == 1) p.k_scales[at] = bad_k ? nan : q;
  if (j == 3) p.v_scales[at] = bad_v ? nan : q;
}

// Eight codes to bf16.
__device__ __forceinline__ uint4 dequant8(const uint2& c, float scale) {
  const uint16_t x[4] = {static_cast<uint16_t>(c.x), static_cast<uint16_t>(c.x >> 16),
                         static_cast<uint16_t>(c.y), static_cast<uint16_t>(c.y >> 16)};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = mul_rn_f32x2(e4m3x2_decode(x[i]), make_float2(scale, scale));
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvCacheArgs p) {
  constexpr int L = D / 16;
  const int j = threadIdx.x % L;
  const unsigned row = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  after_previous();
  if (row >= static_cast<unsigned long long>(p.B) * p.H * p.N) return;
  const unsigned bh = p.by_n(row);
  const int n = static_cast<int>(row - bh * p.N), b = static_cast<int>(p.by_h(bh));
  const int h = static_cast<int>(bh - static_cast<unsigned>(b) * p.H);
  const long long pos = static_cast<long long>(p.begin) + n;
  uint2 ck[2], cv[2];
  ck[0] = ck[1] = cv[0] = cv[1] = make_uint2(0u, 0u);
  float sk = 0.f, sv = 0.f;
  if (pos < seq_len(p, b)) {
    int page, slot;
    if (find_slot(p, b, static_cast<int>(pos), page, slot)) {
      const size_t at = ((static_cast<size_t>(page) * p.H + h) << p.page_shift) + slot;
      const uint2* k = reinterpret_cast<const uint2*>(p.k_codes + at * D) + j;
      const uint2* v = reinterpret_cast<const uint2*>(p.v_codes + at * D) + j;
      ck[0] = k[0];
      ck[1] = k[L];
      cv[0] = v[0];
      cv[1] = v[L];
      sk = p.k_scales[at];
      sv = p.v_scales[at];
    } else {
      sk = sv = __int_as_float(0x7fc00000);  // no page: the row reads as NaN
    }
  }
  uint4* ko = reinterpret_cast<uint4*>(p.k_out + static_cast<size_t>(row) * D) + j;
  uint4* vo = reinterpret_cast<uint4*>(p.v_out + static_cast<size_t>(row) * D) + j;
  ko[0] = dequant8(ck[0], sk);
  ko[L] = dequant8(ck[1], sk);
  vo[0] = dequant8(cv[0], sv);
  vo[L] = dequant8(cv[1], sv);
}

inline unsigned blocks_of(const KvCacheArgs& a, int D) {
  const long long lanes = static_cast<long long>(a.B) * a.H * a.N * (D / 16);
  return static_cast<unsigned>((lanes + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_kv_append(const KvCacheArgs& a, int D, cudaStream_t s) {
  return launch_early(D == 64 ? kv_append_kernel<64> : kv_append_kernel<128>, blocks_of(a, D), kThreads, 0, s, a);
}

cudaError_t launch_kv_read(const KvCacheArgs& a, int D, cudaStream_t s) {
  return launch_early(D == 64 ? kv_read_kernel<64> : kv_read_kernel<128>, blocks_of(a, D), kThreads, 0, s, a);
}

}  // namespace qat
