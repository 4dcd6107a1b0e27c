// attn_decode.cu -- attention of the last T tokens of each sequence over the FP8 key/value cache
// (serving), with P fake-quantized as in training.
//
// Per query row (head, token) and visible key j (j <= its own position):
//   s_j = sm_scale <q, k_j>,  k_j = code_j scale_j;  p_j = exp(s_j - m);  l = sum p_j
//   quantized: per absolute 64-key tile amax = max p, p'_j = E4M3(p_j 448 / amax) amax / 448
//   o = sum p'_j v_j / l;  lse = log2 sum exp(s_j).  A row that sees no key: o = 0, lse = -inf.
//
// What bounds it: the cache is read once, 2 (D + 4) bytes per key and KV head, and every byte
// meets at most 16 query rows, so HBM does.  The kernel is built around keeping loads in flight:
// every warp is its own worker with its own place for a tile's K and V, filled by cp.async, each again
// as soon as it is used (smaller pieces, more of them in flight, took 1 to 7 percent longer); no barrier
// between warps, and all G = Hq / Hkv heads that share a KV head (times T tokens) are rows of one item
// of 8 or 16 rows, so that the cache is read once for all of them (once for each 16 beyond that).
// Measured, 8 KV heads, quantized, in a captured graph:
//   D 128, 32 query heads, 1 token, 64 sequences of 129 to 8192 keys     95 us, 5.9 TB/s of codes and scales
//   D 128, 40 query heads, 1 token, 2 sequences of 250001 and 262144    169 us, 6.4 TB/s
//   D 64,  32 query heads, 3 tokens, 64 sequences of 129 to 8192         65 us, 4.5 TB/s: issue and latency
//                                                                        (its 168 registers spill 4 bytes,
//                                                                        56 where P is not quantized)
//   D 128, 32 query heads, 1 token, one sequence of 1537 keys           9.4 us: two launches and their chains
//                                                                        of loads (prefix sums 1.1 us, table
//                                                                        and first copies 2.3, data 2 to 4,
//                                                                        end to merge 1, merge 2.5 to 4)
// What is left of the first is that the SMs differ by 15 percent in bandwidth: equal ranges end 10 us
// apart.  (Ranges handed out in pieces end together, but every piece cuts an item, and adding the
// partials took what that gained.)
//
// Work split (stream-K).  The batch's units -- 64-key tiles, ordered by sequence, KV head, row tile,
// key, and one more at the head of every (sequence, head, row tile) item for what an item costs beside its
// tiles -- are cut into equal contiguous ranges, one per warp, whatever the sequences' lengths.  (Without
// the item's unit, warps that got many short sequences ended last: 64 sequences of 129 to 8192 keys, 3
// tokens, 64 channels, 104 against 87 us.)  An item inside one range is finished there; an item cut by a
// range boundary leaves unnormalized fp32 partials with their m and l in the workspace, which
// the merge kernels add in an order that the sizes, the table's width and the lengths decide (no atomics: the
// same ones give the same bits; the width bounds the lengths on the host, which chooses the merge by it).
//
// Products: mma.sync m16n8k16 with f16 operands and fp32 sums, the cache as the 16-row operand and
// the query rows as the 8 columns (one column tile for up to 8 rows, else two): S^T = K Q^T and
// O^T = V^T P^T.  E4M3 codes are exact in f16, and become f16 in registers (one conversion per two
// codes), so the scale of a key multiplies its row of S^T, and the scale of a value its row of P^T.
// q (bf16) is brought into f16 by a power of two per row, which is exact for every element above 2^-32
// of the row's largest.  The weights, P times the values' scales, are rounded to f16: by 2^-11 of
// themselves, as each row's are multiplied by a power of two that follows its largest weight so far
// (to about 2^14; what is below 2^-28 of the row's largest is off by 2^-39 of it).  Following each row's weights
// costs nothing where HBM bounds and 1 to 2 percent where issue does, against one bound for all scales of a
// tile, which lost the weights of rows that do not see, or hardly weigh, a value 2^28 times as large.
// With so few rows these products need a tenth of the tensor rate, and a 128-row tcgen05 tile would want the
// codes of V transposed and P in 8 bits with a scale per key; the memory pipeline is what has to be fed.
//
// Operand layout: the order of d in Q K^T and of the output rows in V^T P^T is free, so each lane
// (g = lane / 4, t = lane % 4) takes 16-byte runs of a row: for K chunk t + 4 h of keys g and g + 8
// (k-step s of the run: bytes 4 s .. 4 s + 3), for V the g-th eighth of keys 2t, 2t + 1, 2t + 8, 2t + 9,
// whose bytes are interleaved by key with prmt.  Chunks are XOR-swizzled by row so that these reads are
// free of bank conflicts.  P^T leaves the softmax with a key per lane and becomes the product's operand
// by movmatrix.
#include "qat_internal.h"
#include "qat_quant.cuh"
#include "sm100.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

namespace qat {
namespace {

constexpr int kTile = 64;    // keys per unit
constexpr int kChunk = 16;   // keys that certainly share a page
constexpr int kRows = 16;    // query rows per item at most
constexpr int kMaxCtas = 152;
constexpr int kMaxWarps = 16;
constexpr int kWorkers = kMaxCtas * kMaxWarps;
constexpr float kTinyP = 7.888609052210118e-31f;  // 2^-100: a tile below it counts as zero (448 / amax
                                                  // must stay finite)
constexpr float kPTop = 16384.f;  // the largest weight as an f16 operand
constexpr uint32_t kPTopAt = (127u + 127u + 14u) << 23;  // minus a power of two's bits: those of kPTop over it
constexpr uint32_t kNoPage = 0xffffffffu, kBadPage = 0xfffffffeu;

// NR: column tiles of 8 query rows per item, 1 or 2.  One tile needs half the registers, which
// makes room for more warps (64 ragged sequences, D = 128: 16 warps take 4 percent longer than 12; 16 rows of
// 128 channels with 12 warps and the query rows in shared memory 11 percent longer than 8).
constexpr int warps_of(int D, int NR) { return NR == 1 ? (D == 128 ? 12 : 16) : (D == 128 ? 8 : 12); }

template <int D, int NR>
struct Cfg {
  static constexpr int kWarps = warps_of(D, NR);
  static constexpr int kVAt = kTile * D + 8 * kTile;  // a ring: K codes, the scales of K and V; V codes
  static constexpr int kRing = kVAt + kTile * D;
  static constexpr int kSmem = kWarps * kRing;  // then the warps' sums and B + 1 prefix sums
};

// Workspace: the header, the chains, then the partials: two per worker, [0] of the item its range ends or
// passes through ("head"), [1] of the item it begins and does not end ("tail"), each rows x D sums and
// rows x (m, l).  An item that ranges cut leaves a chain of partials: the tail of the worker in whose range
// it begins, then the heads of the following workers.  Chains are listed by item where there are at most as
// many items as workers (Params::by_item), else by the worker they begin with.
struct Header {
  int workers;
  int pad[31];
};
struct Chain {
  int key;   // by item: the first worker; by worker: the item; -1: none
  int last;  // the worker in whose range the item ends
};
constexpr size_t kPartsAt = sizeof(Header) + kWorkers * sizeof(Chain);
static_assert(kPartsAt % 16 == 0, "partials are read 16 bytes at a time");

struct Params {
  DecodeArgs a;
  int R, rows, mtiles;  // rows of a KV head (Hq / Hkv heads x T tokens), of an item; items of a head
  int prows;            // rows of a partial
  int by_item;
};

__device__ __forceinline__ Header* header_of(const Params& p) { return static_cast<Header*>(p.a.ws); }
__device__ __forceinline__ Chain* chains_of(const Params& p) {
  return reinterpret_cast<Chain*>(static_cast<char*>(p.a.ws) + sizeof(Header));
}
template <int D>
__device__ __forceinline__ float* partial_of(const Params& p, int worker, int which) {
  return reinterpret_cast<float*>(static_cast<char*>(p.a.ws) + kPartsAt) +
         (static_cast<size_t>(worker) * 2 + which) * p.prows * (D + 2);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t codes_to_f16x2(uint16_t c) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
  return h2;
}

// Transposes an 8 x 8 matrix of 16-bit elements, row g's elements 2t and 2t + 1 in lane 4 g + t.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes into shared memory; with `bytes`, that many from global memory and zeros behind them.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// Byte offset of 16-byte chunk c of row r in 16 rows of K or V codes.
template <int D>
__device__ __forceinline__ uint32_t k_off(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ ((r & 1) << 2)) << 4) : r * 64 + (c << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_off(int r, int c) {
  if (D == 128) return r * 128 + ((c ^ (r & 6)) << 4);
  return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1)) << 4);
}

// A place in the batch's list of units.
struct Cursor {
  int b, h, mt, tile, tiles, len;
};

__device__ __forceinline__ int clamp_len(const DecodeArgs& a, int len) {
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  return len > cap ? static_cast<int>(cap) : max(len, 0);
}
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kTile - 1) / kTile : 1; }

// Tiles as the prefix sums have them: the cut and every index hold together even if a length changes
// under the kernel.
__device__ __forceinline__ void enter_seq(const Params& p, const int* prefix, Cursor& c) {
  if (c.b >= p.a.B) return;  // behind the last: not looked at again
  c.tiles = static_cast<unsigned>(prefix[c.b + 1] - prefix[c.b]) / static_cast<unsigned>(p.a.Hkv * p.mtiles);
  c.len = min(clamp_len(p.a, p.a.seq_lens[c.b]), c.tiles * kTile);
}

// The next tile; u: its unit.
__device__ __forceinline__ void advance(const Params& p, const int* prefix, int extra, Cursor& c, int& u) {
  ++u;
  if (++c.tile < c.tiles) return;
  u += extra;
  c.tile = 0;
  if (++c.mt < p.mtiles) return;
  c.mt = 0;
  if (++c.h < p.a.Hkv) return;
  c.h = 0;
  ++c.b;
  enter_seq(p, prefix, c);
}

__device__ __forceinline__ int item_of(const Params& p, const Cursor& c) {
  return (c.b * p.a.Hkv + c.h) * p.mtiles + c.mt;
}

// The item's query rows 8 n + g as f16 times a power of two (exact for all that matters), in the order
// of the K fragments; rf: what the scores of rows 8 n + 2t and 8 n + 2t + 1 are to be multiplied by, with the
// keys' scales times `less`.  Sums of 2^31 times a key's scale leave fp32 for keys above 2^105, so the scales
// are taken 2^-32 times and rf 2^32 times as large, unless a row's is above 2^64 (then scores of such keys do
// not fit fp32 themselves).  What that rounds of the least scales is below 2^-20 of a score.
template <int D, int NR>
__device__ __forceinline__ void load_rows(const Params& p, const Cursor& c, int g, int t,
                                          uint32_t (&qb)[NR][D / 16][2], float2 (&rf)[NR], float& less) {
  int ex[NR];
  bool far = false;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = c.mt * p.rows + g + 8 * n;
    uint4 raw[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < p.R) {
      const uint4* src = reinterpret_cast<const uint4*>(
          p.a.q + ((static_cast<size_t>(c.b) * p.a.Hkv + c.h) * p.R + r) * D);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        raw[2 * h] = src[8 * h + 2 * t];
        raw[2 * h + 1] = src[8 * h + 2 * t + 1];
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&raw[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __bfloat1622float2(b[k]);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // amax in [2^e, 2^(e+1)) goes to [2^14, 2^15)
    int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
    e = min(max(e, -100), 126);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
    ex[n] = e - 14;
    far |= !(ldexpf(p.a.qk_scale, ex[n]) < 18446744073709551616.f);
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&raw[2 * h + i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = __bfloat1622float2(b[k]);
          qb[n][4 * h + 2 * i + (k >> 1)][k & 1] = f16x2(f.x * up, f.y * up);
        }
      }
    }
  }
  far = __any_sync(0xffffffffu, far);
  less = far ? 1.f : 2.3283064365386963e-10f;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const float down = fmaxf(ldexpf(p.a.qk_scale, ex[n] + (far ? 0 : 32)),
                             1.1754943508222875e-38f);  // not zero: it multiplies -inf
    rf[n] = make_float2(__shfl_sync(0xffffffffu, down, 8 * t), __shfl_sync(0xffffffffu, down, 8 * t + 4));
  }
}

template <int MT>
__device__ __forceinline__ void scale_rows(float (&o)[MT][4], float2 f) {
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const float2 a = mul_rn_f32x2(make_float2(o[j][0], o[j][1]), f);
    const float2 b = mul_rn_f32x2(make_float2(o[j][2], o[j][3]), f);
    o[j][0] = a.x; o[j][1] = a.y; o[j][2] = b.x; o[j][3] = b.y;
  }
}

// Over the lanes that share t.
__device__ __forceinline__ float max_over_g(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_over_g(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Two maxima of values >= 0 over the lanes that share t, to 8 bits (rounded towards zero).
__device__ __forceinline__ float2 max_over_g(float2 v) {
  uint32_t x = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, o);
    asm("max.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
  }
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// The bits of the power of two above x >= 0, of 2^-112 .. 2^126 (kPTop over it is a normal number).
__device__ __forceinline__ uint32_t pow2_above(float x) {
  return min(max((__float_as_uint(x) & 0x7f800000u) + 0x00800000u, 15u << 23), 253u << 23);
}
// a / b of two such powers, as far as fp32 reaches.
__device__ __forceinline__ float pow2_ratio(uint32_t a, uint32_t b) {
  const int r = static_cast<int>(a - b) + (127 << 23);
  return __uint_as_float(static_cast<uint32_t>(min(max(r, 1 << 23), 254 << 23)));
}

template <int D, int NR, bool kQuant>
__global__ void __launch_bounds__(32 * Cfg<D, NR>::kWarps, 1) decode_kernel(const Params p) {
  using C = Cfg<D, NR>;
  constexpr int kThreads = 32 * C::kWarps;
  // No static shared memory: it would shift the ring, and cp.async fetches a sector twice when two
  // 16-byte pieces of it do not go to one 32-byte aligned place (64 ragged sequences: 122 against 100 us).
  extern __shared__ __align__(1024) uint8_t smem[];
  int* warp_sum = reinterpret_cast<int*>(smem + C::kSmem);
  int* prefix = warp_sum + C::kWarps;
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  after_previous();

  // prefix[b] = units before sequence b
  const int per_seq = a.Hkv * p.mtiles;
  {
    const int chunk = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * chunk, a.B), b1 = min(b0 + chunk, a.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const int len = a.seq_lens[b];
      const int ok = clamp_len(a, len);
      if (len > ok) atomicOr(a.err, kErrBadPage);
      prefix[b] = tiles_of(ok) * per_seq;
      sum += prefix[b];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    for (int b = b0; b < b1; ++b) {
      const int units = prefix[b];
      prefix[b] = base;
      base += units;
    }
    if (tid == kThreads - 1) prefix[a.B] = base;
    __syncthreads();
  }
  const int tiles = prefix[a.B];
  // workers: as few warps of every CTA as keep the most tiles that one has
  const int ctas = static_cast<int>(gridDim.x);
  const int deep = (tiles + ctas * C::kWarps - 1) / (ctas * C::kWarps);
  const int per_cta = (tiles + ctas * deep - 1) / (ctas * deep);
  const int workers = min(tiles, per_cta * static_cast<int>(gridDim.x));
  if (blockIdx.x == 0 && tid == 0) header_of(p)->workers = workers;
  if (warp >= per_cta) return;
  const int id = blockIdx.x * per_cta + warp;
  if (id >= workers) return;
  // an item's own unit, where ranges are long enough that each holds a tile all the same
  const int extra = tiles / 4 >= workers ? 1 : 0;
  const int W = tiles + extra * a.B * per_seq;
  // u0 = floor(W id / workers), u1 the next one's, by 32-bit divisions: W = each workers + over
  const unsigned each = static_cast<unsigned>(W) / workers, over = W - each * workers;  // over id < kWorkers^2
  int u0 = each * id + over * id / workers;
  const int u1 = each * (id + 1) + over * (id + 1) / workers;

  Cursor cc;  // what is computed next
  {
    int lo = 0, hi = a.B;  // the last b whose units begin at u0 or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] + extra * mid * per_seq <= u0) lo = mid; else hi = mid;
    }
    cc.b = lo;
    enter_seq(p, prefix, cc);
    const int u = u0 - (prefix[lo] + extra * lo * per_seq);
    const int item = u / (cc.tiles + extra), in = u - item * (cc.tiles + extra);
    cc.tile = max(in - extra, 0);
    if (in < extra) ++u0;  // to the item's first tile
    cc.mt = item % p.mtiles;
    cc.h = item / p.mtiles;
  }
  Cursor pc = cc;  // what is loaded next
  int pu = u0;
  uint32_t rows_of = kNoPage;  // lane l: cache row where 16-key chunk 32 (tile / 8) + l begins
  bool all_good = false;       // no chunk of those lies on a bad page
  const uint32_t ring = sm100::smem_addr(smem) + warp * C::kRing;
  // The lane's part of every copy: bytes 16 lane.. of each 512-byte run, by their swizzled places.
  const uint32_t k_dst = k_off<D>(lane / (D / 16), lane % (D / 16));
  const uint32_t v_dst0 = v_off<D>(lane / (D / 16), lane % (D / 16));
  const uint32_t v_dst1 = v_off<D>(lane / (D / 16) + 512 / D, lane % (D / 16)) - 512;

  // Issues the copies of the next tile's K, with the scales of both, or V as one group; an empty group at the
  // end.
  auto produce = [&](auto which, bool fresh) {
    constexpr bool kV = decltype(which)::value;
    if (pu < u1) {
      if (!kV && (fresh || (pc.tile & 7) == 0)) {
        const int pos = ((pc.tile & ~7) * 4 + lane) * kChunk;
        rows_of = kNoPage;
        if (pos < pc.len) {
          const int page = a.table[static_cast<long long>(pc.b) * a.max_pages + (pos >> a.page_shift)];
          rows_of = kBadPage;
          if (page >= 0 && page < a.num_pages)
            rows_of = ((static_cast<uint32_t>(page) * a.Hkv + pc.h) << a.page_shift) +
                      (pos & ((1 << a.page_shift) - 1));
          else
            atomicOr(a.err, kErrBadPage);
        }
        all_good = !__any_sync(0xffffffffu, rows_of == kBadPage);
      }
      const uint8_t* codes = (kV ? a.v_codes : a.k_codes) + 16 * lane;
      const uint32_t dst = ring + (kV ? C::kVAt : 0);
      const int first = (pc.tile & 7) * (kTile / kChunk);
      const int left = pc.len - pc.tile * kTile;  // keys from the tile's first on
      // lanes 0-15: the scales of K, 16-31: of V, four keys each
      const float* scales = (lane & 16) ? a.v_scales : a.k_scales;
      const uint32_t sc_row = kV ? 0 : __shfl_sync(0xffffffffu, rows_of, first + ((lane & 15) >> 2));
      const uint32_t sc_dst = dst + kTile * D + 16 * lane;
      if (left >= kTile && all_good) {
#pragma unroll
        for (int c = 0; c < kTile / kChunk; ++c) {
          const uint8_t* src = codes + static_cast<size_t>(__shfl_sync(0xffffffffu, rows_of, first + c)) * D;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t off = kV ? ((i & 1) ? v_dst1 : v_dst0) : k_dst;
            cp_async16(dst + off + c * kChunk * D + i * 512, src + i * 512);
          }
        }
        if (!kV) cp_async16(sc_dst, scales + sc_row + 4 * (lane & 3));
      } else {  // zeros behind the end, and for bad pages zeros with scale NaN
#pragma unroll 1
        for (int c = 0; c < kTile / kChunk; ++c) {
          const uint32_t rc = __shfl_sync(0xffffffffu, rows_of, first + c);
          const int n = rc < kBadPage ? left - c * kChunk : 0;
          const uint8_t* src = codes + (rc < kBadPage ? static_cast<size_t>(rc) * D : 0);
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t off = kV ? ((i & 1) ? v_dst1 : v_dst0) : k_dst;
            const int r = lane / (D / 16) + i * (512 / D);
            cp_async16(dst + off + c * kChunk * D + i * 512, r < n ? src + i * 512 : codes, r < n ? 16 : 0);
          }
        }
        if (!kV) {
          if (sc_row == kBadPage) {
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(sc_dst), "r"(0x7fc00000u) : "memory");
          } else {
            const int n = sc_row == kNoPage ? 0 : min(max(left - 4 * (lane & 15), 0), 4);
            cp_async16(sc_dst, n > 0 ? scales + sc_row + 4 * (lane & 3) : scales, 4 * n);
          }
        }
      }
      if (kV) advance(p, prefix, extra, pc, pu);
    }
    cp_commit();
  };
  constexpr std::integral_constant<bool, false> kKeys{};
  constexpr std::integral_constant<bool, true> kValues{};
  produce(kKeys, true);
  produce(kValues, false);

  constexpr int KS = D / 16;   // k-steps of K Q^T
  constexpr int MT = D / 16;   // row tiles of V^T P^T; a lane's channels are (D / 8) g + 0 .. D / 8 - 1
  uint32_t qb[NR][KS][2];
  float o[NR][MT][4];
  float2 m[NR], l[NR], rf[NR];  // of rows 8 n + 2t and 8 n + 2t + 1
  float less = 1.f;
  int last[NR][2];              // the newest key each of those rows sees
  float2 bound[NR];             // the rows' largest weights so far, as m is
  bool begun = false;
  if (lane == 0 && !p.by_item) chains_of(p)[id] = Chain{-1, -1};
  int first_tile = cc.tile;    // of the current segment

  for (int u = u0; u < u1;) {
    if (!begun) {
      begun = true;
      first_tile = cc.tile;
      load_rows<D, NR>(p, cc, g, t, qb, rf, less);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        m[n] = make_float2(-INFINITY, -INFINITY);
        l[n] = bound[n] = make_float2(0.f, 0.f);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          last[n][y] = cc.len - a.T + (cc.mt * p.rows + 8 * n + 2 * t + y) % a.T;
#pragma unroll
        for (int j = 0; j < MT; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
      }
    }

    // S^T = K Q^T of 64 keys, times the keys' scales (and, below, the rows'): chunk c's values are
    // keys g and g + 8 of rows 2t, 2t + 1
    float s[NR][4][4];
    float vs[4][2];  // the values' scales of those keys
    cp_wait<1>();
    __syncwarp();
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t slot = ring + hf * (kTile / 2) * D;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          s[n][2 * hf + c][0] = s[n][2 * hf + c][1] = s[n][2 * hf + c][2] = s[n][2 * hf + c][3] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t w[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 x = lds128(slot + 8 * k * D + k_off<D>(g, t + 4 * h));
          w[k][0] = x.x; w[k][1] = x.y; w[k][2] = x.z; w[k][3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t ka[4] = {codes_to_f16x2(static_cast<uint16_t>(w[2 * c][i])),
                                    codes_to_f16x2(static_cast<uint16_t>(w[2 * c + 1][i])),
                                    codes_to_f16x2(static_cast<uint16_t>(w[2 * c][i] >> 16)),
                                    codes_to_f16x2(static_cast<uint16_t>(w[2 * c + 1][i] >> 16))};
#pragma unroll
            for (int n = 0; n < NR; ++n)
              mma16816(s[n][2 * hf + c], ka, qb[n][4 * h + i][0], qb[n][4 * h + i][1]);
          }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t at = ring + kTile * D + 4 * (32 * hf + 16 * c + 8 * y + g);
          const float ks = lds_f(at) * less;
          vs[2 * hf + c][y] = lds_f(at + 4 * kTile);
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            float* x = s[n][2 * hf + c] + 2 * y;
            const float2 z = mul_rn_f32x2(make_float2(x[0], x[1]), make_float2(ks, ks));
            x[0] = z.x;
            x[1] = z.y;
          }
        }
    }
    __syncwarp();
    produce(kKeys, false);

    // mask: only tiles that reach past what some row sees
    const int key0 = cc.tile * kTile + g;
    const bool edge = (cc.tile + 1) * kTile > cc.len - a.T + 1;
    if (edge) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 16 * c + 8 * (i >> 1) > last[n][i & 1]) s[n][c][i] = -INFINITY;
    }

    float amax[NR][2];  // the tile's largest p of the lane's rows
    float2 alpha[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float2 mt = make_float2(s[n][0][0], s[n][0][1]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mt.x = fmaxf(mt.x, fmaxf(s[n][c][0], s[n][c][2]));
        mt.y = fmaxf(mt.y, fmaxf(s[n][c][1], s[n][c][3]));
      }
      mt.x = max_over_g(mt.x);
      mt.y = max_over_g(mt.y);
      const float2 mn = make_float2(fmaxf(m[n].x, mt.x * rf[n].x), fmaxf(m[n].y, mt.y * rf[n].y));
      const float2 neg = make_float2(mn.x == -INFINITY ? 0.f : -mn.x, mn.y == -INFINITY ? 0.f : -mn.y);
      alpha[n] = make_float2(ex2(m[n].x + neg.x), ex2(m[n].y + neg.y));
      m[n] = mn;
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float* x = s[n][c] + 2 * y;
          const float2 e = fma_rn_f32x2(make_float2(x[0], x[1]), rf[n], neg);
          x[0] = ex2(e.x);
          x[1] = ex2(e.y);
          sum = add_rn_f32x2(sum, make_float2(x[0], x[1]));
        }
      l[n] = fma_rn_f32x2(l[n], alpha[n], sum);
      if (kQuant) {  // that of the largest score
        const float2 e = fma_rn_f32x2(mt, rf[n], neg);
        amax[n][0] = ex2(e.x);
        amax[n][1] = ex2(e.y);
      }
    }
    // The rows' scales, 448 / amax and amax / 448: the lanes that share t hold the same rows, so each does
    // one of the divisions (g = 4 n + 2 y + which) and the results go round.
    float quot = 0.f;
    if (kQuant) {
      float x = (g & 2) ? amax[0][1] : amax[0][0];
      if (NR == 2 && (g & 4)) x = (g & 2) ? amax[NR - 1][1] : amax[NR - 1][0];
      if (!(x < kTinyP)) quot = __fdiv_rn((g & 1) ? x : kE4M3Max, (g & 1) ? kE4M3Max : x);
    }
    // The weights, P times the values' scales, and as f16 operands: each row's are multiplied by a power of two
    // that takes the largest so far to 2^13 .. 2^14, and its sums with them.  A weight that the row does not see,
    // or that is nothing beside the others, counts for nothing there, whatever the value's scale.
    uint32_t pb[NR][4][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float2 inv, back;
      if (kQuant) {
        inv.x = __shfl_sync(0xffffffffu, quot, 16 * n + t);
        back.x = __shfl_sync(0xffffffffu, quot, 16 * n + 4 + t);
        inv.y = __shfl_sync(0xffffffffu, quot, 16 * n + 8 + t);
        back.y = __shfl_sync(0xffffffffu, quot, 16 * n + 12 + t);
      }
      float2 top = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float* x = s[n][c] + 2 * y;
          float2 w = make_float2(x[0], x[1]);
          if (kQuant) {
            const float2 q = mul_rn_f32x2(w, inv);
            w = mul_rn_f32x2(e4m3x2_decode(e4m3x2_rn_satfinite(q.x, q.y)), back);
          }
          w = mul_rn_f32x2(w, make_float2(vs[c][y], vs[c][y]));
          if (edge) {  // 0 x NaN: a key that the row does not see may hold anything
            if (key0 + 16 * c + 8 * y > last[n][0]) w.x = 0.f;
            if (key0 + 16 * c + 8 * y > last[n][1]) w.y = 0.f;
          }
          x[0] = w.x;
          x[1] = w.y;
          top.x = fmaxf(top.x, w.x);
          top.y = fmaxf(top.y, w.y);
        }
      top = max_over_g(top);
      const float2 old = bound[n];
      bound[n] = make_float2(fmaxf(old.x * alpha[n].x, top.x), fmaxf(old.y * alpha[n].y, top.y));
      const uint32_t ex = pow2_above(bound[n].x), ey = pow2_above(bound[n].y);
      const float2 f = make_float2(alpha[n].x * pow2_ratio(pow2_above(old.x), ex),
                                   alpha[n].y * pow2_ratio(pow2_above(old.y), ey));
      if (__any_sync(0xffffffffu, f.x != 1.f || f.y != 1.f)) scale_rows<MT>(o[n], f);
      const float2 unit = make_float2(__uint_as_float(kPTopAt - ex), __uint_as_float(kPTopAt - ey));
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float2 w = mul_rn_f32x2(make_float2(s[n][c][2 * y], s[n][c][2 * y + 1]), unit);
          pb[n][c][y] = transpose8x8(f16x2(w.x, w.y));
        }
    }

    // O^T += V^T P^T
    cp_wait<1>();
    __syncwarp();
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t slot = ring + C::kVAt + hf * (kTile / 2) * D;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t base = slot + c * kChunk * D;
        constexpr int W = D / 32;  // words of a lane's run of a row
        uint32_t w[4][W];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * t + (i & 1) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 v = lds128(base + v_off<D>(r, g));
            w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
          } else {
            const uint2 v = lds64(base + v_off<D>(r, g >> 1) + ((g & 1) << 3));
            w[i][0] = v.x; w[i][1] = v.y;
          }
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // bytes of two keys interleaved, two channels
            const uint32_t x = __byte_perm(w[0][i], w[1][i], z ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(w[2][i], w[3][i], z ? 0x7362 : 0x5140);
            const uint32_t va[4] = {codes_to_f16x2(static_cast<uint16_t>(x)),
                                    codes_to_f16x2(static_cast<uint16_t>(x >> 16)),
                                    codes_to_f16x2(static_cast<uint16_t>(y)),
                                    codes_to_f16x2(static_cast<uint16_t>(y >> 16))};
#pragma unroll
            for (int n = 0; n < NR; ++n)
              mma16816(o[n][2 * i + z], va, pb[n][2 * hf + c][0], pb[n][2 * hf + c][1]);
          }
      }
    }
    __syncwarp();
    produce(kValues, false);

    const bool ends = cc.tile + 1 == cc.tiles;
    if (ends || u + 1 >= u1) {  // the segment's end
      begun = false;
      const bool head = first_tile != 0;
      const bool whole = !head && ends;
      if (!head && lane == 0) {
        const long long end = u - cc.tile + cc.tiles;  // the unit behind the item
        const int item = item_of(p, cc);
        if (whole) {
          if (p.by_item) chains_of(p)[item] = Chain{-1, -1};
        } else {
          chains_of(p)[p.by_item ? item : id] = Chain{p.by_item ? id : item, static_cast<int>((end * workers - 1) / W)};
        }
      }
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        l[n].x = sum_over_g(l[n].x);
        l[n].y = sum_over_g(l[n].y);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = 8 * n + 2 * t + y;
          if (cc.mt * p.rows + r >= p.R) continue;
          const float lr = y ? l[n].y : l[n].x, mr = y ? m[n].y : m[n].x;
          const float scale = __uint_as_float(pow2_above(y ? bound[n].y : bound[n].x)) * (1.f / kPTop);
          if (whole) {  // the item's output
            const size_t row = (static_cast<size_t>(cc.b) * a.Hkv + cc.h) * p.R + cc.mt * p.rows + r;
            const bool none = lr == 0.f;
            const float f = none ? 0.f : scale / lr;
            uint32_t w[MT];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(none ? 0.f : o[n][j][y] * f,
                                                             none ? 0.f : o[n][j][2 + y] * f);
              w[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
            uint4* dst = reinterpret_cast<uint4*>(a.o + row * D + D / 8 * g);
#pragma unroll
            for (int j = 0; j < MT / 4; ++j)
              dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            if (g == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : mr + log2f(lr);
          } else {
            float* part = partial_of<D>(p, id, head ? 0 : 1);
            if (g == 0) *reinterpret_cast<float2*>(part + p.prows * D + 2 * r) = make_float2(mr, lr);
#pragma unroll
            for (int j = 0; j < MT / 2; ++j)
              *reinterpret_cast<float4*>(part + r * D + D / 8 * g + 4 * j) =
                  make_float4(o[n][2 * j][y] * scale, o[n][2 * j][2 + y] * scale,
                              o[n][2 * j + 1][y] * scale, o[n][2 * j + 1][2 + y] * scale);
          }
        }
      }
    }
    advance(p, prefix, extra, cc, u);
  }
  cp_wait<0>();
}

// A row of partials being added up: V channels per lane, and the row's m and l.
template <int V>
struct Sum {
  float m, l, acc[V];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
  }
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float (&x)[N][V]) {
    float top = m;
#pragma unroll
    for (int k = 0; k < N; ++k) top = fmaxf(top, ml[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = ex2(m - ref);
    m = top;
    l *= f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float fk = ex2(ml[k].x - ref);
      l = fmaf(ml[k].y, fk, l);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(x[k][i], fk, acc[i]);
    }
  }
};

template <int V>
__device__ __forceinline__ void load_v(float (&x)[V], const float* src) {
  if constexpr (V == 4) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
  } else {
    const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
    x[0] = t.x; x[1] = t.y;
  }
}

// Row r of worker w's partial `which`.
template <int D>
__device__ __forceinline__ void load_partial(const Params& p, int w, int which, int r, int lane, float2& ml,
                                             float (&x)[D / 32]) {
  const float* part = partial_of<D>(p, w, which);
  ml = __ldcg(reinterpret_cast<const float2*>(part + p.prows * D + 2 * r));
  load_v<D / 32>(x, part + r * D + D / 32 * lane);
}

// Adds partials first, first + step, ... up to n of the chain that begins with worker w's tail, kAhead
// loads in flight: none is conditional (behind the end the last one is loaded again and counts as nothing),
// or each would be waited for before the next.
template <int D, int kAhead>
__device__ __forceinline__ void add_chain(const Params& p, int w, int first, int step, int n, int r,
                                          int lane, Sum<D / 32>& sum) {
  for (int i = first; i < n; i += kAhead * step) {
    float x[kAhead][D / 32];
    float2 ml[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int c = min(i + k * step, n - 1);
      load_partial<D>(p, w + c, c == 0 ? 1 : 0, r, lane, ml[k], x[k]);
    }
#pragma unroll
    for (int k = 1; k < kAhead; ++k) {
      if (i + k * step < n) continue;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x[k][j] = 0.f;
    }
    sum.add(ml, x);
  }
}

template <int D>
__device__ __forceinline__ void store_row(const Params& p, int item, int r, int lane,
                                          const Sum<D / 32>& s) {
  constexpr int V = D / 32;
  const size_t row = static_cast<size_t>(item / p.mtiles) * p.R + item % p.mtiles * p.rows + r;
  const bool none = s.l == 0.f;
  const float f = none ? 0.f : 1.f / s.l;
  uint32_t out[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(none ? 0.f : s.acc[2 * i] * f,
                                                   none ? 0.f : s.acc[2 * i + 1] * f);
    out[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint16_t* dst = p.a.o + row * D + V * lane;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = out[0];
  if (lane == 0 && p.a.lse != nullptr) p.a.lse[row] = none ? -INFINITY : s.m + log2f(s.l);
}

// A value into the same shared memory variable of the cluster's first block.
__device__ __forceinline__ void store_first(float* dst, float x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(sm100::smem_addr(dst)));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}

// The kN sums in acc and ml as one: lane x weighs the x-th, then every lane adds its channels of all.
template <int D, int kN>
__device__ __forceinline__ void add_all(const float (*acc)[D], const float (*ml)[2], int lane, Sum<D / 32>& sum) {
  constexpr int V = D / 32;
  const float m = lane < kN ? ml[lane][0] : -INFINITY;
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float f = lane < kN ? ex2(m - (top == -INFINITY ? 0.f : top)) : 0.f;
  float l = lane < kN ? ml[lane][1] * f : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  sum.m = top;
  sum.l = l;
#pragma unroll
  for (int i = 0; i < V; ++i) sum.acc[i] = 0.f;
#pragma unroll
  for (int y = 0; y < kN; ++y) {
    const float fy = __shfl_sync(0xffffffffu, f, y);
#pragma unroll
    for (int i = 0; i < V; ++i) sum.acc[i] = fmaf(acc[y][V * lane + i], fy, sum.acc[i]);
  }
}

// Adds up row r = blockIdx.y of 8 chains, a warp for each; all 8 warps for one after the other where few of
// the block's are long.
constexpr int kEachWarps = 8, kEachAhead = 8;
constexpr int kMergeCtas = 8;  // blocks of a cluster at most

// Row r of the chain at place x of the list: its first worker, length (0: none) and item.
__device__ __forceinline__ void find_chain(const Params& p, int x, int r, int& w, int& n, int& item) {
  const int workers = __ldcg(&header_of(p)->workers);
  w = n = item = 0;
  const int items = p.a.B * p.a.Hkv * p.mtiles;
  if (x >= (p.by_item ? items : kWorkers)) return;
  const int2 raw = __ldcg(reinterpret_cast<const int2*>(chains_of(p) + x));
  item = p.by_item ? x : raw.x;
  w = p.by_item ? raw.x : x;
  // (bounds: an entry beyond the workers' count means nothing, and none may lead outside the workspace)
  if (raw.x >= 0 && item < items && w < workers && raw.y > w && raw.y < workers &&
      item % p.mtiles * p.rows + r < p.R)
    n = raw.y - w + 1;
}

// A chain's partials by all the block's warps, into sum of warp 0.
template <int D, int kWarps, int kAhead>
__device__ __forceinline__ void add_by_block(const Params& p, int w, int first, int step, int n, int r, int warp,
                                             int lane, float (*acc)[D], float (*ml)[2], Sum<D / 32>& sum) {
  sum.clear();
  add_chain<D, kAhead>(p, w, first, step, n, r, lane, sum);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[warp][D / 32 * lane + i] = sum.acc[i];
  if (lane == 0) {
    ml[warp][0] = sum.m;
    ml[warp][1] = sum.l;
  }
  __syncthreads();
  if (warp == 0) add_all<D, kWarps>(acc, ml, lane, sum);
}

template <int D>
__global__ void __launch_bounds__(32 * kEachWarps) merge_each_kernel(const Params p) {
  __shared__ float acc[kEachWarps][D], ml[kEachWarps][2];
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_previous();  // the partials are complete
  int w, n, item;    // lane k: the block's k-th chain
  find_chain(p, blockIdx.x * kEachWarps + min(lane, kEachWarps - 1), r, w, n, item);
  if (lane >= kEachWarps) n = 0;
  // A round of loads takes 1 us, and a chain that all warps share 2 us: a warp takes up to two rounds, and
  // one more for every chain of the block beyond that.
  const int most = kEachAhead * (2 + __popc(__ballot_sync(0xffffffffu, n > 2 * kEachAhead)));
  const int len = __shfl_sync(0xffffffffu, n, warp);
  const int first = __shfl_sync(0xffffffffu, w, warp), it = __shfl_sync(0xffffffffu, item, warp);
  Sum<D / 32> sum;
  if (len > 0 && len <= most) {
    sum.clear();
    add_chain<D, kEachAhead>(p, first, 0, 1, len, r, lane, sum);
    store_row<D>(p, it, r, lane, sum);
  }
  unsigned rest = __ballot_sync(0xffffffffu, n > most);  // the same in every warp
  while (rest != 0) {
    const int k = __ffs(rest) - 1;
    rest &= rest - 1;
    add_by_block<D, kEachWarps, kEachAhead>(p, __shfl_sync(0xffffffffu, w, k), warp, kEachWarps,
                                            __shfl_sync(0xffffffffu, n, k), r, warp, lane, acc, ml, sum);
    if (warp == 0) store_row<D>(p, __shfl_sync(0xffffffffu, item, k), r, lane, sum);
    __syncthreads();
  }
}

// Adds up row r = blockIdx.y of one chain: by a block, or by a cluster of `ctas` blocks whose sums the first
// adds up in its shared memory.
template <int D, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps) merge_long_kernel(const Params p, int ctas) {
  constexpr int V = D / 32;
  __shared__ float acc[kWarps][D], ml[kWarps][2], all_acc[kMergeCtas][D], all_ml[kMergeCtas][2];
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = blockIdx.x / static_cast<unsigned>(ctas), rank = blockIdx.x - x * ctas;
  if (ctas > 1) {  // the cluster's blocks have all started before one writes to another
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
  after_previous();  // the partials are complete
  int w, n, item;
  find_chain(p, x, r, w, n, item);
  if (n == 0) return;  // in every block of the cluster
  Sum<V> sum;
  add_by_block<D, kWarps, 64 / kWarps>(p, w, rank * kWarps + warp, kWarps * ctas, n, r, warp, lane, acc, ml, sum);
  if (ctas > 1) {
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) store_first(&all_acc[rank][V * lane + i], sum.acc[i]);
      if (lane == 0) {
        store_first(&all_ml[rank][0], sum.m);
        store_first(&all_ml[rank][1], sum.l);
      }
      __syncwarp();
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    if (warp == 0) {
      for (int k = ctas; k < kMergeCtas; ++k) {  // blocks that are not there
        if (lane == 0) {
          all_ml[k][0] = -INFINITY;
          all_ml[k][1] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) all_acc[k][V * lane + i] = 0.f;
      }
      __syncwarp();
      add_all<D, kMergeCtas>(all_acc, all_ml, lane, sum);
    }
  }
  if (warp == 0) store_row<D>(p, item, r, lane, sum);
}

template <int D, int NR, bool kQuant>
cudaError_t run(Params p, int ctas, long long units, cudaStream_t s) {
  using C = Cfg<D, NR>;
  const auto bytes = [](int B) { return C::kSmem + sizeof(int) * (C::kWarps + B + 1); };
  const int most = static_cast<int>(units < ctas * C::kWarps ? units : ctas * C::kWarps);  // workers
  const long long items = static_cast<long long>(p.a.B) * p.a.Hkv * p.mtiles;
  p.by_item = items <= most;
  // The limit is that of the largest batch in every call: it is the kernel's, and another thread's call may
  // come between this one's limit and its launch.
  static_assert(bytes(kDecodeMaxBatch) <= 227 * 1024, "the batch's prefix sums fit beside the rings");
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, NR, kQuant>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(bytes(kDecodeMaxBatch)));
  if (e != cudaSuccess) return e;
  e = launch_early(decode_kernel<D, NR, kQuant>, ctas, 32 * C::kWarps, bytes(p.a.B), s, p);
  if (e != cudaSuccess) return e;
  // How many warps add up a chain depends on the partials that an item leaves on average.  Where all chains
  // fit the GPU at two blocks of 16 warps an SM, more blocks share a chain while each has 128 partials.
  const int chains = p.by_item ? static_cast<int>(items) : most, rows = p.R < p.rows ? p.R : p.rows;
  if (items * 16 > most)
    return launch_early(merge_each_kernel<D>, dim3((chains + kEachWarps - 1) / kEachWarps, rows), 32 * kEachWarps, 0,
                        s, p);
  const int room = 2 * ctas;
  if (chains * rows > room) return launch_early(merge_long_kernel<D, 8>, dim3(chains, rows), 256, 0, s, p, 1);
  int n = 1;
  while (n < kMergeCtas && chains * rows * 2 * n <= room && items * 128 * n < most) n *= 2;
  return launch_cluster(n, merge_long_kernel<D, 16>, dim3(chains * n, rows), 512, 0, s, p, n);
}

}  // namespace

namespace {
// Rows of a partial, even so that partials stay 16-byte aligned.
int partial_rows(int R) { return R >= kRows ? kRows : (R + 1) / 2 * 2; }
}  // namespace

size_t decode_workspace_bytes(int R, int D) {
  return kPartsAt + static_cast<size_t>(kMaxCtas) * warps_of(D, R <= 8 ? 1 : 2) * 2 * partial_rows(R) * (D + 2) *
                         sizeof(float);
}

cudaError_t launch_decode(const DecodeArgs& a, int D, int num_sms, cudaStream_t s) {
  Params p;
  p.a = a;
  p.R = a.Hq / a.Hkv * a.T;
  p.rows = p.R <= 8 ? 8 : kRows;
  p.mtiles = (p.R + p.rows - 1) / p.rows;
  p.prows = partial_rows(p.R);
  // one CTA per SM, fewer when the table cannot hold a unit for each
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  const long long units = static_cast<long long>(a.B) * a.Hkv * p.mtiles * ((cap + kTile - 1) / kTile);  // >= 1
  int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  if (units < ctas) ctas = static_cast<int>(units);
  if (p.rows == 8) {
    if (D == 64) return a.quant ? run<64, 1, true>(p, ctas, units, s) : run<64, 1, false>(p, ctas, units, s);
    return a.quant ? run<128, 1, true>(p, ctas, units, s) : run<128, 1, false>(p, ctas, units, s);
  }
  if (D == 64) return a.quant ? run<64, 2, true>(p, ctas, units, s) : run<64, 2, false>(p, ctas, units, s);
  return a.quant ? run<128, 2, true>(p, ctas, units, s) : run<128, 2, false>(p, ctas, units, s);
}

}  // namespace qat
