// attn_tree_sm100.cu -- attention of a drafted tree over the FP8 cache where a KV head has many query rows, on the
// Blackwell tensor core: tcgen05 products with the queries as the 128-row operand.  (Fewer rows: attn_decode.cu,
// whose launch_decode has the rule and both sides' times.)
//
// Per query row (head, token) and key j that it sees:
//   s_j = sm_scale <q, k_j>,  k_j = code_j scale_j;  p_j = exp(s_j - m);  l = sum p_j
//   quantized: per absolute 64-key tile amax = max p, p'_j = E4M3(p_j 448 / amax) amax / 448
//   o = sum p'_j v_j / l;  lse = log2 sum exp(s_j).  A row that sees no key: o = 0, lse = -inf.
//
// What bounds it.  A key and KV head is 2 (D + 4) bytes and 4 D flops for each of up to 128 rows: HBM would be read
// in 47 us for 16 trees of 32 tokens over 2001 to 16384 keys (8 KV heads, 4 query heads each, D 128), the tensor
// core done in 40.  The kernel takes 154: a step of 128 keys goes from warp to warp -- codes, K as an operand, S,
// softmax, P, O -- and takes 2 us (1.7 at D 64) whatever the rows are.  With parts left out of a copy (8 trees of
// 128 rows over 16384 keys, then 126 us): without conversions 113, softmax 101, products 117, all three 79, loads too 61;
// so it is hand-overs and their latencies, and each part's own time comes on top.  64 trees of 64 tokens of 129 to
// 4096 keys (8 query heads each, four items a KV head): 625 to 645 us against 146 of products; with 64 channels 498
// against 73.
//
// An item is a sequence's KV head and 128 of its rows; the batch's 128-key steps are cut into equal ranges, one for a
// CTA, and cut items added up as in cache_split.cuh.  512 threads:
//   warp 0       producer: pages looked up for four steps at once, codes and scales by bulk copies of 16 keys (the
//                keys that certainly share a page), three steps of codes ahead, six of scales (read by the softmax,
//                which ends later); zeros in place of chunks that are not there
//   warp 1       one lane issues S_n = Q K^T (SS) two steps ahead of O += P_n V (TS, P in TMEM over S_n's columns)
//   warps 4-7    E4M3 codes to bf16, exact, in the swizzled layout that the products read
//   warps 8-15   softmax and quantization: two groups that take steps in turn, each a row a thread with a maximum, a
//                sum and an accumulator of its own, added up at the end of a range's part of an item.  (Both groups on
//                one step, a 64-key tile each, wait for each other's maximum: 165 against 156 us, 667 against 655.)
// TMEM (512 columns): S, then P, of even and odd steps [0,128), [128,256); their O [256,256+D), [256+D,256+2D).
// Shared memory: Q, K and V as bf16 operands (32 KB each at D 128), three steps of codes (96 KB), scales.
//
// Roundings to fewer than 32 bits: q is exact (bf16 times a power of two); codes are exact in bf16; the weights,
// p' times the value's scale, are rounded to bf16, 2^-8 relative at most, as TMEM operands of one type with V
// (f16 would be 2^-11 but cannot hold V's scales' range without a power of two for each row and tile; K in f16 took
// 150 against 132 us and lost keys near 2^-105); o is rounded to bf16 once.  448 / amax is an approximate reciprocal,
// 2^-22 off as ex2 is.
//
// Built and not kept, us against the kernel of the time (8 trees of 128 rows, 16384 keys): sixteen softmax warps 128 ->
// 131; K and V converted straight from global memory with loads ahead in registers 126 -> 137 to 165; V in two buffers
// and K two steps ahead 128 -> 134; K and V in two buffers each, codes in three half steps 126 -> 138; scales multiplied
// in twice in place of S written back 126 -> 129; two issuing warps 126 -> 127 to 130; TMEM loads of the softmax 16 or
// 32 keys ahead 128 -> 136 to 186.  Two row tiles beside each other on every step, a group each, with K and V converted
// once for both: 0 to 10 percent faster for even numbers of tiles, 9 to 20 slower for odd ones, and twice the workspace.
#include "cache_split.cuh"
#include "qat_internal.h"
#include "qat_quant.cuh"
#include "sm100.cuh"

#include <cuda_bf16.h>

#include <type_traits>

namespace qat {
namespace {

using namespace sm100;

constexpr int kStep = 128;     // keys of a step
constexpr int kM = 128;        // query rows of an item
constexpr int kThreads = 512;  // warp 0 producer, 1 products, 4-7 converters, 8-15 softmax
constexpr int kStages = 3;     // steps whose codes are on their way or in shared memory
constexpr int kScStages = 6;   // steps whose scales are
constexpr float kRaise = 8.0f; // log2: the running maximum is raised when it is this far behind

template <int D>
struct Tc {
  static constexpr int kChunks = D / 64;                // 128-byte column chunks of a bf16 row
  static constexpr uint32_t kChunkBytes = kStep * 128;  // 128 rows x 64 columns
  static constexpr uint32_t kTileBytes = kChunks * kChunkBytes;
  static constexpr uint32_t kCodes = kStep * D;         // bytes of a step's codes of K, and of V
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kOffQ + kTileBytes;
  static constexpr uint32_t kOffV = kOffK + kTileBytes;
  static constexpr uint32_t kOffRing = kOffV + kTileBytes;        // codes: K, then V, of each stage
  static constexpr uint32_t kOffSc = kOffRing + kStages * 2 * kCodes;  // scales: K, then V
  static constexpr uint32_t kOffBar = kOffSc + kScStages * 8 * kStep;
  static constexpr uint32_t kOffMisc = kOffBar + 320;
  static constexpr uint32_t kOffX = kOffMisc + 64;  // the rows' largest |q|, m and l, [2 groups][128] each
  static constexpr uint32_t kOffSum = kOffX + 3 * 1024;               // the warps' sums, then B + 1 prefix sums
  static constexpr uint32_t kUsed = kOffSum + 4 * (kThreads / 32);
  static constexpr uint32_t kTmemO = 256;
};

enum : uint32_t {
  T_CODES = 0, T_CODES_FREE = T_CODES + kStages, T_SC = T_CODES_FREE + kStages, T_SC_FREE = T_SC + kScStages,
  T_Q = T_SC_FREE + kScStages, T_Q_FREE, T_K, T_K_FREE, T_V, T_V_FREE, T_S, T_P = T_S + 2, T_O_LAST = T_P + 2,
  T_O_FREE, T_DRAIN, T_X, T_COUNT = T_X + 4
};
static_assert(T_COUNT * 8 <= 320, "barrier block");

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Copies `bytes` (a multiple of 16, both addresses on 16-byte boundaries) and completes them on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}
// 32 lanes x 16 columns, as tmem_ld32.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Four E4M3 codes (not NaN) to bf16, exactly: four bits further up, the code's exponent and fraction are those of
// a bf16 number 2^120 times smaller, subnormal codes included.  The bytes are spread with their signs.
__device__ __forceinline__ uint2 codes_to_bf16x4(uint32_t x) {
  uint32_t lo, hi;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(x));
  asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(hi) : "r"(x));
  const uint32_t a = (lo << 4) & 0x87f087f0u, b = (hi << 4) & 0x87f087f0u;
  const uint32_t up = 0x7b807b80u;  // 2^120
  uint2 r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(a), "r"(up));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(b), "r"(up));
  return r;
}

// Bit 7 of a byte is one where the code is a NaN, 0x7f or 0xff: adding one there carries into the sign.  (Behind a byte
// 0xff another bit may be one too.)
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) { return (x + 0x01010101u) ^ x; }
__device__ __forceinline__ void sts2(uint32_t a, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}

// A worker's part of an item: `count` steps from the cursor's on.
__device__ __forceinline__ int segment_steps(const Cursor& c, int u, int u1) { return min(c.tiles - c.tile, u1 - u); }

// The cursor and unit behind a segment.
__device__ __forceinline__ void leave(const Params& p, const int* prefix, int extra, int count, Cursor& c, int& u) {
  u += count - 1;
  c.tile += count - 1;
  advance<kTree, kStep>(p, prefix, extra, c, u);
}

// What hides keys in the step at place `at`: the tree and the end, or the beginnings of windows.
__device__ __forceinline__ bool at_edge(const DecodeArgs& a, const Cursor& c, int at) {
  return (at + 1) * kStep > c.len - a.T ||
         (a.window > 0 && at * kStep < c.len - a.window && (at + 1) * kStep > a.sinks);
}

// The keys of key0 .. key0 + 63 that a row does not see; mask: the tokens it sees; pos: its position.
__device__ __forceinline__ unsigned long long hidden_keys(const DecodeArgs& a, int len, int key0, int pos,
                                                          unsigned long long mask) {
  const int base = len - a.T;
  unsigned long long seen = ones(0, base - key0);
  if (a.window > 0) seen &= ~ones(max(a.sinks - key0, 0), pos - a.window + 1 - key0);
  const int at = base - key0;  // where the first token's key lies
  if (at >= 0)
    seen |= at < 64 ? mask << at : 0ull;
  else
    seen |= at > -64 ? mask >> -at : 0ull;
  return ~seen;
}

// Of 16 codes that lane t of the converters' 128 takes i-th: their row, where they are and where the first eight go (the
// others 16 bytes across).
struct Piece {
  int row;
  uint32_t from, to;
};
template <int D>
__device__ __forceinline__ Piece piece_at(int t, uint32_t ring, uint32_t out, int i) {
  const int g = t >> 2, half = D == 64 ? 0 : (g & 1) ^ (i & 1), row = D == 64 ? g + 32 * i : g + 32 * (i >> 1);
  return Piece{row, ring + row * D + 16 * ((t & 3) + 4 * half),
               out + half * Tc<D>::kChunkBytes + row * 128 + (((2 * t & 6) ^ (row & 7)) << 4)};
}
// NaN operands where lane t's codes are NaN.  (Not inlined, as what follows: the kernel's warps share the instruction cache.)
template <int D>
__device__ __noinline__ void put_nan(int t, uint32_t ring, uint32_t out, int left) {
#pragma unroll 1
  for (int k = 0; k < D / 16 * kStep / 8; ++k) {
    const Piece piece = piece_at<D>(t, ring, out, k >> 4);
    const uint4 x = lds16(piece.from);
    const uint32_t w = (k & 8) ? ((k & 4) ? x.w : x.z) : ((k & 4) ? x.y : x.x);
    if (piece.row < left && (w >> 8 * (k & 3) & 0x7fu) == 0x7fu) sts2((piece.to ^ (2 * k & 16)) + 2 * (k & 7), 0x7fc0);
  }
}

// The channels D / 2 h .. D / 2 (h + 1) - 1 in which a value that the row sees has a NaN code, as bits: in `count` steps
// from `tile` on of sequence and KV head `seq`, read once more (where there are such codes at all: append stores none, but
// a cache may have been filled otherwise).
template <int D>
__device__ __noinline__ unsigned long long nan_channels(const Params& p, const int* prefix, int seq, int row, int tile,
                                                           int count, int h) {
  const DecodeArgs& a = p.a;
  Cursor c;
  c.b = seq / a.Hkv;
  c.h = seq - c.b * a.Hkv;
  enter_seq<kTree, kStep>(p, prefix, c);
  const unsigned long long mask = mask_of(a, c.b, row % a.T);
  const int pos = c.len - a.T + __popcll(mask) - 1;
  unsigned long long nan = 0ull;
#pragma unroll 1
  for (int i = 0; i < 2 * count; ++i) {
    const int key0 = place_of<kTree>(c, tile + (i >> 1)) * kStep + 64 * (i & 1);
    unsigned long long seen = ~hidden_keys(a, c.len, key0, pos, mask);
    while (seen != 0ull) {
      const int key = key0 + __ffsll(seen) - 1;
      seen &= seen - 1;
      const int page = a.table[static_cast<long long>(c.b) * a.max_pages + (key >> a.page_shift)];
      if (page < 0 || page >= a.num_pages) continue;
      const uint32_t at = ((static_cast<uint32_t>(page) * a.Hkv + c.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.v_codes + static_cast<size_t>(at) * D + D / 2 * h);
#pragma unroll 1
      for (int w = 0; w < D / 8; ++w) {
        const uint32_t x = codes[w];
        if (nan_codes(x) & 0x80808080u)
          for (int y = 0; y < 4; ++y) nan |= static_cast<unsigned long long>((x >> 8 * y & 0x7fu) == 0x7fu) << (4 * w + y);
      }
    }
  }
  return nan;
}

template <int D, bool kQuant>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ Params p) {
  using C = Tc<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::kOffBar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile WaitCtl* ctl = reinterpret_cast<volatile WaitCtl*>(gbase + C::kOffMisc + 8);
  // up to the last step with NaN codes in V
  volatile uint32_t* nan_steps = reinterpret_cast<volatile uint32_t*>(gbase + C::kOffMisc + 60);
  int* warp_sum = reinterpret_cast<int*>(gbase + C::kOffSum);
  int* prefix = warp_sum + kThreads / 32;
  const auto bar = [&](uint32_t i) { return bars + 8u * i; };
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    wait_ctl_init(ctl, a.err);
    *nan_steps = 0u;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(T_CODES + i), 1);
      mbar_init(bar(T_CODES_FREE + i), 128);
    }
    for (int i = 0; i < kScStages; ++i) {
      mbar_init(bar(T_SC + i), 1);
      mbar_init(bar(T_SC_FREE + i), 128);
    }
    mbar_init(bar(T_Q), 256);
    mbar_init(bar(T_Q_FREE), 1);
    mbar_init(bar(T_K), 128);
    mbar_init(bar(T_K_FREE), 1);
    mbar_init(bar(T_V), 128);
    mbar_init(bar(T_V_FREE), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(T_S + i), 1);
      mbar_init(bar(T_P + i), 128);
    }
    mbar_init(bar(T_O_LAST), 1);
    mbar_init(bar(T_O_FREE), 256);
    mbar_init(bar(T_DRAIN), 1);
    for (int i = 0; i < 4; ++i) mbar_init(bar(T_X + i), 64);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  after_previous();

  // prefix[b] = steps before sequence b
  const int per_seq = a.Hkv * p.mtiles;
  {
    const int chunk = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * chunk, a.B), b1 = min(b0 + chunk, a.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const int len = a.seq_lens[b], fits = clamp_len(a, len);
      if (len > fits) atomicOr(a.err, kErrBadPage);
      Cursor c;
      find_gap<kTree, kStep>(a, fits, c);
      prefix[b] = (tiles_of<kStep>(fits) - c.gap) * per_seq;
      sum += prefix[b];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int b = b0; b < b1; ++b) {
      const int units = prefix[b];
      prefix[b] = before;
      before += units;
    }
    if (tid == kThreads - 1) prefix[a.B] = before;
    __syncthreads();
  }
  const uint32_t tbase = *tmem_slot;
  const int steps = prefix[a.B], workers = min(steps, static_cast<int>(gridDim.x)), id = blockIdx.x;
  if (id == 0 && tid == 0) header_of(p)->workers = workers;
  // an item's own unit, where ranges are long enough that each holds a step all the same
  const int extra = steps / 4 >= workers ? 1 : 0;
  const int W = steps + extra * a.B * per_seq;
  const unsigned each = static_cast<unsigned>(W) / workers, over = W - each * workers;
  int u0 = 0, u1 = 0;
  Cursor first = {};
  if (id < workers) {
    u0 = each * id + over * id / workers;
    u1 = each * (id + 1) + over * (id + 1) / workers;
    int lo = 0, hi = a.B;  // the last b whose units begin at u0 or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] + extra * mid * per_seq <= u0) lo = mid; else hi = mid;
    }
    first.b = lo;
    enter_seq<kTree, kStep>(p, prefix, first);
    const int u = u0 - (prefix[lo] + extra * lo * per_seq);
    const int item = u / (first.tiles + extra), in = u - item * (first.tiles + extra);
    first.tile = max(in - extra, 0);
    if (in < extra) ++u0;  // to the item's first step
    first.mt = item % p.mtiles;
    first.h = item / p.mtiles;
  }
  Cursor c = first;
  int u = u0;
  bool ok = true;
  const auto wait = [&](uint32_t i, uint32_t parity) { return mbar_wait(bar(i), parity & 1, ctl, a.err); };
  const auto wwait = [&](uint32_t i, uint32_t parity) {  // the same answer in every lane
    return __all_sync(0xffffffffu, wait(i, parity)) != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t n = 0;
    uint32_t rows_of = kNoPage;  // lane l: cache row where chunk l of a group of 4 steps begins
    bool fresh = true;
    while (u < u1) {
      if (fresh || (c.tile & 3) == 0) {
        const int pos = place_of<kTree>(c, (c.tile & ~3) + (lane >> 3)) * kStep + (lane & 7) * kChunk;
        // pages that hold nothing any row sees are not looked up: they may have been given back
        const bool unseen = pos + kChunk <= c.low && pos >= a.sinks;
        rows_of = kNoPage;
        if (pos < c.len && !unseen) {
          const int page = a.table[static_cast<long long>(c.b) * a.max_pages + (pos >> a.page_shift)];
          rows_of = kBadPage;
          if (page >= 0 && page < a.num_pages)
            rows_of = ((static_cast<uint32_t>(page) * a.Hkv + c.h) << a.page_shift) +
                      (pos & ((1 << a.page_shift) - 1));
          else
            atomicOr(a.err, kErrBadPage);
        }
        fresh = false;
      }
      const uint32_t st = n % kStages, sc = n % kScStages;
      if (!(ok = wwait(T_CODES_FREE + st, (n / kStages & 1) ^ 1) && wwait(T_SC_FREE + sc, (n / kScStages & 1) ^ 1)))
        break;
      const uint32_t rc = __shfl_sync(0xffffffffu, rows_of, (c.tile & 3) * 8 + (lane & 7));
      const uint32_t there = __ballot_sync(0xffffffffu, rc < kBadPage) & 0xffu;
      const uint32_t bad = __ballot_sync(0xffffffffu, rc == kBadPage) & 0xffu;
      const uint32_t ring = base + C::kOffRing + st * 2 * C::kCodes, scales = base + C::kOffSc + sc * 8 * kStep;
      for (uint32_t rest = ~there & 0xffu; rest != 0; rest &= rest - 1) {  // zeros; NaN scales for bad pages
        const int k = __ffs(rest) - 1;
        const uint32_t fill = (bad >> k & 1u) ? 0x7fc00000u : 0u;
#pragma unroll
        for (int i = 0; i < kChunk * D / 512; ++i) {
          sts16(ring + k * kChunk * D + 512 * i + 16 * lane, make_uint4(0u, 0u, 0u, 0u));
          sts16(ring + C::kCodes + k * kChunk * D + 512 * i + 16 * lane, make_uint4(0u, 0u, 0u, 0u));
        }
        if (lane < 8)  // lanes 0-3: K's, 4-7: V's
          sts16(scales + (lane >> 2) * 4 * kStep + k * 4 * kChunk + 16 * (lane & 3), make_uint4(fill, fill, fill, fill));
        fence_async();  // a later step's copies go there
      }
      __syncwarp();
      if (lane == 0) {
        const uint32_t chunks = __popc(there);
        mbar_arrive_expect_tx(bar(T_CODES + st), chunks * 2 * kChunk * D);
        mbar_arrive_expect_tx(bar(T_SC + sc), chunks * 2 * 4 * kChunk);
      }
      __syncwarp();
      // lanes 0-7: the chunks' K, 8-15: V, 16-23: K's scales, 24-31: V's
      if (rc < kBadPage) {
        const int k = lane & 7;
        if (lane < 16)
          bulk_load(ring + (lane >> 3) * C::kCodes + k * kChunk * D,
                    (lane < 8 ? a.k_codes : a.v_codes) + static_cast<size_t>(rc) * D, kChunk * D, bar(T_CODES + st));
        else
          bulk_load(scales + (lane >> 3 & 1) * 4 * kStep + k * 4 * kChunk, (lane < 24 ? a.k_scales : a.v_scales) + rc,
                    4 * kChunk, bar(T_SC + sc));
      }
      ++n;
      const int b = c.b, h = c.h;
      advance<kTree, kStep>(p, prefix, extra, c, u);
      fresh = c.b != b || c.h != h;
    }
    // every copy lands before the CTA exits
    for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
      mbar_wait_drain(bar(T_CODES + i % kStages), i / kStages & 1, a.err);
    for (uint32_t i = n > kScStages ? n - kScStages : 0; i < n; ++i)
      mbar_wait_drain(bar(T_SC + i % kScStages), i / kScStages & 1, a.err);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      constexpr uint32_t idS = idesc_bf16_f32(kM, kStep, false), idO = idesc_bf16_f32(kM, D, true);
      uint32_t n = 0, it = 0;
      bool issued = false;
      const auto issue_s = [&](uint32_t k, bool last) {  // S of step k, over P of step k - 2, which its sums have read
        if (!wait(T_K, k)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * C::kChunkBytes + (ks & 3) * 32;
          mma_ss(tbase + (k & 1) * 128, smem_desc_sw128(base + C::kOffQ + off, 16, 1024),
                 smem_desc_sw128(base + C::kOffK + off, 16, 1024), idS, ks > 0 ? 1u : 0u);
        }
        issued = true;
        mma_commit(bar(T_K_FREE));
        mma_commit(bar(T_S + (k & 1)));
        if (last) mma_commit(bar(T_Q_FREE));
        return true;
      };
      for (; u < u1 && ok; ++it) {
        const int count = segment_steps(c, u, u1);
        ok = wait(T_Q, it) && issue_s(n, count == 1) && (count == 1 || issue_s(n + 1, count == 2));
        for (int j = 0; j < count && ok; ++j, ++n) {
          if (!(ok = wait(T_V, n) && wait(T_P + (n & 1), n >> 1))) break;
          if (j == 0 && !(ok = wait(T_O_FREE, it + 1))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < kStep / 16; ++ks)
            mma_ts(tbase + C::kTmemO + (n & 1) * D, tbase + (n & 1) * 128 + 8 * ks,
                   smem_desc_sw128(base + C::kOffV + ks * 2048, C::kChunkBytes, 1024), idO, (j > 1 || ks > 0) ? 1u : 0u);
          mma_commit(bar(T_V_FREE));
          if (j + 1 == count) mma_commit(bar(T_O_LAST));
          if (j + 2 < count && !(ok = issue_s(n + 2, j + 3 == count))) break;
        }
        if (ok) leave(p, prefix, extra, count, c, u);
      }
      if (issued) {
        mma_commit(bar(T_DRAIN));
        mbar_wait_drain(bar(T_DRAIN), 0, a.err);
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ codes to bf16 operands
    // Each step's K and V from E4M3 codes into the 128-byte swizzled layout that the products read, K of the next step
    // before V of this one.  A lane takes 16 codes at a time; groups of four lanes take the halves of two rows
    // crosswise, so that eight lanes are on different banks both reading and writing.
    // NaN codes, which the conversion would make 480, are looked for in a lane's part of a step at once (16 trees of 32
    // tokens 152.0 -> 154.2 us, 64 of 64 tokens 617 -> 630; with a branch at every 16 codes 162 and 657; as the largest of
    // the bf16 numbers 156 and 637; by the two warps with nothing else to do, in the codes as they land, 160 and 686).  Keys
    // get a NaN operand, whose scores are NaN where they count.  A value's would reach rows that do not see it: the step
    // is noted, and the softmax warps look again at the end of their segment.
    const int t = tid & 127;
    constexpr int kEach = kStep * (D / 16) / 128;  // 16-code pieces of a lane
    const auto convert = [&](uint32_t ring, uint32_t out, int left) {  // whether there was a NaN code
      uint32_t nan = 0u;
#pragma unroll 1
      for (int i0 = 0; i0 < kEach; i0 += 2) {
        uint4 x[2];
        Piece at[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          at[i] = piece_at<D>(t, ring, out, i0 + i);
          x[i] = lds16(at[i].from);
        }
        if (left < kStep) {  // behind the end: may hold anything
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (at[i].row >= left) x[i] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint2 w0 = codes_to_bf16x4(x[i].x), w1 = codes_to_bf16x4(x[i].y), w2 = codes_to_bf16x4(x[i].z),
                      w3 = codes_to_bf16x4(x[i].w);
          nan |= nan_codes(x[i].x) | nan_codes(x[i].y) | nan_codes(x[i].z) | nan_codes(x[i].w);
          sts16(at[i].to, make_uint4(w0.x, w0.y, w1.x, w1.y));
          sts16(at[i].to ^ 16, make_uint4(w2.x, w2.y, w3.x, w3.y));
        }
      }
      return (nan & 0x80808080u) != 0;
    };
    const auto left_at = [&](const Cursor& x) { return x.len - place_of<kTree>(x, x.tile) * kStep; };
    const auto do_k = [&](uint32_t n, int left) {
      const uint32_t st = n % kStages;
      if (!wait(T_CODES + st, n / kStages) || !wait(T_K_FREE, n + 1)) return false;
      const uint32_t ring = base + C::kOffRing + st * 2 * C::kCodes;
      if (convert(ring, base + C::kOffK, left)) put_nan<D>(t, ring, base + C::kOffK, left);
      fence_async();
      mbar_arrive(bar(T_K));
      return true;
    };
    int left = 0;
    if (u < u1) ok = do_k(0, left = left_at(c));
    for (uint32_t n = 0; u < u1 && ok; ++n) {
      advance<kTree, kStep>(p, prefix, extra, c, u);
      int next = 0;
      if (u < u1 && !do_k(n + 1, next = left_at(c))) break;
      const uint32_t st = n % kStages;
      if (!wait(T_V_FREE, n + 1)) break;
      if (convert(base + C::kOffRing + st * 2 * C::kCodes + C::kCodes, base + C::kOffV, left)) *nan_steps = n + 1;
      fence_async();
      mbar_arrive(bar(T_V));
      mbar_arrive(bar(T_CODES_FREE + st));
      left = next;
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ softmax, two groups of four warps
    // Group h takes every other step, a thread a row of its S, with a running maximum, a sum and an accumulator of its
    // own, added up at a segment's end: no thread waits for another in between, and the two warps of a scheduler
    // are at different places of a step.
    const int h = (warp - 8) >> 2, quarter = warp & 3, r = 32 * quarter + lane;
    const uint32_t lrow = (32u * quarter) << 16;
    float* xq = reinterpret_cast<float*>(gbase + C::kOffX);  // [2 groups][128]
    float* xm = xq + 256;
    float* xl = xq + 512;
    uint32_t xc = 0;
    const auto exchange = [&]() {  // between the two threads of a row (and their warps)
      tc_fence_before();
      mbar_arrive(bar(T_X + quarter));
      const bool w = wwait(T_X + quarter, xc);
      ++xc;
      tc_fence_after();
      return w;
    };
    // This thread's row of the item at c: half h of it goes to shared memory times a power of two that takes its
    // largest element to 1 .. 2 (times 2^-32, so that products with large scales stay finite, unless that takes
    // rf out of range); scores are S scale_k rf.
    unsigned long long mask = 0ull;
    int pos = 0;
    float rf = 0.f;
    const auto load_q = [&](const Cursor& at) {
      const int row = at.mt * kM + r;
      uint4 x[D / 16];
      float amax = 0.f;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((static_cast<size_t>(at.b) * a.Hkv + at.h) * p.R + row) * D + (D / 2) * h);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) x[i] = row < p.R ? src[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
      }
      xq[h * 128 + r] = amax;
      if (!exchange()) return false;
      amax = fmaxf(amax, xq[(h ^ 1) * 128 + r]);
      int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      e = min(max(e, -100), 126);
      const bool far = !(ldexpf(a.qk_scale, e) < 18446744073709551616.f);
      const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23), less = far ? 1.f : 2.3283064365386963e-10f;
      rf = fmaxf(ldexpf(a.qk_scale, e + (far ? 0 : 32)), 1.1754943508222875e-38f);  // not zero: it multiplies -inf
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = pack_bf16(__uint_as_float(w[k] << 16) * up * less, __uint_as_float(w[k] & 0xffff0000u) * up * less);
        const int piece = h * (D / 16) + i;  // of the row's D / 8
        sts16(base + C::kOffQ + (piece >> 3) * C::kChunkBytes + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
              make_uint4(w[0], w[1], w[2], w[3]));
      }
      const int token = row % a.T;
      mask = mask_of(a, at.b, token);
      pos = at.len - a.T + __popcll(mask) - 1;
      fence_async();
      mbar_arrive(bar(T_Q));
      return true;
    };
    if (warp == 8 && lane == 0 && id < kWorkers && !p.by_item) chains_of(p)[id] = Chain{-1, -1};
    uint32_t first_n = 0, it = 0;  // the segment's first step
    if (u < u1) ok = load_q(c);
    for (; u < u1 && ok; ++it) {
      const int count = segment_steps(c, u, u1);
      float m = -INFINITY, l = 0.f;
      const uint32_t tS = tbase + lrow + 128 * h, tO = tbase + lrow + C::kTmemO + D * h;
      const int j0 = (first_n & 1) ^ h;  // this group's first step of the segment
      for (int j = j0; j < count && ok; j += 2) {
        const uint32_t n = first_n + j, sc = n % kScStages;
        if (!(ok = wwait(T_S + h, n >> 1) && wwait(T_SC + sc, n / kScStages))) break;
        tc_fence_after();
        const uint32_t ks = base + C::kOffSc + sc * 8 * kStep, vs = ks + 4 * kStep;
        const int at = place_of<kTree>(c, c.tile + j);
        const bool edge = at_edge(a, c, at);
        unsigned long long hid0 = 0ull, hid1 = 0ull;
        if (edge) {
          hid0 = hidden_keys(a, c.len, at * kStep, pos, mask);
          hid1 = hidden_keys(a, c.len, at * kStep + 64, pos, mask);
        }
        // S times the keys' scales goes back to where it came from, 32 keys at a time; the largest of each tile
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t sr[32];
          tmem_ld32(tS + 32 * q, sr);
          tmem_wait_ld();
          float* s = reinterpret_cast<float*>(sr);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 k = lds16(ks + 128 * q + 16 * i);
            const float2 lo = mul_rn_f32x2(make_float2(s[4 * i], s[4 * i + 1]),
                                           make_float2(__uint_as_float(k.x), __uint_as_float(k.y)));
            const float2 hi = mul_rn_f32x2(make_float2(s[4 * i + 2], s[4 * i + 3]),
                                           make_float2(__uint_as_float(k.z), __uint_as_float(k.w)));
            s[4 * i] = lo.x; s[4 * i + 1] = lo.y; s[4 * i + 2] = hi.x; s[4 * i + 3] = hi.y;
          }
          if (edge) {
            const uint32_t hq = static_cast<uint32_t>((q < 2 ? hid0 : hid1) >> (32 * (q & 1)));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (hq >> i & 1u) s[i] = -INFINITY;
          }
          tmem_st32(tS + 32 * q, sr);
          float t = fmaxf(s[0], s[1]);
#pragma unroll
          for (int i = 2; i < 32; i += 2) t = fmax3(t, s[i], s[i + 1]);
          if (q < 2) t0 = fmaxf(t0, t); else t1 = fmaxf(t1, t);
        }
        tmem_wait_st();
        const float top = fmaxf(t0, t1) * rf;
        if (__any_sync(0xffffffffu, top > m + kRaise)) {
          float alpha = 1.f;
          if (top > m + kRaise) {
            alpha = ex2(m - top);
            m = top;
          }
          l *= alpha;
          if (j > j0) {  // S of this step is behind every product of this accumulator so far
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * k, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + 32 * k, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        float inv0 = 0.f, back0 = 0.f, inv1 = 0.f, back1 = 0.f;
        if (kQuant) {
          const float a0 = ex2(fmaf(t0, rf, neg)), a1 = ex2(fmaf(t1, rf, neg));
          // (four divisions in place of two approximate reciprocals and two products took 700 of a group's 7700 cycles
          // a step)
          inv0 = a0 < kTinyP ? 0.f : kE4M3Max * rcp(a0);
          inv1 = a1 < kTinyP ? 0.f : kE4M3Max * rcp(a1);
          back0 = a0 < kTinyP ? 0.f : a0 * (1.f / kE4M3Max);
          back1 = a1 < kTinyP ? 0.f : a1 * (1.f / kE4M3Max);
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t sr[32], pk[16];
          tmem_ld32(tS + 32 * q, sr);
          tmem_wait_ld();
          const float* s = reinterpret_cast<const float*>(sr);
          const float inv = q < 2 ? inv0 : inv1, back = q < 2 ? back0 : back1;
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // four keys
            const uint4 vv = lds16(vs + 128 * q + 16 * i);
            const uint32_t v4[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int k = 4 * i + 2 * y;
              const float2 e = fma_rn_f32x2(make_float2(s[k], s[k + 1]), make_float2(rf, rf), make_float2(neg, neg));
              float2 w = make_float2(ex2(e.x), ex2(e.y));
              sum = add_rn_f32x2(sum, w);
              if (kQuant) {
                const float2 x = mul_rn_f32x2(w, make_float2(inv, inv));
                w = mul_rn_f32x2(e4m3x2_decode(e4m3x2_rn_satfinite(x.x, x.y)), make_float2(back, back));
              }
              w = mul_rn_f32x2(w, make_float2(__uint_as_float(v4[2 * y]), __uint_as_float(v4[2 * y + 1])));
              pk[2 * i + y] = pack_bf16(w.x, w.y);
            }
          }
          if (edge) {  // 0 x NaN: a key that the row does not see may hold anything
            const uint32_t hq = static_cast<uint32_t>((q < 2 ? hid0 : hid1) >> (32 * (q & 1)));
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pk[i] &= ((hq >> (2 * i) & 1u) ? 0u : 0xffffu) | ((hq >> (2 * i + 1) & 1u) ? 0u : 0xffff0000u);
          }
          tmem_st16(tS + 16 * q, pk);  // over keys whose scores have been read
        }
        mbar_arrive(bar(T_SC_FREE + sc));
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(T_P + h));
      }
      if (!ok) break;
      // the segment's end: the next one's rows first, whose scores can follow while this one's sums are stored
      const bool head = c.tile != 0, ends = c.tile + count == c.tiles, whole = !head && ends;
      const int row = c.mt * kM + r, item = item_of(p, c), seq = c.b * a.Hkv + c.h, tile = c.tile;
      if (!head && warp == 8 && lane == 0) {
        const long long end = u - c.tile + c.tiles;  // the unit behind the item
        if (whole) {
          if (p.by_item) chains_of(p)[item] = Chain{-1, -1};
        } else {
          chains_of(p)[p.by_item ? item : id] = Chain{p.by_item ? id : item, static_cast<int>((end * workers - 1) / W)};
        }
      }
      xm[h * 128 + r] = m;
      xl[h * 128 + r] = l;
      if (!(ok = exchange())) break;
      const float m0 = xm[r], m1 = xm[128 + r], both = fmaxf(m0, m1), ref = both == -INFINITY ? 0.f : both;
      const float w0 = ex2(m0 - ref), w1 = ex2(m1 - ref);
      const float lr = fmaf(xl[r], w0, xl[128 + r] * w1);
      const bool has0 = count > 1 || (first_n & 1) == 0, has1 = count > 1 || (first_n & 1) == 1;
      leave(p, prefix, extra, count, c, u);
      first_n += count;
      if (u < u1 && !(ok = wwait(T_Q_FREE, it) && load_q(c))) break;
      if (!(ok = wwait(T_O_LAST, it))) break;
      tc_fence_after();
      const bool none = lr == 0.f, in = row < p.R;
      const float f = whole ? (none ? 0.f : 1.f / lr) : 1.f, f0 = w0 * f, f1 = w1 * f;
      float* part = partial_of<D>(p, id, head ? 0 : 1);
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {  // half of the channels, 16 at a time
        uint32_t o0[16], o1[16];
        const uint32_t from = tbase + lrow + C::kTmemO + (D / 2) * h + 16 * k;
        tmem_ld16(from, o0);
        tmem_ld16(from + D, o1);
        tmem_wait_ld();
        if (!in) continue;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          x[i] = (has0 ? __uint_as_float(o0[i]) * f0 : 0.f) + (has1 ? __uint_as_float(o1[i]) * f1 : 0.f);
        if (whole) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = none ? 0u : pack_bf16(x[2 * i], x[2 * i + 1]);
          uint4* dst = reinterpret_cast<uint4*>(a.o + (static_cast<size_t>(seq) * p.R + row) * D + (D / 2) * h + 16 * k);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float4* dst = reinterpret_cast<float4*>(part + r * D + (D / 2) * h + 16 * k);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
      }
      tc_fence_before();
      mbar_arrive(bar(T_O_FREE));
      if (*nan_steps > first_n - count && in) {
        for (unsigned long long nan = nan_channels<D>(p, prefix, seq, row, tile, count, h); nan != 0ull; nan &= nan - 1) {
          const int ch = (D / 2) * h + __ffsll(nan) - 1;
          if (whole)
            a.o[(static_cast<size_t>(seq) * p.R + row) * D + ch] = 0x7fc0;
          else
            part[r * D + ch] = __uint_as_float(0x7fc00000u);
        }
      }
      if (in && h == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(part + p.prows * D + 2 * r) = make_float2(both, lr);
        else if (a.lse != nullptr)
          a.lse[static_cast<size_t>(seq) * p.R + row] = none ? -INFINITY : both + log2f(lr);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
}

template <int D, bool kQuant>
cudaError_t run(Params p, int ctas, int most, cudaStream_t s) {
  using C = Tc<D>;
  // at least 116 KB, so that no two CTAs share an SM (each holds all 512 TMEM columns)
  const auto bytes = [](int B) {
    const size_t n = C::kUsed + 4 * (static_cast<size_t>(B) + 1) + 1024;
    return n > 118784 ? n : 118784;
  };
  const long long items = static_cast<long long>(p.a.B) * p.a.Hkv * p.mtiles;
  p.by_item = items <= most;
  static_assert(C::kUsed + 4 * (kDecodeMaxBatch + 1) + 1024 <= 227 * 1024, "the batch's prefix sums fit");
  cudaError_t e = cudaFuncSetAttribute(tree_kernel<D, kQuant>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(bytes(kDecodeMaxBatch)));
  if (e != cudaSuccess) return e;
  e = launch_early(tree_kernel<D, kQuant>, ctas, kThreads, bytes(p.a.B), s, p);
  if (e != cudaSuccess) return e;
  return launch_merge<D>(p, most, ctas, s);
}

// Rows of a partial, even so that partials stay 16-byte aligned.
int partial_rows(int R) { return R < kM ? (R + 1) / 2 * 2 : kM; }

}  // namespace

size_t tree_workspace_bytes(int R, int D) { return workspace_of(kMaxCtas, partial_rows(R), D); }

cudaError_t launch_tree(const DecodeArgs& a, int D, int num_sms, cudaStream_t s) {
  Params p;
  p.a = a;
  p.R = a.Hq / a.Hkv * a.T;
  p.rows = kM;
  p.mtiles = (p.R + kM - 1) / kM;
  p.prows = partial_rows(p.R);
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  const long long units = static_cast<long long>(a.B) * a.Hkv * p.mtiles * ((cap + kStep - 1) / kStep);
  int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  if (units < ctas) ctas = static_cast<int>(units);
  if (D == 64) return a.quant ? run<64, true>(p, ctas, ctas, s) : run<64, false>(p, ctas, ctas, s);
  return a.quant ? run<128, true>(p, ctas, ctas, s) : run<128, false>(p, ctas, ctas, s);
}

}  // namespace qat
