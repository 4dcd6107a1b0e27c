// qk_norm_rope.cu -- what makes the attention's queries and keys: the RMS norm of every
// head's D channels and the rotation by position, in one pass over the data, and the
// backward of both.
//
//   r = rsqrt(mean_d x_d^2 + eps);  z = x r w          (w NULL: z = x)
//   channels [0, R) in pairs (a, b) -- (i, i + R/2), or (2i, 2i + 1) interleaved -- turned by
//   the angle of their pair:  y_a = A (z_a cos - z_b sin),  y_b = A (z_a sin + z_b cos)
//   channels [R, D):  y = z
//   backward:  dz = A R^T dy;  dw = sum_rows dz x r;  dn = dz w;
//              dx = r (dn - x r mean_d(dn x r))
//
// Angles.  A pair's frequency is a 64-bit fraction of a turn per position, so position x
// phase modulo 2^64 is the angle's fraction of a turn, exact at every 32-bit position: the
// reduction that 32-bit angles lose (at position 10^6 an fp32 angle is off by 0.06 rad)
// costs two integer multiplies, and no table of cosines is read.  The fraction's top 32 bits
// become an angle in [-pi, pi), where the hardware sine and cosine are within 2^-20 absolute;
// the outputs round to bf16 (by up to 2^-8 of themselves).
//
// Work split.  D / 16 lanes hold one row, 16 channels each as two 16-byte chunks chosen so that both
// halves of every pair are in one lane; a warp holds 4 rows (D = 128) or 8 (D = 64) of one token,
// computes the token's angles once and walks the heads of its part, a trip of 4 or 8 heads at a time.
// Of a tensor with half as many heads or fewer it takes 2, 4 or 8 tokens at once instead of leaving
// lanes idle.  A block's 8 warps take consecutive tokens, so that in the head-major output a block
// writes 2 KB (D = 128) runs.
//
// What bounds both directions is HBM; what it takes is bytes in flight.  The rows of the next trips are
// on their way by cp.async, each lane's own 16-byte pieces into its own place in shared memory: no
// registers, no barriers.  Arithmetic is in packed fp32 pairs.  Measured, D = 128, full rotation, norms:
//   B1 H40+40 N32768   forward 197 us, 6.8 TB/s of the 4 bytes a channel read and written
//   B4 H32+32 N8192    forward 158 us, 6.8 TB/s; backward 236 us, 6.8 TB/s of 6 bytes a channel
//   B1 H32+8 N2048     forward 10.6 us, backward 20; B16 N1 2.4 us
// Few heads (D = 64, 3+1 heads, 200000 tokens): forward 71 us, 2.9 TB/s, 61 without the rotation as without the
// norm.  A warp makes one trip of 8 rows and ends: 520 instructions with its start, angles and weights, 74 percent
// of the issue slots.  Backward 112 us, 88 without norm and weights.
// Backward of small sizes (B1 H32+8 N2048): 20 us, 12 without norm and weights; what the sums' second launch,
// each block's start and its sums take of the rest has not been told apart.
// The forward is held to 64 registers, for four blocks an SM, and spills 4 to 40 bytes a thread.
#include "qat_internal.h"
#include "qat_quant.cuh"
#include "sm100.cuh"

#include <cuda_bf16.h>

namespace qat {
namespace {

constexpr int kWarps = 8;
constexpr int kPer = 16;        // channels per lane
constexpr int kFwdStages = 4;   // trips in flight and in hand
constexpr int kBwdStages = 3;
constexpr float kTurnToRad = 1.4629180792671596e-09f;  // 2 pi / 2^32

// A lane's 16 channels as 8 pairs (a, b), packed two by two: in the half layout a is chunk `a` and b
// chunk `b`; interleaved, the first four pairs are chunk `a`, the others chunk `b`.
struct Chan {
  float2 a[4], b[4];
};

__device__ __forceinline__ float2 bf16x2_to_f32x2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool kInter>
__device__ __forceinline__ void unpack(const uint4& ra, const uint4& rb, Chan& v) {
  const uint32_t x[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInter) {
      const float2 p = bf16x2_to_f32x2(x[2 * i]), q = bf16x2_to_f32x2(x[2 * i + 1]);
      v.a[i] = make_float2(p.x, q.x);
      v.b[i] = make_float2(p.y, q.y);
    } else {
      v.a[i] = bf16x2_to_f32x2(x[i]);
      v.b[i] = bf16x2_to_f32x2(x[4 + i]);
    }
  }
}

template <bool kInter>
__device__ __forceinline__ void store(uint4* row, int ca, int cb, const Chan& v) {
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInter) {
      x[2 * i] = f32x2_to_bf16x2(v.a[i].x, v.b[i].x);
      x[2 * i + 1] = f32x2_to_bf16x2(v.a[i].y, v.b[i].y);
    } else {
      x[i] = f32x2_to_bf16x2(v.a[i].x, v.a[i].y);
      x[4 + i] = f32x2_to_bf16x2(v.b[i].x, v.b[i].y);
    }
  }
  row[ca] = make_uint4(x[0], x[1], x[2], x[3]);
  row[cb] = make_uint4(x[4], x[5], x[6], x[7]);
}

// The lane's two 8-channel chunks, whether each is rotated, and the pair index of each chunk's first
// pair.
template <int D, bool kInter>
struct LaneMap {
  int ca, cb;
  bool rot_a, rot_b;  // half layout: both or neither
  int pair_a, pair_b;
  __device__ __forceinline__ LaneMap(int j, int R) {
    constexpr int L = D / kPer;
    if constexpr (kInter) {
      ca = j;
      cb = j + L;
      rot_a = ca < R / 8;
      rot_b = cb < R / 8;
      pair_a = 4 * ca;
      pair_b = 4 * cb;
    } else {
      const int half = R / 16;  // chunks per half of the rotated part
      rot_a = rot_b = j < half;
      ca = rot_a ? j : half + j;  // the other chunks, R / 8 .. D / 8 - 1, in two runs of lanes
      cb = rot_a ? j + half : L + j;
      pair_a = 8 * j;
      pair_b = 8 * j + 4;
    }
  }
  // channel of pair e's member a (b: the next one, or the one of chunk b)
  __device__ __forceinline__ int channel(int e, bool b) const {
    if (kInter) return 8 * (e < 4 ? ca : cb) + 2 * (e & 3) + (b ? 1 : 0);
    return 8 * (b ? cb : ca) + e;
  }
};

// The lane's eight (cos, sin) pairs at a position, times the amplitude; unset for chunks that are not
// rotated.
template <bool kInter, class Map>
__device__ __forceinline__ void lane_angles(const Map& m, const unsigned long long* phases, int pos,
                                            float amplitude, float2 (&c)[4], float2 (&s)[4]) {
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = sn[e] = 0.f;
    if (e < 4 ? m.rot_a : m.rot_b) {
      const unsigned long long turn =
          static_cast<unsigned long long>(static_cast<long long>(pos)) *
          phases[e < 4 ? m.pair_a + e : m.pair_b + e - 4];
      const float ang = static_cast<float>(static_cast<int>(turn >> 32)) * kTurnToRad;
      __sincosf(ang, &sn[e], &cs[e]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = make_float2(cs[2 * i] * amplitude, cs[2 * i + 1] * amplitude);
    s[i] = make_float2(sn[2 * i] * amplitude, sn[2 * i + 1] * amplitude);
  }
}

// v rotated in place by +angle (kBack: by -angle, the transpose).  Channels that are not rotated are
// left alone, not multiplied by (1, 0): an infinity would make its neighbour NaN.
template <bool kBack, class Map>
__device__ __forceinline__ void rotate(const Map& m, Chan& v, const float2 (&c)[4], const float2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!(i < 2 ? m.rot_a : m.rot_b)) continue;
    const float2 a = v.a[i], b = v.b[i];
    const float2 minus = make_float2(-s[i].x, -s[i].y);
    v.a[i] = fma_rn_f32x2(a, c[i], mul_rn_f32x2(b, kBack ? s[i] : minus));
    v.b[i] = fma_rn_f32x2(b, c[i], mul_rn_f32x2(a, kBack ? minus : s[i]));
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// sum_e x_e y_e over the lane's channels
__device__ __forceinline__ float dot16(const Chan& x, const Chan& y) {
  float2 s = mul_rn_f32x2(x.a[0], y.a[0]), t = mul_rn_f32x2(x.b[0], y.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = fma_rn_f32x2(x.a[i], y.a[i], s);
    t = fma_rn_f32x2(x.b[i], y.b[i], t);
  }
  s = add_rn_f32x2(s, t);
  return s.x + s.y;
}

template <bool kInter, class Map>
__device__ __forceinline__ void load_weight(const Map& m, const void* w, int bf16, Chan& v) {
  float* a = reinterpret_cast<float*>(v.a);
  float* b = reinterpret_cast<float*>(v.b);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = m.channel(e, false), j = m.channel(e, true);
    a[e] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
    b[e] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[j]) : static_cast<const float*>(w)[j];
  }
}

// The lane's own 16 bytes from global memory into its own place; zeros (and no access) when !in.
__device__ __forceinline__ void fetch16(uint32_t dst, const uint4* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// kFew: a tensor has so few heads that a warp's rows are of several of its tokens.  (A variant, as the
// lanes' own tokens cost registers: B1 H40+40 N32768 D128 takes 203 us with them, 198 without.)
template <int D, bool kInter, bool kFew>
__global__ void __launch_bounds__(32 * kWarps, 4) norm_rope_kernel(const NormRopeArgs p) {
  constexpr int L = D / kPer;    // lanes per row
  constexpr int RW = 32 / L;     // rows per warp and trip
  __shared__ uint4 ring[kWarps][kFwdStages][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  after_previous();
  bool key;
  unsigned group, part;  // of the tokens; of the tensor's heads, heads_per_part each
  if constexpr (kFew) {  // blocks [0, q_blocks) are the queries', the rest the keys'
    key = blockIdx.x >= static_cast<unsigned>(p.q_blocks);
    const unsigned blk = key ? blockIdx.x - p.q_blocks : blockIdx.x, parts = key ? p.parts - p.q_parts : p.q_parts;
    group = blk / parts;
    part = blk - group * parts;
  } else {  // the parts of both for the same tokens, one after the other
    group = blockIdx.x / static_cast<unsigned>(p.parts);
    part = blockIdx.x - group * static_cast<unsigned>(p.parts);
    key = part >= static_cast<unsigned>(p.q_parts);
    if (key) part -= p.q_parts;
  }
  const NormRopeTensor& t = key ? p.k : p.q;
  const int log_tokens = kFew ? t.log_tokens : 0;
  const unsigned long long first = (static_cast<unsigned long long>(group) * kWarps + warp) << log_tokens;
  if (first >= static_cast<unsigned long long>(p.tokens)) return;
  const int heads = RW >> log_tokens;  // heads of a trip
  const int sub = lane / L % heads;
  unsigned tok = static_cast<unsigned>(first);
  const int h0 = static_cast<int>(part) * p.heads_per_part, h1 = min(h0 + p.heads_per_part, t.H);
  int lim = h1;  // the lane's rows end at lim
  if constexpr (kFew) {
    const unsigned left = static_cast<unsigned>(p.tokens - 1) - tok, ahead = lane / L / heads;
    if (ahead > left) lim = 0;
    tok += min(ahead, left);
  }
  const unsigned b = tok / static_cast<unsigned>(p.N), n = tok - b * static_cast<unsigned>(p.N);
  const LaneMap<D, kInter> m(lane % L, p.R);

  const uint16_t* src = t.x + b * t.sb + n * t.sn;
  const uint32_t mine = sm100::smem_addr(&ring[warp][0][0][lane]);
  int hf = h0 + sub;  // head fetched next
  uint32_t fs = 0;
  auto fetch = [&]() {
    if (hf - sub < h1) {
      const uint4* row = reinterpret_cast<const uint4*>(src + min(hf, h1 - 1) * t.sh);
      fetch16(mine + fs * 1024, row + m.ca, hf < lim);
      fetch16(mine + fs * 1024 + 512, row + m.cb, hf < lim);
      hf += heads;
      fs = fs + 1 == kFwdStages ? 0 : fs + 1;
    }
    fetch_commit();
  };
#pragma unroll
  for (int i = 0; i < kFwdStages - 1; ++i) fetch();

  Chan w;
  if (t.w != nullptr) load_weight<kInter>(m, t.w, p.w_bf16, w);
  float2 c[4], s[4];
  const int pos = p.R > 0 ? p.positions[b * p.pos_sb + n] : 0;
  lane_angles<kInter>(m, p.phases, pos, p.amplitude, c, s);

  uint16_t* dst = t.y + (static_cast<long long>(b) * t.H * p.N + n) * D;
  uint32_t us = 0;
  for (int h = h0 + sub; h - sub < h1; h += heads) {
    fetch();
    fetch_wait<kFwdStages - 1>();
    Chan v;
    unpack<kInter>(lds128(mine + us * 1024), lds128(mine + us * 1024 + 512), v);
    us = us + 1 == kFwdStages ? 0 : us + 1;
    if (t.w != nullptr) {
      const float2 r = both(rsqrtf(row_sum<L>(dot16(v, v)) * (1.f / D) + p.eps));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v.a[i] = mul_rn_f32x2(mul_rn_f32x2(v.a[i], r), w.a[i]);
        v.b[i] = mul_rn_f32x2(mul_rn_f32x2(v.b[i], r), w.b[i]);
      }
    }
    rotate<false>(m, v, c, s);
    if (h < lim)
      store<kInter>(reinterpret_cast<uint4*>(dst + static_cast<long long>(h) * p.N * D), m.ca, m.cb, v);
  }
}

// Backward.  Persistent, so that the weights' gradients leave each block once: block k of a tensor's
// `blocks` walks (token group, head part) items k, k + blocks, ...; each lane keeps the weight gradient of its 16 channels in registers and
// the block's sum goes to its own row of the workspace, which norm_rope_dw_kernel adds in
// block order.  No atomics: the same sizes give the same bits.  The sums are fp32 throughout, off by 4e-7 of the
// gradients' size for 10^6 rows of normal values and by 1e-6 for 8 10^6 (the terms' own fp32 roundings: 1.4e-7).
template <int D, bool kInter>
__global__ void __launch_bounds__(32 * kWarps, 2) norm_rope_bwd_kernel(const NormRopeArgs p) {
  constexpr int L = D / kPer;
  constexpr int RW = 32 / L;
  __shared__ uint4 ring[kWarps][kBwdStages][4][32];  // x and dy; then the warps' weight gradients
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool key = blockIdx.x >= static_cast<unsigned>(p.q_blocks);
  const NormRopeTensor& t = key ? p.k : p.q;
  const int blk = key ? blockIdx.x - p.q_blocks : blockIdx.x;
  const int blocks = key ? gridDim.x - p.q_blocks : p.q_blocks;
  const unsigned parts = key ? p.parts - p.q_parts : p.q_parts;
  const long long items = (p.tokens + (kWarps << t.log_tokens) - 1) / (kWarps << t.log_tokens) * parts;
  const LaneMap<D, kInter> m(lane % L, p.R);
  const int heads = RW >> t.log_tokens;  // heads of a trip
  const int sub = lane / L % heads;
  const bool norm = t.w != nullptr;
  after_previous();

  // The fetches run ahead over the warp's trips: their item, token and head.
  const uint32_t mine = sm100::smem_addr(&ring[warp][0][0][lane]);
  long long fi = blk;
  const uint16_t *fx = nullptr, *fg = nullptr;
  int fh = 0, fh1 = 0;  // heads fetched next, and the part's end; fh = fh1: the next item
  bool fthere = false;
  uint32_t fs = 0;
  // the lane's token of an item and whether there is one; false: the warp has none
  auto locate = [&](long long it, bool& there, unsigned& b, unsigned& n, int& h0, int& h1) {
    const unsigned group = static_cast<unsigned>(it / parts), part = static_cast<unsigned>(it - static_cast<long long>(group) * parts);
    const unsigned long long first = (static_cast<unsigned long long>(group) * kWarps + warp) << t.log_tokens;
    if (first >= static_cast<unsigned long long>(p.tokens)) return false;
    const unsigned last = static_cast<unsigned>(p.tokens - 1);
    there = first + lane / L / heads <= last;
    const unsigned tok = there ? static_cast<unsigned>(first) + lane / L / heads : last;
    b = tok / static_cast<unsigned>(p.N);
    n = tok - b * static_cast<unsigned>(p.N);
    h0 = part * p.heads_per_part;
    h1 = min(h0 + p.heads_per_part, t.H);
    return true;
  };
  auto fetch = [&]() {
    while (fh >= fh1 && fi < items) {  // on to the next item that this warp has a token of
      unsigned b, n;
      if (locate(fi, fthere, b, n, fh, fh1)) {
        fx = t.x + b * t.sb + n * t.sn;
        fg = t.dy + b * t.dy_sb + n * t.dy_sn;
      }
      fi += blocks;
    }
    if (fh < fh1) {
      const int h = fh + sub;
      const bool in = fthere && h < fh1;
      const uint32_t at = mine + fs * 2048;
      const uint4* g = reinterpret_cast<const uint4*>(fg + min(h, fh1 - 1) * t.dy_sh);
      fetch16(at, g + m.ca, in);
      fetch16(at + 512, g + m.cb, in);
      if (norm) {
        const uint4* x = reinterpret_cast<const uint4*>(fx + min(h, fh1 - 1) * t.sh);
        fetch16(at + 1024, x + m.ca, in);
        fetch16(at + 1536, x + m.cb, in);
      }
      fh += heads;
      fs = fs + 1 == kBwdStages ? 0 : fs + 1;
    }
    fetch_commit();
  };
#pragma unroll
  for (int i = 0; i < kBwdStages - 1; ++i) fetch();

  Chan w, dw;
#pragma unroll
  for (int i = 0; i < 4; ++i) dw.a[i] = dw.b[i] = both(0.f);
  if (norm) load_weight<kInter>(m, t.w, p.w_bf16, w);
  uint32_t us = 0;
  for (long long it = blk; it < items; it += blocks) {
    unsigned b, n;
    int h0, h1;
    bool there;
    if (!locate(it, there, b, n, h0, h1)) continue;
    float2 c[4], s[4];
    const int pos = p.R > 0 ? p.positions[b * p.pos_sb + n] : 0;
    lane_angles<kInter>(m, p.phases, pos, p.amplitude, c, s);
    uint16_t* ds = t.y + b * t.y_sb + n * t.y_sn;
    for (int h = h0 + sub; h - sub < h1; h += heads) {
      fetch();
      fetch_wait<kBwdStages - 1>();
      const uint32_t at = mine + us * 2048;
      us = us + 1 == kBwdStages ? 0 : us + 1;
      Chan g;
      unpack<kInter>(lds128(at), lds128(at + 512), g);
      rotate<true>(m, g, c, s);
      if (norm) {
        Chan x;
        unpack<kInter>(lds128(at + 1024), lds128(at + 1536), x);
        const float r = rsqrtf(row_sum<L>(dot16(x, x)) * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // x: the normed channel
          x.a[i] = mul_rn_f32x2(x.a[i], both(r));
          x.b[i] = mul_rn_f32x2(x.b[i], both(r));
          dw.a[i] = fma_rn_f32x2(g.a[i], x.a[i], dw.a[i]);
          dw.b[i] = fma_rn_f32x2(g.b[i], x.b[i], dw.b[i]);
          g.a[i] = mul_rn_f32x2(g.a[i], w.a[i]);
          g.b[i] = mul_rn_f32x2(g.b[i], w.b[i]);
        }
        const float2 dot = both(-row_sum<L>(dot16(g, x)) * (1.f / D));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g.a[i] = mul_rn_f32x2(fma_rn_f32x2(x.a[i], dot, g.a[i]), both(r));
          g.b[i] = mul_rn_f32x2(fma_rn_f32x2(x.b[i], dot, g.b[i]), both(r));
        }
      }
      if (there && h < h1) store<kInter>(reinterpret_cast<uint4*>(ds + h * t.y_sh), m.ca, m.cb, g);
    }
  }
  if (!norm) return;
  fetch_wait<0>();
  float* va = reinterpret_cast<float*>(dw.a);
  float* vb = reinterpret_cast<float*>(dw.b);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
      va[e] += __shfl_xor_sync(0xffffffffu, va[e], o);
      vb[e] += __shfl_xor_sync(0xffffffffu, vb[e], o);
    }
  }
  __syncthreads();  // the ring is free
  float(*red)[D] = reinterpret_cast<float(*)[D]>(&ring[0][0][0][0]);
  if (lane < L) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      red[warp][m.channel(e, false)] = va[e];
      red[warp][m.channel(e, true)] = vb[e];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) sum += red[k][d];
    p.part[static_cast<size_t>(blockIdx.x) * D + d] = sum;
  }
}

// dw[d] = the sum over a tensor's blocks of part[block][d]: a block for 32 channels of a tensor, 32 warps
// that each add every 32nd row, then the warps' sums.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const NormRopeArgs p, int k_blocks, int D) {
  __shared__ float red[32][33];
  const bool key = blockIdx.y == 1;
  const int blocks = key ? k_blocks : p.q_blocks;
  void* out = key ? p.k.dw : p.q.dw;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
  const float* src = p.part + (key ? static_cast<size_t>(p.q_blocks) * D : 0) + d;
  after_previous();  // the blocks' sums are complete
  float sum = 0.f;
#pragma unroll 8
  for (int i = warp; i < blocks; i += 32) sum += __ldcg(src + static_cast<size_t>(i) * D);
  red[warp][lane] = sum;
  __syncthreads();
  sum = red[lane][warp];  // warp w: channel w
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane != 0 || out == nullptr) return;
  if (p.w_bf16)
    static_cast<__nv_bfloat16*>(out)[blockIdx.x * 32 + warp] = __float2bfloat16_rn(sum);
  else
    static_cast<float*>(out)[blockIdx.x * 32 + warp] = sum;
}

// Heads per part: one trip of a warp over its rows while that leaves the GPU short of warps, more (up to
// 16 trips, so that a token's angles are shared and fetches run ahead) when tokens abound, in parts of
// about the same size.
void choose_parts(NormRopeArgs& a, int D, int num_sms) {
  const int rows_per_trip = 32 / (D / kPer);
  const long long trips = a.tokens * ((a.q.H + a.k.H + rows_per_trip - 1) / rows_per_trip);
  long long per = trips / (static_cast<long long>(num_sms) * 64);
  per = per < 1 ? 1 : per > 16 ? 16 : per;
  const int most = a.q.H > a.k.H ? a.q.H : a.k.H;
  const int parts = static_cast<int>((most + per * rows_per_trip - 1) / (per * rows_per_trip));
  a.heads_per_part = parts == 0 ? rows_per_trip
                                : ((most + parts - 1) / parts + rows_per_trip - 1) / rows_per_trip * rows_per_trip;
  a.q_parts = (a.q.H + a.heads_per_part - 1) / a.heads_per_part;
  a.parts = a.q_parts + (a.k.H + a.heads_per_part - 1) / a.heads_per_part;
  for (NormRopeTensor* t : {&a.q, &a.k}) {
    t->log_tokens = 0;
    while (t->H > 0 && t->H << (t->log_tokens + 1) <= rows_per_trip) ++t->log_tokens;
  }
}

long long token_groups(const NormRopeArgs& a, const NormRopeTensor& t) {
  return (a.tokens + (kWarps << t.log_tokens) - 1) / (kWarps << t.log_tokens);
}

template <int D>
cudaError_t run_fwd(const NormRopeArgs& a, unsigned grid, cudaStream_t s) {
  const bool few = a.q.log_tokens + a.k.log_tokens > 0;
  auto kernel = a.interleaved ? (few ? norm_rope_kernel<D, true, true> : norm_rope_kernel<D, true, false>)
                              : (few ? norm_rope_kernel<D, false, true> : norm_rope_kernel<D, false, false>);
  return launch_early(kernel, grid, 32 * kWarps, 0, s, a);
}

template <int D>
cudaError_t run_bwd(const NormRopeArgs& a, int k_blocks, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.q_blocks + k_blocks);
  const cudaError_t e = launch_early(a.interleaved ? norm_rope_bwd_kernel<D, true> : norm_rope_bwd_kernel<D, false>,
                                     grid, 32 * kWarps, 0, s, a);
  if (e != cudaSuccess || (a.q.w == nullptr && a.k.w == nullptr)) return e;
  return launch_early(norm_rope_dw_kernel, dim3(D / 32, 2), 1024, 0, s, a, k_blocks, D);
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeArgs a, int D, int num_sms, cudaStream_t s) {
  choose_parts(a, D, num_sms);
  const long long q_blocks = token_groups(a, a.q) * a.q_parts;
  const long long grid = q_blocks + token_groups(a, a.k) * (a.parts - a.q_parts);
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  a.q_blocks = static_cast<int>(q_blocks);
  return D == 64 ? run_fwd<64>(a, static_cast<unsigned>(grid), s)
                 : run_fwd<128>(a, static_cast<unsigned>(grid), s);
}

cudaError_t launch_norm_rope_bwd(NormRopeArgs a, int D, int num_sms, cudaStream_t s) {
  choose_parts(a, D, num_sms);
  // the blocks are shared out in proportion to the heads, at least one for a tensor that is there
  const int H = a.q.H + a.k.H;
  // two blocks fit an SM: twice as many even out the SMs' different speeds where each has many trips left
  // (B1 H40+40 N32768 D128: 317 us, 335 with one wave), one wave saves a block's start and its sums else
  // (B1 H32+8 N2048 D128: 20.9 against 22.2 us)
  const long long trips = a.tokens * H / (32 / (D / kPer)) / kWarps;  // per warp of a block, of all blocks
  const int most = trips >= 64ll * kNormRopeBwdBlocks ? kNormRopeBwdBlocks
                                                      : (2 * num_sms < kNormRopeBwdBlocks ? 2 * num_sms : kNormRopeBwdBlocks);
  auto share = [&](const NormRopeTensor& t, int parts) {
    if (t.H == 0) return 0;
    long long n = static_cast<long long>(most) * t.H / H;
    if (n > token_groups(a, t) * parts) n = token_groups(a, t) * parts;
    return static_cast<int>(n < 1 ? 1 : n);
  };
  a.q_blocks = share(a.q, a.q_parts);
  const int k_blocks = share(a.k, a.parts - a.q_parts);
  return D == 64 ? run_bwd<64>(a, k_blocks, s) : run_bwd<128>(a, k_blocks, s);
}

}  // namespace qat
