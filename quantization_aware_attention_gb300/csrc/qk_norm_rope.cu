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
// the outputs round to bf16 (2^-9 relative).
//
// Work split.  D / 16 lanes hold one row, 16 channels each as two 16-byte chunks chosen so
// that both halves of every pair are in one lane; a warp holds 4 rows (D = 128) or 8 (D = 64)
// of one token, computes the token's angles once and walks the heads of its part.  A block's
// 8 warps take 8 consecutive tokens, so that in the head-major output a block writes 2 KB
// (D = 128) runs.
#include "qat_internal.h"

#include <cuda_bf16.h>

namespace qat {
namespace {

constexpr int kWarps = 8;
constexpr int kPer = 16;                        // channels per lane
constexpr float kTurnToRad = 1.4629180792671596e-09f;  // 2 pi / 2^32

struct Row16 {
  uint4 a, b;
};

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}

// The lane's two 8-channel chunks, whether each is rotated, and the pair index of each
// chunk's first pair.
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
      ca = rot_a ? j : 2 * j;   // the other chunks in order: R / 8 + 2 (j - half)
      cb = rot_a ? j + half : 2 * j + 1;
      pair_a = pair_b = 8 * j;
    }
  }
};

// The eight (cos, sin) pairs of the lane at a position, times the amplitude; unset for
// chunks that are not rotated.
template <bool kInter, class Map>
__device__ __forceinline__ void lane_angles(const Map& m, const unsigned long long* phases,
                                            int pos, float amplitude, float (&c)[8],
                                            float (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool rot = (kInter && e >= 4) ? m.rot_b : m.rot_a;
    c[e] = s[e] = 0.f;
    if (rot) {
      const int i = kInter ? (e < 4 ? m.pair_a + e : m.pair_b + e - 4) : m.pair_a + e;
      const unsigned long long turn =
          static_cast<unsigned long long>(static_cast<long long>(pos)) * __ldg(phases + i);
      const float ang = static_cast<float>(static_cast<int>(turn >> 32)) * kTurnToRad;
      float sn, cs;
      __sincosf(ang, &sn, &cs);
      c[e] = cs * amplitude;
      s[e] = sn * amplitude;
    }
  }
}

// v: the lane's 16 channels (chunk a, then chunk b), rotated in place by +angle (kBack: by
// -angle, the transpose).
// Channels that are not rotated are left alone, not multiplied by (1, 0): an infinity would
// make its neighbour NaN.
template <bool kInter, bool kBack, class Map>
__device__ __forceinline__ void rotate16(const Map& m, float (&v)[16], const float (&c)[8],
                                         const float (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int ia = kInter ? 2 * e : e, ib = kInter ? 2 * e + 1 : e + 8;
    if (!((kInter && e >= 4) ? m.rot_b : m.rot_a)) continue;
    const float a = v[ia], b = v[ib], sn = kBack ? -s[e] : s[e];
    v[ia] = a * c[e] - b * sn;
    v[ib] = a * sn + b * c[e];
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void load_weight8(const void* w, int bf16, int ch, float* f) {
  if (bf16) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + ch), f);
  } else {
    const float4 x = __ldg(reinterpret_cast<const float4*>(w) + 2 * ch);
    const float4 y = __ldg(reinterpret_cast<const float4*>(w) + 2 * ch + 1);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
  }
}

// Where block `part` of a token's heads lies: parts [0, nq) are the query heads, the rest the
// key heads, `hpp` heads each.
struct Part {
  bool key;
  int h0, h1;
};

__device__ __forceinline__ Part part_of(const NormRopeArgs& p, int part) {
  Part r;
  r.key = part >= p.q_parts;
  r.h0 = (r.key ? part - p.q_parts : part) * p.heads_per_part;
  r.h1 = min(r.h0 + p.heads_per_part, r.key ? p.k.H : p.q.H);
  return r;
}

template <int D, bool kInter>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormRopeArgs p) {
  constexpr int L = D / kPer;    // lanes per row
  constexpr int RW = 32 / L;     // rows per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % p.parts;
  const long long tok = static_cast<long long>(blockIdx.x / p.parts) * kWarps + warp;
  if (tok >= p.tokens) return;
  const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);
  const Part pt = part_of(p, part);
  const NormRopeTensor& t = pt.key ? p.k : p.q;
  const LaneMap<D, kInter> m(lane % L, p.R);
  const int sub = lane / L;

  float w[16];
  if (t.w != nullptr) {
    load_weight8(t.w, p.w_bf16, m.ca, w);
    load_weight8(t.w, p.w_bf16, m.cb, w + 8);
  }
  float c[8], s[8];
  const int pos = p.R > 0 ? __ldg(p.positions + b * p.pos_sb + n) : 0;
  lane_angles<kInter>(m, p.phases, pos, p.amplitude, c, s);

  const uint16_t* src = t.x + b * t.sb + n * t.sn;
  uint16_t* dst = t.y + (static_cast<long long>(b) * t.H * p.N + n) * D;
  for (int h = pt.h0 + sub; h - sub < pt.h1; h += RW) {
    const bool in = h < pt.h1;
    float v[16];
    uint4 ra = make_uint4(0u, 0u, 0u, 0u), rb = ra;
    if (in) {
      const uint16_t* row = src + h * t.sh;
      ra = __ldg(reinterpret_cast<const uint4*>(row) + m.ca);
      rb = __ldg(reinterpret_cast<const uint4*>(row) + m.cb);
    }
    unpack8(ra, v);
    unpack8(rb, v + 8);
    if (t.w != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss += v[i] * v[i];
      const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] * r * w[i];
    }
    rotate16<kInter, false>(m, v, c, s);
    if (in) {
      uint4* out = reinterpret_cast<uint4*>(dst + static_cast<long long>(h) * p.N * D);
      out[m.ca] = pack8(v);
      out[m.cb] = pack8(v + 8);
    }
  }
}

// Backward.  Persistent: block k of a tensor's `blocks` walks (8-token group, head part) items
// k, k + blocks, ...; each lane keeps the weight gradient of its 16 channels in registers and
// the block's sum goes to its own row of the workspace, which norm_rope_dw_kernel adds in
// block order.  No atomics: the same sizes give the same bits.
template <int D, bool kInter>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_bwd_kernel(const NormRopeArgs p) {
  constexpr int L = D / kPer;
  constexpr int RW = 32 / L;
  __shared__ float red[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool key = blockIdx.x >= static_cast<unsigned>(p.q_blocks);
  const NormRopeTensor& t = key ? p.k : p.q;
  const int blk = key ? blockIdx.x - p.q_blocks : blockIdx.x;
  const int blocks = key ? gridDim.x - p.q_blocks : p.q_blocks;
  const int parts = key ? p.parts - p.q_parts : p.q_parts;
  const long long items = (p.tokens + kWarps - 1) / kWarps * parts;
  const LaneMap<D, kInter> m(lane % L, p.R);
  const int sub = lane / L;

  float w[16], dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
  if (t.w != nullptr) {
    load_weight8(t.w, p.w_bf16, m.ca, w);
    load_weight8(t.w, p.w_bf16, m.cb, w + 8);
  }
  for (long long it = blk; it < items; it += blocks) {
    const int part = static_cast<int>(it % parts);
    const long long tok = it / parts * kWarps + warp;
    if (tok >= p.tokens) continue;
    const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);
    const int h0 = part * p.heads_per_part, h1 = min(h0 + p.heads_per_part, t.H);
    float c[8], s[8];
    const int pos = p.R > 0 ? __ldg(p.positions + b * p.pos_sb + n) : 0;
    lane_angles<kInter>(m, p.phases, pos, p.amplitude, c, s);
    const uint16_t* xs = t.x + b * t.sb + n * t.sn;
    const uint16_t* gs = t.dy + b * t.dy_sb + n * t.dy_sn;
    uint16_t* ds = t.y + b * t.y_sb + n * t.y_sn;
    for (int h = h0 + sub; h - sub < h1; h += RW) {
      const bool in = h < h1;
      float g[16];
      uint4 ga = make_uint4(0u, 0u, 0u, 0u), gb = ga, xa = ga, xb = ga;
      if (in) {
        const uint16_t* grow = gs + h * t.dy_sh;
        ga = __ldg(reinterpret_cast<const uint4*>(grow) + m.ca);
        gb = __ldg(reinterpret_cast<const uint4*>(grow) + m.cb);
        if (t.w != nullptr) {
          const uint16_t* row = xs + h * t.sh;
          xa = __ldg(reinterpret_cast<const uint4*>(row) + m.ca);
          xb = __ldg(reinterpret_cast<const uint4*>(row) + m.cb);
        }
      }
      unpack8(ga, g);
      unpack8(gb, g + 8);
      rotate16<kInter, true>(m, g, c, s);
      if (t.w != nullptr) {
        float x[16];
        unpack8(xa, x);
        unpack8(xb, x + 8);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss += x[i] * x[i];
        const float r = rsqrtf(row_sum<L>(ss) * (1.f / D) + p.eps);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] *= r;                 // the normed channel
          dw[i] += g[i] * x[i];
          g[i] *= w[i];
          dot += g[i] * x[i];
        }
        dot = row_sum<L>(dot) * (1.f / D);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = r * (g[i] - x[i] * dot);
      }
      if (in) {
        uint4* out = reinterpret_cast<uint4*>(ds + h * t.y_sh);
        out[m.ca] = pack8(g);
        out[m.cb] = pack8(g + 8);
      }
    }
  }
  if (t.w == nullptr) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      red[warp][8 * m.ca + i] = dw[i];
      red[warp][8 * m.cb + i] = dw[8 + i];
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

// dw[d] = the sum over a tensor's blocks of part[block][d]: one block per tensor, D x 8 threads,
// each adding every eighth row, then the eight sums in order.
template <int D>
__global__ void __launch_bounds__(D * 8) norm_rope_dw_kernel(const NormRopeArgs p, int k_blocks) {
  __shared__ float red[8][D];
  const bool key = blockIdx.x == 1;
  const int blocks = key ? k_blocks : p.q_blocks;
  void* out = key ? p.k.dw : p.q.dw;
  const float* src = p.part + (key ? static_cast<size_t>(p.q_blocks) * D : 0);
  const int d = threadIdx.x % D, lane8 = threadIdx.x / D;
  float sum = 0.f;
  for (int i = lane8; i < blocks; i += 8) sum += src[static_cast<size_t>(i) * D + d];
  red[lane8][d] = sum;
  __syncthreads();
  if (lane8 == 0 && out != nullptr) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += red[i][d];
    if (p.w_bf16)
      static_cast<__nv_bfloat16*>(out)[d] = __float2bfloat16_rn(sum);
    else
      static_cast<float*>(out)[d] = sum;
  }
}

// Heads per part: one trip of a warp over its rows while that leaves the GPU short of warps,
// more (up to 8 trips, so that a token's angles are shared) when tokens abound.
void choose_parts(NormRopeArgs& a, int D, int num_sms) {
  const int rows_per_trip = 32 / (D / kPer);
  const long long trips = a.tokens * ((a.q.H + a.k.H + rows_per_trip - 1) / rows_per_trip);
  long long per = trips / (static_cast<long long>(num_sms) * 64);
  if (per < 1) per = 1;
  if (per > 8) per = 8;
  a.heads_per_part = static_cast<int>(per) * rows_per_trip;
  a.q_parts = (a.q.H + a.heads_per_part - 1) / a.heads_per_part;
  a.parts = a.q_parts + (a.k.H + a.heads_per_part - 1) / a.heads_per_part;
}

template <int D>
cudaError_t run_fwd(const NormRopeArgs& a, unsigned grid, cudaStream_t s) {
  if (a.interleaved)
    norm_rope_kernel<D, true><<<grid, 32 * kWarps, 0, s>>>(a);
  else
    norm_rope_kernel<D, false><<<grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_bwd(const NormRopeArgs& a, int k_blocks, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.q_blocks + k_blocks);
  if (a.interleaved)
    norm_rope_bwd_kernel<D, true><<<grid, 32 * kWarps, 0, s>>>(a);
  else
    norm_rope_bwd_kernel<D, false><<<grid, 32 * kWarps, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (a.q.w == nullptr && a.k.w == nullptr)) return e;
  norm_rope_dw_kernel<D><<<2, D * 8, 0, s>>>(a, k_blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeArgs a, int D, int num_sms, cudaStream_t s) {
  choose_parts(a, D, num_sms);
  const long long grid = (a.tokens + kWarps - 1) / kWarps * a.parts;
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  return D == 64 ? run_fwd<64>(a, static_cast<unsigned>(grid), s)
                 : run_fwd<128>(a, static_cast<unsigned>(grid), s);
}

cudaError_t launch_norm_rope_bwd(NormRopeArgs a, int D, int num_sms, cudaStream_t s) {
  choose_parts(a, D, num_sms);
  // the blocks are shared out in proportion to the heads, at least one for a tensor that is there
  const long long groups = (a.tokens + kWarps - 1) / kWarps;
  const int H = a.q.H + a.k.H;
  auto share = [&](int heads, int parts) {
    if (heads == 0) return 0;
    long long n = static_cast<long long>(kNormRopeBwdBlocks - 1) * heads / H;
    if (n > groups * parts) n = groups * parts;
    return static_cast<int>(n < 1 ? 1 : n);
  };
  a.q_blocks = share(a.q.H, a.q_parts);
  const int k_blocks = share(a.k.H, a.parts - a.q_parts);
  return D == 64 ? run_bwd<64>(a, k_blocks, s) : run_bwd<128>(a, k_blocks, s);
}

}  // namespace qat
