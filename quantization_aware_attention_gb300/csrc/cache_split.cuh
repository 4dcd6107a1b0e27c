// cache_split.cuh -- what the kernels over the FP8 cache share: how a batch's key tiles are cut into equal ranges
// whatever the sequences' lengths, the workspace that holds what the cuts leave, and the kernels that add it up.
//
// The batch's units -- tiles of kUnit keys, ordered by sequence, KV head, row tile, key -- are cut into equal
// contiguous ranges, one per worker (a warp or a block).  An item (sequence, head, row tile) inside one range is
// finished there; an item that a range boundary cuts leaves unnormalized fp32 partials with their m and l in the
// workspace, which the merge kernels add in an order that the sizes, the table's width and the lengths decide.
#pragma once

#include "qat_internal.h"
#include "sm100.cuh"

#include <cuda_bf16.h>

namespace qat {
namespace {

constexpr int kTile = 64;    // keys that share a scale of P
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
// of a kernel's workspace: what partial_of gives each worker, behind the rest
constexpr size_t workspace_of(int workers, int prows, int D) {
  return kPartsAt + static_cast<size_t>(workers) * 2 * prows * (D + 2) * sizeof(float);
}

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

// What the rows may see of the keys before their own: everything, or a window and the sinks; or (the last T
// tokens being a drafted tree) also those of the T that their masks name.
enum { kAll = 0, kWindow = 1, kTree = 2 };

// A place in the batch's list of units.  Where windows leave a gap between the sinks and the keys of the first
// row's window, the gap's whole tiles are not units: `tile` counts the others.
struct Cursor {
  int b, h, mt, tile, tiles, len;
  int gap_at, gap, low;  // tiles from gap_at on lie `gap` further; no row sees keys before `low` but sinks
};

template <int kMask>
__device__ __forceinline__ int place_of(const Cursor& c, int tile) {
  return kMask != kAll && tile >= c.gap_at ? tile + c.gap : tile;
}

template <int kMask, int kUnit = kTile>
__device__ __forceinline__ void find_gap(const DecodeArgs& a, int len, Cursor& c) {
  c.gap_at = c.gap = c.low = 0;
  if (kMask == kAll || a.window == 0) return;
  // the first token's window; a drafted token with an empty mask has the position before it
  c.low = max(len - a.T - a.window + (kMask == kTree ? 0 : 1), 0);
  c.gap_at = (min(a.sinks, len) + kUnit - 1) / kUnit;
  c.gap = max(c.low / kUnit - c.gap_at, 0);
}

__device__ __forceinline__ int clamp_len(const DecodeArgs& a, int len) {
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  return len > cap ? static_cast<int>(cap) : max(len, 0);
}
template <int kUnit = kTile>
__device__ __forceinline__ int tiles_of(int len) {
  return len > 0 ? (len + kUnit - 1) / kUnit : 1;
}

// Tiles as the prefix sums have them: the cut and every index hold together even if a length changes
// under the kernel.
template <int kMask, int kUnit = kTile>
__device__ __forceinline__ void enter_seq(const Params& p, const int* prefix, Cursor& c) {
  if (c.b >= p.a.B) return;  // behind the last: not looked at again
  c.tiles = static_cast<unsigned>(prefix[c.b + 1] - prefix[c.b]) / static_cast<unsigned>(p.a.Hkv * p.mtiles);
  c.len = clamp_len(p.a, p.a.seq_lens[c.b]);
  find_gap<kMask, kUnit>(p.a, c.len, c);
  c.len = min(c.len, (c.tiles + c.gap) * kUnit);
}

// The next tile; u: its unit.
template <int kMask, int kUnit = kTile>
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
  enter_seq<kMask, kUnit>(p, prefix, c);
}

__device__ __forceinline__ unsigned long long mask_of(const DecodeArgs& a, int b, int token) {
  return a.tree[b * a.tree_sb + token] & (~0ull >> (kTreeMaxTokens - a.T));  // bits from T on name no token
}

__device__ __forceinline__ int item_of(const Params& p, const Cursor& c) {
  return (c.b * p.a.Hkv + c.h) * p.mtiles + c.mt;
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

// Adds up what the cuts left: `most` workers at most, `ctas` blocks of the kernel before.
template <int D>
cudaError_t launch_merge(const Params& p, int most, int ctas, cudaStream_t s) {
  const long long items = static_cast<long long>(p.a.B) * p.a.Hkv * p.mtiles;
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
}  // namespace qat
