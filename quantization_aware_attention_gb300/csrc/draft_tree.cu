// draft_tree.cu -- around the attention of a drafted tree: the tokens' masks and positions from their parents,
// and the cache's move of the accepted path behind the text.
//
//   mask(t) = bit t | mask(parent(t)),  position(t) = len - T + popcount(mask(t)) - 1
//   rows len - T + path[i] -> len - T + i  for i < kept;  len' = len - T + kept
//
// Both are a few dependent loads and a launch: in a captured graph the masks of one tree of 16 tokens take 1.1 us, of
// 256 of 64 tokens 1.7; moving 6 of 32 rows for 16 sequences and 8 heads of 128 channels 2.3, 24 of 64 rows for 256
// sequences (26 MB) 6.2 us, 4.2 TB/s.  Called one by one the host takes 4.5 to 5 us for each.  The masks are a warp's
// work for a sequence: six rounds of pointer doubling (each token takes its ancestor's set over and then that one's
// ancestor) in place of a walk of up to 63 steps.  The move is a block's work for a sequence and head: every row is
// read before one is written, so a path may be in any order and name a row twice.
#include "qat_internal.h"

namespace qat {
namespace {

constexpr int kWarpsPerBlock = 4;
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(32 * kWarpsPerBlock) draft_tree_kernel(const DraftTreeArgs a) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  after_previous();
  if (b >= a.B) return;
  const int len = a.seq_lens[b];
  unsigned long long m[2];
  int up[2];     // the ancestor that the set reaches to, -1 at the text
  int pad[2];    // not a token, or behind one that is not
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int t = lane + 32 * y;
    const int parent = t < a.T ? a.parents[b * a.parents_sb + t] : -2;
    pad[y] = parent < -1 || parent >= t;
    m[y] = pad[y] ? 0ull : 1ull << t;
    up[y] = pad[y] ? -1 : parent;
  }
#pragma unroll
  for (int round = 0; round < 6; ++round) {
    unsigned long long nm[2];
    int nup[2], npad[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int from = up[y] & 31;
      const unsigned long long m0 = __shfl_sync(0xffffffffu, m[0], from), m1 = __shfl_sync(0xffffffffu, m[1], from);
      const int u0 = __shfl_sync(0xffffffffu, up[0], from), u1 = __shfl_sync(0xffffffffu, up[1], from);
      const int p0 = __shfl_sync(0xffffffffu, pad[0], from), p1 = __shfl_sync(0xffffffffu, pad[1], from);
      const bool any = up[y] >= 0, high = up[y] >= 32;
      nm[y] = m[y] | (any ? (high ? m1 : m0) : 0ull);
      npad[y] = pad[y] | (any ? (high ? p1 : p0) : 0);
      nup[y] = any ? (high ? u1 : u0) : -1;
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      m[y] = nm[y];
      up[y] = nup[y];
      pad[y] = npad[y];
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int t = lane + 32 * y;
    if (t >= a.T) continue;
    const unsigned long long mask = pad[y] ? 0ull : m[y];
    const long long at = static_cast<long long>(b) * a.T + t;
    a.tree[at] = mask;
    a.positions[at] = len - a.T + __popcll(mask) - 1;
  }
}

// One 16-byte piece of a cached row, or a row's two scales, and where it goes.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv_keep_kernel(const KvKeepArgs a) {
  constexpr int kPieces = 2 * D / 16;                                    // of a row's keys and values
  constexpr int kEach = kTreeMaxTokens * kPieces / kMoveThreads;         // pieces a thread holds at most
  const int h = blockIdx.x % a.H, b = blockIdx.x / a.H;
  after_previous();
  const int len = a.seq_lens[b], want = a.path_lens[b];
  const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
  const long long base = static_cast<long long>(len) - a.T;
  const int kept = min(max(want, 0), a.L);
  if (h == 0 && threadIdx.x == 0) {
    a.new_lens[b] = static_cast<int>(max(base + kept, 0ll));
    if (len > cap) atomicOr(a.err, kErrBadPage);
  }
  // the cache's rows that path entry i goes from and to; false where nothing is to be moved
  const auto find = [&](int i, unsigned& from, unsigned& to) {
    if (i >= kept) return false;
    const int p = a.path[static_cast<long long>(b) * a.L + i];
    if (p < 0 || p >= a.T) {
      atomicOr(a.err, kErrBadPage);
      return false;
    }
    const long long src = base + p, dst = base + i;
    if (p == i || src < 0 || dst < 0) return false;
    if (src >= cap || dst >= cap) {
      atomicOr(a.err, kErrBadPage);
      return false;
    }
    const int* table = a.table + static_cast<long long>(b) * a.max_pages;
    const int ps = table[src >> a.page_shift], pd = table[dst >> a.page_shift];
    if (ps < 0 || ps >= a.num_pages || pd < 0 || pd >= a.num_pages) {
      atomicOr(a.err, kErrBadPage);
      return false;
    }
    const unsigned in = (1u << a.page_shift) - 1;
    from = ((static_cast<unsigned>(ps) * a.H + h) << a.page_shift) + (static_cast<unsigned>(src) & in);
    to = ((static_cast<unsigned>(pd) * a.H + h) << a.page_shift) + (static_cast<unsigned>(dst) & in);
    return true;
  };
  uint4 x[kEach];
  uint4* put[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = threadIdx.x + k * kMoveThreads, c = i % (kPieces / 2);
    const bool value = i / (kPieces / 2) & 1;
    unsigned from, to;
    put[k] = nullptr;
    if (find(i / kPieces, from, to)) {
      uint4* codes = reinterpret_cast<uint4*>(value ? a.v_codes : a.k_codes);
      x[k] = codes[static_cast<size_t>(from) * (D / 16) + c];
      put[k] = codes + static_cast<size_t>(to) * (D / 16) + c;
    }
  }
  float scale = 0.f;
  float* put_scale = nullptr;
  if (threadIdx.x < 2 * kTreeMaxTokens) {
    unsigned from, to;
    if (find(threadIdx.x >> 1, from, to)) {
      float* scales = (threadIdx.x & 1) ? a.v_scales : a.k_scales;
      scale = scales[from];
      put_scale = scales + to;
    }
  }
  __syncthreads();  // every row of the path has been read
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (put[k] != nullptr) *put[k] = x[k];
  if (put_scale != nullptr) *put_scale = scale;
}

}  // namespace

cudaError_t launch_draft_tree(const DraftTreeArgs& a, cudaStream_t s) {
  return launch_early(draft_tree_kernel, (a.B + kWarpsPerBlock - 1) / kWarpsPerBlock, 32 * kWarpsPerBlock, 0, s, a);
}

cudaError_t launch_kv_keep(const KvKeepArgs& a, int D, cudaStream_t s) {
  return launch_early(D == 64 ? kv_keep_kernel<64> : kv_keep_kernel<128>, a.B * a.H, kMoveThreads, 0, s, a);
}

}  // namespace qat
