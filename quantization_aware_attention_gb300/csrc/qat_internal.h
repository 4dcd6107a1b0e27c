// qat_internal.h -- declarations shared by the library's translation units (not ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "qat_attn.h"

namespace qat {

constexpr long long kMaxRows = 2147483647LL;  // rows of a [B*H*N, D] view
constexpr int kMaxBH = 65535;                   // grid y dimension

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Size and mode checks shared by the forward and backward entry points.  Sets *empty
// when there is no query work (B, H or Nq is zero).
inline qat_status_t check_sizes(int B, int H, int Nq, int Nkv, int D, float sm_scale, int causal,
                                int quant_mode, bool* empty) {
  *empty = false;
  if (B < 0 || H < 0 || Nq < 0 || Nkv < 0) return QAT_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return QAT_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !isfinite(sm_scale)) return QAT_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return QAT_ERR_INVALID_ARG;
  if (quant_mode != QAT_QUANT_NONE && quant_mode != QAT_QUANT_P_FP8E4M3_ROW_TILE64 &&
      quant_mode != QAT_QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD)
    return QAT_ERR_INVALID_ARG;
  if (B == 0 || H == 0) {
    *empty = true;
    return QAT_OK;
  }
  if (Nkv < 1) return QAT_ERR_INVALID_ARG;
  const long long bh = static_cast<long long>(B) * H;
  if (bh * Nq > kMaxRows || bh * Nkv > kMaxRows) return QAT_ERR_INVALID_ARG;
  if (bh > kMaxBH) return QAT_ERR_UNSUPPORTED;
  if (causal && Nq != Nkv) return QAT_ERR_UNSUPPORTED;
  if (Nq == 0) *empty = true;
  return QAT_OK;
}

// Backward workspace, each piece 256-byte aligned; query rows are padded per head to a
// multiple of 128:
//   lse_pad, delta   fp32 [B, H, Nq_pad]
//   lse_ext, d_ext   bf16 [B, H, Nq_pad, 16]: -lse / qk_scale and -Delta of each row as
//                    the exact sum of three bf16 terms (elements 0-2, the rest zero)
//   ones             bf16 [128, 16]: 1 in elements 0-2 of every row
// The dK/dV kernel multiplies ones by lse_ext (d_ext) in one extra MMA k-step, so its
// score accumulators come out as S^T - lse / qk_scale and dP^T - Delta.
// With the non-causal dK/dV work cut into ranges (bwd_stream_k_ctas returns G > 0), the
// layout ends with the segments' partial sums, two slots per CTA:
//   part             fp32 [2G][2][128][D], [slot][0] = dV and [slot][1] = dK / sm_scale
struct BwdWorkspace {
  size_t nq_pad, off_lse, off_delta, off_lse_ext, off_d_ext, off_ones, off_part, total;
};

inline BwdWorkspace bwd_workspace_layout(int B, int H, int Nq, int Nkv, int D, int sk_ctas) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  BwdWorkspace w;
  w.nq_pad = (static_cast<size_t>(Nq) + 127) / 128 * 128;
  const size_t rows_pad = static_cast<size_t>(B) * H * w.nq_pad;
  w.off_lse = 0;
  w.off_delta = up(rows_pad * sizeof(float));
  w.off_lse_ext = w.off_delta + up(rows_pad * sizeof(float));
  w.off_d_ext = w.off_lse_ext + up(rows_pad * 32);
  w.off_ones = w.off_d_ext + up(rows_pad * 32);
  w.off_part = w.off_ones + up(128 * 32);
  const size_t part = sk_ctas > 0 ? static_cast<size_t>(sk_ctas) * 2 * 2 * 128 * D * sizeof(float) : 0;
  w.total = w.off_part + up(part);
  if (w.total == 0) w.total = 256;
  return w;
}

// Work split of the non-causal dK/dV kernel.  One CTA runs per SM, so with few (head,
// 128-key block) items the last wave runs ragged: B1 H40 Nkv512 has 160 items of 128
// query blocks each, and 8 CTAs ran two while the rest idled half the time.  Then the
// kernel runs stream-K: the items' (key block, query block) units, in head-major item
// order, are cut into G equal contiguous ranges, one per CTA.  A CTA walks its range
// item by item; an item cut by a range boundary is done in segments, each of which
// stores fp32 partial sums of dV and dK (the CTA's first segment in slot 2c, its last in
// 2c + 1), and one more kernel adds an item's segments in CTA order, so the result stays
// deterministic.  Each range has at least 4 units.  The choice compares estimated
// makespans for 152 SMs, from the sizes alone, so the workspace size is a function of
// the sizes too: ~2 blocks of fixed cost per item without the split, ~5 per segment with
// it (measured: B1 H24 N4608 ran 9% and B2 H8 Nq4096 Nkv1024 17% slower split, where ~2
// per segment had predicted a gain).  With many items the
// ragged wave costs little and the head-major item order, which keeps the CTAs running
// together on one head's Q and dO in L2, is kept: returns 0.
inline int bwd_stream_k_ctas(int B, int H, int Nq, int Nkv) {
  constexpr long long kSms = 152, kMinSeg = 4;
  const long long items = static_cast<long long>(B) * H * ((Nkv + 127) / 128);
  const long long M = (Nq + 127) / 128;
  if (items <= 0 || M < 2) return 0;
  const long long W = items * M;
  if (W > (1ll << 30)) return 0;  // the kernel's range arithmetic is 32-bit
  long long G = W / kMinSeg;
  if (G > kSms) G = kSms;
  if (G < 1) return 0;
  const double classic = static_cast<double>((items + kSms - 1) / kSms) * (M + 2);
  const double per_cta = static_cast<double>(W) / G;
  const double split = per_cta + 5.0 * (per_cta / M + 2.0);
  return split < 0.95 * classic ? static_cast<int>(G) : 0;
}

// [BH, N, D] bf16 viewed as a 3-D TMA tensor (D innermost), 64 x 128 x 1 boxes,
// 128-byte swizzle, zero fill out of bounds.
bool make_bf16_map_3d(CUtensorMap* m, const void* ptr, int D, int N, int BH,
                      int head_rows = -1);
// [BH, N, 16] bf16 as a 3-D TMA tensor with 16 x 128 x 1 boxes, 32-byte swizzle.
bool make_ext_map_3d(CUtensorMap* m, const void* ptr, int N, int BH);

// Arguments of one forward launch (device pointers, validated by the ABI layer).
struct FwdArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* o_q;
  uint16_t* o_hp;
  float* lse;
  int B, H, Nq, Nkv, D;
  float sm_scale;
  float qk_scale;  // sm_scale * log2(e)
  int causal;
  int quant;
  int window, sinks;  // window > 0 (causal only): key j also needs j > i - window or j < sinks;
                      // both at most Nkv
  int kv_head_rows;  // rows between consecutive heads in K/V memory (Nkv unless a chunk)
  float* o_q_f32;    // when set (with o_hp_f32), fp32 outputs replace the bf16 ones; windows: o_hp_f32 alone
  float* o_hp_f32;
};

// Arguments of one backward launch.
struct BwdArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* o_hp;
  const float* lse;
  const uint16_t* dO;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  float* delta;     // fp32 [B, H, Nq_pad] in the workspace (0 in padding rows)
  float* lse_pad;   // fp32 [B, H, Nq_pad] copy of lse (+inf in padding rows)
  uint16_t* lse_ext;  // bf16 [B, H, Nq_pad, 16] (see BwdWorkspace)
  uint16_t* d_ext;    // bf16 [B, H, Nq_pad, 16]
  uint16_t* ones;     // bf16 [128, 16]
  const float* o_f32; // windows: O_hp, then o_hp is null (null: o_hp)
  float* part;        // dK/dV segment sums (BwdWorkspace::off_part) when sk_ctas > 0, or of the
                      // sinks' key blocks when sink_pieces > 1
  const float* k_mean;  // fp32 [D] or null: smooth_k's channel mean (dQ's SMOOTH_K term)
  int sk_ctas;        // 0, or the stream-K CTA bound of bwd_stream_k_ctas (non-causal)
  int B, H, Nq, Nkv, D;
  float sm_scale;
  float qk_scale;
  int causal;
  int window, sinks;  // as FwdArgs
  int sink_pieces;    // window_sink_pieces
  int page_bwd;     // 1: dV from quantized P and Delta from the O passed (O_q)
};

// Sliding windows.  A 128-row query block mt sees the key blocks first .. mt of its rows' windows, and the
// sinks' blocks 0 .. sinks - 1 before them: `count` in all, taken from the diagonal down, so that every
// row has seen a key (its own) after the first and its running maximum is finite from then on.
struct WindowBlocks {
  int first, mt, sinks, count;
#ifdef __CUDACC__
  __device__ __forceinline__ WindowBlocks(int mt_, int window, int sink_keys) : mt(mt_) {
    first = max(mt * 128 + 1 - window, 0) >> 7;
    sinks = min((sink_keys + 127) >> 7, first);
    count = mt - first + 1 + sinks;
  }
  __device__ __forceinline__ int at(int j) const {
    const int inside = mt - first + 1;
    return j < inside ? mt - j : inside + sinks - 1 - j;
  }
#endif
};

#ifdef __CUDACC__
// Ones in bits [from, to), both clamped to 0 .. 64.
__device__ __forceinline__ unsigned long long ones(int from, int to) {
  from = min(max(from, 0), 64);
  to = min(max(to, 0), 64);
  if (to <= from) return 0ull;
  return (~0ull >> (64 - to)) & (~0ull << from);
}
// The keys key0 .. key0 + 63 that a windowed row sees, as bits: one test for each key in place of three comparisons,
// in the two or three blocks of a row that an edge crosses.  B4 H32 N8192 D128 W1024, comparisons / bits: with 4 sinks
// forward 917 / 830 us, backward 1949 / 1852; without sinks 830 / 779 and 1806 / 1734.
__device__ __forceinline__ unsigned long long window_seen(int row, int key0, int window, int sinks, int keys) {
  const int end = min(keys, row + 1) - key0;
  return ones(row + 1 - window - key0, end) | ones(0, min(sinks - key0, end));
}
#endif

// Key blocks of 128 that hold sinks, whose dK and dV sum over all later queries, not a window's: where they are
// few, each is cut into this many pieces of query blocks, whose fp32 sums one more kernel adds in order.  (Every
// CTA gets as many items as the others: with pieces of a quarter of an SM's share of the work, 8 heads of 32768
// tokens with windows of 4096 and 64 sinks took 15 percent longer than without sinks, of which there are 3.)
// A piece has about as many query blocks as another key block's windows, or a 32nd of an SM's share of the work if
// that is more, but 10 blocks if a 16th of the share is (backward, us, with a 16th / this: B4 H32 N8192 D128 W1024 S4
// 1870 / 1803, B1 H8 N131072 D64 W512 S4 1085 / 1040; with a 32nd alone B1 H8 N65536 D128 W512 S4 742 / 780).  None
// is empty, and their sums take at most 1216 slots (160 MB at D 128).
inline int window_sink_pieces(int B, int H, int N, int window, int sinks) {
  const double heads = static_cast<double>(B) * H;
  const int M = (N + 127) / 128, blocks = (sinks + 127) / 128;
  if (blocks == 0) return 1;
  const int each = (window + 254) / 128 < M ? (window + 254) / 128 : M;  // query blocks that see a key block
  if (heads * blocks >= 4 * 152) return 1;
  const double share = heads * (static_cast<double>(blocks) * M + static_cast<double>(M - blocks) * each) / 152.0;
  double piece = share / 32.0;
  if (piece < 10.0) piece = share / 16.0 < 10.0 ? share / 16.0 : 10.0;
  if (piece < each) piece = each;
  int most = static_cast<int>(1216 / (heads * blocks));
  if (most > M - blocks + 1) most = M - blocks + 1;
  const int want = static_cast<int>(ceil(M / (piece < 4.0 ? 4.0 : piece)));
  return want < most ? want : most;
}
inline size_t window_part_bytes(int B, int H, int N, int D, int window, int sinks) {
  const int n = window_sink_pieces(B, H, N, window, sinks);
  if (n <= 1) return 0;
  return static_cast<size_t>(B) * H * ((sinks + 127) / 128) * n * 2 * 128 * D * sizeof(float);
}

// Bits of the device error word: a bounded wait expired; a page index or a sequence length that
// the cache or its table cannot hold.
constexpr unsigned int kErrTimeout = 1u;
constexpr unsigned int kErrBadPage = 2u;

// One of the two tensors of the norm + rotation pass ([B, H, N, D] by element strides; D
// innermost).  H = 0: absent.
struct NormRopeTensor {
  const uint16_t* x;
  long long sb, sh, sn;
  const uint16_t* dy;  // backward only
  long long dy_sb, dy_sh, dy_sn;
  uint16_t* y;         // forward: contiguous output; backward: dx with the strides below
  long long y_sb, y_sh, y_sn;
  const void* w;       // [D] or null: no norm
  void* dw;            // [D] or null
  int H;
  int log_tokens;      // a warp holds rows of 2^log_tokens tokens at once; filled in by the launcher
};

struct NormRopeArgs {
  NormRopeTensor q, k;
  const int* positions;
  long long pos_sb;
  const unsigned long long* phases;  // [R / 2]
  int B, N, R, interleaved, w_bf16;
  long long tokens;                  // B * N
  float amplitude, eps;
  float* part;                       // backward: [blocks][D]
  // work split, filled in by the launcher
  int heads_per_part, q_parts, parts, q_blocks;
};

// Most blocks of the backward of the norm + rotation (its workspace holds D sums for each).
constexpr int kNormRopeBwdBlocks = 608;  // 152 SMs x 4

// Division of x < 2^31 by a divisor known on the host: with s = ceil(log2 d) and
// m = ceil(2^(31 + s) / d) < 2^32, x / d = floor(x m / 2^(31 + s)), as x m / 2^(31 + s) exceeds x / d by
// x / 2^(31 + s) < 1 / d at most.
struct FastDiv {
  unsigned m, s;
  FastDiv() = default;
  explicit FastDiv(unsigned d) : m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<unsigned>(((1ull << (31 + s)) + d - 1) / d);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ unsigned operator()(unsigned x) const {
    return static_cast<unsigned>((static_cast<unsigned long long>(x) * m) >> 31 >> s);
  }
#endif
};

// Append to and read from the FP8 cache.
struct KvCacheArgs {
  const uint16_t *k, *v;             // append: [B, H, N, D] by element strides
  long long k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;
  uint16_t *k_out, *v_out;           // read: contiguous [B, H, N, D]
  uint8_t *k_codes, *v_codes;        // [pages, H, page, D]
  float *k_scales, *v_scales;        // [pages, H, page]
  const int* table;                  // [B, max_pages]
  const int* seq_lens;               // [B]
  const int* new_lens;               // append: [B] or null
  unsigned int* err;
  int B, H, N, begin, num_pages, page_shift, max_pages;
  FastDiv by_n, by_h;
};

// The attention of a few new tokens over the FP8 cache.
struct DecodeArgs {
  const uint16_t* q;                 // [B, Hq, T, D]
  const uint8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  const int* table;
  const int* seq_lens;
  uint16_t* o;                       // [B, Hq, T, D]
  float* lse;                        // [B, Hq, T] or null
  void* ws;
  unsigned int* err;
  int B, Hq, Hkv, T, num_pages, page_shift, max_pages, quant;
  float qk_scale;                    // sm_scale * log2(e)
  int window, sinks;                 // window 0: every key before a row's own; else as FwdArgs, by positions
  const unsigned long long* tree;    // drafted tokens' masks, or null: sequence b's begin at tree + b tree_sb
  long long tree_sb;
};

constexpr int kTreeMaxTokens = 64;     // bits of a mask

// Masks and positions of drafted trees; sequence b's parents begin at parents + b parents_sb.
struct DraftTreeArgs {
  const int* parents;
  long long parents_sb;
  const int* seq_lens;
  unsigned long long* tree;          // [B, T]
  int* positions;                    // [B, T]
  int B, T;
};

// The move of accepted drafted rows behind the text.
struct KvKeepArgs {
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  const int* table;
  const int* seq_lens;
  const int* path;                   // [B, L]
  const int* path_lens;              // [B]
  int* new_lens;                     // [B]
  unsigned int* err;
  int B, H, T, L, num_pages, page_shift, max_pages;
};
constexpr int kDecodeMaxBatch = 4096;  // the kernel keeps the batch's prefix sums in shared memory
constexpr int kDecodeMaxTokens = 16;
size_t decode_workspace_bytes(int R, int D);  // R = Hq / Hkv * T, at most 16 of them
// A tree of R = Hq / Hkv * T rows is the tensor core's (attn_tree_sm100.cu) and not decode_kernel's: see launch_decode.
inline bool tree_is_wide(long long R, int D) { return R > (D == 64 ? 64 : 32); }
size_t tree_workspace_bytes(int R, int D);    // of the tensor core's kernel

#ifdef __CUDACC__
// Launches a kernel that may be brought up while the stream's previous kernel still runs: it begins with
// after_previous(), which waits for that kernel's end and memory, and lets the next one be brought up in
// turn.  In a serving step's chain of kernels of a few microseconds that hides a launch each.
// Such a kernel reads its inputs by plain or L2 loads: the read-only path may only be used for what does not
// change between the kernel's start, which is before the wait, and its end.  launch_cluster: with clusters of
// n blocks along x.
template <class... Par, class... Arg>
cudaError_t launch_cluster(int n, void (*kernel)(Par...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                           const Arg&... arg) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = n;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = n > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, arg...);
}
template <class... Par, class... Arg>
cudaError_t launch_early(void (*kernel)(Par...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         const Arg&... arg) {
  return launch_cluster(1, kernel, grid, block, smem, s, arg...);
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// Kernel launchers (return cudaGetLastError() after the launches).
cudaError_t launch_norm_rope(NormRopeArgs a, int D, int num_sms, cudaStream_t s);
cudaError_t launch_norm_rope_bwd(NormRopeArgs a, int D, int num_sms, cudaStream_t s);
cudaError_t launch_kv_append(const KvCacheArgs& a, int D, cudaStream_t s);
cudaError_t launch_kv_read(const KvCacheArgs& a, int D, cudaStream_t s);
cudaError_t launch_draft_tree(const DraftTreeArgs& a, cudaStream_t s);
cudaError_t launch_kv_keep(const KvKeepArgs& a, int D, cudaStream_t s);
cudaError_t launch_tree(const DecodeArgs& a, int D, int num_sms, cudaStream_t s);
cudaError_t launch_decode(const DecodeArgs& a, int D, int num_sms, cudaStream_t s);
cudaError_t launch_fwd_tc(const FwdArgs& a, unsigned int* err, int num_sms, cudaStream_t s);
// prep + dK/dV + dQ kernels
cudaError_t launch_bwd_tc(const BwdArgs& a, unsigned int* err, int num_sms, cudaStream_t s);
cudaError_t launch_bwd_dq(const BwdArgs& a, unsigned int* err, int num_sms, cudaStream_t s);
cudaError_t launch_channel_mean(const uint16_t* x, float* mean, long long rows, int D,
                                int num_sms, cudaStream_t s);
cudaError_t launch_fake_quant_tokens(const uint16_t* x, const float* mean, uint16_t* out,
                                     float* scales, int BH, int N, int D, cudaStream_t s);
cudaError_t launch_subtract_mean(const uint16_t* x, const float* mean, uint16_t* out,
                                 long long rows, int D, int num_sms, cudaStream_t s);
cudaError_t launch_merge(float* o_q_acc, float* o_hp_acc, float* lse_acc, const float* o_q_part,
                         const float* o_hp_part, const float* lse_part, uint16_t* o_q_out,
                         uint16_t* o_hp_out, long long rows, int D, int num_sms, cudaStream_t s);
cudaError_t launch_debug_quant(const float* p, int rows, int cols, float* deq,
                               float* scales, uint8_t* codes, cudaStream_t s);

// Causal work order.  A causal item (one head x one 128-row block) has between 1 and M
// blocks of work, so the persistent kernels take the longest items first.  Heads are
// taken in groups: inside a group the length classes descend and the group's heads
// alternate within a class, so the CTAs running together touch only a group or two of
// heads and the K/V (or Q/dO) blocks they all stream stay in L2.  With every head in
// one group the order is pure longest-first, which leaves a wave on as many heads as
// there are CTAs and has each CTA fetch its head's blocks from DRAM.
inline int causal_head_group(long long bytes_per_head, int BH) {
  constexpr long long kGroupBytes = 32ll << 20;  // a wave spans about two groups of L2
  long long g = kGroupBytes / (bytes_per_head > 0 ? bytes_per_head : 1);
  if (g < 1) g = 1;
  if (g > BH) g = BH;
  return static_cast<int>(g);
}

#ifdef __CUDACC__
// Item idx of that order -> head bh and length class cls (0 = the longest, M blocks).
__device__ __forceinline__ void causal_item(int idx, int BH, int M, int hgroup, int& bh,
                                            int& cls) {
  const int per = hgroup * M;
  const int gi = idx / per;
  const int h0 = gi * hgroup;
  const int hs = min(hgroup, BH - h0);
  const int j = idx - gi * per;
  cls = j / hs;
  bh = h0 + (j - cls * hs);
}
#endif

// Device-side error word (bounded waits set it); defined in qat_api.cu.
cudaError_t read_and_clear_device_error(unsigned int* out, cudaStream_t s);
// Device address of that word (the first member of the library's device state, looked
// up on every call, so a context created after cudaDeviceReset gets its own) and the SM
// count of the current device (cached).
cudaError_t device_context(unsigned int** err, int* num_sms);

}  // namespace qat
