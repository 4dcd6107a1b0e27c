"""Serving what was trained: the FP8 key/value cache and the attention of new tokens over it.

``KVCache`` quantizes keys and values as they are written to its pages (FP8 E4M3, one absmax scale
per token and head) and reads them back; ``qat_attention_decode`` computes the attention of each
sequence's last tokens over it, with P fake-quantized as in training.  Block tables and lengths are
read on the device, so every call can be captured into a CUDA graph and replayed as they change.
"""

from __future__ import annotations

import torch

from . import capi


class KVCache:
    """Pages of keys and values: ``k`` and ``v`` are torch.float8_e4m3fn [pages, H, page_size, D],
    ``k_scale`` and ``v_scale`` fp32 [pages, H, page_size]; a row's value is its codes times its
    scale.  page_size is 16, 32, 64, 128 or 256, D 64 or 128.

    ``block_table`` (int32 [B, pages per sequence]) and ``seq_lens`` (int32 [B]) place the
    sequences: position i of sequence b is slot i % page_size of page block_table[b, i // page_size].
    Entries outside the cache are never followed: such rows are dropped by ``append``, read as NaN,
    and reported by ``check_device_status`` (or at once with check=True).  ``append`` stores no NaN
    codes; in a cache filled otherwise they count as NaN."""

    def __init__(self, k, v, k_scale, v_scale):
        if not isinstance(k, torch.Tensor) or not k.is_cuda:
            raise ValueError("k must be a CUDA tensor (this library has no CPU path)")
        if k.dim() != 4:
            raise ValueError(f"k must be [pages, H, page_size, D], got shape {tuple(k.shape)}")
        pages, H, page, D = k.shape
        if D not in (64, 128):
            raise ValueError(f"the head dimension must be 64 or 128, got {D}")
        if page not in (16, 32, 64, 128, 256):
            raise ValueError(f"page_size must be 16, 32, 64, 128 or 256, got {page}")
        if pages < 1 or H < 1:
            raise ValueError("a cache has at least one page and one head")
        for name, t, shape, dtype in (("k", k, (pages, H, page, D), torch.float8_e4m3fn),
                                      ("v", v, (pages, H, page, D), torch.float8_e4m3fn),
                                      ("k_scale", k_scale, (pages, H, page), torch.float32),
                                      ("v_scale", v_scale, (pages, H, page), torch.float32)):
            if not isinstance(t, torch.Tensor) or t.device != k.device:
                raise ValueError(f"{name} must be a tensor on {k.device}")
            if t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
            if tuple(t.shape) != shape or not t.is_contiguous() or t.data_ptr() % 16:
                raise ValueError(f"{name} must be contiguous {shape} on a 16-byte boundary, got shape "
                                 f"{tuple(t.shape)}")
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        self.num_pages, self.heads, self.page_size, self.D = pages, H, page, D
        self.device = k.device

    # the tensors the sizes above were checked against
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)

    @classmethod
    def empty(cls, num_pages: int, heads: int, page_size: int, D: int, device="cuda") -> "KVCache":
        """A cache of unwritten pages (their contents are unspecified: nothing past a sequence's
        length is ever used)."""
        def codes():
            return torch.empty((num_pages, heads, page_size, D), dtype=torch.float8_e4m3fn,
                               device=device)

        def scales():
            return torch.empty((num_pages, heads, page_size), dtype=torch.float32, device=device)

        return cls(codes(), codes(), scales(), scales())

    def append(self, k, v, block_table, seq_lens, new_lens=None, check: bool | None = None) -> None:
        """Quantizes new keys and values, bf16 [B, H, N, D] with any strides that have D innermost,
        into their pages.  ``seq_lens`` are the lengths after the append: row n of sequence b goes to
        position seq_lens[b] - N + n, or, with int32 ``new_lens`` [B], to seq_lens[b] - new_lens[b] + n
        for its first new_lens[b] rows (the others are padding; a new_lens above N counts as N).  Rows
        whose position would be negative are dropped.  No two rows may go to one slot."""
        capi.torch_ops().kv_append(self._k, self._v, self._k_scale, self._v_scale, k, v, block_table,
                                   seq_lens, new_lens, check)

    def read(self, block_table, seq_lens, begin: int = 0, length: int | None = None,
             check: bool | None = None):
        """(k, v) of positions [begin, begin + length), bf16 [B, H, length, D] contiguous, zeros behind
        a sequence's end.  Without ``length``: all that the block table can hold."""
        return capi.torch_ops().kv_read(self._k, self._v, self._k_scale, self._v_scale, block_table,
                                        seq_lens, begin, length, check)

    def keep(self, block_table, seq_lens, drafted: int, path, path_lens, check: bool | None = None):
        """After the last ``drafted`` tokens of each sequence were checked: moves the accepted ones' rows behind
        the text before them.  ``path`` (int32 [B, L], L <= drafted <= 64) names drafted tokens in their order in
        the text, the first ``path_lens[b]`` (int32 [B]) of them accepted.  Returns the new lengths, int32
        [B]: seq_lens - drafted + accepted, not below 0.  Rows move as if all were read before one is written; every
        other slot stays as it was.  Entries outside [0, drafted) are not moved and reported as bad
        pages are."""
        return capi.torch_ops().kv_keep(self._k, self._v, self._k_scale, self._v_scale, block_table, seq_lens,
                                        drafted, path, path_lens, check)


def qat_attention_decode(q, cache: KVCache, block_table, seq_lens, sm_scale: float | None = None,
                         quant_mode: int = capi.QUANT_P_FP8E4M3_ROW_TILE64, return_lse: bool = False,
                         workspace: torch.Tensor | None = None, check: bool | None = None,
                         window: int | None = None, sinks: int = 0):
    """Attention of each sequence's last T tokens, q bf16 [B, Hq, T, D], over the cache, which holds
    their own keys and values already: token t is position seq_lens[b] - T + t and sees the keys up to
    its own.  Hq is a multiple of the cache's heads (consecutive query heads share one); T is at most
    16.  Returns o bf16 [B, Hq, T, D], and with ``return_lse`` the base-2 log-sum-exp fp32 [B, Hq, T].
    A row that sees no key gives o = 0, lse = -inf.  The same shapes and lengths give the same bits; a
    block table of another width may round differently.  ``workspace``: uint8, at least
    ``capi.qat_attn_decode_workspace_bytes(Hq, cache.heads, T, D)`` bytes, for one call at a time;
    allocated if None.  ``window``: the token at position i sees only keys j > i - window, and the
    first ``sinks`` keys; nothing else is read, and block table entries of pages that no token sees may be
    anything."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    return capi.torch_ops().decode(cache._k, cache._v, cache._k_scale, cache._v_scale, q, block_table,
                                   seq_lens, None, sm_scale, quant_mode, return_lse, workspace, check, window,
                                   sinks)


def qat_attention_tree(q, cache: KVCache, block_table, seq_lens, tree, sm_scale: float | None = None,
                       quant_mode: int = capi.QUANT_P_FP8E4M3_ROW_TILE64, return_lse: bool = False,
                       workspace: torch.Tensor | None = None, check: bool | None = None,
                       window: int | None = None, sinks: int = 0):
    """Attention of a tree of drafted tokens, q bf16 [B, Hq, T, D] with T up to 64, over the cache: the last T
    slots of each sequence hold their keys and values (appended as they come, seq_lens with them), and
    ``tree`` (int64 [B, T], or [T] for all sequences; from ``qat_draft_tree``) says which of them each token sees:
    bit s of tree[b, t] for token s.  Every token sees the whole text before the tree; with ``window``, only keys
    j > i - window of it, and the first ``sinks``, i being the token's position by its depth, seq_lens[b] - T +
    popcount - 1 (the tree itself is seen by its bits alone, so where a path is longer than the window its tokens see
    ancestors that ``qat_attention_decode`` would leave out).  P's tiles are of 64 slots, so a drafted token's P may
    be quantized in another tile than after ``KVCache.keep``.  Where a KV head has more than 32 query rows (64 channels:
    64) the weights of V are rounded to bf16, else to f16.  Everything else as ``qat_attention_decode``, but that with a
    window the page of key seq_lens - T - window is looked up (a token with an empty mask sees it); the workspace has
    ``capi.qat_attn_tree_workspace_bytes(Hq, cache.heads, T, D)`` bytes."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    if not isinstance(tree, torch.Tensor):
        raise TypeError("tree must be a torch.Tensor")
    return capi.torch_ops().decode(cache._k, cache._v, cache._k_scale, cache._v_scale, q, block_table,
                                   seq_lens, tree, sm_scale, quant_mode, return_lse, workspace, check, window,
                                   sinks)


def qat_draft_tree(parents, seq_lens):
    """(tree, positions) of drafted trees: ``parents`` int32 [B, T] or [T], T up to 64, names for each token the
    earlier one that it continues, -1 for the text (anything else: padding, as is what continues it).  tree
    int64 [B, T] holds each token's own bit and its ancestors' (0 for padding), for ``qat_attention_tree``;
    positions int32 [B, T] are seq_lens - T + depth, for ``qat_qk_norm_rope``.  ``seq_lens`` (int32 [B]) count the
    T tokens, as for the cache."""
    return capi.torch_ops().draft_tree(parents, seq_lens)
