"""Query/key norm and rotary positions in one pass: what makes the q and k that ``attention``
and the key/value cache take, with its backward.

``RopePlan`` holds the rotation's frequencies on the device; ``qat_qk_norm_rope`` applies it,
differentiably.  Angles are exact at every 32-bit position: the plan stores each pair's
frequency as a 64-bit fraction of a turn per position, and the kernel multiplies it by the
position modulo one turn.
"""

from __future__ import annotations

import math

import torch

from . import capi


class RopePlan:
    """The rotation of the first ``rotary_dim`` channels of a head.

    Pair i of rotary_dim / 2 turns by f_i radians per position, f_i = base^(-2i / rotary_dim):
      layout "half"         pairs (i, i + rotary_dim / 2)
      layout "interleaved"  pairs (2i, 2i + 1)
    Scaling for contexts ``factor`` times as long as the trained one:
      "none"
      "linear"  positions divided by factor
      "ntk"     base * factor^(rotary_dim / (rotary_dim - 2))
      "yarn"    pairs that make fewer than ``beta_slow`` turns in ``original_len`` positions are
                divided by factor, those with more than ``beta_fast`` kept, a linear ramp over the
                pairs between; the rotated channels are multiplied by ``amplitude``, by default
                0.1 ln(factor) + 1.
    """

    def __init__(self, rotary_dim: int, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, original_len: int | None = None,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, amplitude: float | None = None,
                 device="cuda"):
        R = int(rotary_dim)
        if R < 16 or R % 16 != 0 or R > 128:
            raise ValueError(f"rotary_dim must be a multiple of 16 in 16..128, got {rotary_dim}")
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
        if scaling not in ("none", "linear", "ntk", "yarn"):
            raise ValueError(f"scaling must be 'none', 'linear', 'ntk' or 'yarn', got {scaling!r}")
        base, factor = float(base), float(factor)
        if not (math.isfinite(base) and base > 1.0):
            raise ValueError(f"base must be finite and above 1, got {base}")
        if not (math.isfinite(factor) and factor >= 1.0):
            raise ValueError(f"factor must be finite and at least 1, got {factor}")
        if scaling == "none" and factor != 1.0:
            raise ValueError("factor applies only together with a scaling")
        self.rotary_dim, self.base, self.layout = R, base, layout
        self.interleaved = layout == "interleaved"
        self.scaling, self.factor = scaling, factor
        self.amplitude = 1.0
        if scaling == "ntk":
            base = base * factor ** (R / (R - 2))
        f = [base ** (-2.0 * i / R) for i in range(R // 2)]
        if scaling == "linear":
            f = [x / factor for x in f]
        elif scaling == "yarn":
            if original_len is None or original_len < 1:
                raise ValueError("yarn needs original_len, the trained context length")
            if not beta_fast > beta_slow > 0:
                raise ValueError("yarn needs beta_fast > beta_slow > 0")

            def pair_of(turns):
                return R * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

            low = max(math.floor(pair_of(beta_fast)), 0)
            high = min(math.ceil(pair_of(beta_slow)), R - 1)
            width = max(high - low, 0.001)
            ramp = [min(max((i - low) / width, 0.0), 1.0) for i in range(R // 2)]
            f = [x / factor * r + x * (1.0 - r) for x, r in zip(f, ramp)]
            self.amplitude = 0.1 * math.log(factor) + 1.0
        if amplitude is not None:
            self.amplitude = float(amplitude)
            if not math.isfinite(self.amplitude):
                raise ValueError("amplitude must be finite")
        self.frequencies = tuple(f)
        bits = [int(x / (2 * math.pi) * 2.0 ** 64) & (2 ** 64 - 1) for x in f]
        self.phases = torch.tensor([b - 2 ** 64 if b >= 2 ** 63 else b for b in bits],
                                   dtype=torch.int64, device=device)
        if not self.phases.is_cuda:
            raise ValueError("device must be a CUDA device (this library has no CPU path)")


def _plan(rope):
    """(phases, rotary_dim, interleaved, amplitude) of a plan, or of none."""
    if rope is None:
        return None, 0, False, 1.0
    if not isinstance(rope, RopePlan):
        raise TypeError("rope must be a RopePlan or None")
    return rope.phases, rope.rotary_dim, rope.interleaved, rope.amplitude


def qat_qk_norm_rope(q, k=None, positions=None, rope: RopePlan | None = None, q_weight=None,
                     k_weight=None, eps: float = 1e-6):
    """Per-head RMS norm (with ``q_weight`` / ``k_weight``, [D] fp32 or bf16) and rotary positions
    (with ``rope`` and int32 ``positions``, [N] or [B, N]) of q [B, Hq, N, D] and k [B, Hk, N, D]
    (or None), bf16; either step may be left out.  Returns (q, k) contiguous [B, H, N, D], what
    ``attention``, the cache and ``qat_attention_decode`` take (only q when k is None).

    The inputs may have any strides with D innermost and rows on 16-byte boundaries: a slice of a
    fused projection, ``x.view(B, N, H, D).transpose(1, 2)``, is read in place.  Differentiable in q,
    k and the weights (once: there is no second derivative, and no forward-mode one); the gradients are
    deterministic, those of q and k in the inputs' order in memory.  Nothing but the inputs is saved for the
    backward.  Forward and backward can be captured into a CUDA graph; while a graph made on the default
    stream lives that ends in the same leaves, or that the backward passes through, that is refused."""
    phases, rotary_dim, interleaved, amplitude = _plan(rope)
    return capi.torch_ops().norm_rope(q, k, positions, phases, q_weight, k_weight, rotary_dim,
                                      interleaved, amplitude, eps)


def qat_qk_norm_rope_backward(q, k, positions, rope, q_weight, k_weight, dq_out, dk_out,
                              eps: float = 1e-6, workspace: torch.Tensor | None = None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qat_qk_norm_rope`` at its inputs, given those of
    its outputs; None for what is absent.  ``workspace``: uint8, at least
    ``capi.qat_qk_norm_rope_bwd_workspace_bytes(D)`` bytes, allocated if None."""
    phases, rotary_dim, interleaved, amplitude = _plan(rope)
    return capi.torch_ops().norm_rope_bwd(q, k, positions, phases, q_weight, k_weight, rotary_dim,
                                          interleaved, amplitude, eps, dq_out, dk_out, workspace)
