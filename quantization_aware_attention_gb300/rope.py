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
from torch.autograd.function import once_differentiable

from . import capi
from .attention import _raise, check_device_status, _check_enabled, device_guard


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


def _rows(t, name, device, B=None, N=None, D=None, H=None):
    """A bf16 [B, H, N, D] tensor the kernels can read in place (D innermost, rows on 16-byte
    boundaries)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, D], got shape {tuple(t.shape)}")
    s = t.shape
    if (B is not None and (s[0] != B or s[2] != N or s[3] != D)) or (H is not None and s[1] != H):
        raise ValueError(f"{name} has shape {tuple(s)}, expected "
                         f"{(B, 'H' if H is None else H, N, D)}")
    if not _readable(t):
        raise ValueError(f"{name} must have D innermost and rows on 16-byte boundaries, got strides "
                         f"{t.stride()}")


def _readable(t) -> bool:
    if t.is_contiguous():
        return t.data_ptr() % 16 == 0
    st, s = t.stride(), t.shape
    return ((st[3] == 1 or s[3] == 1) and t.data_ptr() % 16 == 0
            and all(n <= 1 or x % 8 == 0 for n, x in zip(s[:3], st[:3])))


def _strides(t):
    return None if t.is_contiguous() else t.stride()[:3]


def _operands(q, k, positions, rope, q_weight, k_weight):
    """Checks them; returns the C call's leading arguments in common (after the tensors)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor (this library has no CPU path)")
    dev = q.device
    _rows(q, "q", dev)
    B, Hq, N, D = q.shape
    if D not in (64, 128):
        raise ValueError(f"the head dimension must be 64 or 128, got {D}")
    Hk = 0
    if k is not None:
        _rows(k, "k", dev, B, N, D)
        Hk = k.shape[1]
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight go together")
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor) or w.device != dev:
            raise ValueError(f"{name} must be a tensor on {dev}")
        if w.dtype not in (torch.float32, torch.bfloat16) or w.dtype != q_weight.dtype:
            raise ValueError("the weights must both be torch.float32 or torch.bfloat16")
        if w.dim() != 1 or w.shape[0] != D or not w.is_contiguous() or w.data_ptr() % 16:
            raise ValueError(f"{name} must be contiguous [{D}] on a 16-byte boundary")
    pos_stride = 0
    if rope is None:
        if positions is not None:
            raise ValueError("positions without a RopePlan")
    else:
        if not isinstance(rope, RopePlan):
            raise TypeError("rope must be a RopePlan or None")
        if rope.phases.device != dev:
            raise ValueError(f"the RopePlan lies on {rope.phases.device}, q on {dev}")
        if rope.rotary_dim > D:
            raise ValueError(f"rotary_dim {rope.rotary_dim} exceeds the head dimension {D}")
        if not isinstance(positions, torch.Tensor) or positions.device != dev:
            raise ValueError(f"positions must be a tensor on {dev}")
        if positions.dtype != torch.int32:
            raise ValueError(f"positions must be torch.int32, got {positions.dtype}")
        shape = tuple(positions.shape)
        if shape not in ((N,), (B, N)):
            raise ValueError(f"positions has shape {shape}, expected {(N,)} or {(B, N)}")
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous along the tokens")
        if len(shape) == 2 and B > 1:
            pos_stride = positions.stride(0)
    return B, Hq, Hk, N, D, pos_stride


def _tail(rope):
    if rope is None:
        return 0, 0, 1.0
    return rope.rotary_dim, int(rope.layout == "interleaved"), rope.amplitude


def _forward(q, k, positions, rope, q_weight, k_weight, eps):
    B, Hq, Hk, N, D, pos_stride = _operands(q, k, positions, rope, q_weight, k_weight)
    R, inter, amp = _tail(rope)
    q_out = torch.empty((B, Hq, N, D), dtype=torch.bfloat16, device=q.device)
    k_out = None if k is None else torch.empty((B, Hk, N, D), dtype=torch.bfloat16, device=q.device)
    with device_guard(q.device):
        st = capi.qat_qk_norm_rope(
            q, _strides(q), k, None if k is None else _strides(k), q_out, k_out, positions, pos_stride,
            None if rope is None else rope.phases, q_weight, k_weight,
            q_weight is not None and q_weight.dtype == torch.bfloat16, B, Hq, Hk, N, D, R, inter, amp,
            eps)
    _raise(st, "qat_qk_norm_rope")
    return q_out, k_out


def qat_qk_norm_rope_backward(q, k, positions, rope, q_weight, k_weight, dq_out, dk_out,
                              eps: float = 1e-6, workspace: torch.Tensor | None = None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qat_qk_norm_rope`` at its inputs, given those of
    its outputs; None for what is absent.  dq and dk have the inputs' order in memory."""
    B, Hq, Hk, N, D, pos_stride = _operands(q, k, positions, rope, q_weight, k_weight)
    R, inter, amp = _tail(rope)
    _rows(dq_out, "dq_out", q.device, B, N, D, Hq)
    if (k is None) != (dk_out is None):
        raise ValueError("dk_out goes together with k")
    if k is not None:
        _rows(dk_out, "dk_out", q.device, B, N, D, Hk)

    def grad_of(x):
        if x is None:
            return None
        if x.stride(2) > x.stride(1):  # heads inner, as a projection writes them
            return torch.empty((B, N, x.shape[1], D), dtype=x.dtype, device=x.device).transpose(1, 2)
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)

    dq, dk = grad_of(q), grad_of(k)
    dwq = None if q_weight is None else torch.empty_like(q_weight)
    dwk = None if k_weight is None else torch.empty_like(k_weight)
    if workspace is None and q_weight is not None:
        workspace = torch.empty(capi.qat_qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8,
                                device=q.device)

    def st(x):
        return None if x is None else _strides(x)

    with device_guard(q.device):
        status = capi.qat_qk_norm_rope_bwd(
            q, st(q), k, st(k), dq_out, st(dq_out), dk_out, st(dk_out), positions, pos_stride,
            None if rope is None else rope.phases, q_weight, k_weight,
            q_weight is not None and q_weight.dtype == torch.bfloat16, dq, st(dq), dk, st(dk), dwq, dwk,
            B, Hq, Hk, N, D, R, inter, amp, eps, workspace,
            0 if workspace is None else workspace.numel())
    _raise(status, "qat_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


class QKNormRope(torch.autograd.Function):
    """Forward returns the normed and rotated q (and k); nothing but the inputs is saved, the
    backward recomputes the norm."""

    @staticmethod
    def forward(ctx, q, k, positions, rope, q_weight, k_weight, eps, check):
        ctx.save_for_backward(q, k, positions, q_weight, k_weight)
        ctx.rope, ctx.eps, ctx.check = rope, eps, check
        out = _forward(q, k, positions, rope, q_weight, k_weight, eps)
        return out[0] if k is None else out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out=None):
        q, k, positions, q_weight, k_weight = ctx.saved_tensors

        def ready(d):
            return d if d is None or _readable(d) else d.contiguous()

        dq, dk, dwq, dwk = qat_qk_norm_rope_backward(q, k, positions, ctx.rope, q_weight, k_weight,
                                                     ready(dq_out), ready(dk_out), ctx.eps)
        if ctx.check:
            check_device_status("qat_qk_norm_rope_bwd")
        return dq, dk, None, None, dwq, dwk, None, None


def qat_qk_norm_rope(q, k=None, positions=None, rope: RopePlan | None = None, q_weight=None,
                     k_weight=None, eps: float = 1e-6, check: bool | None = None):
    """Per-head RMS norm (with ``q_weight`` / ``k_weight``, [D] fp32 or bf16) and rotary positions
    (with ``rope`` and int32 ``positions``, [N] or [B, N]) of q [B, Hq, N, D] and k [B, Hk, N, D]
    (or None), bf16; either step may be left out.  Returns (q, k) contiguous [B, H, N, D], what
    ``attention``, the cache and ``qat_attention_decode`` take (only q when k is None).

    The inputs may have any strides with D innermost and rows on 16-byte boundaries: a slice of a
    fused projection, ``x.view(B, N, H, D).transpose(1, 2)``, is read in place.  Differentiable in q,
    k and the weights; the gradients are deterministic."""
    check = _check_enabled(check)
    grad = torch.is_grad_enabled() and any(
        t is not None and t.requires_grad for t in (q, k, q_weight, k_weight))
    if grad:
        out = QKNormRope.apply(q, k, positions, rope, q_weight, k_weight, eps, check)
    else:
        out = _forward(q, k, positions, rope, q_weight, k_weight, eps)
        if k is None:
            out = out[0]
    if check:
        check_device_status("qat_qk_norm_rope")
    return out
