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
from .attention import _raise, device_guard


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


def rows_strides(t, name, device, shape):
    """The element strides {b, h, n} of a bf16 [B, H, N, D] tensor that the kernels can read in place
    (D innermost, rows on 16-byte boundaries), None when it is contiguous.  ``shape`` is what it has
    to be, or None."""
    if (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.device == device
            and (t.shape == shape or (shape is None and t.dim() == 4)) and not t.data_ptr() & 15):
        if t.is_contiguous():
            return None
        b, h, n, d = t.stride()
        if d == 1 and not (b | h | n) & 7:
            return b, h, n
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, D], got shape {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not readable(t):
        raise ValueError(f"{name} must have D innermost and rows on 16-byte boundaries, got strides "
                         f"{t.stride()}")
    return t.stride()[:3]


def readable(t) -> bool:
    """Whether the kernels can read t [B, H, N, D] in place."""
    if t.data_ptr() & 15:
        return False
    if t.is_contiguous():
        return True
    st, s = t.stride(), t.shape
    return st[3] == 1 and all(n <= 1 or x % 8 == 0 for n, x in zip(s[:3], st[:3]))


def _operands(q, k, positions, rope, q_weight, k_weight):
    """Checks them; returns (device, q's strides, k's, B, Hq, Hk, N, D, the positions' stride)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor (this library has no CPU path)")
    dev = q.device
    qs = rows_strides(q, "q", dev, None)
    B, Hq, N, D = q.shape
    if D != 64 and D != 128:
        raise ValueError(f"the head dimension must be 64 or 128, got {D}")
    Hk, ks = 0, None
    if k is not None:
        Hk = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 4 else -1
        ks = rows_strides(k, "k", dev, (B, Hk, N, D))
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight go together")
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    if q_weight is not None:
        wtype = q_weight.dtype if isinstance(q_weight, torch.Tensor) else None
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is None:
                continue
            if not isinstance(w, torch.Tensor) or w.device != dev:
                raise ValueError(f"{name} must be a tensor on {dev}")
            if w.dtype is not wtype or (wtype is not torch.float32 and wtype is not torch.bfloat16):
                raise ValueError("the weights must both be torch.float32 or torch.bfloat16")
            if w.shape != (D,) or not w.is_contiguous() or w.data_ptr() & 15:
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
        if positions.dtype is not torch.int32:
            raise ValueError(f"positions must be torch.int32, got {positions.dtype}")
        if positions.shape == (B, N):
            if B > 1:
                pos_stride = positions.stride(0)
        elif positions.shape != (N,):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {(N,)} or "
                             f"{(B, N)}")
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous along the tokens")
    return dev, qs, ks, B, Hq, Hk, N, D, pos_stride


def _tail(rope):
    if rope is None:
        return None, 0, 0, 1.0
    return rope.phases, rope.rotary_dim, 1 if rope.layout == "interleaved" else 0, rope.amplitude


def _forward(ops, q, k, positions, rope, q_weight, k_weight, eps):
    dev, qs, ks, B, Hq, Hk, N, D, pos_stride = ops
    phases, R, inter, amp = _tail(rope)
    q_out = torch.empty((B, Hq, N, D), dtype=torch.bfloat16, device=dev)
    k_out = None if k is None else torch.empty((B, Hk, N, D), dtype=torch.bfloat16, device=dev)
    with device_guard(dev):
        st = capi.qat_qk_norm_rope(
            q, qs, k, ks, q_out, k_out, positions, pos_stride, phases, q_weight, k_weight,
            q_weight is not None and q_weight.dtype is torch.bfloat16, B, Hq, Hk, N, D, R, inter, amp,
            eps)
    _raise(st, "qat_qk_norm_rope")
    return q_out, k_out


def _backward(ops, q, k, positions, rope, q_weight, k_weight, dq_out, dk_out, eps, workspace=None):
    dev, qs, ks, B, Hq, Hk, N, D, pos_stride = ops
    phases, R, inter, amp = _tail(rope)
    gqs = rows_strides(dq_out, "dq_out", dev, (B, Hq, N, D))
    gks = None if k is None else rows_strides(dk_out, "dk_out", dev, (B, Hk, N, D))

    def grad_of(strides, H):
        if strides is not None and strides[2] > strides[1]:  # heads inner, as a projection writes them
            g = torch.empty((B, N, H, D), dtype=torch.bfloat16, device=dev)
            return g.transpose(1, 2), (N * H * D, D, H * D)
        return torch.empty((B, H, N, D), dtype=torch.bfloat16, device=dev), None

    dq, dqs = grad_of(qs, Hq)
    dk, dks = (None, None) if k is None else grad_of(ks, Hk)
    dwq = dwk = None
    ws_bytes = 0
    if q_weight is not None:
        dwq = torch.empty_like(q_weight)
        dwk = None if k is None else torch.empty_like(k_weight)
        if workspace is None:
            workspace = torch.empty(capi.qat_qk_norm_rope_bwd_workspace_bytes(D), dtype=torch.uint8,
                                    device=dev)
        ws_bytes = workspace.numel()
    with device_guard(dev):
        status = capi.qat_qk_norm_rope_bwd(
            q, qs, k, ks, dq_out, gqs, dk_out, gks, positions, pos_stride, phases, q_weight, k_weight,
            q_weight is not None and q_weight.dtype is torch.bfloat16, dq, dqs, dk, dks, dwq, dwk, B,
            Hq, Hk, N, D, R, inter, amp, eps, workspace, ws_bytes)
    _raise(status, "qat_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def qat_qk_norm_rope_backward(q, k, positions, rope, q_weight, k_weight, dq_out, dk_out,
                              eps: float = 1e-6, workspace: torch.Tensor | None = None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qat_qk_norm_rope`` at its inputs, given those of
    its outputs; None for what is absent.  dq and dk have the inputs' order in memory.  ``workspace``:
    uint8, at least ``capi.qat_qk_norm_rope_bwd_workspace_bytes(D)`` bytes, allocated if None."""
    ops = _operands(q, k, positions, rope, q_weight, k_weight)
    if (k is None) != (dk_out is None):
        raise ValueError("dk_out goes together with k")
    if workspace is not None and (workspace.device != ops[0] or workspace.dtype != torch.uint8
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {ops[0]}")
    return _backward(ops, q, k, positions, rope, q_weight, k_weight, dq_out, dk_out, eps, workspace)


class QKNormRope(torch.autograd.Function):
    """Forward returns the normed and rotated q (and k); nothing but the inputs is saved, the
    backward recomputes the norm."""

    @staticmethod
    def forward(ctx, q, k, positions, rope, q_weight, k_weight, eps):
        ops = _operands(q, k, positions, rope, q_weight, k_weight)
        ctx.save_for_backward(q, k, positions, q_weight, k_weight)
        ctx.rest = ops, rope, eps
        out = _forward(ops, q, k, positions, rope, q_weight, k_weight, eps)
        return out[0] if k is None else out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out=None):
        q, k, positions, q_weight, k_weight = ctx.saved_tensors
        ops, rope, eps = ctx.rest
        if not readable(dq_out):
            dq_out = dq_out.contiguous()
        if dk_out is not None and not readable(dk_out):
            dk_out = dk_out.contiguous()
        dq, dk, dwq, dwk = _backward(ops, q, k, positions, rope, q_weight, k_weight, dq_out, dk_out, eps)
        return dq, dk, None, None, dwq, dwk, None


def qat_qk_norm_rope(q, k=None, positions=None, rope: RopePlan | None = None, q_weight=None,
                     k_weight=None, eps: float = 1e-6):
    """Per-head RMS norm (with ``q_weight`` / ``k_weight``, [D] fp32 or bf16) and rotary positions
    (with ``rope`` and int32 ``positions``, [N] or [B, N]) of q [B, Hq, N, D] and k [B, Hk, N, D]
    (or None), bf16; either step may be left out.  Returns (q, k) contiguous [B, H, N, D], what
    ``attention``, the cache and ``qat_attention_decode`` take (only q when k is None).

    The inputs may have any strides with D innermost and rows on 16-byte boundaries: a slice of a
    fused projection, ``x.view(B, N, H, D).transpose(1, 2)``, is read in place.  Differentiable in q,
    k and the weights; the gradients are deterministic."""
    if torch.is_grad_enabled() and any(
            isinstance(t, torch.Tensor) and t.requires_grad for t in (q, k, q_weight, k_weight)):
        out = QKNormRope.apply(q, k, positions, rope, q_weight, k_weight, eps)
    else:
        ops = _operands(q, k, positions, rope, q_weight, k_weight)
        out = _forward(ops, q, k, positions, rope, q_weight, k_weight, eps)
        if k is None:
            out = out[0]
    return out
