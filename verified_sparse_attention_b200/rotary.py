"""Rotary positions: a rotation plan over vattn_rope_init / vattn_rotate.

Marshalling and argument checks only; the kernels are in libvattn.so.
"""
import torch

from . import _abi

_DTYPES = {torch.float32: _abi.VATTN_FP32, torch.bfloat16: _abi.VATTN_BF16}
_LAYOUTS = {"half": _abi.VATTN_ROPE_HALF, "interleaved": _abi.VATTN_ROPE_INTERLEAVED}
_SCALINGS = {"none": _abi.VATTN_ROPE_NONE, "linear": _abi.VATTN_ROPE_LINEAR, "base": _abi.VATTN_ROPE_BASE,
             "bands": _abi.VATTN_ROPE_BANDS, "yarn": _abi.VATTN_ROPE_YARN}


class Rotary:
    """How a head's components turn with the position (the formulas: include/vattn.h).

    head_dim 64 or 128; the first rot_dim components turn (default: all). layout
    "half" pairs (i, i + rot_dim/2), "interleaved" pairs (2i, 2i+1). scaling
    "none", "linear", "base", "bands" or "yarn" stretches contexts of original_ctx
    by `factor`; amplitude None is the scaling's own.
    """

    def __init__(self, *, head_dim, rot_dim=None, layout="half", base=10000.0, scaling="none", factor=1.0,
                 original_ctx=8192, low=1.0, high=4.0, slow=1.0, fast=32.0, amplitude=None):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout {layout!r}: one of {sorted(_LAYOUTS)}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling {scaling!r}: one of {sorted(_SCALINGS)}")
        if amplitude is not None and not amplitude > 0:
            raise ValueError("amplitude must be positive")
        self.head_dim = head_dim
        self.rot_dim = head_dim if rot_dim is None else rot_dim
        self.plan = _abi.vattn_rope_init(dict(
            head_dim=head_dim, rot_dim=self.rot_dim, layout=_LAYOUTS[layout], scaling=_SCALINGS[scaling], base=base,
            factor=factor, original_ctx=original_ctx, low=low, high=high, slow=slow, fast=fast,
            amplitude=0.0 if amplitude is None else amplitude))

    def rotate(self, x, positions, out=None, transpose=False, stream=None):
        """x [tokens, heads, head_dim] rotated to positions [tokens] (int32, on x's device).

        x may be strided over tokens and heads. out: a tensor like x (x itself to
        rotate in place); new and contiguous by default. transpose: the transposed
        rotation, which turns the gradient of the result into that of x. Autograd
        neither records the call nor sees that out was written; an x that it would
        have to follow is refused (pass x.detach(), or call under torch.no_grad()).
        """
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError("x requires a gradient, and autograd does not record this call: pass x.detach() and rotate "
                             "the result's gradient with transpose=True")
        shape, strides, index = x.shape, x.stride(), x.get_device()
        dtype = _DTYPES.get(x.dtype)
        if len(shape) != 3 or shape[2] != self.head_dim or strides[2] != 1 or dtype is None or index < 0:
            raise ValueError(f"x must be float32 or bfloat16 [tokens, heads, {self.head_dim}] on a CUDA device, with "
                             "contiguous components")
        tokens, heads, _ = shape
        if positions.dtype is not torch.int32 or positions.shape != (tokens,) or not positions.is_contiguous() \
                or positions.get_device() != index:
            raise ValueError("positions must be contiguous int32 [tokens] on x's device")
        if out is None:
            out = _abi.empty_for(stream, (tokens, heads, self.head_dim), dtype=x.dtype, device=x.device)
        elif out.shape != shape or out.dtype is not x.dtype or out.get_device() != index or out.stride(2) != 1:
            raise ValueError("out must be like x")
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(index)
        args = (self.plan, x, out, positions, tokens, heads, dtype, strides[:2], out.stride()[:2], transpose, stream)
        if index == torch.cuda.current_device():
            _abi.vattn_rotate(*args)
        else:
            with torch.cuda.device(index):
                _abi.vattn_rotate(*args)
        return out
