"""Binding of the operators that train the drafter's head (the C ABI's "training the head" section; layouts
and limits are in dflash2.h): the residual's addition with the root-mean-square norm, the LM head's cross
entropy, their gradients, and the norm of many gradients together with their clipping.

Functions carry the C names.  Each has a plan class that checks its arguments once, binds its buffers and
makes each call a single C call (a loop of steps rewrites the bound tensors in place); the function is a plan
made and called once.  There is no CPU or PyTorch fallback, and nothing here builds an autograd graph: a
gradient is a call of its own.

    s = dflash2_residual_norm(x, gamma, residual=r)                              # {"sum", "y"}
    f = dflash2_lm_head_loss(s["y"], W_vocab, labels)                            # {"loss", "lse"}
    b = dflash2_lm_head_loss_grad(s["y"], W_vocab, labels, f["lse"], weights)    # {"d_hidden", "d_W"}
    g = dflash2_residual_norm_grad(s["sum"], gamma, b["d_hidden"])               # {"dx", "dgamma"}
    norm = dflash2_grad_clip([b["d_W"], g["dgamma"]], max_norm=1.0)["norm"]      # scaled in place
"""
from __future__ import annotations

import ctypes
import math

import torch

from .attention import CACHE_TYPES, _int32, _Plan, _ref
from .dflash2 import LossDims, NormDims, TensorArgs, _on_stream, _ptr, library

__all__ = [
    "ResidualNormPlan", "ResidualNormGradPlan", "LossWorkspace", "LossPlan", "LossGradPlan", "GradClipPlan",
    "dflash2_residual_norm", "dflash2_residual_norm_grad", "dflash2_lm_head_loss", "dflash2_lm_head_loss_grad",
    "dflash2_grad_clip", "dflash2_residual_norm_grad_workspace_bytes", "dflash2_lm_head_loss_workspace_bytes",
    "dflash2_lm_head_loss_grad_workspace_bytes", "dflash2_grad_clip_workspace_bytes",
]

BF16 = torch.bfloat16
GRAD_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
NORM_KINDS = {"l2": 0, "max": 1}


def _matrix(t, name):
    """The sizes of a CUDA matrix, which the binding takes the others' from."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    return _int32(t.shape[0], name + "'s rows"), _int32(t.shape[1], name + "'s columns")


def _workspace(nbytes, workspace, device):
    """(scratch as a tensor, its address, bytes): 256-byte aligned, not initialised."""
    if workspace is None:
        if nbytes == 0:
            raise ValueError("invalid or unsupported sizes")
        workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.dtype != torch.uint8 or \
            not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor of torch.uint8")
    elif workspace.get_device() != torch.cuda.current_device():
        raise ValueError("workspace is not on the current device")
    off = (-workspace.data_ptr()) % 256
    if workspace.numel() - off < nbytes or nbytes == 0:
        raise ValueError(f"workspace must hold {nbytes} bytes from a 256-byte boundary on")
    scratch = workspace.view(-1)[off:off + nbytes]
    return scratch, scratch.data_ptr(), nbytes


def _apart(inputs, outputs):
    """Refuses outputs that share memory with an input or with one another: (name, tensor) pairs, and an output's
    third is the names of the inputs that it may be itself (the same elements)."""
    def span(t):
        return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()

    spans = [(n, *span(t)) for n, t in inputs if t is not None and t.numel()]
    for name, t, same in outputs:
        if t is None or not t.numel():
            continue
        lo, hi = span(t)
        for other, lo2, hi2 in spans:
            if lo < hi2 and lo2 < hi and not (other in same and (lo, hi) == (lo2, hi2)):
                raise ValueError(f"{name} overlaps {other}")
        spans.append((name, lo, hi))


class ResidualNormPlan(_Plan):
    """dflash2_residual_norm with its buffers bound; calling returns {"sum", "y", "codes", "scale"}, those asked for.

    sum: True (made where there is a residual), False, or the tensor it goes to; y: the same, made if True.
    codes: a type (torch.float8_e4m3fn or torch.int8) or the tensor they go to; scale goes with them."""

    _name = "dflash2_residual_norm"

    @_on_stream
    def __init__(self, x, gamma, *, residual=None, eps: float = 1e-6, sum=True, y=True, codes=None, scale=None,
                 stream=None):
        N, C = _matrix(x, "x")
        dims = NormDims(N, C)
        if sum is True:
            sum = None if residual is None else torch.empty_like(x)
        if y is True:
            y = torch.empty_like(x)
        sum, y = (None if t is False else t for t in (sum, y))
        if isinstance(codes, torch.dtype):
            if codes not in CACHE_TYPES or codes == BF16:
                raise TypeError(f"codes must be torch.float8_e4m3fn or torch.int8, got {codes}")
            codes = torch.empty((N, C), dtype=torch.uint8, device=x.device).view(codes)
        if codes is None and scale is not None:
            raise ValueError("scale without codes")
        if codes is not None:
            if not isinstance(codes, torch.Tensor) or codes.dtype not in CACHE_TYPES or codes.dtype == BF16:
                raise TypeError("codes must be a tensor of torch.float8_e4m3fn or torch.int8")
            scale = torch.empty(N, dtype=torch.float32, device=x.device) if scale is None else scale
        args = (_ref(dims), _ptr(x, BF16, (N, C), "x"), _ptr(residual, BF16, (N, C), "residual"),
                _ptr(gamma, BF16, (C,), "gamma"), float(eps), _ptr(sum, BF16, (N, C), "sum"),
                _ptr(y, BF16, (N, C), "y"), _ptr(codes, None if codes is None else codes.dtype, (N, C), "codes"),
                0 if codes is None else CACHE_TYPES[codes.dtype], _ptr(scale, torch.float32, (N,), "scale"))
        _apart([("x", x), ("residual", residual), ("gamma", gamma)],
               [("sum", sum, ("x", "residual")), ("y", y, ("x", "residual")), ("codes", codes, ()), ("scale", scale, ())])
        outputs = {n: t for n, t in (("sum", sum), ("y", y), ("codes", codes), ("scale", scale)) if t is not None}
        if not outputs:
            raise ValueError("at least one of sum, y and codes must be asked for")
        self._bind(args, (dims, x, residual, gamma), outputs, stream)


def dflash2_residual_norm_grad_workspace_bytes(N: int, C: int) -> int:
    return int(library().dflash2_residual_norm_grad_workspace_bytes(_ref(NormDims(_int32(N, "N"), _int32(C, "C")))))


class ResidualNormGradPlan(_Plan):
    """dflash2_residual_norm_grad with its buffers bound; calling returns {"dx", "dgamma"}; dgamma=False leaves
    it out."""

    _name = "dflash2_residual_norm_grad"

    @_on_stream
    def __init__(self, z, gamma, dy, *, d_sum=None, eps: float = 1e-6, dx=None, dgamma=None, workspace=None,
                 stream=None):
        N, C = _matrix(z, "z")
        dims = NormDims(N, C)
        dx = torch.empty_like(z) if dx is None else dx
        outputs = {"dx": dx}
        ws, ptr, nbytes = None, None, 0
        if dgamma is False:
            dgamma = None
        else:
            dgamma = torch.empty(C, dtype=torch.float32, device=z.device) if dgamma is None else dgamma
            outputs["dgamma"] = dgamma
            ws, ptr, nbytes = _workspace(dflash2_residual_norm_grad_workspace_bytes(N, C), workspace, z.device)
        args = (_ref(dims), _ptr(z, BF16, (N, C), "z"), _ptr(gamma, BF16, (C,), "gamma"), _ptr(dy, BF16, (N, C), "dy"),
                _ptr(d_sum, BF16, (N, C), "d_sum"), float(eps), _ptr(dx, BF16, (N, C), "dx"),
                _ptr(dgamma, torch.float32, (C,), "dgamma"), ptr, nbytes)
        _apart([("z", z), ("gamma", gamma), ("dy", dy), ("d_sum", d_sum)],
               [("dx", dx, ("dy", "d_sum")), ("dgamma", dgamma, ()), ("workspace", ws, ())])
        self._bind(args, (dims, z, gamma, dy, d_sum, ws), outputs, stream)


def _loss_dims(N, H, V):
    return LossDims(_int32(N, "N"), _int32(H, "H"), _int32(V, "V"))


def dflash2_lm_head_loss_workspace_bytes(N: int, H: int, V: int) -> int:
    return int(library().dflash2_lm_head_loss_workspace_bytes(_ref(_loss_dims(N, H, V))))


def dflash2_lm_head_loss_grad_workspace_bytes(N: int, H: int, V: int) -> int:
    return int(library().dflash2_lm_head_loss_grad_workspace_bytes(_ref(_loss_dims(N, H, V))))


class LossWorkspace:
    """Device scratch of dflash2_lm_head_loss and, with `grad`, of dflash2_lm_head_loss_grad too (256-byte aligned, its
    status word zeroed on the current stream when allocated); dflash2_check_device_status takes it.  It serves other
    sizes that need no more (fewer rows may: up to 128 are held twice)."""

    def __init__(self, N: int, H: int, V: int, *, grad: bool = True, device=None):
        n = dflash2_lm_head_loss_workspace_bytes(N, H, V)
        if n == 0:
            raise ValueError(f"invalid or unsupported sizes N={N}, H={H}, V={V}")
        if grad:
            n = max(n, dflash2_lm_head_loss_grad_workspace_bytes(N, H, V))
        self.tensor = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.tensor.data_ptr()) % 256
        self.view = self.tensor[off:off + n]
        self.view[:256].zero_()
        self.nbytes = n

    @property
    def ptr(self) -> int:
        return self.view.data_ptr()


def _head(hidden, W_vocab, labels, workspace, grad):
    """Sizes, checked addresses and workspace that the loss and its gradient share."""
    N, H = _matrix(hidden, "hidden")
    V, _ = _matrix(W_vocab, "W_vocab")
    args = (_ptr(hidden, BF16, (N, H), "hidden"), _ptr(W_vocab, BF16, (V, H), "W_vocab"),
            _ptr(labels, torch.int32, (N,), "labels"))
    need = (dflash2_lm_head_loss_grad_workspace_bytes if grad else dflash2_lm_head_loss_workspace_bytes)(N, H, V)
    if workspace is None:
        workspace = LossWorkspace(N, H, V, grad=grad, device=hidden.device)
    elif workspace.nbytes < need or need == 0:
        raise ValueError("workspace too small for these sizes")
    elif workspace.tensor.get_device() != torch.cuda.current_device():
        raise ValueError("workspace is not on the current device")
    return N, H, V, args, workspace


class LossPlan(_Plan):
    """dflash2_lm_head_loss with its buffers bound; calling returns {"loss", "lse"}."""

    _name = "dflash2_lm_head_loss"

    @_on_stream
    def __init__(self, hidden, W_vocab, labels, *, loss=None, lse=None, workspace: LossWorkspace | None = None,
                 stream=None):
        N, H, V, args, ws = _head(hidden, W_vocab, labels, workspace, False)
        loss, lse = (torch.empty(N, dtype=torch.float32, device=hidden.device) if t is None else t for t in (loss, lse))
        dims = _loss_dims(N, H, V)
        self.workspace = ws
        args = (_ref(dims), *args, _ptr(loss, torch.float32, (N,), "loss"), _ptr(lse, torch.float32, (N,), "lse"),
                ws.ptr, ws.nbytes)
        _apart([("hidden", hidden), ("W_vocab", W_vocab), ("labels", labels)],
               [("loss", loss, ()), ("lse", lse, ()), ("workspace", ws.view, ())])
        self._bind(args, (dims, hidden, W_vocab, labels, ws), {"loss": loss, "lse": lse}, stream)


class LossGradPlan(_Plan):
    """dflash2_lm_head_loss_grad with its buffers bound; calling returns {"d_hidden", "d_W"}; False for either leaves
    it out.  d_W is made as bfloat16, or given as a tensor of bfloat16 or float32."""

    _name = "dflash2_lm_head_loss_grad"

    @_on_stream
    def __init__(self, hidden, W_vocab, labels, lse, grad, *, d_hidden=None, d_W=None,
                 workspace: LossWorkspace | None = None, stream=None):
        N, H, V, args, ws = _head(hidden, W_vocab, labels, workspace, True)
        d_hidden = torch.empty_like(hidden) if d_hidden is None else None if d_hidden is False else d_hidden
        d_W = torch.empty_like(W_vocab) if d_W is None else None if d_W is False else d_W
        if d_hidden is None and d_W is None:
            raise ValueError("d_hidden and d_W are both left out")
        if d_W is not None and (not isinstance(d_W, torch.Tensor) or d_W.dtype not in (BF16, torch.float32)):
            raise TypeError("d_W must be a tensor of torch.bfloat16 or torch.float32")
        dims = _loss_dims(N, H, V)
        self.workspace = ws
        args = (_ref(dims), *args, _ptr(lse, torch.float32, (N,), "lse"), _ptr(grad, torch.float32, (N,), "grad"),
                _ptr(d_hidden, BF16, (N, H), "d_hidden"),
                _ptr(d_W, None if d_W is None else d_W.dtype, (V, H), "d_W"),
                0 if d_W is None else GRAD_TYPES[d_W.dtype], ws.ptr, ws.nbytes)
        _apart([("hidden", hidden), ("W_vocab", W_vocab), ("labels", labels), ("lse", lse), ("grad", grad)],
               [("d_hidden", d_hidden, ()), ("d_W", d_W, ()), ("workspace", ws.view, ())])
        outputs = {n: t for n, t in (("d_hidden", d_hidden), ("d_W", d_W)) if t is not None}
        self._bind(args, (dims, hidden, W_vocab, labels, lse, grad, ws), outputs, stream)


def dflash2_grad_clip_workspace_bytes(n: int) -> int:
    return int(library().dflash2_grad_clip_workspace_bytes(_int32(n, "n")))


def _dense(t, name):
    """Address of a tensor that fills its memory without gaps, in whatever order (a transposed weight's gradient)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on the current device "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.device(...))")
    if t.dtype not in GRAD_TYPES:
        raise TypeError(f"{name} must be one of {[str(d) for d in GRAD_TYPES]}, got {t.dtype}")
    at = 1
    for stride, size in sorted((t.stride(i), t.size(i)) for i in range(t.dim()) if t.size(i) != 1):
        if stride != at and t.numel():
            raise ValueError(f"{name} must fill its memory without gaps")
        at *= size
    return t.data_ptr()


class GradClipPlan(_Plan):
    """dflash2_grad_clip with its tensors bound; calling returns {"norm", "tensors"}: a float32 tensor without
    dimensions (one of a single element may be given) and the clipped gradients, `tensors` themselves or `out`, tensors
    of the same types, shapes and strides.  Without max_norm the norm alone is taken and the gradients stay as they
    are."""

    _name = "dflash2_grad_clip"

    @_on_stream
    def __init__(self, tensors, *, max_norm: float | None = None, kind: str = "l2", out=None, norm=None,
                 workspace=None, stream=None):
        tensors = tuple(tensors)
        if kind not in NORM_KINDS:
            raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}, got {kind!r}")
        if max_norm is None and out is not None:
            raise ValueError("out without max_norm")
        if max_norm is not None and not (math.isfinite(max_norm) and max_norm >= 0):
            raise ValueError("max_norm must be finite and not negative")
        outs = tensors if out is None else tuple(out)
        if len(outs) != len(tensors):
            raise ValueError(f"out must hold {len(tensors)} tensors, got {len(outs)}")
        table = (TensorArgs * max(1, len(tensors)))()
        spans = []
        for i, (t, o) in enumerate(zip(tensors, outs)):
            p = _dense(t, f"tensors[{i}]")
            if o is not t and (_dense(o, f"out[{i}]") is None or o.dtype != t.dtype or o.shape != t.shape or
                               o.stride() != t.stride()):
                raise ValueError(f"out[{i}] must have the type, shape and strides of tensors[{i}]")
            table[i] = TensorArgs(p, None if max_norm is None else o.data_ptr(), t.numel(), GRAD_TYPES[t.dtype])
            nbytes = t.numel() * t.element_size()
            if nbytes:
                spans.append((p, p + nbytes, f"tensors[{i}]"))
                if max_norm is not None and o.data_ptr() != p:
                    spans.append((o.data_ptr(), o.data_ptr() + nbytes, f"out[{i}]"))
        device = tensors[0].device if tensors else torch.device("cuda", torch.cuda.current_device())
        norm = torch.empty((), dtype=torch.float32, device=device) if norm is None else norm
        norm_ptr = _ptr(norm, torch.float32, (1,) if isinstance(norm, torch.Tensor) and norm.dim() else (), "norm")
        spans.append((norm_ptr, norm_ptr + 4, "norm"))
        ws, ptr, nbytes = _workspace(dflash2_grad_clip_workspace_bytes(len(tensors)), workspace, device)
        spans.append((ptr, ptr + nbytes, "workspace"))
        spans.sort()
        for a, b in zip(spans, spans[1:]):
            if b[0] < a[1]:
                raise ValueError(f"{a[2]} and {b[2]} overlap")
        outputs = {"norm": norm}
        if max_norm is not None:
            outputs["tensors"] = outs
        self._bind((table, len(tensors), NORM_KINDS[kind], float(max_norm or 0.0),
                    norm_ptr, ptr, nbytes), (table, tensors, outs, ws), outputs, stream)


def dflash2_residual_norm(x, gamma, *, residual=None, eps: float = 1e-6, sum=True, y=True, codes=None, scale=None,
                          stream=None):
    """z = x + residual, y = z / sqrt(mean(z^2) + eps) * gamma for rows [N, C]; returns the outputs asked for
    (ResidualNormPlan) as a dict."""
    return ResidualNormPlan(x, gamma, residual=residual, eps=eps, sum=sum, y=y, codes=codes, scale=scale,
                            stream=stream)()


def dflash2_residual_norm_grad(z, gamma, dy, *, d_sum=None, eps: float = 1e-6, dx=None, dgamma=None, workspace=None,
                               stream=None):
    """The gradient of dflash2_residual_norm at z, with d_sum added; returns {"dx", "dgamma"}."""
    return ResidualNormGradPlan(z, gamma, dy, d_sum=d_sum, eps=eps, dx=dx, dgamma=dgamma, workspace=workspace,
                                stream=stream)()


def dflash2_lm_head_loss(hidden, W_vocab, labels, *, loss=None, lse=None, workspace=None, stream=None):
    """The cross entropy of labels int32 [N] under hidden [N, H] and W_vocab [V, H], without the logits; rows whose
    label lies outside the vocabulary are ignored.  Returns {"loss", "lse"} float32 [N]."""
    return LossPlan(hidden, W_vocab, labels, loss=loss, lse=lse, workspace=workspace, stream=stream)()


def dflash2_lm_head_loss_grad(hidden, W_vocab, labels, lse, grad, *, d_hidden=None, d_W=None, workspace=None,
                              stream=None):
    """Its gradient, from the forward pass's lse and the gradient of each row's loss; returns {"d_hidden", "d_W"}."""
    return LossGradPlan(hidden, W_vocab, labels, lse, grad, d_hidden=d_hidden, d_W=d_W, workspace=workspace,
                        stream=stream)()


def dflash2_grad_clip(tensors, *, max_norm: float | None = None, kind: str = "l2", out=None, norm=None, workspace=None,
                      stream=None):
    """The norm ("l2" or "max") of all elements of `tensors` together and, with max_norm, the tensors scaled so that
    it is at most that, in place or into `out`; returns {"norm", "tensors"}."""
    return GradClipPlan(tensors, max_norm=max_norm, kind=kind, out=out, norm=norm, workspace=workspace,
                        stream=stream)()
