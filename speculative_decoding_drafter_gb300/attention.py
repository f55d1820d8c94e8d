"""Binding of the attention-side operators: rotary positions, the paged cache, attention over it
(the C ABI's "attention of the drafter's layers" section; layouts and limits are in dflash2.h).

Functions carry the C names.  Each has a plan class that checks its arguments once, binds its
buffers and makes each call a single C call (a loop of steps rewrites the bound tensors in
place); the function is a plan made and called once.  There is no CPU or PyTorch fallback.

    cache = PagedCache.allocate(pages, page_size=64, heads=8, dim=128, dtype=torch.float8_e4m3fn)
    batch = TokenBatch(token_start, kv_len, page_table, tokens=N, max_new=T)
    table = dflash2_rope_table(max_pos, rot=128)
    dflash2_cache_append(cache, batch, k, v, q=q, q_out=q, table=table)
    out = dflash2_paged_attention(q, cache, batch, causal=False)["out"]
"""
from __future__ import annotations

import ctypes
import math

import torch

from .dflash2 import (AttentionArgs, CacheArgs, DFlash2Error, HeadRows, RopeArgs, RopeScaling, TokenArgs, _check,
                      _on_stream, _ptr, _stream, library)

__all__ = [
    "PagedCache", "TokenBatch", "AttentionWorkspace", "RopePlan", "CacheAppendPlan", "CacheReadPlan",
    "PagedAttentionPlan", "dflash2_rope_table", "dflash2_rope", "dflash2_cache_append", "dflash2_cache_read",
    "dflash2_paged_attention", "dflash2_paged_attention_workspace_bytes",
]

CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}
ROPE_KINDS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3, "band": 4}


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _int32(value, name):
    """A count as the C ABI takes it (ctypes would cut it to 32 bits without a word)."""
    value = int(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def _rows(t, N, heads, dim, name):
    """df2_heads of a bf16 tensor [N, heads, dim] whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on the current device "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.device(...))")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if tuple(t.shape) != (N, heads, dim):
        raise ValueError(f"{name} must have shape {(N, heads, dim)}, got {tuple(t.shape)}")
    if t.numel() and t.stride(2) != 1 and dim > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return HeadRows(t.data_ptr(), _int32(heads, name + "'s heads"), t.stride(0), t.stride(1))


def _heads_of(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [tokens, heads, dim], got {tuple(t.shape)}")
    return t.shape[1]


def _table(table, interleaved):
    if table is None:
        return None
    if not isinstance(table, torch.Tensor) or table.dim() != 3 or table.shape[1] != 2:
        raise ValueError("table must be a float32 tensor [max_pos, 2, rot / 2]")
    shape = tuple(table.shape)
    return RopeArgs(_ptr(table, torch.float32, shape, "table"), _int32(shape[0], "max_pos"),
                    _int32(2 * shape[2], "rot"), int(bool(interleaved)))


class PagedCache:
    """One layer's paged keys and values [pages, heads, page_size, dim]: bfloat16, or float8_e4m3fn / int8
    with float32 scales [pages, heads, page_size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if not isinstance(k, torch.Tensor) or not k.is_cuda:
            raise TypeError("k must be a CUDA tensor")
        if k.dtype not in CACHE_TYPES:
            raise TypeError(f"k must be one of {[str(t) for t in CACHE_TYPES]}, got {k.dtype}")
        if k.dim() != 4:
            raise ValueError(f"k must have shape [pages, heads, page_size, dim], got {tuple(k.shape)}")
        quantised = k.dtype != torch.bfloat16
        if quantised != (k_scale is not None) or quantised != (v_scale is not None):
            raise ValueError("8-bit caches have k_scale and v_scale, bfloat16 caches have none")
        shape = tuple(k.shape)
        self.k, self.v, self.k_scale, self.v_scale = self._keep = k, v, k_scale, v_scale
        pages, heads, page_size, dim = (_int32(n, name) for n, name in zip(shape, ("pages", "heads", "page_size", "dim")))
        self.args = CacheArgs(pages, page_size, heads, dim, CACHE_TYPES[k.dtype], _ptr(k, k.dtype, shape, "k"),
                              _ptr(v, k.dtype, shape, "v"), _ptr(k_scale, torch.float32, shape[:3], "k_scale"),
                              _ptr(v_scale, torch.float32, shape[:3], "v_scale"))

    @classmethod
    def allocate(cls, pages: int, page_size: int, heads: int, dim: int, dtype=torch.bfloat16, device="cuda"):
        """A cache of zeros."""
        shape = (pages, heads, page_size, dim)
        if dtype == torch.bfloat16:
            return cls(torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device))
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
        return cls(k, v, *(torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))

    @property
    def heads(self) -> int:
        return self.args.heads

    @property
    def dim(self) -> int:
        return self.args.dim


class TokenBatch:
    """The new tokens of a batch of sequences: token_start int32 [B + 1], kv_len int32 [B] (new tokens
    included), page_table int32 [B, max_pages]; tokens = token_start[B], no sequence has more than max_new.
    max_new may be larger than tokens (a loop's block length, a short last batch).  It sets how many rows
    attention plans for: give it where sequences have few tokens each, it is taken as `tokens` if not given
    (64 sequences of one token are then planned as one of 64: the same results, slower)."""

    def __init__(self, token_start, kv_len, page_table, *, tokens: int, max_new: int | None = None):
        if not isinstance(kv_len, torch.Tensor) or not kv_len.is_cuda:
            raise TypeError("kv_len must be a CUDA tensor")
        B = kv_len.shape[0] if kv_len.dim() else 0
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be an int32 tensor [B, max_pages]")
        self.token_start, self.kv_len, self.page_table = self._keep = token_start, kv_len, page_table
        self.tokens = _int32(tokens, "tokens")
        max_new = self.tokens if max_new is None else min(_int32(max_new, "max_new"), self.tokens)
        self.args = TokenArgs(_int32(B, "sequences"), self.tokens, max_new,
                              _int32(page_table.shape[1], "max_pages"),
                              _ptr(token_start, torch.int32, (B + 1,), "token_start"),
                              _ptr(kv_len, torch.int32, (B,), "kv_len"),
                              _ptr(page_table, torch.int32, (B, page_table.shape[1]), "page_table"))


def dflash2_paged_attention_workspace_bytes(cache: PagedCache, batch: TokenBatch, q_heads: int) -> int:
    return int(library().dflash2_paged_attention_workspace_bytes(ctypes.byref(cache.args), ctypes.byref(batch.args),
                                                                 _int32(q_heads, "q_heads")))


class AttentionWorkspace:
    """Device scratch of dflash2_paged_attention (256-byte aligned, its status word zeroed on the current
    stream when allocated); dflash2_check_device_status takes it."""

    def __init__(self, cache: PagedCache, batch: TokenBatch, q_heads: int, device=None):
        n = dflash2_paged_attention_workspace_bytes(cache, batch, q_heads)
        if n == 0:
            raise ValueError("invalid or unsupported cache, tokens or q_heads")
        self.tensor = torch.empty(n + 256, dtype=torch.uint8, device=device or cache.k.device)
        off = (-self.tensor.data_ptr()) % 256
        self.view = self.tensor[off:off + n]
        self.view[:256].zero_()
        self.nbytes = n

    @property
    def ptr(self) -> int:
        return self.view.data_ptr()


class _Plan:
    """A C call with its arguments checked and bound.  Calling launches it on the stream the plan was
    given, or else on the current stream of the call, and returns the bound outputs (a dict of its own
    each time).  What is bound stays so, and alive, whatever becomes of names and dicts around it."""

    _name = ""

    def _bind(self, args, keep, outputs, stream):
        self._fn = getattr(library(), self._name)
        self._device = torch.cuda.current_device()
        self._args, self._keep, self.outputs = args, keep, outputs
        self._several = isinstance(outputs, dict)
        self._bound = dict(outputs) if self._several else outputs
        self._handle = None if stream is None else _stream(stream)

    def __call__(self):
        handle = self._handle
        st = self._fn(*self._args, _current_stream(self._device) if handle is None else handle)
        if st:
            raise DFlash2Error(st, self._name)
        return self._bound.copy() if self._several else self._bound


# the raw handle without building a stream object, which costs as much as the launch
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _out_like(x):
    return torch.empty(x.shape, dtype=x.dtype, device=x.device)


class RopePlan(_Plan):
    """dflash2_rope with its buffers bound; calling returns the rotated rows."""

    _name = "dflash2_rope"

    @_on_stream
    def __init__(self, x, positions, table, *, interleaved: bool = False, inverse: bool = False, out=None,
                 stream=None):
        heads = _heads_of(x, "x")
        N, dim = x.shape[0], x.shape[2]
        xr = _rows(x, N, heads, dim, "x")
        pos = _ptr(positions, torch.int32, (N,), "positions")
        rope = _table(table, interleaved)
        if rope is None:
            raise ValueError("table must be a float32 tensor [max_pos, 2, rot / 2]")
        out = _out_like(x) if out is None else out
        yr = _rows(out, N, heads, dim, "out")
        self._bind((_ref(rope), _int32(N, "tokens"), _int32(dim, "dim"), _ref(xr), pos, int(bool(inverse)), _ref(yr)),
                   (rope, xr, yr, x, positions, table), out, stream)


class CacheAppendPlan(_Plan):
    """dflash2_cache_append with its buffers bound; calling returns the cache's tensors (and the rotated
    queries) as a dict."""

    _name = "dflash2_cache_append"

    @_on_stream
    def __init__(self, cache: PagedCache, batch: TokenBatch, k, v, *, q=None, q_out=None, table=None,
                 interleaved: bool = False, stream=None):
        N, dim = batch.tokens, cache.dim
        kr, vr = _rows(k, N, cache.heads, dim, "k"), _rows(v, N, cache.heads, dim, "v")
        qr = qo = None
        outputs = {"k_cache": cache.k, "v_cache": cache.v}
        if cache.k_scale is not None:
            outputs.update(k_scale=cache.k_scale, v_scale=cache.v_scale)
        if q is not None:
            heads = _heads_of(q, "q")
            qr = _rows(q, N, heads, dim, "q")
            q_out = _out_like(q) if q_out is None else q_out
            qo = _rows(q_out, N, heads, dim, "q_out")
            outputs["q"] = q_out
        elif q_out is not None:
            raise ValueError("q_out without q")
        rope = _table(table, interleaved)
        self._bind((_ref(cache.args), _ref(batch.args), _ref(rope), _ref(qr), _ref(qo), _ref(kr), _ref(vr)),
                   (cache, batch, rope, qr, qo, kr, vr, k, v, q, table), outputs, stream)


class CacheReadPlan(_Plan):
    """dflash2_cache_read with its buffers bound; calling returns {"k", "v"} bf16 [tokens, heads, dim]."""

    _name = "dflash2_cache_read"

    @_on_stream
    def __init__(self, cache: PagedCache, batch: TokenBatch, *, k_out=None, v_out=None, stream=None):
        shape = (batch.tokens, cache.heads, cache.dim)
        if k_out is None and v_out is None:
            k_out, v_out = (torch.empty(shape, dtype=torch.bfloat16, device=cache.k.device) for _ in range(2))
        outputs, rows = {}, []
        for name, t in (("k", k_out), ("v", v_out)):
            rows.append(None if t is None else _rows(t, *shape, name + "_out"))
            if t is not None:
                outputs[name] = t
        self._bind((_ref(cache.args), _ref(batch.args), _ref(rows[0]), _ref(rows[1])), (cache, batch, rows), outputs,
                   stream)


class PagedAttentionPlan(_Plan):
    """dflash2_paged_attention with its buffers bound; calling returns {"out", "lse"}."""

    _name = "dflash2_paged_attention"

    @_on_stream
    def __init__(self, q, cache: PagedCache, batch: TokenBatch, *, causal: bool = True, window: int = 0,
                 scale: float | None = None, out=None, lse=None, workspace: AttentionWorkspace | None = None,
                 stream=None):
        heads = _heads_of(q, "q")
        N, dim = batch.tokens, cache.dim
        qr = _rows(q, N, heads, dim, "q")
        out = _out_like(q) if out is None else out
        outr = _rows(out, N, heads, dim, "out")
        if lse is None:
            lse = torch.empty((N, heads), dtype=torch.float32, device=q.device)
        elif lse is False:
            lse = None
        opts = AttentionArgs(dim ** -0.5 if scale is None else float(scale), int(bool(causal)),
                             _int32(min(int(window), 2 ** 31 - 1), "window"))  # past every position: no limit
        if not math.isfinite(opts.scale):
            raise ValueError("scale must be finite")
        ws = workspace
        if ws is None:
            ws = AttentionWorkspace(cache, batch, heads)
        elif ws.nbytes < dflash2_paged_attention_workspace_bytes(cache, batch, heads):
            raise ValueError("workspace too small for these sizes")
        self.workspace = ws
        outputs = {"out": out} if lse is None else {"out": out, "lse": lse}
        self._bind((_ref(cache.args), _ref(batch.args), _ref(opts), _ref(qr), _ref(outr),
                    _ptr(lse, torch.float32, (N, heads), "lse"), ws.ptr, ws.nbytes), (cache, batch, opts, qr, outr, q, ws),
                   outputs, stream)


@_on_stream
def dflash2_rope_table(max_pos: int, rot: int, *, theta: float = 10000.0, kind: str = "plain", factor: float = 1.0,
                       original_len: float = 0.0, low: float = 1.0, high: float = 32.0, multiplier: float = 1.0,
                       out=None, stream=None):
    """Cosines and sines [max_pos, 2, rot / 2] float32 of position * frequency; `kind` is one of "plain",
    "linear", "base", "ramp", "band" (df2_rope_kind), the latter four stretched by `factor`."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(ROPE_KINDS)}, got {kind!r}")
    max_pos, rot = _int32(max_pos, "max_pos"), _int32(rot, "rot")
    if out is None:
        if max_pos < 1 or rot < 2 or rot % 2:
            raise ValueError("max_pos must be positive and rot even and positive")
        out = torch.empty((max_pos, 2, rot // 2), dtype=torch.float32, device="cuda")
    s = RopeScaling(ROPE_KINDS[kind], theta, factor, original_len, low, high, multiplier)
    st = library().dflash2_rope_table(ctypes.byref(s), max_pos, rot,
                                      _ptr(out, torch.float32, (max_pos, 2, rot // 2), "out"), _stream(stream))
    _check(st, "dflash2_rope_table")
    return out


def dflash2_rope(x, positions, table, *, interleaved: bool = False, inverse: bool = False, out=None, stream=None):
    """Rows [N, heads, dim] rotated by positions int32 [N]; inverse: the other way (the gradient).  Returns out."""
    return RopePlan(x, positions, table, interleaved=interleaved, inverse=inverse, out=out, stream=stream)()


def dflash2_cache_append(cache: PagedCache, batch: TokenBatch, k, v, *, q=None, q_out=None, table=None,
                         interleaved: bool = False, stream=None):
    """Rotates (with a table) and writes the new tokens' keys and values; returns the cache's tensors and q."""
    return CacheAppendPlan(cache, batch, k, v, q=q, q_out=q_out, table=table, interleaved=interleaved,
                           stream=stream)()


def dflash2_cache_read(cache: PagedCache, batch: TokenBatch, *, k_out=None, v_out=None, stream=None):
    """The tokens' keys and values out of the cache, bf16; returns {"k", "v"}."""
    return CacheReadPlan(cache, batch, k_out=k_out, v_out=v_out, stream=stream)()


def dflash2_paged_attention(q, cache: PagedCache, batch: TokenBatch, *, causal: bool = True, window: int = 0,
                            scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """Attention of the new tokens' queries over the cache (scale defaults to dim ** -0.5); returns
    {"out", "lse"}; pass lse=False to leave it out."""
    return PagedAttentionPlan(q, cache, batch, causal=causal, window=window, scale=scale, out=out, lse=lse,
                              workspace=workspace, stream=stream)()
