"""Plain forms, in float64 and loops over sequences, of the attention-side operators, and the bounds the
GPU tests hold the kernels to (derived from the formats, not from runs)."""
import math

import torch

BF16 = torch.bfloat16
TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
EPS32 = 2.0 ** -24  # half a unit in the last place of float32, relative
EPS16 = 2.0 ** -8   # ... of bfloat16 (8 significand bits)
EPS_F16 = 2.0 ** -11  # ... of float16 (11)


def rotate(x, table, positions, interleaved, inverse=False):
    """x [N, heads, dim] -> float64."""
    x = x.double()
    c, s = table[positions.long(), 0].double()[:, None], table[positions.long(), 1].double()[:, None]
    s = -s if inverse else s
    half = table.shape[2]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    y = x.clone()
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def rotate_bound(x, y):
    """Three float32 roundings of numbers up to |a| + |b| (<= 2 max |row|), then one to bfloat16."""
    return EPS16 * y.abs() + 8 * EPS32 * x.double().abs().amax(-1, keepdim=True) + 2.0 ** -133


def rotate32(x, table, positions, interleaved):
    """The rotation in float32 with every product and sum rounded: what is quantised."""
    x = x.float()
    c, s = table[positions.long(), 0][:, None], table[positions.long(), 1][:, None]
    half = table.shape[2]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ra, rb = a * c - b * s, b * c + a * s
    y = x.clone()
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ra, rb
    else:
        y[..., :half], y[..., half:2 * half] = ra, rb
    return y


def quantise(x, dtype):
    """Codes and scales of float32 rows on the CPU (IEEE float32 operations, one by one)."""
    x = x.cpu().float()
    m = x.abs().amax(-1, keepdim=True)
    m = torch.where(torch.isnan(x).any(-1, keepdim=True), torch.full_like(m, math.nan), m)
    finite = torch.isfinite(m)
    held = finite & (m >= 1e-30)
    top = torch.full_like(m, TOP[dtype])
    one = torch.ones_like(m)
    y = torch.where(held, x * (top / torch.where(held, m, one)), torch.zeros_like(x))
    codes = y.round().clamp(-127, 127).to(torch.int8) if dtype == torch.int8 else y.to(torch.float8_e4m3fn)
    scale = torch.where(held, m / top, torch.where(finite, torch.zeros_like(m), torch.full_like(m, math.nan)))
    return codes, scale.squeeze(-1)


class Batch:
    """A ragged batch on the CPU: lengths, new tokens, a shuffled page table; `spare` page-table columns
    hold ids that no call may use."""

    def __init__(self, lens, news, page_size, seed=0, spare=1, poison=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.news, self.page_size = list(lens), list(news), page_size
        need = [max(0, -(-n // page_size)) for n in lens]
        self.pages = sum(need) + 2
        ids = torch.randperm(self.pages, generator=g)
        width = max(need) + spare
        self.table = torch.full((len(lens), width), 2 ** 31 - 1 if poison else 0, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n].to(torch.int32)
            at += n
        self.start = torch.tensor([0] + list(news)).cumsum(0).to(torch.int32)
        self.N = int(self.start[-1])

    def on_gpu(self, at):
        return at.TokenBatch(self.start.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.table.cuda(),
                             tokens=self.N, max_new=max(self.news))

    def places(self):
        """(sequence, position, page, slot) of every new token; page -1 for padding."""
        out = []
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            for p in range(n - m, n):
                out.append((b, p, int(self.table[b, p // self.page_size]) if p >= 0 else -1, p % self.page_size))
        return out


def attend(q, k, v, lens, news, scale, causal, window):
    """float64 attention; k, v: lists of [len, kv_heads, dim] float64.  Returns out, sum p |v|, lse."""
    outs, mags, lses, at = [], [], [], 0
    for b, (n, m) in enumerate(zip(lens, news)):
        qb = q[at:at + m].double()
        at += m
        heads, kvh = qb.shape[1], k[b].shape[1]
        g = heads // kvh
        pos = torch.arange(n - m, n)[:, None]
        j = torch.arange(n)[None]
        seen = (j <= pos) if causal else torch.ones(m, n, dtype=torch.bool)
        if window:
            seen = seen & (j > pos - window)
        seen = seen.to(qb.device)
        kk, vv = k[b].repeat_interleave(g, 1), v[b].repeat_interleave(g, 1)
        s = torch.einsum("thd,jhd->htj", qb, torch.nan_to_num(kk, 0.0, 0.0, 0.0)) * scale
        s = s.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(s, -1) if n else torch.full((heads, m), -math.inf, dtype=torch.float64, device=q.device)
        p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
        outs.append(torch.einsum("htj,jhd->thd", p, vv))
        mags.append(torch.einsum("htj,jhd->thd", p, vv.abs()))
        lses.append(lse.T)
    return torch.cat(outs), torch.cat(mags), torch.cat(lses)


def attend_bound(out, mag):
    """The result's rounding to bfloat16; each probability rounded once to bfloat16 before its product
    (relative 2^-8, so at most 2^-8 sum p |v| in all); scores and sums in float32 (2^-13 of sum p |v|
    allows a score error of 2^-14, 128 terms of 2^-24 times scores up to 8)."""
    return EPS16 * out.abs() + (EPS16 + 2.0 ** -13) * mag + 1e-30


def tile_values(n, heads, dim, device="cuda"):
    """Value rows of one 1: channel d is that of the key tiles t with t mod dim == d, so that it counts them."""
    v = torch.zeros(n, heads, dim, device=device)
    p = torch.arange(n, device=device)
    v[p, :, (p // 128) % dim] = 1
    return v


def tile_bound(want, squares, eps_p):
    """For such values: a result's rounding to bfloat16; each probability rounded to nearest, independently (seven times
    the root of the sum of squares: 1e-10 that a result passes it); float32 sums of positive terms."""
    return EPS16 * want.abs() + 7 * eps_p * squares.sqrt() + 2.0 ** -13 * want.abs()
