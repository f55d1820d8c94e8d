"""One drafter layer and the selector head around the paged cache: what a drafting loop runs each step.

    python examples/draft_step.py [--sequences 4] [--steps 3] [--cache bf16|e4m3|int8]

Each step a block of T draft positions per sequence goes through the local convolution, the q/k/v
projection, rotary positions with the cache write, attention over the sequence so far (a draft block
sees all of itself), the output projection and the selector head, whose draft then counts as accepted:
the sequences grow by T.  Weights are random; the point is the calls and their buffers, which are bound
once and reused.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_drafter_gb300 import attention as at  # noqa: E402
from speculative_decoding_drafter_gb300 import dflash2 as df  # noqa: E402

BF16 = torch.bfloat16
TYPES = {"bf16": BF16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class DraftStep:
    """Weights, cache and bound calls of one drafter layer with its selector head."""

    def __init__(self, B, T, H=1024, q_heads=8, kv_heads=2, dim=128, V=8192, k=8, D=64, page_size=16, max_len=512,
                 cache_type="bf16", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, scale=None):
            s = shape[-1] ** -0.5 if scale is None else scale
            return (torch.randn(*shape, device="cuda", generator=g) * s).to(BF16)

        self.B, self.T, self.H, self.q_heads, self.kv_heads, self.dim, self.k = B, T, H, q_heads, kv_heads, dim, k
        self.embed, self.w_qkv = w(V, H, scale=1.0), w((q_heads + 2 * kv_heads) * dim, H)
        self.w_out, self.head = w(H, q_heads * dim), w(V, H)
        self.conv_base = torch.zeros(2, H, dtype=BF16, device="cuda")
        self.conv_base[0] = 1
        self.conv_dyn = torch.randn(B * T, 2, H // 16, device="cuda", generator=g) * 0.1
        self.gamma = torch.ones(H, dtype=BF16, device="cuda")
        self.W_sel, self.pred_cb, self.succ_cb = w(D, H), w(V, D, scale=0.1), w(V, D, scale=0.1)
        self.table = at.dflash2_rope_table(max_len, dim)
        # a page table with the pages of the sequences side by side
        per = -(-max_len // page_size)
        pages = torch.arange(B * per, dtype=torch.int32, device="cuda").view(per, B).t().contiguous()
        self.cache = at.PagedCache.allocate(B * per, page_size, kv_heads, dim, TYPES[cache_type])
        self.kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
        start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
        self.tokens = at.TokenBatch(start, self.kv_len, pages, tokens=B * T, max_new=T)
        # buffers, and the calls bound to them
        self.qkv = torch.empty(B * T, q_heads + 2 * kv_heads, dim, dtype=BF16, device="cuda")
        q, key, v = self.qkv.split([q_heads, kv_heads, kv_heads], 1)
        self.append = at.CacheAppendPlan(self.cache, self.tokens, key, v, q=q, q_out=q, table=self.table)
        self.attend = at.PagedAttentionPlan(q, self.cache, self.tokens, causal=False)
        self.workspace = df.Workspace(df.make_dims(B, T, H, V, k, D))

    def __call__(self, ids, anchor):
        """Token ids [B, T] of the block (masks or the last draft) and the anchors [B] -> draft ids [B, T]."""
        x = self.embed[ids.long()].view(self.B * self.T, self.H)
        x_prev = self.embed[anchor.long()]
        h = df.dflash2_dynamic_conv(x, self.conv_base, self.conv_dyn, self.T, x_prev=x_prev, gamma=self.gamma)
        torch.matmul(h, self.w_qkv.t(), out=self.qkv.view(self.B * self.T, -1))
        self.kv_len += self.T  # the block's own rows count as held from here on
        self.append()
        self.out = self.attend()["out"]
        hidden = x + self.out.reshape(self.B * self.T, -1) @ self.w_out.t()
        _, draft = df.dflash2_select(hidden, self.head, self.W_sel, self.pred_cb, self.succ_cb, anchor, self.k, self.T,
                                     workspace=self.workspace)
        return draft


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--sequences", type=int, default=4)
    p.add_argument("--steps", type=int, default=3)
    p.add_argument("--cache", choices=sorted(TYPES), default="bf16")
    a = p.parse_args(argv)
    T = 8
    step = DraftStep(a.sequences, T, cache_type=a.cache, max_len=max(64, a.steps * T))
    ids = torch.zeros(a.sequences, T, dtype=torch.int32, device="cuda")
    anchor = torch.arange(a.sequences, dtype=torch.int32, device="cuda")
    for n in range(a.steps):
        ids = step(ids, anchor)
        anchor = ids[:, -1].contiguous()
        print(f"step {n}: {int(step.kv_len[0])} tokens held, draft {ids.tolist()}")
    df.dflash2_check_device_status(step.attend.workspace)
    return ids


if __name__ == "__main__":
    main()
