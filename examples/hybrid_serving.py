"""Serving a small hybrid model: gated-delta-rule layers with their states,
and a softmax-attention layer over a paged cache.

Two sequences of different length are run through three layers (two of the
gated delta rule, one of attention) the way a server does: the prompts in chunks
(each chunk's keys and values go into the cache, its tokens attend to everything
cached, and the rule's layers carry their states from chunk to chunk), then token
by token.  The same tokens in one pass give the same outputs, up to rounding.

    python examples/hybrid_serving.py [--fmt bf16|e4m3|int8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_rule_gb300 as gdr  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 8, 2, 128, 16
WIDTH = HEADS * DIM
FORMATS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class PagedCache:
    """Pages of keys and values, and the table of the pages that each sequence
    owns.  ``extend`` takes pages from the free list as sequences grow."""

    def __init__(self, n_seqs, n_pages, max_pages, fmt, device):
        shape = (n_pages, PAGE, KV_HEADS, DIM)
        self.k = torch.zeros(shape, device=device).to(FORMATS[fmt])
        self.v = torch.zeros(shape, device=device).to(FORMATS[fmt])
        scales = (n_pages, KV_HEADS, PAGE)
        self.scales = {} if fmt == "bf16" else dict(k_scale=torch.zeros(scales, device=device),
                                                    v_scale=torch.zeros(scales, device=device))
        self.free = list(range(n_pages))[::-1]
        self.owned = [[] for _ in range(n_seqs)]
        self.lens = [0] * n_seqs
        self.max_pages, self.device = max_pages, device

    def extend(self, new_tokens):
        for i, n in enumerate(new_tokens):
            self.lens[i] += n
            while len(self.owned[i]) * PAGE < self.lens[i]:
                self.owned[i].append(self.free.pop())
        table = [p + [0] * (self.max_pages - len(p)) for p in self.owned]
        self.table = torch.tensor(table, dtype=torch.int32, device=self.device)
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device=self.device)

    def attend(self, q, k, v, cu, longest):
        args = (self.k, self.v, self.table, self.kv_lens, cu)
        gdr.gdr_cache_write(k, v, *args, **self.scales)
        return gdr.gdr_paged_attn(q, *args, max_seqlen=longest, **self.scales)[0]


class HybridModel:
    def __init__(self, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen) * shape[0] ** -0.5).to(torch.bfloat16).to(device)

        self.rule = [dict(qkv=weight(WIDTH, 3 * WIDTH), gate=weight(WIDTH, 2 * HEADS),
                          out=weight(WIDTH, WIDTH)) for _ in range(2)]
        self.attn = dict(q=weight(WIDTH, WIDTH), kv=weight(WIDTH, 2 * KV_HEADS * DIM),
                         out=weight(WIDTH, WIDTH))

    def start(self, n_seqs, n_pages, max_pages, fmt, device="cuda"):
        """States of the rule's layers [sequences, heads, K, V] and the cache."""
        states = [torch.zeros(n_seqs, HEADS, DIM, DIM, device=device) for _ in self.rule]
        return states, PagedCache(n_seqs, n_pages, max_pages, fmt, device)

    def forward(self, x, lens, states, cache):
        """One step over packed new tokens x [tokens, WIDTH], ``lens`` of each
        sequence; the states and the cache move on."""
        cu = torch.tensor([0] + lens, device=x.device).cumsum(0).to(torch.int32)
        cache.extend(lens)
        T, longest = x.shape[0], max(lens)
        for i, w in enumerate(self.rule):
            if i == 1:  # the attention layer lies between the rule's two
                h = norm(x)
                q = (h @ self.attn["q"]).view(1, T, HEADS, DIM)
                kv = (h @ self.attn["kv"]).view(1, T, 2, KV_HEADS, DIM)
                o = cache.attend(q, kv[:, :, 0], kv[:, :, 1], cu, longest)
                x = x + o.reshape(T, WIDTH) @ self.attn["out"]
            h = norm(x)
            qkv = (h @ w["qkv"]).view(1, T, 3, HEADS, DIM)
            q, k = (norm(qkv[:, :, j]) * DIM ** -0.5 for j in (0, 1))
            gates = (h @ w["gate"]).float().view(1, T, 2, HEADS)
            g = torch.nn.functional.logsigmoid(gates[:, :, 0] + 3.0).contiguous()
            beta = gates[:, :, 1].sigmoid().contiguous()
            if longest == 1:  # a decode step: the states are read and written in place
                o = gdr.gdr_recurrent_fwd(q, k, qkv[:, :, 2], g, beta, cu, state=states[i])
            else:
                o, states[i] = gdr.gdr_chunk_fwd(q, k, qkv[:, :, 2], g, beta, cu, h0=states[i],
                                                 max_seqlen=longest)
            x = x + o.reshape(T, WIDTH) @ w["out"]
        return x


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def main(fmt="bf16", prompts=(150, 70), steps=4, chunk=64):
    """Largest relative difference between the served tokens' outputs and the
    same tokens' in one pass."""
    model, n = HybridModel(), len(prompts)
    gen = torch.Generator().manual_seed(1)
    total = [p + steps for p in prompts]
    seqs = [torch.randn(t, WIDTH, generator=gen).to(torch.bfloat16).cuda() for t in total]
    pages = [-(-t // PAGE) for t in total]

    states, cache = model.start(n, sum(pages), max(pages), fmt)
    served, at = [[] for _ in seqs], [0] * n
    while at != total:
        # a chunk of what is left of each prompt, then a token at a time
        left = [p - a for p, a in zip(prompts, at)]
        lens = [min(max(0, x), chunk) for x in left] if max(left) > 0 else [1] * n
        x = torch.cat([s[a:a + m] for s, a, m in zip(seqs, at, lens)])
        y = model.forward(x, lens, states, cache)
        for i, part in enumerate(y.split(lens)):
            served[i].append(part)
        at = [a + m for a, m in zip(at, lens)]

    states, cache = model.start(n, sum(pages), max(pages), fmt)
    whole = model.forward(torch.cat(seqs), total, states, cache)
    served = torch.cat([torch.cat(s) for s in served]).float()
    return float((served - whole.float()).norm() / whole.float().norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--fmt", choices=sorted(FORMATS), default="bf16")
    a = ap.parse_args()
    print(f"{a.fmt} cache: served against one pass, relative difference {main(a.fmt):.2e}")
