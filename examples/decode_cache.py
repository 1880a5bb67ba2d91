"""Decoding over the paged 4-bit key/value cache: a prompt, steps of single
tokens, beams that fork, and pages that are moved together.

A stack of attention layers with random weights stands in for a model: per layer
a fused projection gives queries, keys and values, the keys and values are
appended (keys rotated, both quantized to 4 bits), the queries attend over the
cache, and an output projection is added to the residual stream.  The next token
of a row is drawn from the last layer's output.

    python examples/decode_cache.py                      # 4 rows, 256 tokens of prompt, 64 steps
    python examples/decode_cache.py --rows 32 --prompt 4000 --steps 32 --layers 8
    python examples/decode_cache.py --prompt 4000 --budget 1024   # rows cut to their 1024 heaviest positions

It prints the error of the first layer's attention against exact attention over
the unquantized keys and values, and the time of a step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hadamard_rotation_preprocessing_amd as hr  # noqa: E402


class Decoder:
    """Attention layers whose keys and values live in one pool of pages."""

    def __init__(self, layers, rows, positions, q_heads, kv_heads, head_dim, vocab=256, page=64, device="cuda", seed=0,
                 budget=0):
        g = torch.Generator(device=device).manual_seed(seed)
        width = q_heads * head_dim
        self.q_heads, self.kv_heads, self.head_dim, self.page = q_heads, kv_heads, head_dim, page
        self.spec = hr.CacheSpec(kv_heads, head_dim, page, hr.QSpec("int", 4, head_dim, False, "bf16"))
        self.width = -(-positions // page)
        self.pages = rows * self.width + rows
        self.pool = hr.cache_pool(self.spec, self.pages, layers, device)

        def weight(n, m):
            return (torch.randn((n, m), generator=g, device=device) / n ** 0.5).bfloat16()
        self.embed = torch.randn((vocab, width), generator=g, device=device).bfloat16()
        self.qkv = [weight(width, (q_heads + 2 * kv_heads) * head_dim) for _ in range(layers)]
        self.out = [weight(width, width) for _ in range(layers)]
        self.head = weight(width, vocab)
        self.table = torch.full((rows, self.width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=device)
        # with a budget: the attention weight that each position has got so far
        self.budget = budget
        self.weights = torch.zeros((layers, rows, kv_heads, self.width * page), device=device) if budget else None

    def schedule(self, parents, grow):
        """Row i continues row parents[i] (-1: a new one), grown by grow[i]."""
        step = hr.cache_update(self.pool, self.spec, self.table, self.lens, parents, grow)
        self.table, self.lens = step["table"], step["lens"]
        if self.budget:
            self.weights = self.weights[:, parents.clamp(min=0).long()]     # (a new row's are written before they are read)
        return step["status"]

    def evict(self):
        """Cuts the rows to the budget: 4 first positions, the newest eighth, and the
        heaviest of the others; layer by layer and head by head."""
        r = hr.cache_evict(self.pool, self.spec, self.table, self.lens, self.weights, self.budget, min(4, self.budget // 8),
                           self.budget // 8)
        self.table, self.lens = r["table"], r["lens"]
        return r["status"]

    def forward(self, tokens, new):
        """tokens int64 [rows * new], row by row; returns logits of each row's last token."""
        x = self.embed[tokens]
        hq, hk, d = self.q_heads, self.kv_heads, self.head_dim
        self.first = None
        for i, (wi, wo) in enumerate(zip(self.qkv, self.out)):
            y = torch.nn.functional.layer_norm(x, x.shape[-1:])
            qkv = (y @ wi).view(-1, hq + 2 * hk, d)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]     # read in place, as slices
            hr.cache_append(self.pool[i], self.spec, k, v, self.table, self.lens)
            o = hr.cache_attention(q, self.pool[i], self.spec, self.table, self.lens, max_q=new, lse=bool(self.budget))
            if self.budget:
                o, lse = o
                hr.cache_weights(q, self.pool[i], self.spec, self.table, self.lens, lse, self.weights[i], max_q=new)
            if i == 0:
                self.first = (q, k, v, o)
            x = x + o.reshape(x.shape) @ wo
        return x.view(-1, new, x.shape[-1])[:, -1] @ self.head

    def compact(self):
        r = hr.cache_compact(self.pool, self.spec, self.table, self.lens)
        self.table = r["table"]
        return r["status"]


def exact(q, k, v):
    """Causal attention of one row's prompt over the keys and values as they were."""
    rep = q.shape[1] // k.shape[1]
    q, k, v = (t.float().transpose(0, 1).contiguous() for t in (q, k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)))
    s = torch.matmul(q, k.transpose(1, 2).contiguous()) / q.shape[-1] ** 0.5
    n = s.shape[-1]
    s = s.masked_fill(torch.ones((n, n), dtype=torch.bool, device=s.device).triu(1), float("-inf"))
    return torch.matmul(s.softmax(-1), v).transpose(0, 1)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--rows", type=int, default=4)
    p.add_argument("--prompt", type=int, default=256)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--q-heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--budget", type=int, default=0, help="positions that a row keeps (0: all)")
    a = p.parse_args(argv)
    dev = "cuda"
    m = Decoder(a.layers, a.rows, a.prompt + a.steps, a.q_heads, a.kv_heads, a.head_dim, device=dev, budget=a.budget)
    g = torch.Generator(device=dev).manual_seed(1)
    fresh = torch.full((a.rows,), -1, dtype=torch.int32, device=dev)
    m.schedule(fresh, torch.full_like(fresh, a.prompt))
    prompt = torch.randint(0, m.embed.shape[0], (a.rows, a.prompt), generator=g, device=dev)
    logits = m.forward(prompt.reshape(-1), a.prompt)
    q, k, v, o = (t[: a.prompt] for t in m.first)
    want = exact(q, k, v)
    error = (torch.linalg.vector_norm(o.float() - want) / torch.linalg.vector_norm(want)).item()
    print("prompt of %d rows x %d tokens; first layer's attention within %.3g of exact keys and values" % (a.rows, a.prompt, error))

    same = torch.arange(a.rows, dtype=torch.int32, device=dev)
    one = torch.ones_like(same)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for step in range(a.steps):
        # every eighth step the last row gives way to a second continuation of
        # the first: full pages are shared, the one being filled is copied
        parents = same.clone()
        if step % 8 == 7:
            parents[-1] = 0
        if a.budget and step % 8 == 0:
            m.evict()
        status = m.schedule(parents, one)
        p = torch.softmax(logits[parents.long()].float(), -1)
        token = torch.multinomial(p, 1, generator=g)[:, 0]
        logits = m.forward(token, 1)
    end.record()
    torch.cuda.synchronize()
    used, lacking, copied, free = status.tolist()
    if lacking:
        raise SystemExit("%d pages were lacking" % lacking)
    live = m.compact().tolist()
    print("%d steps, %.1f us each; %d of %d pages in use, the last step copied %d; after compaction %s"
          % (a.steps, begin.elapsed_time(end) * 1e3 / max(a.steps, 1), used, m.pages, copied, live))
    print("lengths %s, logits finite: %s" % (m.lens.tolist()[:8], bool(torch.isfinite(logits).all())))
    return error, logits


if __name__ == "__main__":
    main()
