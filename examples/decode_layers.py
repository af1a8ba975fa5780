"""Prompt, decode and verify steps of a small stack of W4 layers over the paged 8-bit cache.

    python examples/decode_layers.py [--layers 4] [--kind int8|fp8] [--steps 16] [--candidates 3]
        [--rope-base 10000] [--share 2048 [--share-from 2048]] [--temperature 0.8 [--top-k 50] [--top-p 0.95] [--min-p 0.02]]

Every weight product, the cache and its attention, the rotation and the sampling
are the library's; torch allocates, normalises the hidden rows (root mean square, no
learned factor) and adds the residuals.  Weights are random (synthetic.quantized_weights), so what is
generated means nothing: the example shows how the entry points fit together.
A step brings some tokens of each request (a prompt, one token, or candidates
to verify), and its bookkeeping (w4a16_kv_plan) is made once for all layers:

  plan -> per layer: q/k/v products -> (head norms, positions rotated in) -> append -> attention
       -> o product -> MLP -> LM head -> largest logits, or tokens drawn from them

Requests that begin with the same tokens can share their pages (Stack.share): from some 2000 of
them on, steps of few tokens a request read these once for all requests (w4a16_kv_attention_shared).
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import decode_w4a16_affine_amd as w4  # noqa: E402
import synthetic  # noqa: E402

KINDS = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}


class Weights:
    """One packed matrix [N, K] on the GPU: weights of mean 0, scaled to outputs of unit size."""

    def __init__(self, N, K, seed):
        w = synthetic.quantized_weights(N, K, seed=seed)
        self.qw = torch.from_numpy(np.ascontiguousarray(w.qw).view(np.int32)).cuda()
        s = torch.from_numpy(w.scales.view(np.int16)).view(torch.bfloat16).cuda().float()
        s = s / (0.056 * K ** 0.5)          # code * s has standard deviation 0.056: codes 4.6, s 0.011 +- 0.005
        self.s, self.b = s.to(torch.bfloat16), (-7.5 * s).to(torch.bfloat16)
        self.N = N

    def __iter__(self):
        return iter((self.qw, self.s, self.b))

    def __call__(self, x):
        return (w4.matmul if x.shape[0] <= w4.MAX_M else w4.matmul_prefill)(x, *self)


class Layer:
    def __init__(self, hidden, ffn, q_heads, kv_heads, dim, seed):
        self.q, self.o = Weights(q_heads * dim, hidden, seed), Weights(hidden, q_heads * dim, seed + 1)
        self.k, self.v = Weights(kv_heads * dim, hidden, seed + 2), Weights(kv_heads * dim, hidden, seed + 3)
        self.gate_up, self.down = Weights(2 * ffn, hidden, seed + 4), Weights(hidden, ffn, seed + 5)
        norms = 1 + 0.2 * torch.randn((2, dim), generator=torch.Generator().manual_seed(seed + 6))
        self.q_norm, self.k_norm = norms.to(torch.bfloat16).cuda()

    def qkv(self, x):
        out = [torch.empty((x.shape[0], w.N), dtype=torch.bfloat16, device=x.device) for w in (self.q, self.k, self.v)]
        if x.shape[0] <= w4.MAX_M:          # one launch for the three
            w4.w4a16_matmul_grouped(x, [(*w, y) for w, y in zip((self.q, self.k, self.v), out)])
        else:
            for w, y in zip((self.q, self.k, self.v), out):
                w4.w4a16_matmul_prefill(x, *w, y)
        return out

    def mlp(self, x):
        if x.shape[0] <= w4.MAX_M:
            h = torch.empty((x.shape[0], self.gate_up.N // 2), dtype=torch.bfloat16, device=x.device)
            w4.w4a16_matmul_geglu(x, *self.gate_up, h)
        else:
            gate, up = self.gate_up(x).float().chunk(2, dim=1)
            h = (torch.nn.functional.gelu(gate) * up).to(torch.bfloat16)
        return self.down(h)


def norm(x):
    return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def give_back(table, lens, kept, page):
    """The pages that requests cut from `lens` to `kept` tokens no longer reach; they leave the block table.

    w4a16_kv_plan takes every page past a request's length from the free list, so a page that rejected candidates
    opened belongs there again: left in the table, the next plan would write over it and nobody would hold it."""
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    reach = lambda n: (n[:, None] + page - 1) // page  # noqa: E731
    gone = (col >= reach(kept)) & (col < reach(lens)) & (table >= 0)
    pages = table[gone]
    table[gone] = -1
    return pages


class Stack:
    """Layers with a paged cache for `requests` requests of at most max_len tokens."""

    def __init__(self, layers=2, hidden=2560, ffn=10240, q_heads=10, kv_heads=2, dim=256, vocab=4096, requests=4,
                 max_len=2048, page=64, kind="int8", window=0, seed=0, rope_base=None, share_from=2048):
        self.embedding = Weights(vocab, hidden, seed + 100)      # tied: gathered rows in, LM head out
        self.layers = [Layer(hidden, ffn, q_heads, kv_heads, dim, seed + 1000 * (i + 1)) for i in range(layers)]
        self.heads, self.dim, self.page, self.max_len, self.window = (q_heads, kv_heads), dim, page, max_len, window
        width = -(-max_len // page)
        self.caches = [w4.kv_cache(requests * width, kv_heads, dim, page, dtype=KINDS[kind]) for _ in range(layers)]
        self.free = torch.randperm(requests * width).to(torch.int32).cuda()
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros((requests,), dtype=torch.int32, device="cuda")
        self.held = [0] * requests                               # the same on the host
        # with a base: queries and keys normed for each head and turned by their positions
        self.inv_freq = None if rope_base is None else rope_base ** (-torch.arange(0, dim, 2) / dim).float().cuda()
        self.shared = 0                                          # entries that all requests begin with
        self.shared_len = torch.zeros((1,), dtype=torch.int32, device="cuda")
        # fewer shared entries are read by each request for itself: joining partial results takes longer (4 requests, 10
        # heads of 256 over 2: behind 512 entries 10.7 us instead of 9.1, 2048 12.1 and 12.5, 16384 23 instead of 28)
        self.share_from = share_from

    def step(self, tokens, counts):
        """tokens [T]: counts[r] of each request, in request order.  (logits' argmax [T], final hidden rows [T, hidden])"""
        held = [n + c for n, c in zip(self.held, counts)]
        longest = max(held, default=0)
        if longest > self.max_len:      # (past the block table's columns tokens have no slot: they would be lost)
            raise ValueError(f"a request of {longest} tokens in a stack of max_len {self.max_len}")
        new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        # where the tokens go: once for all layers
        seq, start, slots, used = w4.kv_plan(self.lens, new, self.free, self.table, tokens.numel(), self.page)
        positions = None
        if self.inv_freq is not None:
            positions = torch.cat([torch.arange(n, n + c) for n, c in zip(self.held, counts)]).int().cuda()
        x = w4.gather_rows(*self.embedding, tokens).float()
        for layer, cache in zip(self.layers, self.caches):
            q, k, v = (t.view(t.shape[0], -1, self.dim) for t in layer.qkv(norm(x)))
            if positions is not None:
                w4.w4a16_qk_norm_rope(q, k, layer.q_norm, layer.k_norm, self.inv_freq, positions, q, k)
            w4.w4a16_kv_append(k, v, slots, *cache)
            a = self.attention(q, cache, seq, start, max(counts))
            x = x + layer.o(a.flatten(1)).float()
            x = x + layer.mlp(norm(x)).float()
        h = norm(x)
        best = torch.cat([w4.lmhead_argmax(part, *self.embedding, want_logits=False)[0] for part in h.split(w4.MAX_M)])
        # the pages are taken, the tokens held (a program that rejects candidates keeps fewer: see keep)
        taken = int(used)
        if taken > self.free.numel():
            raise RuntimeError("out of cache pages")
        self.free = self.free[taken:].contiguous()
        self.lens, self.held = seq, held
        return best, h

    def attention(self, q, cache, seq, start, most):
        rows = most * (self.heads[0] // self.heads[1])
        if self.shared and self.shared >= self.share_from and not self.window and rows <= 64:
            return w4.kv_attention_shared(q, *cache, self.table, seq, start, self.shared_len, most, max_shared=self.shared,
                                          max_own=self.max_len - self.shared)
        return w4.kv_attention(q, *cache, self.table, seq, start, most, max_len=self.max_len, window=self.window)

    def share(self, tokens):
        """All requests begin with these tokens, a whole number of pages, which are brought and held once."""
        n = tokens.numel()
        if any(self.held) or n % self.page or n > self.max_len:
            raise ValueError(f"{n} tokens to share: whole pages of {self.page}, up to {self.max_len}, before any other step")
        self.step(tokens, [n] + [0] * (len(self.held) - 1))
        self.table[1:] = self.table[0]
        self.lens, self.held = torch.full_like(self.lens, n), [n] * len(self.held)
        self.shared = n
        self.shared_len.fill_(n)

    def draw(self, h, uniforms, temperature, top_k=0, top_p=1.0, min_p=0.0):
        """Tokens drawn from the logits of final hidden rows h [R, hidden] by numbers uniforms [R] in [0, 1)."""
        each = lambda v, dtype: torch.full(uniforms.shape, v, dtype=dtype, device="cuda")  # noqa: E731
        return w4.sample(self.embedding(h), uniforms, each(temperature, torch.float32), each(top_k, torch.int32),
                         each(top_p, torch.float32), each(min_p, torch.float32))[0]

    def keep(self, lens):
        """Keeps the first lens[r] tokens of each request: the candidates behind them were rejected."""
        if any(n > h for n, h in zip(lens, self.held)):
            raise ValueError(f"requests hold {self.held} tokens, {lens} asked to keep")
        if min(lens) < self.shared:
            raise ValueError(f"{lens} asked to keep of requests that share {self.shared}")
        kept = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.free = torch.cat([give_back(self.table, self.lens, kept, self.page), self.free])
        self.lens, self.held = kept, list(lens)

    def verify(self, tokens, guesses):
        """One token and some candidates of each request (tokens [R], guesses [R, k]) in one step; those candidates
        stay that agree with the stack's own choice up to there.  (the next tokens [R], how many stayed [R])"""
        batch = torch.cat([tokens[:, None], guesses], dim=1)
        held = self.held
        best, _ = self.step(batch.flatten(), [batch.shape[1]] * len(held))
        best = best.view(batch.shape)
        stay = (best[:, :-1] == guesses).int().cumprod(1).sum(1)
        self.keep([n + 1 + s for n, s in zip(held, stay.tolist())])
        return best.gather(1, stay[:, None]).flatten(), stay


def last_of(counts):
    return torch.tensor(np.cumsum(counts) - 1, device="cuda")


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--kind", choices=sorted(KINDS), default="int8")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--candidates", type=int, default=3)
    ap.add_argument("--rope-base", type=float, help="norm queries and keys and rotate positions in, with this base")
    ap.add_argument("--share", type=int, default=0, help="tokens that all requests begin with (whole pages of 64)")
    ap.add_argument("--share-from", type=int, default=2048, help="shared tokens from which steps read them once for all")
    ap.add_argument("--temperature", type=float, default=0.0, help="draw tokens (0: take the largest logits)")
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=1.0)
    ap.add_argument("--min-p", type=float, default=0.0)
    a = ap.parse_args()
    prompts = [700, 64, 333, 5]
    stack = Stack(layers=a.layers, kind=a.kind, rope_base=a.rope_base, max_len=2048 + a.share, share_from=a.share_from)
    generator = torch.Generator().manual_seed(1)
    if a.share:
        stack.share(torch.randint(0, 4096, (a.share,), dtype=torch.int32, generator=torch.Generator().manual_seed(2)).cuda())
    tokens = torch.randint(0, 4096, (sum(prompts),), dtype=torch.int32, generator=generator).cuda()

    def choose(best, h):
        if not a.temperature:
            return best
        uniforms = torch.rand((h.shape[0],), generator=generator).cuda()
        return stack.draw(h, uniforms, a.temperature, a.top_k, a.top_p, a.min_p)

    last = last_of(prompts)
    best, h = stack.step(tokens, prompts)
    tokens = choose(best[last], h[last])
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        tokens = choose(*stack.step(tokens, [1] * len(prompts)))
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) / a.steps * 1e3
    print(f"{a.layers} layers, {len(prompts)} requests, {a.kind} cache: {ms:.2f} ms a decode step; "
          f"lengths {stack.lens.tolist()}, last tokens {tokens.tolist()}")
    # verify steps; the candidates are guesses (the token itself), so most are rejected
    stayed = 0
    for _ in range(a.steps):
        tokens, stay = stack.verify(tokens, tokens[:, None].expand(-1, a.candidates))
        stayed += int(stay.sum())
    print(f"{a.steps} verify steps of {a.candidates} candidates: {stayed} stayed; lengths {stack.lens.tolist()}, "
          f"{stack.free.numel()} pages free")


if __name__ == "__main__":
    main()
