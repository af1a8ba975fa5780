"""A serving step's operators in their order (include/w4a16_step.h beside w4a16_kv.h): plan, head norms with rotation,
append, attention behind shared entries, sampling, each fed by the ones before; and the example stack with all of them.

Each operator's output is held to its definition on the inputs that it was given."""
import os
import sys

import numpy as np
import pytest
import torch

import decode_w4a16_affine_amd as w4
import kv_reference
import step_reference as ref
from parity import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w4.step_lib()
    yield
    torch.cuda.synchronize()


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def f64(t):
    return t.cpu().double().numpy()


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("graph", [False, True])
def test_a_prompt_shared_and_three_steps(kind, graph):
    """Three requests behind a prompt of 96 tokens (six pages); single tokens, then candidates; once in a graph that is
    replayed for steps of the same sizes."""
    say("step together", kind, graph)
    R, H, G, D, page, vocab, S = 3, 2, 4, 128, 16, 5000, 96
    rng = np.random.default_rng(23)
    bf16 = lambda *n: torch.from_numpy(rng.normal(size=n)).to(torch.bfloat16).cuda()  # noqa: E731
    cache = w4.kv_cache(60, H, D, page, {"int8": torch.int8, "fp8": torch.float8_e4m3fn}[kind])
    qw, kw = (1 + 0.1 * bf16(2, D)).to(torch.bfloat16)
    inv_freq = torch.tensor(10000.0 ** (-np.arange(D // 2) / (D // 2)), dtype=torch.float32, device="cuda")
    head = bf16(vocab, H * G * D).float() * 0.05
    free = i32(rng.permutation(60))
    table = torch.full((R, 16), -1, dtype=torch.int32, device="cuda")

    def rope(q, k, positions):
        qo, ko = w4.qk_norm_rope(q, k, qw, kw, inv_freq, positions)
        for x, y, w in ((q, qo, qw), (k, ko, kw)):
            want, bound = ref.rope(f64(x), f64(w), 0.0, np.float64(np.float32(1e-6)), True, f64(inv_freq),
                                   positions.cpu().numpy()[None], None, False)
            assert (np.abs(f64(y) - want) <= bound + ref.BF16_STEP * (np.abs(want) + bound)).all()
        return qo, ko

    # the prompt, as request 0's alone
    q, k, v = bf16(S, H * G, D), bf16(S, H, D), bf16(S, H, D)
    seq, start, slots, used = w4.kv_plan(i32([0] * R), i32([S, 0, 0]), free, table, S, page)
    _, k = rope(q, k, torch.arange(S, device="cuda", dtype=torch.int32))
    w4.w4a16_kv_append(k, v, slots, *cache)
    free = free[int(used):].contiguous()
    table[1:] = table[0]
    lens = i32([S] * R)
    shared_len = i32([S])
    for counts in ([1, 1, 1], [1, 1, 1], [1, 1, 1], [4, 2, 5]):
        T = sum(counts)
        q, k, v = bf16(T, H * G, D), bf16(T, H, D), bf16(T, H, D)
        seq, start, slots, used = w4.kv_plan(lens, i32(counts), free, table, T, page)
        positions = torch.cat([torch.arange(int(n), int(n) + c) for n, c in zip(lens, counts)]).int().cuda()
        q, k = rope(q, k, positions)
        bounds = dict(max_new=max(counts), max_shared=S, max_own=64)
        need = w4.w4a16_kv_attention_shared_workspace_bytes(T, R, max(counts), S, 64, H * G, *cache)
        ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
        ws2 = torch.empty((w4.w4a16_sample_workspace_bytes(T, vocab),), dtype=torch.uint8, device="cuda")
        out, logits = torch.empty_like(q), torch.empty((T, vocab), device="cuda")
        tokens, share = torch.empty((T,), dtype=torch.int32, device="cuda"), torch.empty((T,), device="cuda")
        u = torch.from_numpy(rng.random(T)).float().cuda()
        temperature, top_k = torch.full((T,), 0.9, device="cuda"), i32([40] * T)

        def after_append():
            w4.w4a16_kv_attention_shared(q, *cache, table, seq, start, shared_len, out, ws, **bounds)
            logits.copy_(out.flatten(1).float() @ head.T)
            w4.w4a16_sample(logits, u, temperature, top_k, None, None, tokens, share, ws2)

        w4.w4a16_kv_append(k, v, slots, *cache)
        if graph:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                after_append()
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                after_append()
            tokens.fill_(-5)
            out.fill_(float("nan"))
            g.replay()
        else:
            after_append()
        torch.cuda.synchronize()
        kc, vc = kv_reference.to_values(cache[0], False), kv_reference.to_values(cache[1], True)
        ks, vs = (kv_reference.host_scales(t) for t in cache[2:])
        want, tol = ref.shared_attention(f64(q), kc, ks, vc, vs, table.cpu().numpy(), seq.tolist(), start.tolist(),
                                         D ** -0.5, S, 64)
        assert (np.abs(f64(out) - want) <= tol).all()
        x = f64(logits)
        for t in range(T):
            token, part = ref.sample(x[t], float(u[t]), float(temperature[t]), 40)
            assert int(tokens[t]) == token
            assert abs(float(share[t]) - part) <= (ref.F32_STEP + vocab * 2.0 ** -50) * part
        free = free[int(used):].contiguous()
        lens = seq
    assert lens.tolist() == [S + 3 + c for c in (4, 2, 5)]


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_the_example_stack_with_all_of_them(kind):
    """It runs; the hidden rows behind shared pages are those of the plain attention over the same pages (bound: some
    ten bf16 roundings of 2^-9 a layer for two layers, 2-norm: 4%), and drawn tokens are the vocabulary's."""
    import decode_layers as ex

    say("example", kind)
    g = torch.Generator().manual_seed(7)
    prompt, own = (torch.randint(0, 1024, (n,), dtype=torch.int32, generator=g).cuda() for n in (96, 33))
    rows = []
    for shared in (True, False):
        s = ex.Stack(layers=2, ffn=2560, vocab=1024, requests=3, max_len=192, page=32, kind=kind, rope_base=10000.0)
        s.share(prompt)
        assert s.lens.tolist() == [96] * 3 and s.free.numel() == 3 * 6 - 3
        if not shared:
            s.shared = 0                  # (the pages stay; every request reads them by itself)
        _, h = s.step(own, [30, 2, 1])
        _, h1 = s.step(own[:3], [1, 1, 1])
        _, h2 = s.step(own[:9], [2, 4, 3])
        rows.append(torch.cat([h, h1, h2]))
        u = torch.linspace(0, 0.99, 9).cuda()
        drawn = s.draw(h2, u, 0.8, top_k=50, top_p=0.95, min_p=0.01)
        assert ((drawn >= 0) & (drawn < 1024)).all()
        best = w4.matmul_prefill(h2, *s.embedding).float().argmax(1)
        assert (s.draw(h2, u, 0.0) == best).all()
        assert s.lens.tolist() == [129, 103, 101]
        if shared:
            with pytest.raises(ValueError, match="share"):
                s.keep([129, 103, 95])
    diff = float((rows[0].float() - rows[1].float()).norm() / rows[1].float().norm())
    print("relative difference", diff)
    assert diff < 0.04
    with pytest.raises(ValueError, match="share"):
        s.share(prompt)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_the_example_stack_reads_shared_entries_by_their_number(kind, monkeypatch):
    """From share_from shared entries on by one call for all requests, else each for itself; the hidden rows are the same
    (to the bound above)."""
    import decode_layers as ex

    say("example, share_from", kind)
    g = torch.Generator().manual_seed(9)
    prompt, own = (torch.randint(0, 1024, (n,), dtype=torch.int32, generator=g).cuda() for n in (64, 9))
    calls = []
    call = w4.kv_attention_shared
    monkeypatch.setattr(w4, "kv_attention_shared", lambda *a, **k: (calls.append(1), call(*a, **k))[1])
    rows = []
    for share_from, made in ((64, 4), (0, 4), (65, 0)):
        s = ex.Stack(layers=2, ffn=2560, vocab=1024, requests=3, max_len=128, page=32, kind=kind, rope_base=10000.0,
                     share_from=share_from)
        s.share(prompt)
        calls.clear()
        _, h = s.step(own, [5, 3, 1])
        _, h1 = s.step(own[:3], [1, 1, 1])
        assert len(calls) == made
        rows.append(torch.cat([h, h1]).float())
    assert torch.equal(rows[0], rows[1])
    diff = float((rows[0] - rows[2]).norm() / rows[2].norm())
    print("relative difference", diff)
    assert diff < 0.04
