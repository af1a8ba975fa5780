"""The example stack (examples/decode_layers.py): prompt, decode and verify steps agree with each other.

The same tokens brought one by one, as a verify batch, or as one prompt give
the same hidden rows up to rounding: bf16 rounding of every layer's activations
(relative 2^-9 each, some ten roundings a layer) and the cache's codes, which
depend on the order in which a page's scale grows (int8: half a step of 1/127
of a page's largest entry, about 1/250 of it, an entry's own size being a third
of that: 2^-6.5 relative; E4M3: 2^-4.5).  The rows are compared in the 2-norm,
where independent roundings average over the elements: bounds of 4% (int8) and
8% (E4M3) for two layers.
"""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu
BOUND = {"int8": 0.04, "fp8": 0.08}


def rel(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("window", [0, 50])
def test_steps_agree_however_tokens_arrive(kind, window):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_layers as ex

    make = lambda: ex.Stack(layers=2, ffn=2560, vocab=1024, requests=2, max_len=192, page=32, kind=kind,  # noqa: E731
                            window=window)
    g = torch.Generator().manual_seed(5)
    first, second = (torch.randint(0, 1024, (n,), dtype=torch.int32, generator=g).cuda() for n in (90, 41))
    whole = make()
    _, h = whole.step(torch.cat([first, second]), [90, 41])
    # two prompts, then three single tokens, then five candidates, of each request
    s = make()
    rows = []
    for counts in ([82, 33], [1, 1], [1, 1], [1, 1], [5, 5]):
        lo = [int(n) for n in s.lens]
        part = torch.cat([t[a:a + n] for t, a, n in zip((first, second), lo, counts)])
        _, out = s.step(part, counts)
        rows.append(out.split(counts))
    got = torch.cat([torch.cat([r[i] for r in rows]) for i in range(2)])
    assert s.lens.tolist() == [90, 41]
    err = rel(got, h)
    print(kind, window, "relative difference", err)
    assert err < BOUND[kind]
    assert rel(h[1:90], h[:89]) > 0.5        # (rows of different tokens do differ)
    # the two stacks' pages lie elsewhere and another request follows: nothing of either is seen by the other
    alone = make()
    _, h1 = alone.step(first, [90, 0])
    assert rel(h1, h[:90]) < BOUND[kind]
