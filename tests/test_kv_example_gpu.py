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


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_rejected_candidates_leave_no_trace(kind):
    """Verify steps that reject some candidates, over page ends: the pages are all there afterwards, and the rows of the
    accepted tokens are those of one prompt (within the bound above: rejected tokens are of the same kind, so the
    scales that they may leave behind are those of some more tokens in the page)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_layers as ex

    make = lambda: ex.Stack(layers=2, ffn=2560, vocab=1024, requests=2, max_len=192, page=16, kind=kind)  # noqa: E731
    g = torch.Generator().manual_seed(9)
    first, second, junk = (torch.randint(0, 1024, (n,), dtype=torch.int32, generator=g).cuda() for n in (90, 70, 64))
    _, want = make().step(torch.cat([first, second]), [90, 70])
    s = make()
    _, h = s.step(torch.cat([first[:45], second[:30]]), [45, 30])
    rows = [list(h.split([45, 30]))]
    accepted = [(1, 3), (2, 1), (4, 4), (1, 2), (3, 2), (4, 3), (2, 4), (4, 4)]
    for a, b in accepted:
        lo = s.lens.tolist()
        # the accepted tokens, then wrong candidates, of each request; seven tokens each, so that pages are opened
        part = torch.cat([first[lo[0]:lo[0] + a], junk[:7 - a], second[lo[1]:lo[1] + b], junk[-(7 - b):]])
        _, h = s.step(part, [7, 7])
        rows.append([h[:a], h[7:7 + b]])
        s.keep([lo[0] + a, lo[1] + b])
        held = s.table[s.table >= 0].tolist()
        assert sorted(held + s.free.tolist()) == list(range(24)) and len(held) == sum(-(-n // 16) for n in s.lens.tolist())
    n = s.lens.tolist()
    assert n == [45 + sum(a for a, _ in accepted), 30 + sum(b for _, b in accepted)]
    for r, (at, count) in enumerate(((0, n[0]), (90, n[1]))):
        assert rel(torch.cat([x[r] for x in rows]), want[at:at + count]) < BOUND[kind]
    with pytest.raises(ValueError, match="asked to keep"):
        s.keep([n[0] + 1, n[1]])


def test_verify_keeps_the_stack_s_own_choices():
    """A candidate that is the stack's own next token stays, and what follows a wrong one does not."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_layers as ex

    prompt = torch.randint(0, 1024, (41,), dtype=torch.int32, generator=torch.Generator().manual_seed(3)).cuda()

    def verify(change):
        s = ex.Stack(layers=1, ffn=2560, vocab=1024, requests=2, max_len=128, page=16)
        best, _ = s.step(prompt, [30, 11])
        after, stay = s.verify(*change(best[ex.last_of([30, 11])]))
        assert s.lens.tolist() == [31 + int(stay[0]), 12 + int(stay[1])]
        assert s.free.numel() == 16 - sum(-(-n // 16) for n in s.lens.tolist())
        return after, stay.tolist()

    wrong = torch.zeros((2, 5), dtype=torch.int32, device="cuda")
    own, stay = verify(lambda t: (t, wrong))
    assert stay == [0, 0] and 0 not in own.tolist()
    guesses = wrong.clone()
    guesses[0, 0] = own[0]
    _, stay = verify(lambda t: (t, guesses))
    assert stay == [1, 0]
    guesses[1, 0] = own[1]
    _, stay = verify(lambda t: (t, guesses))
    assert stay == [1, 1]


def test_a_request_longer_than_the_stack_is_refused():
    """Nothing is written, taken or counted by a step that would pass max_len; one that just fits is fine."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_layers as ex

    s = ex.Stack(layers=1, ffn=2560, vocab=1024, requests=2, max_len=40, page=16)
    tokens = torch.arange(61, dtype=torch.int32, device="cuda")
    s.step(tokens[:50], [30, 20])
    before = [t.clone().view(torch.uint8) for t in (*s.caches[0], s.table, s.free, s.lens)]
    with pytest.raises(ValueError, match="41 tokens in a stack of max_len 40"):
        s.step(tokens[:12], [11, 1])
    for t, b in zip((*s.caches[0], s.table, s.free, s.lens), before):
        assert torch.equal(t.view(torch.uint8), b)
    s.step(tokens[:11], [10, 1])
    assert s.lens.tolist() == [40, 21]
