"""The key/value cache's binding without a GPU: host tensors that report a GPU stand in for device ones, and a recorder
for the library."""
import contextlib

import pytest
import torch

import decode_w4a16_affine_amd as w4
from decode_w4a16_affine_amd import kv


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    gpu = 1

    def get_device(self):
        return self.gpu


def gpu(t):
    return t.as_subclass(OnGpu)


class Library:
    """Records each call and the GPU that was current in it."""

    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.state["device"], args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    state = {"device": 0}

    @contextlib.contextmanager
    def device(dev):
        before, state["device"] = state["device"], dev
        try:
            yield
        finally:
            state["device"] = before

    lib = Library(state)
    monkeypatch.setattr(kv, "kv_lib", lambda: lib)
    monkeypatch.setattr(kv, "_current_device", lambda: state["device"])
    monkeypatch.setattr(kv, "_current_stream", lambda dev: 1000 + dev)
    monkeypatch.setattr(torch.cuda, "device", device)
    return lib


def step(T=3, R=2, H=2, G=2, D=64, page=16):
    """Arguments of a step's calls."""
    cache = tuple(gpu(t) for t in w4.kv_cache(4, H, D, page, device="cpu"))
    q, kv_rows = (gpu(torch.zeros((T, n, D), dtype=torch.bfloat16)) for n in (H * G, H))
    i = lambda *shape: gpu(torch.zeros(shape, dtype=torch.int32))  # noqa: E731
    return cache, q, kv_rows, i(T), i(R), i(R + 1), i(R, 5), i(1)


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_tensors_gpu(library, current):
    """With another GPU current, the tensors' own is made current for the call, and its stream is taken."""
    cache, q, rows, slots, seq, start, table, one = step()
    library.state["device"] = current
    w4.w4a16_kv_plan(seq, seq, one, table, seq, start, slots, one, 16)
    w4.kv_plan(seq, seq, one, table, 3, 16)
    w4.w4a16_kv_append(rows, rows, slots, *cache)
    w4.w4a16_kv_attention(q, *cache, table, seq, start, q, None, 2)
    w4.kv_attention(q, *cache, table, seq, start, 2)
    out = gpu(torch.zeros((1, 2, 16, 64)))
    w4.w4a16_kv_dequant(*cache, one, out, out)
    w4.kv_dequant(*cache, one)
    launches = [c for c in library.calls if "workspace" not in c[0]]
    assert [c[0] for c in launches] == ["w4a16_kv_plan", "w4a16_kv_plan", "w4a16_kv_append", "w4a16_kv_attention",
                                        "w4a16_kv_attention", "w4a16_kv_dequant", "w4a16_kv_dequant"]
    for name, device, args in launches:
        assert device == 1 and args[-1] == 1001, name
    assert library.state["device"] == current


@pytest.mark.parametrize("wide", [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40, -2 ** 31 - 1, -2 ** 32 + 5])
def test_numbers_past_32_bits_are_refused(library, wide):
    """Cut to their low bits, 2^32 tokens a request would be none (rows left unwritten) and a window of 2^32 + 1 be 1."""
    cache, q, rows, slots, seq, start, table, one = step()
    refuse = lambda what: pytest.raises(ValueError, match=f"{what}.* must fit 32 bits")  # noqa: E731
    with refuse("page"):
        w4.w4a16_kv_plan(seq, seq, one, table, seq, start, slots, one, wide)
    for args in ((3, wide), (wide, 16)):
        with refuse("tokens, page"):
            w4.kv_plan(seq, seq, one, table, *args)
    for kw in (dict(max_new=wide), dict(max_new=2, max_len=wide), dict(max_new=2, window=wide)):
        with refuse("max_new, max_len, window"):
            w4.w4a16_kv_attention(q, *cache, table, seq, start, q, None, **kw)
        with refuse("max_new, max_len, window"):
            w4.kv_attention(q, *cache, table, seq, start, **kw)
    for at in range(6):
        numbers = [3, 2, 2, 64, 0, 4]
        numbers[at] = wide
        with refuse("tokens, requests"):
            w4.w4a16_kv_attention_workspace_bytes(*numbers, *cache)
    assert library.calls == []


def test_numbers_of_32_bits_reach_the_library(library):
    cache, q, rows, slots, seq, start, table, one = step()
    for n in (2 ** 31 - 1, -2 ** 31, -1):       # (what they mean is the library's to judge)
        w4.w4a16_kv_attention(q, *cache, table, seq, start, q, None, n, max_len=n, window=n)
        w4.w4a16_kv_plan(seq, seq, one, table, seq, start, slots, one, n)
    assert len(library.calls) == 6
