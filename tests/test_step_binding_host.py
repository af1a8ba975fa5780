"""A serving step's binding without a GPU: host tensors that report a GPU stand in for device ones, and a recorder for
the library (those of test_kv_binding_host.py)."""
import contextlib

import pytest
import torch

import decode_w4a16_affine_amd as w4
from decode_w4a16_affine_amd import step
from test_kv_binding_host import Library, OnGpu, gpu


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
    monkeypatch.setattr(step, "step_lib", lambda: lib)
    monkeypatch.setattr(step, "_current_device", lambda: state["device"])
    monkeypatch.setattr(step, "_raw_stream", lambda stream, dev: 1000 + dev if stream is None else stream)
    monkeypatch.setattr(torch.cuda, "device", device)
    return lib


def z(*shape, dtype=torch.bfloat16):
    return gpu(torch.zeros(shape, dtype=dtype))


def _on(dev, t):
    t = gpu(t)
    t.gpu = dev
    return t


def i32(*shape):
    return z(*shape, dtype=torch.int32)


def f32(*shape):
    return z(*shape, dtype=torch.float32)


def calls(out=True):
    """Every function with arguments that it takes."""
    cache = tuple(gpu(t) for t in w4.kv_cache(4, 2, 64, 16, device="cpu"))
    q, k, f, pos = z(3, 4, 64), z(3, 2, 64), f32(32), i32(3)
    attn = (q, *cache, i32(2, 4), i32(2), i32(3), i32(1))
    bounds = dict(max_new=2, max_shared=20, max_own=30)
    x, u = f32(3, 50), f32(3)
    ws = z(1 << 20, dtype=torch.uint8)
    return {
        "w4a16_qk_norm_rope": [lambda **s: w4.w4a16_qk_norm_rope(q, k, z(64), None, f, pos, q, k, **s),
                               lambda **s: w4.qk_norm_rope(q, k, z(64), None, f, pos, **s)],
        "w4a16_kv_attention_shared": [lambda **s: w4.w4a16_kv_attention_shared(*attn, q, ws, **bounds, **s),
                                      lambda **s: w4.kv_attention_shared(*attn, **bounds, **s)],
        "w4a16_sample": [lambda **s: w4.w4a16_sample(x, u, u, i32(3), u, None, i32(3), u, ws, **s),
                         lambda **s: w4.sample(x, u, u, i32(3), u, None, **s)],
    }


@pytest.mark.parametrize("name", ["w4a16_qk_norm_rope", "w4a16_kv_attention_shared", "w4a16_sample"])
@pytest.mark.parametrize("form", [0, 1])
def test_calls_run_on_their_tensors_gpu(library, name, form):
    """With another GPU current the call goes to theirs and its stream, and the other is current again afterwards."""
    for current in (1, 0):
        library.state["device"], library.calls = current, []
        calls()[name][form]()
        (made,) = [c for c in library.calls if c[0] == name]
        assert made[1] == OnGpu.gpu and made[2][-1] == 1000 + OnGpu.gpu
        assert library.state["device"] == current


@pytest.mark.parametrize("name", ["w4a16_qk_norm_rope", "w4a16_kv_attention_shared", "w4a16_sample"])
def test_a_stream_of_the_caller_s_is_passed_on(library, name):
    calls()[name][0](stream=77)
    (made,) = [c for c in library.calls if c[0] == name]
    assert made[2][-1] == 77 and made[1] == OnGpu.gpu


def test_tensors_of_two_gpus_are_refused(library):
    other = _on(0, torch.zeros((3, 2, 64), dtype=torch.bfloat16))
    q, f, pos = z(3, 4, 64), f32(32), i32(3)
    with pytest.raises(ValueError, match="one device"):
        w4.qk_norm_rope(q, other, inv_freq=f, positions=pos)
    with pytest.raises(ValueError, match="one device"):
        w4.w4a16_qk_norm_rope(q, None, None, None, f, pos, _on(0, torch.zeros((3, 4, 64), dtype=torch.bfloat16)), None)
    x, u = f32(3, 50), _on(0, torch.zeros(3))
    with pytest.raises(ValueError, match="one device"):
        w4.sample(x, u)
    with pytest.raises(ValueError, match="one device"):
        w4.w4a16_sample(x, f32(3), None, None, None, None, _on(0, torch.zeros(3, dtype=torch.int32)), None, None)
    cache = tuple(gpu(t) for t in w4.kv_cache(4, 2, 64, 16, device="cpu"))
    with pytest.raises(ValueError, match="one device"):
        w4.kv_attention_shared(q, *cache, i32(2, 4), i32(2), i32(3), _on(0, torch.zeros(1, dtype=torch.int32)), max_new=2,
                               max_shared=20, max_own=30)
    assert all(c[0].endswith("_workspace_bytes") for c in library.calls)
