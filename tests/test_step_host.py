"""Checks of a serving step's entry points (include/w4a16_step.h) that need no GPU: exports, refusals before anything is
launched (fake, never dereferenced pointers), the binding's checks, and the test oracle's own pins."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import decode_w4a16_affine_amd as w4
import step_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w4a16_step.h")

OK, ENULL, ESHAPE, EUNSUP, EALIGN, EWS = range(6)
A16 = 0x10000


@pytest.fixture(scope="module")
def L():
    return w4.step_lib()


def header_text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_every_declared_symbol_is_exported(L):
    names = set(re.findall(r"\b(w4a16_[a-z0-9_]+)\s*\(", header_text()))
    assert names == set(w4.STEP_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def constant(name):
    m = re.search(rf"#define W4A16_{name} (?:\(1 << (\d+)\)|(\d+))", header_text())
    return 1 << int(m.group(1)) if m.group(1) else int(m.group(2))


def test_rope_constants_match_the_header():
    assert constant("ROPE_MAX_AXES") == w4.ROPE_MAX_AXES
    assert constant("ROPE_NORM") == w4.ROPE_NORM and constant("ROPE_INTERLEAVED") == w4.ROPE_INTERLEAVED


def test_rope_refuses_bad_arguments(L):
    def rope(q=A16, qs=256, k=A16, ks=128, qw=A16, kw=A16, f=A16, pos=A16, sec=None, axes=1, qo=A16, qos=256, ko=A16, kos=128,
             flags=1, T=3, HQ=4, H=2, D=64, rot=64):
        sec = None if sec is None else (ctypes.c_int * len(sec))(*sec)
        return L.w4a16_qk_norm_rope(q, qs, k, ks, qw, kw, 0.0, f, pos, sec, axes, qo, qos, ko, kos, 1e-6, flags, T, HQ, H, D,
                                    rot, None)

    for bad in (dict(D=0), dict(D=96), dict(D=512), dict(flags=4), dict(flags=-1), dict(axes=0), dict(axes=5),
                dict(axes=-1)):
        assert rope(**bad) == EUNSUP, bad
    for bad in (dict(T=-1), dict(T=2 ** 20 + 1), dict(HQ=-1), dict(H=-1), dict(HQ=2 ** 16 + 1), dict(H=2 ** 16 + 1),
                dict(rot=-8), dict(rot=72), dict(rot=12), dict(qs=248), dict(ks=120), dict(qs=257), dict(kos=132),
                dict(qos=255), dict(qs=2 ** 40 + 8), dict(axes=2, sec=[16, 15]), dict(axes=2, sec=[33, -1]),
                dict(axes=3, sec=[16, 17, 0]), dict(axes=2, sec=[2 ** 31 - 1, 2 ** 31 - 1])):
        assert rope(**bad) == ESHAPE, bad
    for bad in ("q", "k", "f", "pos", "qo", "ko"):
        assert rope(**{bad: None}) == ENULL, bad
    assert rope(axes=2) == ENULL
    for bad in ("q", "k", "qw", "kw", "f", "qo", "ko"):
        assert rope(**{bad: A16 + 8}) == EALIGN, bad
    assert rope(pos=A16 + 2) == EALIGN
    assert rope(T=0) == OK and rope(HQ=0, H=0) == OK
    assert rope(T=0, q=None, k=None) == OK




def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_rope_binding_refuses_bad_tensors():
    q, k, f, pos = host(3, 4, 64), host(3, 2, 64), host(32, dtype=torch.float32), host(3, dtype=torch.int32)
    for bad, kind in ((dict(q=q.float()), TypeError), (dict(q=q[0]), ValueError), (dict(k=host(2, 2, 64)), ValueError),
                      (dict(k=host(3, 2, 128)), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                      (dict(q=None, k=None), ValueError), (dict(inv_freq=f.double()), TypeError),
                      (dict(inv_freq=f[None]), ValueError), (dict(positions=pos.long()), TypeError),
                      (dict(positions=pos[:2]), ValueError), (dict(positions=None), ValueError),
                      (dict(inv_freq=None), ValueError), (dict(sections=[16, 16]), ValueError),
                      (dict(sections=[31], positions=pos[None]), ValueError), (dict(sections=[]), ValueError),
                      (dict(sections=[33, -1], positions=host(2, 3, dtype=torch.int32)), ValueError),
                      (dict(sections=[8, 8, 8, 4, 4], positions=host(5, 3, dtype=torch.int32)), ValueError),
                      (dict(q_weight=host(32)), ValueError), (dict(k_weight=host(64, dtype=torch.float32)), TypeError),
                      (dict(), ValueError)):      # (host tensors)
        with pytest.raises(kind):
            w4.qk_norm_rope(**{**dict(q=q, k=k, inv_freq=f, positions=pos), **bad})
    with pytest.raises(ValueError):
        w4.w4a16_qk_norm_rope(q, k, None, None, f, pos, q, None)
    with pytest.raises(ValueError):
        w4.w4a16_qk_norm_rope(q, k, None, None, f, pos, q[:, :3], k)


def test_rope_definition_by_hand():
    """Two elements a pair, a quarter turn, weights and the two ways of pairing."""
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 40] = 3.0, 5.0, 2.0
    f = np.zeros(32)
    f[0] = np.pi / 2
    y, _ = ref.rope(x, None, 0.0, 0.0, False, f, np.array([[1]]), None, False)
    assert np.allclose([y[0, 0, 0], y[0, 0, 32], y[0, 0, 1], y[0, 0, 40]], [0, 3, 5, 2])
    y, _ = ref.rope(x, None, 0.0, 0.0, False, f, np.array([[1]]), None, True)
    assert np.allclose([y[0, 0, 0], y[0, 0, 1], y[0, 0, 40]], [-5, 3, 2])
    f[:] = np.pi / 2
    y, _ = ref.rope(x, None, 0.0, 0.0, False, f, np.array([[0], [1]]), [8, 24], False)      # pair 8 is of axis 1
    assert np.allclose([y[0, 0, 0], y[0, 0, 8], y[0, 0, 40]], [3, -2, 0])
    w = np.full(64, 0.5)
    y, _ = ref.rope(x, w, 1.0, 0.0, True, np.zeros(0), np.array([[0]]), None, False)
    assert np.allclose(y[0, 0, 0], 3 * 1.5 / np.sqrt(38 / 64))
