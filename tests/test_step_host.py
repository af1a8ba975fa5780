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


def test_sample_constants_match_the_header():
    assert constant("SAMPLE_MAX_ROWS") == w4.SAMPLE_MAX_ROWS and constant("SAMPLE_MAX_N") == w4.SAMPLE_MAX_N


def test_sample_refuses_bad_arguments(L):
    need = L.w4a16_sample_workspace_bytes(3, 1000)

    def sample(x=A16, dtype=1, stride=1000, u=A16, t=A16, k=A16, p=A16, m=A16, tokens=A16, share=A16, ws=A16, ws_bytes=need,
               M=3, N=1000):
        return L.w4a16_sample(x, dtype, stride, u, t, k, p, m, tokens, share, ws, ws_bytes, M, N, None)

    for bad in (dict(dtype=2), dict(dtype=-1)):
        assert sample(**bad) == EUNSUP, bad
    for bad in (dict(M=-1), dict(M=65537), dict(N=-1), dict(N=2 ** 20 + 1, stride=2 ** 21), dict(stride=999),
                dict(stride=-1), dict(stride=2 ** 40 + 1)):
        assert sample(**bad) == ESHAPE, bad
    for bad in ("x", "tokens"):
        assert sample(**{bad: None}) == ENULL, bad
    for bad in ("x", "u", "t", "k", "p", "m", "tokens", "share"):
        assert sample(**{bad: A16 + 2}) == EALIGN, bad
    assert sample(x=A16 + 1, dtype=0) == EALIGN
    assert need > 0 and sample(ws=None) == EWS and sample(ws_bytes=need - 1) == EWS and sample(ws=A16 + 8) == EALIGN
    assert sample(M=0) == OK and sample(M=0, x=None, tokens=None, ws=None, ws_bytes=0) == OK
    # rows go through in turns of 16384 chunks of 8192 tokens
    ws = L.w4a16_sample_workspace_bytes
    assert ws(65536, 2 ** 20) == ws(64, 2 ** 20) < 200 << 20 and ws(65536, 1) == ws(8192, 1) > ws(8191, 1)
    assert ws(0, 5) == 0 and ws(5, 0) == 0
    assert L.w4a16_sample_workspace_bytes(-1, 5) == 0 and L.w4a16_sample_workspace_bytes(5, 2 ** 20 + 1) == 0


def test_sample_binding_refuses_bad_tensors():
    x, f, i = host(3, 50, dtype=torch.float32), host(3, dtype=torch.float32), host(3, dtype=torch.int32)
    for bad, kind in ((dict(logits=x.double()), TypeError), (dict(logits=x[0]), ValueError), (dict(logits=x.T), ValueError),
                      (dict(logits=x[:1].expand(3, 50)), ValueError), (dict(uniforms=f.double()), TypeError),
                      (dict(uniforms=f[:2]), ValueError), (dict(temperature=f[:, None]), ValueError),
                      (dict(top_k=f), TypeError), (dict(top_k=i[:1]), ValueError), (dict(top_p=i), TypeError),
                      (dict(min_p=i), TypeError), (dict(), ValueError)):      # (host tensors)
        with pytest.raises(kind):
            w4.sample(**{**dict(logits=x, uniforms=f), **bad})
    for tokens, share, ws in ((f, f, None), (i[:1], f, None), (i, i, None), (i, f[:2], None), (i, f, f), (None, f, None)):
        with pytest.raises((TypeError, ValueError)):
            w4.w4a16_sample(x, f, None, None, None, None, tokens, share, ws)
    with pytest.raises(ValueError):
        w4.w4a16_sample_workspace_bytes(2 ** 33, 5)
    with pytest.raises(ValueError, match="32 bits"):      # (its low 32 bits would be no rows)
        w4.sample(torch.empty((2 ** 32, 0)))


def test_sample_definition_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.05, 0.4, 0.05]))
    pick = lambda u, **kw: ref.sample(x, u, **kw)[0]  # noqa: E731
    assert [pick(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.54, 0.56, 0.94, 0.96, 1.5)] == [0, 0, 1, 1, 2, 2, 3, 3, 4, 4]
    assert [pick(u, top_k=1) for u in (0.0, 0.99)] == [1, 1]                 # the lower index of equal ones
    assert [pick(u, top_k=2) for u in (0.49, 0.51)] == [1, 3]
    assert [pick(u, top_p=0.3) for u in (0.0, 0.99)] == [1, 1]
    assert [pick(u, top_p=0.5) for u in (0.49, 0.51)] == [1, 3]
    assert pick(0.99, top_p=0.85) == 3 and pick(0.0, top_p=0.85) == 0
    assert pick(0.0, min_p=0.3) == 1 and pick(0.0, min_p=0.2) == 0
    assert pick(0.99, top_k=4, top_p=0.99) == 3 and pick(0.53, top_k=4) == 2    # 0.05 of 0.95: the lower index
    assert ref.sample(x, 0.2, top_k=2)[1] == pytest.approx(0.5)
    assert pick(0.9, temperature=0.0) == 1 and pick(None) == 1
    assert pick(0.9, min_p=2.0) == 1 and pick(0.9, top_p=0.0) == 1
    x[2] = -np.inf
    assert ref.sample(x, 0.525)[0] == 1 and ref.sample(x, 1.0)[0] == 4
    assert ref.sample(np.full(3, -np.inf), 0.5) == (-1, 0.0)
    x[4] = np.inf
    assert ref.sample(x, 0.0) == (4, 1.0)
    x[3] = np.nan
    assert ref.sample(x, 0.0)[0] == 3


def cache(k=A16, v=A16, ks=A16, vs=A16, kind=0, pages=8, heads=2, page=64, dim=128):
    return ctypes.byref(w4.KVCache(k, v, ks, vs, kind, pages, heads, page, dim))


def test_shared_attention_refuses_bad_arguments(L):
    sizes = (3, 3, 2, 500, 100, 8)
    need = L.w4a16_kv_attention_shared_workspace_bytes(*sizes, cache())
    assert need > 0

    def attn(q=A16, stride=1024, c=None, table=A16, width=10, seq=A16, start=A16, s=A16, out=A16, T=3, R=3, new=2, shared=500,
             own=100, HQ=8, ws=A16, ws_bytes=need):
        return L.w4a16_kv_attention_shared(q, stride, cache() if c is None else c, table, width, seq, start, s, out, 0.1, T, R, new, shared,
                                           own, HQ, ws, ws_bytes, None)

    for bad in (dict(kind=2), dict(dim=96), dict(page=48)):
        assert attn(c=cache(**bad)) == EUNSUP, bad
    for bad in (dict(heads=0), dict(heads=1025), dict(pages=-1), dict(pages=2 ** 25), dict(pages=0)):
        assert attn(c=cache(**bad)) == ESHAPE, bad
    for bad in (dict(T=-1), dict(T=2 ** 20 + 1), dict(R=-1), dict(R=2 ** 20 + 1), dict(new=-1), dict(shared=-1), dict(own=-1),
                dict(shared=2 ** 28 + 1), dict(own=2 ** 28 + 1), dict(HQ=0), dict(HQ=7), dict(width=-1),
                dict(width=2 ** 22 + 1), dict(stride=1016), dict(stride=1028), dict(stride=2 ** 40 + 8)):
        assert attn(**bad) == ESHAPE, bad
    assert attn(HQ=130, stride=2 ** 20) == EUNSUP                   # 65 heads a cache head
    assert attn(new=17) == EUNSUP                                   # 17 tokens of 4 heads: over 64 rows
    assert attn(T=2 ** 20, R=2 ** 20, c=cache(heads=8), HQ=512, new=1, stride=2 ** 20) == ESHAPE
    for bad in ("q", "table", "seq", "start", "s", "out"):
        assert attn(**{bad: None}) == ENULL, bad
    for bad in ("q", "out"):
        assert attn(**{bad: A16 + 8}) == EALIGN, bad
    for bad in ("table", "seq", "start", "s"):
        assert attn(**{bad: A16 + 2}) == EALIGN, bad
    for bad in ("k", "v"):
        assert attn(c=cache(**{bad: None})) == ENULL and attn(c=cache(**{bad: A16 + 8})) == EALIGN
    assert attn(ws_bytes=need - 1) == EWS and attn(ws=None) == EWS and attn(ws=A16 + 8) == EALIGN
    assert attn(c=ctypes.POINTER(w4.KVCache)()) == ENULL
    for empty in (dict(T=0), dict(R=0), dict(new=0)):
        assert attn(**empty, q=None, ws=None, ws_bytes=0) == OK, empty
    ws = L.w4a16_kv_attention_shared_workspace_bytes
    assert ws(0, 3, 2, 500, 100, 8, cache()) == 0 and ws(3, 3, 17, 500, 100, 8, cache()) == 0
    assert ws(3, 3, 2, 0, 0, 8, cache()) == 0
    # few rows: 500 entries in four parts of 128; two chunks of 128 for 100 that may begin inside one
    assert need == 3 * 8 * (4 + 2) * (128 + 5) * 4
    # more: tiles of 64 for a workgroup a CU, 8000 entries in 16 parts of eight
    assert ws(64, 64, 1, 8000, 100, 32, cache(heads=8)) == 64 * 32 * (16 + 2) * (128 + 5) * 4


def test_shared_attention_binding_refuses_bad_tensors():
    c = w4.kv_cache(4, 2, 64, 16, device="cpu")
    i = lambda *n: host(*n, dtype=torch.int32)  # noqa: E731
    good = dict(q=host(3, 4, 64), block_table=i(2, 5), seq_lens=i(2), token_start=i(3), shared_len=i(1), max_new=2,
                max_shared=20, max_own=30)
    for bad, kind in ((dict(q=host(3, 4, 128)), ValueError), (dict(q=good["q"].float()), TypeError),
                      (dict(block_table=i(3, 5)), ValueError), (dict(seq_lens=i(2).long()), TypeError),
                      (dict(token_start=i(2)), ValueError), (dict(shared_len=i(2)), ValueError),
                      (dict(shared_len=i(1).float()), TypeError), (dict(max_own=2 ** 31), ValueError),
                      (dict(max_shared=2 ** 40), ValueError), (dict(), ValueError)):      # (host tensors)
        with pytest.raises(kind):
            kw = {**good, **bad}
            w4.kv_attention_shared(kw.pop("q"), *c, **kw)
    for out, ws in ((host(3, 4, 128), None), (host(3, 4, 64).float(), None), (host(3, 4, 64), host(5))):
        with pytest.raises((TypeError, ValueError)):
            kw = dict(good)
            w4.w4a16_kv_attention_shared(kw.pop("q"), *c, **kw, out=out, workspace=ws)


def test_shared_entries_by_hand():
    table = np.array([[3, 1, 7], [9, 4, 5]])
    assert ref.entry_table(table, [5, 6], 2, 3, 2).tolist() == [[6, 7, 2, 3, 14, -1], [6, 7, 2, 9, 10, -1]]
    assert ref.entry_table(table, [5, 2], 2, 0, 9).tolist() == [[6, 7, 2, 3, 14], [18, 19, 8, 9, 10]]


@pytest.mark.parametrize("N", [1, 8192, 8193, 100003, 262144, 1 << 20])
def test_sampling_takes_turns_of_8192_chunks(L, N):
    """A chunk is 8192 logits: no more rows than 8192 chunks hold have workspace, whatever a call's rows."""
    ws = L.w4a16_sample_workspace_bytes
    turn = 8192 // -(-N // 8192)
    assert ws(turn - 1, N) < ws(turn, N) == ws(turn + 1, N) == ws(65536, N)
    assert ws(turn, N) < 153 * 10 ** 6


def test_rope_without_queries_and_keys_is_refused_on_a_stream_too():
    for stream in (None, 0):
        with pytest.raises(ValueError, match="both None"):
            w4.qk_norm_rope(None, None, stream=stream)
