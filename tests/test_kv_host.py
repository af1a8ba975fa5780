"""Checks of the key/value cache's entry points that need no GPU: exports,
refusals before anything is launched (fake, never dereferenced pointers), the
binding's shape checks, and the test oracle's own pins."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import decode_w4a16_affine_amd as w4
import kv_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "w4a16_kv.h")

OK, ENULL, ESHAPE, EUNSUP, EALIGN, EWS = range(6)
A16 = 0x10000
A4 = 0x20004


@pytest.fixture(scope="module")
def L():
    return w4.kv_lib()


def header_text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_every_declared_symbol_is_exported(L):
    names = set(re.findall(r"\b(w4a16_kv_[a-z0-9_]+)\s*\(", header_text()))
    assert names == set(w4.KV_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def test_binding_constants_match_the_header():
    text = header_text()
    for name, value in (("REQUESTS", w4.KV_MAX_REQUESTS), ("TOKENS", w4.KV_MAX_TOKENS), ("WIDTH", w4.KV_MAX_WIDTH)):
        m = re.search(rf"#define W4A16_KV_MAX_{name} \(1 << (\d+)\)", text)
        assert m and 1 << int(m.group(1)) == value, name
    for name, value in (("HEADS", w4.KV_MAX_HEADS), ("GROUP", w4.KV_MAX_GROUP)):
        m = re.search(rf"#define W4A16_KV_MAX_{name} (\d+)", text)
        assert m and int(m.group(1)) == value, name
    assert re.search(rf"W4A16_KV_INT8 = {w4.KV_INT8}\b", text) and re.search(rf"W4A16_KV_FP8 = {w4.KV_FP8}\b", text)


def cache(k=A16, v=A16, ks=A16, vs=A16, kind=0, pages=8, heads=2, page=64, dim=128):
    return ctypes.byref(w4.KVCache(k, v, ks, vs, kind, pages, heads, page, dim))


BAD_CACHES = [
    (dict(kind=2), EUNSUP), (dict(kind=-1), EUNSUP), (dict(dim=96), EUNSUP), (dict(dim=0), EUNSUP),
    (dict(dim=512), EUNSUP), (dict(page=8), EUNSUP), (dict(page=48), EUNSUP), (dict(page=512), EUNSUP),
    (dict(page=0), EUNSUP), (dict(heads=0), ESHAPE), (dict(heads=1025), ESHAPE), (dict(pages=-1), ESHAPE),
    (dict(pages=2 ** 25, page=64), ESHAPE), (dict(pages=2 ** 31 - 1, page=16), ESHAPE),
    (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(ks=None), ENULL), (dict(vs=None), ENULL),
    (dict(k=A4), EALIGN), (dict(v=A16 + 8), EALIGN), (dict(ks=A16 + 1), EALIGN), (dict(vs=A16 + 1), EALIGN),
]


def test_plan_refuses_bad_arguments(L):
    def plan(ctx=A16, new=A16, free=A16, nf=8, table=A16, width=4, seq=A16, start=A16, slots=A16, used=A16, R=2, T=3,
             page=64):
        return L.w4a16_kv_plan(ctx, new, free, nf, table, width, seq, start, slots, used, R, T, page, None)

    for page in (0, 8, 24, 512, -16):
        assert plan(page=page) == EUNSUP
    for bad in (dict(R=-1), dict(R=2 ** 20 + 1), dict(T=-1), dict(T=2 ** 20 + 1), dict(nf=-1), dict(width=-1),
                dict(width=2 ** 22 + 1)):
        assert plan(**bad) == ESHAPE, bad
    for bad in ("ctx", "new", "free", "table", "seq", "start", "slots", "used"):
        assert plan(**{bad: None}) == ENULL, bad
        assert plan(**{bad: A16 + 2}) == EALIGN, bad


def test_append_refuses_bad_arguments(L):
    def app(k=A16, ks=256, v=A16, vs=256, slots=A16, T=4, pages=8):
        return L.w4a16_kv_append(k, ks, v, vs, slots, cache(pages=pages), T, None)

    for args, want in BAD_CACHES:
        assert L.w4a16_kv_append(A16, 256, A16, 256, A16, cache(**args), 4, None) == want, args
    assert L.w4a16_kv_append(A16, 256, A16, 256, A16, None, 4, None) == ENULL
    assert app(T=-1) == ESHAPE and app(T=2 ** 20 + 1) == ESHAPE
    for bad in (0, 248, 257, -256, 2 ** 41):
        assert app(ks=bad) == ESHAPE and app(vs=bad) == ESHAPE, bad
    for name in ("k", "v", "slots"):
        assert app(**{name: None}) == ENULL, name
    assert app(k=A4) == EALIGN and app(v=A16 + 8) == EALIGN and app(slots=A16 + 2) == EALIGN
    assert app(T=0, k=None, v=None, slots=None) == OK
    assert app(pages=0, k=None) == OK


def test_attention_refuses_bad_arguments(L):
    def att(q=A16, qs=1024, table=A16, width=4, seq=A16, start=A16, out=A16, window=0, T=3, R=2, mn=2, ml=256, HQ=8,
            ws=A16, wb=1 << 40, **cache_args):
        return L.w4a16_kv_attention(q, qs, cache(**cache_args), table, width, seq, start, out, 1.0, window, T, R, mn,
                                    ml, HQ, ws, wb, None)

    for args, want in BAD_CACHES:
        assert att(**args) == want, args
    for bad in (dict(T=-1), dict(T=2 ** 20 + 1), dict(R=-1), dict(R=2 ** 20 + 1), dict(mn=-1), dict(ml=-1),
                dict(ml=2 ** 29 + 1), dict(window=-1), dict(HQ=0), dict(HQ=7), dict(HQ=-2), dict(width=-1),
                dict(width=2 ** 22 + 1), dict(qs=1023), dict(qs=1016), dict(qs=1028), dict(qs=2 ** 41)):
        assert att(**bad) == ESHAPE, bad
    assert att(HQ=130, qs=130 * 128) == EUNSUP          # 65 query heads a cache head
    assert att(pages=0) == ESHAPE
    assert att(T=2 ** 19, HQ=512, heads=512, qs=512 * 128) == ESHAPE           # a launch of over 2^22 workgroups
    assert att(T=2 ** 20, HQ=2048, heads=1024, qs=2048 * 128) == ESHAPE        # T * HQ = 2^31
    assert att(pages=2 ** 21, page=16, heads=1024) == ESHAPE                  # pages * heads = 2^31
    for name in ("q", "table", "seq", "start", "out"):
        assert att(**{name: None}) == ENULL, name
    assert att(q=A4) == EALIGN and att(out=A16 + 8) == EALIGN and att(table=A16 + 2) == EALIGN
    assert att(seq=A16 + 1) == EALIGN and att(start=A16 + 2) == EALIGN
    for empty in (dict(T=0), dict(R=0), dict(mn=0)):
        assert att(q=None, out=None, **empty) == OK, empty


def test_attention_workspace_rules(L):
    def ws(T=4, R=4, mn=1, ml=4096, window=0, HQ=8, **cache_args):
        return L.w4a16_kv_attention_workspace_bytes(T, R, mn, ml, window, HQ, cache(**cache_args))

    assert ws(T=-1) == 0 and ws(HQ=7) == 0 and ws(dim=96) == 0 and ws(ml=2 ** 29 + 1) == 0
    need = ws()
    if need:
        def att(wsp, wb):
            return L.w4a16_kv_attention(A16, 1024, cache(), A16, 64, A16, A16, A16, 1.0, 0, 4, 4, 1, 4096, 8, wsp, wb,
                                        None)
        assert att(A16, need - 1) == EWS and att(None, need) == EWS and att(A16 + 8, need) == EALIGN


def test_attention_workspace_is_sized_by_the_rows_that_can_need_it(L):
    """(D + 5) floats a row and chunk, for the rows of T tokens or of R requests of 64 / G tokens, whichever is less."""
    def ws(T, R, mn, ml=4096, HQ=32, heads=8, **cache_args):
        return L.w4a16_kv_attention_workspace_bytes(T, R, mn, ml, 0, HQ, cache(heads=heads, **cache_args))

    row = 133 * 4               # D 128
    assert ws(256, 256, 1) == 256 * 32 * 16 * row                # 4096 entries: chunks of 256
    assert ws(256, 256, 16) == ws(256, 256, 1)                   # a bound of more tokens than there are
    assert ws(600, 256, 4) == 600 * 32 * 16 * row
    assert ws(1024, 256, 4) == 1024 * 32 * 16 * row == ws(1500, 256, 4)
    # single tokens beside a prompt chunk, behind histories of up to 131072 (64 chunks): not 4.5 GB
    assert ws(2255, 256, 2000, ml=131072) == 2255 * 32 * 64 * row
    assert ws(8192, 256, 2000, ml=131072) == 256 * 16 * 32 * 64 * row
    # statistics end on 16 bytes; one chunk needs nothing
    assert ws(1, 1, 1, HQ=1, heads=1) == (16 * 128 + (16 * 5 + 3) // 4 * 4) * 4
    assert ws(256, 256, 1, ml=128) == 0


def test_attention_refuses_a_missing_or_small_workspace(L):
    """4096 entries lie in several chunks: a workspace is needed, and its absence refused."""
    need = L.w4a16_kv_attention_workspace_bytes(4, 4, 1, 4096, 0, 8, cache())
    assert need > 0

    def att(ws, size):
        return L.w4a16_kv_attention(A16, 1024, cache(), A16, 64, A16, A16, A16, 1.0, 0, 4, 4, 1, 4096, 8, ws, size, None)
    assert att(A16, need - 1) == EWS and att(A16, 0) == EWS and att(None, need) == EWS and att(A16 + 8, need) == EALIGN


def test_dequant_refuses_bad_arguments(L):
    for args, want in BAD_CACHES:
        assert L.w4a16_kv_dequant(cache(**args), A16, 3, A16, A16, None) == want, args
    dq = L.w4a16_kv_dequant
    assert dq(None, A16, 3, A16, A16, None) == ENULL
    assert dq(cache(), A16, -1, A16, A16, None) == ESHAPE
    assert dq(cache(), None, 3, A16, A16, None) == ENULL and dq(cache(), A16, 3, None, A16, None) == ENULL
    assert dq(cache(), A16, 3, A16, None, None) == ENULL
    assert dq(cache(), A16 + 2, 3, A16, A16, None) == EALIGN and dq(cache(), A16, 3, A16 + 4, A16, None) == EALIGN
    assert dq(cache(k=None), None, 0, None, None, None) == OK


def test_dequant_refuses_more_pages_than_a_launch_holds(L):
    """2^24 pages of 256 threads are 2^32 on a grid's axis: an argument error, not a refused launch."""
    text = header_text()
    assert re.search(r"#define W4A16_KV_MAX_DEQUANT \(\(1 << 24\) - 1\)", text) and w4.KV_MAX_DEQUANT == 2 ** 24 - 1
    for count in (2 ** 24, 2 ** 31 - 1):
        assert L.w4a16_kv_dequant(cache(), A16, count, A16, A16, None) == ESHAPE
    # (the largest count goes on to the pointers' checks)
    assert L.w4a16_kv_dequant(cache(), None, 2 ** 24 - 1, A16, A16, None) == ENULL


def test_binding_checks_shapes_before_the_library():
    bf, i32 = torch.bfloat16, torch.int32
    kc, vc, ks, vs = w4.kv_cache(4, 2, 64, 16, device="cpu")
    q = torch.zeros((3, 4, 64), dtype=bf)
    kv = torch.zeros((3, 2, 64), dtype=bf)
    slots, table = torch.zeros((3,), dtype=i32), torch.zeros((2, 5), dtype=i32)
    seq, start = torch.zeros((2,), dtype=i32), torch.zeros((3,), dtype=i32)
    one = torch.zeros((1,), dtype=i32)

    def raises(kind, match, fn, *a, **k):
        with pytest.raises(kind, match=match):
            fn(*a, **k)

    app = w4.w4a16_kv_append
    raises(TypeError, "k_cache must be", app, kv, kv, slots, kc.float(), vc, ks, vs)
    raises(TypeError, "v_cache must be", app, kv, kv, slots, kc, vc.to(torch.float8_e4m3fn), ks, vs)
    raises(ValueError, "v_cache must have shape", app, kv, kv, slots, kc, vc.transpose(2, 3), ks, vs)
    raises(ValueError, "k_scales must have shape", app, kv, kv, slots, kc, vc, ks[:, :1], vs)
    raises(TypeError, "v_scales must be", app, kv, kv, slots, kc, vc, ks, vs.float())
    raises(ValueError, "k_cache must be 4-D", app, kv, kv, slots, kc[0], vc, ks, vs)
    raises(ValueError, "k must have shape", app, kv[:, :1], kv, slots, kc, vc, ks, vs)
    raises(ValueError, "v must be dense", app, kv, kv.transpose(1, 2).contiguous().transpose(1, 2), slots, kc, vc, ks, vs)
    raises(TypeError, "slot_map must be", app, kv, kv, slots.long(), kc, vc, ks, vs)
    raises(ValueError, "slot_map must have shape", app, kv, kv, slots[:2], kc, vc, ks, vs)
    raises(ValueError, "same tokens", app, kv, kv[:2], slots, kc, vc, ks, vs)
    raises(ValueError, "on the GPU", app, kv, kv, slots, kc, vc, ks, vs)
    att = w4.w4a16_kv_attention
    raises(TypeError, "q must be", att, q.float(), kc, vc, ks, vs, table, seq, start, q, None, 1)
    raises(ValueError, "q must have shape", att, q[:, :, :32], kc, vc, ks, vs, table, seq, start, q, None, 1)
    raises(ValueError, "token_start must have shape", att, q, kc, vc, ks, vs, table, seq, start[:2], q, None, 1)
    raises(ValueError, "block_table must have shape", att, q, kc, vc, ks, vs, table[:1], seq, start, q, None, 1)
    raises(ValueError, "out must have shape", att, q, kc, vc, ks, vs, table, seq, start, q[:2], None, 1)
    raises(TypeError, "workspace must be", att, q, kc, vc, ks, vs, table, seq, start, q, one, 1)
    raises(ValueError, "on the GPU", att, q, kc, vc, ks, vs, table, seq, start, q, None, 1)
    plan = w4.w4a16_kv_plan
    raises(ValueError, "new_lens must have shape", plan, seq, one, one, table, seq, start, slots, one, 16)
    raises(ValueError, "block_table must have shape", plan, seq, seq, one, table[0], seq, start, slots, one, 16)
    raises(ValueError, "pages_used must have shape", plan, seq, seq, one, table, seq, start, slots, seq, 16)
    raises(TypeError, "free_pages must be", plan, seq, seq, one.long(), table, seq, start, slots, one, 16)
    raises(ValueError, "on the GPU", plan, seq, seq, one, table, seq, start, slots, one, 16)
    raises(ValueError, "k_out must have shape", w4.w4a16_kv_dequant, kc, vc, ks, vs, one, kv.float(), kv.float())


# ---- the oracle's own pins ------------------------------------------------------------

def test_oracle_scales_against_every_bf16_magnitude():
    """scale_of is the smallest admissible number: checked against its neighbours for all positive bf16 numbers."""
    bits = np.arange(1, 0x7F80, 7, dtype=np.int32)
    for b in bits:
        a = float(torch.tensor([b], dtype=torch.int16).view(torch.bfloat16).double())
        s = ref.scale_of(a, "int8")
        t = torch.tensor([s], dtype=torch.float64).to(torch.bfloat16)
        assert float(t.double()) == s                                   # a bf16 number
        below = float((t.view(torch.int16) - 1).view(torch.bfloat16).double())
        assert s * 127 >= a and (s == 2.0 ** -100 or below * 127 < a), a
        s = ref.scale_of(a, "fp8")
        assert math.frexp(s)[0] == 0.5 and s * 448 >= a and (s == 2.0 ** -100 or s / 2 * 448 < a), a
    assert ref.scale_of(0.0, "int8") == ref.scale_of(0.0, "fp8") == 2.0 ** -100
    assert math.isnan(ref.scale_of(math.inf, "int8")) and math.isnan(ref.scale_of(math.nan, "fp8"))


def test_oracle_codes_against_all_e4m3_numbers():
    every = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mids = (every[1:] + every[:-1]) / 2
    assert np.array_equal(ref.nearest_code(every, "fp8"), every)
    # a midpoint goes to the neighbour with the even last bit, a hair beside it to the nearer one
    even = np.where(np.arange(len(mids)) % 2 == 0, every[:-1], every[1:])
    assert np.array_equal(ref.nearest_code(mids, "fp8"), even)
    assert np.array_equal(ref.nearest_code(mids * (1 + 1e-9), "fp8"), every[1:])
    assert np.array_equal(ref.nearest_code(-mids * (1 - 1e-9), "fp8"), -every[:-1])


def test_oracle_attention_against_a_direct_sum():
    """One head, no scales other than 1, against a sum written with Python floats; planted faults are seen."""
    rng = np.random.default_rng(3)
    page, D, n = 16, 64, 37
    kc, vc = (np.round(rng.uniform(-9, 9, (4, 1, page, D))) for _ in range(2))
    ones = np.ones((4, 1))
    table = np.array([[2, 0, 3]])
    q = rng.standard_normal((2, 1, D))
    out, tol = ref.attention(q, kc, ones, vc, ones, table, [n], [0, 2], 0.1, 20)
    for t in range(2):
        pos = n - 2 + t
        js = range(pos - 19, pos + 1)
        k = [kc[table[0, j // page], 0, j % page] for j in js]
        v = [vc[table[0, j // page], 0, j % page] for j in js]
        e = [math.exp(0.1 * float(sum(q[t, 0, d] * kk[d] for d in range(D)))) for kk in k]
        for d in range(0, D, 9):
            assert abs(out[t, 0, d] - sum(w * vv[d] for w, vv in zip(e, v)) / sum(e)) < 1e-12
    for fault in (dict(table=[[2, 0, 1]]), dict(seq=[n - 1]), dict(window=21), dict(scale=0.101)):
        other, _ = ref.attention(q, kc, ones, vc, ones, np.array(fault.get("table", table)), fault.get("seq", [n]),
                                 [0, 2], fault.get("scale", 0.1), fault.get("window", 20))
        assert (np.abs(other - out) > tol).any(), fault


def test_oracle_append_and_plan_by_hand():
    codes, scales = np.zeros((2, 1, 16, 1)), np.zeros((2, 1))
    ref.append(np.array([[[127.0]], [[1.0]]]), [14, 15], codes, scales, "int8")
    # a run that does not begin its page keeps the larger scale: old 0, new 1
    assert scales[0, 0] == 1 and codes[0, 0, 14, 0] == 127 and codes[0, 0, 15, 0] == 1
    ref.append(np.array([[[10.0]]]), [16], codes, scales, "int8")
    assert scales[1, 0] == ref.scale_of(10.0, "int8")
    ref.append(np.array([[[254.0]]]), [17], codes, scales, "int8")
    assert scales[1, 0] == 2 and codes[1, 0, 0, 0] == 5 and codes[1, 0, 1, 0] == 127
    table, seq, start, slots, used = ref.plan([15, 0], [2, 17], [9, 8, 7], [[4, 5, 6], [1, 2, 3]], 21, 16)
    assert table.tolist() == [[4, 9, -1], [8, 7, -1]] and seq == [17, 17] and start == [0, 2, 19] and used == 3
    assert slots[:3] == [79, 144, 128] and slots[18] == 112 and slots[19:] == [-1, -1]
