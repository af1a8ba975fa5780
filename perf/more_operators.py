"""What a serving step runs around the cache and the products as workloads: sizes, inputs, plain forms, exact values.

Three operators (all in decode_w4a16_affine_amd):
  * rope:   norms of queries and keys for each head and the position rotation, in one pass between the q/k/v
            products and w4a16_kv_append; positions of one axis, or of several (time, height, width);
  * shared: attention of decode and verify steps over the paged 8-bit cache for a batch whose requests begin with
            the same entries, which are read once for all of them;
  * sample: tokens drawn from logits with temperature, top-k, top-p and min-p of each row, from given random numbers.

rope.  y = x / sqrt(mean(x^2) + eps) * weight over a head's D elements; pair i (elements i and i + rot / 2, or 2 i and
2 i + 1) of the first `rot` elements turns by position * inv_freq[i]; with several axes, pair i takes its position
from the axis whose section it lies in.

shared.  Row at position pos of request r attends entries 0 .. pos; entry j lies in page table[0][j / P] for
j < shared and table[r][j / P] from there on.

sample.  w = exp((logit - largest) / temperature).  In the order of falling logits (ties: lowest index first), a token
is kept if fewer than top_k come before it (0: all), if the weights before it sum to less than top_p of those that
top_k kept, and if w >= min_p; the first always is.  The token is the first in index order whose running sum of kept
weights exceeds u times their sum; temperature 0 takes the largest logit.  Also returned: the token's share of the
kept weights.

`own` chooses between the plain forms (elementary torch operations) and the framework's kernels; both take what
`prepare` returns.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
QMAX = {"int8": 127.0, "fp8": 448.0}
TORCH_TYPE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
BASE = 1000000.0        # of the rotation's frequencies
EPS = 1e-6
NEG_INF = float("-inf")


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one user, one token (10 query heads and 2 cache heads of 256): the latency of a single decode layer
        dict(name="rope_token", op="rope", tokens=1, prompts=0, q_heads=10, kv_heads=2, dim=256, rot=256, style="half",
             sections="", norm=True, packed=False, pos_hi=9000, spread=1),
        # a serving batch of decode steps at far positions, q, k and v parts of one projected row
        dict(name="rope_batch", op="rope", tokens=48, prompts=0, q_heads=32, kv_heads=8, dim=128, rot=128, style="half",
             sections="", norm=True, packed=True, pos_hi=120001, spread=2),
        # three prompts at once, half of each head rotated in neighbouring pairs
        dict(name="rope_prompt", op="rope", tokens=11801, prompts=3, q_heads=32, kv_heads=8, dim=128, rot=64,
             style="pairs", sections="", norm=True, packed=False, pos_hi=12000, spread=3),
        # a prompt of video frames between text: positions of time, height and width
        dict(name="rope_axes", op="rope", tokens=4099, prompts=1, q_heads=16, kv_heads=4, dim=128, rot=128, style="half",
             sections="16,24,24", norm=True, packed=True, pos_hi=2000, spread=4),
        # one user: a token of a large vocabulary
        dict(name="sample_single", op="sample", rows=1, vocab=262144, dtype="fp32", params="all", spread=5),
        # a serving batch whose requests ask for different things, greedy ones among them
        dict(name="sample_batch", op="sample", rows=48, vocab=262144, dtype="bf16", params="mixed", spread=6),
        # nucleus sampling over a vocabulary of odd size: rows that begin off every alignment
        dict(name="sample_nucleus", op="sample", rows=16, vocab=100003, dtype="fp32", params="top_p", spread=7),
        # a large batch that is only tempered: every logit counts
        dict(name="sample_free", op="sample", rows=256, vocab=262144, dtype="fp32", params="free", spread=8),
        # a few requests behind a short common instruction
        dict(name="shared_small", op="shared", kind="int8", requests=8, q_heads=10, kv_heads=2, dim=256, page=64,
             shared=1501, own_lo=5, own_hi=300, new_lo=1, new_hi=1, spread=9),
        # a serving batch behind a long common instruction with examples
        dict(name="shared_batch", op="shared", kind="fp8", requests=64, q_heads=32, kv_heads=8, dim=128, page=32,
             shared=8000, own_lo=50, own_hi=2000, new_lo=1, new_hi=1, spread=10),
        # many questions about one very long document
        dict(name="shared_long", op="shared", kind="int8", requests=24, q_heads=32, kv_heads=8, dim=128, page=128,
             shared=100001, own_lo=20, own_hi=900, new_lo=1, new_hi=1, spread=11),
        # speculative verify steps: k + 1 candidate tokens a request
        dict(name="shared_verify", op="shared", kind="fp8", requests=16, q_heads=16, kv_heads=4, dim=64, page=16,
             shared=6000, own_lo=30, own_hi=600, new_lo=2, new_hi=6, spread=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["rope", "sample", "shared"])
    spread = rng.randrange(1, 1 << 20)
    if op == "sample":
        vocab = _log_int(rng, 1000, 262144)
        return dict(op="sample", rows=_log_int(rng, 1, min(256, (256 << 18) // vocab)), vocab=vocab,
                    dtype=rng.choice(["fp32", "bf16"]), params=rng.choice(["all", "mixed", "top_k", "top_p", "min_p", "free"]),
                    spread=spread)
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = rng.choice([1, 2, 4, 5, 8]) * kv_heads
    if op == "rope":
        most = min(16384, 11801 * 40 * 128 // ((q_heads + kv_heads) * dim))
        tokens = _log_int(rng, 1, most)
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        sections = ""
        if rng.random() < 0.3:
            a = rng.randrange(1, rot // 2 - 1)
            b = rng.randrange(a + 1, rot // 2)
            sections = ",".join(str(n) for n in (a, b - a, rot // 2 - b))
        return dict(op="rope", tokens=tokens, prompts=rng.choice([0, 1, 3]) if tokens > 2 else 0, q_heads=q_heads,
                    kv_heads=kv_heads, dim=dim, rot=rot, style=rng.choice(["half", "pairs"]), sections=sections,
                    norm=rng.random() < 0.8, packed=rng.random() < 0.5, pos_hi=_log_int(rng, 100, 1000000), spread=spread)
    new_lo, new_hi = (1, 1) if rng.random() < 0.6 else (2, rng.randrange(3, 9))
    requests = _log_int(rng, 2, 64)
    # at most the listed products, and 100 MB of common entries and of others
    most = int(min(3.9e10 / (4 * requests * new_hi * q_heads * dim), 1e8 / (2 * kv_heads * dim)))
    shared = _log_int(rng, 20, max(21, min(100001, most)))
    if rng.random() < 0.4:      # whole pages only, as a server shares them
        shared = -(-shared // 128) * 128
    own_hi = _log_int(rng, new_hi + 1, max(new_hi + 2, min(2000, int(1e8 / (2 * kv_heads * dim * requests)))))
    return dict(op="shared", kind=rng.choice(["int8", "fp8"]), requests=requests, q_heads=q_heads, kv_heads=kv_heads,
                dim=dim, page=rng.choice([16, 32, 64, 128]), shared=shared, own_lo=new_hi, own_hi=own_hi, new_lo=new_lo,
                new_hi=new_hi, spread=spread)


def _pages(tokens, page):
    return -(-tokens // page)


def _lengths(case):
    """(entries behind the shared ones, new tokens among them) of each request: of the case alone, not of the seed."""
    rng = random.Random(case["spread"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["requests"])]
    return [max(n, rng.randint(case["own_lo"], case["own_hi"])) for n in new], new


def _positions(case):
    """[axes][tokens]: of the case alone."""
    rng = random.Random(case["spread"])
    tokens, hi = case["tokens"], case["pos_hi"]
    axes = len(case["sections"].split(",")) if case["sections"] else 1
    if not case["prompts"]:      # single tokens of as many requests
        return [[rng.randrange(hi) for _ in range(tokens)] for _ in range(axes)]
    rows = [[] for _ in range(axes)]
    cuts = sorted(rng.sample(range(1, tokens), case["prompts"] - 1))
    for lo, end in zip([0] + cuts, cuts + [tokens]):
        first = rng.randrange(hi)
        # frames of 12 x 20 patches behind 37 tokens of text, which count on all axes alike
        for i in range(end - lo):
            patch = i - 37
            steps = (patch // 240, patch // 20 % 12, patch % 20) if axes > 1 and patch >= 0 else None
            for a in range(axes):
                rows[a].append(first + (37 + steps[a] if steps else i))
    return rows


def _params(case):
    """Temperature, top_k, top_p and min_p of each row (None: off for all), of the case alone."""
    rng = random.Random(case["spread"])
    rows, kind = range(case["rows"]), case["params"]
    temperature = [rng.uniform(0.5, 1.2) for _ in rows]
    top_k = top_p = min_p = None
    if kind == "mixed":
        temperature = [rng.choice([0.0, t, t, t]) for t in temperature]
        top_k = [rng.choice([0, 0, 20, 64, 1000]) for _ in rows]
        top_p = [rng.choice([1.0, 1.0, 0.8, 0.95]) for _ in rows]
        min_p = [rng.choice([0.0, 0.0, 0.02, 0.1]) for _ in rows]
    if kind in ("all", "top_k"):
        top_k = [rng.choice([20, 50, 64]) for _ in rows]
    if kind in ("all", "top_p"):
        top_p = [rng.uniform(0.7, 0.98) for _ in rows]
    if kind in ("all", "min_p"):
        min_p = [rng.uniform(0.001, 0.1) for _ in rows]
    return temperature, top_k, top_p, min_p


# ---- inputs -------------------------------------------------------------------

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _f32(values):
    return torch.tensor(values, dtype=torch.float32, device=DEVICE)


def _filled(gen, pages, heads, page, dim, kind, transposed):
    """Codes and bf16 scales of `pages` pages of normal entries."""
    shape = (pages, heads, dim, page) if transposed else (pages, heads, page, dim)
    codes = torch.empty(shape, dtype=TORCH_TYPE[kind], device=DEVICE)
    scales = torch.empty((pages, heads), dtype=torch.bfloat16, device=DEVICE)
    step = max(1, (1 << 28) // (heads * page * dim))
    for p in range(0, pages, step):
        x = torch.randn((min(step, pages - p),) + shape[1:], generator=gen, device=DEVICE)
        s = (x.abs().amax((2, 3)) * (1.01 / QMAX[kind])).to(torch.bfloat16)
        scales[p:p + step] = s
        y = x / s.float()[:, :, None, None]
        codes[p:p + step] = torch.round(y).clamp(-127, 127).to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    st = {"op": case["op"]}
    if case["op"] == "rope":
        T, HQ, H, D = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        x = torch.randn((T, HQ + 2 * H, D), generator=gen, device=DEVICE)
        x *= torch.linspace(0.3, 4.0, HQ + 2 * H, device=DEVICE)[None, :, None]      # heads of different sizes
        x = x.to(torch.bfloat16)
        q, k = x[:, :HQ], x[:, HQ:HQ + H]
        if not case["packed"]:
            q, k = q.contiguous(), k.contiguous()
        weights = 1.0 + 0.3 * torch.randn((2, D), generator=gen, device=DEVICE)
        weights = weights.to(torch.bfloat16) if case["norm"] else (None, None)
        half = case["rot"] // 2
        inv_freq = _f32([BASE ** (-i / half) for i in range(half)])
        positions = _i32(_positions(case))
        sections = [int(n) for n in case["sections"].split(",")] if case["sections"] else None
        return dict(st, q=q, k=k, q_weight=weights[0], k_weight=weights[1], inv_freq=inv_freq, norm=case["norm"],
                    positions=positions if sections else positions[0], sections=sections, pairs=case["style"] == "pairs")
    if case["op"] == "sample":
        M, N = case["rows"], case["vocab"]
        logits = torch.randn((M, N), generator=gen, device=DEVICE) * 2.0
        # some tokens of each row stand out, as after a trained head
        some = torch.randint(0, N, (M, 60), generator=gen, device=DEVICE)
        logits.scatter_reduce_(1, some, 6.0 + 6.0 * torch.rand((M, 60), generator=gen, device=DEVICE), "amax")
        logits[:, N - N // 100:] = NEG_INF       # padding of the vocabulary
        logits = logits.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
        temperature, top_k, top_p, min_p = _params(case)
        opt = lambda v, f: None if v is None else f(v)  # noqa: E731
        return dict(st, logits=logits, uniforms=torch.rand((M,), generator=gen, device=DEVICE),
                    temperature=_f32(temperature), top_k=opt(top_k, _i32), top_p=opt(top_p, _f32), min_p=opt(min_p, _f32))
    owned, new = _lengths(case)
    page, shared, heads, dim, kind = case["page"], case["shared"], case["kv_heads"], case["dim"], case["kind"]
    whole = shared // page          # pages that all requests hold; a page that the prefix ends in is each one's own
    need = [_pages(shared + n, page) for n in owned]
    pages = whole + sum(n - whole for n in need) + 5
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((len(new), max(need)), -1, dtype=torch.int32, device=DEVICE)
    table[:, :whole] = order[:whole]
    at = whole
    for r, n in enumerate(need):
        table[r, whole:n] = order[at:at + n - whole]
        at += n - whole
    st["k_cache"], st["k_scales"] = _filled(gen, pages, heads, page, dim, kind, False)
    st["v_cache"], st["v_scales"] = _filled(gen, pages, heads, page, dim, kind, True)
    q = torch.randn((sum(new), case["q_heads"], dim), generator=gen, device=DEVICE)
    q *= torch.linspace(0.5, 3.0, case["q_heads"], device=DEVICE)[None, :, None]     # heads of different sharpness
    return dict(st, q=q.to(torch.bfloat16), block_table=table, seq_lens=_i32([shared + n for n in owned]),
                token_start=_i32([sum(new[:r]) for r in range(len(new) + 1)]), shared_len=_i32([shared]),
                shared=shared, max_new=max(new), max_own=max(owned), scale=1.0 / math.sqrt(dim))


# ---- one pass -----------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import decode_w4a16_affine_amd as w4

    if st["op"] == "rope":
        q, k = w4.qk_norm_rope(st["q"], st["k"], st["q_weight"], st["k_weight"], st["inv_freq"], st["positions"],
                               eps=EPS, norm=st["norm"], interleaved=st["pairs"], sections=st["sections"])
        return {"q": q, "k": k}
    if st["op"] == "sample":
        tokens, share = w4.sample(st["logits"], st["uniforms"], st["temperature"], st["top_k"], st["top_p"], st["min_p"])
        return {"tokens": tokens, "share": share}
    return w4.kv_attention_shared(st["q"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                                  st["block_table"], st["seq_lens"], st["token_start"], st["shared_len"],
                                  max_new=st["max_new"], max_shared=st["shared"], max_own=st["max_own"],
                                  scale=st["scale"])


def _run_plain(st):
    return {"rope": _rope_plain, "sample": _sample_plain, "shared": _shared_plain}[st["op"]](st)


def _rope_plain(st):
    positions, half = st["positions"], st["inv_freq"].numel()
    if st["sections"]:
        axis = torch.tensor([a for a, n in enumerate(st["sections"]) for _ in range(n)], device=DEVICE)
        positions = positions[axis].T                                    # [T, pairs]
    else:
        positions = positions[:, None]
    angle = positions.double() * st["inv_freq"].double()                   # far positions: 32 bits would lose turns
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = []
    for x, weight in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
        x = x.float()
        if st["norm"]:
            x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight.float()
        y = x.clone()
        if st["pairs"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            y[..., :half], y[..., half:2 * half] = a * cos - b * sin, a * sin + b * cos
        out.append(y.to(torch.bfloat16))
    return {"q": out[0], "k": out[1]}


def _sample_plain(st):
    """In 64 bits throughout: whether a token is kept or drawn is decided next to a border."""
    v = st["logits"].double()
    M, N = v.shape
    temperature = st["temperature"].double()[:, None]
    greedy = ~(temperature > 0)
    scale = torch.where(greedy, 1.0, temperature)
    ordered, index = torch.sort(v, dim=1, descending=True, stable=True)
    w = torch.exp((ordered - ordered[:, :1]) / scale)
    place = torch.arange(N, device=DEVICE)[None, :]
    keep = place == place
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep = (place < k) | (k <= 0)
    if st["top_p"] is not None:
        left = torch.where(keep, w, 0.0)
        before = torch.cumsum(left, 1) - left
        p = st["top_p"].double()[:, None]
        keep = keep & ((before < p * left.sum(1, keepdim=True)) | (p >= 1.0))
    if st["min_p"] is not None:
        keep = keep & (w >= st["min_p"].double()[:, None])
    keep = (keep & ~greedy) | (place == 0)
    kept = torch.zeros_like(v).scatter_(1, index, torch.where(keep, w, 0.0))
    running = torch.cumsum(kept, 1)
    total = running[:, -1:]
    tokens = (running <= st["uniforms"].double()[:, None] * total).sum(1, keepdim=True)
    last = (kept > 0).to(torch.int32).mul_(place + 1).amax(1, keepdim=True) - 1
    tokens = torch.minimum(tokens, last)
    share = kept.gather(1, tokens) / total
    return {"tokens": tokens[:, 0].to(torch.int32), "share": share[:, 0].float()}


def _values(st, table, transposed):
    """Entries [..., heads, columns * page, D] of a table [..., columns]."""
    codes, scales = (st["v_cache"], st["v_scales"]) if transposed else (st["k_cache"], st["k_scales"])
    x = codes[table].float() * scales[table].float()[..., None, None]
    if transposed:
        x = x.transpose(-1, -2)
    x = x.transpose(-4, -3)
    return x.reshape(x.shape[:-3] + (x.shape[-3] * x.shape[-2], x.shape[-1]))


def _shared_plain(st):
    """The common entries once for all rows, each request's own after them, one softmax over both."""
    table = st["block_table"].clamp(min=0).long()
    R, width = table.shape
    tokens, HQ, D = st["q"].shape
    H, page = st["k_cache"].shape[1:3]
    group, most, shared = HQ // H, st["max_new"], st["shared"]
    start, seq = st["token_start"], st["seq_lens"]
    count = start[1:] - start[:-1]
    i = torch.arange(most, device=DEVICE, dtype=torch.int32)[None, :]
    rows = (start[:-1, None] + i).clamp(max=tokens - 1).long()
    q = st["q"].float()[rows].reshape(R, most, H, group, D).permute(2, 0, 1, 3, 4).reshape(H, R, most * group, D)
    pos = ((seq - count)[:, None] + i).repeat_interleave(group, dim=1)                # [R, rows]
    # the common entries
    columns = _pages(shared, page)
    k, v = (_values(st, table[0, :columns], t)[:, :shared] for t in (False, True))
    j = torch.arange(shared, device=DEVICE, dtype=torch.int32)
    near = torch.matmul(q.reshape(H, -1, D), k.transpose(1, 2)).view(H, R, -1, shared) * st["scale"]
    near = near.masked_fill_(j > pos[..., None], NEG_INF)
    # each request's own
    first = shared // page
    ko, vo = (_values(st, table[:, first:], t).transpose(0, 1) for t in (False, True))      # [H, R, L, D]
    j = first * page + torch.arange(ko.shape[2], device=DEVICE, dtype=torch.int32)
    far = torch.matmul(q, ko.transpose(2, 3)) * st["scale"]
    far = far.masked_fill_((j > pos[..., None]) | (j < shared), NEG_INF)
    top = torch.maximum(near.amax(3, keepdim=True), far.amax(3, keepdim=True))
    near, far = torch.exp(near.sub_(top)), torch.exp(far.sub_(top))
    total = near.sum(3, keepdim=True) + far.sum(3, keepdim=True)
    out = torch.matmul(near.view(H, -1, shared), v).view(H, R, -1, D) + torch.matmul(far, vo)
    out = (out / total).view(H, R, most, group, D).permute(1, 2, 0, 3, 4).reshape(R, most, HQ, D)
    return out[i < count[:, None]].to(torch.bfloat16)


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    if case["op"] == "rope":
        elements = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        axes = len(case["sections"].split(",")) if case["sections"] else 1
        # rows read and written, positions, frequencies and weights; squares, factors and rotation
        return {"bytes": 4 * elements + 4 * case["tokens"] * axes + 2 * case["rot"] + 4 * case["dim"],
                "flops": 7 * elements}
    if case["op"] == "sample":
        size = case["rows"] * case["vocab"]
        return {"bytes": size * (4 if case["dtype"] == "fp32" else 2) + 28 * case["rows"], "flops": 4 * size}
    owned, new = _lengths(case)
    page, row, q_row = case["page"], case["kv_heads"] * case["dim"], case["q_heads"] * case["dim"]
    entries = case["shared"] + sum(owned)
    pages = _pages(case["shared"], page) + sum(_pages(case["shared"] + n, page) - case["shared"] // page for n in owned)
    pairs = sum(n * (case["shared"] + o) - n * (n - 1) // 2 for o, n in zip(owned, new))
    return {"bytes": 2 * entries * row + 4 * sum(new) * q_row + pages * (4 + 4 * case["kv_heads"]),
            "flops": 4 * pairs * q_row}


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _rope_exact, "sample": _sample_exact, "shared": _shared_exact}[case["op"]](case, st)


def _rope_exact(case, st):
    """Each pair as a complex number."""
    half, D = case["rot"] // 2, case["dim"]
    rows = torch.tensor(_positions(case), dtype=torch.float64, device=DEVICE)
    turn = torch.empty((case["tokens"], half), dtype=torch.float64, device=DEVICE)
    sizes = [int(n) for n in case["sections"].split(",")] if case["sections"] else [half]
    lo = 0
    for a, n in enumerate(sizes):
        turn[:, lo:lo + n] = torch.outer(rows[a], st["inv_freq"][lo:lo + n].double())
        lo += n
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]
    if case["style"] == "pairs":
        re = torch.arange(half, device=DEVICE) * 2
        im = re + 1
    else:
        re = torch.arange(half, device=DEVICE)
        im = re + half
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        if case["norm"]:
            x = x * (D / (x.square().sum(2, keepdim=True) + D * EPS)).sqrt() * st[name + "_weight"].double()
        z = torch.complex(x[..., re], x[..., im]) * turn
        x[..., re], x[..., im] = z.real, z.imag
        out[name] = x
    return out


def _sample_exact(case, st):
    """Row by row: shares of the ordered tokens, cut, and searched in index order."""
    temperature, top_k, top_p, min_p = _params(case)
    as_f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    tokens, shares = [], []
    for r in range(case["rows"]):
        x = st["logits"][r].double()
        order = torch.argsort(-x, stable=True)
        t = as_f32(temperature[r])
        if t == 0:
            tokens.append(int(order[0]))
            shares.append(1.0)
            continue
        logs = (x[order] - x[order[0]]) / t
        n = int((logs > NEG_INF).sum())
        if top_k is not None and top_k[r] > 0:
            n = min(n, top_k[r])
        share = torch.softmax(logs[:n], 0)
        if top_p is not None and top_p[r] < 1.0:
            n = 1 + int((torch.cumsum(share, 0)[:-1] < as_f32(top_p[r])).sum())
        if min_p is not None and min_p[r] > 0:
            n = min(n, max(1, int((logs >= math.log(as_f32(min_p[r]))).sum())))
        kept, _ = torch.sort(order[:n])
        weight = torch.exp((x[kept] - x[order[0]]) / t)
        running = torch.cumsum(weight, 0)
        at = int(torch.searchsorted(running, st["uniforms"][r].double() * running[-1], right=True))
        at = min(at, n - 1)
        tokens.append(int(kept[at]))
        shares.append(float(weight[at] / running[-1]))
    return {"tokens": _i32(tokens), "share": torch.tensor(shares, dtype=torch.float64, device=DEVICE)}


def _shared_exact(case, st):
    """Request by request and cache head by cache head, over one list of entries."""
    owned, new = _lengths(case)
    page, shared, dim, group = case["page"], case["shared"], case["dim"], case["q_heads"] // case["kv_heads"]
    if sum(shared + o for o in owned) * case["kv_heads"] * dim > 2e11:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
    begin = 0
    for r, (o, n) in enumerate(zip(owned, new)):
        length = shared + o
        at = torch.arange(length, device=DEVICE)
        ids = torch.where(at < shared, st["block_table"][0, at // page], st["block_table"][r, at // page]).long()
        pos = length - n + torch.arange(n, device=DEVICE)
        for h in range(case["kv_heads"]):
            k = st["k_cache"][ids, h, at % page].double() * st["k_scales"][ids, h].double()[:, None]
            v = st["v_cache"][ids, h, :, at % page].double() * st["v_scales"][ids, h].double()[:, None]
            for g in range(h * group, (h + 1) * group):
                s = (st["q"][begin:begin + n, g].double() @ k.T) / math.sqrt(dim)
                s[at[None, :] > pos[:, None]] = NEG_INF
                out[begin:begin + n, g] = torch.softmax(s, 1) @ v
        begin += n
    return out
