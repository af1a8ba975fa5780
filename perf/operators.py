"""The paged 8-bit key/value cache operators as workloads: sizes, inputs, plain forms, exact values.

Four operators that a decode program runs between the q/k/v product and the
o product of a layer (all in decode_w4a16_affine_amd):
  * plan:      block tables and slot maps built on the GPU from request lengths;
  * append:    new keys and values quantized into 8-bit pages with one scale a
               page and head (and read back as values);
  * attention: causal grouped-query attention of one token, of a verify batch
               or of a prompt chunk over such a cache.

The cache: keys [pages, heads, page, D], values [pages, heads, D, page], both
int8 or float8_e4m3fn, with bf16 scales [pages, heads] each; a value is
code * scale.  The scale of a page and head is chosen from the largest
magnitude a of its entries: int8 takes the smallest bf16 number >= a / 127,
float8_e4m3fn the smallest power of two >= a / 448, both at least 2^-100.  A
page that is filled over several calls keeps the larger of its old and its
new scale; where it grows, the page's earlier codes are encoded again.

`own` chooses between the plain forms (elementary torch operations in 32 bits)
and the framework's kernels; both take what `prepare` returns.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
QMAX = {"int8": 127.0, "fp8": 448.0}
TORCH_TYPE = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}
TINY = 2.0 ** -100      # the smallest scale
NEG_INF = float("-inf")


# ---- cases --------------------------------------------------------------------

def listed():
    """Every size is a case's own: requests and lengths are spread by `spread` over [lo, hi]."""
    return [
        # one user, one token, a short history: the latency of a single decode layer
        # (10 query heads and 2 cache heads of 256: the 2560 <- 2560 and 512 <- 2560 projections)
        dict(name="attn_single", op="attention", kind="int8", requests=1, q_heads=10, kv_heads=2, dim=256, page=64,
             ctx_lo=716, ctx_hi=716, new_lo=1, new_hi=1, window=0, spread=1),
        # a serving batch of decode steps with ragged histories, 4 query heads a cache head
        dict(name="attn_batch", op="attention", kind="fp8", requests=48, q_heads=32, kv_heads=8, dim=128, page=32,
             ctx_lo=300, ctx_hi=6000, new_lo=1, new_hi=1, window=0, spread=2),
        # few requests with very long histories: the whole chip has to share each of them
        dict(name="attn_long", op="attention", kind="int8", requests=3, q_heads=32, kv_heads=8, dim=128, page=128,
             ctx_lo=90001, ctx_hi=120001, new_lo=1, new_hi=1, window=0, spread=3),
        # speculative verify: k + 1 candidate tokens a request at once
        dict(name="attn_verify", op="attention", kind="int8", requests=16, q_heads=10, kv_heads=2, dim=256, page=64,
             ctx_lo=1000, ctx_hi=9000, new_lo=2, new_hi=6, window=0, spread=4),
        # the sliding-window layers of the same kind of model: only the last 512 positions count
        dict(name="attn_window", op="attention", kind="fp8", requests=96, q_heads=16, kv_heads=4, dim=64, page=16,
             ctx_lo=100, ctx_hi=3100, new_lo=1, new_hi=1, window=512, spread=5),
        # one whole prompt of an odd length, nothing cached before it
        dict(name="attn_prompt", op="attention", kind="fp8", requests=1, q_heads=10, kv_heads=2, dim=256, page=64,
             ctx_lo=0, ctx_hi=0, new_lo=4099, new_hi=4099, window=0, spread=6),
        # chunks of several prompts, each behind the part that is cached already
        dict(name="attn_chunks", op="attention", kind="int8", requests=4, q_heads=32, kv_heads=8, dim=128, page=64,
             ctx_lo=0, ctx_hi=12000, new_lo=200, new_hi=2000, window=0, spread=7),
        # a decode step's keys and values into running pages
        dict(name="append_token", op="append", kind="int8", requests=64, kv_heads=8, dim=128, page=16,
             ctx_lo=1, ctx_hi=4000, new_lo=1, new_hi=1, spread=8),
        # a verify batch's candidates, across page ends
        dict(name="append_verify", op="append", kind="fp8", requests=24, kv_heads=2, dim=256, page=64,
             ctx_lo=1, ctx_hi=9000, new_lo=2, new_hi=6, spread=9),
        # prompt chunks: whole pages at once, the first and the last of each in part
        dict(name="append_prompt", op="append", kind="int8", requests=3, kv_heads=8, dim=128, page=64,
             ctx_lo=0, ctx_hi=700, new_lo=1001, new_hi=6001, spread=10),
        # the bookkeeping of one decode step
        dict(name="plan_step", op="plan", requests=40, page=64, ctx_lo=0, ctx_hi=16000, new_lo=1, new_hi=1, long=0,
             spread=11),
        # the bookkeeping of a large step in which some prompts arrive among decoding requests
        dict(name="plan_mixed", op="plan", requests=701, page=32, ctx_lo=0, ctx_hi=30000, new_lo=1, new_hi=2000,
             long=16, spread=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["attention", "attention", "attention", "attention", "append", "append", "plan"])
    spread = rng.randrange(1, 1 << 20)
    if op == "plan":
        return dict(op="plan", requests=_log_int(rng, 1, 1000), page=rng.choice([16, 32, 64, 128]), ctx_lo=0,
                    ctx_hi=_log_int(rng, 500, 30000), new_lo=1, new_hi=_log_int(rng, 1, 2000),
                    long=rng.randrange(0, 12), spread=spread)
    kind = rng.choice(["int8", "fp8"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        requests = _log_int(rng, 1, 128)
        new_hi = rng.choice([1, rng.randrange(2, 8), _log_int(rng, 100, 12000 // requests + 101)])
        new_lo = 1 if new_hi < 100 else new_hi // 4
        return dict(op="append", kind=kind, requests=requests, kv_heads=kv_heads, dim=dim, page=page, ctx_lo=0,
                    ctx_hi=_log_int(rng, 1, 6000), new_lo=new_lo, new_hi=new_hi, spread=spread)
    group = rng.choice([1, 2, 4, 5, 8])
    form = rng.choice(["token", "token", "verify", "chunk"])
    if form == "chunk":
        requests = _log_int(rng, 1, 4)
        new_hi = _log_int(rng, 64, 4000 // requests)
        new_lo = max(1, new_hi // 5)
        ctx_hi = _log_int(rng, 1, 8000)
    else:
        new_lo, new_hi = (1, 1) if form == "token" else (2, rng.randrange(3, 9))
        requests = _log_int(rng, 1, 128)
        # at most 300 MB of keys and values
        most = int(3e8 / (2 * kv_heads * dim * requests))
        ctx_hi = _log_int(rng, 30, max(31, min(most, 100000)))
    window = rng.choice([0, 0, 0, 512, rng.randrange(30, 2000)])
    return dict(op="attention", kind=kind, requests=requests, q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                page=page, ctx_lo=ctx_hi // rng.choice([2, 8, 40]), ctx_hi=ctx_hi, new_lo=new_lo, new_hi=new_hi,
                window=window, spread=spread)


def _lengths(case):
    """(tokens cached before, new tokens) of each request: of the case alone, not of the seed."""
    rng = random.Random(case["spread"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["requests"])]
    if case["op"] == "plan":
        new = [1] * case["requests"]
        for r in rng.sample(range(case["requests"]), min(case["long"], case["requests"])):
            new[r] = rng.randint(case["new_lo"], case["new_hi"])
    else:
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["requests"])]
    return ctx, new


def _pages(tokens, page):
    return -(-tokens // page)


# ---- inputs -------------------------------------------------------------------

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _tables(ctx, new, page, gen, spare=7):
    """Block table [R, widest] of distinct pages in random order, -1 past a request's need; number of pages."""
    need = [_pages(c + n, page) for c, n in zip(ctx, new)]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    width = max(1, max(need))
    need_t = _i32(need)
    first = torch.cumsum(need_t, 0, dtype=torch.int32) - need_t
    col = torch.arange(width, device=DEVICE, dtype=torch.int32)
    at = (first[:, None] + col[None, :]).clamp(max=pages - 1)
    return torch.where(col[None, :] < need_t[:, None], order[at.long()], _i32([-1])), pages


def _scale_of(amax, kind):
    """The scale of a page and head whose largest magnitude is amax (fp32 tensor), in fp32."""
    s = amax / torch.full_like(amax, QMAX[kind])     # by a number, the division would be a product
    low = 0xFFFF if kind == "int8" else 0x7FFFFF    # up to the next bf16 number, or the next power of two
    s = ((s.view(torch.int32) + low) & ~low).view(torch.float32)
    return s.clamp(min=TINY)


def _encode(x, s, kind):
    y = x / s
    return torch.round(y).to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)


def _filled(gen, pages, heads, page, dim, kind, transposed):
    """Codes and bf16 scales of `pages` full pages of normal entries."""
    shape = (pages, heads, dim, page) if transposed else (pages, heads, page, dim)
    codes = torch.empty(shape, dtype=TORCH_TYPE[kind], device=DEVICE)
    scales = torch.empty((pages, heads), dtype=torch.bfloat16, device=DEVICE)
    step = max(1, (1 << 28) // max(1, heads * page * dim))
    for p in range(0, pages, step):     # in parts: the 32-bit entries of a long cache are large
        x = torch.randn((min(step, pages - p),) + shape[1:], generator=gen, device=DEVICE)
        s = _scale_of(x.abs().amax((2, 3)), kind)
        scales[p:p + step] = s.to(torch.bfloat16)
        codes[p:p + step] = _encode(x, s[:, :, None, None], kind)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    ctx, new = _lengths(case)
    page = case["page"]
    st = {"op": case["op"], "page": page, "max_new": max(new), "tokens": sum(new)}
    if case["op"] == "plan":
        held = [_pages(c, page) for c in ctx]
        table, pages = _tables(ctx, [0] * len(ctx), page, gen, spare=sum(new) // page + len(ctx) + 5)
        used = set(table[table >= 0].tolist())
        free = torch.tensor([p for p in range(pages) if p not in used], dtype=torch.int32, device=DEVICE)
        free = free[torch.randperm(free.numel(), generator=gen, device=DEVICE)]
        width = max(_pages(c + n, page) for c, n in zip(ctx, new)) + 1
        block_table = torch.full((len(ctx), width), -1, dtype=torch.int32, device=DEVICE)
        block_table[:, :table.shape[1]] = table[:, :width]
        assert max(held) <= width
        return dict(st, ctx_lens=_i32(ctx), new_lens=_i32(new), free_pages=free, block_table=block_table)
    table, pages = _tables(ctx, new, page, gen)
    heads, dim, kind = case["kv_heads"], case["dim"], case["kind"]
    st.update(kind=kind, block_table=table, seq_lens=_i32([c + n for c, n in zip(ctx, new)]),
              token_start=_i32([sum(new[:r]) for r in range(len(new) + 1)]))
    if case["op"] == "attention":
        st["k_cache"], st["k_scales"] = _filled(gen, pages, heads, page, dim, kind, False)
        st["v_cache"], st["v_scales"] = _filled(gen, pages, heads, page, dim, kind, True)
        q = torch.randn((st["tokens"], case["q_heads"], dim), generator=gen, device=DEVICE)
        # heads of different sharpness: logits of spread 0.5 to 3
        q *= torch.linspace(0.5, 3.0, case["q_heads"], device=DEVICE)[None, :, None]
        st.update(q=q.to(torch.bfloat16), scale=1.0 / math.sqrt(dim), window=case["window"],
                  max_len=max(c + n for c, n in zip(ctx, new)))
        return st
    # append: pages that hold each request's earlier tokens, the rest empty
    k_cache = torch.zeros((pages, heads, page, dim), dtype=TORCH_TYPE[kind], device=DEVICE)
    v_cache = torch.zeros((pages, heads, dim, page), dtype=TORCH_TYPE[kind], device=DEVICE)
    k_scales = torch.zeros((pages, heads), dtype=torch.bfloat16, device=DEVICE)
    v_scales = torch.zeros_like(k_scales)
    touched, slots = [], []
    tables = table.cpu()
    for r, (c, n) in enumerate(zip(ctx, new)):
        first = c // page
        mine = tables[r, first:_pages(c + n, page)].tolist()
        touched += mine
        held = c - first * page
        if held:    # the running page: earlier entries of half the new ones' spread, so that scales grow
            kc, ks = _filled(gen, 1, heads, page, dim, kind, False)
            vc, vs = _filled(gen, 1, heads, page, dim, kind, True)
            k_cache[mine[0], :, :held] = kc[0, :, :held]
            v_cache[mine[0], :, :, :held] = vc[0, :, :, :held]
            k_scales[mine[0]] = ks[0] * 0.5
            v_scales[mine[0]] = vs[0] * 0.5
        pos = torch.arange(c, c + n)
        slots.append(tables[r, pos // page].long() * page + pos % page)
    # keys and values as two parts of one projected row a token
    kv = torch.randn((st["tokens"], 2, heads, dim), generator=gen, device=DEVICE).to(torch.bfloat16)
    st.update(k=kv[:, 0], v=kv[:, 1], slot_map=torch.cat(slots).to(torch.int32).to(DEVICE), pages=_i32(touched),
              k_cache=k_cache, v_cache=v_cache, k_scales=k_scales, v_scales=v_scales)
    return st


# ---- one pass -----------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import decode_w4a16_affine_amd as w4

    if st["op"] == "plan":
        seq_lens, token_start, slot_map, pages_used = w4.kv_plan(
            st["ctx_lens"], st["new_lens"], st["free_pages"], st["block_table"], st["tokens"], st["page"])
        return {"block_table": st["block_table"], "seq_lens": seq_lens, "token_start": token_start,
                "slot_map": slot_map, "pages_used": pages_used}
    cache = (st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"])
    if st["op"] == "append":
        w4.w4a16_kv_append(st["k"], st["v"], st["slot_map"], *cache)
        k, v = w4.kv_dequant(*cache, st["pages"])
        return {"k": k, "v": v, "k_scales": st["k_scales"], "v_scales": st["v_scales"]}
    return w4.kv_attention(st["q"], *cache, st["block_table"], st["seq_lens"], st["token_start"], st["max_new"],
                           max_len=st["max_len"], scale=st["scale"], window=st["window"])


def _run_plain(st):
    return {"plan": _plan_plain, "append": _append_plain, "attention": _attention_plain}[st["op"]](st)


def _owner(token_start, tokens):
    """Request and index within the request of each token."""
    tok = torch.arange(tokens, device=DEVICE, dtype=torch.int32)
    r = torch.searchsorted(token_start[1:], tok, right=True)
    return r, tok - token_start[r]


def _plan_plain(st):
    ctx, new, page, free, table = st["ctx_lens"], st["new_lens"], st["page"], st["free_pages"], st["block_table"]
    seq = ctx + new
    start = torch.zeros(ctx.numel() + 1, dtype=torch.int32, device=DEVICE)
    start[1:] = torch.cumsum(new, 0, dtype=torch.int32)
    held = (ctx + page - 1) // page
    need = (seq + page - 1) // page - held
    last = torch.cumsum(need, 0, dtype=torch.int32)
    col = torch.arange(table.shape[1], device=DEVICE, dtype=torch.int32)[None, :]
    pick = (last - need)[:, None] + col - held[:, None]
    fresh = free[pick.clamp(0, free.numel() - 1).long()]
    fresh = torch.where((col < (held + need)[:, None]) & (pick < free.numel()), fresh, -1)
    table.copy_(torch.where(col < held[:, None], table, fresh))
    r, t = _owner(start, st["tokens"])
    pos = ctx[r] + t
    at = table[r, (pos // page).long()]
    slots = torch.where(at >= 0, at * page + pos % page, -1)
    return {"block_table": table, "seq_lens": seq, "token_start": start, "slot_map": slots, "pages_used": last[-1:]}


def _append_plain(st):
    kind = st["kind"]
    page = st["page"]
    pages = st["pages"].long()
    slots = st["slot_map"].long()
    local = torch.full((st["k_cache"].shape[0],), -1, dtype=torch.long, device=DEVICE)
    local[pages] = torch.arange(pages.numel(), device=DEVICE)
    at, off = local[slots // page], slots % page
    # the first slot that this call writes in each page: earlier ones are kept
    begin = torch.full((pages.numel(),), page, dtype=torch.long, device=DEVICE).scatter_reduce(0, at, off, "amin")
    kept = torch.arange(page, device=DEVICE)[None, :] < begin[:, None]
    out = {}
    out["k"] = _append_one(st["k"], st["k_cache"], st["k_scales"], False, pages, at, off, kept, kind)
    out["v"] = _append_one(st["v"], st["v_cache"], st["v_scales"], True, pages, at, off, kept, kind)
    out["k_scales"], out["v_scales"] = st["k_scales"], st["v_scales"]
    return out


def _append_one(x, cache, scales, transposed, pages, at, off, kept, kind):
    """Writes x [T, heads, D] into the pages; returns the pages' values [n, heads, page, D]."""
    x = x.float()
    amax = torch.zeros((pages.numel(), x.shape[1]), device=DEVICE)
    amax = amax.scatter_reduce(0, at[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
    old_s = torch.where(kept[:, :1], scales[pages].float(), 0.0)
    new_s = torch.maximum(old_s, _scale_of(amax, kind))
    old = cache[pages]
    wide = old.float().transpose(2, 3) if transposed else old.float()
    grown = (new_s > old_s)[:, :, None, None] & kept[:, None, :, None]
    again = _encode(wide * old_s[:, :, None, None], new_s[:, :, None, None], kind).float()
    codes = torch.where(grown, again, wide)
    codes[at, :, off] = _encode(x, new_s[at][:, :, None], kind).float()
    cache[pages] = (codes.transpose(2, 3) if transposed else codes).to(cache.dtype)
    scales[pages] = new_s.to(torch.bfloat16)
    return codes * new_s[:, :, None, None]


def _attention_plain(st):
    q, table = st["q"].float(), st["block_table"].clamp(min=0).long()
    tokens, q_heads, dim = q.shape
    requests, width = table.shape
    heads, page = st["k_cache"].shape[1], st["page"]
    length = width * page
    k = st["k_cache"][table].float() * st["k_scales"][table].float()[..., None, None]     # [R, W, H, P, D]
    k = k.permute(0, 2, 1, 3, 4).reshape(requests, heads, length, dim)
    v = st["v_cache"][table].float() * st["v_scales"][table].float()[..., None, None]     # [R, W, H, D, P]
    v = v.permute(0, 2, 1, 4, 3).reshape(requests, heads, length, dim)
    start, seq, most = st["token_start"], st["seq_lens"], st["max_new"]
    count = start[1:] - start[:-1]
    t = torch.arange(most, device=DEVICE, dtype=torch.int32)[None, :]
    rows = (start[:-1, None] + t).clamp(max=tokens - 1).long()
    grouped = q[rows].reshape(requests, most, heads, q_heads // heads, dim).permute(0, 2, 1, 3, 4)
    grouped = grouped.reshape(requests, heads, most * (q_heads // heads), dim)
    logits = torch.matmul(grouped, k.transpose(2, 3)) * st["scale"]
    pos = (seq - count)[:, None] + t                                                          # [R, most]
    j = torch.arange(length, device=DEVICE, dtype=torch.int32)
    seen = j[None, None, :] <= pos[:, :, None]
    if st["window"]:
        seen = seen & (j[None, None, :] > pos[:, :, None] - st["window"])
    seen = seen.repeat_interleave(q_heads // heads, dim=1)[:, None]
    logits = logits.masked_fill_(~seen, NEG_INF)
    top = logits.amax(3, keepdim=True)
    top = torch.where(top == NEG_INF, 0.0, top)
    p = torch.exp(logits.sub_(top))
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    out = out.reshape(requests, heads, most, q_heads // heads, dim).permute(0, 2, 1, 3, 4)
    out = out.reshape(requests, most, q_heads, dim)
    r, i = _owner(start, tokens)
    return out[r, i.long()].to(torch.bfloat16)


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    ctx, new = _lengths(case)
    page = case["page"]
    if case["op"] == "plan":
        width = max(_pages(c + n, page) for c, n in zip(ctx, new)) + 1
        taken = sum(_pages(c + n, page) - _pages(c, page) for c, n in zip(ctx, new))
        held = sum(_pages(c, page) for c in ctx)
        # lengths, tables and free pages read; the new and empty table entries, lengths and slots written
        words = 2 * len(ctx) + held + taken + (len(ctx) * width - held) + 2 * len(ctx) + 2 + sum(new)
        return {"bytes": 4 * words, "flops": 8 * (len(ctx) + sum(new))}
    row = case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        pages = sum(_pages(c + n, page) - c // page for c, n in zip(ctx, new))
        # bf16 rows read, codes written; the touched pages' codes read and their fp32 values written
        return {"bytes": 2 * (sum(new) * row * 3 + pages * page * row * 5 + pages * case["kv_heads"] * 6),
                "flops": 2 * (sum(new) * row * 3 + pages * page * row)}
    kv = pairs = 0
    for c, n in zip(ctx, new):
        window = case["window"] or c + n
        kv += min(c + n, window + n - 1)
        pairs += sum(min(c + t + 1, window) for t in range(n))
    q_row = case["q_heads"] * case["dim"]
    table = sum(_pages(c + n, page) for c, n in zip(ctx, new))
    return {"bytes": 2 * kv * row + 4 * sum(new) * q_row + table * (4 + 4 * case["kv_heads"]),
            "flops": 4 * pairs * q_row}


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return None     # whole numbers only
    if case["op"] == "append":
        return _append_exact(case, st)
    return _attention_exact(case, st)


def _attention_exact(case, st):
    """Request by request and cache head by cache head."""
    ctx, new = _lengths(case)
    if sum((c + n) * n for c, n in zip(ctx, new)) * case["q_heads"] * case["dim"] > 4e13:
        return None
    page, heads, group = case["page"], case["kv_heads"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEVICE)
    begin = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        ids = st["block_table"][r, :_pages(c + n, page)].long()
        lo = max(0, c + 1 - case["window"]) if case["window"] else 0
        for h in range(heads):
            k = st["k_cache"][ids, h].double() * st["k_scales"][ids, h].double()[:, None, None]
            v = st["v_cache"][ids, h].double() * st["v_scales"][ids, h].double()[:, None, None]
            k = k.reshape(-1, case["dim"])[lo:c + n]
            v = v.transpose(1, 2).reshape(-1, case["dim"])[lo:c + n]
            at = torch.arange(lo, c + n, device=DEVICE)
            for g in range(h * group, (h + 1) * group):
                s = (st["q"][begin:begin + n, g].double() @ k.T) / math.sqrt(case["dim"])
                own_pos = torch.arange(c, c + n, device=DEVICE)[:, None]
                hidden = at[None, :] > own_pos
                if case["window"]:
                    hidden |= own_pos - at[None, :] >= case["window"]
                s[hidden] = NEG_INF
                out[begin:begin + n, g] = torch.softmax(s, 1) @ v
        begin += n
    return out


def _exact_scale(amax, kind):
    """64-bit form of the scale rule of one number."""
    m, e = math.frexp(amax / QMAX[kind])
    if kind == "int8":
        return max(TINY, math.ldexp(math.ceil(m * 256), e - 8))
    return max(TINY, math.ldexp(1.0, e - 1 if m == 0.5 else e))


def _exact_codes(y, kind):
    """The nearest code of each 64-bit value, ties to even."""
    if kind == "int8":
        return torch.round(y)
    _, e = torch.frexp(y)
    step = (e.clamp(min=-5).long() - 4 + 1023 << 52).view(torch.float64)    # 4 significant bits, none below 2^-9
    return torch.round(y / step) * step


def _append_exact(case, st):
    """Page by page."""
    ctx, new = _lengths(case)
    page, kind, heads = case["page"], case["kind"], case["kv_heads"]
    got = {}
    for name, transposed in (("k", False), ("v", True)):
        scales = st[name + "_scales"].double().clone()
        values, begin = [], 0
        x_all = st[name].double()
        biggest = x_all.abs().amax(2).cpu()
        for r, (c, n) in enumerate(zip(ctx, new)):
            for b in range(c // page, _pages(c + n, page)):
                p = int(st["block_table"][r, b])
                lo, hi = max(c, b * page), min(c + n, (b + 1) * page)
                t0, t1, o0 = begin + lo - c, begin + hi - c, lo - b * page
                old = st[name + "_cache"][p].double()
                old = old.transpose(1, 2) if transposed else old
                was = scales[p].tolist()
                s = [_exact_scale(float(a), kind) for a in biggest[t0:t1].amax(0)]
                s = [max(a, w) if o0 else a for a, w in zip(s, was)]
                s_t = torch.tensor(s, dtype=torch.float64, device=DEVICE)[:, None, None]
                codes = old.clone()
                for h in range(heads):
                    if o0 and s[h] > was[h]:
                        codes[h, :o0] = _exact_codes(old[h, :o0] * was[h] / s_t[h], kind)
                codes[:, o0:o0 + hi - lo] = _exact_codes(x_all[t0:t1].transpose(0, 1) / s_t, kind)
                scales[p] = s_t[:, 0, 0]
                values.append(codes * s_t)
            begin += n
        got[name] = torch.stack(values)
        got[name + "_scales"] = scales
    return got
