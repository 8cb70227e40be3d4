"""The serving operators over the 4-bit key/value cache, as they are measured.

  tables     block tables and slot maps of one scheduling step, from request lengths
  append     the step's new keys and values into the cache (group-32 signed 4-bit codes, one
             step size per group), and the written tokens back as the values they stand for
  attention  softmax attention of a ragged batch of queries over the paged cache

Quantizer of the cache: for a group of 32 channels of one token and head with largest magnitude m,
Delta = fl(m / 7) rounded up to 5 significant bits (so that Delta times any code is exactly a bf16),
limited to 2^100, and 0 where fl(m / 7) < 2^-100; code = clamp(rint(v / Delta), -8, 7), 0 where
Delta is 0.  A byte holds channel 2j in its low nibble and channel 2j + 1 in its high nibble.

Sizes: the heads of the 8B-class stack (32 query heads, 8 key/value heads of 128: hidden 4096, keys
and values 1024 wide) and of the 1B-class stack (32 and 8 of 64: hidden 2048, keys and values 512
wide); draws add other head groupings, page sizes and windows.
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------------- cases
def listed():
    att8 = dict(op="attention", q_heads=32, kv_heads=8, dim=128, window=0)
    att1 = dict(op="attention", q_heads=32, kv_heads=8, dim=64, window=0)
    return [
        # one decode step of a small batch: each request takes one token, few take a page
        dict(name="tables_step", op="tables", batch=32, held=4000, new=1, page=64),
        # admission of a wave of prompts: every page and slot of 1000 requests
        dict(name="tables_prompts", op="tables", batch=1000, held=0, new=1023, page=16),
        # the new tokens of a 48-request decode step of the 8B-class stack, cut from stacked qkv rows
        dict(name="append_step", op="append", tokens=48, kv_heads=8, dim=128, page=64, dtype="bf16", stacked=True),
        # a 16k-token prefill batch of the 8B-class stack
        dict(name="append_prompts", op="append", tokens=16411, kv_heads=8, dim=128, page=64, dtype="bf16", stacked=True),
        # a short prompt of the 1B-class stack, keys and values in float32
        dict(name="append_f32", op="append", tokens=777, kv_heads=8, dim=64, page=16, dtype="f32", stacked=False),
        # one user, one token, a chat of about a thousand tokens: latency
        dict(att8, name="decode_one", batch=1, new=1, least=999, most=999, page=64),
        # an ordinary decode batch of ragged contexts
        dict(att8, name="decode_batch", batch=64, new=1, least=511, most=8200, page=64),
        # one user with a very long document
        dict(att8, name="decode_long", batch=1, new=1, least=131071, most=131071, page=64),
        # the small model with small pages, a sliding window and many requests
        dict(att1, name="decode_window", batch=128, new=1, least=77, most=4001, page=16, window=1024),
        # a few drafted tokens of each request verified at once
        dict(att8, name="verify_draft", batch=16, new=5, least=700, most=6007, page=32),
        # the prompt of a new request
        dict(att8, name="prefill", batch=1, new=4096, least=4096, most=4096, page=64),
        # chunks of three long prompts, the earlier chunks already in the cache
        dict(att1, name="prefill_chunks", batch=3, new=1501, least=2000, most=9001, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        page = rng.choice([16, 32, 64, 128])
        op = rng.choice(["tables", "append", "attention", "attention"])
        if op == "tables":
            c = dict(op=op, batch=_log(rng, 1, 2000), held=rng.choice([0, _log(rng, 1, 20000)]),
                     new=rng.choice([1, _log(rng, 1, 1024)]), page=page)
            if c["batch"] * c["new"] > 1023000:
                continue
        elif op == "append":
            c = dict(op=op, tokens=_log(rng, 1, 16411), kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]),
                     page=page, dtype=rng.choice(["bf16", "bf16", "f32"]), stacked=rng.random() < 0.5)
        else:
            kv = rng.choice([1, 2, 4, 8])
            group = rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
            c = dict(op=op, q_heads=kv * group, kv_heads=kv, dim=rng.choice([64, 128, 128]),
                     window=rng.choice([0, 0, 0, _log(rng, 100, 4000)]), batch=1, new=1, least=1, most=1, page=page)
            if c["q_heads"] > 64:
                continue
            kind = rng.choice(["one", "batch", "draft", "prompt", "chunk"])
            if kind == "one":
                c.update(most=_log(rng, 1, 131071))
                c["least"] = c["most"]
            elif kind in ("batch", "draft"):
                c.update(batch=_log(rng, 2, 128), new=1 if kind == "batch" else rng.randint(2, 9), most=_log(rng, 64, 8200))
                c["least"] = rng.randint(c["new"], c["most"])
            else:
                c.update(batch=rng.randint(1, 3), new=_log(rng, 17, 4096))
                c["least"] = c["most"] = c["new"]
                if kind == "chunk":
                    c["most"] = c["new"] + _log(rng, 1, 8000)
                    c["least"] = rng.randint(c["new"], c["most"])
            scores = c["batch"] * c["q_heads"] * c["new"] * c["most"]
            if scores > 1.4e9 or c["batch"] * c["most"] * c["kv_heads"] * c["dim"] > 1.1e9:
                continue
        if _cost(c) <= most:
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# --------------------------------------------------------- lengths: a function of the case alone
def _lens(c):
    """Tokens of each request, the step's new ones among them: spread over least..most."""
    return [c["most"] - int((c["most"] - c["least"]) * ((i * 0.6180339887) % 1.0)) for i in range(c["batch"])]


def _table_lens(c):
    """(held, new) of each request of a tables case; in a case of several new tokens every request has its own number."""
    held = [0 if c["held"] == 0 else max(1, int(c["held"] * (0.3 + 0.7 * ((i * 0.6180339887) % 1.0)))) for i in range(c["batch"])]
    new = [1 if c["new"] == 1 else max(1, int(c["new"] * (1.0 - ((i * 0.7548776662) % 1.0)))) for i in range(c["batch"])]
    return held, new


def _pages(n, page):
    return -(-n // page)


def _attended(c):
    """(query, key) pairs of one head, and cached tokens that any query attends to, over the batch."""
    pairs = tokens = 0
    for n in _lens(c):
        first, w = n - c["new"], c["window"]
        if w:
            pairs += sum(min(p + 1, w) for p in range(first, n))
            tokens += min(n, c["new"] + w - 1)
        else:
            pairs += c["new"] * first + c["new"] * (c["new"] + 1) // 2
            tokens += n
    return pairs, tokens


def work(case):
    c = case
    if c["op"] == "tables":
        held, new = _table_lens(c)
        pages = sum(_pages(h + n, c["page"]) - _pages(h, c["page"]) for h, n in zip(held, new))
        # lengths in, new pages from the free list into the table, slots, total lengths and offsets out
        return {"bytes": 4 * (4 * c["batch"] + 1 + 2 * pages + sum(new)), "flops": 0}
    d = c["dim"]
    token = 2 * c["kv_heads"] * (d // 2 + 2 * (d // 32))  # codes and step sizes of a cached token
    if c["op"] == "append":
        n, value = c["tokens"], 2 * c["tokens"] * c["kv_heads"] * d
        # k and v in, the cache entries written and read back, the values out in bf16; slots in twice
        return {"bytes": value * (2 if c["dtype"] == "bf16" else 4) + 2 * n * token + value * 2 + 8 * n, "flops": 4 * value}
    pairs, tokens = _attended(c)
    qo = 2 * 2 * c["batch"] * c["new"] * c["q_heads"] * d
    return {"bytes": tokens * token + qo, "flops": 4 * pairs * c["q_heads"] * d}


# ------------------------------------------------------------------------------------- inputs
def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _kv(g, n, heads, dim):
    """Keys or values: normal, a few channels of each head several times larger, as projections give them."""
    gain = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device="cuda"))
    x = torch.randn(n, heads, dim, generator=g, device="cuda")
    return x.mul_(gain)


def _filled_cache(g, pages, page, heads, dim):
    """A cache whose every slot holds quantized tokens: codes [pages, heads, page, dim / 2], step sizes [pages, heads, page, dim / 32]."""
    out = []
    for _ in range(2):
        codes = torch.empty(pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
        steps = torch.empty(pages, heads, page, dim // 32, dtype=torch.bfloat16, device="cuda")
        gain = torch.exp(0.5 * torch.randn(heads, 1, dim, generator=g, device="cuda"))
        some = max(1, (1 << 27) // (heads * page * dim))
        for a in range(0, pages, some):
            x = torch.randn(min(some, pages - a), heads, page, dim, generator=g, device="cuda") * gain
            codes[a:a + some], steps[a:a + some] = _quantize(x)
        out += [codes, steps]
    return out


def prepare(case, seed):
    c, g = case, _rand(seed)
    s = {"case": c}
    if c["op"] == "tables":
        held, new = _table_lens(c)
        most = max(_pages(h + n, c["page"]) for h, n in zip(held, new))
        start = [_pages(h, c["page"]) for h in held]
        fresh = sum(_pages(h + n, c["page"]) for h, n in zip(held, new)) - sum(start)
        names = torch.randperm(sum(start) + fresh + 64, generator=g, device="cuda").to(torch.int32)
        at = torch.arange(most, device="cuda")[None, :]
        first = torch.tensor([0] + start, device="cuda").cumsum(0)[:-1, None]
        table = torch.where(at < torch.tensor(start, device="cuda")[:, None],
                            names[(first + at).clamp(max=names.numel() - 1)], torch.full_like(names[:1], -1))
        s.update(lengths=torch.tensor(held, dtype=torch.int32, device="cuda"),
                 new=torch.tensor(new, dtype=torch.int32, device="cuda"), table=table.contiguous(),
                 free=names[sum(start):].contiguous(), slots=sum(new))
        return s
    if c["op"] == "append":
        n, h, d, p = c["tokens"], c["kv_heads"], c["dim"], c["page"]
        pages = _pages(n, p) + 8
        k, v = _kv(g, n, h, d), _kv(g, n, h, d)
        if c["dtype"] == "bf16":
            k, v = k.bfloat16(), v.bfloat16()
        if c["stacked"]:  # the rows of a stacked projection: queries, keys, values
            rows = torch.cat([torch.zeros(n, 4 * h, d, dtype=k.dtype, device="cuda"), k, v], 1)
            k, v = rows[:, 4 * h:5 * h], rows[:, 5 * h:]
        # whole pages in any order, the tokens of a page in order
        page = torch.randperm(pages, generator=g, device="cuda")[:_pages(n, p)]
        slots = (page[:, None] * p + torch.arange(p, device="cuda")).reshape(-1)[:n].to(torch.int32)
        cache = []
        for _ in range(2):
            cache += [torch.zeros(pages, h, p, d // 2, dtype=torch.uint8, device="cuda"),
                      torch.zeros(pages, h, p, d // 32, dtype=torch.bfloat16, device="cuda")]
        s.update(k=k, v=v, slots=slots, cache=cache)
        return s
    lens = _lens(c)
    count = [_pages(n, c["page"]) for n in lens]
    total = sum(count) + 3
    s["cache"] = _filled_cache(g, total, c["page"], c["kv_heads"], c["dim"])
    names = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(max(count), device="cuda")[None, :]
    have = torch.tensor(count, device="cuda")[:, None]
    first = torch.tensor([0] + count, device="cuda").cumsum(0)[:-1, None]
    s["table"] = torch.where(at < have, names[(first + at).clamp(max=total - 1)], torch.full_like(names[:1], -1)).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = torch.arange(c["batch"] + 1, dtype=torch.int32, device="cuda") * c["new"]
    s["q"] = torch.randn(c["batch"] * c["new"], c["q_heads"], c["dim"], generator=g, device="cuda").bfloat16()
    s["scale"] = c["dim"] ** -0.5
    return s


# -------------------------------------------------------------------------------- plain forms
def _quantize(x):
    """Codes (two to a byte) and step sizes of x [..., dim]."""
    y = x.float().unflatten(-1, (-1, 32))
    d = y.abs().amax(-1)
    d = d / torch.full_like(d, 7)  # a division: by a number it may become a product with 1/7, which misses exact quotients
    low = (1 << 19) - 1  # 5 significant bits are all but the last 19 of the 23 stored; the carry of rounding up moves on
    step = (d.view(torch.int32).add(low) & ~low).view(torch.float32).clamp(max=2.0 ** 100)
    step = torch.where(d < 2.0 ** -100, torch.zeros_like(step), step)
    code = torch.round(y / step.unsqueeze(-1)).clamp(-8, 7)
    code = torch.where(step.unsqueeze(-1) == 0, torch.zeros_like(code), code).to(torch.int16).flatten(-2) & 15
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), step.bfloat16()


def _values(codes, steps):
    """What codes [..., dim / 2] and step sizes [..., dim / 32] stand for, in float32."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int8)
    n = torch.where(n > 7, n - 16, n).float()
    return (n.unflatten(-1, (-1, 32)) * steps.float().unsqueeze(-1)).flatten(-2)


def _plain_tables(s):
    c, table = s["case"], s["table"]
    p, most, total = c["page"], table.shape[1], s["slots"]
    held, new = s["lengths"].long(), s["new"].long()
    have = ((held + p - 1) // p).clamp(max=most)
    need = ((held + new + p - 1) // p).clamp(max=most)
    extra = need - have
    before = extra.cumsum(0) - extra
    at = torch.arange(most, device=table.device)[None, :]
    src = before[:, None] + at - have[:, None]
    page = torch.where(src < s["free"].numel(), s["free"][src.clamp(0, s["free"].numel() - 1)], -1)
    table.copy_(torch.where((at >= have[:, None]) & (at < need[:, None]), page, table))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    tok = torch.arange(total, device=table.device)
    b = torch.searchsorted(cu[1:], tok, right=True).clamp(max=new.numel() - 1)
    pos = held[b] + tok - cu[b]
    page = table[b, (pos // p).clamp(max=most - 1)].long()
    slots = torch.where((tok < cu[-1]) & (pos // p < most) & (page >= 0), page * p + pos % p, -1)
    return {"table": table, "slots": slots.int(), "lens": (held + new).int(), "cu": cu.int(), "taken": extra.sum().int()}


def _plain_append(s):
    kc, ks, vc, vs = s["cache"]
    p, at = kc.shape[2], s["slots"].long()
    page, row = at // p, at % p
    out = {}
    for name, x, codes, steps in (("k", s["k"], kc, ks), ("v", s["v"], vc, vs)):
        codes[page, :, row], steps[page, :, row] = _quantize(x)
        out[name] = _values(codes[page, :, row], steps[page, :, row]).bfloat16()
    return out


def _plain_attention(s):
    c = s["case"]
    kc, ks, vc, vs = s["cache"]
    q, cu, lens = s["q"], s["cu"].long(), s["lens"].long()
    p, most, t, heads = c["page"], c["most"], c["new"], c["kv_heads"]
    group = c["q_heads"] // heads
    pos = torch.arange(most, device=q.device)
    page = s["table"][:, pos // p].long().clamp(min=0)  # [batch, most]
    k = _values(kc[page, :, pos % p], ks[page, :, pos % p])  # [batch, most, heads, dim]
    tok = cu[:-1, None] + torch.arange(t, device=q.device)
    qb = q[tok.clamp(max=q.shape[0] - 1)].float().unflatten(2, (heads, group))  # [batch, t, heads, group, dim]
    sc = torch.einsum("bthgd,blhd->bhgtl", qb, k) * s["scale"]
    del k
    last = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(t, device=q.device)  # position of each query
    see = pos[None, None, :] <= last[:, :, None]
    if c["window"]:
        see &= pos[None, None, :] > last[:, :, None] - c["window"]
    sc = sc.masked_fill_(~see[:, None, None], float("-inf"))
    sc = (sc - sc.amax(-1, keepdim=True)).exp_()
    sc = sc / sc.sum(-1, keepdim=True)
    v = _values(vc[page, :, pos % p], vs[page, :, pos % p]).masked_fill_((pos[None, :] >= lens[:, None])[..., None, None], 0)
    o = torch.einsum("bhgtl,blhd->bthgd", sc, v).flatten(2, 3)
    return {"out": o.flatten(0, 1).bfloat16()}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention}[op](s)
    import int4_group_wise_b200 as q4
    if op == "tables":
        lens, cu, slots, taken = q4.kv4_tables(s["lengths"], s["new"], s["table"], s["free"], s["case"]["page"], s["slots"])
        return {"table": s["table"], "slots": slots, "lens": lens, "cu": cu, "taken": taken}
    cache = q4.KV4Cache(*s["cache"])
    if op == "append":
        q4.kv4_append(cache, s["k"], s["v"], s["slots"])
        k, v = q4.kv4_gather(cache, s["slots"])
        return {"k": k, "v": v}
    return {"out": q4.kv4_attention(s["q"], cache, s["table"], s["lens"], s["cu"], scale=s["scale"], window=s["case"]["window"])}


# ------------------------------------------------------------------------- by definition, 64 bits
def _exact_values(x):
    """The values that x's codes stand for, from the quantizer's definition."""
    y = x.double().reshape(*x.shape[:-1], -1, 32)
    d = y.abs().max(-1).values / 7
    unit = torch.exp2(torch.floor(torch.log2(d)) - 4)  # the fifth significant bit
    step = (torch.ceil(d / unit) * unit).clamp(max=2.0 ** 100)
    step = torch.where(d < 2.0 ** -100, 0.0, step)[..., None]
    code = torch.where(step > 0, (y / step).round().clamp(-8, 7), 0.0)
    return (code * step).reshape(x.shape)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "tables":
        held, new = _table_lens(c)
        table, free, p = s["table"].cpu(), s["free"].cpu().tolist(), c["page"]
        rows, slots, cu, taken = table.tolist(), [], [0], 0
        for b, (h, n) in enumerate(zip(held, new)):
            for i in range(_pages(h, p), _pages(h + n, p)):
                rows[b][i] = free[taken]
                taken += 1
            slots += [rows[b][x // p] * p + x % p for x in range(h, h + n)]
            cu.append(cu[-1] + n)
        i32 = torch.int32
        return {"table": torch.tensor(rows, dtype=i32), "slots": torch.tensor(slots, dtype=i32),
                "lens": torch.tensor([h + n for h, n in zip(held, new)], dtype=i32), "cu": torch.tensor(cu, dtype=i32),
                "taken": torch.tensor(taken, dtype=i32)}
    if c["op"] == "append":
        return {"k": _exact_values(s["k"]), "v": _exact_values(s["v"])}
    kc, ks, vc, vs = s["cache"]
    p, group = c["page"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c)):
        pages = s["table"][b, :_pages(n, p)].long()
        rows = slice(b * c["new"], (b + 1) * c["new"])
        at = torch.arange(n - c["new"], n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None, :]
        hide = (key > at) | ((key <= at - c["window"]) if c["window"] else (key < 0))
        for h in range(c["kv_heads"]):
            kv = []
            for codes, steps in ((kc, ks), (vc, vs)):
                byte = codes[pages, h].reshape(-1, c["dim"] // 2)[:n].long()
                code = torch.stack([byte % 16, byte // 16], 2).reshape(n, c["dim"]).double()
                code = code - 16 * (code >= 8)
                kv.append(code * steps[pages, h].reshape(-1, c["dim"] // 32)[:n].double().repeat_interleave(32, 1))
            for j in range(h * group, (h + 1) * group):
                z = (s["q"][rows, j].double() @ kv[0].T * s["scale"]).masked_fill(hide, -math.inf)
                out[rows, j] = torch.softmax(z, 1) @ kv[1]
    return {"out": out}
