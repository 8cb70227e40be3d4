"""GPU parity of the 4-bit key/value cache's calls with the plain 64-bit implementation in kv4_ref.py: tables
and packed bytes exactly, attention within the bounds derived there."""
import math

import numpy as np
import pytest
import torch

import int4_group_wise_b200 as q4
import kv4_ref as ref

pytestmark = pytest.mark.gpu
I32 = torch.int32


# ---------------------------------------------------------------------------------------- tables
def _tables_case(B, held, new, page, seed, free=None, most=None, pad=0):
    rng = np.random.default_rng(seed)
    lengths = rng.integers(0, held + 1, B)
    fresh = rng.integers(0, new + 1, B)
    need = -(-(lengths + fresh) // page)
    most = int(max(1, need.max())) if most is None else most
    n_pages = int(need.sum()) + 7
    names = torch.from_numpy(rng.permutation(n_pages).astype(np.int32))
    table = torch.full((B, most), -5, dtype=I32)
    at = 0
    for b in range(B):
        have = min(most, -(-int(lengths[b]) // page))
        table[b, :have] = names[at:at + have]
        at += have
    fl = names[at:] if free is None else names[at:at + free]
    return (torch.from_numpy(lengths.astype(np.int32)), torch.from_numpy(fresh.astype(np.int32)), table, fl,
            int(fresh.sum()) + pad)


def _check_tables(lengths, fresh, table, free, page, num_slots):
    lens, cu, slots, taken, want = ref.tables(lengths, fresh, table, free.tolist(), page, num_slots)
    t = table.cuda()
    a, b, c, d = q4.kv4_tables(lengths.cuda(), fresh.cuda(), t, free.cuda(), page, num_slots)
    assert a.tolist() == lens and b.tolist() == cu and d.item() == taken
    assert c.tolist() == slots
    assert torch.equal(t.cpu(), want)


@pytest.mark.parametrize("B,held,new,page", [(1, 0, 1, 16), (1, 100, 1, 128), (3, 50, 40, 32), (33, 500, 1, 64),
                                             (511, 300, 20, 16), (512, 0, 65, 64), (513, 99, 3, 32),
                                             (1500, 40, 300, 16)])
def test_tables(B, held, new, page):
    _check_tables(*_tables_case(B, held, new, page, seed=B + held)[:4], page,
                  _tables_case(B, held, new, page, seed=B + held)[4])


def test_tables_padding_and_short_room():
    """Entries past the last token are -1; tokens past num_slots get no entry, the tables are the same."""
    for pad in (0, 1, 37, -5):
        l, f, t, fr, n = _tables_case(20, 100, 30, 16, seed=5, pad=pad)
        _check_tables(l, f, t, fr, 16, n)
    l, f, t, fr, _ = _tables_case(20, 100, 30, 16, seed=5)
    _check_tables(l, f, t, fr, 16, 0)


def test_tables_short_free_list_and_short_rows():
    for free in (0, 1, 9):
        l, f, t, fr, n = _tables_case(12, 60, 90, 16, seed=8, free=free, pad=3)
        _check_tables(l, f, t, fr, 16, n)
    l, f, t, fr, n = _tables_case(12, 60, 90, 16, seed=9, most=3)
    _check_tables(l, f, t, fr, 16, n)


def test_tables_no_new_tokens_and_negative_entries():
    l = torch.tensor([0, 17, -3, 40], dtype=I32)
    f = torch.tensor([0, 0, 4, -9], dtype=I32)
    t = torch.full((4, 4), -1, dtype=I32)
    t[1, :2] = torch.tensor([3, 4], dtype=I32)
    t[3, :3] = torch.tensor([7, 8, 9], dtype=I32)
    _check_tables(l, f, t, torch.arange(20, 30, dtype=I32), 16, 9)


def test_tables_largest_batch_and_strided_rows():
    l, f, t, fr, n = _tables_case(16384, 20, 5, 16, seed=3)
    lens, cu, slots, taken, want = ref.tables(l, f, t, fr.tolist(), 16, n)
    wide = torch.full((16384, t.shape[1] + 3), 77, dtype=I32, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    a, b, c, d = q4.kv4_tables(l.cuda(), f.cuda(), wide[:, :t.shape[1]], fr.cuda(), 16, n)
    assert a.tolist() == lens and b.tolist() == cu and c.tolist() == slots and d.item() == taken
    assert torch.equal(wide[:, :t.shape[1]].cpu(), want) and bool((wide[:, t.shape[1]:] == 77).all())


def test_tables_unaligned_slots_and_huge_lengths():
    """slots that start on an odd word take scalar stores; lengths whose sum passes 2^31 are cut, nothing is
    written out of range."""
    l, f, t, fr, n = _tables_case(9, 30, 30, 16, seed=11)
    room = torch.full((n + 9,), 123, dtype=I32, device="cuda")
    _, _, slots, _, _ = ref.tables(l, f, t, fr.tolist(), 16, n)
    q4.kv4_tables(l.cuda(), f.cuda(), t.cuda(), fr.cuda(), 16, n, slots=room[1:n + 1])
    assert room[1:n + 1].tolist() == slots and room[0].item() == 123 and bool((room[n + 1:] == 123).all())
    big = torch.tensor([2 ** 31 - 1, 2 ** 31 - 1, 5], dtype=I32)
    t = torch.full((3, 2), -1, dtype=I32).cuda()
    lens, cu, s, taken = q4.kv4_tables(big.cuda(), big.cuda(), t, torch.arange(4, dtype=I32).cuda(), 16, 40)
    assert lens.tolist() == [2 ** 31 - 1, 2 ** 31 - 1, 10] and cu.tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert bool((s == -1).all()) and taken.item() == 0


# ---------------------------------------------------------------------------------------- append, gather
def _append_values(n, h, d, seed, kind):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, d, generator=g) * torch.exp(0.5 * torch.randn(h, d, generator=g))
    if kind == "grid":      # multiples of half a 5-bit step: every quotient is a tie or exact
        x = torch.randint(-16, 15, (n, h, d), generator=g).float() * 0.5 * 1.1875
        x[..., ::32] = 7 * 1.1875
    elif kind == "edges":
        x[0] = 0
        x.view(-1)[5] = 1e-38
        x[n // 2] *= 1e-33
        x[n // 3] *= 1e36
        x[-1] = 3e38
        x.view(-1)[-d - 3] = math.inf
        x.view(-1)[-2 * d - 40 % d] = math.nan
        x.view(-1)[d + 1] = -math.inf
    return x


@pytest.mark.parametrize("n,h,d,page,dtype,kind", [
    (1, 1, 64, 16, torch.bfloat16, "normal"), (2, 1, 64, 16, torch.float32, "normal"), (7, 3, 128, 32, torch.bfloat16, "normal"),
    (130, 8, 128, 64, torch.bfloat16, "grid"), (61, 2, 64, 128, torch.float32, "grid"),
    (33, 5, 64, 16, torch.float32, "normal"), (40, 2, 128, 16, torch.float32, "edges"),
    (40, 3, 64, 16, torch.bfloat16, "edges"), (2049, 8, 128, 64, torch.bfloat16, "normal")])
def test_append_and_gather(n, h, d, page, dtype, kind):
    k, v = _append_values(n, h, d, n + d, kind).to(dtype), _append_values(n, h, d, n + d + 1, kind).to(dtype)
    pages = -(-n // page) + 3
    perm = torch.randperm(pages * page, generator=torch.Generator().manual_seed(n))[:n].to(I32)
    perm[n // 2] = -1
    if n > 8:
        perm[3], perm[4] = pages * page, 2 ** 31 - 1        # past the cache: skipped
    cache = q4.kv4_cache(pages, page, h, d)
    for t in cache:
        t.fill_(3)
    rows = torch.cat([torch.zeros(n, 2 * h, d).to(dtype), k, v], 1).cuda()
    q4.kv4_append(cache, rows[:, 2 * h:3 * h], rows[:, 3 * h:], perm.cuda())
    ok = (perm >= 0) & (perm < pages * page)
    at = perm[ok].long()
    for x, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        q, s = ref.quantize(x[ok])
        want_c = torch.full((pages, h, page, d // 2), 3, dtype=torch.uint8)
        want_s = torch.full((pages, h, page, d // 32), 3, dtype=torch.bfloat16)
        want_c[at // page, :, at % page] = ref.pack(q)
        want_s[at // page, :, at % page] = s.bfloat16()
        assert torch.equal(s.bfloat16().float(), s)         # a step has at most 5 significant bits
        assert torch.equal(scales.cpu().view(torch.int16), want_s.view(torch.int16))
        assert torch.equal(codes.cpu(), want_c)
    gk, gv = q4.kv4_gather(cache, perm.cuda())
    for x, got in ((k, gk), (v, gv)):
        q, s = ref.quantize(x)
        want = q.double() * s.double().repeat_interleave(32, -1)
        want[~ok] = 0
        assert torch.equal(want.bfloat16().double(), want)  # code * step is exactly a bf16
        assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("n,h,d,page,dtype,kind", [
    (4001, 8, 128, 64, torch.float32, "normal"), (4001, 8, 128, 16, torch.float32, "edges"),
    (9001, 7, 64, 32, torch.bfloat16, "edges"), (5003, 6, 128, 128, torch.bfloat16, "grid")])
def test_append_and_gather_large(n, h, d, page, dtype, kind):
    """Batches large enough for several words per thread."""
    test_append_and_gather(n, h, d, page, dtype, kind)


@pytest.mark.parametrize("copies", [1, 9])
def test_append_every_bf16_against_every_step(copies):
    """All bf16 significands at every exponent that gives a code other than 0, and some below, against every 5-bit
    step; some groups hold a NaN, an infinity or values near the type's ends.  Small and large batches."""
    groups = []
    for s in range(16, 32):
        v = (torch.arange(256).float() * 2.0 ** -4)[None] * 2.0 ** torch.arange(-14, 8)[:, None].float()
        v = v[v <= 7 * s / 16]
        v = torch.cat([v, -v, torch.zeros(-2 * v.numel() % 31)]).view(-1, 31)
        groups.append(torch.cat([torch.full((v.shape[0], 1), 7 * s / 16), v], 1))
    x = torch.cat(groups)
    x = torch.cat([x, x * 2.0 ** 90, x * 2.0 ** -90])
    for i, bad in enumerate((math.nan, math.inf, -math.inf, 3e38, -1e-38)):
        x[11 + 40 * i:3000:200, 7 * i] = bad
    x[4000, :] = math.nan
    x = x[: x.shape[0] // 4 * 4].view(-1, 1, 128).bfloat16()
    q, s = ref.quantize(x)
    n = x.shape[0]
    cache = q4.kv4_cache(-(-copies * n // 16), 16, 1, 128)
    q4.kv4_append(cache, x.repeat(copies, 1, 1).cuda(), x.flip(0).repeat(copies, 1, 1).cuda(),
                  torch.arange(copies * n, dtype=I32).cuda())
    flat = lambda t: t.cpu().transpose(1, 2).flatten(0, 1)[:copies * n].view(copies, n, 1, -1)  # noqa: E731
    for codes, scales, wq, ws in ((cache.k_codes, cache.k_scales, q, s), (cache.v_codes, cache.v_scales, q.flip(0), s.flip(0))):
        assert bool((flat(codes) == ref.pack(wq)).all()) and bool((flat(scales).float() == ws).all())


def test_append_quantizer_error():
    """Against the values themselves: a code's value is off by at most half a step, and the step is at most
    17/16 of m / 7 (5 significant bits rounded up: at most one part in 16)."""
    x = _append_values(64, 4, 128, 2, "normal")
    cache = q4.kv4_cache(1, 64, 4, 128)
    s = torch.arange(64, dtype=I32).cuda()
    q4.kv4_append(cache, x.cuda(), x.cuda(), s)
    k, _ = q4.kv4_gather(cache, s)
    m = x.double().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 7
    err = (k.cpu().double() - x.double()).unflatten(-1, (-1, 32)).abs()
    assert bool((err <= 0.5 * m * 17 / 16 * (1 + 2.0 ** -22)).all())


def test_append_division_is_the_binary32_quotient():
    """Every 5-bit step significand against dense float32 values around the code boundaries."""
    g = torch.Generator().manual_seed(1)
    groups = []
    for s in range(16, 32):
        step = np.float32(s / 16)
        v = torch.arange(-15, 14, 2).float().repeat_interleave(64) * 0.5 * float(step)
        v = (v.numpy().view(np.int32) + torch.randint(-3, 4, (v.numel(),), generator=g).numpy().astype(np.int32)).view(np.float32)
        v = torch.from_numpy(v)[: v.size // 31 * 31].view(-1, 31)
        groups.append(torch.cat([torch.full((v.shape[0], 1), float(np.float32(7) * step)), v], 1))
    x = torch.cat(groups)
    n = x.shape[0] // 4 * 4
    x = x[:n].reshape(-1, 1, 128).contiguous()
    q, s = ref.quantize(x)
    cache = q4.kv4_cache(-(-x.shape[0] // 16), 16, 1, 128)
    slots = torch.arange(x.shape[0], dtype=I32)
    q4.kv4_append(cache, x.cuda(), x.cuda(), slots.cuda())
    at = slots.long()
    assert torch.equal(cache.k_codes.cpu()[at // 16, :, at % 16], ref.pack(q))
    assert torch.equal(cache.v_scales.cpu()[at // 16, :, at % 16].float(), s)


# ---------------------------------------------------------------------------------------- attention
def _batch(lens, nqs, page, heads, dim, q_heads, seed, spare=2, extra_rows=0):
    g = torch.Generator().manual_seed(seed)
    count = [max(0, -(-n // page)) for n in lens]
    total = sum(count) + spare
    cache = ref.make_cache(total, heads, page, dim, seed)
    names = torch.randperm(total, generator=g).to(I32)
    table = torch.full((len(lens), max(1, max(count))), -1, dtype=I32)
    at = 0
    for b, c in enumerate(count):
        table[b, :c] = names[at:at + c]
        at += c
    cu = torch.tensor([0] + list(np.cumsum(nqs)), dtype=I32)
    q = torch.randn(int(cu[-1]) + extra_rows, q_heads, dim, generator=g).bfloat16()
    return q, cache, table, torch.tensor(lens, dtype=I32), cu


def _run(q, cache, table, lens, cu, scale=None, causal=True, window=0, **kw):
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    q4.kv4_attention(q.cuda(), q4.KV4Cache(*(t.cuda() for t in cache)), table.cuda(), lens.cuda(), cu.cuda(),
                     scale=scale, causal=causal, window=window, out=out, lse=lse, **kw)
    q4.sync_check()
    return out.cpu(), lse.cpu()


def _check(q, cache, table, lens, cu, scale=None, causal=True, window=0):
    out, lse = _run(q, cache, table, lens, cu, scale, causal, window)
    sc = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    want, wl, tol, ltol = ref.attention(q, cache, table, lens, cu, float(np.float32(sc)), causal, window)
    none = torch.isnan(wl)
    assert bool((out[none] == 7.0).all()) and bool((lse[none] == 7.0).all())     # rows of no request
    o, l, want, wl, tol, ltol = out[~none].double(), lse[~none].double(), want[~none], wl[~none], tol[~none], ltol[~none]
    empty = torch.isinf(wl)
    assert bool((o[empty] == 0).all()) and bool((l[empty] == -math.inf).all())
    err = (o - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), int((err > tol).sum()))
    lerr = (l - wl).abs()[~empty]
    assert bool((lerr <= ltol[~empty]).all()), float((lerr / ltol[~empty]).max())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attention_single_tokens(dim, page):
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1000]
    _check(*_batch(lens, [1] * len(lens), page, 2, dim, 8, seed=page + dim))


@pytest.mark.parametrize("dim,q_heads,heads", [(64, 1, 1), (128, 1, 1), (128, 8, 8), (64, 32, 8), (128, 5, 1),
                                               (64, 14, 2), (128, 16, 1), (64, 17, 1), (128, 64, 1), (64, 128, 2)])
def test_attention_head_groups(dim, q_heads, heads):
    _check(*_batch([77, 300, 1], [1, 1, 1], 16, heads, dim, q_heads, seed=q_heads))
    _check(*_batch([77, 300, 9], [4, 1, 3], 32, heads, dim, q_heads, seed=q_heads + 1))


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_queries_of_every_length(dim):
    """Requests without queries, without cached tokens, with more queries than tokens (the first see
    nothing), short drafts and prompts in one batch."""
    lens = [50, 0, 0, 3, 40, 130, 129, 260, 17, 1]
    nqs = [0, 0, 2, 7, 40, 3, 129, 33, 17, 1]
    _check(*_batch(lens, nqs, 16, 2, dim, 8, seed=dim))
    _check(*_batch(lens, nqs, 64, 1, dim, 5, seed=dim + 1), causal=False)


@pytest.mark.parametrize("window", [1, 2, 17, 128, 1000])
def test_attention_window(window):
    _check(*_batch([1, 130, 400, 1500], [1, 1, 1, 1], 16, 2, 64, 8, seed=window), window=window)
    _check(*_batch([5, 130, 400, 1500], [5, 9, 70, 21], 32, 1, 128, 8, seed=window + 1), window=window)
    _check(*_batch([300, 700], [300, 260], 64, 1, 128, 4, seed=window + 2), window=window)


def test_attention_window_past_short_requests():
    """More queries than tokens under a window: negative positions see nothing."""
    _check(*_batch([3, 2], [9, 300], 16, 1, 64, 2, seed=4), window=2)


@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
def test_attention_long_request_is_split(dim, page):
    """One request over every CTA, and the same beside short ones."""
    _check(*_batch([20011], [1], page, 1, dim, 4, seed=dim))
    _check(*_batch([3, 9001, 1, 40], [1, 2, 1, 1], page, 2, dim, 8, seed=dim + 1))


def test_attention_many_ragged_requests():
    rng = np.random.default_rng(0)
    lens = rng.integers(1, 90, 700).tolist()
    _check(*_batch(lens, [1] * 700, 16, 1, 64, 4, seed=1))
    nqs = [int(rng.integers(0, min(6, n) + 1)) for n in lens]
    _check(*_batch(lens, nqs, 32, 1, 64, 2, seed=2))


@pytest.mark.parametrize("dim,q_heads,heads,page", [(128, 8, 2, 64), (64, 8, 2, 16), (128, 7, 1, 128), (64, 3, 3, 32)])
def test_attention_prompts(dim, q_heads, heads, page):
    for lens, nqs in (([513], [513]), ([700, 300], [100, 300]), ([255, 256, 257], [255, 256, 257])):
        _check(*_batch(lens, nqs, page, heads, dim, q_heads, seed=sum(lens) + dim))
    _check(*_batch([400, 150], [200, 150], page, heads, dim, q_heads, seed=dim), causal=False)


def test_attention_prompt_on_long_context():
    """Few query tiles on a long context: the keys are split and joined."""
    _check(*_batch([5000], [40], 64, 1, 128, 4, seed=1))
    _check(*_batch([3001], [129], 16, 1, 64, 2, seed=2), window=700)


@pytest.mark.parametrize("dim,new,q_heads,heads", [(64, 5, 8, 2), (128, 5, 8, 2), (64, 3, 7, 1), (128, 20, 1, 1),
                                                   (128, 1, 17, 1), (64, 1, 24, 1)])
def test_attention_drafts(dim, new, q_heads, heads):
    """17 to 24 rows per request and kv head, requests enough for tiles of 24 rows; one request with more, one
    with none."""
    rng = np.random.default_rng(dim + new)
    B = 70 // heads
    lens = rng.integers(new, 400, B).tolist()
    nqs = [new] * B
    nqs[3], nqs[5], nqs[7] = 0, 2 * new, max(0, new - 2)
    lens[0], lens[5] = 1500, 2 * new
    _check(*_batch(lens, nqs, 32, heads, dim, q_heads, seed=dim + q_heads))
    _check(*_batch(lens, nqs, 16, heads, dim, q_heads, seed=dim + q_heads + 1), window=100)


def test_attention_many_prompts():
    """More requests of many rows than a warp has lanes, and groups of 32 of them without any."""
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 300, 75).tolist()
    nqs = [int(rng.integers(1, n + 1)) for n in lens]
    _check(*_batch(lens, nqs, 16, 1, 64, 4, seed=3))
    lens = [40] * 70 + [200, 130] + [1] * 90
    nqs = [0] * 70 + [200, 90] + [1] * 90
    _check(*_batch(lens, nqs, 64, 2, 128, 64, seed=4))


def test_attention_window_of_any_size():
    """A window near 2^31 is no window, for requests with more queries than tokens too."""
    for nqs in ([5, 1], [200, 90]):
        a = _batch([3, 300], nqs, 16, 1, 64, 4, seed=2)
        want = _run(*a)
        for window in (2 ** 31 - 1, 2 ** 40):
            got = _run(*a, window=window)
            assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("lens,nqs,q_heads", [
    ([300, 40], [1, 1], 4), ([5000, 300], [1, 1], 4), ([300, 40], [2, 2], 4), ([300, 40], [4, 4], 4), ([5000], [4], 4),
    ([150] * 70, [5] * 70, 4), ([300], [300], 4), ([5000], [40], 4), ([600, 300], [130, 1], 4)])
def test_attention_nan_queries_stay_in_their_rows(lens, nqs, q_heads):
    """A NaN in one query head gives NaN there, in the output and in the log-sum-exp, and leaves every other row's
    bits alone; the output may take the queries' place."""
    for dim in (64, 128):
        q, cache, table, lens_t, cu = _batch(lens, nqs, 64, 1, dim, q_heads, seed=dim)
        out, lse = _run(q, cache, table, lens_t, cu)
        at = int(cu[-1]) // 2
        dirty = q.clone()
        dirty[at, 1, 5] = math.nan
        got, gl = _run(dirty, cache, table, lens_t, cu)
        assert bool(torch.isnan(got[at, 1]).all()) and math.isnan(float(gl[at, 1]))
        got[at, 1], gl[at, 1] = out[at, 1], lse[at, 1]
        assert torch.equal(got.view(torch.int16), out.view(torch.int16)) and torch.equal(gl, lse)
        place = q.cuda()
        q4.kv4_attention(place, q4.KV4Cache(*(t.cuda() for t in cache)), table.cuda(), lens_t.cuda(), cu.cuda(), out=place)
        q4.sync_check()
        assert torch.equal(place.cpu().view(torch.int16), out.view(torch.int16))


def test_attention_large_and_small_scores():
    """Scores that leave one key all the weight, equal scores, and a scale other than 1/sqrt(D)."""
    q, cache, table, lens, cu = _batch([300, 129, 700], [1, 20, 300], 64, 1, 128, 4, seed=6)
    _check(q * 30, cache, table, lens, cu)
    _check(q * 0, cache, table, lens, cu)
    _check(q, cache, table, lens, cu, scale=0.5)
    _check(q, cache, table, lens, cu, scale=1e-6)
    # maxima that keep growing along the keys: the running maximum is moved again and again
    kc, ks, vc, vs = (t.clone() for t in cache)
    for b in range(3):
        n = int(lens[b])
        for j in range(n):
            pg = int(table[b, j // 64])
            ks[pg, :, j % 64] = 0.0625 * 2.0 ** (j * 6 // n)
    _check(q, (kc, ks, vc, vs), table, lens, cu)


def test_attention_ignores_what_lies_past_the_lengths():
    """NaN and infinite steps in pages' ends, in spare pages and before the window change nothing; entries of
    the table outside the cache are left out; rows past the last request stay as they are."""
    for lens, nqs, window, page in (([70, 33, 200], [1, 1, 1], 0, 64), ([70, 33, 500], [1, 5, 40], 0, 32),
                                    ([500, 300], [1, 1], 50, 16), ([500, 300], [2, 150], 50, 16)):
        q, cache, table, tl, cu = _batch(lens, nqs, page, 2, 64, 4, seed=page, extra_rows=3)
        base, blse = _run(q, cache, table, tl, cu, window=window)
        dirty = [t.clone() for t in cache]
        used = torch.zeros(cache[0].shape[0], page, dtype=torch.bool)
        for b, n in enumerate(lens):
            first = max(0, n - nqs[b] - window + 1) if window else 0
            for j in range(first, n):
                used[int(table[b, j // page]), j % page] = True
        for i in range(2):
            dirty[2 * i].transpose(1, 2)[~used] = 0x9C
            dirty[2 * i + 1].transpose(1, 2)[~used] = math.nan if i else math.inf
        out, lse = _run(q, dirty, table, tl, cu, window=window)
        assert torch.equal(out.view(torch.int16), base.view(torch.int16)) and torch.equal(lse, blse)
        assert bool((out[-3:] == 7.0).all())
        if window:                                            # pages before the window given back
            t2 = table.clone()
            for b, n in enumerate(lens):
                t2[b, :max(0, n - nqs[b] - window + 1) // page] = -1
            out, lse = _run(q, dirty, t2, tl, cu, window=window)
            assert torch.equal(out.view(torch.int16), base.view(torch.int16)) and torch.equal(lse, blse)


def test_attention_bad_pages_are_left_out():
    for nqs in ([1, 1], [3, 100]):
        q, cache, table, lens, cu = _batch([300, 260], nqs, 32, 2, 64, 4, seed=3)
        table[0, 2] = -1
        table[0, 5] = cache[0].shape[0]
        table[1, 0] = 2 ** 31 - 1
        table[1, 8] = -2 ** 31
        _check(q, cache, table, lens, cu)
    q, cache, table, lens, cu = _batch([100], [1], 64, 1, 128, 4, seed=3)
    table.fill_(-1)
    _check(q, cache, table, lens, cu)                         # nothing left: zeros
    lens[0] = 2 ** 31 - 1                                     # cut to the table
    _check(q, cache, torch.zeros_like(table), lens, cu)


def test_attention_wrong_offsets_stay_in_bounds():
    """cu_q that is not ascending or leaves [0, N]: no fault, and requests with right offsets are right."""
    q, cache, table, lens, cu = _batch([64, 64, 64], [2, 2, 2], 64, 1, 64, 2, seed=3)
    want, _ = _run(q, cache, table, lens, cu)
    for bad in ([0, 2, 1, 99], [0, 2, -7, -1], [0, 2, 2 ** 31 - 1, 4]):
        out, _ = _run(q, cache, table, lens, torch.tensor(bad, dtype=I32))
        assert torch.equal(out[:1], want[:1])


def test_attention_strided_inputs():
    q, cache, table, lens, cu = _batch([90, 500], [1, 30], 32, 2, 128, 4, seed=8)
    want, wl = _run(q, cache, table, lens, cu)
    rows = torch.randn(q.shape[0], 9, 128).bfloat16().cuda()
    rows[:, 3:7] = q.cuda()
    wide = torch.full((2, table.shape[1] + 5), -9, dtype=I32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = table.cuda()
    out = q4.kv4_attention(rows[:, 3:7], q4.KV4Cache(*(t.cuda() for t in cache)), wide[:, 2:2 + table.shape[1]],
                           torch.cat([lens, lens]).cuda()[:2], cu.cuda())
    assert torch.equal(out.cpu(), want)


def test_attention_is_deterministic():
    for lens, nqs in (([5000, 3], [1, 1]), ([900, 40], [200, 3])):
        a = _batch(lens, nqs, 64, 2, 128, 8, seed=1)
        first = _run(*a)
        for _ in range(10):
            again = _run(*a)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_offsets_past_32_bits():
    """A cache of 5.4 GB: pages whose byte offset passes 2^32."""
    heads, page, dim = 8, 128, 128
    pages = (5 << 30) // (heads * page * dim // 2)
    kc, ks, vc, vs = ref.make_cache(4, heads, page, dim, 1)
    cache = q4.kv4_cache(pages, page, heads, dim)
    at = torch.tensor([0, pages // 2, pages - 2, pages - 1])
    for big, small in zip(cache, (kc, ks, vc, vs)):
        big[at.cuda()] = small.cuda()
    order = torch.tensor([[2, 0, 3, 1]])
    q = torch.randn(34, 8, dim, generator=torch.Generator().manual_seed(2)).bfloat16()
    lens, cu = torch.tensor([500, 400], dtype=I32), torch.tensor([0, 1, 34], dtype=I32)
    tab = at[order].to(I32).repeat(2, 1)
    out = q4.kv4_attention(q.cuda(), cache, tab.cuda(), lens.cuda(), cu.cuda()).cpu().double()
    want, _, tol, _ = ref.attention(q, (kc, ks, vc, vs), order.to(I32).repeat(2, 1), lens, cu, float(np.float32(dim ** -0.5)))
    assert bool(((out - want).abs() <= tol).all())
    x = torch.randn(3, heads, dim).bfloat16().cuda()
    s = torch.tensor([0, pages * page - 1, (pages - 2) * page + 5], dtype=I32).cuda()
    q4.kv4_append(cache, x, x, s)
    k, _ = q4.kv4_gather(cache, s)
    c, st = ref.quantize(x.cpu())
    assert torch.equal(k.cpu().double(), c.double() * st.double().repeat_interleave(32, -1))


# ---------------------------------------------------------------------------------------- together
def _steps(news, page, heads, dim, q_heads, seed):
    """Decode and prompt steps as a server makes them: tables, append, attention; compared after each with the
    64-bit attention over the tokens' own quantized values."""
    B, g = len(news[0]), torch.Generator().manual_seed(seed)
    total = [sum(n[b] for n in news) for b in range(B)]
    pages = sum(-(-t // page) for t in total) + 3
    cache = q4.kv4_cache(pages, page, heads, dim)
    table = torch.full((B, max(-(-t // page) for t in total)), -1, dtype=I32, device="cuda")
    free = torch.randperm(pages, generator=g).to(I32).cuda()
    lens, used = torch.zeros(B, dtype=I32, device="cuda"), 0
    for new in news:
        n = sum(new)
        k, v = (torch.randn(n, heads, dim, generator=g).bfloat16().cuda() for _ in range(2))
        q = torch.randn(n, q_heads, dim, generator=g).bfloat16()
        lens, cu, slots, taken = q4.kv4_tables(lens, torch.tensor(new, dtype=I32).cuda(), table, free[used:], page, n)
        q4.kv4_append(cache, k, v, slots)
        out = q4.kv4_attention(q.cuda(), cache, table, lens, cu)
        used += int(taken)
        want, _, tol, _ = ref.attention(q, [t.cpu() for t in cache], table.cpu(), lens.cpu(), cu.cpu(),
                                        float(np.float32(dim ** -0.5)))
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
    q4.sync_check()


def test_steps_of_a_server():
    _steps([[30, 5, 100], [1, 1, 1], [1, 1, 0], [2, 40, 1], [1, 1, 1]], 16, 2, 64, 8, seed=1)
    _steps([[70, 300], [1, 1], [9, 1]], 64, 1, 128, 8, seed=2)


def test_steps_in_captured_graphs():
    """A padded step captured once and replayed with new lengths and values, two graphs alive, each with its
    own outputs: the same as eager calls."""
    heads, dim, q_heads, page, room, B = 2, 128, 8, 32, 12, 4
    g = torch.Generator().manual_seed(3)

    def make():
        d = dict(cache=q4.kv4_cache(40, page, heads, dim), table=torch.full((B, 9), -1, dtype=I32, device="cuda"),
                 lens=torch.zeros(B, dtype=I32, device="cuda"), new=torch.zeros(B, dtype=I32, device="cuda"),
                 free=torch.arange(40, dtype=I32, device="cuda"),
                 k=torch.zeros(room, heads, dim, device="cuda"), v=torch.zeros(room, heads, dim, device="cuda"),
                 q=torch.zeros(room, q_heads, dim, dtype=torch.bfloat16, device="cuda"),
                 out=torch.zeros(room, q_heads, dim, dtype=torch.bfloat16, device="cuda"))
        return d

    def step(d):
        lens, cu, slots, taken = q4.kv4_tables(d["lens"], d["new"], d["table"], d["free"], page, room)
        q4.kv4_append(d["cache"], d["k"], d["v"], slots)
        q4.kv4_attention(d["q"], d["cache"], d["table"], lens, cu, out=d["out"])
        return lens

    eager, caught, graphs = [make(), make()], [make(), make()], []
    side = torch.cuda.Stream()
    for d in caught:
        with torch.cuda.stream(side):
            step(d)
        side.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            d["after"] = step(d)
        graphs.append(gr)
    for i, new in enumerate(([3, 1, 0, 2], [1, 1, 1, 1], [5, 0, 0, 7], [1, 0, 1, 1])):
        for a, e, gr in zip(caught, eager, graphs):
            k, v = torch.randn(room, heads, dim, generator=g), torch.randn(room, heads, dim, generator=g)
            q = torch.randn(room, q_heads, dim, generator=g).bfloat16()
            for d in (a, e):
                d["k"].copy_(k)
                d["v"].copy_(v)
                d["q"].copy_(q)
                d["new"].copy_(torch.tensor(new, dtype=I32))
            gr.replay()
            e["after"] = step(e)
        torch.cuda.synchronize()
        for a, e in zip(caught, eager):
            n = sum(new)
            assert torch.equal(a["out"][:n], e["out"][:n]) and torch.equal(a["table"], e["table"])
            for d in (a, e):
                used = int((-(-d["after"] // page)).sum()) - int((-(-d["lens"] // page)).sum())
                d["free"].copy_(torch.roll(d["free"], -used))
                d["lens"].copy_(d["after"])
    q4.sync_check()


def test_calls_on_a_side_stream():
    """stream=: inputs made on that stream, outputs and workspace of that stream's pool."""
    q, cache, table, lens, cu = _batch([600, 90], [1, 30], 32, 2, 64, 8, seed=4)
    want, _ = _run(q, cache, table, lens, cu)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dq, dc = q.cuda(), q4.KV4Cache(*(t.cuda() for t in cache))
        dt, dl, dcu = table.cuda(), lens.cuda(), cu.cuda()
    out = [q4.kv4_attention(dq, dc, dt, dl, dcu, stream=side) for _ in range(3)]
    side.synchronize()
    q4.sync_check(side)
    for o in out:
        assert torch.equal(o.cpu(), want)


# ---------------------------------------------------------------------------------------- refusals
def test_refusals_of_the_binding():
    q, cache, table, lens, cu = _batch([20, 20], [1, 1], 16, 2, 64, 4, seed=1)
    dc = q4.KV4Cache(*(t.cuda() for t in cache))
    q, table, lens, cu = q.cuda(), table.cuda(), lens.cuda(), cu.cuda()
    call = lambda **kw: q4.kv4_attention(**{**dict(q=q, cache=dc, block_table=table, seq_lens=lens, cu_q=cu), **kw})  # noqa: E731
    with pytest.raises(TypeError):
        call(q=q.float())
    with pytest.raises(TypeError):
        call(q=q.cpu())
    with pytest.raises(ValueError):
        call(q=q[:, :3])
    with pytest.raises(ValueError):
        call(q=q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        call(cu_q=cu[:2])
    with pytest.raises(TypeError):
        call(seq_lens=lens.long())
    with pytest.raises(ValueError):
        call(block_table=table.t())
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(window=-1),
               dict(window=4, causal=False)):
        with pytest.raises(q4.Qat4Error) as e:
            call(**kw)
        assert e.value.status == 2
    wide = torch.zeros((2, 900), dtype=I32, device="cuda")
    with pytest.raises(q4.Qat4Error) as e:
        call(block_table=wide, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    with pytest.raises(q4.Qat4Error) as e:               # rows of 20 bytes past a 16-byte boundary
        call(q=torch.zeros(2 * 260, dtype=torch.bfloat16, device="cuda").as_strided((2, 4, 64), (260, 64, 1)))
    assert e.value.status == 3
    x = torch.zeros(3, 2, 64, device="cuda")
    s = torch.zeros(3, dtype=I32, device="cuda")
    with pytest.raises(TypeError):
        q4.kv4_append(dc, x.half(), x.half(), s)
    with pytest.raises(TypeError):
        q4.kv4_append(dc, x, x.bfloat16(), s)
    with pytest.raises(ValueError):
        q4.kv4_append(dc, x, x[:2], s)
    with pytest.raises(ValueError):
        q4.kv4_append(dc, x, x, s[:2])
    with pytest.raises(ValueError):
        q4.kv4_append(dc._replace(k_scales=dc.k_scales[:1]), x, x, s)
    with pytest.raises(q4.Qat4Error):
        q4.kv4_tables(lens, lens, table, s, 16, 4, seq_lens=lens)
    with pytest.raises(ValueError):
        q4.kv4_tables(lens, lens.clone(), table, s, 48, 4)
    with pytest.raises(ValueError):
        q4.kv4_tables(lens, lens.clone(), table[:1], s, 16, 4)
    assert q4.kv4_attention(q[:0], dc, table, lens, cu * 0).shape == (0, 4, 64)
    q4.kv4_append(dc, x[:0], x[:0], s[:0])
    assert q4.kv4_gather(dc, s[:0])[0].shape == (0, 2, 64)
    q4.sync_check()
