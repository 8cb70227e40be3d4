"""Attention over millions of cached tokens.  A block table may name a page again and again, so a few pages stand for a long
context: a token's weight is its exponential times the number of times that its page is named."""
import math

import pytest
import torch

import int4_group_wise_b200 as q4
import kv4_ref as ref

pytestmark = pytest.mark.gpu
I32 = torch.int32
PAGE, PAGES = 128, 8


def _long(batch, nq, tokens, q_heads, dim, seed, growing=False):
    """A batch of requests of `tokens` tokens over PAGES pages.  Values are positive, so that what a sum loses shows in its
    mean; `growing`: the pages come in the order of ever larger scores, which move the running maxima."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = q4.kv4_cache(PAGES, PAGE, 1, dim)
    rand = lambda lo, hi, shape: torch.randint(lo, hi, shape, generator=g, device="cuda")        # noqa: E731
    kcodes, vcodes = rand(-8, 8, (PAGES, 1, PAGE, dim)), rand(1, 8, (PAGES, 1, PAGE, dim))
    cache.k_codes.copy_(ref.pack(kcodes.to(torch.int8)))
    cache.v_codes.copy_(ref.pack(vcodes.to(torch.int8)))
    cache.k_scales.fill_(0.25)
    cache.v_scales.copy_((1 + rand(0, 16, cache.v_scales.shape) / 16).bfloat16())
    blocks = tokens // PAGE
    if growing:
        # a channel that every query has at 1 raises the scores page by page
        kcodes[..., 0] = torch.arange(-4, 4, device="cuda").view(PAGES, 1, 1)
        cache.k_codes.copy_(ref.pack(kcodes.to(torch.int8)))
        order = torch.arange(blocks, device="cuda") * PAGES // blocks
        order = torch.stack([order.roll(b * 977 % 64) for b in range(batch)])
        order[:, :64] = 0
    else:
        order = rand(0, PAGES, (batch, blocks))
    q = torch.randn((batch * nq, q_heads, dim), generator=g, device="cuda")
    if growing:
        q[..., 0] = 24.0 * math.sqrt(dim)
    count = torch.stack([(order == i).sum(1) for i in range(PAGES)], 1).double()
    return q.bfloat16(), cache, order.to(I32).contiguous(), count


@pytest.mark.parametrize("growing", [False, True])
@pytest.mark.parametrize("batch,nq,tokens,q_heads,dim", [
    (500, 1, 1 << 22, 4, 64), (500, 1, 1 << 22, 4, 128), (500, 1, 1 << 22, 8, 128), (500, 2, 1 << 22, 8, 64),
    (250, 5, 1 << 22, 4, 64), (160, 64, 1 << 20, 4, 64), (40, 64, 1 << 21, 4, 128), (1, 2048, 1 << 20, 8, 64)])
def test_sums_over_millions_of_tokens(batch, nq, tokens, q_heads, dim, growing):
    """Every element within the bound of kv4_ref.attention (of the values' sum, which is the output here), with the sums' part
    (n 2^-22 there) held to 2^-11; and their mean error within 2^-11 too, which the roundings' signs average out.  A sum
    cut to its own bits is low by 2^-12 at most (kKaFold, kKpFold).  A rounding to bf16 is 2^-8 at most, over sqrt(3) in the
    mean square: that of the output over the root of the number of elements, that of a weight by its share p of the
    row, so the root of sum p^2 over the rows' number; four times both."""
    q, cache, table, count = _long(batch, nq, tokens, q_heads, dim, seed=nq + dim, growing=growing)
    lens = torch.full((batch,), tokens, dtype=I32, device="cuda")
    cu = (torch.arange(batch + 1, device="cuda") * nq).to(I32)
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = q4.kv4_attention(q, cache, table, lens, cu, causal=False, lse=lse)
    q4.sync_check()
    k = ref.values(cache.k_codes.cpu(), cache.k_scales.cpu()).view(PAGES * PAGE, dim).cuda()
    v = ref.values(cache.v_codes.cpu(), cache.v_scales.cpu()).view(PAGES * PAGE, dim).cuda()
    scale = float(torch.tensor(dim ** -0.5, dtype=torch.float32))
    far, total, shares, number = 0.0, 0.0, 0.0, 0
    for b in range(0, batch, 50):
        rows = slice(b * nq, min(b + 50, batch) * nq)
        weight = count[b:b + 50].repeat_interleave(PAGE, 1).repeat_interleave(nq, 0)[:, None]
        x = q[rows].double()
        s = x @ k.T * scale + torch.log(weight)
        p = s.softmax(-1)
        want = p @ v
        mag = (x.abs() @ k.abs().T).amax(-1, keepdim=True)
        r = 4 * scale * (dim + 4) * 2.0 ** -23 * mag + 2.0 ** -20 + 2.0 ** -11
        err = out[rows].double() - want
        far = max(far, float((err.abs() / ((2.0 ** -8 + 1.01 * 2.0 ** -8 + 2 * r) * want)).max()))
        total += float((err / want).sum())
        number += err.numel()
        shares += float((p * p).sum())
        lerr = (lse[rows].double() - torch.logsumexp(s, -1)).abs()
        # a lane's sum has n / 8 terms at most, one rounding each
        assert bool((lerr <= r[..., 0] + tokens / 8 * 2.0 ** -24).all())
    assert far <= 1.0, far
    noise = 4 * (2.0 ** -8 / math.sqrt(3)) * (math.sqrt(1 / number) + math.sqrt(shares) / (number / dim))
    assert abs(total / number) <= 2.0 ** -11 + noise, (total / number, noise)


@pytest.mark.parametrize("batch,nq,tokens,dim", [(500, 1, 1 << 20, 64), (130, 5, 1 << 22, 128), (40, 64, 1 << 18, 64), (2, 300, 1 << 18, 128)])
def test_joined_sums_of_rows_apart(batch, nq, tokens, dim):
    """Where sums are joined in the workspace, a request whose table names no page gives zeros, a NaN in a query stays in its
    row, the other rows keep their bits, and the output may take the queries' place."""
    q, cache, table, _ = _long(batch, nq, tokens, 4, dim, seed=dim)
    lens = torch.full((batch,), tokens, dtype=I32, device="cuda")
    cu = (torch.arange(batch + 1, device="cuda") * nq).to(I32)
    lse, lse2 = torch.zeros(q.shape[:2], device="cuda"), torch.zeros(q.shape[:2], device="cuda")
    want = q4.kv4_attention(q, cache, table, lens, cu, lse=lse)
    dirty, none = q.clone(), table.clone()
    none[0] = -1
    dirty[nq + nq // 2, 2, 7] = math.nan
    got = q4.kv4_attention(dirty, cache, none, lens, cu, lse=lse2)
    assert not bool(got[:nq].any()) and bool((lse2[:nq] == -math.inf).all())
    assert bool(torch.isnan(got[nq + nq // 2, 2]).all()) and math.isnan(float(lse2[nq + nq // 2, 2]))
    got[:nq], lse2[:nq] = want[:nq], lse[:nq]
    got[nq + nq // 2, 2], lse2[nq + nq // 2, 2] = want[nq + nq // 2, 2], lse[nq + nq // 2, 2]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(lse2, lse)
    place = q.clone()
    q4.kv4_attention(place, cache, table, lens, cu, out=place)
    q4.sync_check()
    assert torch.equal(place.view(torch.int16), want.view(torch.int16))
