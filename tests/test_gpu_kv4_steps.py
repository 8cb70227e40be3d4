"""Caches with step sizes that kv4_append does not write: any bf16 from 0 to 2^100.  A value is step * code rounded
to bf16 once (include/qat4.h), for every significand of 8 bits and every code, in the gather call and in each
attention kernel."""
import math

import numpy as np
import pytest
import torch

import int4_group_wise_b200 as q4
import kv4_ref as ref
from test_gpu_kv4 import _batch, _check, _run

pytestmark = pytest.mark.gpu
I32 = torch.int32

# the requests and heads that reach each attention kernel: clusters and the grid-wide split with tiles of 4, 8, 16
# and 24 rows, prompts in one part and in several
KERNELS = [([300, 40], [1, 1], 4), ([300, 40], [2, 2], 4), ([300, 40], [4, 4], 4), ([5000, 300], [1, 1], 4),
           ([5000, 300], [2, 2], 4), ([5000, 300], [4, 4], 4), ([150] * 70, [5] * 70, 4), ([300], [300], 4),
           ([5000], [40], 4), ([600, 300], [130, 1], 4)]


def _values(codes, scales):
    """float64 of step * code rounded to bf16 (the product of 8 and 4 bits is exact in float32)."""
    return (ref.unpack(codes).float() * scales.float().repeat_interleave(32, -1)).bfloat16().double()


def _steps(shape, exponents, seed, most=128):
    """bf16 steps with every significand (`most` = 128: 8 bits) at the given exponents; exponent -127 is the subnormals."""
    g = torch.Generator().manual_seed(seed)
    n = math.prod(shape)
    e = torch.tensor(exponents)[torch.randint(len(exponents), (n,), generator=g)] + 127
    s = torch.arange(n) % 128
    s = s - s % (128 // most)
    return ((e << 7) | s).to(torch.int16).view(torch.bfloat16).view(shape)


@pytest.mark.parametrize("exponents", [[0], [-3, 5], [-100, 100], [-126, -127], [-127, 99]])
def test_gather_every_step_and_code(exponents):
    """16 codes by 128 significands, at ordinary exponents, at the ends of what append writes, among the subnormals
    and near the largest step that is allowed."""
    for dim in (64, 128):
        codes = torch.arange(2 * 16 * dim).view(2, 1, 16, dim) + torch.arange(16)[:, None]     # every code in every group
        codes = ((codes & 15) - 8).to(torch.int8)
        pages = 64
        packed = ref.pack(codes).repeat(pages // 2, 1, 1, 1)
        ks, vs = (_steps((pages, 1, 16, dim // 32), exponents, s) for s in (0, 1))
        cache = q4.KV4Cache(*(t.cuda() for t in (packed, ks, packed.flip(3).contiguous(), vs)))
        slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(2)).to(I32)
        k, v = q4.kv4_gather(cache, slots.cuda())
        at = slots.long()
        for got, (c, s) in ((k, cache[:2]), (v, cache[2:])):
            want = _values(c.cpu()[at // 16, :, at % 16], s.cpu()[at // 16, :, at % 16])
            assert torch.equal(got.cpu().double(), want)


def _own_batch(lens, nqs, q_heads, dim, seed, exponents, most=128):
    q, cache, table, tl, cu = _batch(lens, nqs, 64, 1, dim, q_heads, seed)
    kc, ks, vc, vs = cache
    g = torch.Generator().manual_seed(seed + 1)
    kc, vc = (torch.randint(0, 256, kc.shape, generator=g, dtype=torch.uint8) for _ in range(2))
    return q, (kc, _steps(ks.shape, exponents, seed + 2, most), vc, _steps(vs.shape, exponents, seed + 3, most)), table, tl, cu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,nqs,q_heads", KERNELS)
def test_attention_to_one_key(lens, nqs, q_heads, dim):
    """A window of one token: a query sees its own key alone, its weight is 1 and the output is the value itself.  The
    query is a one at one channel: the log-sum-exp is that channel of the key.  Roundings of the latter: scale * log2(e)
    (2 steps of 2^-24), the score (1), log2 and the product with ln 2 (4), relative; and exp2 and log2 of about 1,
    2^-21 absolute."""
    q, cache, table, tl, cu = _own_batch(lens, nqs, q_heads, dim, dim + len(lens), [-2, -1, 0, 1])
    q.zero_()
    n = q.shape[0]
    ch = (7 * torch.arange(n)[:, None] + 29 * torch.arange(q_heads)) % dim
    q.scatter_(2, ch[..., None], 1.0)
    out, lse = _run(q, cache, table, tl, cu, scale=1.0, window=1)
    for b in range(len(lens)):
        rows = torch.arange(int(cu[b]), int(cu[b + 1]))
        pos = int(tl[b]) - nqs[b] + rows - int(cu[b])
        pg, off = table[b, pos // 64].long(), pos % 64
        k, v = _values(cache[0][pg, 0, off], cache[1][pg, 0, off]), _values(cache[2][pg, 0, off], cache[3][pg, 0, off])
        assert torch.equal(out[rows].double(), v[:, None].expand(-1, q_heads, -1))
        want = k.gather(1, ch[rows])
        assert bool(((lse[rows].double() - want).abs() <= 7 * 2.0 ** -24 * want.abs() + 2.0 ** -20).all())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,nqs,q_heads", KERNELS)
def test_attention_to_code_zero(lens, nqs, q_heads, dim):
    """Codes 0 are zeros whatever the step: outputs are 0, and the log-sum-exp the logarithm of the number of keys (log2 and
    the product with ln 2: 4 steps of 2^-24)."""
    q, cache, table, tl, cu = _own_batch(lens, nqs, q_heads, dim, dim + 7, [-2, 3, 100])
    cache[0].zero_()
    cache[2].zero_()
    out, lse = _run(q, cache, table, tl, cu)
    assert not bool(out.any())
    for b in range(len(lens)):
        rows = torch.arange(int(cu[b]), int(cu[b + 1]))
        want = torch.log((int(tl[b]) - nqs[b] + 1 + rows - int(cu[b])).double())[:, None]
        assert bool(((lse[rows].double() - want).abs() <= 4 * 2.0 ** -24 * want).all())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,nqs,q_heads", KERNELS)
def test_attention_to_any_steps(lens, nqs, q_heads, dim, monkeypatch):
    """Random codes under steps of 8 bits, and under a mix in which some spans of tokens have short steps only."""
    monkeypatch.setattr(ref, "values", _values)
    q, cache, table, tl, cu = _own_batch(lens, nqs, q_heads, dim, dim + 11, [-4, -3])
    _check(q, cache, table, tl, cu)
    short = _steps(cache[1].shape, [-4, -3], 5, most=32)                      # 6 significant bits
    for t in (cache[1], cache[3]):
        t[:, :, :32] = short[:, :, :32]
    cache[1][:, :, 40] = short[:, :, 40]
    _check(q, cache, table, tl, cu)
    cache[3][:, :, 32:] = short[:, :, 32:]                                    # values short throughout, keys not
    _check(q, cache, table, tl, cu, window=90)


def test_long_and_short_steps_agree():
    """A request's bits do not depend on what steps other requests of the batch, or tokens it does not see, have."""
    q, cache, table, tl, cu = _batch([300, 260], [1, 40], 32, 1, 128, 4, seed=9)
    want, lse = _run(q[:1], cache, table[:1], tl[:1], cu[:2])
    wide = [t.clone() for t in cache]
    for i in (1, 3):
        wide[i][table[1, :9].long()] = _steps((9,) + cache[i].shape[1:], [-2], 3)
        wide[i][int(table[0, 9]), :, 12:] = _steps((1, 20, 4), [-2], 4)       # past the length
    got, l2 = _run(q[:1], wide, table[:1], tl[:1], cu[:2])
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(l2, lse)
    assert np.isfinite(float(l2[0, 0]))
