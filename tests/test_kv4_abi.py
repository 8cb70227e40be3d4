"""The 4-bit key/value cache's calls without a GPU: bad arguments are rejected on the host before anything is
launched, and the plain 64-bit implementation that judges the kernels is itself pinned."""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

import int4_group_wise_b200 as q4
import kv4_ref as ref

A, MIS4, MIS1 = 0x10000, 0x20004, 0x20001


class _Cache(ct.Structure):
    """qat4_kv4_cache of include/qat4.h."""
    _fields_ = ([(n, ct.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] + [("num_pages", ct.c_int64)] +
                [(n, ct.c_int32) for n in ("page_size", "kv_heads", "head_dim")])


def _cache(**kw):
    d = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, num_pages=10, page_size=16, kv_heads=2, head_dim=64)
    d.update(kw)
    return _Cache(*d.values())


BAD_CACHES = [(dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(page_size=8), 2), (dict(page_size=48), 2),
              (dict(page_size=256), 2), (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(kv_heads=0), 2),
              (dict(kv_heads=1025), 2), (dict(num_pages=0), 2), (dict(num_pages=1 << 28), 2), (dict(v_codes=MIS4), 3)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(kw, code):
    L, c = q4.lib(), ct.byref(_cache(**kw))
    assert L.qat4_kv4_append(c, A, A, 1, 128, 128, A, 4, None) == code
    assert L.qat4_kv4_gather(c, A, 4, A, A, None) == code
    assert L.qat4_kv4_attention(A, 256, 4, 4, c, A, 8, 8, A, A, 2, 0.1, 1, 0, A, None, A, 1 << 30, None) == code
    assert L.qat4_kv4_append(None, A, A, 1, 128, 128, A, 4, None) == 1


def test_append_and_gather_validation():
    L, c = q4.lib(), ct.byref(_cache())
    f = L.qat4_kv4_append
    assert f(c, None, A, 1, 128, 128, A, 4, None) == 1
    assert f(c, A, A, 1, 128, 128, None, 4, None) == 1
    assert f(c, A, A, 2, 128, 128, A, 4, None) == 4
    assert f(c, A, A, 1, 120, 128, A, 4, None) == 2          # rows overlap
    assert f(c, A, A, 1, 128, 128, A, -1, None) == 2
    assert f(c, A, A, 1, 132, 128, A, 4, None) == 3          # rows leave the 16-byte grid
    assert f(c, MIS4, A, 0, 128, 128, A, 4, None) == 3
    assert f(c, A, A, 0, 128, 128, MIS1, 4, None) == 3
    assert f(c, None, None, 0, 128, 128, None, 0, None) == 0  # no token: nothing to do
    g = L.qat4_kv4_gather
    assert g(c, A, 4, None, A, None) == 1
    assert g(c, A, -2, A, A, None) == 2
    assert g(c, A, 4, A, MIS4, None) == 3
    assert g(c, None, 0, None, None, None) == 0


def _tables(**kw):
    d = dict(lengths=0x10000, new=0x11000, B=4, table=0x12000, stride=8, most=8, free=0x13000, nfree=9, page=16,
             lens=0x14000, cu=0x15000, slots=0x16000, n=40, taken=0x17000)
    d.update(kw)
    return q4.lib().qat4_kv4_tables(*d.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(lengths=None), 1), (dict(table=None), 1), (dict(free=None), 1), (dict(slots=None), 1), (dict(taken=None), 1),
    (dict(B=0), 2), (dict(B=16385), 2), (dict(most=0), 2), (dict(stride=7), 2), (dict(nfree=-1), 2), (dict(n=-1), 2),
    (dict(page=24), 2), (dict(lens=0x10000), 2), (dict(cu=0x11008), 2), (dict(slots=0x10000 - 4 * 39), 2),
    (dict(table=0x11000), 2), (dict(lengths=0x10002), 3), (dict(slots=0x16001), 3)])
def test_tables_validation(kw, code):
    assert _tables(**kw) == code


def test_attention_validation():
    L, c = q4.lib(), ct.byref(_cache())
    assert q4.kv4_attention_workspace_bytes(4, 2, 4, 2, 64, 16, 8) == 0      # one launch of clusters: none
    need = q4.kv4_attention_workspace_bytes(4, 2, 4, 2, 64, 16, 800)
    assert need > 0
    base = dict(q=A, qs=256, N=4, Hq=4, c=c, t=A, ts=800, mb=800, lens=A, cu=A, B=2, scale=0.1, causal=1, window=0, out=A,
                lse=None, ws=A, wb=need)

    def f(**kw):
        return L.qat4_kv4_attention(*{**base, **kw}.values(), None)
    for kw in (dict(q=None), dict(t=None), dict(lens=None), dict(cu=None), dict(out=None), dict(ws=None, wb=need)):
        assert f(**kw) == 1, kw
    for kw in (dict(N=-1), dict(B=0), dict(B=65537), dict(Hq=5), dict(Hq=0), dict(Hq=130, qs=130 * 64), dict(qs=248),
               dict(mb=0), dict(ts=799), dict(scale=0.0), dict(scale=-0.5), dict(scale=math.nan), dict(scale=math.inf),
               dict(scale=3e38), dict(causal=2), dict(window=-1), dict(window=3, causal=0), dict(N=1 << 30),
               dict(mb=(1 << 26) + 1, ts=1 << 27)):
        assert f(**kw) == 2, kw
    for kw in (dict(q=MIS4), dict(qs=260), dict(out=MIS4), dict(ws=MIS4), dict(t=MIS1), dict(lse=MIS1), dict(cu=MIS1)):
        assert f(**kw) == 3, kw
    assert f(wb=need - 1) == 5
    assert f(N=0, q=None, out=None) == 0                      # no query: nothing to do
    for bad in ((-1, 2, 4, 2, 64, 16, 800), (4, 0, 4, 2, 64, 16, 800), (4, 2, 5, 2, 64, 16, 800), (4, 2, 4, 2, 80, 16, 800),
                (4, 2, 4, 2, 64, 16, 0)):
        assert q4.kv4_attention_workspace_bytes(*bad) == 0


def test_binding_packs_the_c_struct():
    c = _cache()
    assert q4._pack_cache(*(getattr(c, n) for n, _ in c._fields_)) == bytes(c)


def test_binding_refuses_host_tensors_and_bad_caches():
    with pytest.raises(TypeError):
        q4.kv4_append(q4.kv4_cache(2, 16, 1, 64, device="cpu"), torch.zeros(1, 1, 64), torch.zeros(1, 1, 64),
                      torch.zeros(1, dtype=torch.int32))
    for bad in ((2, 15, 1, 64), (2, 16, 1, 80), (0, 16, 1, 64), (2, 16, 0, 64)):
        with pytest.raises(ValueError):
            q4.kv4_cache(*bad, device="cpu")


# ------------------------------------------------------------------------ the reference implementation
def test_reference_quantizer_by_hand():
    """m = 7: step 1, codes are the rounded values (half to even); m = 7.1: fl(7.1/7) = 1.0142... rounds up to
    17/16; an all-zero group and one below 7 * 2^-100 have step 0."""
    x = torch.zeros(4, 32)
    x[0, :6] = torch.tensor([7.0, -6.5, 2.5, 3.5, -0.5, 0.75])
    x[1, :3] = torch.tensor([7.1, -7.1, 1.0625 * 2.5])
    x[3, :2] = torch.tensor([6.9 * 2.0 ** -100, -2.0 ** -120])
    q, s = ref.quantize(x)
    assert s[:, 0].tolist() == [1.0, 1.0625, 0.0, 0.0]
    assert q[0, :6].tolist() == [7, -6, 2, 4, 0, 1]
    assert q[1, :3].tolist() == [7, -7, 2]
    assert not q[2:].any()
    assert torch.equal(ref.unpack(ref.pack(q)), q.to(torch.int16))


def test_reference_values_are_bf16():
    q, s = ref.quantize(torch.randn(50, 128) * torch.exp(3 * torch.randn(50, 1)))
    v = q.double() * s.double().repeat_interleave(32, -1)
    assert torch.equal(v.bfloat16().double(), v)


def test_reference_attention_against_differences_of_lse():
    """The output is the gradient of the log-sum-exp with respect to a score's key bias: with one value row
    changed, out moves by its weight; and a single visible key is copied."""
    cache = ref.make_cache(6, 1, 16, 64, 0)
    table = torch.tensor([[4, 1, 3]], dtype=torch.int32)
    q = torch.randn(3, 2, 64).bfloat16()
    out, lse, _, _ = ref.attention(q, cache, table, [40], [0, 3], 0.125)
    q2 = q.double()
    h = 1e-5
    k = ref.values(cache[0][[4, 1, 3], 0].flatten(0, 1)[:40], cache[1][[4, 1, 3], 0].flatten(0, 1)[:40])
    v = ref.values(cache[2][[4, 1, 3], 0].flatten(0, 1)[:40], cache[3][[4, 1, 3], 0].flatten(0, 1)[:40])
    for i in range(3):
        s = q2[i, 1] @ k[:38 + i].T * 0.125
        assert abs(float(torch.logsumexp(s, 0) - lse[i, 1])) < 1e-12
        w = torch.zeros(38 + i, dtype=torch.float64)
        for j in range(38 + i):
            e = torch.zeros_like(s)
            e[j] = h
            w[j] = (torch.logsumexp(s + e, 0) - torch.logsumexp(s - e, 0)) / (2 * h)
        assert torch.allclose(w @ v[:38 + i], out[i, 1], atol=1e-8)
    one, l1, _, _ = ref.attention(q[:1], cache, table, [1], [0, 1], 0.125)
    assert torch.allclose(one[0, 0], v[0]) and np.isfinite(float(l1[0, 0]))


def test_reference_tables_by_hand():
    table = torch.tensor([[5, -1, -1], [-1, -1, -1]], dtype=torch.int32)
    lens, cu, slots, taken, t = ref.tables([15, 0], [3, 17], table, [9, 2, 7], 16, 21)
    assert lens == [18, 17] and cu == [0, 3, 20] and taken == 3
    assert t.tolist() == [[5, 9, -1], [2, 7, -1]]
    assert slots == [95, 144, 145] + list(range(32, 48)) + [112, -1]
