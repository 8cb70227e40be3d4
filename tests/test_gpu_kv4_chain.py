"""The cache's calls and the product on the packed export in one stream, as the layers of a decode step make them.  Each
call may start before the one ahead of it has ended, so a captured chain is compared bit by bit with the same calls
synchronised one by one."""
import pytest
import torch

import int4_group_wise_b200 as q4

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _layers(n_layers, tokens, lens, q_heads, heads, dim, seed):
    """Caches, o-projections and a step's stacked rows for every layer; requests of lens[b] tokens held."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    page, B = 32, len(lens)
    blocks = -(-(max(lens) + tokens) // page)
    table = torch.randperm(B * blocks, generator=g, device="cuda").to(I32).view(B, blocks)
    free = torch.zeros(0, dtype=I32, device="cuda")
    d = dict(table=table, free=free, page=page, lens=torch.tensor(lens, dtype=I32, device="cuda"),
             new=torch.tensor([tokens] * B, dtype=I32, device="cuda"), layers=[])
    for _ in range(n_layers):
        cache = q4.kv4_cache(B * blocks, page, heads, dim)
        x = torch.randn((2, B * blocks * page, heads, dim), generator=g, device="cuda")
        q4.kv4_append(cache, x[0], x[1], torch.arange(B * blocks * page, dtype=I32, device="cuda"))
        W = 0.02 * torch.randn((512, q_heads * dim), generator=g, device="cuda")
        delta = (W.abs().unflatten(1, (-1, 32)).amax(2) / 7).contiguous()
        packed, scales = q4.pack_w4a16(W, delta)
        d["layers"].append(dict(cache=cache, packed=packed, scales=scales, y=torch.empty((B * tokens, 512), device="cuda")))
    return d


def _step(d, qkv, out, q_heads, heads, between=lambda: None):
    """All layers on one output buffer; out None: the attention writes over its queries."""
    n = qkv.shape[1]
    dim = qkv.shape[3]
    lens, cu, slots, _ = q4.kv4_tables(d["lens"], d["new"], d["table"], d["free"], d["page"], n)
    between()
    ys = []
    for x, q, lay in zip(qkv, d["q"], d["layers"]):
        q4.kv4_append(lay["cache"], x[:, q_heads:q_heads + heads], x[:, q_heads + heads:], slots)
        between()
        if out is None:
            q.copy_(x[:, :q_heads])
            between()
            o = q4.kv4_attention(q, lay["cache"], d["table"], lens, cu, out=q)
        else:
            o = q4.kv4_attention(x[:, :q_heads], lay["cache"], d["table"], lens, cu, out=out)
        between()
        ys.append(q4.w4a16_gemv(o.view(n, q_heads * dim), lay["packed"], lay["scales"], y=lay["y"]))
        between()
    return ys


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens,lens,q_heads,heads,dim", [(1, [300], 32, 8, 128), (1, [900, 31, 4000, 77], 32, 8, 64),
                                                           (5, [513, 60], 8, 2, 128), (40, [700], 4, 1, 128)])
def test_attention_then_product(tokens, lens, q_heads, heads, dim, in_place):
    n = tokens * len(lens)
    d = _layers(6, tokens, lens, q_heads, heads, dim, seed=dim + tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.zeros((6, n, q_heads + 2 * heads, dim), dtype=torch.bfloat16, device="cuda")
    d["q"] = [torch.zeros((n, q_heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    out = None if in_place else torch.zeros((n, q_heads, dim), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(d, qkv, out, q_heads, heads)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = _step(d, qkv, out, q_heads, heads)
    for _ in range(4):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in ys]
        for y in ys:
            y.fill_(7.0)
        torch.cuda.synchronize()
        want = _step(d, qkv, out, q_heads, heads, between=torch.cuda.synchronize)
        for a, b in zip(got, want):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all()) and bool(a.any())
    q4.sync_check()


@pytest.mark.parametrize("B,nq,heads,n,room", [(1, 40, 8, 1 << 29, 10240), (4, 1, 64, 1 << 30, 4)])
def test_product_behind_a_long_attention(B, nq, heads, n, room):
    """The product's bounded waits begin when the kernel ahead of it has ended: an attention of six seconds (a chunk of
    40 tokens on 2^29 in a batch padded to 10240, whose 8 items leave most SMs to the product; four requests of 2^30
    tokens, the longest allowed) does not run them out.  All keys weigh the same and all values are one: outputs of exactly
    one, and the log-sum-exp log(n) (log2 and the product with ln 2, 4 steps of 2^-24)."""
    dim, page, R = 64, 128, 32768                # more stages for a CTA of the product than its ring holds
    cache = q4.kv4_cache(1, page, heads, dim)
    cache.v_codes.fill_(0x11)
    cache.v_scales.fill_(1.0)
    table = torch.zeros((B, n // page), dtype=I32, device="cuda")
    lens, cu = torch.full((B,), n, dtype=I32, device="cuda"), nq * torch.arange(B + 1, dtype=I32, device="cuda")
    rows = B * nq
    q = torch.zeros((room, heads, dim), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((room, heads), device="cuda")
    C = heads * dim
    packed, scales = torch.full((R, C // 2), 0x11, dtype=torch.uint8, device="cuda"), torch.ones((R, C // 32), device="cuda").half()
    y = q4.w4a16_gemv(q[:rows].view(rows, C) + 1, packed, scales)
    torch.cuda.synchronize()
    assert bool((y == C).all())
    out = q4.kv4_attention(q, cache, table, lens, cu, causal=False, lse=lse)
    y = q4.w4a16_gemv(out[:rows].view(rows, C), packed, scales)
    q4.sync_check()
    assert bool((out[:rows] == 1).all()) and bool((y == C).all())
    want = torch.log(torch.tensor(float(n), dtype=torch.float64))
    assert bool(((lse[:rows].cpu().double() - want).abs() <= 4 * 2.0 ** -24 * want).all())
