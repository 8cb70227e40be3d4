"""What the bounds of kv4_ref.py cannot see on long contexts: every key counted once, wherever a request is cut, and the
weights' full 16 bits in tiles of 4 rows."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from test_gpu_kv4 import _batch, _run

pytestmark = pytest.mark.gpu

# (lengths, queries, query heads, kv heads, page): the grid-wide split with tiles of 4, 8, 16 and 24 rows; clusters;
# prompts in one part and in several; decode tokens beside a chunk of a prompt
CUTS = [([20011], [1], 4, 1, 64), ([9001, 3, 4100, 129], [1, 1, 1, 1], 8, 2, 16), ([20011], [2], 4, 1, 128),
        ([12000, 777], [4, 3], 4, 1, 32), ([300] * 66 + [9000], [5] * 67, 4, 1, 64), ([4096], [1], 4, 1, 16),
        ([2049, 128], [3, 1], 4, 1, 64), ([777], [777], 8, 2, 64), ([16000], [40], 4, 1, 64), ([9000, 300], [129, 1], 4, 1, 32),
        ([700] * 20 + [5000], [1] * 20 + [300], 8, 2, 64), ([129] * 70 + [3000], [1] * 70 + [20], 8, 1, 16)]


def _uniform(lens, nqs, q_heads, heads, page, dim, seed):
    """A batch whose queries are zero, so that every key that a query sees weighs the same, and whose values are one at
    channel (token + head) % dim and zero elsewhere."""
    q, cache, table, tl, cu = _batch(lens, nqs, page, heads, dim, q_heads, seed)
    q.zero_()
    kc, ks, vc, vs = (t.clone() for t in cache)
    codes = torch.zeros((kc.shape[0], heads, page, dim), dtype=torch.int8)
    vs.fill_(1.0)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        pg, off = table[b, pos // page].long(), pos % page
        for h in range(heads):
            codes[pg, h, off, (pos + h) % dim] = 1
    return q, (kc, ks, ref.pack(codes), vs), table, tl, cu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 3000])
@pytest.mark.parametrize("lens,nqs,q_heads,heads,page", CUTS)
def test_every_key_counts_once(lens, nqs, q_heads, heads, page, window, dim):
    """Weights are 1/n: the log-sum-exp is log(n) (log2 and the product with ln 2, 4 steps of 2^-24; one key more or less is
    1/n, at least 2^-15), and a channel's output is the number of its tokens over n.  The sums and the product with 1/n are
    exact to 2^-22, the rounding to bf16 2^-8: at 128 channels and up to 12000 tokens a count is at most 94 and met to 0.37, so that
    one token more or less, itself rounded, shows there too."""
    q, cache, table, tl, cu = _uniform(lens, nqs, q_heads, heads, page, dim, seed=len(lens) + dim)
    out, lse = _run(q, cache, table, tl, cu, window=window)
    group = q_heads // heads
    for b in range(len(lens)):
        rows = torch.arange(int(cu[b]), int(cu[b + 1]))
        pos = lens[b] - nqs[b] + rows - int(cu[b])
        lo = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
        n = (pos + 1 - lo).double()
        want = torch.log(n)[:, None]
        assert bool(((lse[rows].double() - want).abs() <= 4 * 2.0 ** -24 * want).all())
        ch = torch.arange(dim)
        for h in range(heads):
            # tokens j in [lo, pos] with (j + h) % dim == ch
            upto = lambda m: torch.div(m[:, None] - 1 - (ch - h) % dim, dim, rounding_mode="floor") + 1   # noqa: E731  below m
            count = (upto(pos + 1) - upto(lo)).double()
            assert bool((count.sum(1) == n).all()) 
            got = out[rows, h * group:(h + 1) * group].double() * n[:, None, None]
            err = (got - count[:, None]).abs()
            assert bool((err <= (2.0 ** -8 + 2.0 ** -22) * count[:, None]).all()), float(err.max())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [[2, 2], [2] * 80, [6, 40, 300], [5000, 64], [9001]])
def test_tiles_of_four_rows_keep_16_bits_of_the_weights(lens, dim):
    """Tokens in pairs of nearly the same key and opposite values: what is left of a pair is the difference of its weights, and
    with it the rounding of each, 2^-16 in these tiles (2^-8, and 2^-8 of what that left).  The bound of kv4_ref.attention with
    that in the place of 2^-8."""
    q_heads, page = 4, 16
    q, cache, table, tl, cu = _batch(lens, [1] * len(lens), page, 1, dim, q_heads, seed=dim + len(lens))
    codes = [ref.unpack(cache[0]).to(torch.int8), ref.unpack(cache[2]).to(torch.int8)]
    ks, vs = cache[1].clone(), cache[3].clone()
    q = q * (2.0 if max(lens) > 2 else 1.0)
    for b, n in enumerate(lens):
        pos = torch.arange(0, n - 1, 2)
        pg, off = table[b, pos // page].long(), pos % page           # a pair never crosses a page
        for t in (codes[0], codes[1], ks, vs):
            t[pg, :, off + 1] = t[pg, :, off]
        codes[0][pg, :, off + 1, 5] = codes[0][pg, :, off, 5] ^ 1    # one code of the key differs by one
        codes[1][pg, :, off] = codes[1][pg, :, off].clamp(min=-7)
        codes[1][pg, :, off + 1] = -codes[1][pg, :, off]
    cache = (ref.pack(codes[0]), ks, ref.pack(codes[1]), vs)
    out, _ = _run(q, cache, table, tl, cu)
    scale = float(np.float32(dim ** -0.5))
    for b, n in enumerate(lens):
        idx = table[b, :-(-n // page)].long()
        k = ref.values(cache[0][idx, 0].flatten(0, 1)[:n], ks[idx, 0].flatten(0, 1)[:n])
        v = ref.values(cache[2][idx, 0].flatten(0, 1)[:n], vs[idx, 0].flatten(0, 1)[:n])
        x = q[b].double()
        p = (x @ k.T * scale).softmax(1)
        want, mass = p @ v, p @ v.abs()
        r = 4 * scale * (dim + 4) * 2.0 ** -23 * (x.abs() @ k.abs().T).amax(1, keepdim=True) + 2.0 ** -20 + n * 2.0 ** -22
        tol = 2.0 ** -8 * want.abs() + (1.01 * 2.0 ** -16 + r) * mass + r * want.abs()
        err = (out[b].double() - want).abs()
        assert bool((err <= tol).all()), (b, float((err / tol).max()))
