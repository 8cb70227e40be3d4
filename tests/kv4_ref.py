"""Plain 64-bit implementation of the 4-bit key/value cache (CPU, torch): quantizer, tables, attention, and
the error bounds of the kernels' attention derived from it."""
import math

import numpy as np
import torch


def quantize(x):
    """(codes int8, step float32) of x [..., D] (float32 values): step [..., D / 32], by the definition in
    include/qat4.h; binary32 divisions as numpy does them."""
    y = x.to(torch.float32).numpy().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(all="ignore"):
        m = np.fmax.reduce(np.abs(y), axis=-1)                  # passes NaN over
        m = np.where(np.isnan(m), np.float32(0), m).astype(np.float32)
        d = (m / np.float32(7)).astype(np.float32)
        up = ((d.view(np.uint32).astype(np.uint64) + 0x7FFFF) & 0xFFF80000).astype(np.uint32).view(np.float32)
        step = np.where(d < np.float32(2.0 ** -100), np.float32(0), np.minimum(up, np.float32(2.0 ** 100))).astype(np.float32)
        q = np.rint((y / step[..., None]).astype(np.float32))
        q = np.where(np.isnan(q), -8, np.clip(q, -8, 7))        # clamp as max then min with NaN passed over
        q = np.where(step[..., None] == 0, 0, q)
    return torch.from_numpy(q.astype(np.int8).reshape(x.shape)), torch.from_numpy(step)


def pack(codes):
    n = codes.to(torch.int16) & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)


def unpack(codes):
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int16)
    return torch.where(n > 7, n - 16, n)


def values(codes, scales):
    """float64 values of packed codes [..., D / 2] and bf16 steps [..., D / 32]."""
    return unpack(codes).double() * scales.double().repeat_interleave(32, -1)


def make_cache(pages, heads, page, dim, seed, spread=0.4):
    """Packed cache of random tokens on the CPU, in the form append writes."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        gain = torch.exp(spread * torch.randn(heads, 1, dim, generator=g))
        q, s = quantize(torch.randn(pages, heads, page, dim, generator=g) * gain)
        out += [pack(q), s.bfloat16()]
    return out


def tables(lengths, new, table, free, page, num_slots):
    B, most = table.shape
    table = table.clone()
    cu, slots, taken = [0], [], 0
    for b in range(B):
        h, n = max(0, int(lengths[b])), max(0, int(new[b]))
        for i in range(min(most, -(-h // page)), min(most, -(-(h + n) // page))):
            table[b, i] = int(free[taken]) if taken < len(free) else -1
            taken += 1
        for x in range(h, h + n):
            p = int(table[b, x // page]) if x // page < most else -1
            slots.append(p * page + x % page if p >= 0 else -1)
        cu.append(cu[-1] + n)
    slots = (slots + [-1] * num_slots)[:num_slots]
    lens = [max(0, int(a)) + max(0, int(b)) for a, b in zip(lengths, new)]
    return lens, cu, slots, taken, table


def attention(q, cache, table, lens, cu, scale, causal=True, window=0):
    """out, lse in float64 and their error bounds, for q bf16 [N, Hq, D] on the CPU.  Rows of no request are
    NaN in all four.

    Bound of out.  Keys, values and products are exact.  A score's float32 sum of D products is off by at
    most (D + 4) 2^-23 sum |q k| (one step per addition and a few of the scaling), so a weight's exponent is
    off by d = scale (D + 4) 2^-23 max sum |q k| and the row's maximum by as much; exp2 adds 2^-21 and the
    subtraction of the maximum 2^-23 |scale q k|, both well inside 4 d + 2^-20.  A weight rounded to bf16 is
    off by 2^-8 of itself, the sums of n weights and n products by n 2^-23 of theirs, and the result by its
    rounding to bf16, 2^-8 |out|.  With A = sum p |v| this gives
        |err| <= 2^-8 |out| + (1.01 2^-8 + r) A + r |out|,  r = 4 d + 2^-20 + n 2^-22.
    Bound of lse: r + 2^-22 |lse|."""
    kc, ks, vc, vs = cache
    P, D, Hkv = kc.shape[2], kc.shape[3] * 2, kc.shape[1]
    N, Hq, _ = q.shape
    group = Hq // Hkv
    out = torch.full((N, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((N, Hq), math.nan, dtype=torch.float64)
    tol, ltol = out.clone(), lse.clone()
    for b in range(len(lens)):
        a, e = int(cu[b]), int(cu[b + 1])
        nq, n = e - a, min(int(lens[b]), table.shape[1] * P)
        if nq <= 0:
            continue
        pos = torch.arange(n - nq, n)[:, None]
        key = torch.arange(n)[None, :]
        pages = table[b, :-(-n // P)].long()
        good = (pages >= 0) & (pages < kc.shape[0])
        see = good.repeat_interleave(P)[:n][None, :].expand(nq, n).clone()
        if causal:
            see &= key <= pos
        if window:
            see &= key > pos - window
        idx = torch.where(good, pages, torch.zeros_like(pages))
        none = ~see.any(1)
        for h in range(Hkv):
            k = values(kc[idx, h].flatten(0, 1)[:n], ks[idx, h].flatten(0, 1)[:n])
            v = values(vc[idx, h].flatten(0, 1)[:n], vs[idx, h].flatten(0, 1)[:n])
            anyone = see.any(0)
            k[~anyone] = 0
            v[~anyone] = 0
            for j in range(h * group, (h + 1) * group):
                x = q[a:e, j].double()
                s = (x @ k.T * scale).masked_fill(~see, -math.inf)
                mx = s.amax(1, keepdim=True) if n else torch.full((nq, 1), -math.inf, dtype=torch.float64)
                mx = torch.where(torch.isinf(mx), torch.zeros_like(mx), mx)
                w = torch.exp(s - mx)
                tot = w.sum(1, keepdim=True)
                p = w / torch.where(tot > 0, tot, torch.ones_like(tot))
                o = p @ v
                mag = ((x.abs() @ k.abs().T) * see).amax(1, keepdim=True) if n else torch.zeros(nq, 1, dtype=torch.float64)
                r = 4 * scale * (D + 4) * 2.0 ** -23 * mag + 2.0 ** -20 + n * 2.0 ** -22
                out[a:e, j] = o
                tol[a:e, j] = 2.0 ** -8 * o.abs() + (1.01 * 2.0 ** -8 + r) * (p @ v.abs()) + r * o.abs() + 1e-30
                l = (mx + torch.log(tot))[:, 0]
                l[none] = -math.inf
                lse[a:e, j] = l
                ltol[a:e, j] = torch.where(none, torch.zeros_like(l), r[:, 0] + 2.0 ** -22 * l.abs())
    return out, lse, tol, ltol
