"""How far a decode output over the block-scaled cache may be from its 64-bit form, from the inputs and
from the arithmetic that include/pgd.h states, and inputs whose outputs cancel, so that an error of
the weights is not hidden behind the output's rounding to bf16."""
import numpy as np
import torch

import block_scaled as bsc

D = 128


def split_query(q: np.ndarray) -> np.ndarray:
    """The two E4M3 terms of a query [n_q][128] added up, with a head's power-of-two scale that puts
    its largest element into [128, 256)."""
    top = np.abs(q).max(-1, keepdims=True)
    s = np.exp2(np.floor(np.log2(np.where(top > 0, top, 1.0))) - 7)
    x = q / s
    hi = bsc.VALUES[bsc.e4m3_codes(x)]
    return (hi + bsc.VALUES[bsc.e4m3_codes(x - hi)]) * s


def weight_terms(x: np.ndarray, terms: int) -> np.ndarray:
    """x as `terms` E4M3 numbers, each the rounding of 2^5 times what the ones before it leave."""
    got, left = np.zeros_like(x), x.copy()
    for i in range(terms):
        t = bsc.VALUES[bsc.e4m3_codes(left * 2.0 ** (5 * i))] * 2.0 ** (-5 * i)
        got, left = got + t, left - t
    return got


def bound(q, k, v, v_scale, scale, fp32):
    """One sequence's output and the bound of its error, [n_q][128]: q [n_q][128], k / v
    [n][n_kv][128] and v's scales [n][n_kv], all in 64 bits.

    The score of a token, a sum of 128 exact products in fp32 (truncated at worst: 2^-23 a step) and
    four more roundings, is off by at most scale * sum |dq k| + 2^-16 scale sum |q k| + 2^-22 |s| (dq:
    what the query's two terms leave; none in fp32); the exponential's argument, in log2 units and
    relative to a reference that may hold log2 of the V scale, by 2^-23 (|s| + |max| + 128) ln 2 more,
    the exponential itself by 2^-22.  A weight off by the factor exp(e) moves numerator and denominator
    by at most e^e - 1 of its share in each.  The numerator's weight (times V's scale) is held to 2^-12
    of itself and 2^-24 of the head's largest (not so in fp32: one rounding).  Sums: fp32 steps over
    the n tokens, 2^-23 each, and the roundings of a merge of the parts, n / 32 + 256 of them with
    room.  The output is rounded to bf16, by 2^-8 of itself at most."""
    n_q, n, n_kv = q.shape[0], k.shape[0], k.shape[1]
    G = n_q // n_kv
    out, tol = np.zeros((n_q, D)), np.zeros((n_q, D))
    left = np.zeros_like(q) if fp32 else np.abs(q - split_query(q))
    sums = (n / 32 + 256) * 2.0 ** -23
    for h in range(n_q):
        kh, vh, sv = k[:, h // G], v[:, h // G], v_scale[:, h // G]
        s = kh @ q[h] * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        e = scale * (np.abs(kh) @ left[h] + 2.0 ** -16 * (np.abs(kh) @ np.abs(q[h])))
        e += 2.0 ** -22 * np.abs(s) + 2.0 ** -23 * (np.abs(s) + np.abs(s).max() + 128) + 2.0 ** -22
        e = np.expm1(e)
        share = w * (e + sums + (2.0 ** -24 if fp32 else 2.0 ** -12))
        out[h] = w @ vh
        mag = w @ np.abs(vh)
        tol[h] = share @ np.abs(vh) + (w @ e + sums) * mag
        if not fp32:
            codes = np.abs(vh) / sv[:, None]
            tol[h] += 2.0 ** -24 * (w * sv).max() * codes.sum(0)
        tol[h] = 1.01 * tol[h]  # (products of the relative errors)
        tol[h] += 2.0 ** -8 * np.abs(out[h]) + 2.0 ** -126
    return out, tol


def check(got, out, tol, label=""):
    g = got.detach().float().cpu().double().numpy() if isinstance(got, torch.Tensor) else got
    assert np.isfinite(g).all(), "%s: not finite" % label
    over = np.abs(g - out) / tol
    assert over.max() <= 1, "%s: off by %.3g of its bound" % (label, over.max())


def cancelling_cache(n_seq, n_kv, G, bs, seed, scale):
    """(cache, query): each sequence two blocks, the second part full; in each block two tokens that
    hold nearly all of the weight.  Every V row is plus (first block) or minus (second) one pattern,
    and the second block's V scale is what makes the blocks' parts of the output cancel.  The heads
    of a KV head are alike, and a query's elements are those that two E4M3 terms hold exactly."""
    r = np.random.default_rng(seed)
    ctx = [int(bs + r.integers(2, bs + 1)) for _ in range(n_seq)]
    c = bsc.make_cache(ctx, n_kv, bs, seed=seed)
    q = torch.from_numpy(r.standard_normal((n_seq, n_kv, D)) * 0.25).to(torch.bfloat16)
    q = torch.where(q.abs() < q.abs().amax(-1, keepdim=True) / 256, torch.zeros_like(q), q)
    q = q.repeat_interleave(G, 1)
    assert (split_query(bsc.f64(q).reshape(-1, D)) == bsc.f64(q).reshape(-1, D)).all()
    c.k_scales.fill_(2.0 ** -7)
    for b, n in enumerate(ctx):
        for g in range(n_kv):
            x = bsc.f64(q[b, g * G])
            # the other tokens' keys lie against the query: scores of -14 and less
            against = -np.sign(x) * min(3.5, 14 / scale / np.abs(x).sum())
            pattern = bsc.e4m3_codes(r.uniform(64, 448, D) * r.choice([-1, 1], D))
            for j in range(2):
                blk, m = int(c.tables[b, j]), min(bs, n - j * bs)
                k = np.tile(against, (m, 1))
                heavy = r.choice(m, 2, replace=False)
                k[heavy] = r.standard_normal((2, D)) * 0.4
                c.k[blk, g, :m] = torch.from_numpy(bsc.e4m3_codes(k * 2.0 ** 7))
                c.v[blk, g, :m] = torch.from_numpy(pattern ^ np.uint8(128 * j))
                c.v_scales[blk, g] = 1.0
            s = c.rows("k", b, n)[:, g] @ x * scale
            w = np.exp(s - s.max())
            c.v_scales[int(c.tables[b, 1]), g] = w[:bs].sum() / w[bs:].sum()
    return c, q


def v_scales(c, b, n):
    """V's scale of every token of a sequence, [n][n_kv]."""
    nblk = -(-n // c.bs)
    return bsc.f64(c.v_scales)[c.tables[b, :nblk].long().numpy()].repeat(c.bs, 0)[:n]


def bounds_of(c, q, scale, fp32):
    got = [bound(bsc.f64(q[b]), c.rows("k", b, n), c.rows("v", b, n), v_scales(c, b, n), scale, fp32)
           for b, n in enumerate(c.ctx)]
    return np.stack([x for x, _ in got]), np.stack([t for _, t in got])
