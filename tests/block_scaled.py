"""Plain 64-bit forms of the block-scaled 8-bit cache and of block-sparse decode attention, and the
inputs of their tests.  Everything here runs on the CPU, token by token or block by block, from
the definitions in include/pgd.h; it shares no code with the package.

Pools here are row-major: codes uint8 [NB][n_kv][bs][128], bf16 rows [NB][n_kv][bs][128].
`tile8` / `untile8` (and inputs.tile_pool / untile_pool for bf16) convert to the pool layout.
"""
import dataclasses
import math

import numpy as np
import torch

from paged_gqa_decode_kv_gb300 import inputs

D = 128
NAN_CODE = 0x7F


# ------------------------------------------------------------------------------ E4M3, scales
def e4m3_values() -> np.ndarray:
    """The value of every code, from its bits."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


VALUES = e4m3_values()
_POS = VALUES[:127]  # 0 .. 448, ascending


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even code, saturating; NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.nan_to_num(np.abs(x), nan=0.0, posinf=1e300), 448.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.isnan(x), NAN_CODE, c)
    return (c + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def least_pow2(amax: float, top: float) -> float:
    """2^e, e the smallest integer >= -100 with amax <= top * 2^e."""
    e = -100
    while amax > top * 2.0 ** e:
        e += 1
    return 2.0 ** e


def tile8(codes: torch.Tensor) -> torch.Tensor:
    NB, n_kv, bs, d = codes.shape
    return codes.reshape(NB, n_kv, bs // 8, 8, d // 16, 16).permute(0, 1, 2, 4, 3, 5).contiguous()


def untile8(pool: torch.Tensor) -> torch.Tensor:
    NB, n_kv, rg = pool.shape[:3]
    return pool.permute(0, 1, 2, 4, 3, 5).reshape(NB, n_kv, rg * 8, D)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


# ----------------------------------------------------------------------------------- inputs
@dataclasses.dataclass
class Cache:
    """A paged cache on the CPU, row-major, with every slot that holds no token spoiled."""
    tables: torch.Tensor      # int32 [B][MB], -1 where unused
    ctx: list                 # tokens of every sequence
    bs: int
    k: torch.Tensor           # codes uint8 or bf16 rows [NB][n_kv][bs][128]
    v: torch.Tensor
    k_scales: torch.Tensor    # fp32 [NB][n_kv], or None (bf16)
    v_scales: torch.Tensor

    @property
    def n_kv(self):
        return self.k.shape[1]

    def values(self, which: str) -> np.ndarray:
        """[NB][n_kv][bs][128] in 64 bits."""
        x, s = getattr(self, which), getattr(self, which + "_scales")
        return f64(x) if s is None else VALUES[x.numpy()] * f64(s)[:, :, None, None]

    def rows(self, which: str, b: int, n: int) -> np.ndarray:
        """The first n tokens of sequence b: [n][n_kv][128] in 64 bits."""
        nb = -(-n // self.bs)
        x = self.values(which)[self.tables[b, :nb].long().numpy()]
        return x.transpose(0, 2, 1, 3).reshape(nb * self.bs, self.n_kv, D)[:n]

    def cuda(self):
        """(k, v, k_scales, v_scales, tables, context_lens) as the calls take them."""
        if self.k_scales is None:
            k, v = inputs.tile_pool(self.k), inputs.tile_pool(self.v)
        else:
            k, v = tile8(self.k), tile8(self.v)
        up = lambda t: None if t is None else t.cuda()
        return (k.cuda(), v.cuda(), up(self.k_scales), up(self.v_scales), self.tables.cuda(),
                torch.tensor(self.ctx, dtype=torch.int32).cuda())


def make_cache(ctx, n_kv, bs, fp8=True, seed=1, room=0, scale_spread=2, spoil=True) -> Cache:
    """A cache of the given contexts; `room` more tokens fit behind each.  Codes are those of
    normal values; the scales powers of two over 2 * scale_spread + 1 binades."""
    g = torch.Generator().manual_seed(seed)
    nblk = [max(1, -(-(c + room) // bs)) for c in ctx]
    total, MB = sum(nblk), max(nblk) + 1
    NB = total + 3
    perm = torch.randperm(NB, generator=g).to(torch.int32)
    tables = torch.full((len(ctx), MB), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = perm[at:at + n]
        at += n
    held = torch.zeros(NB, bs, dtype=torch.bool)
    for b, c in enumerate(ctx):
        for j in range(-(-c // bs)):
            held[int(tables[b, j]), :min(bs, c - j * bs)] = True
    shape = (NB, n_kv, bs, D)
    ks = vs = None
    pools = []
    for _ in range(2):
        x = torch.randn(shape, generator=g)
        if fp8:
            x = (x * 110).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            bad = torch.tensor(NAN_CODE, dtype=torch.uint8)
        else:
            x, bad = x.to(torch.bfloat16), torch.tensor(float("nan"), dtype=torch.bfloat16)
        pools.append(torch.where(held[:, None, :, None], x, bad) if spoil else x)
    if fp8:
        ks, vs = [torch.exp2(torch.randint(-7 - scale_spread, -6 + scale_spread, (NB, n_kv),
                                           generator=g).float()) for _ in range(2)]
    return Cache(tables, list(ctx), bs, pools[0], pools[1], ks, vs)


def make_query(B, n_q, seed=2, std=1.0) -> torch.Tensor:
    return (torch.randn(B, n_q, D, generator=torch.Generator().manual_seed(seed)) * std).to(
        torch.bfloat16)


# -------------------------------------------------------------------------------- definitions
def append(c: Cache, k_new: torch.Tensor, v_new: torch.Tensor, positions, starts) -> None:
    """kv_append_fp8b on the cache itself; k_new / v_new [N][n_kv][128]."""
    for new, codes, scales in ((k_new, c.k, c.k_scales), (v_new, c.v, c.v_scales)):
        x = f64(new)
        for b, p in enumerate(positions):
            n = starts[b + 1] - starts[b]
            for j in range(p // c.bs, -(-(p + n) // c.bs) if n else 0):
                blk = int(c.tables[b, j])
                s0, s1 = max(0, p - j * c.bs), min(c.bs, p + n - j * c.bs)
                r0 = starts[b] + j * c.bs + s0 - p
                for g in range(c.n_kv):
                    y = x[r0:r0 + s1 - s0, g]
                    fin = np.abs(y[np.isfinite(y)])
                    s = least_pow2(float(fin.max()) if fin.size else 0.0, 448.0)
                    if s0:
                        old = float(scales[blk, g])
                        s = max(s, old)
                        if s != old:
                            early = VALUES[codes[blk, g, :s0].numpy()] * (old / s)
                            codes[blk, g, :s0] = torch.from_numpy(e4m3_codes(early))
                    codes[blk, g, s0:s1] = torch.from_numpy(e4m3_codes(y / s))
                    scales[blk, g] = s


def attention(q: torch.Tensor, k: np.ndarray, v: np.ndarray, scale: float):
    """One sequence: q [n_q][128], k / v [n][n_kv][128] -> (output [n_q][128], weighted mean of
    |v|, the same shape)."""
    n_q, n_kv = q.shape[0], k.shape[1]
    G = n_q // n_kv
    out, mag = np.zeros((n_q, D)), np.zeros((n_q, D))
    for h in range(n_q):
        s = k[:, h // G] @ f64(q[h]) * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        out[h] = w @ v[:, h // G]
        mag[h] = w @ np.abs(v[:, h // G])
    return out, mag


def paged(c: Cache, q: torch.Tensor, scale: float):
    got = [attention(q[b], c.rows("k", b, n), c.rows("v", b, n), scale)
           for b, n in enumerate(c.ctx)]
    return np.stack([x for x, _ in got]), np.stack([m for _, m in got])


def bounds(c: Cache, b: int, j: int, g: int, n: int):
    """Bounds of block j of sequence b (context n) and head g: (lower, upper, scale)."""
    x = c.values("k")[int(c.tables[b, j]), g, :min(c.bs, n - j * c.bs)]
    s = least_pow2(float(np.abs(x).max()), 127.0)
    return np.floor(x.min(0) / s), np.ceil(x.max(0) / s), s


def select(q: torch.Tensor, lower, upper, scales, W, first, last):
    """Selected blocks of one sequence and KV head: q [G][128], bounds [n][128], scales [n]."""
    n = len(scales)
    if n <= W:
        return list(range(n))
    score = np.full(n, -math.inf)
    for h in range(q.shape[0]):
        x = f64(q[h])
        f = least_pow2(float(np.abs(x).max()), 127.0)
        r = np.rint(x / f)
        score = np.maximum(score, (np.maximum(r, 0) * upper + np.minimum(r, 0) * lower).sum(1) * f)
    score = score * scales
    score[:first] = math.inf
    score[n - last:] = math.inf
    return sorted(sorted(range(n), key=lambda j: (-score[j], j))[:W])


def selected(c: Cache, q: torch.Tensor, chosen, scale: float):
    """Attention over chosen[b][g] (block lists): (output, weighted mean of |v|)."""
    n_q, G = q.shape[1], q.shape[1] // c.n_kv
    out, mag = np.zeros((len(c.ctx), n_q, D)), np.zeros((len(c.ctx), n_q, D))
    for b, n in enumerate(c.ctx):
        k, v = c.rows("k", b, n), c.rows("v", b, n)
        for g in range(c.n_kv):
            at = [t for j in chosen[b][g] for t in range(j * c.bs, min(n, (j + 1) * c.bs))]
            hs = slice(g * G, (g + 1) * G)
            out[b, hs], mag[b, hs] = attention(q[b, hs], k[at, g:g + 1], v[at, g:g + 1], scale)
    return out, mag


def close(got: torch.Tensor, want: np.ndarray, mag: np.ndarray, p_err: float = 2.0 ** -8,
          label: str = "") -> None:
    """A decode output against its 64-bit form.

    Element by element, with w_t the weights and mag = sum_t w_t |v_t|: each weight carries a
    relative rounding of at most p_err (2^-8: bf16, or two E4M3 terms, 2^-4 each), and the score
    it is the exponential of an absolute error that stays below 2^-8 here (fp32 sums of 128
    products of size < 32: 128 * 32 * 2^-24 = 2^-12, and queries split to 2^-17 of their largest),
    so numerator and denominator are off by at most (p_err + 2^-8) each; the result is then
    rounded to bf16, by at most 2^-8 of itself: |got - want| <= 2 (p_err + 2^-8) mag + 2^-8 |want|.

    As a whole: the roundings are independent of the values' signs, so in the 2-norm the
    error stays within 2^-8 (weights) + 2^-8 (output) of the result's."""
    g = got.detach().float().cpu().double().numpy()
    assert np.isfinite(g).all(), "%s: not finite" % label
    err = np.abs(g - want)
    tol = 2 * (p_err + 2.0 ** -8) * mag + 2.0 ** -8 * np.abs(want) + 1e-30
    assert (err <= tol).all(), "%s: off by %.3g of its bound" % (label, float((err / tol).max()))
    rel = np.linalg.norm(g - want) / max(np.linalg.norm(want), 1e-300)
    assert rel <= p_err + 2.0 ** -8, "%s: %.3g in the 2-norm" % (label, rel)
