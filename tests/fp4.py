"""Plain 64-bit forms of the 4-bit cache (E2M1 codes, an E4M3 scale per token, head and 16 dims), of
rotary positions and of block tables, and the bound of an attention output's error.

Shares no code with the package: values and roundings are worked out from the formats' bits, layouts
from the byte places that include/pgd.h gives."""
import numpy as np
import torch

import block_scaled as bsc

D, GROUP = 128, 1152
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
CODES = np.concatenate([E2M1, -E2M1])


def _places(is_v):
    """(byte, is the high nibble, scale byte) of token t and dim i of a group, [16][128] each."""
    t, i = np.arange(16)[:, None], np.arange(D)[None, :]
    if is_v:
        byte = i // 64 * 512 + i % 8 * 64 + t // 4 * 16 + i // 8 % 8 * 2 + t % 4 // 2
        return byte, t % 2 + 0 * i == 1, 1024 + t // 4 * 32 + i // 16 * 4 + t % 4
    return t * 64 + i // 2, i % 2 + 0 * t == 1, 1024 + t * 8 + i // 16


def unpack(pool, is_v):
    """Pool uint8 [NB][n_kv][bs/16][1152] -> codes [NB][n_kv][bs][128], scale bytes [..][bs][8]."""
    x = np.asarray(pool)
    byte, high, sc = _places(is_v)
    c = x[..., byte]
    c = np.where(high, c >> 4, c & 15)
    s = x[..., sc[:, ::16]]
    NB, n_kv, ng = x.shape[:3]
    return c.reshape(NB, n_kv, ng * 16, D), s.reshape(NB, n_kv, ng * 16, 8)


def pack(codes, scales, is_v):
    """The other way."""
    NB, n_kv, bs = codes.shape[:3]
    c = codes.reshape(NB, n_kv, bs // 16, 16, D).astype(np.uint8)
    out = np.zeros((NB, n_kv, bs // 16, GROUP), np.uint8)
    byte, high, sc = _places(is_v)
    for t in range(16):
        for half in (False, True):
            m = high[t] == half
            out[..., byte[t][m]] |= c[..., t, :][..., m] << (4 if half else 0)
        out[..., sc[t, ::16]] = scales.reshape(NB, n_kv, bs // 16, 16, 8)[..., t, :]
    return out


def values(codes, scales, S):
    """What codes [...][128] with scale bytes [...][8] stand for."""
    return CODES[codes] * np.repeat(bsc.VALUES[scales], 16, -1) * S


def quantise(x, S):
    """bf16 values [...][128] (in 64 bits) -> codes, scale bytes."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        g = x.reshape(*x.shape[:-1], 8, 16)
        m = np.abs(g).max(-1)  # (NaN wins)
        s = bsc.e4m3_codes(np.minimum(m / (6 * S), 1e30))
        f = bsc.VALUES[s] * S
        y = np.abs(g) / np.where(f > 0, f, 1.0)[..., None]
        y = np.where((f > 0)[..., None], np.minimum(np.nan_to_num(y, nan=0.0, posinf=6.0), 6.0),
                     0.0)
        hi = np.minimum(np.searchsorted(E2M1, y), 7)
        lo = np.maximum(hi - 1, 0)
        up, down = E2M1[hi] - y, y - E2M1[lo]
        code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        code = code + 8 * np.signbit(g)
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


class Cache:
    """A paged 4-bit cache on the CPU, row-major; slots that hold no token have NaN scales."""

    def __init__(self, ctx, n_kv, bs, seed=1, room=0, S=(0.5, 2.0)):
        r = np.random.default_rng(seed)
        self.ctx, self.n_kv, self.bs, self.S = list(ctx), n_kv, bs, S
        nblk = [-(-(n + room) // bs) for n in ctx]
        self.NB = sum(nblk) + 3
        MB = max(nblk + [1])
        perm = r.permutation(self.NB)
        self.tables = np.full((len(ctx), MB), -1, np.int32)
        at = 0
        for b, n in enumerate(nblk):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        self.codes, self.scales = [], []
        for S1 in S:
            x = r.standard_normal((self.NB, n_kv, bs, D)) * np.exp(
                0.3 * r.standard_normal((self.NB, n_kv, bs, 1)))
            c, s = quantise(bsc.f64(torch.from_numpy(x).to(torch.bfloat16)), S1)
            for b, n in enumerate(ctx):
                for j in range(nblk[b]):
                    s[self.tables[b, j], :, max(0, min(bs, n - j * bs)):] = 0x7F
            self.codes.append(c)
            self.scales.append(s)

    def cuda(self):
        """(k, v, tables, context_lens) as the calls take them."""
        pools = [torch.from_numpy(pack(c, s, i == 1)).cuda()
                 for i, (c, s) in enumerate(zip(self.codes, self.scales))]
        return (*pools, torch.from_numpy(self.tables).cuda(),
                torch.tensor(self.ctx, dtype=torch.int32).cuda())

    def take(self, k, v):
        """Replaces the contents by pools'."""
        for i, p in enumerate((k, v)):
            self.codes[i], self.scales[i] = unpack(p.cpu().numpy(), i == 1)

    def rows(self, which, b, n, lo=0):
        """Tokens lo .. n - 1 of sequence b: [n - lo][n_kv][128]."""
        p = np.arange(lo, n)
        blk = self.tables[b, p // self.bs]
        return values(self.codes[which][blk, :, p % self.bs],
                      self.scales[which][blk, :, p % self.bs], self.S[which])

    def append(self, k_new, v_new, positions, starts):
        """k_new, v_new [N][n_kv][128] bf16 tensors."""
        for i, x in enumerate((k_new, v_new)):
            c, s = quantise(bsc.f64(x), self.S[i])
            for b, p0 in enumerate(positions):
                for n in range(starts[b], starts[b + 1]):
                    p = p0 + n - starts[b]
                    blk = self.tables[b, p // self.bs]
                    self.codes[i][blk, :, p % self.bs] = c[n]
                    self.scales[i][blk, :, p % self.bs] = s[n]


def scales_kw(c):
    return dict(k_scale=c.S[0], v_scale=c.S[1])


def bound(q, k, v, scale):
    """One sequence's output and the bound of its error, [n_q][128], from q [n_q][128] and k, v
    [n][n_kv][128] in 64 bits.

    Score: 128 exact products added in fp32 (truncated at worst: 2^-23 a step, 2^-16 in all), a query
    element off by 2^-39 of the head's largest, four more roundings; the exponential's argument in
    log2 units by 2^-23 (|s| + |max| + 128) ln 2 more and the exponential itself by 2^-22.  A weight
    off by the factor exp(e) moves numerator and denominator by at most e^e - 1 of its share in each.
    The numerator's weight is an f16 number: 2^-11 of itself, and 2^-32 of the largest below its normal
    range.  Sums: fp32 steps, 2^-23 each, at most n / 8 of them in a lane's sum, 256 in merges.  The
    output is rounded to bf16, by 2^-8 of itself."""
    n_q, n, n_kv = q.shape[0], k.shape[0], k.shape[1]
    G = n_q // n_kv
    out, tol = np.zeros((n_q, D)), np.zeros((n_q, D))
    sums = (n / 8 + 256) * 2.0 ** -23
    for h in range(n_q):
        kh, vh = k[:, h // G], v[:, h // G]
        s = kh @ q[h] * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        e = scale * (2.0 ** -16 * (np.abs(kh) @ np.abs(q[h])) +
                     2.0 ** -39 * np.abs(q[h]).max() * np.abs(kh).sum(1))
        e += 2.0 ** -22 * np.abs(s) + 2.0 ** -23 * (np.abs(s) + np.abs(s).max() + 128) + 2.0 ** -22
        e = np.expm1(e)
        out[h] = w @ vh
        mag = w @ np.abs(vh)
        tol[h] = (w * (e + sums + 2.0 ** -11)) @ np.abs(vh) + (w @ e + sums) * mag
        tol[h] += 2.0 ** -32 * w.max() * np.abs(vh).sum(0)
        tol[h] = 1.01 * tol[h] + 2.0 ** -8 * np.abs(out[h]) + 2.0 ** -126
    return out, tol


def bounds_of(c, q, scale, ctx=None):
    got = [bound(bsc.f64(q[b]), c.rows(0, b, n), c.rows(1, b, n), scale)
           for b, n in enumerate(ctx or c.ctx)]
    return np.stack([x for x, _ in got]), np.stack([t for _, t in got])


def turned(x, positions, freq, first, interleaved, factor):
    """Rows [T][heads][d] (64 bits) with rotary dims turned, and the bound of a bf16 result's error.

    freq: the 2^-64 turns of every pair, taken modulo a turn in whole numbers.  The kernel's fraction
    of a turn is cut to 32 bits and rounded to fp32's 24, as is its angle (2^-22 radians), its sine
    and cosine are off by 2^-21.2, and three roundings of 2^-24 follow, so each of the two products by
    at most 2^-20 of |x| factor (2^-22 + 2^-21.2 + 3 * 2^-24 < 2^-20); then bf16: 2^-8 of the
    result."""
    half = len(freq)
    turn = np.array([[((int(p) * int(f)) % (1 << 64)) / 2.0 ** 64 for f in freq]
                     for p in positions]).reshape(len(positions), half)
    c, s = np.cos(2 * np.pi * turn)[:, None] * factor, np.sin(2 * np.pi * turn)[:, None] * factor
    i = np.arange(half)
    a, b = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + i + half)
    y, tol = x.copy(), np.zeros_like(x)
    u, w = x[..., a], x[..., b]
    y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    tol[..., a] = tol[..., b] = (np.abs(u) + np.abs(w)) * abs(factor) * 2.0 ** -20
    rot = np.zeros(x.shape[-1], bool)
    rot[a], rot[b] = True, True
    tol = np.where(rot, tol + 2.0 ** -8 * np.abs(y) + 2.0 ** -133, 0.0)
    return y, tol


class Tables:
    """The state of grow_tables and trim_tables on the host, one request after another."""

    def __init__(self, tables, ctx, refs, bs):
        self.tables, self.ctx = [list(map(int, r)) for r in tables], list(map(int, ctx))
        self.refs, self.bs = list(map(int, refs)), bs

    @property
    def NB(self):
        return len(self.refs)

    def bits(self):
        w = [0] * ((self.NB + 31) // 32)
        for i, r in enumerate(self.refs):
            if r == 0:
                w[i // 32] |= 1 << i % 32
        return [x - (1 << 32) if x >> 31 else x for x in w]

    def grow(self, new, N):
        """The outputs of grow_tables, as a dict of lists."""
        bs, B = self.bs, len(self.ctx)
        MB = len(self.tables[0]) if B else 1
        counts, copies, need = [], [], []
        for b in range(B):
            n, t = self.ctx[b], new[b]
            bad = n < 0 or t < 0 or n + t > MB * bs
            t = 0 if bad else t
            shared = False
            if t and n % bs:
                last = self.tables[b][n // bs]
                if not 0 <= last < self.NB:
                    t = 0
                else:
                    shared = self.refs[last] > 1
            counts.append(t)
            copies.append(shared)
            need.append((-(-(n + t) // bs) - -(-n // bs) if t else 0) + shared)
        free = [i for i, r in enumerate(self.refs) if r == 0]
        out = dict(positions=list(self.ctx), token_starts=[0] * (B + 1), slots=[-1] * N,
                   token_positions=[0] * N, copy_src=[-1] * B, copy_dst=[-1] * B)
        if sum(counts) > N or sum(need) > len(free):
            over = sum(counts) > N
            out["result"] = [2 if over else 1, 0, 0 if over else sum(need) - len(free), 0]
            return out
        at, n = 0, 0
        gone = []
        for b in range(B):
            p0, t = self.ctx[b], counts[b]
            j = -(-p0 // bs)
            out["token_starts"][b] = n
            if copies[b]:
                j -= 1
                out["copy_src"][b], out["copy_dst"][b] = self.tables[b][j], free[at]
                gone.append(self.tables[b][j])
            for i in range(need[b]):
                self.tables[b][j + i] = free[at]
                self.refs[free[at]] = 1
                at += 1
            for p in range(p0, p0 + t):
                out["slots"][n] = self.tables[b][p // bs] * bs + p % bs
                out["token_positions"][n] = p
                n += 1
            self.ctx[b] += t
        for i in gone:
            self.refs[i] -= 1
        out["token_starts"][B] = n
        out["result"] = [0, at, 0, n]
        return out

    def trim(self, keep):
        for b, k in enumerate(keep):
            n = self.ctx[b]
            if k < 0 or n < 0 or n > len(self.tables[b]) * self.bs or k >= n:
                continue
            for j in range(-(-k // self.bs), -(-n // self.bs)):
                i = self.tables[b][j]
                self.tables[b][j] = -1
                if 0 <= i < self.NB and self.refs[i] > 0:
                    self.refs[i] -= 1
            self.ctx[b] = k
