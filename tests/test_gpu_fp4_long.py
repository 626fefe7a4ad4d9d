"""The 4-bit attention next to the largest B * n_kv * MB * bs (2^35), with values that tell which tokens
were read: what a part, a boundary between parts or a merge weight left out would change."""
import numpy as np
import pytest
import torch

import block_scaled as bsc
import fp4
import paged_gqa_decode_kv_gb300 as pgd

pytestmark = pytest.mark.gpu


def test_every_part_of_the_longest_contexts_counts():
    """Equal weights (all keys 0).  Dim r < 64 of a value is 1 in the r-th 64th of a context and 0
    elsewhere; dims from 64 on belong to one block each: the ends, the places where 6, 7 or 8 equal parts
    meet, and others, each with 2688 in its dim."""
    n_kv, bs, MB, runs = 4, 32, (1 << 22) + 1, 64
    B = (1 << 30) // (n_kv * MB)
    c = fp4.Cache([2 * runs * bs], n_kv, bs, S=(1.0, 1.0))
    ids = c.tables[0, :2 * runs]
    one, most = 0x38, 0x7E  # scales 1 and 448
    c.codes[0][:], c.scales[0][:] = 0, one
    c.codes[1][:], c.scales[1][:] = 0, one
    for d, i in enumerate(ids):
        c.codes[1][i, :, :, d] = 2 if d < runs else 7  # 1, 6
        if d >= runs:
            c.scales[1][i] = most
    assert c.rows(1, 0, 33).max() == 1 and c.rows(1, 0, 65 * 32)[-1].max() == 2688
    row = ids[np.arange(MB) * runs // MB]
    cuts = {n: [p * (MB // n) + min(p, MB % n) for p in range(n + 1)] for n in (6, 7, 8)}
    at = {0, MB - 1} | {i - d for cut in cuts.values() for i in cut[1:-1] for d in (0, 1)}
    r = np.random.default_rng(5)
    while len(at) < runs:
        at.add(int(r.integers(MB)))
    at = sorted(at)
    row[at] = ids[runs:]
    k, v, _, _ = c.cuda()
    q = bsc.make_query(B, n_kv).cuda()
    table = torch.from_numpy(row.astype(np.int32)).cuda().repeat(B, 1)
    lens = torch.full((B,), MB * bs, dtype=torch.int32, device="cuda")
    got = bsc.f64(pgd.paged_decode_attention_fp4(None, q, k, v, table, lens, 128 ** -0.5))
    assert pgd.device_errors(clear=True) == 0

    def mean(row):
        return np.where(np.arange(128) < runs, 1.0, 2688.0) * np.bincount(
            row, minlength=c.NB)[ids] / len(row)

    want = mean(row)
    # A warp takes at most 2^30 steps over 4 * 608 warps that run at once; a lane's sum has 4 terms a
    # step, each rounded (2^-24), an output 2 products, each cut (2^-23); a thousand roundings more in
    # merges, then bf16 (2^-8).
    steps = 2 ** 30 / (4 * 608)
    tol = (steps * (4 * 2.0 ** -24 + 2 * 2.0 ** -23) + 2.0 ** -14 + 2.0 ** -8) * want
    assert (want > 0).all() and (tol < 0.22 * want).all()
    # (a part or a block at its end left out, or read twice, would be seen)
    for cut in cuts.values():
        for i, j in zip(cut, cut[1:]):
            assert (np.abs(mean(np.delete(row, slice(i, j))) - want) > tol).any()
            for one_block in (i, j - 1):
                for other in (np.delete(row, one_block), np.append(row, row[one_block])):
                    assert (np.abs(mean(other) - want) > tol).any()
    err = np.abs(got - want)
    assert (err <= tol).all(), (err / want).max()
