"""The bound of attention_error.py without a GPU: outputs computed as the header states stay within
it, outputs with a part of that arithmetic left out do not."""
import numpy as np
import pytest

import attention_error as ae
import block_scaled as bsc

SCALE = 128 ** -0.5


def _attend(c, q, scale, terms, split=True):
    """Outputs with weights in `terms` E4M3 terms and queries in two (split) or one, the rest in 64
    bits."""
    out = np.zeros(q.shape)
    G = q.shape[1] // c.n_kv
    for b, n in enumerate(c.ctx):
        x = bsc.f64(q[b])
        if split:
            x = ae.split_query(x)
        else:
            s = np.exp2(np.floor(np.log2(np.abs(x).max(-1, keepdims=True))) - 7)
            x = bsc.VALUES[bsc.e4m3_codes(x / s)] * s
        k, v, sv = c.rows("k", b, n), c.rows("v", b, n), ae.v_scales(c, b, n)
        for h in range(q.shape[1]):
            s = k[:, h // G] @ x[h] * scale
            p = np.exp(s - s.max())
            ref = (p * sv[:, h // G]).max()
            w = 16 * p * sv[:, h // G] / ref
            w = w if terms is None else ae.weight_terms(w, terms)
            out[b, h] = w @ (v[:, h // G] / sv[:, h // G, None]) / 16 * ref / p.sum()
    return out


@pytest.mark.parametrize("bs", [16, 32])
def test_cancelling_outputs_show_the_third_term(bs):
    c, q = ae.cancelling_cache(24, 4, 1, bs, 5, SCALE)
    out, tol = ae.bounds_of(c, q, SCALE, False)
    ae.check(_attend(c, q, SCALE, 3), out, tol)
    with pytest.raises(AssertionError, match="of its bound"):
        ae.check(_attend(c, q, SCALE, 2), out, tol)
    # the bound of fp32 weights
    out, tol = ae.bounds_of(c, q, SCALE, True)
    ae.check(_attend(c, q, SCALE, None), out, tol)
    with pytest.raises(AssertionError, match="of its bound"):
        ae.check(_attend(c, q, SCALE, 2), out, tol)


def test_ordinary_outputs_show_a_query_in_one_term():
    c = bsc.make_cache([300, 40], 2, 16, seed=3)
    q = bsc.make_query(2, 8)
    out, tol = ae.bounds_of(c, q, SCALE, False)
    ae.check(_attend(c, q, SCALE, 3), out, tol)
    with pytest.raises(AssertionError, match="of its bound"):
        ae.check(_attend(c, q, SCALE, 3, split=False), out, tol)
