"""Pins of the oracle's packed-prompt attention and of the quantised values
it is given: torch's causal SDPA, the multi-query oracle, closed forms."""

import numpy as np
import pytest
import torch

from oracle import attention, kvcache


@pytest.mark.parametrize("lens,prefix", [([5, 1, 9], [0, 0, 0]), ([3, 0, 7], [4, 2, 0])])
def test_equals_sdpa_and_the_multi_query_oracle(lens, prefix):
    rng = np.random.default_rng(7)
    Hq, Hkv, D = 6, 2, 16
    kv = [a + b for a, b in zip(lens, prefix)]
    qs, ks = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(kv)])
    q, k, v = (rng.standard_normal((n, h, D)) for n, h in ((qs[-1], Hq), (ks[-1], Hkv), (ks[-1], Hkv)))
    out, out_abs = attention.prompt_attention(q, k, v, qs, 0.3, ks)
    for b, (n, m) in enumerate(zip(lens, kv)):
        if n == 0:
            continue
        qb, kb, vb = q[qs[b]:qs[b + 1]], k[ks[b]:ks[b + 1]], v[ks[b]:ks[b + 1]]
        want = attention.multi_query_attention(qb, kb, vb, 0.3)
        np.testing.assert_allclose(out[qs[b]:qs[b + 1]], want, rtol=1e-12, atol=1e-13)
        t = [torch.from_numpy(x).transpose(0, 1) for x in (qb, kb, vb)]
        mask = torch.ones(n, m, dtype=torch.bool).tril(m - n)
        ref = torch.nn.functional.scaled_dot_product_attention(t[0], t[1], t[2], attn_mask=mask, scale=0.3,
                                                               enable_gqa=True)
        np.testing.assert_allclose(out[qs[b]:qs[b + 1]], ref.transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)
        want_abs = attention.multi_query_attention(qb, kb, np.abs(vb), 0.3)
        np.testing.assert_allclose(out_abs[qs[b]:qs[b + 1]], want_abs, rtol=1e-12)


def test_closed_forms():
    v = np.arange(12.0).reshape(4, 1, 3)
    q, k = np.zeros((4, 1, 3)), np.ones((4, 1, 3))
    out, _ = attention.prompt_attention(q, k, v, [0, 4], 1.0)
    np.testing.assert_allclose(out[:, 0], np.cumsum(v[:, 0], axis=0) / np.arange(1, 5)[:, None])
    # more queries than rows: the first ones sit before the first row
    out, _ = attention.prompt_attention(q, k[:2], v[:2], [0, 4], 1.0, [0, 2])
    assert (out[:2] == 0).all() and (out[2] == v[0]).all()
    # rows of no sequence
    out, _ = attention.prompt_attention(q, k, v, [1, 3], 1.0)
    assert (out[0] == 0).all() and (out[3] == 0).all() and (out[1] == v[1]).all()


@pytest.mark.parametrize("qmode,window", [("int4", 0), ("int4", 16), ("fp8", 32)])
def test_sequence_values_are_what_decode_attends_to(qmode, window):
    rng = np.random.default_rng(3)
    k, v = (rng.standard_normal((50, 2, 64)).astype(np.float32) for _ in range(2))
    q = rng.standard_normal((4, 64))
    kd, vd = (kvcache.sequence_values(x, 4, qmode, 64, window) for x in (k, v))
    want = kvcache.sequence_attention_quant(q, k, v, 0.125, 4, qmode, 64, window)
    np.testing.assert_allclose(attention.sequence_attention(q, kd, vd, 0.125), want, rtol=1e-12)
    np.testing.assert_allclose(attention.prompt_attention(q[None], kd, vd, [0, 1], 0.125, [0, 50])[0][0], want,
                               rtol=1e-10)
