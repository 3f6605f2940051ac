"""Pins of oracle/scored.py (CPU): torch's attention with explicit masks, the
plain and verify references, closed forms of the cap and the bias, and a tree
whose masks form a chain."""
import math

import numpy as np
import pytest

from oracle import ckv_oracle as O
from oracle import scored as S

torch = pytest.importorskip("torch")


def _qkv(n, H, Hkv, T, D, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((n, H, D)), r.standard_normal((Hkv, T, D)), r.standard_normal((Hkv, T, D))


@pytest.mark.parametrize("window,prefix,docs", [(0, 0, False), (5, 0, False), (0, 20, False), (0, 0, True), (7, 18, True)])
def test_causal_rows_match_sdpa(window, prefix, docs):
    n, H, Hkv, T, D = 9, 4, 2, 23, 8
    q, k, v = _qkv(n, H, Hkv, T, D)
    doc = (np.arange(T - n, T) // 6) * 6 if docs else None
    at, key_at, see = S.causal_rows(T, n, window, prefix, doc)
    for i in range(n):  # the definition, key by key
        for p in range(T):
            want = (p <= T - n + i or p < prefix) and (not window or T - n + i - p < window)
            want = want and (doc is None or p >= doc[i])
            assert see[i, p] == want
    o, lse = S.scored_attention(q, k, v, at, key_at, see, 0.3)
    kk, vv = (torch.from_numpy(np.repeat(x, H // Hkv, 0)) for x in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), kk, vv, attn_mask=torch.from_numpy(see), scale=0.3).transpose(0, 1)
    assert np.allclose(o, ref.numpy(), atol=1e-12)


def test_unmasked_rows_are_the_verify_reference():
    n, H, Hkv, T, D = 5, 6, 3, 17, 8
    q, k, v = _qkv(n, H, Hkv, T, D, 1)
    o, lse = S.scored_attention(q, k, v, *S.causal_rows(T, n), 0.5)
    ro, rl = O.verify_decode_reference(q, k, v, T, 0.5)
    assert np.allclose(o, ro, atol=1e-12) and np.allclose(lse, rl, atol=1e-12)


def test_cap_and_bias_closed_forms():
    # One key: o = v, lse = the logit itself.
    q, k = np.full((1, 1, 4), 3.0), np.full((1, 1, 4), 2.0)
    at, key_at, see = S.causal_rows(1, 1)
    _, lse = S.scored_attention(q, k, k, at, key_at, see, 1.0, softcap=10.0)
    assert lse[0, 0] == pytest.approx(10.0 * math.tanh(2.4), abs=1e-14)
    # Equal logits: the weights of distances 0, 1, 2 are 1, e^-s, e^-2s.
    z, v = np.zeros((1, 3, 4)), np.eye(4)[None, :3]
    o, _ = S.scored_attention(np.zeros((1, 1, 4)), z, v, *S.causal_rows(3, 1), 1.0, slopes=[0.7])
    w = np.exp(-0.7 * np.array([2, 1, 0]))
    assert np.allclose(o[0, 0, :3], w / w.sum(), atol=1e-15)


def test_a_chain_is_a_verify_batch_and_siblings_do_not_meet():
    n, H, Hkv, T, D = 6, 2, 1, 15, 8
    q, k, v = _qkv(n, H, Hkv, T, D, 2)
    chain = [(1 << (i + 1)) - 1 for i in range(n)]
    for w in (0, 4):
        a, b = S.tree_rows(T, chain, w), S.causal_rows(T, n, w)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1]) and np.array_equal(a[2], b[2])
    at, key_at, see = S.tree_rows(T, [1, 3, 5], 0)  # two children of node 0: both at depth 1
    assert list(at - (T - 3)) == [0, 1, 1] and list(key_at[-3:]) == list(at)
    assert not see[2, T - 2] and see[2, T - 3] and see[2, T - 1]
    o, lse = S.scored_attention(q[:1], k[:, :1], v[:, :1], *S.tree_rows(1, [0]), 1.0)
    assert np.all(o == 0) and np.all(np.isneginf(lse))


def test_accepted_positions():
    assert list(S.accepted_positions(8, 4, [0, 3])) == [0, 1, 2, 3, 4, 7, 6, 7]
    assert list(S.accepted_positions(5, 3, [2, 1, 2])) == [0, 1, 4, 3, 4]
