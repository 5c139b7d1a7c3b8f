"""Pins of the conditioning oracle: closed forms and identities that need no other code."""
import numpy as np
import pytest

import oracle


def test_norm_is_unit_rms_and_matches_the_relayout_norm():
    x = np.random.default_rng(1).normal(size=(5, 3, 24))
    y = oracle.qk_norm_rope(x, eps=0.0)
    assert np.allclose(np.mean(y * y, -1), 1.0)
    g = np.linspace(0.5, 1.5, 24)
    assert np.allclose(oracle.qk_norm_rope(x, g, 1e-3).reshape(5, -1),
                       oracle.rmsnorm_heads(x.reshape(5, -1), g, 24, 1e-3))


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_rotation_is_a_complex_product_and_keeps_lengths(pairing):
    rng = np.random.default_rng(2)
    D, n = 16, 7
    x = rng.normal(size=(n, 2, D))
    table = oracle.rope_table(n, D)
    pos = np.array([0, 3, 6, 1, 1, -1, n])
    y0 = oracle.qk_norm_rope(x, eps=0.0)
    y = oracle.qk_norm_rope(x, eps=0.0, table=table, pos=pos, pairing=pairing)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(y0, axis=-1))
    assert np.array_equal(y[[0, 5, 6]], y0[[0, 5, 6]])          # position 0, and positions outside the table
    pair = (lambda z: z[..., 0::2] + 1j * z[..., 1::2]) if pairing == "interleaved" else (
        lambda z: z[..., :D // 2] + 1j * z[..., D // 2:])
    w = table[pos[1], :, 0] + 1j * table[pos[1], :, 1]
    assert np.allclose(pair(y[1]), pair(y0[1]) * w)


def test_interleaved_rotation_matches_the_relayout_rotation():
    x = np.random.default_rng(3).normal(size=(6, 2, 8))
    y = oracle.qk_norm_rope(x, eps=0.0, table=oracle.rope_table(6, 8), pos=np.arange(6))
    ref = oracle.rope_heads(oracle.qk_norm_rope(x, eps=0.0).reshape(6, -1), np.arange(6), 8)
    assert np.allclose(y.reshape(6, -1), np.asarray(ref).reshape(6, -1))


def _kv(rng, l, h, d):
    return rng.normal(size=(l, h, d)), rng.normal(size=(l, h, d))


def test_no_key_one_key_and_equal_keys():
    rng = np.random.default_rng(4)
    q = rng.normal(size=(1, 2, 3, 2, 4))
    o, lse, _ = oracle.conditioned(q, [[_kv(rng, 0, 2, 4)]])
    assert not o.any() and np.all(lse == -np.inf)
    k, v = _kv(rng, 1, 2, 4)
    o, lse, _ = oracle.conditioned(q, [[(k, v)]])
    assert np.allclose(o, v[0]) and np.allclose(lse[0, 1, 0, 2], q[0, 1, 2, 0] @ k[0, 0] / 2)
    v = rng.normal(size=(5, 2, 4))
    o, _, _ = oracle.conditioned(q, [[(np.repeat(k, 5, 0), v)]])
    assert np.allclose(o, v.mean(0))


def test_segments_are_one_sequence_and_their_merge():
    rng = np.random.default_rng(5)
    q = rng.normal(size=(2, 1, 3, 4, 8))
    a, b = _kv(rng, 6, 2, 8), [_kv(rng, 5, 2, 8), _kv(rng, 2, 2, 8)]
    o, lse, _ = oracle.conditioned(q, [[a], b])
    for i in range(2):
        whole = (np.concatenate((a[0], b[i][0])), np.concatenate((a[1], b[i][1])))
        o1, l1, _ = oracle.conditioned(q[i:i + 1], [[whole]])
        assert np.allclose(o[i], o1[0]) and np.allclose(lse[i], l1[0])
    oa, la, _ = oracle.conditioned(q, [[a]])
    ob, lb, _ = oracle.conditioned(q, [b])
    m = np.logaddexp(la, lb)
    wa, wb = (np.exp(x - m).transpose(0, 1, 3, 2)[..., None] for x in (la, lb))
    assert np.allclose(m, lse) and np.allclose(wa * oa + wb * ob, o)


def test_sets_and_grouped_heads():
    rng = np.random.default_rng(6)
    q = rng.normal(size=(4, 1, 2, 6, 8))
    sets = [_kv(rng, 3, 2, 8), _kv(rng, 4, 2, 8)]
    o, _, _ = oracle.conditioned(q, [sets])
    one, _, _ = oracle.conditioned(q[3:, :, :, 5:], [[tuple(x[:, 1:] for x in sets[1])]])
    assert np.allclose(o[3, 0, :, 5], one[0, 0, :, 0])
