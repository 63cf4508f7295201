"""Pins of the oracle's head norms with rotation, paged append and attention over a cache:
closed forms, differences of the forward pass, invariances and the oracle's own
self-attention on the same tokens."""
import numpy as np
import pytest

from oracle import dark_oracle as O

LAYOUTS = [(0, False), (4, False), (8, False), (8, True), (6, True)]


def _x(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("dims,inter", LAYOUTS)
def test_rotation_keeps_lengths_and_depends_on_distance(dims, inter):
    q, k = _x(1, 1, 2, 1, 8), _x(2, 1, 2, 1, 8)
    at = lambda x, p: O.rotate(x, np.array([[p]]), dims, interleaved=inter)
    np.testing.assert_allclose((at(q, 71) ** 2).sum(-1), (q ** 2).sum(-1), rtol=1e-12)
    np.testing.assert_allclose((at(q, 71) * at(k, 60)).sum(-1), (at(q, 11) * at(k, 0)).sum(-1),
                               rtol=1e-10)
    np.testing.assert_array_equal(at(q, 5)[..., dims:], q[..., dims:])
    np.testing.assert_allclose(O.rotate(at(q, 9), np.array([[9]]), dims, interleaved=inter,
                                        transpose=True), q, rtol=1e-12)


def test_rotation_worked_example():
    # position 2, base 100, dims 4: frequencies 1 and 100^(-1/2) = 0.1
    x = np.array([1.0, 0.0, 0.0, 1.0, 7.0]).reshape(1, 1, 1, 5)
    got = O.rotate(x, np.array([[2]]), 4, base=100.0)[0, 0, 0]
    # pairs (0, 2) = (1, 0) by 2 rad and (1, 3) = (0, 1) by 0.2 rad
    np.testing.assert_allclose(got, [np.cos(2), -np.sin(0.2), np.sin(2), np.cos(0.2), 7.0])
    got = O.rotate(x, np.array([[2]]), 4, base=100.0, interleaved=True)[0, 0, 0]
    np.testing.assert_allclose(got, [np.cos(2), np.sin(2), -np.sin(0.2), np.cos(0.2), 7.0])


@pytest.mark.parametrize("dims,inter", LAYOUTS)
@pytest.mark.parametrize("gheads", [0, 1, 3])
def test_backward_against_differences(dims, inter, gheads):
    x, dy = _x(3, 2, 3, 2, 8), _x(4, 2, 3, 2, 8)
    gamma = None if gheads == 0 else 1.0 + 0.3 * _x(5, gheads, 8)
    pos = np.array([[3, 11], [0, 200]])
    f = lambda x_, g_: (dy * O.norm_rope(x_, g_, 1e-3, pos, dims, interleaved=inter)).sum()
    dx, dg = O.norm_rope_backward(x, gamma, 1e-3, pos, dy, dims, interleaved=inter)
    h = 1e-6
    for idx in [(0, 0, 0, 0), (1, 2, 1, 7), (0, 1, 1, 3), (1, 0, 0, 5)]:
        e = np.zeros_like(x)
        e[idx] = h
        assert abs((f(x + e, gamma) - f(x - e, gamma)) / (2 * h) - dx[idx]) < 1e-7
    if gamma is not None:
        assert dg.shape == gamma.shape
        for idx in [(0, 0), (gheads - 1, 6)]:
            e = np.zeros_like(gamma)
            e[idx] = h
            assert abs((f(x, gamma + e) - f(x, gamma - e)) / (2 * h) - dg[idx]) < 1e-7


def _cache(seed, B, Hk, page, d, lens, prefix):
    rng = np.random.default_rng(seed)
    per = max(1, -(-max(lens) // page))
    shared = -(-prefix // page)
    n = B * per + shared + 1
    order = rng.permutation(n)
    pools = [rng.standard_normal((n, Hk, page, d)) for _ in range(2)]
    return pools, order[:B * per].reshape(B, per), order[B * per:B * per + shared]


def test_append_then_read_back():
    pools, table, _ = _cache(6, 2, 3, 4, 8, [11, 11], 0)
    k, v = _x(7, 2, 3, 6, 8), _x(8, 2, 3, 6, 8)
    lens, new = [5, 0], [6, 3]
    kp, vp = O.kv_append(*pools, k, v, table, lens, new)
    for b in range(2):
        for h in range(3):
            rows = O.cache_rows(kp, table[b], lens[b] + new[b], h)
            np.testing.assert_array_equal(rows[lens[b]:], k[b, h, :new[b]])
            np.testing.assert_array_equal(rows[:lens[b]],
                                          O.cache_rows(pools[0], table[b], lens[b], h))
    # rows behind the last token stay
    assert (kp != pools[0]).any(axis=(1, 3)).sum() == sum(new)
    assert (vp != pools[1]).any(axis=(1, 3)).sum() == sum(new)


@pytest.mark.parametrize("prefix", [0, 5])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_over_the_cache_is_attention_over_its_tokens(prefix, causal):
    B, H, Hk, d, T = 2, 4, 2, 8, 3
    lens = [7, 3]
    (kp, vp), table, shared = _cache(9, B, Hk, 4, d, lens, prefix)
    geom = np.eye(6, d)[None] + 0.3 * _x(10, H, 6, d)
    q = _x(11, B, H, T, d)
    got = O.cache_attention(q, kp, vp, geom, table, lens, shared, prefix, causal)
    for b in range(B):
        full = [np.stack([np.concatenate([O.cache_rows(x, shared, prefix, h // 2),
                                          O.cache_rows(x, table[b], lens[b], h // 2)])
                          for h in range(H)])[None] for x in (kp, vp)]
        n = prefix + lens[b]
        if causal:                    # the queries are the last T tokens of n
            qq = np.concatenate([np.zeros((1, H, n - T, d)), q[b:b + 1]], axis=2)
            ref = O.exact_attention(qq, *full, geom, causal=True)[:, :, n - T:]
        else:
            ref = O.exact_attention(q[b:b + 1], *full, geom)
        np.testing.assert_allclose(got[b:b + 1], ref, rtol=1e-11, atol=1e-12)


def test_queries_that_see_nothing_are_zero():
    (kp, vp), table, shared = _cache(12, 2, 1, 4, 4, [0, 2], 0)
    q = _x(13, 2, 1, 4, 4)
    geom = np.eye(4)[None]
    out = O.cache_attention(q, kp, vp, geom, table, [0, 2])
    assert np.all(out[0] == 0) and np.all(out[1] != 0)
    # causal: the first T - lens queries are padding, with a prefix too
    (kp, vp), table, shared = _cache(14, 2, 1, 4, 4, [0, 2], 3)
    out = O.cache_attention(q, kp, vp, geom, table, [0, 2], shared, 3, causal=True)
    assert np.all(out[0] == 0) and np.all(out[1, :, :2] == 0) and np.all(out[1, :, 2:] != 0)
