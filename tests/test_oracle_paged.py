"""Pins for the paged-cache oracle: results from outside its own formulas."""

import math
import random

import numpy as np
import pytest

import oracle.decode_oracle as dec
import oracle.paged_oracle as pg
from helpers import ensure_built


def test_attention_of_shuffled_pages_is_the_decode_oracles():
    rng = np.random.default_rng(1)
    L, S, H, Hkv, D, ps = 2, 3, 4, 2, 8, 4
    lens, W, P = [9, 0, 4], 3, 9
    K, V = rng.standard_normal((2, L, P, ps, Hkv, D))
    q = rng.standard_normal((L, S, H, D))
    table = rng.permutation(P).reshape(S, W)
    out, lse, ob, lb = pg.attention(q, K, V, table, lens)
    for l in range(L):
        for b in range(S):
            for h in range(H):
                if lens[b] == 0:
                    assert not out[l, b, h].any() and lse[l, b, h] == -math.inf
                    continue
                k = np.array([K[l, table[b, j // ps], j % ps, h // 2] for j in range(lens[b])])
                v = np.array([V[l, table[b, j // ps], j % ps, h // 2] for j in range(lens[b])])
                o, z = dec.decode_attention(q[l, b, h], k, v)
                np.testing.assert_allclose(out[l, b, h], o, rtol=1e-12, atol=1e-12)
                assert lse[l, b, h] == pytest.approx(z, abs=1e-12)
                assert (ob[l, b, h] > 0).all() and lb[l, b, h] > 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_laws(interleaved):
    """Lengths stay, rotating by a then b is rotating by a + b, the dot product of two rotated
    rows depends on the difference of their angles alone."""
    rng = np.random.default_rng(2)
    x, y = rng.standard_normal((2, 1, 1, 12))
    a, b = rng.standard_normal((2, 1, 4))
    r = lambda z, t: pg.rotate(z, t, interleaved)  # noqa: E731
    np.testing.assert_allclose(np.linalg.norm(r(x, a)), np.linalg.norm(x), rtol=1e-13)
    np.testing.assert_allclose(r(r(x, a), b), r(x, a + b), atol=1e-13)
    np.testing.assert_allclose((r(x, a) * r(y, b)).sum(), (r(x, a - b) * y).sum(), atol=1e-12)
    np.testing.assert_array_equal(r(x, a)[..., 8:], x[..., 8:])
    quarter = pg.rotate(np.arange(4.0).reshape(1, 1, 4), np.full((1, 2), math.pi / 2), interleaved, 2.0)
    want = [-2, 0, -6, 4] if interleaved else [-4, -6, 0, 2]
    np.testing.assert_allclose(quarter[0, 0], want, atol=1e-12)


def test_norm_has_unit_mean_square():
    x = np.array([[3.0, 4.0]])
    np.testing.assert_allclose(pg.norm(x, np.ones(2), 0.0), x / math.sqrt(12.5))
    assert pg.norm(np.zeros((1, 4)), np.ones(4), 1e-6).any() == False  # noqa: E712


def test_compact_keeps_the_set_and_moves_the_least():
    assert pg.compact([5, 0, 7, 2], 8) == [0, 5, 2, 7]
    assert pg.compact([1, 0, 2], 3) == [0, 1, 2]
    rng = random.Random(3)
    for _ in range(50):
        length = rng.randrange(1, 40)
        want = rng.sample(range(length), rng.randrange(0, length + 1))
        got = pg.compact(want, length)
        assert sorted(got) == sorted(want)
        assert sum(s != j for s, j in enumerate(got)) == sum(j >= len(want) for j in want)
    with pytest.raises(ValueError):
        pg.compact([1, 1], 4)


def test_update_by_row_replay():
    """Random steps against a model of rows alone: every sequence reads its own rows through
    its table, references count the holders, and no row of another sequence is overwritten."""
    rng = random.Random(4)
    ps, P, W = 4, 60, 8
    store = {}                       # (page, slot) -> value
    rows, table, lens = [[]], [[-1] * W], [0]
    tag = 0
    for step in range(120):
        n_out = rng.randrange(1, 6)
        parents = [rng.randrange(-1, len(rows)) for _ in range(n_out)]
        new = [rng.randrange(0, min(W * ps, (len(rows[p]) if p >= 0 else 0) + 6) + 1) for p in parents]
        t2, ref, free, copies = pg.update(table, lens, parents, new, P, ps)
        assert free >= 0
        for src, dst, n in copies:
            for r in range(n):
                store[dst, r] = store[src, r]
        held = [x for t in t2 for x in t if x >= 0]
        assert [held.count(x) for x in range(P)] == ref and free == ref.count(0)
        rows = [(rows[p][:n] if p >= 0 else []) for p, n in zip(parents, new)]
        for b in range(n_out):
            assert [x >= 0 for x in t2[b]] == [i < -(-new[b] // ps) for i in range(W)]
            for j in range(len(rows[b]), new[b]):            # the step's new rows
                tag += 1
                rows[b].append(tag)
                store[t2[b][j // ps], j % ps] = tag
        table, lens = t2, new
        for b in range(n_out):
            assert [store[table[b][j // ps], j % ps] for j in range(lens[b])] == rows[b]


def test_update_hands_out_the_lowest_pages_and_reports_a_shortfall():
    out, ref, free, copies = pg.update([[3, 1]], [6], [0, 0], [7, 6], 5, 4)
    assert out == [[3, 1], [3, 0]] and ref == [1, 1, 0, 2, 0] and free == 2
    assert copies == [(1, 0, 2)]
    out, ref, free, _ = pg.update([[0, -1]], [4], None, [8], 1, 4)
    assert out == [[0, -1]] and free == -1


def test_rope_frequencies():
    ensure_built()
    from kv_cache_eviction_snapkv_gb300 import api
    i = np.arange(32)
    plain, one = api.kvsel_rope_frequencies(64, 10000.0)
    want = 10000.0 ** (-i / 32)
    np.testing.assert_allclose(plain.numpy(), want, rtol=2 ** -24)
    assert one == 1.0
    lin, _ = api.kvsel_rope_frequencies(64, 10000.0, api.KVSEL_ROPE_LINEAR, 4.0)
    np.testing.assert_allclose(lin.numpy(), want / 4, rtol=2 ** -24)
    # the changed base stretches the slowest pair by the whole factor, the fastest not at all
    base, _ = api.kvsel_rope_frequencies(64, 10000.0, api.KVSEL_ROPE_BASE, 8.0)
    assert base[0] == 1.0
    assert float(base[-1]) == pytest.approx(want[-1] / 8, rel=1e-6)
    parts, s = api.kvsel_rope_frequencies(64, 10000.0, api.KVSEL_ROPE_PARTS, 8.0, 4096, 1.0, 32.0)
    turns = 4096 * want / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    np.testing.assert_allclose(parts.numpy(), want * keep + want / 8 * (1 - keep), rtol=2 ** -23)
    assert s == pytest.approx(1 + 0.1 * math.log(8), rel=1e-6)
    assert keep.min() == 0 and keep.max() == 1
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(base=1.0), dict(factor=0.5), dict(kind=4),
                dict(kind=2, rot_dim=2), dict(kind=3, original_len=0), dict(kind=3, low=2.0, high=1.0),
                dict(base=float("nan"))):
        with pytest.raises(api.KvselError) as e:
            api.kvsel_rope_frequencies(**{"rot_dim": 64, "original_len": 4096, **bad})
        assert e.value.status == api.KVSEL_ERR_INVALID_ARG
