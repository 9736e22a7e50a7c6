"""Pins of the paged-cache oracle: rotations keep lengths and compose by angle, the norm is
scale-free, bounds bound, selections keep what they must, attention equals the dense form."""

import math

import numpy as np
import pytest

from oracle import paged as op
from oracle.attention import dense_causal_rows

D = 128


@pytest.mark.parametrize("rot,pairs", [(128, False), (64, False), (32, True), (16, True), (0, False)])
def test_rotation_keeps_lengths_and_leaves_the_rest(rot, pairs):
    rng = np.random.default_rng(rot)
    x = rng.standard_normal((3, 2, D))
    ang = op.rope_table(50, max(rot, 2))[[1, 7, 49]][:, :rot].astype(np.float64)
    y = op.norm_rope(x, None, 0.0, ang, rot, pairs)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-6)
    assert np.array_equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("pairs", [False, True])
def test_rotated_products_depend_on_the_distance_only(pairs):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, D)), rng.standard_normal((1, 1, D))
    inv = 1e4 ** (-np.arange(0, D, 2) / D)
    ang = lambda p: np.concatenate([np.cos(p * inv), np.sin(p * inv)])[None]
    dot = lambda a, b: float(np.sum(op.norm_rope(q, None, 0, ang(a), D, pairs) *
                                    op.norm_rope(k, None, 0, ang(b), D, pairs)))
    assert dot(9, 4) == pytest.approx(dot(1005, 1000), abs=1e-9)
    assert dot(9, 4) != pytest.approx(dot(9, 5), abs=1e-3)


def test_norm_is_scale_free_and_has_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((4, 1, D))
    y = op.norm_rope(x, np.ones(D), 0.0, np.zeros((4, 0)), 0, False)
    assert np.allclose(np.mean(y * y, axis=-1), 1.0)
    assert np.allclose(op.norm_rope(1e3 * x, np.ones(D), 0.0, np.zeros((4, 0)), 0, False), y)
    assert np.all(op.norm_rope(0 * x, np.ones(D), 1e-6, np.zeros((4, 0)), 0, False) == 0)


def test_page_bounds_bound_every_logit():
    rng = np.random.default_rng(3)
    k = rng.standard_normal((6, 16, D)).astype(np.float32).astype(np.float64)
    q = rng.standard_normal((3, D))
    u = op.page_bounds(q, k.min(1), k.max(1))
    logits = np.einsum("hd,prd->hpr", q, k)
    assert np.all(u >= logits.max(axis=(0, 2)) - 1e-5)
    same = np.repeat(k[:, :1], 16, axis=1)                    # equal rows: the bound is the logit
    assert np.allclose(op.page_bounds(q, same.min(1), same.max(1)),
                       np.einsum("hd,pd->hp", q, same[:, 0]).max(0), rtol=1e-6)


def test_select_pages_keeps_sink_recent_and_best():
    u = np.array([5, 1, 9, 9, 2, 9, 0], np.float32)
    score = lambda a, b: u[a - 1:b - 1]
    got = op.select_pages(pos=16 * 9 + 3, page=16, sink=1, local=2, top=2, score=score)
    assert got.tolist() == [0, 3, 4, 8, 9]                    # ties: pages 3 and 4 before 6
    assert op.select_pages(-1, 16, 1, 1, 1, score).size == 0
    assert op.select_pages(16 * 3, 16, 1, 2, 1, score).tolist() == [0, 1, 2, 3]
    assert op.select_pages(16 * 9, 16, 20, 1, 0, score).tolist() == list(range(10))


def test_attend_equals_dense_attention():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal((40, D)) for _ in range(3))
    ref, lref = dense_causal_rows(q, k, v, [0, 17, 39])
    for i, r in enumerate((0, 17, 39)):
        o, lse, w = op.attend(q[r], k[:r + 1], v[:r + 1], 1 / math.sqrt(D))
        assert np.allclose(o, ref[i]) and lse == pytest.approx(lref[i])
        assert np.all(w >= np.abs(o) - 1e-12)
    o, lse, _ = op.attend(q[0], k[:0], v[:0], 1.0)
    assert lse == -math.inf and np.all(o == 0)


def test_sequence_rows_follow_the_table():
    cache = np.arange(5 * 2 * 4 * D, dtype=np.float64).reshape(5, 2, 4, D)
    rows = op.sequence_rows(cache, [3, 1], 1, 6)
    assert np.array_equal(rows[:4], cache[3, 1]) and np.array_equal(rows[4:], cache[1, 1, :2])
