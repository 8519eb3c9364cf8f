"""Pins of oracle.operators: hand-worked examples and independent recomputations (CPU)."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import operators as op

SIG = dict(sigmoid=True, n_groups=1, topk_groups=1, group_best=1, renormalise=True, weight_scale=1.0)


def test_norm_worked_example():
    # s = (3, -4) + (0, 8) = (3, 4): mean square 12.5, y = s / sqrt(12.5) * (1, 2)
    s, y, scale = op.add_rmsnorm([[3.0, -4.0]], [[0.0, 8.0]], [1.0, 2.0], 0.0)
    assert s.tolist() == [[3.0, 4.0]]
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]], rtol=1e-15)
    assert np.allclose(scale, [8 / math.sqrt(12.5) / 448], rtol=1e-15)
    s, y, scale = op.add_rmsnorm([[0.0, 0.0]], None, [1.0, 2.0], 1e-6)
    assert y.tolist() == [[0.0, 0.0]] and scale.tolist() == [1.0]


def test_norm_against_torch():
    x = np.random.default_rng(0).normal(size=(5, 33))
    y = op.add_rmsnorm(x, None, np.ones(33), 1e-5)[1]
    assert np.allclose(y, torch.nn.functional.rms_norm(torch.from_numpy(x), (33,), eps=1e-5).numpy(), rtol=1e-12)


def test_select_worked_example():
    # sigmoid(0) = 1/2, sigmoid(ln 3) = 3/4, sigmoid(-ln 3) = 1/4
    l = [0.0, math.log(3), -math.log(3), 0.0]
    idx, w, _ = op.select_token(l, None, 2, **SIG)
    assert idx == [1, 0] and np.allclose(w, [0.6, 0.4])
    # the bias takes expert 2 ahead (1/4 + 0.6) but its weight is its own score
    idx, w, _ = op.select_token(l, [0, 0, 0.6, 0], 2, **{**SIG, "weight_scale": 2.0})
    assert idx == [2, 1] and np.allclose(w, [2 * 0.25, 2 * 0.75])
    # two groups {0, 1}, {2, 3}: by the best one the first stays, by the best two with the bias the second
    two = dict(SIG, n_groups=2, topk_groups=1)
    assert op.select_token(l, None, 2, **two)[0] == [1, 0]
    assert op.select_token(l, [0, 0, 0.3, 0.3], 2, **{**two, "group_best": 2})[0] == [3, 2]


def test_select_softmax_matches_torch_topk():
    l = np.random.default_rng(1).normal(size=(50, 24))
    idx, w = op.select_experts(l, None, 5, **{**SIG, "sigmoid": False, "renormalise": False})
    p, i = torch.softmax(torch.from_numpy(l), 1).topk(5)
    assert np.array_equal(idx, i.numpy()) and np.allclose(w, p.numpy(), rtol=1e-12)


def test_select_groups_against_every_subset():
    rng = np.random.default_rng(2)
    for _ in range(20):
        l, b = rng.normal(size=12), 0.1 * rng.normal(size=12)
        r = dict(SIG, n_groups=4, topk_groups=2, group_best=2)
        idx, w, c = op.select_token(l, b, 3, **r)
        s = 1 / (1 + np.exp(-l)) + b
        worth = lambda g: np.sort(s[3 * g:3 * g + 3])[-2:].sum()                       # noqa: E731
        pair = max(itertools.combinations(range(4), 2), key=lambda p: sum(map(worth, p)))
        allowed = [e for e in range(12) if e // 3 in pair]
        best = max(itertools.combinations(allowed, 3), key=lambda p: s[list(p)].sum())
        assert sorted(idx) == sorted(best) and s[idx[0]] >= s[idx[1]] >= s[idx[2]]


def test_select_out_of_service_and_ties():
    r = dict(SIG, sigmoid=False)
    assert op.select_token([1.0] * 4, None, 2, **r)[:2] == ([0, 1], [0.5, 0.5])
    assert op.select_token([-math.inf, math.nan, 2.0, -math.inf], None, 2, **r)[:2] == ([2, -1], [1.0, 0.0])
    assert op.select_token([-math.inf] * 3, None, 2, **r)[:2] == ([-1, -1], [0.0, 0.0])
    assert op.select_token([0.0, math.inf, 1.0], None, 2, **r)[:2] == ([1, 2], [1.0, 0.0])
    # scores far below fp32's range keep their ratio when renormalised
    w = op.select_token([-200.0, -200.0 + math.log(3)], None, 2, **SIG)[1]
    assert np.allclose(w, [0.75, 0.25])


def test_w4_worked_example_and_round_trip():
    q = np.zeros((1, 32), np.uint8)
    q[0, :4] = [8, 9, 0, 15]
    codes = op.w4_pack(q)
    assert codes[0, 0] == 8 | 9 << 4 and codes[0, 1] == 0 | 15 << 4
    w = op.w4_dequant(codes, [[0.5]], None, 32)
    assert w[0, :4].tolist() == [0.0, 0.5, -4.0, 3.5] and (w[0, 4:] == -4.0).all()
    w = op.w4_dequant(codes, [[0.5]], np.array([[9 + 16]], np.uint8), 32)   # the low four bits of the zero point
    assert w[0, :4].tolist() == [-0.5, 0.0, -4.5, 3.0]


@pytest.mark.parametrize("group", [32, 64])
def test_w4_dequant_against_a_scalar_loop(group):
    rng = np.random.default_rng(3)
    q, s, z = rng.integers(0, 16, (3, 128)), rng.normal(size=(3, 128 // group)), rng.integers(0, 16, (3, 128 // group))
    w = op.w4_dequant(op.w4_pack(q), s, z.astype(np.uint8), group)
    for n in range(3):
        for k in range(128):
            assert w[n, k] == (q[n, k] - z[n, k // group]) * s[n, k // group]


def test_w4_experts_against_the_dense_expert():
    from oracle import moe
    rng = np.random.default_rng(4)
    w13, w2, x = rng.normal(size=(2, 64, 32)), rng.normal(size=(2, 32, 32)), rng.normal(size=(5, 32))
    y = op.w4_expert_rows(x, lambda e: w13[e], lambda e: w2[e], [2, 3])
    for r in range(5):
        e = 0 if r < 2 else 1
        ref = moe.swiglu_ffn(x[r:r + 1], w13[e], w2[e])
        assert np.allclose(y[r], ref[0], rtol=1e-12)
