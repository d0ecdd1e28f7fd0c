"""The plain fp64 statements of routing, combine and MXFP4 pinned by hand-worked cases, identities and
differences (CPU): what the GPU tests compare with has to be right by itself."""
import numpy as np
import pytest

import plain


def test_fp4_hand_worked_block():
    x = np.zeros((1, 32))
    x[0, :16] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -6.0, 7.9, -0.0, 0.26, 0.24, -0.75, 1.0, 3.0]
    code, s = plain.quantize_fp4(x)
    assert s[0, 0] == 127                                    # amax 7.9: e = 2 - 2 = 0
    #        4    .25  .75  1.25 1.75 2.5  3.5  5    -6   7.9  -0   .26  .24  -.75 1    3
    want = [6, 0, 2, 2, 4, 4, 6, 6, 8 + 7, 7, 8, 1, 0, 8 + 2, 2, 5]
    assert code[0, :16].tolist() == want


@pytest.mark.parametrize("amax,byte", [(1.0, 125), (4.0, 127), (6.0, 127), (8.0, 128), (2.0 ** -125, 0),
                                       (2.0 ** -124, 1), (2.0 ** -133, 0), (3.3e38, 252), (0.0, 0)])
def test_fp4_scale_bytes(amax, byte):
    x = np.zeros((1, 32))
    x[0, 5] = -amax
    assert plain.quantize_fp4(x)[1][0, 0] == byte


def test_fp4_special_blocks_and_round_trip():
    x = np.ones((1, 64))
    x[0, 3], x[0, 4] = np.nan, -1.0
    code, s = plain.quantize_fp4(x)
    assert s.tolist() == [[255, 125]] and code[0, 0] == 7 and code[0, 4] == 15
    g = np.random.default_rng(0)
    y = g.standard_normal((5, 96))
    code, s = plain.quantize_fp4(y)
    v = plain.values_fp4(plain.pack(code), s)
    again = plain.quantize_fp4(v)
    assert np.array_equal(again[0], code) and np.array_equal(again[1], s)
    assert np.array_equal(plain.unpack(plain.pack(code)), code)


def test_route_hand_worked():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0, np.nan]])
    ids, w = plain.route(x, 3)
    assert ids.tolist() == [[1, 2, 4]]                       # the tie between 1 and 2 goes to the lower index
    e = np.exp([0.0, 0.0, -1.0])
    assert np.allclose(w[0], e / e.sum())
    ids, w = plain.route(x, 6, renormalize=False, scale=2.0)
    assert ids.tolist() == [[1, 2, 4, 0, -1, -1]] and np.isclose(w.sum(), 2.0)
    # The bias moves the choice, not the weights.
    ids, w = plain.route(np.zeros((1, 4)), 2, score="sigmoid", bias=[0, 0.1, 0, 0.2])
    assert ids.tolist() == [[3, 1]] and np.allclose(w, 0.5)
    # Groups of two: by the sum of two, group 1 (1 + 1) beats group 0 (1.9 + 0); by the largest it does not.
    y = np.log(np.array([[1.9, 1e-9, 1.0, 1.0]]))
    assert plain.route(y, 1, groups=2, topk_groups=1, group_score="max")[0].tolist() == [[0]]
    assert plain.route(y, 1, groups=2, topk_groups=1, group_score="top2")[0].tolist() == [[2]]
    # Nothing to choose from, and logits at the type's lowest value.
    assert plain.route(np.full((1, 3), -np.inf), 2)[0].tolist() == [[-1, -1]]
    low = np.full((1, 3), -3.3e38)
    assert plain.route(low, 2)[0].tolist() == [[0, 1]] and np.allclose(plain.route(low, 2)[1], 0.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_is_the_difference_quotient(score, renormalize):
    g = np.random.default_rng(1)
    x, dw = g.standard_normal((4, 9)), g.standard_normal((4, 3))
    x[1, 2] = -np.inf
    ids, _ = plain.route(x, 3, score=score)
    ids[2, 2] = -1
    d, size = plain.route_backward(dw, x, ids, score=score, renormalize=renormalize, scale=1.7)
    h = 1e-6
    for t in range(4):
        for e in range(9):
            if not np.isfinite(x[t, e]):
                assert d[t, e] == 0
                continue
            up, down = x[t].copy(), x[t].copy()
            up[e] += h
            down[e] -= h
            diff = sum(dw[t] * (plain.weights_of(up, ids[t], score, renormalize, 1.7)
                                - plain.weights_of(down, ids[t], score, renormalize, 1.7))) / (2 * h)
            assert abs(diff - d[t, e]) < 1e-8
            assert abs(d[t, e]) <= size[t, e] + 1e-15


def test_plan_and_layout_hand_worked():
    off, slot_row, counts = plain.plan(np.array([[2, 0], [-1, 2], [0, 5]]), 3)
    assert counts.tolist() == [2, 0, 2] and off.tolist() == [0, 2, 2, 6]
    assert slot_row.tolist() == [[2, 0], [~4, 3], [1, ~5]]
    lay = plain.grouped_layout(np.arange(1, 7, dtype=np.uint8).reshape(6, 1), off, 1024)
    assert [lay[0], lay[16], lay[512], lay[512 + 16], lay[512 + 48]] == [1, 2, 3, 4, 6] and lay.sum() == 21


def test_combine_gradient_is_the_difference_quotient():
    g = np.random.default_rng(2)
    ids = np.array([[0, 2], [2, -1], [1, 0]])
    _, slot_row, _ = plain.plan(ids, 3)
    rows, w, dy = g.standard_normal((6, 5)), g.standard_normal((3, 2)), g.standard_normal((3, 5))
    d_rows, dw, _ = plain.combine_backward(dy, rows, slot_row, w)
    f = lambda r, v: (plain.combine(r, slot_row, v)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    for i in np.ndindex(rows.shape):
        up, down = rows.copy(), rows.copy()
        up[i] += h
        down[i] -= h
        assert abs((f(up, w) - f(down, w)) / (2 * h) - d_rows[i]) < 1e-8
    for i in np.ndindex(w.shape):
        up, down = w.copy(), w.copy()
        up[i] += h
        down[i] -= h
        assert abs((f(rows, up) - f(rows, down)) / (2 * h) - dw[i]) < 1e-8
