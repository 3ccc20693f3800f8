"""The oracle's row-wise steps on threads give the bits of the same steps in one piece (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import _rows


def cases():
    rng = np.random.default_rng(3)
    H, W = rng.standard_normal((300, 24)), 0.3 * rng.standard_normal((5003, 24))
    y = rng.integers(0, 5003, 300)
    y[::7] = oracle.IGNORE_INDEX
    a = rng.standard_normal(300)
    cu = np.array([0, 40, 90, 200, 290])
    return [lambda: oracle.lce_large_f64(H, W, y), lambda: oracle.lce_large_f64(H, W, y, row_block=64, grads=False),
            lambda: oracle.head_gradients_f64(H, W, y, a, temperature=0.7), lambda: oracle.policy_f64(H, W, y, a),
            lambda: oracle.preference_f64(H, W, y, cu), lambda: oracle.logprobs_f64(H, W, y, top_k=5),
            lambda: oracle.logprobs_backward_f64(H, W, y, a, a)]


@pytest.mark.parametrize("k", range(7))
def test_threads_change_no_bit(monkeypatch, k):
    monkeypatch.setattr(_rows, "_CORES", 7)
    monkeypatch.setattr(_rows, "_pool", None)
    many = cases()[k]()
    assert _rows._pool is not None
    monkeypatch.setattr(_rows, "_CORES", 1)
    one = cases()[k]()
    assert many.keys() == one.keys()
    for name in one:
        assert np.array_equal(many[name], one[name]), name


@pytest.mark.parametrize("kw", [{}, dict(row_block=64, grads=False), dict(reduction=oracle.SUM, grad_loss=-2.0),
                                dict(n_valid_override=7)])
def test_full_size_form_is_the_definition_bit_for_bit(monkeypatch, kw):
    monkeypatch.setattr(_rows, "_CORES", 7)
    monkeypatch.setattr(_rows, "_pool", None)
    rng = np.random.default_rng(5)
    H, W = (rng.integers(0, 1 << 16, s).astype(np.uint16) & 0xBFFF for s in ((600, 24), (5003, 24)))   # finite, below 2
    y = rng.integers(0, 5003, 600)
    y[::7] = oracle.IGNORE_INDEX
    want = oracle.lce_bf16(H, W, y, **kw)
    ref = oracle.lce_f64(oracle.decode_bf16(H), oracle.decode_bf16(W), y, **kw)
    monkeypatch.setattr(oracle, "LARGE", 1)
    got = oracle.lce_bf16(H, W, y, **kw)
    assert _rows._pool is not None and got.keys() == want.keys() == ref.keys()
    for name in got:
        assert np.array_equal(got[name], want[name]) and np.array_equal(got[name], ref[name]), name


def test_pieces_cover_the_rows_once(monkeypatch):
    monkeypatch.setattr(_rows, "_CORES", 5)
    monkeypatch.setattr(_rows, "_pool", None)
    for rows, columns in ((0, 10), (1, 1 << 20), (3, 1 << 20), (17, 1 << 16), (1000, 8), (100, 5000)):
        seen = np.zeros(rows, int)

        def step(a, b):
            seen[a:b] += 1
        _rows.by_rows(step, rows, columns)
        assert (seen == 1).all()


def test_a_failing_piece_is_raised(monkeypatch):
    monkeypatch.setattr(_rows, "_CORES", 4)
    monkeypatch.setattr(_rows, "_pool", None)

    def step(a, b):
        raise ValueError("no")
    with pytest.raises(ValueError, match="no"):
        _rows.by_rows(step, 100, 1 << 16)
