"""Pins of the float64 definitions in oracle/score.py (CPU only): finite
differences, the plain attention oracle where nothing is modified, closed
forms, and the block rule of the quantiser."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import fp8 as F
from oracle import score as S


def _inputs(seed, b=2, hq=4, hkv=2, n=9, d=6):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in ((b, hq, n, d), (b, hkv, n, d), (b, hkv, n, d), (b, hq, n, d))]


@pytest.mark.parametrize("window,causal", [((-1, -1), False), ((-1, 0), True), ((3, 2), False)])
def test_unmodified_scores_are_plain_attention(window, causal):
    q, k, v, do = _inputs(0)
    o, lse = S.forward(q, k, v, 0.3, window=window)
    ro, rl = A.forward(q, k, v, 0.3, False, window)
    assert np.abs(o - ro).max() < 1e-13 and np.abs(lse - rl).max() < 1e-13
    for got, ref in zip(S.backward(q, k, v, do, 0.3, window=window), A.backward(q, k, v, do, 0.3, False, window)):
        assert np.abs(got - ref).max() < 1e-12


@pytest.mark.parametrize("cap,slopes,masked", [(1.5, None, False), (0.0, (0.5, 0.25, 0.1, 0.0), True),
                                               (2.0, (0.3, 0.2, 0.1, 0.05), True)])
def test_gradients_match_finite_differences(cap, slopes, masked):
    q, k, v, do = _inputs(1)
    ids = np.array([[0, 0, 0, 1, 1, 1, 1, -1, -1], [0] * 9])
    ranges = S.mask_rows(2, 9, ids, [5, 2], True) if masked else None
    grads = S.backward(q, k, v, do, 0.4, ranges, (-1, -1), cap, slopes)

    def loss(*args):
        return (S.forward(*args, 0.4, ranges, (-1, -1), cap, slopes)[0] * do).sum()

    r = np.random.default_rng(2)
    for i, grad in enumerate(grads):
        for _ in range(12):
            at = tuple(int(r.integers(s)) for s in grad.shape)
            args = [q.copy(), k.copy(), v.copy()]
            args[i][at] += 1e-5
            up = loss(*args)
            args[i][at] -= 2e-5
            assert abs((up - loss(*args)) / 2e-5 - grad[at]) < 1e-7


def test_mask_rows_by_definition():
    r = np.random.default_rng(3)
    ids = np.array([np.repeat([0, 1, 0, -1], [3, 4, 2, 3]), r.integers(0, 2, 12)])
    for causal in (True, False):
        for prefix in (None, [2, 5]):
            got = S.mask_rows(2, 12, ids, prefix, causal)
            for b in range(2):
                run = np.concatenate([[0], np.cumsum(ids[b][1:] != ids[b][:-1])])
                for i in range(12):
                    see = [j for j in range(12) if ids[b][i] >= 0 and run[j] == run[i]
                           and (not causal or j <= i or (prefix is not None and j < prefix[b]))]
                    lo, hi = got[b, i]
                    assert list(range(lo, hi)) == see


def test_an_empty_row_has_no_output_and_no_gradient():
    q, k, v, do = _inputs(4)
    ranges = S.mask_rows(2, 9, np.array([[0] * 5 + [-1] * 4] * 2), None, False)
    o, lse = S.forward(q, k, v, 0.3, ranges, cap=2.0)
    assert not o[:, :, 5:].any() and np.isneginf(lse[:, :, 5:]).all() and np.isfinite(lse[:, :, :5]).all()
    dq, dk, dv = S.backward(q, k, v, do, 0.3, ranges, cap=2.0)
    assert not dq[:, :, 5:].any() and not dk[:, :, 5:].any() and not dv[:, :, 5:].any()


def test_a_large_cap_changes_nothing_and_a_small_one_flattens():
    q, k, v, _ = _inputs(5)
    assert np.abs(S.forward(q, k, v, 0.3, cap=1e6)[0] - S.forward(q, k, v, 0.3)[0]).max() < 1e-9
    assert np.abs(S.forward(q, k, v, 0.3, cap=1e-6)[0] - v.repeat(2, 1).mean(2, keepdims=True)).max() < 1e-5


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_turns_back(interleaved):
    r = np.random.default_rng(6)
    x = r.standard_normal((2, 3, 7, 10))
    a = r.uniform(0, 6, (7, 4))
    y = S.rotate(x, np.cos(a), np.sin(a), interleaved)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.abs((y ** 2).sum(-1) - (x ** 2).sum(-1)).max() < 1e-12
    assert np.abs(S.rotate(y, np.cos(a), np.sin(a), interleaved, inverse=True) - x).max() < 1e-14
    # a difference of positions is all that a product of two rotated rows sees
    p = S.rotate(np.broadcast_to(x[0, 0, 0], (7, 10)), np.cos(np.arange(7)[:, None] * a[0]), np.sin(np.arange(7)[:, None] * a[0]), interleaved)
    assert abs(p[1] @ p[3] - p[4] @ p[6]) < 1e-12
    if not interleaved:
        cos, sin = F.rope_tables(7, 10)
        assert np.abs(S.rotate(x, cos, sin) - F.rope_f64(x, cos, sin)).max() < 1e-14


def test_appending_a_whole_block_at_once_is_the_quantiser():
    r = np.random.default_rng(7)
    x = r.standard_normal((1, 2, 200, 64)).astype(np.float32)
    codes, fac = F.quantize_blocks(x)
    c0, f0 = np.zeros((2, 300, 64), np.uint8), np.ones((2, 3), np.float32)
    c, f = S.append_sequence(c0, f0, 0, x[0])
    assert np.array_equal(c[:, :200], codes[0]) and np.array_equal(f[:, :2], fac[0]) and not c[:, 200:].any()


def test_appending_row_by_row_moves_the_factor_and_keeps_half_a_step():
    x = np.ones((1, 4, 64)) * np.array([0.3, 1.7, 20.0, 0.01])[None, :, None]
    c, f = np.zeros((1, 128, 64), np.uint8), np.ones((1, 1), np.float32)
    for i in range(4):
        c, f = S.append_sequence(c, f, i, x[:, i:i + 1])
    assert f[0, 0] == 2.0 ** -4    # 20 * 2^4 = 320 <= 448
    back = F.e4m3_decode(c[0, :4]) * f[0, 0]
    # each row was rounded at most twice: once when appended, once when the factor moved
    assert (np.abs(back - x[0]) <= 2 * np.maximum(np.abs(x[0]) * 2.0 ** -4, 2.0 ** -14)).all()


def test_decode_is_the_last_row():
    q, k, v, _ = _inputs(8)
    for cap, slopes, left in ((0.0, None, -1), (1.5, (0.5, 0.25, 0.1, 0.0), 4)):
        o, lse = S.forward(q, k, v, 0.3, window=(left, 0), cap=cap, slopes=slopes)
        od, ld, mag = S.decode(q[:, :, 8], k, v, [9, 9], 0.3, cap, slopes, left)
        assert np.abs(od - o[:, :, 8]).max() < 1e-13 and np.abs(ld - lse[:, :, 8]).max() < 1e-13
        assert (mag >= np.abs(od) - 1e-15).all()
    o, lse, _ = S.decode(q[:, :, 8], k, v, [0, 1], 0.3)
    assert not o[0].any() and np.isneginf(lse[0]).all() and np.abs(o[1] - v[1, :, 0].repeat(2, 0)).max() < 1e-15
