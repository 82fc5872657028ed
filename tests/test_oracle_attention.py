"""Pins of the float64 oracle of cross attention and of the norm with the position rotation: closed forms,
invariants, a naive loop and central differences."""

import numpy as np
import pytest

from oracle import attention as att
from oracle import norm_rope as nr


def _inputs(rng, R=2, G=3, Lq=2, Lk=5, H=4, Hk=2, D=8):
    q = rng.standard_normal((R * G, Lq, H, D))
    k, v = rng.standard_normal((R, Lk, Hk, D)), rng.standard_normal((R, Lk, Hk, D))
    return q, k, v, rng.standard_normal(q.shape)


def test_forward_is_the_naive_loop():
    rng = np.random.default_rng(0)
    q, k, v, _ = _inputs(rng)
    keep = att.attended(2, 5, [3, 5], rng.random((2, 5)) < 0.8)
    keep[0, 0] = keep[1, 4] = True
    out, lse = att.forward(q, k, v, keep, 0.3)
    for b in range(6):
        for i in range(2):
            for h in range(4):
                e = {n: np.exp(0.3 * q[b, i, h] @ k[b // 3, n, h // 2]) for n in range(5) if keep[b // 3, n]}
                total = sum(e.values())
                want = sum(e[n] / total * v[b // 3, n, h // 2] for n in e)
                assert np.allclose(out[b, i, h], want, rtol=1e-12, atol=1e-13)
                assert np.isclose(lse[b, i, h], np.log(total), rtol=1e-12)


def test_one_key_and_none():
    rng = np.random.default_rng(1)
    q, k, v, g = _inputs(rng, R=3, G=1)
    keep = att.attended(3, 5, [1, 0, 5])
    k[1], v[1] = np.nan, np.nan           # nothing of an empty state is read
    out, lse = att.forward(q, k, v, keep, 0.5)
    assert np.allclose(out[0], np.repeat(v[0, 0], 2, axis=0)[None])
    assert not out[1].any() and np.all(lse[1] == -np.inf)
    dq, dk, dv = att.backward(q, k, v, g, keep, 0.5)
    assert not dq[1].any() and not dk[1].any() and not dv[1].any()
    assert np.allclose(dq[0], 0.0, atol=1e-14) and not dk[0, 1:].any()   # a softmax over one key is constant


def test_masked_places_have_no_influence():
    rng = np.random.default_rng(2)
    q, k, v, g = _inputs(rng)
    keep = rng.random((2, 5)) < 0.6
    keep[:, 1] = True
    want = att.forward(q, k, v, keep, 0.4)[0], *att.backward(q, k, v, g, keep, 0.4)
    k[~keep], v[~keep] = np.nan, np.inf
    got = att.forward(q, k, v, keep, 0.4)[0], *att.backward(q, k, v, g, keep, 0.4)
    assert all(np.array_equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_attention_gradients_are_central_differences(which):
    rng = np.random.default_rng(3)
    q, k, v, g = _inputs(rng)
    keep = att.attended(2, 5, [4, 5])
    grads = dict(zip("qkv", att.backward(q, k, v, g, keep, 0.7)))
    x = {"q": q, "k": k, "v": v}
    for _ in range(8):
        u = rng.standard_normal(x[which].shape)
        h = 1e-5
        f = [(g * att.forward(*(x[n] + (s * h * u if n == which else 0.0) for n in "qkv"), keep, 0.7)[0]).sum()
             for s in (1, -1)]
        assert np.isclose((f[0] - f[1]) / (2 * h), (grads[which] * u).sum(), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_depends_on_the_difference_of_positions(interleaved):
    rng = np.random.default_rng(4)
    f = 10.0 ** -np.arange(3)
    q, k = rng.standard_normal((1, 1, 1, 8)), rng.standard_normal((1, 1, 1, 8))
    turn = lambda x, p: nr.rotate(x, np.array([[p]]), f, interleaved)  # noqa: E731
    a = (turn(q, 7) * turn(k, 3)).sum()
    assert np.isclose(a, (turn(q, 104) * turn(k, 100)).sum(), rtol=1e-12)
    assert np.isclose(a, (turn(q, 4) * k).sum(), rtol=1e-12)
    assert np.allclose(np.linalg.norm(turn(q, 5)), np.linalg.norm(q))
    assert np.array_equal(turn(q, 5)[..., 6:], q[..., 6:])            # the rest of the head is not turned
    assert np.allclose(nr.rotate(turn(q, 5), np.array([[5]]), f, interleaved, -1.0), q)
    quarter = nr.rotate(np.eye(8)[None, None, :1], np.array([[1]]), [np.pi / 2], interleaved)
    assert np.allclose(quarter[0, 0, 0], np.eye(8)[1], atol=1e-15)    # (1, 0) -> (0, 1)


def test_norm_has_unit_mean_square():
    rng = np.random.default_rng(5)
    x = 3.0 * rng.standard_normal((2, 3, 2, 16))
    y = nr.forward(x, np.ones(16), np.arange(6).reshape(2, 3), [0.5, 0.1], 0.0, True)
    assert np.allclose((y * y).mean(axis=-1), 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients_are_central_differences(interleaved):
    rng = np.random.default_rng(6)
    x, w, dy = rng.standard_normal((2, 3, 2, 16)), rng.standard_normal(16), rng.standard_normal((2, 3, 2, 16))
    pos, fr = rng.integers(-50, 50, (2, 3)), 10.0 ** -np.arange(4)
    dx, dw = nr.backward(x, w, pos, fr, 1e-3, interleaved, dy)
    for _ in range(8):
        u, t, h = rng.standard_normal(x.shape), rng.standard_normal(16), 1e-5
        f = [(dy * nr.forward(x + s * h * u, w, pos, fr, 1e-3, interleaved)).sum() for s in (1, -1)]
        assert np.isclose((f[0] - f[1]) / (2 * h), (dx * u).sum(), rtol=1e-7, atol=1e-8)
        f = [(dy * nr.forward(x, w + s * h * t, pos, fr, 1e-3, interleaved)).sum() for s in (1, -1)]
        assert np.isclose((f[0] - f[1]) / (2 * h), (dw * t).sum(), rtol=1e-7, atol=1e-8)


def test_error_bounds_hold_for_a_rounded_evaluation():
    """The bounds the GPU tests use, on a float32 evaluation with P, dS and results rounded to half precision."""
    rng = np.random.default_rng(7)
    half = lambda x: x.astype(np.float16).astype(np.float64)  # noqa: E731
    q, k, v, g = (half(x) for x in _inputs(rng, Lk=33, D=16))
    keep = att.attended(2, 33, [33, 20])
    t_out, t_dq, t_dk, t_dv = att.error_bounds(q, k, v, g, keep, 0.25, 2.0 ** -11, 2.0 ** -11, 2.0 ** -25)
    p = half(att.probabilities(q, k, keep, 0.25)[1])
    out = half((p @ att._per_query(v, 6, 4)).transpose(0, 2, 1, 3))
    assert np.all(np.abs(out - att.forward(q, k, v, keep, 0.25)[0]) <= t_out)
    gh = g.transpose(0, 2, 1, 3)
    dv = half(att._summed(p.transpose(0, 1, 3, 2) @ gh, 2, 2))
    dq, dk, want = att.backward(q, k, v, g, keep, 0.25)
    assert np.all(np.abs(dv - want) <= t_dv)
    # the bounds are of the size of the rounding, not vacuous
    for t, x in ((t_out, out), (t_dq, dq), (t_dk, dk), (t_dv, want)):
        assert np.median(t) < 0.02 * np.abs(x).max()
