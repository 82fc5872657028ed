"""The example denoiser: its operators together as a network uses them, against the oracle, through training and the
sampler."""

import os
import sys

import numpy as np
import pytest

from gpu_util import say, torch_dev
from oracle import attention as att
from oracle import norm_rope as nr
from workloads import Workload

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

WL = Workload("small_chain", "", 4, 2, 3, 4, 12, 52, (5,), 1.0, (0.0, 1.0), None, 3)


def _numpy_eps(model, x, states, kv_len, pos_q, pos_k):
    """The network's forward in float64 with the oracle's operators."""
    f = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    B, (R, L, _) = x.shape[0], states.shape
    i, j = np.triu_indices(64, 1)
    full = np.zeros((B, 64, 64))
    full[:, i, j] = f(x)
    full += full.transpose(0, 2, 1)
    q = (full @ f(model.wq)).reshape(B, 64, model.heads, model.dim)
    kv = (f(states) @ f(model.wkv)).reshape(R, L, 2, model.heads_kv, model.dim)
    q = nr.forward(q, f(model.nq), pos_q.cpu().numpy(), model.freqs, 1e-6, False)
    k = nr.forward(kv[:, :, 0], f(model.nk), pos_k.cpu().numpy(), model.freqs, 1e-6, False)
    a, _ = att.forward(q, k, kv[:, :, 1], att.attended(R, L, kv_len.cpu().numpy()), model.dim ** -0.5)
    y = a.reshape(B, 64, -1) @ f(model.wo) + full @ f(model.skip)
    return 0.5 * (y + y.transpose(0, 2, 1))[:, i, j]


def test_prediction_matches_oracle():
    """float32 throughout: each of the network's five products sums at most 128 terms, 5 x 128 x 2^-24 = 4e-5 of the
    absolute sums in the worst case, and a normalised head's scores are of order sqrt(dim), so their errors pass through
    the softmax at their own size: 1e-4 of the largest value bounds both."""
    import attention_denoiser as ex

    torch, dev = torch_dev()
    say("denoiser forward against the oracle")
    inputs = ex.setup(WL, 77, 48, 1, dev)
    model = ex.Denoiser(48, seed=2).to(dev)
    x = torch.randn(24, 2016, generator=torch.Generator().manual_seed(3)).to(dev)
    for states in inputs[:2]:   # conditional, null
        got = model(x, states, *inputs[2:]).detach().double().cpu().numpy()
        want = _numpy_eps(model, x, states, *inputs[2:])
        assert np.abs(got - want).max() <= 1e-4 * np.abs(want).max()


def test_gradients_against_differences():
    """Directional derivatives of the loss for every parameter: the central difference with h = 2^-7 is off by the
    loss's curvature (h^2) and by its float32 rounding 2^-22 / h, both below 1e-3 of the gradient's size times the
    direction's."""
    import attention_denoiser as ex

    torch, dev = torch_dev()
    say("denoiser gradients against central differences")
    inputs = ex.setup(WL, 50, 48, 4, dev)
    model = ex.Denoiser(48, seed=5).to(dev)
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(24, 2016, generator=gen).to(dev)
    g = torch.randn(24, 2016, generator=gen).to(dev) / 2016 ** 0.5
    (model(x, inputs[0], *inputs[2:]) * g).sum().backward()
    for name, w in model.named_parameters():
        u = torch.randn(w.shape, generator=gen).to(dev)
        u /= u.norm()
        want = float((w.grad.double() * u.double()).sum())
        f = []
        with torch.no_grad():
            for s in (2.0 ** -7, -2.0 ** -7):
                w.add_(s * u)
                f.append(float((model(x, inputs[0], *inputs[2:]).double() * g.double()).sum()))
                w.sub_(s * u)
        size = float(w.grad.norm())
        assert abs((f[0] - f[1]) * 2.0 ** 6 - want) <= 1e-3 * size + 1e-3, name


def test_training_lowers_the_loss_and_samples_are_finite():
    import attention_denoiser as ex

    torch, dev = torch_dev()
    say("denoiser training and sampling")
    inputs = ex.setup(WL, 77, 48, 7, dev)
    model = ex.Denoiser(48, seed=8).to(dev)
    losses = ex.train(model, WL, inputs, 25, 9)
    assert np.isfinite(losses).all() and np.mean(losses[-5:]) < 0.7 * np.mean(losses[:3])
    x = ex.sample(model, WL, inputs, 5, 9)
    again = ex.sample(model, WL, inputs, 5, 9)
    assert torch.isfinite(x).all() and torch.equal(x, again)
