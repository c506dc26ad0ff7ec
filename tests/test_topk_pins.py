"""Pins of the top-k and top-k distillation oracles against things other than themselves (CPU only):
torch.topk and torch.logsumexp; the whole-row loss oracle (a list of every token is the whole row);
torch's autograd and central differences for the gradient; closed forms of special cases."""

import numpy as np
import pytest

from oracle import opd_oracle as O
from oracle import topk as T


def test_topk_row_matches_torch():
    torch = pytest.importorskip("torch")
    y = np.random.default_rng(0).normal(0, 3, 301)
    v, i, r = T.topk_row(y, 17)
    tv, ti = torch.topk(torch.tensor(y), 17)
    assert np.array_equal(v, tv.numpy()) and np.array_equal(i, ti.numpy())
    rest = torch.tensor(y).scatter(0, ti, -np.inf)
    assert abs(r - float(torch.logsumexp(rest, 0))) < 1e-12


def test_topk_row_ties_and_masked_rows():
    v, i, r = T.topk_row([1.0, 2.0, 2.0, 2.0, -np.inf], 2)
    assert i.tolist() == [1, 2] and v.tolist() == [2.0, 2.0]
    assert abs(r - np.log(np.exp(2) + np.exp(1))) < 1e-12
    v, i, r = T.topk_row([-np.inf] * 4, 3)
    assert i.tolist() == [0, 1, 2] and r == -np.inf


@pytest.mark.parametrize("tau", [0.02, np.inf])
@pytest.mark.parametrize("alpha", [0.0, 0.6, 1.0])
def test_a_list_of_every_token_is_the_whole_row(alpha, tau):
    rng = np.random.default_rng(5)
    z, y = rng.normal(0, 2, 50), rng.normal(0, 2, 50)
    order = rng.permutation(50)
    loss, info = T.row_loss(z, order, y[order], -np.inf, alpha, min(tau, 1e9))
    dz, _ = T.row_grad(z, order, y[order], -np.inf, alpha, min(tau, 1e9))
    ref, whole = O.row_grad(z, y, alpha, tau)
    assert abs(loss - whole["loss"]) < 1e-12
    assert np.allclose(dz, ref, rtol=0, atol=1e-14)


def _autograd(z, index, logit, rest, alpha, tau, kl):
    torch = pytest.importorskip("torch")
    zt = torch.tensor(z, dtype=torch.float64, requires_grad=True)
    idx = torch.tensor(np.asarray(index))
    others = torch.ones(len(z), dtype=torch.bool)
    others[idx] = False
    c = torch.cat([zt[idx], torch.logsumexp(zt[others], 0)[None]])
    t = torch.tensor(np.append(logit, rest))
    lp, lq = torch.log_softmax(c, 0), torch.log_softmax(t, 0)
    term = lp.exp() * (lp - lq) if kl == "reverse" else lq.exp() * (lq - lp)
    term = torch.where(term <= tau, term, torch.full_like(term, tau))
    a = int(np.argmax(logit))
    loss = alpha * term.sum() - (1 - alpha) * lp[a]
    loss.backward()
    return float(loss.detach()), zt.grad.numpy()


@pytest.mark.parametrize("kl", ["reverse", "forward"])
@pytest.mark.parametrize("tau", [0.01, 50.0])
@pytest.mark.parametrize("k", [1, 3, 20, 29])
def test_loss_and_gradient(kl, tau, k):
    rng = np.random.default_rng(k)
    y = rng.normal(0, 3, 30)
    z = y + rng.normal(0, 1.5, 30)
    v, i, r = T.topk_row(y, k)
    loss, _ = T.row_loss(z, i, v, r, 0.7, tau, kl)
    dz, _ = T.row_grad(z, i, v, r, 0.7, tau, kl)
    ref, grad = _autograd(z, i, v, r, 0.7, tau, kl)
    assert abs(loss - ref) < 1e-12 and np.allclose(dz, grad, rtol=0, atol=1e-13)
    h = 1e-6
    for j in range(30):
        e = np.zeros(30)
        e[j] = h
        d = (T.row_loss(z + e, i, v, r, 0.7, tau, kl)[0] - T.row_loss(z - e, i, v, r, 0.7, tau, kl)[0]) / (2 * h)
        assert abs(d - dz[j]) < 1e-8
    assert abs(dz.sum()) < 1e-13  # a softmax does not see a constant


def test_entries_that_do_not_count():
    rng = np.random.default_rng(9)
    z = rng.normal(0, 2, 20)
    full = T.row_loss(z, [4, 7], [2.0, 1.0], 0.5, 0.5, 0.1)
    padded = T.row_loss(z, [4, -1, 7, 4, 25], [2.0, 9.0, 1.0, 8.0, 9.0], 0.5, 0.5, 0.1)
    assert full[0] == padded[0]
    for index, logit in (([-1, -1], [1.0, 2.0]), ([3, 4], [-np.inf, -np.inf])):
        assert T.row_loss(z, index, logit, 0.5, 0.5, 0.1)[0] == 0.0
        assert not T.row_grad(z, index, logit, 0.5, 0.5, 0.1)[0].any()


def test_zero_probabilities():
    z = np.array([1.0, 0.5, -np.inf, 0.0])
    # the teacher gives nothing to the others: an infinite reverse term, clipped; no forward term
    loss, info = T.row_loss(z, [0, 1], [1.0, 0.0], -np.inf, 1.0, 0.25, "reverse")
    assert np.isinf(info["term"][-1]) and np.isfinite(loss)
    loss, info = T.row_loss(z, [0, 1], [1.0, 0.0], -np.inf, 1.0, np.inf, "forward")
    assert info["term"][-1] == 0.0 and np.isfinite(loss)
    # the drafter gives nothing to a listed token: the other way round
    loss, info = T.row_loss(z, [0, 2], [1.0, 0.0], 0.5, 1.0, 0.25, "forward")
    assert np.isinf(info["term"][1]) and np.isfinite(loss)
    dz, info = T.row_grad(z, [0, 2], [1.0, 0.0], 0.5, 1.0, np.inf, "reverse")
    assert info["term"][1] == 0.0 and np.isfinite(dz).all() and dz[2] == 0.0
