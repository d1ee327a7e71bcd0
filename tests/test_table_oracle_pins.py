"""The float64 oracle of the item-table operators against other things than itself:
central differences of its losses, and torch's float64 autograd of the definitions."""
import numpy as np
import pytest
import torch

from oracle import table_oracle as O


def draw(T, V, D, K, seed):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, D)), r.standard_normal((V, D)) / np.sqrt(D), r.integers(0, V, (T, K)).astype(np.int32),
            2.0 * r.standard_normal((T, K)), r)


def differences(f, x, dx, h=1e-6):
    return (f(x + h * dx) - f(x - h * dx)) / (2 * h)


@pytest.mark.parametrize("tau,reduction", [(1.0, "mean"), (0.6, "sum"), (2.5, "mean")])
def test_distill_gradients_are_differences(tau, reduction):
    H, E, ids, lg, r = draw(7, 13, 5, 4, 1)
    ids[0, 1] = -1
    ids[2] = -1
    ids[3, 2] = ids[3, 0]                       # a repeated id
    lg[4, 3] = -np.inf
    mask = np.ones(7, np.uint8)
    mask[5] = 0
    w = r.uniform(-2, 2, 7)
    w[6] = 0.0
    kw = dict(ids=ids, logits=lg, mask=mask, weights=w, tau=tau, reduction=reduction)
    ref = O.distill(H, E, **kw)
    assert ref.valid.tolist() == [True, True, False, True, True, False, False]
    for _ in range(3):
        a, b = r.standard_normal(H.shape), r.standard_normal(E.shape)
        assert np.isclose(differences(lambda x: O.distill(x, E, **kw).loss, H, a), (ref.dH * a).sum(), rtol=1e-6, atol=1e-8)
        assert np.isclose(differences(lambda x: O.distill(H, x, **kw).loss, E, b), (ref.dE * b).sum(), rtol=1e-6, atol=1e-8)


def test_distill_is_the_kl_divergence():
    H, E, ids, lg, _ = draw(6, 11, 4, 3, 2)
    for t in range(6):
        ids[t] = [t, t + 1, t + 2]
    tau = 1.7
    ref = O.distill(H, E, ids, lg, tau=tau)
    Ht = torch.tensor(H, requires_grad=True)
    Et = torch.tensor(E, requires_grad=True)
    q = torch.zeros(6, 11, dtype=torch.float64).scatter_(1, torch.tensor(ids).long(), torch.softmax(torch.tensor(lg) / tau, 1))
    lp = torch.log_softmax(Ht @ Et.T / tau, 1)
    loss = tau * tau * torch.nn.functional.kl_div(lp, q, reduction="batchmean")
    loss.backward()
    assert abs(loss.item() - ref.loss) < 1e-12 * (1 + abs(ref.loss))
    np.testing.assert_allclose(Ht.grad.numpy(), ref.dH, rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(Et.grad.numpy(), ref.dE, rtol=1e-10, atol=1e-13)


def test_preference_gradients_are_differences_and_autograd():
    H, E, _, _, r = draw(14, 9, 6, 1, 3)
    ids = r.integers(0, 9, 14).astype(np.int32)
    ids[3] = -1
    off = O.offsets_of([3, 0, 4, 5], first=1)                 # one empty sequence; rows 0 and 13 outside
    ref_lp = r.standard_normal(4)
    mask = np.ones(14, np.uint8)
    mask[5] = 0
    kw = dict(ids=ids, offsets=off, ref=ref_lp, mask=mask, beta=0.7)
    ref = O.preference(H, E, **kw)
    assert not ref.valid[[0, 3, 5, 13]].any() and ref.valid.sum() == 10
    for _ in range(3):
        a, b = r.standard_normal(H.shape), r.standard_normal(E.shape)
        assert np.isclose(differences(lambda x: O.preference(x, E, **kw).loss, H, a), (ref.dH * a).sum(), rtol=1e-6, atol=1e-9)
        assert np.isclose(differences(lambda x: O.preference(H, x, **kw).loss, E, b), (ref.dE * b).sum(), rtol=1e-6, atol=1e-9)
    Ht, Et = torch.tensor(H, requires_grad=True), torch.tensor(E, requires_grad=True)
    lp = torch.log_softmax(Ht @ Et.T, 1)
    L = [sum((lp[t, ids[t]] for t in range(off[i], off[i + 1]) if ids[t] >= 0 and mask[t]), torch.zeros((), dtype=torch.float64))
         for i in range(4)]
    x = [0.7 * ((L[2 * p] - L[2 * p + 1]) - (ref_lp[2 * p] - ref_lp[2 * p + 1])) for p in range(2)]
    loss = -torch.nn.functional.logsigmoid(torch.stack(x)).mean()
    loss.backward()
    assert abs(loss.item() - ref.loss) < 1e-12
    np.testing.assert_allclose(Ht.grad.numpy(), ref.dH, rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(Et.grad.numpy(), ref.dE, rtol=1e-10, atol=1e-13)


def test_embed_against_torch():
    r = np.random.default_rng(4)
    E = r.standard_normal((10, 3))
    ids = np.array([1, -1, 9, 1, 1, 0])
    W = torch.tensor(E, requires_grad=True)
    g = r.standard_normal((6, 3))
    keep = torch.tensor(ids >= 0)[:, None]
    out = torch.where(keep, 2.5 * torch.nn.functional.embedding(torch.tensor(ids).clamp(min=0), W), torch.zeros(()).double())
    out.backward(torch.tensor(g))
    np.testing.assert_allclose(out.detach().numpy(), O.embed(E, ids, 2.5), rtol=1e-14)
    np.testing.assert_allclose(W.grad.numpy(), O.embed_grad(g, ids, 10, 2.5), rtol=1e-13, atol=1e-15)
