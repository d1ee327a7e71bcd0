"""NaN in the item table, in states and in weights reaches the outputs that depend on it, whichever column of a
tile it falls on."""
import numpy as np
import pytest
import torch

from vocabulary_label_bce_b200 import api

pytestmark = pytest.mark.gpu


def draw(T, V, D, K=2, seed=60):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = torch.randn(T, D, device="cuda", generator=g).to(torch.bfloat16)
    E = (torch.randn(V, D, device="cuda", generator=g) / np.sqrt(D)).to(torch.bfloat16)
    ids = torch.randint(0, 50, (T, K), device="cuda", generator=g).int()
    lg = torch.randn(T, K, device="cuda", generator=g)
    return H, E, ids, lg


# below 8e6 logits the log-sum-exp pass gives the sums, from there on the dH pass
SIZES = [(20, 200, 64), (20, 200, 200), (520, 16001, 64), (520, 16001, 136)]


@pytest.mark.parametrize("T,V,D", SIZES)
def test_a_nan_row_of_the_table(T, V, D):
    H, E, ids, lg = draw(T, V, D)
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    for v in range(64, 64 + (32 if T == 20 else 16)):       # not a target; 32 columns share an arithmetic
        bad = E.clone()
        bad[v, 5] = float("nan")
        loss, lse = api.distill_forward(H, bad, ids, lg)
        assert torch.isnan(loss) and torch.isnan(lse).all(), v
        loss, logp, lse = api.preference_forward(H, bad, ids[:, 0], off)
        assert torch.isnan(loss) and torch.isnan(logp).all() and torch.isnan(lse).all(), v
        loss, lse, dH, dE = api.distill_forward_backward(H, bad, ids, lg)
        assert torch.isnan(loss) and all(torch.isnan(x).all() for x in (lse, dH, dE)), v


@pytest.mark.parametrize("T,V,D", SIZES)
def test_a_nan_target_row(T, V, D):
    H, E, ids, lg = draw(T, V, D)
    ids[7, 1] = 90
    E[90] = float("nan")
    loss, lse, dH, dE = api.distill_forward_backward(H, E, ids, lg)
    assert torch.isnan(loss) and all(torch.isnan(x).all() for x in (lse, dH, dE))


@pytest.mark.parametrize("T,V,D", SIZES)
def test_a_nan_state(T, V, D):
    H, E, ids, lg = draw(T, V, D)
    for t in range(1, 17, 3):
        bad = H.clone()
        bad[t, 3] = float("nan")
        rest = torch.arange(T, device="cuda") != t
        loss, lse, dH, dE = api.distill_forward_backward(bad, E, ids, lg)
        assert torch.isnan(loss) and torch.isnan(lse[t]) and torch.isnan(dH[t]).all() and torch.isnan(dE).all(), t
        assert torch.isfinite(lse[rest]).all() and torch.isfinite(dH[rest]).all(), t
        loss2, lse2 = api.distill_forward(bad, E, ids, lg)
        dH, dE = api.distill_backward(bad, E, ids, lg, lse2)
        assert torch.isnan(loss2) and torch.isnan(lse2[t]) and torch.isnan(dH[t]).all() and torch.isnan(dE).all(), t
        assert torch.isfinite(lse2[rest]).all() and torch.isfinite(dH[rest]).all(), t


@pytest.mark.parametrize("T,V,D", SIZES)
def test_a_nan_weight_or_reference(T, V, D):
    H, E, ids, lg = draw(T, V, D)
    for t in range(0, 16, 3):
        w = torch.ones(T, device="cuda")
        w[t] = float("nan")
        rest = torch.arange(T, device="cuda") != t
        loss, lse, dH, dE = api.distill_forward_backward(H, E, ids, lg, None, w)
        assert torch.isnan(loss) and torch.isfinite(lse).all() and torch.isnan(dE).all(), t
        assert torch.isnan(dH[t]).all() and torch.isfinite(dH[rest]).all(), t
    off = torch.tensor([0, 5, 9, 14, T], dtype=torch.int32, device="cuda")
    ref = torch.tensor([0.0, 0.0, float("nan"), 0.0], device="cuda")
    loss, logp, lse, dH, dE = api.preference_forward_backward(H, E, ids[:, 0], off, ref)
    assert torch.isnan(loss) and torch.isfinite(logp).all() and torch.isfinite(lse).all() and torch.isnan(dE).all()
    assert torch.isfinite(dH[:9]).all() and torch.isnan(dH[9:]).all()
