"""Teacher logits of any finite size: the row's maximum is subtracted before the division by tau.

q = softmax(l / tau).  l is fp32 and given; l - max is rounded once (u = 2^-24 of itself), its product with the rounded
1 / tau twice more, and expf and the division add 4 u: a weight with |l - max| / tau <= 30 is off by at most
(4 * 30 + 8) u < 1e-5 of itself."""
import numpy as np
import pytest
import torch

from oracle import table_oracle as O
from vocabulary_label_bce_b200 import api

pytestmark = pytest.mark.gpu
LOW = float(np.finfo(np.float32).min)


def run(lg, tau):
    r = np.random.default_rng(62)
    T, K = lg.shape
    H = torch.from_numpy(r.standard_normal((T, 64)).astype(np.float32)).to(torch.bfloat16)
    E = torch.from_numpy((r.standard_normal((300, 64)) / 8).astype(np.float32)).to(torch.bfloat16)
    ids = np.stack([r.permutation(300)[:K] for _ in range(T)]).astype(np.int32)
    loss, lse, dH, dE = api.distill_forward_backward(H.cuda(), E.cuda(), torch.from_numpy(ids).cuda(),
                                                     torch.from_numpy(lg).cuda(), temperature=tau)
    return O.distill(H.double().numpy(), E.double().numpy(), ids, lg, tau=tau), float(loss), dH, dE, H, E


@pytest.mark.parametrize("tau", [0.5, 0.01, 4.0])
@pytest.mark.parametrize("top", [1e4, -1e6, 3e38, LOW])
def test_large_logits(top, tau):
    """Differences that fp32 can hold at that size, down to 20 tau below the top."""
    r = np.random.default_rng(63)
    lg = np.full((40, 5), top, np.float32)
    step = np.spacing(np.float32(min(abs(top), 3e38)))
    lg[:20, 1:] = (np.float64(top) - np.minimum(step * r.integers(0, 9, (20, 4)), 20 * tau)).astype(np.float32)
    lg[:20, 1:] = np.where(np.isfinite(lg[:20, 1:]), lg[:20, 1:], top)
    ref, loss, dH, dE, H, E = run(lg, tau)
    p, q = ref.p, ref.q
    zt = 2.0 ** -16 * (np.abs(H.double().numpy()) @ np.abs(E.double().numpy()).T).max()    # of a student's logit
    tol = (p * (2.0 ** -8 + 2 * zt / tau + 3e-4) + q * 1e-4) * ref.s * tau                 # as for ordinary logits
    for got, want, t in ((dH, ref.dH, tol @ np.abs(E.double().numpy())), (dE, ref.dE, tol.T @ np.abs(H.double().numpy()))):
        got = got.double().cpu().numpy()
        assert np.isfinite(got).all() and (np.abs(got - want) <= t + 1e-12).all()
    assert np.isfinite(loss) and abs(loss - ref.loss) <= tau * tau * (1e-4 + 2 * zt / tau) + 1e-5 * abs(ref.loss)


def test_one_slot_far_above_the_others():
    lg = np.array([[3e38, -3e38, 0.0], [LOW, LOW, -np.inf], [1.0, -3e38, 1.0]], np.float32)
    ref, loss, dH, dE, H, E = run(lg, 0.5)
    assert np.isfinite(ref.loss) and abs(loss - ref.loss) <= 1e-4 * (1 + abs(ref.loss))
    assert torch.isfinite(dH).all() and torch.isfinite(dE).all()
    assert np.linalg.norm(dH.double().cpu().numpy() - ref.dH) <= 2.0 ** -8 * np.linalg.norm(ref.dH)
