"""The lookup's gradient with ids out of range: it is the gradient of what the lookup gives (a zero row for such an
entry), and the status says that there was one."""
import numpy as np
import pytest
import torch

from vocabulary_label_bce_b200 import api, binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N,V,D", [(4, 50, 64), (3000, 700, 40), (20_000, 700, 7), (20_000, 300_000, 8),
                                   (200_000, 5000, 8), (4_200_000, 900, 8)])
def test_the_other_entries_keep_their_gradient(N, V, D, accumulate):
    g = torch.Generator(device="cuda").manual_seed(61)
    ids = (torch.rand(N, device="cuda", generator=g) ** 2 * V).int()
    good = ids.clone()
    at = torch.tensor([1, N // 2, N - 1], device="cuda")
    ids[at] = torch.tensor([V, -2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    good[at] = -1
    dX = torch.randn(N, D, device="cuda", generator=g)
    old = torch.randn(V, D, device="cuda", generator=g)
    ws = torch.empty(B.cutbce_embed_workspace_size(N, V, D), dtype=torch.uint8, device="cuda")

    def grad(i):
        return api.embed_backward(dX, i, V, scale=0.5, out=old.clone(), accumulate=accumulate, workspace=ws)
    want = grad(good)
    assert B.cutbce_read_status(ws) == 0 and want.any() and not torch.equal(want, old)
    assert torch.equal(grad(ids), want) and B.cutbce_read_status(ws) == B.ERR_TARGET_RANGE


def test_through_autograd():
    E = torch.randn(100, 64, device="cuda").requires_grad_()
    ids = torch.tensor([[3, 100, 7], [-1, 3, 2 ** 40]], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    X = api.embed(E, ids, 2.0, status=status)
    assert int(status) == B.ERR_TARGET_RANGE
    dX = torch.randn_like(X)
    X.backward(dX)
    want = torch.zeros_like(E)
    want[3] = 2 * (dX[0, 0] + dX[1, 1])
    want[7] = 2 * dX[0, 2]
    assert np.abs((E.grad - want).detach().cpu().numpy()).max() <= 4 * 2.0 ** -24 * 2 * float(dX.abs().max()) * 2
