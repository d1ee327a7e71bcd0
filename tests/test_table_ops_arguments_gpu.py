"""What the torch-facing losses take: offsets and masks of other types than the kernels'."""
import pytest
import torch

from vocabulary_label_bce_b200 import api

pytestmark = pytest.mark.gpu


def draw(T=30, V=100, D=64):
    g = torch.Generator(device="cuda").manual_seed(64)
    H = torch.randn(T, D, device="cuda", generator=g).to(torch.bfloat16)
    E = (torch.randn(V, D, device="cuda", generator=g) / 8).to(torch.bfloat16)
    return H, E, torch.randint(0, V, (T,), device="cuda", generator=g).int()


@pytest.mark.parametrize("bad", [2 ** 32, 2 ** 32 + 15, -2 ** 32, 2 ** 31, 2 ** 40 + 20])
def test_far_offsets_do_not_wrap(bad):
    H, E, y = draw()
    for at in range(3):
        off = torch.tensor([0, 15, 30], device="cuda")
        off[at] = bad
        assert torch.isnan(api.preference_forward(H, E, y, off)[0]), at


def test_offsets_are_integers():
    H, E, y = draw()
    want = api.preference_forward(H, E, y, torch.tensor([0, 15, 30], dtype=torch.int32, device="cuda"))
    for dt in (torch.int64, torch.int16, torch.uint8):
        got = api.preference_forward(H, E, y, torch.tensor([0, 15, 30], dtype=dt, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ValueError, match="integers"):
        api.preference_forward(H, E, y, torch.tensor([0.0, 15.0, 30.0], device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bool, torch.float32, torch.bfloat16, torch.int64, torch.int32])
def test_masks_of_any_type(dtype):
    """As for cut_bce, a mask of another type counts where it is not zero."""
    H, E, y = draw()
    m = torch.arange(30, device="cuda") % 3 != 0
    other = m.to(dtype) * (256 if dtype == torch.int64 else 1) if dtype != torch.bool else m
    off = torch.tensor([0, 15, 30], device="cuda")
    u8 = m.to(torch.uint8)
    for a, b in zip(api.preference_forward_backward(H, E, y, off, mask=other),
                    api.preference_forward_backward(H, E, y, off, mask=u8)):
        assert torch.equal(a, b)
    lg = torch.zeros(30, 1, device="cuda")
    for a, b in zip(api.distill_forward_backward(H, E, y[:, None], lg, other),
                    api.distill_forward_backward(H, E, y[:, None], lg, u8)):
        assert torch.equal(a, b)
    loss = api.distill_loss(H.requires_grad_(), E, y[:, None], lg, other)
    loss.backward()
    assert torch.equal(H.grad != 0, m[:, None].expand(30, 64))
