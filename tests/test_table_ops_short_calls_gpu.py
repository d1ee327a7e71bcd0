"""Short calls on either side of the rules that choose how their rows are sorted out: T to 1,024 positions, T K to
16,384 slots, P to 1,024 pairs.  Neighbours give the same bits row by row, and a long list of slots costs no more than
its share."""
import pytest
import torch

from vocabulary_label_bce_b200 import api

pytestmark = pytest.mark.gpu


def draw(T, K, V=600, D=64):
    g = torch.Generator(device="cuda").manual_seed(70)
    H = torch.randn(T, D, device="cuda", generator=g).to(torch.bfloat16)
    E = (torch.randn(V, D, device="cuda", generator=g) / 8).to(torch.bfloat16)
    ids = torch.randint(-1, V, (T, K), device="cuda", generator=g).int()
    return H, E, ids, 2 * torch.randn(T, K, device="cuda", generator=g)


@pytest.mark.parametrize("K", [1, 15, 16, 17, 64, 128])
def test_rows_do_not_depend_on_the_length_of_the_call(K):
    H, E, ids, lg = draw(1100, K)
    mask = torch.arange(1100, device="cuda") % 7 != 0
    _, want = api.distill_forward(H, E, ids, lg, mask)
    for T in (16384 // K - 1, 16384 // K, 16384 // K + 1, 1000, 1024, 1025):
        if 0 < T <= 1100:
            _, lse = api.distill_forward(H[:T], E, ids[:T], lg[:T], mask[:T])
            assert torch.allclose(lse, want[:T], rtol=0, atol=2e-6 * 16), T
            assert torch.equal(lse == 0, want[:T] == 0), T


def device_ms(f):
    for _ in range(3):
        f()
    best = 1e9
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(20):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 20)
    return best


def test_many_slots_in_a_short_call():
    """One position more leaves the form of short calls: 1,024 positions of 128 slots took twice as long as 1,025."""
    H, E, ids, lg = draw(1025, 128, V=2048)
    short = device_ms(lambda: api.distill_forward(H[:1024], E, ids[:1024], lg[:1024]))
    longer = device_ms(lambda: api.distill_forward(H, E, ids, lg))
    assert short < 1.5 * longer, (short, longer)
