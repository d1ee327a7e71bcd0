"""A captured call replayed on other inputs gives the bits of an eager call on them: nothing is kept from one replay to
the next (counts of rows, targets, status, NaN notes)."""
import pytest
import torch

from vocabulary_label_bce_b200 import api

pytestmark = pytest.mark.gpu


def capture(call):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    return g, out


@pytest.mark.parametrize("T,V,K", [(70, 500, 3), (900, 4000, 40), (600, 16001, 5)])
def test_losses(T, V, K):
    gen = torch.Generator(device="cuda").manual_seed(80)
    H = torch.randn(T, 64, device="cuda", generator=gen).to(torch.bfloat16)
    E = (torch.randn(V, 64, device="cuda", generator=gen) / 8).to(torch.bfloat16)
    ids = torch.randint(0, V, (T, K), device="cuda", generator=gen).int()
    lg = torch.randn(T, K, device="cuda", generator=gen)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    w = torch.ones(T, device="cuda")
    off = torch.tensor([0, T // 3, T // 2, T - 4, T], dtype=torch.int32, device="cuda")
    y = ids[:, 0].clone()
    calls = (lambda: api.distill_forward_backward(H, E, ids, lg, mask, w, 1.5),
             lambda: api.preference_forward_backward(H, E, y, off, mask=mask, beta=0.2))
    graphs = [capture(c) for c in calls]

    def changes():
        yield lambda: None
        yield lambda: mask.copy_(torch.arange(T, device="cuda") % 3 != 0)
        yield lambda: (w.copy_(torch.randn(T, device="cuda", generator=gen)), off.copy_(torch.tensor([0, 0, 9, 9, T // 2])))
        yield lambda: mask.zero_()
        yield lambda: (mask.fill_(1), H[5, 3].fill_(float("nan")))
        yield lambda: (H.copy_(torch.randn_like(H)), ids[1, K - 1].fill_(V), y[2].fill_(-2))          # a data error
        yield lambda: (ids.copy_(ids % 7), y.copy_(y.abs() % 3))
        yield lambda: E.mul_(6)                                                                        # peaked rows
    for n, change in enumerate(changes()):
        change()
        for call, (graph, out) in zip(calls, graphs):
            graph.replay()
            want = call()
            torch.cuda.synchronize()
            bad = torch.isnan(want[0]) and n == 5
            assert torch.isnan(out[0]) if bad else all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) and
                                                       torch.equal(a.isnan(), b.isnan()) for a, b in zip(out, want)), n
            assert bool(torch.isnan(want[0])) == (n in (4, 5)), n


@pytest.mark.parametrize("N,V", [(300, 70), (40_000, 3000)])
def test_lookup_gradient(N, V):
    gen = torch.Generator(device="cuda").manual_seed(81)
    ids = torch.randint(-1, V, (N,), device="cuda", generator=gen).int()
    dX = torch.randn(N, 40, device="cuda", generator=gen)
    graph, out = capture(lambda: api.embed_backward(dX, ids, V))
    for change in (lambda: None, lambda: ids.copy_(ids % 5), lambda: ids[:9].fill_(V + 3), lambda: ids.fill_(-1),
                   lambda: ids.copy_(torch.randint(0, V, (N,), device="cuda", generator=gen))):
        change()
        graph.replay()
        assert torch.equal(out, api.embed_backward(dX, ids, V))
