"""The item-table operators where element offsets pass 32 bits: V D > 2^31.

The oracle is the float64 formula, formed on the device over pieces of the table.  Tolerances as in
test_table_ops_gpu.py, with what a table this long adds: a thread sums up to V / 148 / 4 = 14,200
exponentials (14,200 u = 8.5e-4 of the row's sum, so of p), and a CTA's share of dH has up to
V / 148 = 56,800 terms (3.4e-3).
"""
import pytest
import torch

from vocabulary_label_bce_b200 import api

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8
V, D, T, K = 8_400_005, 256, 33, 5
PIECE = 600_000


@pytest.fixture(scope="module")
def table():
    g = torch.Generator(device="cuda").manual_seed(40)
    E = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for v in range(0, V, PIECE):
        E[v:v + PIECE] = torch.randn(min(PIECE, V - v), D, device="cuda", generator=g) / 16
    yield E
    del E
    torch.cuda.empty_cache()


def pieces(E):
    for v in range(0, len(E), PIECE):
        yield v, E[v:v + PIECE].double()


def test_distillation(table):
    g = torch.Generator(device="cuda").manual_seed(41)
    H = torch.randn(T, D, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randint(0, V, (T, K), device="cuda", generator=g).int()
    ids[0, :3] = torch.tensor([V - 1, V - 2, 2 ** 31 // D], device="cuda")
    ids[1, 0] = V - 1
    lg = torch.randn(T, K, device="cuda", generator=g)
    loss, lse, dH, dE = api.distill_forward_backward(H, table, ids, lg)

    h, q = H.double(), torch.softmax(lg.double(), 1)
    zs = [h @ e.T for _, e in pieces(table)]
    want_lse = torch.logsumexp(torch.stack([torch.logsumexp(z, 1) for z in zs]), 0)
    zt = 2.0 ** -16 * torch.stack([(h.abs() @ e.abs().T).amax(1) for _, e in pieces(table)]).amax(0)
    lt = zt + 4e-5 + 8.5e-4 + 4 * U * want_lse.abs()
    assert ((lse.double() - want_lse).abs() <= lt).all()
    zk = (h[:, None, :] * table[ids.long()].double()).sum(2)
    want_loss = (q * (q.log() - zk + want_lse[:, None])).sum(1).mean()
    assert abs(float(loss) - float(want_loss)) <= float((2 * lt + 1e-4).mean())

    r = (zt + lt + 2e-4)[:, None]
    sparse_rows, inv = torch.unique(ids.long().reshape(-1), return_inverse=True)
    pairs = (q.reshape(-1, 1) / T) * h.repeat_interleave(K, 0)
    sparse = torch.zeros(len(sparse_rows), D, dtype=torch.float64, device="cuda").index_add_(0, inv, pairs)
    sparse_abs = torch.zeros_like(sparse).index_add_(0, inv, pairs.abs())
    want_dH, tol_dH = torch.zeros(T, D, dtype=torch.float64, device="cuda"), 0
    for (v, e), z in zip(pieces(table), zs):
        p = torch.exp(z - want_lse[:, None]) / T
        want_dH += p @ e
        tol_dH = tol_dH + (p * (BF + r + 3.4e-3)) @ e.abs()
        want, tol = p.T @ h, (p * (BF + r)).T @ h.abs()
        here = (sparse_rows >= v) & (sparse_rows < v + len(e))
        want.index_add_(0, sparse_rows[here] - v, -sparse[here])
        tol.index_add_(0, sparse_rows[here] - v, 1e-4 * sparse_abs[here])
        err = (dE[v:v + len(e)].double() - want).abs()
        assert (err <= tol + 4 * U * want.abs() + 1e-30).all(), v
    qe = (q[:, :, None] / T) * table[ids.long()].double()
    want_dH -= qe.sum(1)
    tol_dH = tol_dH + 1e-4 * qe.abs().sum(1) + 4 * U * want_dH.abs()
    assert ((dH.double() - want_dH).abs() <= tol_dH).all()


def test_lookup_and_its_gradient(table):
    g = torch.Generator(device="cuda").manual_seed(42)
    ids = torch.randint(V - 400, V, (500,), device="cuda", generator=g).int()
    ids[:5] = torch.tensor([0, V - 1, 2 ** 31 // D - 1, 2 ** 31 // D, -1], device="cuda")
    X = api.embed_forward(table, ids)
    assert torch.equal(X[:4], table[ids[:4].long()]) and not X[4].any() and torch.equal(X[5:], table[ids[5:].long()])
    dX = torch.randn(500, D, device="cuda", generator=g)
    dE = api.embed_backward(dX, ids, V)
    real = ids >= 0
    rows, inv, n = torch.unique(ids[real].long(), return_inverse=True, return_counts=True)
    want = torch.zeros(len(rows), D, dtype=torch.float64, device="cuda").index_add_(0, inv, dX[real].double())
    size = torch.zeros_like(want).index_add_(0, inv, dX[real].abs().double())
    assert ((dE[rows].double() - want).abs() <= U * (n[:, None] + 2) * size + U * want.abs()).all()
    dE[rows] = 0
    assert not any(dE[v:v + PIECE].any() for v in range(0, V, PIECE))


@pytest.mark.parametrize("V", [1, 900, 40_000, 5_000_000])
@pytest.mark.parametrize("N", [16_384, 16_385, 131_072, 131_073, 262_145, 1_000_003, 4_194_305])
def test_many_entries(N, V):
    """Sizes at which the sort takes another form.  A sum of fp32 terms is off by at most u times its
    longest chain of additions, of the sum of their sizes; the chains here are far shorter than
    N / 64 + 4096."""
    g = torch.Generator(device="cuda").manual_seed(43)
    ids = (torch.rand(N, device="cuda", generator=g) ** 3 * V).int()
    ids[::17] = -1
    dX = torch.randn(N, 8, device="cuda", generator=g)
    dE = api.embed_backward(dX, ids, V, out=torch.full((V, 8), float("nan"), device="cuda"))
    real = ids >= 0
    rows = ids[real].long()
    want = torch.zeros(V, 8, dtype=torch.float64, device="cuda").index_add_(0, rows, dX[real].double())
    size = torch.zeros(V, 8, dtype=torch.float64, device="cuda").index_add_(0, rows, dX[real].double().abs())
    assert ((dE.double() - want).abs() <= U * (N / 64 + 4096) * size).all()
    assert torch.equal(dE, api.embed_backward(dX, ids, V))
