"""Refusals of the item-table operators, on the host and before any launch: the C
entries with arguments they reject, and the torch-facing calls."""
import ctypes

import pytest
import torch

from vocabulary_label_bce_b200 import api, binding as B

P = ctypes.c_void_p
FAKE, WS = 0x10000, 0x40000


def distill(**kw):
    p = B.cutbce_distill_problem(100, 1000, 64, 8, B.BF16, 0, FAKE, FAKE, FAKE, FAKE, None, None, 1.0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def preference(**kw):
    p = B.cutbce_preference_problem(100, 1000, 64, 5, B.BF16, 0, FAKE, FAKE, FAKE, FAKE, None, None, 0.1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


INV, UNS = B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED
COMMON = [("T", 0, INV), ("T", (1 << 24) - 255, UNS), ("V", 0, INV), ("V", (1 << 31) - 1, UNS), ("D", 0, INV),
          ("D", 60, UNS), ("D", 264, UNS), ("dtype", B.F32, UNS), ("reduction", 2, INV), ("reduction", -1, INV)]


@pytest.mark.parametrize("field,value,expect", COMMON + [
    ("K", 0, INV), ("K", 129, UNS), ("temperature", 0.0, INV), ("temperature", -1.0, INV),
    ("temperature", float("nan"), INV), ("temperature", float("inf"), INV), ("temperature", 1e-39, INV),
    ("temperature", 1e30, INV)])
def test_distill_problem_errors(field, value, expect):
    with pytest.raises(B.CutBCEError) as e:
        B.cutbce_distill_workspace_size(distill(**{field: value}), B.OUT_LOSS)
    assert e.value.status == expect


@pytest.mark.parametrize("field,value,expect", COMMON + [("P", 0, INV), ("P", 1 << 30, UNS), ("beta", float("nan"), INV),
                                                         ("beta", float("inf"), INV)])
def test_preference_problem_errors(field, value, expect):
    with pytest.raises(B.CutBCEError) as e:
        B.cutbce_preference_workspace_size(preference(**{field: value}), B.OUT_LOSS)
    assert e.value.status == expect


@pytest.mark.parametrize("make,size", [(distill, B.cutbce_distill_workspace_size),
                                       (preference, B.cutbce_preference_workspace_size)])
def test_workspace_sizes(make, size):
    p = make(T=12800, V=876000)
    loss = size(p, B.OUT_LOSS)
    both = size(p, B.OUT_LOSS | B.OUT_DH | B.OUT_DE)
    assert size(p, B.OUT_DH) < both and size(p, B.OUT_DE) < both and loss < both
    assert both < 12800 * 876000 * 4 / 50              # no T V term
    for bad in (0, 8, -1):
        with pytest.raises(B.CutBCEError) as e:
            size(p, bad)
        assert e.value.status == INV


def test_pairs_limit():
    with pytest.raises(B.CutBCEError) as e:            # T K is limited by the sort of the pairs
        B.cutbce_distill_workspace_size(distill(T=1 << 22, K=64), B.OUT_DE)
    assert e.value.status == UNS


def test_compute_calls_reject_before_launch():
    lib = B.load_library()
    d, p = distill(), preference()
    n = B.cutbce_distill_workspace_size(d, 7)
    m = B.cutbce_preference_workspace_size(p, 7)
    r = ctypes.byref
    big = 1 << 40
    assert lib.cutbce_distill_forward(None, FAKE, None, WS, big, None) == INV
    assert lib.cutbce_distill_forward(r(d), None, None, WS, big, None) == INV               # nothing wanted
    assert lib.cutbce_distill_forward(r(d), FAKE, None, None, big, None) == INV             # no workspace
    assert lib.cutbce_distill_forward(r(d), FAKE, None, WS + 16, big, None) == INV          # misaligned workspace
    assert lib.cutbce_distill_forward(r(d), FAKE + 4, None, WS, big, None) == INV           # misaligned loss
    assert lib.cutbce_distill_forward(r(d), FAKE, FAKE + 2, WS, big, None) == INV           # misaligned lse
    assert lib.cutbce_distill_forward_backward(r(d), None, None, FAKE, FAKE, FAKE, FAKE, WS, n // 2, None) == B.ERR_WORKSPACE
    assert lib.cutbce_preference_forward_backward(r(p), None, None, FAKE, FAKE, FAKE, FAKE, FAKE, WS, m // 2,
                                                  None) == B.ERR_WORKSPACE
    assert lib.cutbce_distill_backward(r(d), None, None, None, FAKE, FAKE, WS, big, None) == INV   # no lse
    assert lib.cutbce_distill_backward(r(d), None, FAKE, None, None, None, WS, big, None) == INV   # no gradient
    assert lib.cutbce_distill_backward(r(d), None, FAKE, None, FAKE + 8, None, WS, big, None) == INV
    for field, bad in (("H", FAKE + 8), ("E", FAKE + 2), ("H", None), ("E", None), ("ids", None), ("ids", FAKE + 1),
                       ("logits", None), ("logits", FAKE + 2), ("weights", FAKE + 2)):
        assert lib.cutbce_distill_forward(r(distill(**{field: bad})), FAKE, None, WS, big, None) == INV, field
    for field, bad in (("offsets", None), ("offsets", FAKE + 2), ("ref_logp", FAKE + 1)):
        assert lib.cutbce_preference_forward(r(preference(**{field: bad})), FAKE, None, None, WS, big, None) == INV, field
    for opts, expect in (((2, 0), UNS), ((0, 4), INV), ((0, -1), INV)):
        o = B.cutbce_grad_options(*opts)
        assert lib.cutbce_distill_forward_backward(r(d), r(o), None, FAKE, None, FAKE, None, WS, big, None) == expect
        assert lib.cutbce_preference_backward(r(p), r(o), FAKE, None, FAKE, None, WS, big, None) == expect


def test_embed_rejects_before_launch():
    lib = B.load_library()

    def fwd(E=FAKE, V=100, D=64, dtype=B.BF16, ids=FAKE, N=10, X=FAKE, status=None):
        return lib.cutbce_embed_forward(E, V, D, dtype, ids, N, 1.0, X, status, None)
    assert fwd(E=None) == fwd(ids=None) == fwd(X=None) == fwd(N=0) == fwd(V=0) == fwd(D=0) == fwd(D=-8) == INV
    assert fwd(E=FAKE + 1) == fwd(X=FAKE + 1) == fwd(ids=FAKE + 2) == fwd(status=FAKE + 1) == INV
    assert fwd(dtype=2) == fwd(D=16385) == fwd(N=1 << 28) == fwd(V=(1 << 31) - 1) == UNS
    n = B.cutbce_embed_workspace_size(10, 100, 64)

    def bwd(dX=FAKE, dtype=B.BF16, ids=FAKE, N=10, V=100, D=64, dE=FAKE, gd=0, acc=0, ws=WS, size=n):
        return lib.cutbce_embed_backward(dX, dtype, ids, N, V, D, 1.0, dE, gd, acc, ws, size, None)
    assert bwd(dX=None) == bwd(ids=None) == bwd(dE=None) == bwd(ws=None) == bwd(ws=WS + 16) == bwd(N=0) == INV
    assert bwd(dE=FAKE + 2) == bwd(dE=FAKE + 1, gd=1) == bwd(acc=2) == INV
    assert bwd(gd=2) == bwd(dtype=5) == bwd(N=1 << 28) == UNS
    assert bwd(size=n - 1) == B.ERR_WORKSPACE


def test_workspace_without_size():
    lib = B.load_library()
    assert lib.cutbce_embed_workspace_size(10, 100, 64, None) == INV
    assert lib.cutbce_distill_workspace_size(ctypes.byref(distill()), 1, None) == INV
    assert lib.cutbce_distill_workspace_size(None, 1, None) == INV
    assert lib.cutbce_preference_workspace_size(None, 1, None) == INV


def _cpu(T=4, V=9, D=16, K=2):
    H = torch.zeros(T, D, dtype=torch.bfloat16)
    E = torch.zeros(V, D, dtype=torch.bfloat16)
    return H, E, torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)


def test_torch_calls_refuse():
    H, E, ids, lg = _cpu()
    for call in (lambda: api.distill_forward(H, E, ids, lg), lambda: api.embed_forward(E, ids),
                 lambda: api.preference_forward(H, E, ids[:, 0], torch.tensor([0, 2, 4])),
                 lambda: api.embed_backward(H, ids[:, 0], 9)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="detach"):
        api.distill_loss(H, E, ids, lg.clone().requires_grad_())
    with pytest.raises(ValueError, match="detach"):
        api.preference_loss(H, E, ids[:, 0], torch.tensor([0, 2, 4]), torch.zeros(2, requires_grad=True))
    with pytest.raises(ValueError, match="accumulate needs out"):
        api.embed_backward(H, ids[:, 0], 9, accumulate=True)
    with pytest.raises(ValueError, match="dX must be"):
        api.embed_backward(H, ids[:2, 0], 9)
    with pytest.raises(ValueError, match="out must be"):
        api.embed_backward(H, ids[:, 0], 9, out=torch.zeros(8, 16))


def test_problem_makers_refuse():
    H, E, ids, lg = _cpu()
    make = B.make_distill_problem
    assert make(H, E, ids, lg).K == 2
    bad = [(H.float(), E, ids, lg), (H, E[:, :8], ids, lg), (H, E, ids.long(), lg), (H, E, ids, lg.double()),
           (H, E, ids, lg[:, :1]), (H, E, ids[:3], lg[:3]), (H.t().contiguous().t(), E, ids, lg),
           (H, E, ids[:, 0], lg[:, 0])]
    for args in bad:
        with pytest.raises(ValueError):
            make(*args)
    for kw in (dict(mask=torch.ones(4)), dict(mask=torch.ones(3, dtype=torch.uint8)), dict(weights=torch.ones(4).double()),
               dict(weights=torch.ones(5)), dict(reduction="mean_elements")):
        with pytest.raises(ValueError):
            make(H, E, ids, lg, **kw)
    pref = B.make_preference_problem
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    y = ids[:, 0].contiguous()
    assert pref(H, E, y, off).P == 1
    for args in ((H, E, y, off[:2]), (H, E, y, off[:1]), (H, E, y, off.long()), (H, E, y[:3], off),
                 (H, E, y, off, torch.zeros(3)), (H, E, y, off, torch.zeros(2).double())):
        with pytest.raises(ValueError):
            pref(*args)
    with pytest.raises(ValueError):
        B.make_grad_options(torch.zeros(4, 16), torch.zeros(9, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.make_grad_options(torch.zeros(4, 16, dtype=torch.float16), None)
    with pytest.raises(ValueError):
        B.make_grad_options(None, None)
