"""The item-table operators on the GPU against their float64 oracle.

Tolerances.  u = 2^-24 (half a step of fp32), b = 2^-8 (half a step of bf16).
 * A logit is an fp32 sum of at most 256 products: |dz| <= zt = 2^-16 max_v sum_d |h_d e_vd|.
 * lse is 1-Lipschitz in the logits; 2^x carries at most 2.7e-6 (FMA-pipe polynomial; the SFU's
   2^x is within 2^-22) and the rounding of its argument, at most 2^-23 |x| ln 2 with |x| <= 150
   where a term matters: 1.3e-5; the sums add fewer than 256 values a thread here: 256 u = 1.6e-5.
   With the final roundings |dlse| <= lt = zt / tau + 4e-5 + 4 u |lse|.
 * p: relative error r = zt / tau + lt + 1e-4 (polynomial 7.5e-5, argument 1.3e-5) before bf16,
   then b.  The dense sum over v (or t) of |p e| (|p h|) is therefore off by at most
   (b + r + 1e-4) of itself (the last term: fp32 accumulation of at most 1200 terms, 7.2e-5), the
   sparse sum by at most 1e-4 of itself (q: expf and a division, 1e-5 for logits up to 40).
   The output adds u, or b when it is bf16; preference factors add |dx| from the log-probabilities.
Everything is checked element by element against these bounds.
"""
import numpy as np
import pytest
import torch

from oracle import table_oracle as O
from vocabulary_label_bce_b200 import api, binding as B

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(x):
    """float64 values of x rounded to bf16, and the device tensor."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def host(t):
    return t.double().cpu().numpy()


def bounds(ref, H, E, tau, bits):
    """Tolerances of lse, dH and dE (see above); H with the rows that do not count zeroed."""
    zt = 2.0 ** -16 * (np.abs(ref.H) @ np.abs(E).T).max(1) if len(E) else 0
    lt = zt / tau + 4e-5 + 4 * U * np.abs(ref.lse)
    r = zt / tau + lt + 2e-4
    out = BF if bits == 16 else 4 * U
    return SimpleTol(zt, lt, r, out)


class SimpleTol:
    def __init__(self, zt, lt, r, out):
        self.zt, self.lt, self.r, self.out = zt, lt, r, out

    def dH(self, ref, E, scale, extra):
        w = np.abs(ref.w)[:, None] * scale
        e = np.abs(E)
        return w * ((ref.p @ e) * (BF + self.r[:, None]) + (ref.q @ e) * 1e-4 + extra[:, None] * ((ref.p + ref.q) @ e)) + self.out * np.abs(ref.dH) + 1e-30

    def dE(self, ref, scale, extra):
        w = np.abs(ref.w)[:, None] * scale
        h = np.abs(ref.H)
        return (w * ref.p * (BF + self.r[:, None])).T @ h + (w * ref.q * 1e-4).T @ h + (w * extra[:, None] * (ref.p + ref.q)).T @ h + self.out * np.abs(ref.dE) + 1e-30


def close(got, want, tol, what):
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)), what
    worst = np.max(err / tol) if err.size else 0.0
    assert worst <= 1.0, (what, worst, float(err.max()))
    return worst


# ---------------------------------------------------------------- distillation
def draw_distill(T, V, D, K, seed, h=1.0, mask=None, weights=None, holes=True):
    r = np.random.default_rng(seed)
    Hf, H = bf16(h * r.standard_normal((T, D)))
    Ef, E = bf16(r.standard_normal((V, D)) / np.sqrt(D))
    ids = r.integers(0, V, (T, K)).astype(np.int32)
    lg = (2.0 * r.standard_normal((T, K)) + 3.0).astype(np.float32)
    if holes:
        ids[r.random((T, K)) < 0.15] = -1
        lg[r.random((T, K)) < 0.05] = -np.inf
        lg[ids < 0] = np.nan                              # an empty slot's logit is not looked at
    m = None
    if mask == "random":
        m = (r.random(T) < 0.8).astype(np.uint8)
    elif mask == "none":
        m = np.zeros(T, np.uint8)
    w = None
    if weights == "mixed":
        w = r.uniform(-2, 2, T).astype(np.float32)
        w[::7] = 0.0
    elif weights == "negative":
        w = -r.uniform(0.5, 2, T).astype(np.float32)
    if m is not None:                                     # what masked rows hold is not looked at
        Hf[m == 0] = np.nan
        H = dev(Hf).to(torch.bfloat16)
        ids[m == 0] = 2 ** 31 - 1
        lg[m == 0] = np.inf
        Hf = np.where((m == 0)[:, None], 0.0, Hf)
    return Hf, H, Ef, E, ids, lg, m, w


def check_distill(c, tau=1.0, reduction="mean", g=None, bits=32, entry="fused"):
    Hf, H, Ef, E, ids, lg, m, w = c
    ref = O.distill(Hf, Ef, ids, np.where(ids >= 0, lg, 0.0), m, w, tau, reduction, 1.0 if g is None else g)
    args = (H, E, dev(ids), dev(lg), None if m is None else dev(m), None if w is None else dev(w))
    kw = dict(temperature=tau, reduction=reduction, grad_loss=None if g is None else torch.tensor(g, device="cuda"),
              grad_dtype=torch.bfloat16 if bits == 16 else torch.float32)
    if entry == "fused":
        loss, lse, dH, dE = api.distill_forward_backward(*args, **kw)
    else:
        loss, lse = api.distill_forward(*args, temperature=tau, reduction=reduction)
        dH, dE = api.distill_backward(*args[:4], lse, *args[4:], **kw)
    t = bounds(ref, Hf, Ef, tau, bits)
    V = ref.valid
    close(host(lse)[V], ref.lse[V], t.lt[V], "lse")
    assert np.all(host(lse)[~V] == 0)
    assert abs(float(loss) - ref.loss) <= tau * tau * ref.s * (np.abs(ref.w) * (2 * t.lt + 1e-4))[V].sum() + 1e-6 * abs(ref.loss) + 1e-30
    scale = abs(1.0 if g is None else g) * ref.s * tau
    close(host(dH), ref.dH, t.dH(ref, Ef, scale, np.zeros(len(Hf))), "dH")
    assert np.all(host(dH)[~V] == 0)
    close(host(dE), ref.dE, t.dE(ref, scale, np.zeros(len(Hf))), "dE")
    return ref, loss, lse, dH, dE


DISTILL = [
    dict(T=1, V=1, D=8, K=1), dict(T=1, V=2, D=64, K=2), dict(T=3, V=127, D=40, K=5), dict(T=129, V=129, D=72, K=7),
    dict(T=128, V=128, D=64, K=128), dict(T=200, V=1000, D=128, K=16, mask="random"),
    dict(T=257, V=2049, D=136, K=33, mask="random", weights="mixed"), dict(T=130, V=640, D=192, K=3, weights="mixed"),
    dict(T=300, V=1537, D=256, K=16, mask="random", weights="negative"), dict(T=64, V=3000, D=200, K=4, weights="mixed"),
    dict(T=513, V=5000, D=64, K=8, mask="random", weights="mixed"), dict(T=40, V=20000, D=64, K=16),
]


@pytest.mark.parametrize("entry", ["fused", "split"])
@pytest.mark.parametrize("case", DISTILL, ids=lambda c: "_".join(f"{k}{v}" for k, v in c.items()))
def test_distill_matches_oracle(case, entry):
    check_distill(draw_distill(seed=5, **case), tau=1.0, entry=entry)


@pytest.mark.parametrize("tau,reduction,g,bits", [(0.5, "sum", None, 32), (3.0, "mean", -2.5, 16), (1.3, "sum", 0.25, 16)])
def test_distill_options(tau, reduction, g, bits):
    check_distill(draw_distill(T=150, V=700, D=64, K=6, seed=6, mask="random", weights="mixed"), tau, reduction, g, bits)


@pytest.mark.parametrize("entry", ["fused", "split"])
@pytest.mark.parametrize("D,h", [(64, 30.0), (256, 12.0), (64, 8.0), (128, 60.0)])
def test_distill_large_logits(D, h, entry):
    # peaked rows whose bound lies far above their largest logit: the log-sum-exp pass gives the
    # reference (at 1.0e6 logits and more the fused call takes the row sums in its dH pass)
    check_distill(draw_distill(T=140, V=8000, D=D, K=4, seed=7, h=h), entry=entry)


def test_distill_large_problem_takes_the_row_sums():
    c = draw_distill(T=260, V=9000, D=64, K=8, seed=8, mask="random", weights="mixed")
    a = check_distill(c, entry="fused")
    b = check_distill(c, entry="split")
    assert torch.allclose(a[2], b[2], rtol=0, atol=4e-5)


# from 8e6 logits on the dH pass takes the row sums itself, with a bound as reference
FUSED = [dict(T=520, V=16001, D=64, K=8), dict(T=520, V=16001, D=64, K=8, mask="random", weights="mixed"),
         dict(T=700, V=15003, D=72, K=5, mask="random"), dict(T=640, V=15000, D=200, K=3, weights="negative"),
         dict(T=600, V=16100, D=256, K=4, mask="random", weights="mixed")]


@pytest.mark.parametrize("h", [1.0, 30.0])
@pytest.mark.parametrize("case", FUSED, ids=lambda c: "_".join(f"{k}{v}" for k, v in c.items()))
def test_distill_with_row_sums_in_the_dh_pass(case, h):
    # h = 30: the bound lies more than 70 (log2) above the logits, so the log-sum-exp pass runs first
    check_distill(draw_distill(seed=33, h=h, **case), tau=1.2)


@pytest.mark.parametrize("how", ["masked", "zero weight", "empty slots", "infinite logits"])
def test_distill_nothing_counts(how):
    c = list(draw_distill(T=70, V=300, D=64, K=3, seed=9, holes=False))
    if how == "masked":
        c[6] = np.zeros(70, np.uint8)
        c[4][:] = 2 ** 31 - 1
    elif how == "zero weight":
        c[7] = np.zeros(70, np.float32)
    elif how == "empty slots":
        c[4][:] = -1
    else:
        c[5][:] = -np.inf
    ref, loss, lse, dH, dE = check_distill(tuple(c))
    assert float(loss) == 0 and not ref.valid.any() and not dE.any() and not dH.any() and not lse.any()


def test_distill_bad_teacher_value_stays_in_its_terms():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=20, V=100, D=64, K=3, seed=10, holes=False)
    lg[4, 1] = np.nan
    loss, lse, dH, dE = api.distill_forward_backward(H, E, dev(ids), dev(lg))
    assert torch.isnan(loss) and torch.isnan(dH[4]).all() and torch.isfinite(lse).all()
    rows = [t for t in range(20) if t != 4]
    assert torch.isfinite(dH[rows]).all()


@pytest.mark.parametrize("bad", [-2, 100, 2 ** 31 - 1, -2 ** 31])
def test_distill_reports_bad_ids(bad):
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=20, V=100, D=64, K=3, seed=11, holes=False)
    ids[7, 2] = bad
    di, dl = dev(ids), dev(lg)                             # a problem holds pointers, not its tensors
    p = B.make_distill_problem(H, E, di, dl)
    ws = torch.empty(B.cutbce_distill_workspace_size(p, 7), dtype=torch.uint8, device="cuda")
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    B.cutbce_distill_forward(p, loss, None, ws)
    assert B.cutbce_read_status(ws) == B.ERR_TARGET_RANGE
    dH, dE = torch.empty(20, 64, device="cuda"), torch.empty(100, 64, device="cuda")
    B.cutbce_distill_forward_backward(p, None, None, loss, None, dH, dE, ws)
    assert B.cutbce_read_status(ws) == B.ERR_TARGET_RANGE
    torch.cuda.synchronize()


# ---------------------------------------------------------------- preference
def draw_preference(lengths, V, D, seed, first=0, extra=0, h=1.0, mask=False, holes=True):
    r = np.random.default_rng(seed)
    off = O.offsets_of(lengths, first)
    T = int(off[-1]) + extra
    Hf, H = bf16(h * r.standard_normal((T, D)))
    Ef, E = bf16(r.standard_normal((V, D)) / np.sqrt(D))
    ids = r.integers(0, V, T).astype(np.int32)
    if holes and T > 3:
        ids[r.random(T) < 0.1] = -1
    m = (r.random(T) < 0.85).astype(np.uint8) if mask else None
    if m is not None:
        ids[m == 0] = -7
        Hf[m == 0] = np.nan
        H = dev(Hf).to(torch.bfloat16)
        Hf = np.where((m == 0)[:, None], 0.0, Hf)
    ref = (-np.log(V) * np.asarray(lengths) + r.standard_normal(len(lengths))).astype(np.float32)
    return Hf, H, Ef, E, ids, off, ref, m


def check_preference(c, beta=0.1, reduction="mean", g=None, bits=32, entry="fused", with_ref=True):
    Hf, H, Ef, E, ids, off, rl, m = c
    rl = rl if with_ref else None
    ref = O.preference(Hf, Ef, np.where(ids < 0, -1, ids), off, rl, m, beta, reduction, 1.0 if g is None else g)
    args = (H, E, dev(ids))
    kw = dict(offsets=dev(off), ref_logp=None if rl is None else dev(rl), mask=None if m is None else dev(m), beta=beta,
              reduction=reduction)
    gk = dict(grad_loss=None if g is None else torch.tensor(g, device="cuda"),
              grad_dtype=torch.bfloat16 if bits == 16 else torch.float32)
    if entry == "fused":
        loss, logp, lse, dH, dE = api.preference_forward_backward(*args, **kw, **gk)
    else:
        loss, logp, lse = api.preference_forward(*args, **kw)
        dH, dE = api.preference_backward(*args, lse, **kw, **gk)
    t = bounds(ref, Hf, Ef, 1.0, bits)
    V = ref.valid
    close(host(lse)[V], ref.lse[V], t.lt[V], "lse")
    assert np.all(host(lse)[~V] == 0)
    seq = np.full(len(Hf), -1)
    for i in range(len(off) - 1):
        seq[off[i]:off[i + 1]] = i
    lt = np.array([(t.lt + t.zt)[(seq == i) & V].sum() for i in range(len(off) - 1)])
    close(host(logp), ref.logp, lt + 4 * U * np.abs(ref.logp) + 1e-30, "logp")
    xt = abs(beta) * (lt[0::2] + lt[1::2] + 4 * U * (0 if rl is None else np.abs(rl[0::2]) + np.abs(rl[1::2])))
    assert abs(float(loss) - ref.loss) <= ref.s * xt.sum() + 1e-6 * abs(ref.loss) + 1e-30
    # sigmoid(-x) changes by at most a factor e^|dx|
    extra = np.array([np.expm1(xt[s // 2]) if s >= 0 else 0.0 for s in seq]) + 1e-6
    scale = abs(1.0 if g is None else g) * ref.s * abs(beta)
    close(host(dH), ref.dH, t.dH(ref, Ef, scale, extra), "dH")
    assert np.all(host(dH)[~V] == 0)
    close(host(dE), ref.dE, t.dE(ref, scale, extra), "dE")
    return ref, loss, logp, lse, dH, dE


PREF = [
    dict(lengths=[1, 1], V=1, D=8), dict(lengths=[1, 0], V=50, D=64), dict(lengths=[0, 0, 3, 5], V=129, D=40),
    dict(lengths=[0, 0], V=10, D=64, extra=4), dict(lengths=[127, 129], V=300, D=64),
    dict(lengths=[128, 128, 64, 1], V=1000, D=128, mask=True), dict(lengths=[200, 3], V=2049, D=256, first=5, extra=9),
    dict(lengths=[7] * 40, V=777, D=136, mask=True), dict(lengths=[300, 17, 0, 90, 45, 45], V=5000, D=192, mask=True),
    dict(lengths=[100, 100], V=20000, D=64, first=3, mask=True),
]


@pytest.mark.parametrize("entry", ["fused", "split"])
@pytest.mark.parametrize("case", PREF, ids=lambda c: f"L{len(c['lengths'])}_T{sum(c['lengths'])}_V{c['V']}_D{c['D']}")
def test_preference_matches_oracle(case, entry):
    check_preference(draw_preference(seed=12, **case), entry=entry)


@pytest.mark.parametrize("beta,reduction,g,bits,with_ref", [(0.5, "sum", None, 16, True), (2.0, "mean", -1.5, 32, False),
                                                             (-0.3, "mean", 3.0, 16, True), (0.0, "sum", None, 32, True)])
def test_preference_options(beta, reduction, g, bits, with_ref):
    c = draw_preference([20, 25, 60, 13], V=600, D=64, seed=13, mask=True)
    check_preference(c, beta, reduction, g, bits, with_ref=with_ref)


def test_preference_large_logits():
    check_preference(draw_preference([70, 60], V=9000, D=64, seed=14, h=30.0), beta=0.01)
    check_preference(draw_preference([70, 60], V=9000, D=256, seed=15, h=12.0), beta=0.01, entry="split")


@pytest.mark.parametrize("D,h", [(64, 1.0), (64, 30.0), (136, 1.0), (256, 12.0)])
def test_preference_with_row_sums_in_the_dh_pass(D, h):
    check_preference(draw_preference([150, 130, 0, 100, 120, 97], V=16001, D=D, seed=34, h=h, mask=True), beta=0.02)


def test_nothing_counts_in_a_large_problem():
    c = list(draw_distill(T=530, V=16000, D=64, K=2, seed=35, holes=False))
    c[6] = np.zeros(530, np.uint8)
    ref, loss, lse, dH, dE = check_distill(tuple(c))
    assert float(loss) == 0 and not dE.any() and not dH.any()


def test_preference_far_apart_pairs():
    # x far from zero on both sides: loss near -x and near 0, factors 1 and (almost) 0
    c = list(draw_preference([4, 4, 4, 4, 4, 4], V=100, D=64, seed=16, holes=False))
    c[6] = np.array([0, 0, 4000, 0, 0, 4000], np.float32)
    check_preference(tuple(c), beta=0.5)


def test_preference_padded_batch_equals_packed():
    Hf, H, Ef, E, ids, off, rl, m = draw_preference([6, 6, 6, 6], V=90, D=64, seed=17)
    a = api.preference_forward_backward(H, E, dev(ids), dev(off), dev(rl))
    b = api.preference_forward_backward(H.view(4, 6, 64), E, dev(ids).view(4, 6), None, dev(rl))
    assert b[2].shape == (4, 6) and b[3].shape == (4, 6, 64)
    for x, y in zip(a, b):
        assert torch.equal(x.reshape(-1), y.reshape(-1))


@pytest.mark.parametrize("how", ["descending", "negative", "past the end", "id"])
def test_preference_reports_bad_data(how):
    Hf, H, Ef, E, ids, off, rl, m = draw_preference([6, 6, 6, 6], V=90, D=64, seed=18, holes=False)
    if how == "descending":
        off[2] = 3
    elif how == "negative":
        off[0] = -4
    elif how == "past the end":
        off[-1] = 2 ** 31 - 1
    else:
        ids[11] = 90
    di, do, dr = dev(ids), dev(off), dev(rl)
    p = B.make_preference_problem(H, E, di, do, dr)
    ws = torch.empty(B.cutbce_preference_workspace_size(p, 7), dtype=torch.uint8, device="cuda")
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    dH, dE = torch.empty(24, 64, device="cuda"), torch.empty(90, 64, device="cuda")
    B.cutbce_preference_forward_backward(p, None, None, loss, None, None, dH, dE, ws)
    assert B.cutbce_read_status(ws) == B.ERR_TARGET_RANGE
    torch.cuda.synchronize()


# ---------------------------------------------------------------- lookup
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (1, 5, 64), (64, 1000, 64), (77, 10, 7), (1000, 333, 200), (5, 9, 2050)])
def test_embed_forward(N, V, D, dtype):
    r = np.random.default_rng(20)
    E = dev(r.standard_normal((V, D)).astype(np.float32)).to(dtype)
    ids = r.integers(-1, V, N).astype(np.int32)
    X = api.embed_forward(E, dev(ids), scale=3.3)
    want = O.embed(host(E), ids, float(np.float32(3.3)))
    close(host(X), want, (BF if dtype == torch.bfloat16 else U) * np.abs(want) + U * np.abs(want) + 1e-38, "X")


def test_embed_forward_odd_bases_shapes_and_bad_ids():
    r = np.random.default_rng(21)
    flat = dev(r.standard_normal(1 + 50 * 64).astype(np.float32))
    E = flat[1:].view(50, 64)                             # rows start 4 bytes off a 16-byte boundary
    ids = dev(r.integers(0, 50, (3, 4)).astype(np.int64))
    assert torch.equal(api.embed_forward(E, ids), E[ids])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    X = api.embed_forward(E, torch.tensor([3, 50, -2, 2 ** 40, -1], device="cuda"), status=status)
    assert int(status) == B.ERR_TARGET_RANGE and torch.equal(X[0], E[3]) and not X[1:].any()
    assert api.embed_forward(E, ids[:0]).shape == (0, 4, 64)
    assert torch.equal(api.embed_forward(E.t().contiguous().t(), ids), E[ids])


EMBED_GRAD = [
    dict(N=1, V=1, D=1), dict(N=1, V=7, D=64), dict(N=33, V=1, D=64), dict(N=1000, V=10, D=64), dict(N=1025, V=2048, D=8),
    dict(N=777, V=2047, D=7), dict(N=5000, V=100000, D=64), dict(N=4096, V=5000000, D=8), dict(N=70000, V=500, D=24),
    dict(N=3000, V=40, D=256), dict(N=700, V=30, D=1100), dict(N=1100003, V=3000, D=4), dict(N=2300000, V=70000, D=8),
]


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                       (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("case", EMBED_GRAD, ids=lambda c: f"N{c['N']}_V{c['V']}_D{c['D']}")
def test_embed_backward(case, dtype, out):
    N, V, D = case["N"], case["V"], case["D"]
    r = np.random.default_rng(22)
    ids = np.minimum((V * r.random(N) ** 3).astype(np.int32), V - 1)      # the small ids are hot
    ids[r.random(N) < 0.05] = -1
    dX = dev(r.standard_normal((N, D)).astype(np.float32)).to(dtype)
    dE = api.embed_backward(dX, dev(ids), V, scale=0.7, grad_dtype=out)
    x = host(dX)
    s = float(np.float32(0.7))
    want, absum = O.embed_grad(x, ids, V, s), O.embed_grad(np.abs(x), ids, V, s)
    # an fp32 sum of n terms, at most n - 1 additions deep, then the factor and one rounding
    n = np.bincount(ids[ids >= 0], minlength=V)[:, None]
    close(host(dE), want, U * (n + 2) * absum + (BF if out == torch.bfloat16 else U) * np.abs(want) + 1e-38, "dE")
    assert torch.equal(dE, api.embed_backward(dX, dev(ids), V, scale=0.7, grad_dtype=out))     # the same bits again


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_embed_backward_accumulates(out):
    r = np.random.default_rng(23)
    N, V, D = 900, 400, 64
    ids = r.integers(0, 100, N).astype(np.int32)
    dX = dev(r.standard_normal((N, D)).astype(np.float32)).to(torch.bfloat16)
    old = dev(r.standard_normal((V, D)).astype(np.float32)).to(out)
    got = api.embed_backward(dX, dev(ids), V, out=old.clone(), accumulate=True)
    plain = api.embed_backward(dX, dev(ids), V, grad_dtype=torch.float32)
    assert torch.equal(got, (old.float() + plain).to(out))                 # the fp32 sum, added and rounded once
    assert torch.equal(got[100:], old[100:])
    fresh = torch.full((V, D), float("nan"), dtype=out, device="cuda")
    assert torch.equal(api.embed_backward(dX, dev(ids), V, out=fresh), plain.to(out))


def test_embed_backward_edges():
    dX = torch.randn(4, 64, device="cuda")
    none = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    assert not api.embed_backward(dX, none, 50).any()
    old = torch.randn(50, 64, device="cuda")
    assert torch.equal(api.embed_backward(dX, none, 50, out=old.clone(), accumulate=True), old)
    assert not api.embed_backward(dX[:0], none[:0], 50, out=old.clone()).any()
    assert torch.equal(api.embed_backward(dX[:0], none[:0], 50, out=old.clone(), accumulate=True), old)
    ws = torch.empty(B.cutbce_embed_workspace_size(4, 50, 64), dtype=torch.uint8, device="cuda")
    bad = torch.tensor([1, 2, 50, 3], dtype=torch.int32, device="cuda")
    B.cutbce_embed_backward(dX, bad, torch.empty(50, 64, device="cuda"), ws)
    assert B.cutbce_read_status(ws) == B.ERR_TARGET_RANGE
    base = torch.randn(1 + 4 * 64, device="cuda")
    odd = base[1:].view(4, 64)                                             # rows off the 16-byte boundary
    ids = torch.tensor([3, 3, 0, 3], dtype=torch.int32, device="cuda")
    assert torch.equal(api.embed_backward(odd, ids, 5), api.embed_backward(odd.clone(), ids, 5))


# ---------------------------------------------------------------- as they are used
def test_accumulate_into_outputs():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=100, V=500, D=64, K=4, seed=24, mask="random")
    p = B.make_distill_problem(H, E, *(keep := (dev(ids), dev(lg), dev(m))))
    ws = torch.empty(B.cutbce_distill_workspace_size(p, 7), dtype=torch.uint8, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        dH, dE = torch.empty(100, 64, device="cuda"), torch.empty(500, 64, device="cuda")
        B.cutbce_distill_forward_backward(p, None, None, None, None, dH, dE, ws)
        oH, oE = torch.randn(100, 64, device="cuda").to(dt), torch.randn(500, 64, device="cuda").to(dt)
        aH, aE = oH.clone(), oE.clone()
        B.cutbce_distill_forward_backward(p, B.make_grad_options(aH, aE, 3), None, None, None, aH, aE, ws)
        assert torch.equal(aH, (oH.float() + dH).to(dt)) and torch.equal(aE, (oE.float() + dE).to(dt))
    assert keep


def test_one_gradient_alone_and_repeats_give_the_same_bits():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=300, V=7000, D=64, K=4, seed=25, mask="random", weights="mixed")
    args = (H, E, dev(ids), dev(lg), dev(m), dev(w))
    loss, lse, dH, dE = api.distill_forward_backward(*args)
    for _ in range(3):
        again = api.distill_forward_backward(*args)
        assert all(torch.equal(x, y) for x, y in zip((loss, lse, dH, dE), again))
    only = api.distill_forward_backward(*args, want_dE=False)
    assert only[3] is None and torch.equal(only[2], dH) and torch.equal(only[0], loss)
    l2, lse2 = api.distill_forward(*args)
    _, _, none, dE2 = api.distill_forward_backward(*args, want_dH=False)
    _, dE3 = api.distill_backward(*args[:4], lse2, *args[4:], want_dH=False)
    # the lse handed over is in natural units: back in the log2 domain it may be two fp32 steps
    # (2^-22 |lse|) off, which moves p by about 1e-6 and may flip roundings of p to bf16
    for other in (dE2, dE3):
        assert none is None and torch.allclose(other, dE, rtol=2 * BF, atol=1e-6)


def test_autograd_matches_the_calls():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=60, V=300, D=64, K=4, seed=26, mask="random")
    H = torch.nan_to_num(H)
    Hl, El = H.view(3, 20, 64).clone().requires_grad_(), E.clone().requires_grad_()
    i, l, mm = dev(ids).view(3, 20, 4), dev(lg).view(3, 20, 4), dev(m).view(3, 20)
    (2.0 * api.distill_loss(Hl, El, i, l, mm, temperature=1.5)).backward()
    loss, lse = api.distill_forward(H, E, dev(ids), dev(lg), dev(m), temperature=1.5)
    dH, dE = api.distill_backward(H, E, dev(ids), dev(lg), lse, dev(m), temperature=1.5,
                                  grad_loss=torch.tensor(2.0, device="cuda"), grad_dtype=torch.bfloat16)
    assert torch.equal(Hl.grad.view(60, 64), dH) and torch.equal(El.grad, dE)
    y, off = dev(np.maximum(ids[:, 0], -1) % 300), torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    Hl.grad = El.grad = None
    loss, logp = api.preference_loss(Hl.view(60, 64), El, y, off, beta=0.2)
    assert not logp.requires_grad
    loss.backward()
    l2, logp2, lse, dH, dE = api.preference_forward_backward(H, E, y, off, beta=0.2, grad_dtype=torch.bfloat16)
    assert torch.equal(logp, logp2) and abs(float(loss) - float(l2)) < 1e-6
    assert torch.allclose(Hl.grad.view(60, 64).float(), dH.float(), rtol=0.02, atol=1e-5)
    X = api.embed(El, y.view(3, 20), 8.0)
    El.grad = None
    X.backward(torch.ones_like(X))
    assert torch.equal(El.grad, api.embed_backward(torch.ones_like(X), y.view(3, 20), 300, 8.0, grad_dtype=torch.bfloat16))


def tied_step(E, ids, teacher, dE=None):
    """One step of a model whose table is its input and its output: lookup, a trunk, the
    distillation loss on the teacher's top items, and both gradients into one dE."""
    X = api.embed_forward(E, ids, scale=8.0)
    Wt = torch.linspace(-1, 1, 64 * 64, device="cuda").view(64, 64).to(torch.bfloat16) / 8
    H = X @ Wt
    tid, tlg = B.cutbce_topk(teacher.view(-1, 64), E, 8)
    loss, lse, dH, dE = api.distill_forward_backward(H, E, tid.view(4, -1, 8), tlg.view(4, -1, 8), (ids >= 0).to(torch.uint8),
                                                     temperature=2.0, dE_out=dE)
    dX = dH.to(torch.bfloat16) @ Wt.t()
    return loss, api.embed_backward(dX, ids, E.shape[0], scale=8.0, out=dE, accumulate=True), X, H, tid, tlg, dX


def test_a_tied_step():
    r = np.random.default_rng(27)
    Ef, E = bf16(r.standard_normal((700, 64)) / 8)
    _, teacher = bf16(r.standard_normal((4, 30, 64)))
    ids = r.integers(0, 700, (4, 30)).astype(np.int32)
    ids[:, 25:] = -1
    loss, dE, X, H, tid, tlg, dX = tied_step(E, dev(ids), teacher)
    ref = O.distill(host(H).reshape(120, 64), Ef, tid.cpu().numpy(), tlg.cpu().numpy(), ids.reshape(-1) >= 0, tau=2.0)
    assert abs(float(loss) - ref.loss) <= 1e-4 * (1 + abs(ref.loss))
    want = ref.dE + O.embed_grad(host(dX).reshape(120, 64), ids.reshape(-1), 700, 8.0)
    t = bounds(ref, host(H).reshape(120, 64), Ef, 2.0, 32)
    scale = ref.s * 2.0
    tol = t.dE(ref, scale, np.zeros(120)) + 64 * U * O.embed_grad(np.abs(host(dX)).reshape(120, 64), ids.reshape(-1), 700, 8.0)
    close(host(dE), want, tol + 4 * U * np.abs(want), "tied dE")


def test_preference_with_its_reference_model():
    r = np.random.default_rng(28)
    Ef, E = bf16(r.standard_normal((500, 64)) / 8)
    Rf, Rm = bf16(r.standard_normal((50, 64)))
    Hf, H = bf16(Rf + 0.3 * r.standard_normal((50, 64)))
    ids, off = r.integers(0, 500, 50).astype(np.int32), O.offsets_of([13, 12, 20, 5])
    _, ref_lp, _ = api.preference_forward(Rm, E, dev(ids), dev(off))
    loss, logp, lse, dH, dE = api.preference_forward_backward(H, E, dev(ids), dev(off), ref_lp, beta=0.3)
    want_ref = O.preference(Rf, Ef, ids, off).logp
    ref = O.preference(Hf, Ef, ids, off, want_ref, beta=0.3)
    assert abs(float(loss) - ref.loss) <= 1e-4
    close(host(logp), ref.logp, 1e-2 + 0 * ref.logp, "logp")
    # the reference itself gives x = 0: loss ln 2
    same, *_ = api.preference_forward(Rm, E, dev(ids), dev(off), ref_lp)
    assert abs(float(same) - np.log(2)) < 1e-5


def test_captured_graphs_beside_each_other():
    r = np.random.default_rng(29)
    Ef, E = bf16(r.standard_normal((600, 64)) / 8)
    teachers = [bf16(r.standard_normal((4, 16, 64)))[1] for _ in range(2)]
    inputs = [dev(r.integers(0, 600, (4, 16)).astype(np.int32)) for _ in range(2)]
    want = [tied_step(E, i, t)[:2] for i, t in zip(inputs, teachers)]
    graphs, outs = [], []
    for i, t in zip(inputs, teachers):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            tied_step(E, i, t)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tied_step(E, i, t)[:2])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):               # both in flight at once
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_three_streams_at_once():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=200, V=4000, D=64, K=4, seed=30)
    lg = np.nan_to_num(lg)
    args = (H, E, dev(ids), dev(lg))
    want = api.distill_forward_backward(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(api.distill_forward_backward(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for o in got for x, y in zip(o, want))


def test_captured_backward_beside_an_eager_graph():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=200, V=4000, D=64, K=4, seed=32)
    args = dev(ids), dev(np.nan_to_num(lg))
    Hl, El = H.clone().requires_grad_(), E.clone().requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    # an eager graph of the same leaves on another stream: refused before the capture breaks
    elsewhere = api.distill_loss(Hl, El, *args)
    with pytest.raises(RuntimeError, match="another stream"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            api.distill_loss(Hl, El, *args)
    assert torch.isfinite(elsewhere)
    del elsewhere
    # on the captured stream it may live through the capture
    with torch.cuda.stream(s):
        eager = api.distill_loss(Hl, El, *args)
        torch.autograd.grad(api.distill_loss(Hl, El, *args), (Hl, El))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        loss = api.distill_loss(Hl, El, *args)
        grads = torch.autograd.grad(loss, (Hl, El))
    g.replay()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ge = torch.autograd.grad(eager, (Hl, El))
    torch.cuda.synchronize()
    assert torch.equal(loss, eager) and all(torch.equal(a, b) for a, b in zip(grads, ge))


def test_bad_ids_give_a_nan_loss():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=30, V=100, D=64, K=3, seed=36, holes=False)
    ids[11, 1] = 100
    assert torch.isnan(api.distill_forward(H, E, dev(ids), dev(lg))[0])
    y, off = dev(ids[:, 1]), torch.tensor([0, 15, 30], dtype=torch.int32, device="cuda")
    assert torch.isnan(api.preference_forward(H, E, y, off)[0])
    # more positions than the short form takes
    big = H.repeat(50, 1)
    assert torch.isnan(api.distill_forward(big, E, dev(ids).repeat(50, 1), dev(lg).repeat(50, 1))[0])


def test_calls_by_keyword_and_refusals_on_the_device():
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=30, V=100, D=64, K=3, seed=37, holes=False)
    i, l = dev(ids), dev(lg)
    a = api.distill_forward_backward(H, E, i, l)
    b = api.distill_forward_backward(E=E, H=H, teacher_logits=l, teacher_ids=i)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(api.embed_forward(ids=i, E=E), api.embed_forward(E, i))
    g = torch.tensor(2.0)
    for bad in (dict(grad_loss=g), dict(grad_loss=g.cuda().repeat(2)), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                dict(workspace=torch.empty(1 << 20, device="cuda")), dict(want_dH=False, want_dE=False),
                dict(accumulate_dE=True), dict(dE_out=torch.empty(99, 64, device="cuda")),
                dict(dE_out=torch.empty(100, 64)), dict(dE_out=torch.empty(100, 64, device="cuda"), grad_dtype=torch.bfloat16),
                dict(grad_dtype=torch.float16)):
        with pytest.raises(ValueError):
            api.distill_forward_backward(H, E, i, l, **bad)
    with pytest.raises(ValueError):
        api.distill_forward(H, E, i, l.cpu())
    with pytest.raises(ValueError):
        api.distill_backward(H, E, i, l, torch.zeros(29, device="cuda"))
    with pytest.raises(B.CutBCEError) as e:
        api.distill_forward(H, E, i, l, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == B.ERR_WORKSPACE
    p = B.make_distill_problem(H, E, i, l)
    ws = torch.empty(B.cutbce_distill_workspace_size(p, 7), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty((), dtype=torch.float64, device="cuda"), torch.empty(30, device="cuda")
    for args in ((loss.float(), lse), (loss, lse.double()), (loss, lse[:29])):
        with pytest.raises(ValueError):
            B.cutbce_distill_forward(p, *args, ws)
    with pytest.raises(ValueError):
        B.cutbce_distill_backward(p, None, lse, None, torch.empty(29, 64, device="cuda"), None, ws)


def test_workspace_guards():
    """Nothing outside the requested workspace is written."""
    Hf, H, Ef, E, ids, lg, m, w = draw_distill(T=131, V=1333, D=72, K=5, seed=31, mask="random")
    i, l, mm = dev(ids), dev(lg), dev(m)
    p = B.make_distill_problem(H, E, i, l, mm)
    n = B.cutbce_distill_workspace_size(p, 7)
    buf = torch.full((n + 512 + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    dH, dE = torch.empty(131, 72, device="cuda"), torch.empty(1333, 72, device="cuda")
    loss = torch.empty((), dtype=torch.float64, device="cuda")
    B.cutbce_distill_forward_backward(p, None, None, loss, None, dH, dE, buf[256:256 + n])
    assert B.cutbce_read_status(buf[256:]) == 0
    assert (buf[:256] == 0xA5).all() and (buf[256 + n:] == 0xA5).all()
    x = torch.randn(777, 40, device="cuda")
    ids = torch.randint(0, 50, (777,), dtype=torch.int32, device="cuda")
    n = B.cutbce_embed_workspace_size(777, 50, 40)
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    big = torch.full((52, 40), 7.0, device="cuda")
    B.cutbce_embed_backward(x, ids, big[1:51], buf[256:256 + n])
    assert (buf[:256] == 0xA5).all() and (buf[256 + n:] == 0xA5).all() and (big[0] == 7).all() and (big[51] == 7).all()
