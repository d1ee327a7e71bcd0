"""Softmax losses on peaked rows: states aligned with their next item, where the target's probability is
near 1 (or the student's weights near the teacher's) and dz = w (p - q) is a small difference.

Tolerances.  u = 2^-24, b = 2^-8 (half steps of fp32 and bf16).
 * A logit z is an fp32 sum of at most 256 products: |dz| <= zt = 2^-16 max_v sum_d |h_d e_vd|.  An exponential
   relative to another of its row is off by a factor of at most 1 + r, r = 2 zt / tau + 2e-4 (2^x: 7.5e-5 and the
   rounding of its argument, 1.3e-5, on either side).
 * An item that is not a target contributes p e (p h), rounded once to bf16: (b + r) of itself, and 1e-4 for the fp32
   accumulation.
 * A target contributes (p - q) e.  p = t / (t + rest) moves by p (1 - p) r at most, and the fp32 operations that form
   p - q and add it over the K targets are off by at most 8 (K + 2) u of p + q.
So a row whose dz is small has a small tolerance: it goes with p of the others and 1 - p of the target, not with p.
 * lse and the loss: a row's loss is its own size times r, and 8 u for each of the terms of its sum.
"""
import numpy as np
import pytest
import torch

from oracle import table_oracle as O
from vocabulary_label_bce_b200 import api

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8


def bf16(x):
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def aligned_rows(T, V, D, lo, hi, seed):
    """H [T, D] along the row of its next item y, with logits of it from lo to hi; E [V, D] of unit rows."""
    r = np.random.default_rng(seed)
    E = r.standard_normal((V, D)) / np.sqrt(D)
    Ef, Ed = bf16(E)
    y = r.integers(0, V, T).astype(np.int32)
    y[:3] = [0, V - 1, V // 2][:min(3, T)]
    n2 = (Ef[y] ** 2).sum(1)
    H = Ef[y] * (r.permutation(np.linspace(lo, hi, T)) / n2)[:, None]
    Hf, Hd = bf16(H)
    return Hf, Hd, Ef, Ed, y, r


def tolerances(ref, E, tau, K, scale):
    zt = 2.0 ** -16 * (np.abs(ref.H) @ np.abs(E).T).max(1)
    r = (2 * zt / tau + 2e-4)[:, None]
    is_t = ref.q != 0
    per = np.where(is_t, ref.p * (1 - ref.p) * r + 8 * (K + 2) * U * (ref.p + ref.q), ref.p * (BF + r + 1e-4))
    per = per * np.abs(ref.w)[:, None] * scale
    return zt, per @ np.abs(E) + 4 * U * np.abs(ref.dH) + 1e-30, per.T @ np.abs(ref.H) + 4 * U * np.abs(ref.dE) + 1e-30


def close(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - want) / tol))
    assert worst <= 1.0, (what, worst)


SIZES = [dict(T=60, V=3000, D=64), dict(T=300, V=5000, D=136), dict(T=520, V=20000, D=64), dict(T=450, V=20000, D=72),
         dict(T=410, V=20011, D=256)]


def name(c):
    return "_".join(f"{k}{v}" for k, v in c.items())


@pytest.mark.parametrize("entry", ["fused", "split", "dE only"])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=name)
def test_distill_to_the_next_item(size, weights, entry):
    """One target a row, p from about 1/2 to within 1e-4 of 1."""
    T = size["T"]
    Hf, H, Ef, E, y, r = aligned_rows(lo=11, hi=24, seed=50, **size)
    ids, lg = y[:, None], np.zeros((T, 1), np.float32)
    w = r.uniform(0.5, 2, T).astype(np.float32) * np.where(r.random(T) < 0.3, -1, 1).astype(np.float32) if weights else None
    check_distill(Hf, H, Ef, E, ids, lg, w, 1.0, 1, entry)


@pytest.mark.parametrize("entry", ["fused", "split", "dE only"])
@pytest.mark.parametrize("K", [3, 20, 40, 128])
def test_distill_to_its_own_distribution(K, entry):
    """The teacher's weights are the student's up to a factor e^0.02, some ids are there twice, some slots are empty."""
    T, V, D, tau = 430, 20000, 64, 1.3
    Hf, H, Ef, E, y, r = aligned_rows(T, V, D, 11, 24, 51)
    z = Hf @ Ef.T
    ids = np.argsort(-z, axis=1)[:, :K].astype(np.int32)
    ids = r.permuted(ids, axis=1)
    lg = np.take_along_axis(z, ids.astype(np.int64), 1) + 0.02 * r.standard_normal((T, K))
    ids[::5, K - 1] = ids[::5, 0]                          # an id twice: half of its weight in either slot
    lg[::5, 0] -= tau * np.log(2)
    lg[::5, K - 1] = lg[::5, 0]
    ids[1::5, K // 2] = -1
    check_distill(Hf, H, Ef, E, ids, lg.astype(np.float32), None, tau, K, entry)


def check_distill(Hf, H, Ef, E, ids, lg, w, tau, K, entry):
    ref = O.distill(Hf, Ef, ids, lg, None, w, tau, "mean")
    wd = None if w is None else torch.from_numpy(w).cuda()
    args = H, E, torch.from_numpy(ids).cuda(), torch.from_numpy(lg).cuda(), None, wd
    if entry == "fused":
        loss, lse, dH, dE = api.distill_forward_backward(*args, temperature=tau)
    else:
        loss, lse = api.distill_forward(*args, temperature=tau)
        dH, dE = api.distill_backward(*args[:4], lse, *args[4:], temperature=tau, want_dH=entry != "dE only")
    zt, tol_dH, tol_dE = tolerances(ref, Ef, tau, K, ref.s * tau)
    if entry == "dE only":                                 # p from the lse alone: half a step of it, and of its scaling
        extra = (8 * U * (np.abs(ref.lse) + 2))[:, None] * ref.p * np.abs(ref.w)[:, None] * ref.s * tau
        tol_dE = tol_dE + extra.T @ np.abs(ref.H)
    if dH is not None:
        close(dH, ref.dH, tol_dH, "dH")
    close(dE, ref.dE, tol_dE, "dE")
    # tau^2 KL(q || p): its terms q ln(q / p) are off by q du, du = (1 - p) r and a few u of the terms themselves
    q = ref.q
    with np.errstate(divide="ignore", invalid="ignore"):
        size = np.where(q > 0, q * (np.abs(np.log(q)) + 2), 0).sum(1)
    rest = 1 - (ref.p * (q > 0)).sum(1)
    du = (2 * zt / tau + 2e-4) * (rest + (0 if K == 1 else 1)) + 16 * U * size
    assert abs(float(loss) - ref.loss) <= tau * tau * ref.s * (np.abs(ref.w) * du).sum()


@pytest.mark.parametrize("entry", ["fused", "split"])
@pytest.mark.parametrize("size", SIZES, ids=name)
def test_preference_of_a_trained_model(size, entry):
    T = size["T"]
    Hf, H, Ef, E, y, r = aligned_rows(lo=11, hi=24, seed=52, **size)
    off = O.offsets_of([T // 4, T // 4 - 3, T // 8, T - 2 * (T // 4) + 3 - T // 8])
    rl = np.zeros(4, np.float32)
    ref = O.preference(Hf, Ef, y, off, rl, None, 0.3)
    args = H, E, torch.from_numpy(y).cuda()
    kw = dict(offsets=torch.from_numpy(off).cuda(), ref_logp=torch.from_numpy(rl).cuda(), beta=0.3)
    if entry == "fused":
        loss, logp, lse, dH, dE = api.preference_forward_backward(*args, **kw)
    else:
        loss, logp, lse = api.preference_forward(*args, **kw)
        dH, dE = api.preference_backward(*args, lse, **kw)
    zt, tol_dH, tol_dE = tolerances(ref, Ef, 1.0, 1, ref.s * 0.3)
    # log p of a position is -ln(1 + rest / t): off by (1 - p) r; the factors move by e^|dx| - 1
    py = (ref.p * ref.q).sum(1)
    row = (2 * zt + 2e-4) * (1 - py) + 16 * U
    if entry == "split":                                   # x from the lse of the forward, an fp32 number
        row = row + 4 * U * np.abs(ref.lse)
    seq = np.repeat(np.arange(4), np.diff(off))
    lt = np.array([row[seq == i].sum() for i in range(4)])
    if entry == "fused":
        close(logp, ref.logp, lt + 4 * U * np.abs(ref.logp), "logp")
    grow = np.expm1(0.3 * (lt[0::2] + lt[1::2]))[seq // 2] + 1e-6
    ext = grow[:, None] * np.abs(ref.p - ref.q) * np.abs(ref.w)[:, None] * ref.s * 0.3
    close(dH, ref.dH, tol_dH + ext @ np.abs(Ef), "dH")
    close(dE, ref.dE, tol_dE + ext.T @ np.abs(Hf), "dE")


@pytest.mark.parametrize("T,V", [(40, 3000), (420, 20000)])
def test_errors_of_a_peaked_gradient_in_the_norm(T, V):
    """Every target above p = 0.9: what remains is the rounding of the others' p, 2^-8 of each at most."""
    Hf, H, Ef, E, y, r = aligned_rows(T, V, 64, 20, 24, 53)
    ref = O.distill(Hf, Ef, y[:, None], np.zeros((T, 1)))
    _, _, dH, dE = api.distill_forward_backward(H, E, torch.from_numpy(y[:, None]).cuda(), torch.zeros(T, 1, device="cuda"))
    assert (ref.p * ref.q).sum(1).min() > 0.9
    for got, want in ((dH, ref.dH), (dE, ref.dE)):
        assert np.linalg.norm(got.double().cpu().numpy() - want) <= 2 * BF * np.linalg.norm(want)


def test_one_target_in_every_position():
    """A hot item: its tile of the dE pass leaves it out of every row."""
    T, V, D = 700, 12000, 64
    Hf, H, Ef, E, y, r = aligned_rows(T, V, D, 8, 16, 54)
    ids = np.stack([y, np.full(T, 4321, np.int32)], 1).astype(np.int32)
    lg = np.zeros((T, 2), np.float32)
    check_distill(Hf, H, Ef, E, ids, lg, np.where(np.arange(T) % 3, 1.0, -0.5).astype(np.float32), 1.0, 2, "fused")


def test_every_item_a_target():
    """K = V: no item is left to the dense part."""
    T, V, D = 300, 128, 64
    Hf, H, Ef, E, y, r = aligned_rows(T, V, D, 4, 10, 55)
    ids = np.stack([r.permutation(V) for _ in range(T)]).astype(np.int32)
    lg = r.standard_normal((T, V)).astype(np.float32)
    for entry in ("fused", "split"):
        check_distill(Hf, H, Ef, E, ids, lg, None, 1.0, V, entry)


@pytest.mark.parametrize("entry", ["fused", "split", "dE only"])
@pytest.mark.parametrize("T,V", [(60, 3000), (430, 20000)])
def test_a_teacher_far_from_the_student(T, V, entry):
    """Weights over five decades on items that the student all but rules out: each keeps its own accuracy."""
    Hf, H, Ef, E, y, r = aligned_rows(T, V, 64, 18, 24, 56)
    ids = np.stack([(y[t] + 1 + r.permutation(V - 1)[:5]) % V for t in range(T)]).astype(np.int32)
    lg = np.tile(np.array([0, -3, -6, -9, -12], np.float32), (T, 1))
    check_distill(Hf, H, Ef, E, ids, lg, None, 1.0, 5, entry)
