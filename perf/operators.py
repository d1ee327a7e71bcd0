"""Timing cases of the item-table operators: row lookup and its gradient, and the
softmax losses over the whole table (distillation from a teacher's top logits, paired
preference loss).  `run` computes a case either in plain torch (own = False) or through
the library's torch-facing calls (own = True)."""
import math

import torch

own = False

KINDS = ("embed", "embed_grad", "distill", "distill_grad", "pref", "pref_grad")


def listed():
    return [
        # the newest item of each of 64 sequences, looked up at serving time
        {"name": "embed_step", "kind": "embed", "N": 64, "V": 100000, "D": 64, "dtype": "bf16", "zipf": 1.1},
        # the input of one SASRec-style training step: 64 sequences of 200 items
        {"name": "embed_sasrec", "kind": "embed", "N": 12800, "V": 876000, "D": 64, "dtype": "bf16", "zipf": 1.05},
        # the gradient of that input with respect to the whole table
        {"name": "embed_grad_sasrec", "kind": "embed_grad", "N": 12800, "V": 876000, "D": 64, "dtype": "bf16",
         "zipf": 1.05},
        # a long batch in fp32 with odd sizes: hot items hold thousands of tokens each
        {"name": "embed_grad_long_f32", "kind": "embed_grad", "N": 200003, "V": 100000, "D": 200, "dtype": "f32",
         "zipf": 1.1},
        # the distillation loss of a handful of positions over a small table: latency
        {"name": "distill_loss_tiny", "kind": "distill", "B": 4, "N": 16, "pad": 2, "V": 2048, "D": 32, "K": 4,
         "tau": 1.0},
        # validation loss over the full table
        {"name": "distill_loss_sasrec", "kind": "distill", "B": 64, "N": 200, "pad": 40, "V": 876000, "D": 64, "K": 16,
         "tau": 1.0},
        # a training step over a small catalog
        {"name": "distill_grad_small", "kind": "distill_grad", "B": 32, "N": 200, "pad": 30, "V": 100000, "D": 64,
         "K": 8, "tau": 2.0},
        # a training step of the SASRec-style head
        {"name": "distill_grad_sasrec", "kind": "distill_grad", "B": 64, "N": 200, "pad": 40, "V": 876000, "D": 64,
         "K": 16, "tau": 1.0},
        # a wide head
        {"name": "distill_grad_wide", "kind": "distill_grad", "B": 16, "N": 512, "pad": 51, "V": 1000000, "D": 256,
         "K": 16, "tau": 1.5},
        # scoring a few pairs of short sequences against a small table: latency
        {"name": "pref_loss_tiny", "kind": "pref", "P": 3, "N": 11, "V": 2047, "D": 40, "beta": 0.1},
        # preference tuning over a small catalog
        {"name": "pref_grad_small", "kind": "pref_grad", "P": 32, "N": 100, "V": 100000, "D": 64, "beta": 0.1},
        # preference tuning of the SASRec-style head
        {"name": "pref_grad_sasrec", "kind": "pref_grad", "P": 32, "N": 200, "V": 876000, "D": 64, "beta": 0.1},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(KINDS)
    if kind.startswith("embed"):
        D = 8 * _log_int(rng, 1, 32)
        V = _log_int(rng, 2, 1000000)
        N = _log_int(rng, 1, 250000)
        return {"kind": kind, "N": N, "V": V, "D": D, "dtype": rng.choice(("bf16", "f32")),
                "zipf": rng.choice((1.05, 1.1))}
    D = 8 * _log_int(rng, 2, 32)
    V = _log_int(rng, 100, 1000000)
    most = max(1, int(7.0e9 / V))
    if kind.startswith("distill"):
        B = _log_int(rng, 1, 64)
        N = _log_int(rng, 2, 512)
        N = max(2, min(N, most // B, 12800 // B))
        return {"kind": kind, "B": B, "N": N, "pad": rng.randrange(0, 1 + N // 4), "V": V, "D": D,
                "K": min(_log_int(rng, 1, 64), V), "tau": rng.choice((0.7, 1.0, 2.0))}
    P = _log_int(rng, 1, 32)
    N = _log_int(rng, 1, 200)
    return {"kind": kind, "P": P, "N": max(1, min(N, most // (2 * P))), "V": V, "D": D,
            "beta": rng.choice((0.05, 0.1, 0.5))}


def _zipf(n, V, s, g):
    # bounded Zipf(s), id = rank, by inverse CDF
    p = torch.arange(1, V + 1, device="cuda", dtype=torch.float64) ** -s
    c = torch.cumsum(p, 0)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * c[-1]
    return torch.searchsorted(c, u).clamp_(max=V - 1).to(torch.int32)


def _normal(shape, std, dtype, g):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _lengths(case):
    # ragged lengths, fixed by the case: from N down to about N / 2
    n = case["N"]
    return [n - (7 * i) % (n // 2 + 1) for i in range(2 * case["P"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    V, D, kind = case["V"], case["D"], case["kind"]
    if kind.startswith("embed"):
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        ids = _zipf(case["N"], V, case["zipf"], g)
        ids[torch.rand(case["N"], generator=g, device="cuda") < 0.05] = -1          # padding
        s = {"case": case, "ids": ids, "scale": math.sqrt(D)}
        if kind == "embed":
            s["E"] = _normal((V, D), 1 / math.sqrt(D), dt, g)
        else:
            s["dX"] = _normal((case["N"], D), 1.0, dt, g)
        return s
    E = _normal((V, D), 1 / math.sqrt(D), torch.bfloat16, g)
    if kind.startswith("distill"):
        B, N, K = case["B"], case["N"], case["K"]
        T = B * N
        mask = torch.ones((B, N), device="cuda", dtype=torch.uint8)
        mask[:, N - case["pad"]:] = 0
        ids = torch.randint(0, V, (T, K), generator=g, device="cuda", dtype=torch.int32)
        logits = torch.sort(2.0 * torch.randn((T, K), generator=g, device="cuda") + 4.0, dim=1, descending=True)[0]
        if K > 1:
            ids[torch.rand(T, generator=g, device="cuda") < 0.1, K - 1] = -1        # a list one entry short
        return {"case": case, "E": E, "H": _normal((T, D), 1.0, torch.bfloat16, g), "ids": ids,
                "logits": logits.contiguous(), "mask": mask.reshape(T)}
    lens = _lengths(case)
    T = sum(lens)
    off = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    ids = _zipf(T, V, 1.05, g)
    ids[torch.rand(T, generator=g, device="cuda") < 0.03] = -1                      # padding inside a sequence
    ref = -torch.tensor(lens, device="cuda", dtype=torch.float32) * math.log(V)
    ref = ref + torch.randn(len(lens), generator=g, device="cuda")
    return {"case": case, "E": E, "H": _normal((T, D), 1.0, torch.bfloat16, g), "ids": ids, "off": off, "ref": ref}


# ---------------------------------------------------------------- plain forms
def _softmax_grads(P, lse_rows, coef, H, E, sparse_rows, sparse_ids, sparse_coef):
    """dH and dE of sum coef (P - Y) with P [T, V] fp32 in place; one rounding at the end."""
    P.mul_(coef[:, None])
    P.index_put_((sparse_rows, sparse_ids), -sparse_coef, accumulate=True)
    return (P @ E.float()).to(torch.bfloat16), (P.t() @ H.float()).to(torch.bfloat16)


def _plain_distill(s):
    c = s["case"]
    tau = c["tau"]
    H, E, ids, valid = s["H"], s["E"], s["ids"], s["mask"] != 0
    slot = ids >= 0
    tl = torch.where(slot, s["logits"] / tau, torch.full_like(s["logits"], -math.inf))
    tl = tl - tl.amax(1, keepdim=True)
    q = tl.exp()
    qs = q.sum(1, keepdim=True)
    q = q / qs
    logq = torch.where(slot, tl - qs.log(), torch.zeros_like(tl))
    Z = H.float() @ E.float().t()
    Z.div_(tau)
    zk = torch.gather(Z, 1, ids.clamp(min=0).long())
    m = Z.amax(1)
    Z.sub_(m[:, None]).exp_()
    S = Z.sum(1)
    lse = m + S.log()
    row = tau * tau * (q * (logq - zk + lse[:, None])).sum(1)
    n = valid.sum()
    loss = (torch.where(valid, row, torch.zeros_like(row)).double().sum() / n).float()
    lse = torch.where(valid, lse, torch.zeros_like(lse))
    if c["kind"] == "distill":
        return {"loss": loss, "lse": lse}
    coef = torch.where(valid, tau / n.float(), torch.zeros_like(S))
    Z.div_(S[:, None])
    rows = torch.arange(ids.shape[0], device="cuda")[:, None].expand_as(ids)
    dH, dE = _softmax_grads(Z, lse, coef, H, E, rows, ids.clamp(min=0).long(), torch.where(slot, q, 0 * q) * coef[:, None])
    return {"loss": loss, "lse": lse, "dH": dH, "dE": dE}


def _plain_pref(s):
    c = s["case"]
    H, E, ids, off, ref = s["H"], s["E"], s["ids"], s["off"], s["ref"]
    T, nseq = ids.shape[0], 2 * c["P"]
    valid = ids >= 0
    seq = torch.searchsorted(off[1:].contiguous(), torch.arange(T, device="cuda", dtype=torch.int32), right=True)
    Z = H.float() @ E.float().t()
    y = ids.clamp(min=0).long()
    zy = torch.gather(Z, 1, y[:, None])[:, 0]
    m = Z.amax(1)
    Z.sub_(m[:, None]).exp_()
    S = Z.sum(1)
    lse = m + S.log()
    lp = torch.where(valid, zy - lse, torch.zeros_like(lse))
    logp64 = torch.zeros(nseq, device="cuda", dtype=torch.float64).index_add_(0, seq, lp.double())
    d = (logp64 - ref.double()).view(-1, 2)
    x = c["beta"] * (d[:, 0] - d[:, 1])
    soft = torch.clamp(-x, min=0) + torch.log1p(torch.exp(-x.abs()))
    loss, logp = soft.mean().float(), logp64.float()
    lse = torch.where(valid, lse, torch.zeros_like(lse))
    if c["kind"] == "pref":
        return {"loss": loss, "logp": logp, "lse": lse}
    w = c["beta"] / (1 + torch.exp(x)) / c["P"]
    w = torch.stack((w, -w), 1).view(-1).float()[seq]
    w = torch.where(valid, w, torch.zeros_like(w))
    Z.div_(S[:, None])
    dH, dE = _softmax_grads(Z, lse, w, H, E, torch.arange(T, device="cuda"), y, w)
    return {"loss": loss, "logp": logp, "lse": lse, "dH": dH, "dE": dE}


def _plain_embed(s):
    ids = s["ids"].long()
    real = (ids >= 0)[:, None]
    if s["case"]["kind"] == "embed":
        x = s["E"][ids.clamp(min=0)].float() * s["scale"]
        return torch.where(real, x, torch.zeros_like(x)).to(s["E"].dtype)
    g = s["dX"].float() * s["scale"]
    g = torch.where(real, g, torch.zeros_like(g))
    out = torch.zeros((s["case"]["V"], s["case"]["D"]), device="cuda", dtype=torch.float32)
    return out.index_add_(0, ids.clamp(min=0), g).to(s["dX"].dtype)


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from vocabulary_label_bce_b200 import api
    c = s["case"]
    kind = c["kind"]
    if kind == "embed":
        return api.embed_forward(s["E"], s["ids"], scale=s["scale"])
    if kind == "embed_grad":
        return api.embed_backward(s["dX"], s["ids"], c["V"], scale=s["scale"], grad_dtype=s["dX"].dtype)
    if kind == "distill":
        loss, lse = api.distill_forward(s["H"], s["E"], s["ids"], s["logits"], s["mask"], temperature=c["tau"])
        return {"loss": loss.float(), "lse": lse}
    if kind == "distill_grad":
        loss, lse, dH, dE = api.distill_forward_backward(s["H"], s["E"], s["ids"], s["logits"], s["mask"],
                                                         temperature=c["tau"], grad_dtype=torch.bfloat16)
        return {"loss": loss.float(), "lse": lse, "dH": dH, "dE": dE}
    if kind == "pref":
        loss, logp, lse = api.preference_forward(s["H"], s["E"], s["ids"], s["off"], s["ref"], beta=c["beta"])
        return {"loss": loss.float(), "logp": logp, "lse": lse}
    loss, logp, lse, dH, dE = api.preference_forward_backward(s["H"], s["E"], s["ids"], s["off"], s["ref"],
                                                              beta=c["beta"], grad_dtype=torch.bfloat16)
    return {"loss": loss.float(), "logp": logp, "lse": lse, "dH": dH, "dE": dE}


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind.startswith("embed"):
        return _plain_embed(state)
    return _plain_distill(state) if kind.startswith("distill") else _plain_pref(state)


def work(case):
    kind, V, D = case["kind"], case["V"], case["D"]
    if kind.startswith("embed"):
        N, e = case["N"], 2 if case["dtype"] == "bf16" else 4
        if kind == "embed":
            return {"bytes": 4 * N + e * D * (min(N, V) + N), "flops": N * D}
        return {"bytes": 4 * N + e * D * N + e * D * V, "flops": 2 * N * D}
    if kind.startswith("distill"):
        T = case["B"] * case["N"]
        n = case["B"] * (case["N"] - case["pad"])
        b = 2 * D * (n + V) + 8 * n * case["K"] + T + 4 * T
    else:
        T = n = sum(_lengths(case))
        b = 2 * D * (n + V) + 8 * T + 4 * (2 * case["P"] + 1)
    if kind.endswith("grad"):
        return {"bytes": b + 2 * D * (T + V), "flops": 6 * n * V * D}
    return {"bytes": b, "flops": 2 * n * V * D}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_head(H, E, valid, coef_of, sparse, scale):
    """Row log-sum-exps of scale * H E^T and, with coef_of, the gradients of the head, in slices of rows."""
    T, V = H.shape[0], E.shape[0]
    step = max(1, min(T, int(1.0e9 // V)))
    E64, H64 = E.double(), H.double()
    lse = torch.zeros(T, device="cuda", dtype=torch.float64)
    for a in range(0, T, step):
        lse[a:a + step] = torch.logsumexp(scale * (H64[a:a + step] @ E64.T), dim=1)
    lse = lse * valid
    if coef_of is None:
        return lse, None, None
    coef = coef_of(lse)
    dH, dE = torch.zeros_like(H64), torch.zeros_like(E64)
    rows, cols, share = sparse
    for a in range(0, T, step):
        G = torch.exp(scale * (H64[a:a + step] @ E64.T) - lse[a:a + step, None]) * coef[a:a + step, None]
        dH[a:a + step] = G @ E64
        dE += G.T @ H64[a:a + step]
    amount = coef[rows] * share
    dH.index_add_(0, rows, -amount[:, None] * E64[cols])
    dE.index_add_(0, cols, -amount[:, None] * H64[rows])
    return lse, dH, dE


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "embed":
        ids = s["ids"].long()
        x = torch.zeros((case["N"], case["D"]), device="cuda", dtype=torch.float64)
        k = ids >= 0
        x[k] = s["E"].double()[ids[k]] * s["scale"]
        return x
    if kind == "embed_grad":
        ids = s["ids"].long()
        k = ids >= 0
        out = torch.zeros((case["V"], case["D"]), device="cuda", dtype=torch.float64)
        out.index_put_((ids[k],), s["dX"][k].double() * s["scale"], accumulate=True)
        return out
    grad = kind.endswith("grad")
    H, E, ids = s["H"], s["E"], s["ids"].long()
    T = H.shape[0]
    H64, E64 = H.double(), E.double()
    if kind.startswith("distill"):
        tau, K = case["tau"], case["K"]
        valid = (s["mask"] != 0).double()
        n = valid.sum()
        t, k = torch.nonzero((ids >= 0) & (s["mask"] != 0)[:, None], as_tuple=True)
        v = ids[t, k]
        tq = torch.full((T, K), -math.inf, device="cuda", dtype=torch.float64)
        tq[ids >= 0] = s["logits"].double()[ids >= 0] / tau
        logq = torch.log_softmax(tq, 1)[t, k]
        q = logq.exp()
        lse, dH, dE = _exact_head(H, E, valid, (lambda l: tau * valid / n) if grad else None, (t, v, q), 1 / tau)
        term = tau * tau * q * (logq - (H64[t] * E64[v]).sum(1) / tau + lse[t])
        out = {"loss": term.sum() / n, "lse": lse}
    else:
        valid = (ids >= 0).double()
        t = torch.nonzero(ids >= 0)[:, 0]
        off = s["off"].tolist()
        which = torch.cat([torch.full((off[i + 1] - off[i],), i, device="cuda") for i in range(2 * case["P"])])
        zy = (H64 * E64[ids.clamp(min=0)]).sum(1)
        kept = {}

        def coef(lse):
            lp = torch.zeros(2 * case["P"], device="cuda", dtype=torch.float64)
            lp.index_add_(0, which, (zy - lse) * valid)
            x = case["beta"] * ((lp[0::2] - s["ref"].double()[0::2]) - (lp[1::2] - s["ref"].double()[1::2]))
            kept["logp"], kept["loss"] = lp, -torch.nn.functional.logsigmoid(x).mean()
            w = case["beta"] * torch.sigmoid(-x) / case["P"]
            sign = 1.0 - 2.0 * (which % 2).double()
            return sign * w[which // 2] * valid

        lse, dH, dE = _exact_head(H, E, valid, coef if grad else None, (t, ids[t], torch.ones_like(zy)[t]), 1.0)
        if not grad:
            coef(lse)
        out = {"loss": kept["loss"], "logp": kept["logp"], "lse": lse}
    if grad:
        out["dH"], out["dE"] = dH, dE
    return out
