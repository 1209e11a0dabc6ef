"""What the operators around the expert layer are measured on: the norm in front of it (forward and backward), the
router's balance loss (forward and backward), and the orthogonalised update of the expert weights.

A case is one call of one operator.  `run` computes it in plain torch operations in 32 bits, or, where `own` is true,
through the framework's entry points.  `exact` gives the same outputs in 64 bits."""
import math

import torch

own = False

COEFS = (3.4445, -4.7750, 2.0315)  # the quintic Newton-Schulz step, five times
STEPS = 5
NORM_EPS = 1e-5
ORTHO_EPS = 1e-7


def listed():
    return [
        # the norm before the layer of the tiny configuration (T=512, H=128): latency is all there is
        dict(name="norm_fwd_t512_h128", op="norm_fwd", T=512, H=128, kind="layer", bias=True, residual=False,
             dtype="bf16"),
        # the residual sum and the norm in front of a layer of the 235B shape, one 16,384-token sequence
        dict(name="norm_fwd_res_t16384_h4096", op="norm_fwd", T=16384, H=4096, kind="layer", bias=True, residual=True,
             dtype="bf16"),
        # its backward at the 30B shape, the residual path's gradient added, weight and bias gradients reduced
        dict(name="norm_bwd_res_t16384_h2048", op="norm_bwd", T=16384, H=2048, kind="layer", bias=True, residual=True,
             dtype="bf16"),
        # an fp32 model of odd width, RMS kind, a ragged last batch
        dict(name="norm_bwd_t4999_h1000_fp32", op="norm_bwd", T=4999, H=1000, kind="rms", bias=False, residual=False,
             dtype="fp32"),
        # the balance loss of the tiny configuration
        dict(name="balance_fwd_t512_e8", op="balance_fwd", T=512, E=8, k=2, S=1, masked=False),
        # four packed sequences with padding at the 30B routing shape
        dict(name="balance_fwd_t16384_e128_s4", op="balance_fwd", T=16384, E=128, k=8, S=4, masked=True),
        # its gradient added to the d_logits that the layer's backward left, one sequence
        dict(name="balance_bwd_t16384_e128", op="balance_bwd", T=16384, E=128, k=8, S=1, masked=False),
        # a large batch over an expert count that is no multiple of four
        dict(name="balance_bwd_t131072_e250_s32", op="balance_bwd", T=131072, E=250, k=8, S=32, masked=True),
        # W_gate of the tiny configuration: eight small matrices, latency
        dict(name="ortho_b8_128x64", op="ortho", B=8, R=128, C=64, dtype="bf16", momentum=False),
        # dW_gate of the 30B shape, straight from the layer's backward
        dict(name="ortho_b128_2048x768", op="ortho", B=128, R=2048, C=768, dtype="bf16", momentum=False),
        # dW_down of the 235B shape for an eighth of the experts, through fp32 momentum
        dict(name="ortho_b16_1536x4096_mom", op="ortho", B=16, R=1536, C=4096, dtype="bf16", momentum=True),
        # a few fp32 matrices of odd sizes
        dict(name="ortho_b3_1000x333_fp32", op="ortho", B=3, R=1000, C=333, dtype="fp32", momentum=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance_fwd", "balance_bwd", "ortho", "ortho"])
    if op.startswith("norm"):
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        T = _log(rng, 1, max(1, (1 << 26) // H))
        return dict(op=op, T=T, H=H, kind=rng.choice(["layer", "rms"]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op.startswith("balance"):
        E = rng.choice([8, 16, 60, 64, 128, 128, 160, 250, 256])
        S = rng.choice([1, 1, 2, 4, 8, 32])
        L = _log(rng, 1, (1 << 17) // S)
        return dict(op=op, T=S * L, E=E, k=min(E, rng.choice([1, 2, 4, 6, 8, 16])), S=S, masked=rng.random() < 0.5)
    n = _log(rng, 24, 1536)
    m = max(n, min(4096, int(n * rng.uniform(1.0, 6.0))))
    if rng.random() < 0.6:
        n, m = max(8, n // 64 * 64), max(8, m // 64 * 64)
    B = _log(rng, 1, max(1, min(256, (1 << 27) // (n * m))))
    R, C = (n, m) if rng.random() < 0.5 else (m, n)
    return dict(op="ortho", B=B, R=R, C=C, dtype=rng.choice(["bf16", "bf16", "fp32"]), momentum=rng.random() < 0.4)


# ------------------------------------------------------------------------------------------------ inputs

_T = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)

    def randn(*s, dtype=torch.float32):
        return torch.randn(*s, generator=g, device="cuda", dtype=dtype)

    op, t = case["op"], {}
    if op.startswith("norm"):
        T, H, dt = case["T"], case["H"], _T[case["dtype"]]
        # activations: channels of uneven scale around uneven means
        x = (randn(T, H) * torch.exp(0.5 * randn(H)) + 0.3 * randn(H)).to(dt)
        t["weight"] = (1 + 0.1 * randn(H)).to(dt)
        t["bias"] = (0.1 * randn(H)).to(dt) if case["bias"] else None
        if op == "norm_fwd":
            t["x"], t["residual"] = x, randn(T, H).to(dt) if case["residual"] else None
        else:
            t["x"], t["dy"] = x, randn(T, H).to(dt)
            t["d_sum"] = randn(T, H).to(dt) if case["residual"] else None
            f = x.float()
            mu = f.mean(1) if case["kind"] == "layer" else torch.zeros(T, device="cuda")
            var = ((f - mu[:, None]) ** 2).mean(1)
            t["stats"] = torch.stack([mu, torch.rsqrt(var + NORM_EPS)], 1).contiguous()  # the forward's
    elif op.startswith("balance"):
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        L = T // S
        t["logits"] = randn(T, E) + 0.7 * randn(E)  # uneven expert loads
        t["topk_idx"] = torch.topk(t["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        t["mask"] = None
        if case["masked"]:  # each sequence is padded at its end; the last of several is empty
            n = torch.randint(max(1, L // 2), L + 1, (S,), generator=g, device="cuda")
            if S > 1:
                n[-1] = 0
            t["mask"] = (torch.arange(L, device="cuda")[None, :] < n[:, None]).reshape(T).to(torch.uint8)
        if op == "balance_bwd":
            valid = torch.ones(T, device="cuda") if t["mask"] is None else t["mask"].float()
            t["lse"] = torch.logsumexp(t["logits"], 1)  # what the forward leaves
            lse = torch.where(valid > 0, t["lse"], torch.full_like(t["lse"], float("inf")))
            t["lse"] = lse.contiguous()
            t["tokens"] = valid.reshape(S, L).sum(1).to(torch.int32)
            oh = torch.zeros(T, E, device="cuda").scatter_add_(1, t["topk_idx"].long(), valid[:, None].expand(T, k))
            t["counts"] = oh.reshape(S, L, E).sum(1).to(torch.int32).contiguous()
            t["d_logits"] = 1e-3 * randn(T, E)  # from the layer's backward
    else:
        B, R, C = case["B"], case["R"], case["C"]
        # a weight gradient: a product over tokens whose channels have uneven scales
        K = 2 * min(R, C)
        a = (randn(B, R, K) * torch.exp(0.3 * randn(B, R, 1))).to(torch.bfloat16)
        b = (randn(B, K, C) / math.sqrt(K)).to(torch.bfloat16)
        t["update"] = (torch.bmm(a, b).float() * 1e-3).to(_T[case["dtype"]])
        t["momentum"] = None
        if case["momentum"]:
            t["momentum"] = randn(B, R, C) * 5e-3 + t["update"].float()
    return t


def prepare(case, seed):
    # "out": the buffers of the last call's results, handed to the next one, as a training loop does
    state = {"case": case, "t": _inputs(case, seed), "op": None, "out": None}
    try:
        from dropless_mixture_experts_top_gb300 import moe
    except ImportError:
        return state
    op, t = case["op"], state["t"]
    if op.startswith("norm") and hasattr(moe, "Norm"):
        state["op"] = moe.Norm(case["T"], case["H"], kind=case["kind"], dtype=case["dtype"], bias=case["bias"],
                               eps=NORM_EPS)
    elif op.startswith("balance") and hasattr(moe, "BalanceLoss"):
        state["op"] = moe.BalanceLoss(case["T"], case["E"], case["k"], sequences=case["S"])
    elif op == "ortho" and hasattr(moe, "Orthogonaliser"):
        state["op"] = moe.Orthogonaliser(case["B"], case["R"], case["C"], dtype=case["dtype"],
                                         coefs=[COEFS] * STEPS, eps=ORTHO_EPS)
    return state


# ------------------------------------------------------------------------------------------------ one pass

G_BAL, G_Z = 1e-2, 1e-3  # loss coefficients
BETA = 0.95


def run(state):
    return (_run_own if own else _run_plain)(state["case"], state["t"], state["op"], state)


def _run_own(case, t, op, state):
    kind, out = case["op"], state["out"]
    if kind == "norm_fwd":
        out = op.forward(t["x"], t["weight"], t["bias"], residual=t["residual"], out=out)
    elif kind == "norm_bwd":
        out = op.backward(t["dy"], t["x"], t["weight"], t["stats"], d_sum=t["d_sum"], grads=out)
    elif kind == "balance_fwd":
        out = op.forward(t["logits"], t["topk_idx"], mask=t["mask"], out=out)
    elif kind == "balance_bwd":
        return op.backward(t["logits"], t["counts"], t["tokens"], t["lse"], G_BAL, G_Z, d_logits=t["d_logits"])
    else:
        out = op.update(t["update"], momentum=t["momentum"], beta=BETA, nesterov=True, out=out)
        state["out"] = out
        return {"out": out, "momentum": t["momentum"]}
    state["out"] = out
    return out


def _run_plain(case, t, op, state):
    kind = case["op"]
    if kind == "norm_fwd":
        x = t["x"].float()
        h = t["x"]
        if t["residual"] is not None:
            h = (x + t["residual"].float()).to(t["x"].dtype)
            x = h.float()
        mu = x.mean(1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
        c = x - mu
        rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + NORM_EPS)
        y = c * rstd * t["weight"].float()
        if t["bias"] is not None:
            y = y + t["bias"].float()
        return {"y": y.to(t["x"].dtype), "sum": h if t["residual"] is not None else None,
                "stats": torch.cat([mu, rstd], 1)}
    if kind == "norm_bwd":
        mu, rstd = t["stats"][:, :1], t["stats"][:, 1:]
        dy = t["dy"].float()
        xh = (t["x"].float() - mu) * rstd
        g = dy * t["weight"].float()
        dx = g - xh * (g * xh).mean(1, keepdim=True)
        if case["kind"] == "layer":
            dx = dx - g.mean(1, keepdim=True)
        dx = dx * rstd
        if t["d_sum"] is not None:
            dx = dx + t["d_sum"].float()
        return {"dx": dx.to(t["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0) if case["bias"] else None}
    if kind.startswith("balance"):
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        logits = t["logits"]
        if kind == "balance_fwd":
            valid = torch.ones(T, device=logits.device) if t["mask"] is None else t["mask"].float()
            top = logits.max(1, keepdim=True).values
            e = torch.exp(logits - top)
            z = e.sum(1, keepdim=True)
            lse = (top + torch.log(z))[:, 0]
            p = e / z * valid[:, None]
            hot = torch.zeros_like(p).scatter_add_(1, t["topk_idx"].long(), valid[:, None].expand(T, k))
            counts = hot.reshape(S, T // S, E).sum(1)
            n = valid.reshape(S, T // S).sum(1)
            some = (n > 0).float()
            probs = p.reshape(S, T // S, E).sum(1) / n.clamp(min=1)[:, None]
            f = counts / (k * n.clamp(min=1))[:, None]
            bal = E * (f * probs).sum() / some.sum().clamp(min=1)
            lz = (lse * lse * valid).sum() / n.sum().clamp(min=1)
            return {"loss": torch.stack([bal, lz]), "counts": counts.to(torch.int32), "probs": probs,
                    "tokens": n.to(torch.int32), "lse": torch.where(valid > 0, lse, torch.full_like(lse, math.inf))}
        n = t["tokens"].float()
        some = (n > 0).float().sum().clamp(min=1)
        f = t["counts"].float() / (k * n.clamp(min=1))[:, None]
        coef = G_BAL * E / (some * n.clamp(min=1))
        f = f.repeat_interleave(T // S, 0)
        coef = coef.repeat_interleave(T // S, 0)[:, None]
        valid = torch.isfinite(t["lse"])[:, None]
        lse = torch.where(valid, t["lse"][:, None], torch.zeros_like(t["lse"][:, None]))
        p = torch.exp(logits - lse)
        d = coef * p * (f - (f * p).sum(1, keepdim=True)) + (2 * G_Z / n.sum().clamp(min=1)) * lse * p
        t["d_logits"].add_(torch.where(valid, d, torch.zeros_like(d)))
        return t["d_logits"]
    u = t["update"].float()
    if t["momentum"] is not None:
        t["momentum"].mul_(BETA).add_(u)
        u = u + BETA * t["momentum"]
    tall = case["R"] > case["C"]
    x = u.transpose(1, 2) if tall else u
    x = x / torch.sqrt((x * x).sum((1, 2), keepdim=True)).clamp(min=ORTHO_EPS)
    a, b, c = COEFS
    for _ in range(STEPS):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return {"out": (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous(), "momentum": t["momentum"]}


# ------------------------------------------------------------------------------------------------ the least work

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, el, H = case["T"] * case["H"], 2 if case["dtype"] == "bf16" else 4, case["H"]
        io = (2 if op == "norm_fwd" else 3) + (2 if op == "norm_fwd" else 1) * case["residual"]
        return {"bytes": io * n * el + 8 * case["T"] + H * (2 * el + 8), "flops": (8 if op == "norm_fwd" else 14) * n}
    if op.startswith("balance"):
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        if op == "balance_fwd":
            return {"bytes": T * (4 * E + 4 * k + 4 + case["masked"]) + 8 * S * E, "flops": 6 * T * E}
        return {"bytes": T * (12 * E + 4) + 4 * S * E, "flops": 10 * T * E}
    B, n, m = case["B"], min(case["R"], case["C"]), max(case["R"], case["C"])
    el = 2 if case["dtype"] == "bf16" else 4
    # two symmetric products (one triangle each) and the product with X, per step
    flops = STEPS * B * (float(n) * n * m + float(n) ** 3 + 2.0 * n * n * m)
    return {"bytes": B * n * m * (el + 2 + 8 * case["momentum"]), "flops": flops}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    t, op = _inputs(case, seed), case["op"]
    d = {k: v.double() if v is not None and v.is_floating_point() else v for k, v in t.items()}
    if op == "norm_fwd":
        # h as the operator stores it (rounded to its type), everything after it in 64 bits
        h = d["x"]
        if t["residual"] is not None:
            h = (t["x"].float() + t["residual"].float()).to(t["x"].dtype).double()
        m1 = h.sum(1) / case["H"]
        mu = m1 if case["kind"] == "layer" else torch.zeros_like(m1)
        var = torch.sum((h - mu.unsqueeze(1)).pow(2), 1) / case["H"]
        r = 1.0 / torch.sqrt(var + NORM_EPS)
        y = torch.einsum("th,t,h->th", h - mu.unsqueeze(1), r, d["weight"])
        if d["bias"] is not None:
            y = y + d["bias"]
        return {"y": y, "sum": h if t["residual"] is not None else None, "stats": torch.stack([mu, r], 1)}
    if op == "norm_bwd":
        mu, r = d["stats"][:, 0], d["stats"][:, 1]
        xh = torch.einsum("th,t->th", d["x"] - mu.unsqueeze(1), r)
        gy = d["dy"] * d["weight"]
        along = torch.einsum("th,th->t", gy, xh) / case["H"]
        dx = gy - torch.einsum("t,th->th", along, xh)
        if case["kind"] == "layer":
            dx -= gy.sum(1, keepdim=True) / case["H"]
        dx = torch.einsum("th,t->th", dx, r)
        if d["d_sum"] is not None:
            dx += d["d_sum"]
        return {"dx": dx, "dweight": torch.einsum("th,th->h", d["dy"], xh),
                "dbias": torch.einsum("th->h", d["dy"]) if case["bias"] else None}
    if op.startswith("balance"):
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        valid = torch.ones(T, device="cuda", dtype=torch.bool) if t["mask"] is None else t["mask"].bool()
        seq = torch.arange(T, device="cuda") // (T // S)
        p = torch.softmax(d["logits"], 1)
        lse = torch.logsumexp(d["logits"], 1)
        n = torch.bincount(seq[valid], minlength=S).double()
        slot = (seq[:, None] * E + t["topk_idx"].long())[valid].reshape(-1)
        counts = torch.bincount(slot, minlength=S * E).reshape(S, E)
        f = counts.double() / (k * n.clamp(min=1)).unsqueeze(1)
        s_used = max(1, int((n > 0).sum()))
        n_all = max(1.0, float(n.sum()))
        if op == "balance_fwd":
            probs = torch.zeros(S, E, device="cuda", dtype=torch.float64).index_add_(0, seq[valid], p[valid])
            probs = probs / n.clamp(min=1).unsqueeze(1)
            loss = torch.stack([E * torch.sum(f * probs) / s_used, torch.sum(lse[valid] ** 2) / n_all])
            return {"loss": loss, "counts": None, "probs": probs, "tokens": None,
                    "lse": torch.where(valid, lse, torch.full_like(lse, math.inf))}
        w = G_BAL * E / (s_used * n.clamp(min=1))
        dp = w[seq].unsqueeze(1) * f[seq]  # d L_b / d p
        grad = p * dp - p * torch.sum(p * dp, 1, keepdim=True) + p * (2 * G_Z * lse / n_all).unsqueeze(1)
        return torch.where(valid.unsqueeze(1), grad, torch.zeros_like(grad)) + d["d_logits"]
    u, m = d["update"], None
    if t["momentum"] is not None:
        m = BETA * d["momentum"] + u
        u = u + BETA * m
    if case["R"] > case["C"]:
        u = u.mT
    norm = torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True).clamp(min=ORTHO_EPS)
    # on the small Gram matrices alone: each step multiplies X by a polynomial of X X^T, and all of them commute
    A = torch.bmm(u / norm, (u / norm).mT)
    Q = torch.eye(A.shape[1], device="cuda", dtype=torch.float64).expand_as(A)
    for _ in range(STEPS):
        P = COEFS[1] * A + COEFS[2] * torch.bmm(A, A)
        P.diagonal(dim1=1, dim2=2).add_(COEFS[0])
        Q = torch.bmm(P, Q)
        A = torch.bmm(torch.bmm(P, A), P)
    x = torch.bmm(Q, u / norm)
    return {"out": x.mT.contiguous() if case["R"] > case["C"] else x, "momentum": m}
