"""What the gate, the AdamW step and the dense layer are measured on: how a router's logits become a routing (sigmoid or
softmax scores, a bias for balance, groups), its gradient and the bias' step; one optimiser step over many tensors with
states in 32 or 8 bits; a matrix product with bias, activation and residual, forward and backward.

A case is one call of one operator.  `run` computes it in plain torch operations, or, where `own` is true, through the
framework's entry points.  `exact` gives the same outputs in 64 bits."""
import math

import torch

own = False

ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, decay=0.1)
BLOCK = 256  # elements that share a scale in 8-bit states
RATE = 1e-3  # of the gate's bias


def listed():
    return [
        # routing of the tiny configuration (T=512, E=8, top-2), softmax: latency is all there is
        dict(name="gate_fwd_t512_e8", op="gate_fwd", T=512, E=8, k=2, score="softmax", bias=False, groups=1, kept=1,
             best=1, renorm=True, scale=1.0),
        # the 30B routing shape with sigmoid scores and a bias for balance
        dict(name="gate_fwd_t16384_e128_bias", op="gate_fwd", T=16384, E=128, k=8, score="sigmoid", bias=True, groups=1,
             kept=1, best=1, renorm=True, scale=1.0),
        # a large batch over 256 experts in 8 groups, 4 of them kept by their two best experts
        dict(name="gate_fwd_t131072_e256_g8", op="gate_fwd", T=131072, E=256, k=8, score="sigmoid", bias=True, groups=8,
             kept=4, best=2, renorm=True, scale=2.5),
        # the gradient of that routing at the 30B shape, and the bias' step
        dict(name="gate_bwd_t16384_e128", op="gate_bwd", T=16384, E=128, k=8, score="sigmoid", bias=True, groups=1,
             kept=1, best=1, renorm=True, scale=1.0),
        # softmax weights that are not renormalised: every logit has a gradient; a large batch, no power of two of experts
        dict(name="gate_bwd_t100000_e250_softmax", op="gate_bwd", T=100000, E=250, k=6, score="softmax", bias=False,
             groups=1, kept=1, best=1, renorm=False, scale=16.0),
        # all tensors of a block of the tiny configuration: norm, router, experts; latency
        dict(name="adamw_block_tiny", op="adamw", H=128, I=64, E=8, layers=1, param="fp32", grad="bf16", state="fp32"),
        # the router, norm and 16 experts of the 235B shape, fp32 master weights with bf16 copies
        dict(name="adamw_h4096_i1536_e16", op="adamw", H=4096, I=1536, E=16, layers=1, param="fp32", grad="bf16",
             state="fp32"),
        # the same in 8-bit states
        dict(name="adamw_h4096_i1536_e16_8bit", op="adamw", H=4096, I=1536, E=16, layers=1, param="fp32", grad="bf16",
             state="8bit"),
        # a dense layer of the tiny configuration: latency
        dict(name="linear_fwd_t512_128x64", op="linear_fwd", T=512, K=128, N=64, act="gelu", bias=True, residual=False),
        # the down projection of a dense expert at the 235B shape, added to the routed experts' output
        dict(name="linear_fwd_t16384_1536x4096_res", op="linear_fwd", T=16384, K=1536, N=4096, act="none", bias=True,
             residual=True),
        # the up projection's backward at that shape
        dict(name="linear_bwd_t16384_4096x1536", op="linear_bwd", T=16384, K=4096, N=1536, act="silu", bias=True,
             residual=False),
        # a ragged batch and odd widths
        dict(name="linear_bwd_t777_1000x520", op="linear_bwd", T=777, K=1000, N=520, act="gelu", bias=True, residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate_fwd", "gate_fwd", "gate_bwd", "adamw", "adamw", "linear_fwd", "linear_bwd"])
    if op.startswith("gate"):
        E = rng.choice([8, 16, 60, 64, 128, 128, 160, 250, 256])
        k = min(E, rng.choice([1, 2, 4, 6, 8, 16]))
        groups, kept, best, bias = 1, 1, 1, rng.random() < 0.6
        if rng.random() < 0.4:
            groups = rng.choice([g for g in (2, 4, 5, 8, 10) if E % g == 0 and E // g >= 2])
            kept = rng.randint(-(-k * groups // E), groups)
            best = rng.choice([1, 2])
        return dict(op=op, T=_log(rng, 1, 131072), E=E, k=k, score=rng.choice(["softmax", "sigmoid", "sigmoid"]),
                    bias=bias, groups=groups, kept=kept, best=best, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 1.0, 2.5, 16.0]))
    if op == "adamw":
        H, I = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 192)
        if rng.random() < 0.3:
            H, I = H + rng.randint(1, 7), I + rng.randint(1, 7)
        E, layers = _log(rng, 1, max(1, min(64, 300_000_000 // (3 * H * I)))), 1
        if H * I * E < 10_000_000:
            layers = rng.randint(1, 3)
        return dict(op=op, H=H, I=I, E=E, layers=layers, param=rng.choice(["fp32", "fp32", "bf16"]),
                    grad=rng.choice(["bf16", "fp32"]), state=rng.choice(["fp32", "8bit"]))
    K, N = 8 * _log(rng, 8, 768), 8 * _log(rng, 4, 768)
    T = _log(rng, 1, max(1, min(32768, 100_000_000_000 // (K * N))))
    return dict(op=op, T=T, K=K, N=N, act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.7,
                residual=op == "linear_fwd" and rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------ inputs

_T = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _shapes(case):
    """The tensors of a block: norm weight and bias, router, experts; matrices alone decay."""
    H, I, E = case["H"], case["I"], case["E"]
    one = [(H,), (H,), (H, max(8, E)), (E, H, I), (E, H, I), (E, I, H)]
    return one * case["layers"]


def _layout(case):
    """(elements, offset in the states) of every tensor: each starts on a block of its own."""
    sizes = [math.prod(s) for s in _shapes(case)]
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    return sizes, at


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6971 + 29)

    def randn(*s, dtype=torch.float32):
        return torch.randn(*s, generator=g, device="cuda", dtype=dtype)

    op, t = case["op"], {}
    if op.startswith("gate"):
        T, E, k = case["T"], case["E"], case["k"]
        t["logits"] = randn(T, E) + 0.7 * randn(E)  # uneven expert loads
        # a bias that has been moved up and down in steps of its rate
        t["bias"] = torch.round(20 * randn(E)) * RATE if case["bias"] else None
        if op == "gate_bwd":
            r = _gate_plain(case, t)
            t.update(topk_idx=r["topk_idx"], topk_w=r["topk_w"], counts=r["counts"])
            t["d_topk_w"] = randn(T, k)
    elif op == "adamw":
        sizes, at = _layout(case)
        shapes = _shapes(case)
        t["params"] = [(0.02 * randn(*s)).to(_T[case["param"]]) for s in shapes]
        # gradients of uneven scale, as the rows of a layer's are
        t["grads"] = [(1e-3 * randn(*s) * torch.exp(randn(s[0]).view(-1, *[1] * (len(s) - 1)))).to(_T[case["grad"]])
                      for s in shapes]
        n = at[-1]
        if case["state"] == "fp32":
            m, v = 1e-3 * randn(n), 1e-6 * randn(n).square()
            for i, size in enumerate(sizes):  # the states of no element are zero
                m[at[i] + size:at[i + 1]] = 0
                v[at[i] + size:at[i + 1]] = 0
            t["state"] = {"m": m, "v": v}
        else:
            f8 = torch.float8_e4m3fn
            t["state"] = {"m": randn(n).mul_(100).clamp_(-448, 448).to(f8),
                          "v": randn(n).abs_().mul_(100).clamp_(0.01, 448).to(f8),
                          "m_scale": torch.rand(n // BLOCK, generator=g, device="cuda") * 2e-5 + 1e-6,
                          "v_scale": torch.rand(n // BLOCK, generator=g, device="cuda") * 2e-5 + 1e-5}
            for i, size in enumerate(sizes):
                t["state"]["m"].view(torch.uint8)[at[i] + size:at[i + 1]] = 0
                t["state"]["v"].view(torch.uint8)[at[i] + size:at[i + 1]] = 0
        t["state"]["step"] = torch.tensor([0, 9, 0, 0], dtype=torch.int32, device="cuda")  # status, steps so far, -, -
        t["copies"] = [p.to(torch.bfloat16) for p in t["params"]] if case["param"] == "fp32" else None
    else:
        T, K, N = case["T"], case["K"], case["N"]
        t["x"] = randn(T, K).to(torch.bfloat16)
        t["W"] = (randn(K, N) / math.sqrt(K)).to(torch.bfloat16)
        t["bias"] = (0.1 * randn(N)).to(torch.bfloat16) if case["bias"] else None
        if op == "linear_fwd":
            t["residual"] = randn(T, N).to(torch.bfloat16) if case["residual"] else None
        else:
            t["dy"] = randn(T, N).to(torch.bfloat16)
            t["z"] = randn(T, N).to(torch.bfloat16) if case["act"] != "none" else None  # what the forward keeps
    return t


def prepare(case, seed):
    # "out": the buffers of the last call's results, handed to the next one, as a training loop does
    state = {"case": case, "t": _inputs(case, seed), "op": None, "out": None}
    if own:
        from dropless_mixture_experts_top_gb300 import moe
        op = case["op"]
        if op.startswith("gate"):
            state["op"] = moe.Gate(case["T"], case["E"], case["k"], score=case["score"], groups=case["groups"],
                                   top_groups=case["kept"], group_best=case["best"], renormalise=case["renorm"],
                                   scale=case["scale"])
        elif op == "adamw":
            state["op"] = moe.AdamW(_shapes(case), param=case["param"], grad=case["grad"], state=case["state"],
                                    weight_decay=[ADAM["decay"] * (len(s) > 1) for s in _shapes(case)],
                                    beta1=ADAM["beta1"], beta2=ADAM["beta2"], eps=ADAM["eps"])
        else:
            state["op"] = moe.Linear(case["T"], case["K"], case["N"], activation=case["act"], bias=case["bias"])
    return state


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state["case"], state["t"], state["op"], state)


def _run_own(case, t, op, state):
    kind, out = case["op"], state["out"]
    if kind == "gate_fwd":
        state["out"] = out = op.forward(t["logits"], bias=t["bias"], out=out)
        return out
    if kind == "gate_bwd":
        state["out"] = out = op.backward(t["logits"], t["topk_idx"], t["topk_w"], t["d_topk_w"], d_logits=out)
        if t["bias"] is not None:
            op.update_bias(t["bias"], t["counts"], RATE)
        return {"d_logits": out, "bias": t["bias"]}
    if kind == "adamw":
        op.step(t["params"], t["grads"], t["state"], ADAM["lr"], copies=t["copies"])
        return {"params": t["params"], "copies": t["copies"], "state": t["state"]}
    if kind == "linear_fwd":
        state["out"] = out = op.forward(t["x"], t["W"], t["bias"], residual=t["residual"], out=out)
    else:
        state["out"] = out = op.backward(t["dy"], t["x"], t["W"], t["z"], grads=out)
    return out


def _gate_plain(case, t):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    logits = t["logits"]
    wide = logits.double()  # which experts: scores next to each other differ by less than 32 bits hold
    if case["score"] == "softmax":
        e = torch.exp(wide - wide.max(1, keepdim=True).values)
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-wide))
    c = s + t["bias"].double() if t["bias"] is not None else s
    order = c if t["bias"] is not None else wide
    if G > 1:
        top = (order if case["best"] == 1 else c).reshape(T, G, E // G).topk(case["best"], dim=2).values.sum(2)
        groups = torch.sort(top, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, groups, True)
        order = torch.where(keep.repeat_interleave(E // G, 1), order, torch.full_like(order, -math.inf))
    idx = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.float().gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    flat = idx.reshape(-1)
    slots = torch.sort(flat, stable=True).indices  # expert by expert, tokens ascending
    rows = torch.empty_like(slots).scatter_(0, slots, torch.arange(T * k, device=slots.device))
    counts = torch.zeros(E, dtype=torch.int64, device=slots.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)])
    i32 = torch.int32
    return {"topk_idx": idx.to(i32), "topk_w": w, "counts": counts.to(i32), "offsets": offsets.to(i32),
            "row_of_slot": rows.to(i32).reshape(T, k), "slot_of_row": slots.to(i32), "w_row": w.reshape(-1)[slots]}


def _gate_grad_plain(case, t):
    idx, d = t["topk_idx"].long(), t["d_topk_w"]
    logits, scale = t["logits"], case["scale"]
    if case["score"] == "sigmoid":
        l = logits.gather(1, idx)
        s = 1 / (1 + torch.exp(-l))
        far = 1 / (1 + torch.exp(l))  # 1 - s
        if case["renorm"]:
            n = s / s.sum(1, keepdim=True)
            at = scale * n * far * (d - (n * d).sum(1, keepdim=True))
        else:
            at = scale * s * far * d
        return torch.zeros_like(logits).scatter_(1, idx, at)
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    n = p.gather(1, idx)
    if case["renorm"]:
        n = n / n.sum(1, keepdim=True)
        return torch.zeros_like(logits).scatter_(1, idx, scale * n * (d - (n * d).sum(1, keepdim=True)))
    out = p * (-scale * (n * d).sum(1, keepdim=True))
    return out.scatter_add_(1, idx, scale * n * d)


def _to_8bit(x, least):
    """Blocks of x as e4m3 values and their scales; `least`: a positive value keeps at least the smallest code."""
    most = x.abs().amax(1, keepdim=True).clamp(min=1e-30)
    q = x * (448.0 / most)
    if least:
        q = torch.where((x > 0) & (q < 2.0 ** -9), torch.full_like(q, 2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn), (most * (1 / 448.0))[:, 0]


def _adamw_plain(case, t, i, corr1, corr2):
    sizes, at = _layout(case)
    st, n, lo, hi = t["state"], sizes[i], at[i], at[i + 1]
    b1, b2, lr, eps = ADAM["beta1"], ADAM["beta2"], ADAM["lr"], ADAM["eps"]
    decay = ADAM["decay"] if t["params"][i].dim() > 1 else 0.0
    g, p = t["grads"][i].reshape(-1).float(), t["params"][i].reshape(-1).float()
    eight = case["state"] == "8bit"
    if eight:
        blocks = slice(lo // BLOCK, hi // BLOCK)
        m = st["m"][lo:hi].view(-1, BLOCK).float() * st["m_scale"][blocks, None]
        r = st["v"][lo:hi].view(-1, BLOCK).float() * st["v_scale"][blocks, None]
        m, v = m.reshape(-1)[:n], (r * r).reshape(-1)[:n]
    else:
        m, v = st["m"][lo:lo + n], st["v"][lo:lo + n]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * (g * g)
    r = torch.sqrt(v)
    p = p * (1 - lr * decay) - (lr / corr1) * m / (r / torch.sqrt(corr2) + eps)
    t["params"][i].copy_(p.view_as(t["params"][i]))
    if t["copies"] is not None:
        t["copies"][i].copy_(p.view_as(t["params"][i]))
    if eight:
        pad = (0, hi - lo - n)
        m, m_scale = _to_8bit(torch.nn.functional.pad(m, pad).view(-1, BLOCK), False)
        r, v_scale = _to_8bit(torch.nn.functional.pad(r, pad).view(-1, BLOCK), True)
        st["m"][lo:hi].copy_(m.reshape(-1))
        st["v"][lo:hi].copy_(r.reshape(-1))
        st["m_scale"][blocks] = m_scale
        st["v_scale"][blocks] = v_scale
    else:
        m_old, v_old = st["m"][lo:lo + n], st["v"][lo:lo + n]
        m_old.copy_(m)
        v_old.copy_(v)


_ACT = {
    "none": (lambda z: z, lambda z: torch.ones_like(z)),
    "relu": (lambda z: z.clamp(min=0), lambda z: (z > 0).to(z.dtype)),
    "silu": (lambda z: z * torch.sigmoid(z), lambda z: torch.sigmoid(z) * (1 + z * (1 - torch.sigmoid(z)))),
}


def _gelu_inner(z):
    return math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)


def _gelu(z):
    return 0.5 * z * (1 + torch.tanh(_gelu_inner(z)))


def _gelu_slope(z):
    h = torch.tanh(_gelu_inner(z))
    return 0.5 * (1 + h) + 0.5 * z * (1 - h * h) * (math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z))


_ACT["gelu"] = (_gelu, _gelu_slope)


def _run_plain(case, t, op, state):
    kind = case["op"]
    if kind == "gate_fwd":
        return _gate_plain(case, t)
    if kind == "gate_bwd":
        d = _gate_grad_plain(case, t)
        if t["bias"] is not None:
            c = t["counts"].long()
            t["bias"].add_(torch.sign(c.sum() - case["E"] * c).float(), alpha=RATE)
        return {"d_logits": d, "bias": t["bias"]}
    if kind == "adamw":
        steps = t["state"]["step"]
        steps[1] += 1
        n = steps[1].double()  # the number of steps stays on the device
        corr1, corr2 = (1 - ADAM["beta1"] ** n).float(), (1 - ADAM["beta2"] ** n).float()
        [_adamw_plain(case, t, i, corr1, corr2) for i in range(len(t["params"]))]
        return {"params": t["params"], "copies": t["copies"], "state": t["state"]}
    act, slope = _ACT[case["act"]]
    if kind == "linear_fwd":
        z = t["x"].float() @ t["W"].float()
        if t["bias"] is not None:
            z = z + t["bias"].float()
        y = act(z)
        if t["residual"] is not None:
            y = y + t["residual"].float()
        return {"y": y.to(torch.bfloat16), "z": z.to(torch.bfloat16) if case["act"] != "none" else None}
    dz = t["dy"].float()
    if t["z"] is not None:
        dz = dz * slope(t["z"].float())
    return {"dx": (dz @ t["W"].float().T).to(torch.bfloat16), "dW": (t["x"].float().T @ dz).to(torch.bfloat16),
            "dbias": dz.sum(0) if case["bias"] else None}


# ------------------------------------------------------------------------------------------------ the least work

def work(case):
    op = case["op"]
    if op.startswith("gate"):
        T, E, k = case["T"], case["E"], case["k"]
        if op == "gate_fwd":
            return {"bytes": T * (4 * E + 20 * k) + 4 * E, "flops": 10 * T * E}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * (4 * E + 16 * k + (4 * E if dense else 0)), "flops": (8 * T * E if dense else 12 * T * k)}
    if op == "adamw":
        n = _layout(case)[0]
        el = {"bf16": 2, "fp32": 4}
        each = 2 * el[case["param"]] + el[case["grad"]] + (2 if case["param"] == "fp32" else 0)
        each += 16 if case["state"] == "fp32" else 4 + 16 / BLOCK
        return {"bytes": each * sum(n), "flops": 16 * sum(n)}
    T, K, N = case["T"], case["K"], case["N"]
    act = case["act"] != "none"
    if op == "linear_fwd":
        return {"bytes": 2 * (T * K + K * N + T * N * (1 + case["residual"] + act)), "flops": 2 * T * K * N}
    return {"bytes": 2 * (2 * T * K + 2 * K * N + T * N * (1 + act)), "flops": 4 * T * K * N}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    t, op = _inputs(case, seed), case["op"]
    if op.startswith("gate"):
        T, E, k, scale = case["T"], case["E"], case["k"], case["scale"]
        l = t["logits"].double()
        s = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
        if op == "gate_fwd":
            c = s if t["bias"] is None else s + t["bias"].double()
            if case["groups"] > 1:
                per = c.unflatten(1, (case["groups"], -1))
                best = torch.sort(per, dim=2, descending=True).values[..., :case["best"]].sum(-1)
                # a group's place: those that are better, and the equal ones in front of it
                before = (best[:, None, :] > best[:, :, None]).sum(2)
                c = torch.where((before < case["kept"]).unsqueeze(2), per, torch.full_like(per, -1e9)).flatten(1)
            idx = torch.argsort(c, dim=1, descending=True, stable=True)[:, :k]
            w = torch.take_along_dim(s, idx, 1)
            w = scale * (w / w.sum(1, keepdim=True) if case["renorm"] else w)
            by = torch.argsort(idx.flatten(), stable=True)
            return {"topk_idx": None, "topk_w": w, "counts": None, "offsets": None, "row_of_slot": None,
                    "slot_of_row": None, "w_row": w.flatten()[by]}
        # by the chain rule over all experts: d s, then through softmax or sigmoid
        idx = t["topk_idx"].long()
        chosen = torch.zeros_like(s).scatter_(1, idx, 1.0)
        d = torch.zeros_like(s).scatter_(1, idx, t["d_topk_w"].double())
        if case["renorm"]:
            total = (s * chosen).sum(1, keepdim=True)
            ds = scale * chosen * (d / total - (s * d).sum(1, keepdim=True) / total ** 2)
        else:
            ds = scale * d
        if case["score"] == "softmax":
            dl = s * ds - s * (s * ds).sum(1, keepdim=True)
        else:
            dl = ds * s * torch.sigmoid(-l)
        b = None
        if t["bias"] is not None:
            c = t["counts"].double()
            b = t["bias"].double() + RATE * torch.sign(c.mean() - c)
        return {"d_logits": dl, "bias": b}
    if op == "adamw":
        sizes, at = _layout(case)
        n, eight, st = 10, case["state"] == "8bit", t["state"]
        b1, b2, lr = ADAM["beta1"], ADAM["beta2"], ADAM["lr"]
        ms = torch.zeros(at[-1], dtype=torch.float64, device="cuda")
        vs, params = torch.zeros_like(ms), []
        for i, p in enumerate(t["params"]):
            lo, hi = at[i], at[i] + sizes[i]
            m, v, g, w = st["m"][lo:hi].double(), st["v"][lo:hi].double(), t["grads"][i].double().flatten(), p.double().flatten()
            if eight:
                block = torch.arange(lo, hi, device="cuda") // BLOCK
                m, v = m * st["m_scale"].double()[block], (v * st["v_scale"].double()[block]).square()
            m = torch.lerp(g, m, b1)
            v = torch.lerp(g.square(), v, b2)
            step = lr * (m / (1 - b1 ** n)) / ((v / (1 - b2 ** n)).sqrt() + ADAM["eps"])
            w = w - lr * (ADAM["decay"] if p.dim() > 1 else 0.0) * w - step
            params.append(w.view(p.shape))
            ms[lo:hi], vs[lo:hi] = m, v.sqrt() if eight else v
        state = {"m": ms, "v": vs, "step": None}
        if eight:
            for name, x in (("m", ms), ("v", vs)):
                s = x.view(-1, BLOCK).abs().amax(1).clamp(min=1e-30) / 448
                state[name] = (x.view(-1, BLOCK) / s[:, None]).flatten()  # in units of the scale, not rounded
                state[name + "_scale"] = s
        return {"params": params, "copies": params if t["copies"] is not None else None, "state": state}
    d = {k: v.double() if v is not None else None for k, v in t.items()}
    z = {"none": None, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[case["act"]]
    if op == "linear_fwd":
        y = torch.einsum("tk,kn->tn", d["x"], d["W"])
        if d["bias"] is not None:
            y += d["bias"]
        out = z(y) if z else y
        return {"y": out + d["residual"] if d["residual"] is not None else out, "z": y if z else None}
    dz = d["dy"]
    if z:
        at = d["z"].requires_grad_()
        dz, = torch.autograd.grad(z(at), at, d["dy"])
    return {"dx": torch.einsum("tn,kn->tk", dz, d["W"]), "dW": torch.einsum("tk,tn->kn", d["x"], dz),
            "dbias": dz.sum(0) if case["bias"] else None}
