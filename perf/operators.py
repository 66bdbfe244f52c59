"""The training-step operators around the optimizer, as timed cases: the gated
feed-forward product (forward; forward and backward), the block norms with
gate and residual scale (forward; backward) and distillation from a teacher's
top logits (forward; forward and gradient; forward, then backward).

`run` has two forms of each.  With `own` false it computes the formulas in
elementary torch operations in float32, rounded once at the end; with `own`
true it makes the calls of this repository's package.  `exact` evaluates the
definitions in float64.

Formulas, with x [T, D], W_g and W_u [F, D]:
  feed-forward   g = x W_g^T, u = x W_u^T, h = act(g) * u;
                 dg = dh * u * act'(g), du = dh * act(g);
                 dx = dg W_g + du W_u, dW_g = dg^T x, dW_u = du^T x.
  block norm     r' = scale * r + gate * N_post(y),  z = N_pre(r'), where
                 N(v) = (v - mean) / sqrt(var + eps) * w + b (layer) or
                 v / sqrt(mean(v^2) + eps) * w (rms); z sees r' unrounded.
  distillation   p = softmax(teacher / tau) over the row's valid entries,
                 q = softmax(logits / tau):
                 loss = kd * tau^2 * sum_k p_k (log p_k - log q_{id_k})
                        + ce * (logsumexp(logits) - logits[label]).
"""
import math

import torch

own = False

SILU, GELU_TANH, GELU = 0, 1, 2          # activations, as the package numbers them
NONE, RMS, LAYER = 0, 1, 2               # kinds of norm
EPS = 1e-5


# ------------------------------------------------------------------- the cases

def _ff(name, mode, T, D, F, act):
    return {"name": name, "op": "ff", "mode": mode, "T": T, "D": D, "F": F, "act": act}


def _norm(name, mode, T, D, kind, gates, f32, bias):
    """gates: rows of the gate matrix (0: no gate; 1: one learned gate; else a gate for each T / gates tokens)."""
    return {"name": name, "op": "norm", "mode": mode, "T": T, "D": D, "kind": kind, "gates": gates, "f32": f32,
            "bias": bias, "scale": 1.0 if gates else 0.75}


def _loss(name, mode, T, V, K, tau, kd, ce, f32):
    return {"name": name, "op": "loss", "mode": mode, "T": T, "V": V, "K": K, "tau": tau, "kd": kd, "ce": ce, "f32": f32}


def listed():
    return [
        # one token through a GPT-2 350M sized layer: sampling from the model between training steps; latency
        _ff("ff token 350M", "forward", 1, 1024, 4096, SILU),
        # a small batch of tokens through a GPT-Neo 2.7B sized layer: the weights' bytes bound it
        _ff("ff 24 tokens 2.7B", "forward", 24, 2560, 10240, GELU_TANH),
        # a ragged micro-batch of GPT-2 XL 1.5B training, forward and backward
        _ff("ff train 1.5B ragged", "train", 1023, 1600, 6400, GELU),
        # a full micro-batch of GPT-Neo 6.7B training, forward and backward: the largest matrix products
        _ff("ff train 6.7B", "train", 8192, 4096, 16384, SILU),
        # one token's norms, GPT-2 350M width; latency
        _norm("norm token 350M", "forward", 1, 1024, RMS, 1, False, False),
        # the norms of a full micro-batch, GPT-Neo 6.7B width
        _norm("norm forward 6.7B", "forward", 16384, 4096, RMS, 1, False, False),
        # an odd width and a float32 residual stream with layer norms and biases
        _norm("norm backward odd", "backward", 3001, 1601, LAYER, 0, True, True),
        # the backward of a full micro-batch of eight sequences, each with its own gate
        _norm("norm backward 6.7B", "backward", 16384, 4096, RMS, 8, False, False),
        # one row of GPT-2's vocabulary: a held-out token scored against its teacher; latency
        _loss("loss row", "forward", 1, 50257, 16, 1.0, 1.0, 0.0, False),
        # a held-out batch's losses
        _loss("loss forward", "forward", 4096, 50257, 64, 1.0, 1.0, 0.0, False),
        # the loss and its gradient for a full micro-batch, with the labels' term mixed in
        _loss("loss train", "train", 8192, 50257, 64, 2.0, 0.7, 0.3, False),
        # a wide odd vocabulary with float32 logits, as autograd runs it: forward, then backward
        _loss("loss wide float32", "split", 1001, 128001, 100, 1.5, 1.0, 0.5, True),
    ]


def _between(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Three of four sizes are multiples of 8, as model widths are; the others come as they fall."""
    n = _between(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["ff", "norm", "loss"])
    if op == "ff":
        D, F = _size(rng, 256, 4096), _size(rng, 512, 16384)
        T = _between(rng, 1, 8192)
        c = _ff("", rng.choice(["forward", "train"]), T, D, F, rng.choice([SILU, GELU_TANH, GELU]))
    elif op == "norm":
        D, T = _size(rng, 64, 8192), _between(rng, 1, 16384)
        T = min(T, 16384 * 4096 // D)
        gates = rng.choice([0, 1, 1, 2, 7, T])
        if gates > 1:
            gates = min(gates, T)
            T = T // gates * gates
        c = _norm("", rng.choice(["forward", "backward"]), T, D, rng.choice([RMS, LAYER]), gates,
                  rng.random() < 0.25, rng.random() < 0.5)
    else:
        V, T = _size(rng, 500, 160000), _between(rng, 1, 8192)
        f32 = rng.random() < 0.25
        T = max(1, min(T, 8192 * 50257 // (V * (2 if f32 else 1))))
        c = _loss("", rng.choice(["forward", "train", "split"]), T, V, _between(rng, 1, 128),
                  rng.choice([1.0, 1.5, 2.0, 4.0]), rng.choice([1.0, 0.7]), rng.choice([0.0, 0.3]), f32)
    del c["name"]
    return c


def work(case):
    T = case["T"]
    if case["op"] == "ff":
        D, F = case["D"], case["F"]
        if case["mode"] == "forward":
            return {"bytes": 2 * (T * D + 2 * F * D + T * F), "flops": 4 * T * F * D + 8 * T * F}
        return {"bytes": 2 * (2 * T * D + 4 * F * D + 2 * T * F), "flops": 12 * T * F * D + 20 * T * F}
    if case["op"] == "norm":
        D, r = case["D"], 4 if case["f32"] else 2
        chans = 2 * D * (2 + (2 if case["bias"] else 0) + case["gates"])
        if case["mode"] == "forward":
            return {"bytes": T * D * (2 * r + 4) + chans, "flops": 14 * T * D}
        return {"bytes": T * D * (3 * r + 6) + 2 * chans, "flops": 40 * T * D}
    V, K, e = case["V"], case["K"], 4 if case["f32"] else 2
    rows = T * (K * 12 + 8 + 4 + 4)
    if case["mode"] == "forward":
        return {"bytes": T * V * e + rows, "flops": 6 * T * V}
    return {"bytes": 2 * T * V * e + rows, "flops": 10 * T * V}


# ------------------------------------------------------------------ the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 13)
    bf = torch.bfloat16

    def normal(*shape, std=1.0, mean=0.0, dtype=bf):
        out = torch.empty(shape, device=dev, dtype=dtype)
        flat = out.view(-1)
        step = 1 << 26
        for i in range(0, flat.numel(), step):
            n = min(step, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, generator=gen, device=dev) * std + mean
        return out

    def empty(*shape, dtype=bf):
        return torch.empty(shape, device=dev, dtype=dtype)

    T, s = case["T"], dict(case)
    if case["op"] == "ff":
        D, F = case["D"], case["F"]
        # normalised activations against weights of standard deviation 0.02, or
        # 1 / sqrt(D) where the layer is narrow: pre-activations of order one
        std = max(0.02, D ** -0.5)
        s.update(x=normal(T, D), w_gate=normal(F, D, std=std), w_up=normal(F, D, std=std), h=empty(T, F))
        if case["mode"] == "train":
            s.update(dh=normal(T, F, std=1e-2), saved=empty(2, T, F, dtype=torch.float32), dx=empty(T, D),
                     dw_gate=empty(F, D), dw_up=empty(F, D))
        return s
    if case["op"] == "norm":
        D, G, rd = case["D"], case["gates"], torch.float32 if case["f32"] else bf
        r = normal(T, D, std=2.0, dtype=rd)
        r[:, :: max(1, D // 4)] *= 8                   # a few channels of a residual stream are far larger than the rest
        s.update(r=r, y=normal(T, D, std=0.5, mean=0.1), post_w=normal(D, std=0.2, mean=1.0),
                 pre_w=normal(D, std=0.2, mean=1.0), post_b=None, pre_b=None, gate=None)
        if case["bias"]:
            s.update(post_b=normal(D, std=0.1), pre_b=normal(D, std=0.1))
        if G:
            s["gate"] = normal(G, D, std=0.3, mean=0.5)
        if case["mode"] == "forward":
            s.update(r_out=empty(T, D, dtype=rd), z=empty(T, D))
        else:
            s.update(dr_out=normal(T, D, std=1e-2, dtype=rd), dz=normal(T, D, std=1e-2), dr=empty(T, D, dtype=rd),
                     dy=empty(T, D), dpost_w=empty(D), dpre_w=empty(D), dpost_b=empty(D) if case["bias"] else None,
                     dpre_b=empty(D) if case["bias"] else None, dgate=empty(G, D) if G else None)
        return s
    V, K, dt = case["V"], case["K"], torch.float32 if case["f32"] else bf
    K = min(K, V)
    logits = normal(T, V, std=2.0, dtype=dt)
    # distinct ids: an arithmetic walk over the vocabulary; the teacher's logits fall off by random gaps
    start = torch.randint(0, V, (T, 1), generator=gen, device=dev)
    pace = torch.randint(1, max(2, V // K + 1), (T, 1), generator=gen, device=dev)
    ids = (start + pace * torch.arange(K, device=dev)) % V
    gaps = -torch.log(torch.rand(T, K, generator=gen, device=dev).clamp_min(1e-6))
    teacher = 14.0 - torch.cumsum(gaps, 1) * (6.0 / K ** 0.5)
    for i in range(0, T, 1024):                       # the student agrees with the teacher in part
        t = slice(i, i + 1024)
        logits[t] = logits[t].scatter_add(1, ids[t], (0.7 * teacher[t]).to(dt))
    labels = torch.where(torch.rand(T, generator=gen, device=dev) < 0.8, ids[:, 0],
                         torch.randint(0, V, (T,), generator=gen, device=dev))
    if T > 3:                                          # padding: rows without a teacher, without a label, with neither
        u = torch.rand(T, generator=gen, device=dev)
        ids[u < 0.05] = -1
        labels[(u > 0.02) & (u < 0.10)] = -100
        labels[u < 0.01] = -100
        ids[:, K // 2:][(u > 0.9)] = -1                # and rows with fewer entries than the others
    weight = torch.full((T,), 1.0 / T, device=dev)
    s.update(logits=logits, ids=ids, teacher=teacher.contiguous(), labels=labels, weight=weight,
             loss=empty(T, dtype=torch.float32))
    if case["mode"] != "forward":
        s["dlogits"] = empty(T, V, dtype=dt)
    if case["mode"] == "split":
        s["stats"] = empty(T, 2, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- one pass each

def run(s):
    if own:
        return {"ff": _own_ff, "norm": _own_norm, "loss": _own_loss}[s["op"]](s)
    return {"ff": _plain_ff, "norm": _plain_norm, "loss": _plain_loss}[s["op"]](s)


def _own_ff(s):
    import bit_blockwise_adamw_gb300 as q8
    if s["mode"] == "forward":
        q8.q8_gated_ff_forward(s["x"], s["w_gate"], s["w_up"], s["h"], s["act"])
        return {"h": s["h"]}
    q8.q8_gated_ff_forward(s["x"], s["w_gate"], s["w_up"], s["h"], s["act"], saved=s["saved"])
    q8.q8_gated_ff_backward(s["x"], s["w_gate"], s["w_up"], s["dh"], s["dx"], s["dw_gate"], s["dw_up"], s["act"],
                            saved=s["saved"])
    return {k: s[k] for k in ("h", "dx", "dw_gate", "dw_up")}


def _own_norm(s):
    import bit_blockwise_adamw_gb300 as q8
    chans = dict(post_weight=s["post_w"], post_bias=s["post_b"], pre_weight=s["pre_w"], pre_bias=s["pre_b"],
                 gate=s["gate"], residual_scale=s["scale"], eps=EPS)
    if s["mode"] == "forward":
        q8.q8_block_norm_forward(s["r"], s["y"], s["r_out"], s["z"], s["kind"], s["kind"], **chans)
        return {"r_out": s["r_out"], "z": s["z"]}
    q8.q8_block_norm_backward(s["r"], s["y"], s["dr_out"], s["dz"], s["dr"], s["dy"], s["kind"], s["kind"], **chans,
                              dpost_weight=s["dpost_w"], dpost_bias=s["dpost_b"], dpre_weight=s["dpre_w"],
                              dpre_bias=s["dpre_b"], dgate=s["dgate"])
    return {k: s[k] for k in ("dr", "dy", "dpost_w", "dpre_w", "dpost_b", "dpre_b", "dgate") if s[k] is not None}


def _own_loss(s):
    import bit_blockwise_adamw_gb300 as q8
    opts = dict(labels=s["labels"], temperature=s["tau"], kd_weight=s["kd"], ce_weight=s["ce"])
    if s["mode"] == "forward":
        q8.q8_distill_topk_forward(s["logits"], s["ids"], s["teacher"], s["loss"], **opts)
        return {"loss": s["loss"]}
    if s["mode"] == "train":
        q8.q8_distill_topk_forward(s["logits"], s["ids"], s["teacher"], s["loss"], dlogits=s["dlogits"],
                                   row_weight=s["weight"], **opts)
    else:
        q8.q8_distill_topk_forward(s["logits"], s["ids"], s["teacher"], s["loss"], stats=s["stats"], **opts)
        q8.q8_distill_topk_backward(s["logits"], s["ids"], s["teacher"], s["stats"], s["dlogits"],
                                    row_weight=s["weight"], **opts)
    return {"loss": s["loss"], "dlogits": s["dlogits"]}


def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == SILU:
        e = 1.0 / (1.0 + torch.exp(-g))
        return g * e, e * (1.0 + g * (1.0 - e))
    if kind == GELU_TANH:
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
    cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2 * math.pi))


def _plain_ff(s):
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, s["act"])
    h = (a * u).bfloat16()
    if s["mode"] == "forward":
        return {"h": h}
    dh = s["dh"].float()
    dg, du = dh * u * da, dh * a
    return {"h": h, "dx": (dg @ wg + du @ wu).bfloat16(), "dw_gate": (dg.t() @ x).bfloat16(),
            "dw_up": (du.t() @ x).bfloat16()}


def _stats(v, kind):
    """The normalised rows and the reciprocal of each row's root."""
    if kind == LAYER:
        v = v - v.mean(1, keepdim=True)
    rs = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * rs, rs


def _affine(n, w, b):
    return n * w if b is None else n * w + b


def _norm_grad(dn, n, rs, kind):
    """The gradient of the rows from that of the normalised rows."""
    d = dn - n * (dn * n).mean(1, keepdim=True)
    return rs * (d - dn.mean(1, keepdim=True) if kind == LAYER else d)


def _plain_norm(s):
    f = {k: None if s[k] is None else s[k].float() for k in ("post_w", "post_b", "pre_w", "pre_b", "gate")}
    r, y, kind, G, (T, D) = s["r"].float(), s["y"].float(), s["kind"], s["gates"], s["y"].shape
    yn, yrs = _stats(y, kind)
    post = _affine(yn, f["post_w"], f["post_b"])
    gate = f["gate"].repeat_interleave(T // G, 0) if G else None
    r_out = s["scale"] * r + (post if gate is None else gate * post)
    rn, rrs = _stats(r_out, kind)
    if s["mode"] == "forward":
        return {"r_out": r_out.to(s["r"].dtype), "z": _affine(rn, f["pre_w"], f["pre_b"]).bfloat16()}
    dz = s["dz"].float()
    d = s["dr_out"].float() + _norm_grad(dz * f["pre_w"], rn, rrs, kind)
    dpost = d if gate is None else d * gate
    out = {"dr": (s["scale"] * d).to(s["r"].dtype), "dy": _norm_grad(dpost * f["post_w"], yn, yrs, kind).bfloat16(),
           "dpost_w": (dpost * yn).sum(0).bfloat16(), "dpre_w": (dz * rn).sum(0).bfloat16()}
    if s["bias"]:
        out.update(dpost_b=dpost.sum(0).bfloat16(), dpre_b=dz.sum(0).bfloat16())
    if G:
        out["dgate"] = (d * post).view(G, T // G, D).sum(1).bfloat16()
    return out


def _plain_loss(s):
    z, tau, kd, ce = s["logits"].float(), s["tau"], s["kd"], s["ce"]
    valid, ids = s["ids"] >= 0, s["ids"].clamp_min(0)
    taught = valid.any(1)
    t = torch.where(valid, s["teacher"].float() / tau, -math.inf)
    top = torch.where(taught, t.amax(1), 0.0)
    pe = torch.where(valid, torch.exp(t - top[:, None]), 0.0)
    p = pe / torch.where(taught, pe.sum(1), 1.0)[:, None]
    most = z.amax(1, keepdim=True)
    qe = torch.exp((z - most) / tau)
    qs = qe.sum(1, keepdim=True)
    logq = (z.gather(1, ids) - most) / tau - torch.log(qs)
    loss = kd * tau * tau * torch.where(p > 0, p * (torch.log(p) - logq), 0.0).sum(1)
    labelled = s["labels"] >= 0
    label = s["labels"].clamp_min(0)[:, None]
    if ce:
        e = torch.exp(z - most)
        es = e.sum(1, keepdim=True)
        loss = loss + ce * torch.where(labelled, (torch.log(es) + most - z.gather(1, label))[:, 0], 0.0)
    if s["mode"] == "forward":
        return {"loss": loss}
    w = s["weight"]
    d = (qe / qs) * (kd * tau * w * taught)[:, None]
    d = d.scatter_add(1, ids, -(kd * tau * w)[:, None] * p)
    if ce:
        d = d + (e / es) * (ce * w * labelled)[:, None]
        d = d.scatter_add(1, label, -(ce * w * labelled)[:, None])
    return {"loss": loss, "dlogits": d.to(s["logits"].dtype)}


# ------------------------------------------------------------ float64 definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"ff": _exact_ff, "norm": _exact_norm, "loss": _exact_loss}[case["op"]](s)


def _exact_ff(s):
    T, D, F = s["T"], s["D"], s["F"]
    if T * D * F * (12 if s["mode"] == "train" else 4) > 1.2e13:
        return None
    x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()
    g = torch.matmul(x, wg.mT).requires_grad_(s["mode"] == "train")
    u = torch.matmul(x, wu.mT).requires_grad_(s["mode"] == "train")
    if s["act"] == SILU:
        h = g * torch.sigmoid(g) * u
    else:
        h = torch.nn.functional.gelu(g, approximate="tanh" if s["act"] == GELU_TANH else "none") * u
    if s["mode"] == "forward":
        return {"h": h}
    dg, du = torch.autograd.grad(h, (g, u), s["dh"].double())
    return {"h": h.detach(), "dx": torch.matmul(dg, wg) + torch.matmul(du, wu), "dw_gate": torch.matmul(dg.mT, x),
            "dw_up": torch.matmul(du.mT, x)}


def _exact_norm(s):
    """The definition in float64, its gradients by automatic differentiation of it, some rows at a time."""
    T, D, G = s["T"], s["D"], s["gates"]
    back = s["mode"] == "backward"
    names = [k for k in ("post_w", "post_b", "pre_w", "pre_b", "gate") if s[k] is not None]
    par = {k: s[k].double().requires_grad_(back) for k in names}

    def norm(v, w, b):
        if s["kind"] == LAYER:
            return torch.nn.functional.layer_norm(v, (D,), w, b, EPS)
        n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w
        return n if b is None else n + b

    got = {k: [] for k in (("dr", "dy") if back else ("r_out", "z"))}
    sums = {k: 0.0 for k in names}
    group = torch.arange(T, device=s["y"].device) // max(1, T // max(1, G))
    step = max(1, (1 << 26) // D)
    for i in range(0, T, step):
        t = slice(i, i + step)
        r, y = s["r"][t].double().requires_grad_(back), s["y"][t].double().requires_grad_(back)
        post = norm(y, par["post_w"], par.get("post_b"))
        r_out = s["scale"] * r + (post * par["gate"][group[t]] if G else post)
        z = norm(r_out, par["pre_w"], par.get("pre_b"))
        if not back:
            got["r_out"].append(r_out)
            got["z"].append(z)
            continue
        total = (r_out * s["dr_out"][t].double()).sum() + (z * s["dz"][t].double()).sum()
        grads = torch.autograd.grad(total, [r, y] + [par[k] for k in names])
        got["dr"].append(grads[0])
        got["dy"].append(grads[1])
        for k, v in zip(names, grads[2:]):
            sums[k] = sums[k] + v
    out = {k: torch.cat(v) for k, v in got.items()}
    if back:
        out.update({"d" + k: v for k, v in sums.items()})
    return out


def _exact_loss(s):
    """Row by row of the definition: log-softmax of both sides, in float64."""
    tau, kd, ce, back = s["tau"], s["kd"], s["ce"], s["mode"] != "forward"
    T, V = s["logits"].shape
    loss, grad = [], []
    step = max(1, (1 << 26) // V)
    for i in range(0, T, step):
        t = slice(i, i + step)
        z = s["logits"][t].double().requires_grad_(back)
        ids, labels = s["ids"][t], s["labels"][t]
        some = (ids >= 0).any(1)
        teach = s["teacher"][t].double().div(tau).masked_fill(ids < 0, -1e300)
        logp = torch.log_softmax(teach, 1)
        logq = torch.log_softmax(z / tau, 1).gather(1, ids.clamp_min(0))
        p = logp.exp() * (ids >= 0)
        row = kd * tau ** 2 * (p * (logp.clamp_min(-1e4) - logq)).sum(1) * some
        if ce:
            nll = torch.nn.functional.cross_entropy(z, labels, ignore_index=-100, reduction="none")
            row = row + ce * nll
        loss.append(row.detach())
        if back:
            grad.append(torch.autograd.grad((row * s["weight"][t].double()).sum(), z)[0].to(torch.float64))
    if not back:
        return {"loss": torch.cat(loss)}
    return {"loss": torch.cat(loss), "dlogits": torch.cat(grad)}
