"""The operators at the two ends of a training step, as timed cases: the token
embedding (lookup with a scale; its table's gradient), and between the backward
pass and the optimizer the norm of all gradients and their clipping.

`run` has two forms of each.  With `own` false it computes the formulas in
elementary torch operations in float32, rounded once at the end (long sums of
squares are joined in float64); with `own` true it makes the calls of this
repository's package.  `exact` evaluates the definitions in float64.

Formulas, with a table W [V, D], ids [T] and gradients g_i of any sizes:
  lookup    out[t] = scale * W[ids[t]], zeros where ids[t] lies outside [0, V)
  gradient  dW[v] = scale * (sum of dout[t] with ids[t] = v), zeros where none
  norm      n = sqrt(sum over all tensors and elements of g^2)
  clipping  g' = c * g with c = min(1, max_norm / (n + 1e-6))
"""
import math

import numpy as np
import torch

own = False

BF, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F32}
SLOT = 64                                # a tensor's place in a flat buffer starts at a multiple of so many elements


# ------------------------------------------------------------------- the cases

def _embed(name, mode, T, V, D, scale, dt, pad=0.0, none=0.0):
    """pad: share of tokens that are one same token (padding with a row of its own); none: of tokens without a row."""
    return {"name": name, "op": "embed", "mode": mode, "T": T, "V": V, "D": D, "scale": scale, "dt": dt, "pad": pad, "none": none}


def _model(name, mode, L, d, ffn, ctx, V=50257, only="all"):
    """The gradients of a transformer as its optimizer gets them; only "vectors": of its norms and biases alone."""
    return {"name": name, "op": "grads", "mode": mode, "L": L, "d": d, "ffn": ffn, "ctx": ctx, "V": V, "only": only,
            "dt": "bf16", "out": "bf16", "max": 1.0}


def _ragged(name, mode, count, lo, hi, dt, out, limit):
    """`count` tensors of odd and even sizes between lo and hi, from one to the other by equal factors."""
    return {"name": name, "op": "grads", "mode": mode, "count": count, "lo": lo, "hi": hi, "dt": dt, "out": out, "max": limit}


def listed():
    return [
        # one token of a GPT-2 350M sized table: sampling from the model between training steps; latency
        _embed("embed token 350M", "forward", 1, 50257, 1024, 1.0, "bf16"),
        # a full micro-batch of GPT-Neo 6.7B width, rows scaled by the root of the width
        _embed("embed forward 6.7B", "forward", 16384, 50257, 4096, 64.0, "bf16"),
        # an odd width into a float32 residual stream, some positions without a token
        _embed("embed forward odd", "forward", 3001, 50257, 1601, 1.0, "f32", none=0.03),
        # the gradient of a handful of tokens, GPT-Neo 2.7B: nearly all of the table's rows are zeros
        _embed("embed grad 24 tokens 2.7B", "grad", 24, 50257, 2560, 1.0, "bf16"),
        # an odd width and float32 gradients, ragged batch with padding
        _embed("embed grad odd", "grad", 3001, 50257, 1601, 1.0, "f32", pad=0.2, none=0.03),
        # the gradient of a full micro-batch, GPT-Neo 6.7B
        _embed("embed grad 6.7B", "grad", 16384, 50257, 4096, 64.0, "bf16"),
        # a large batch of short padded texts, GPT-2 350M: half of all tokens are the padding token
        _embed("embed grad padded 350M", "grad", 262144, 50257, 1024, 1.0, "bf16", pad=0.5),
        # one flat tensor of a million gradients; latency
        _ragged("norm flat 1M", "norm", 1, 1 << 20, 1 << 20, "bf16", "bf16", 1.0),
        # the norms' and biases' gradients of GPT-2 350M, clipped (training them alone); latency
        _model("clip vectors 350M", "clip", 24, 1024, 4096, 1024, only="vectors"),
        # float32 gradients summed over micro-batches, of odd sizes, clipped to the bf16 that the optimizer takes
        _ragged("clip odd float32", "clip", 37, 1001, 9000001, "f32", "bf16", 0.5),
        # all gradients of GPT-2 XL 1.5B, clipped
        _model("clip 1.5B", "clip", 48, 1600, 6400, 1024),
        # the norm of all gradients of GPT-Neo 6.7B: the largest read
        _model("norm 6.7B", "norm", 32, 4096, 16384, 2048),
    ]


def _between(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Three of four sizes are multiples of 8, as model widths are; the others come as they fall."""
    n = _between(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["forward", "grad", "model", "ragged"])
    if op in ("forward", "grad"):
        V, D = _size(rng, 500, 160000), _size(rng, 64, 8192)
        V = min(V, 50257 * 4096 // D)
        T = min(_between(rng, 1, 262144), 262144 * 1024 // D)
        c = _embed("", op, T, V, D, rng.choice([1.0, 1.0, 64.0, 0.7]), rng.choice(["bf16", "bf16", "f32"]),
                   rng.choice([0.0, 0.0, 0.2, 0.5]), rng.choice([0.0, 0.0, 0.03]))
    elif op == "model":
        d = _size(rng, 256, 4096)
        c = _model("", rng.choice(["norm", "clip"]), rng.randint(2, 48), d, 4 * d, rng.choice([1024, 2048]),
                   _size(rng, 500, 50257), rng.choice(["all", "all", "vectors"]))
        c["L"] = max(1, min(c["L"], 1600000000 // (12 * d * d) - 50257 // (12 * d)))
    else:
        hi = _between(rng, 1000, 30000000)
        c = _ragged("", rng.choice(["norm", "clip"]), _between(rng, 1, 300), _between(rng, 1, min(hi, 5000)), hi,
                    rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.choice([0.5, 1.0, 1e9]))
    del c["name"]
    return c


def _sizes(c):
    """The tensors' numbers of elements."""
    if "count" in c:
        n = max(1, c["count"] - 1)
        return [int(round(c["lo"] * (c["hi"] / c["lo"]) ** (i / n))) for i in range(c["count"])]
    d, ffn = c["d"], c["ffn"]
    vectors = [d, d, 3 * d, d, d, d, ffn, d]
    block = vectors if c["only"] == "vectors" else [d, d, 3 * d * d, 3 * d, d * d, d, d, d, d * ffn, ffn, ffn * d, d]
    return ([] if c["only"] == "vectors" else [c["V"] * d, c["ctx"] * d]) + block * c["L"] + [d, d]


def _shares(V):
    """The probability of the i-th most frequent token: 1 / (i + 1), as words fall off."""
    return np.log1p(1.0 / np.arange(1, V + 1)) / math.log(V + 1)


def work(case):
    if case["op"] == "embed":
        T, V, D, e = case["T"], case["V"], case["D"], 4 if case["dt"] == "f32" else 2
        free = (1.0 - case["none"]) * (1.0 - case["pad"])                # tokens of the text itself
        if case["mode"] == "forward":
            rows = float(-np.expm1(T * np.log1p(-free * _shares(V))).sum())  # distinct rows, expected
            return {"bytes": rows * D * 2 + T * D * e + T * 8, "flops": T * D}
        return {"bytes": (1.0 - case["none"]) * T * D * e + V * D * 2 + T * 8, "flops": T * D}
    n, e, o = sum(_sizes(case)), 4 if case["dt"] == "f32" else 2, 4 if case["out"] == "f32" else 2
    if case["mode"] == "norm":
        return {"bytes": n * e + 4, "flops": 2 * n}
    return {"bytes": n * (e + o) + 4, "flops": 3 * n}


# ------------------------------------------------------------------ the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)

    def normal(shape, std, dtype):
        out = torch.empty(shape, device=dev, dtype=dtype)
        flat, step = out.view(-1), 1 << 26
        for i in range(0, flat.numel(), step):
            n = min(step, flat.numel() - i)
            flat[i:i + n] = torch.randn(n, generator=gen, device=dev) * std
        return out

    s = dict(case)
    if case["op"] == "embed":
        T, V, D, dt = case["T"], case["V"], case["D"], DT[case["dt"]]
        u = torch.rand(T, generator=gen, device=dev, dtype=torch.float64)
        rank = (torch.exp(u * math.log(V + 1)) - 1.0).long().clamp_(0, V - 1)
        ids = torch.randperm(V, generator=gen, device=dev)[rank]         # frequent tokens lie anywhere in the table
        ids[torch.rand(T, generator=gen, device=dev) < case["pad"]] = V // 2
        ids[torch.rand(T, generator=gen, device=dev) < case["none"]] = -1
        s["ids"] = ids
        if case["mode"] == "forward":
            s.update(table=normal((V, D), 0.02, BF), out=torch.empty(T, D, device=dev, dtype=dt))
        else:
            s.update(dout=normal((T, D), 1e-3, dt), dtable=torch.empty(V, D, device=dev, dtype=BF))
        return s
    sizes = _sizes(case)
    scale = torch.exp(torch.randn(len(sizes), generator=gen, device=dev)).tolist()      # layers' gradients differ in size
    grads = [normal((n,), 1e-3 * k, DT[case["dt"]]) for n, k in zip(sizes, scale)]
    for g in grads[:2]:
        g[:: 997] *= 100                                                 # outliers
    s.update(grads=grads, norm=torch.empty(1, device=dev))
    if case["mode"] == "clip":                                           # one buffer holds all clipped gradients
        ends = np.cumsum([-(-n // SLOT) * SLOT for n in sizes]).tolist()
        s["flat"] = torch.zeros(ends[-1], device=dev, dtype=DT[case["out"]])
        s["clipped"] = [s["flat"][e - -(-n // SLOT) * SLOT:][:n] for n, e in zip(sizes, ends)]
    return s


# ---------------------------------------------------------------- one pass each

def run(s):
    if own:
        return (_own_embed if s["op"] == "embed" else _own_grads)(s)
    return (_plain_embed if s["op"] == "embed" else _plain_grads)(s)


def _own_embed(s):
    import bit_blockwise_adamw_gb300 as q8
    if s["mode"] == "forward":
        q8.q8_embedding_forward(s["ids"], s["table"], s["out"], scale=s["scale"])
        return {"out": s["out"]}
    q8.q8_embedding_backward(s["ids"], s["dout"], s["dtable"], scale=s["scale"])
    return {"dtable": s["dtable"]}


def _own_grads(s):
    import bit_blockwise_adamw_gb300 as q8
    if s["mode"] == "norm":
        q8.q8_grad_norm(s["grads"], s["norm"])
        return {"norm": s["norm"]}
    q8.q8_clip_grads(s["grads"], s["max"], s["norm"], out=s["clipped"])
    return {"norm": s["norm"], "clipped": s["flat"]}


def _plain_embed(s):
    ids, V = s["ids"], s["V"]
    known = (ids >= 0) & (ids < V)
    if s["mode"] == "forward":
        rows = s["table"][ids.clamp(0, V - 1)].float() * s["scale"]
        return {"out": torch.where(known[:, None], rows, 0.0).to(DT[s["dt"]])}
    total = torch.zeros(V, s["D"], device=ids.device)
    rows = torch.where(known[:, None], s["dout"].float(), 0.0)
    total.index_add_(0, ids.clamp(0, V - 1), rows)
    return {"dtable": (total * s["scale"]).bfloat16()}


def _plain_norm(grads):
    squares = torch.stack([(g.float() * g.float()).sum(dtype=torch.float64) for g in grads])
    return squares.sum().sqrt().float().view(1)


def _plain_grads(s):
    n = _plain_norm(s["grads"])
    if s["mode"] == "norm":
        return {"norm": n}
    c = (s["max"] / (n + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * c) for g, o in zip(s["grads"], s["clipped"])]
    return {"norm": n, "clipped": s["flat"]}


# ------------------------------------------------------------ float64 definitions

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "embed":
        return _exact_lookup(s) if s["mode"] == "forward" else _exact_gradient(s)
    n = math.sqrt(sum(float(torch.linalg.vector_norm(p.double())) ** 2 for g in s["grads"] for p in g.split(1 << 27)))
    out = {"norm": torch.full((1,), n, dtype=torch.float64, device="cuda")}
    if s["mode"] == "clip":
        c = min(1.0, s["max"] / (n + 1e-6))
        out["clipped"] = torch.cat([torch.nn.functional.pad(g.double() * c, (0, -g.numel() % SLOT)) for g in s["grads"]])
    return out


def _exact_lookup(s):
    """A row of zeros stands behind the table for the positions without a token."""
    table = torch.nn.functional.pad(s["table"].double(), (0, 0, 0, 1))
    return {"out": s["scale"] * table[torch.where(s["ids"] < 0, s["V"], s["ids"])]}


def _exact_gradient(s):
    """Sorted tokens, running sums down the columns, and their differences at each token's last place; in exact
    whole numbers, so that the differences lose nothing: 2^-44 of a gradient of order 1e-3 is 2^-34 of it."""
    ids, V, D = s["ids"], s["V"], s["D"]
    order = torch.argsort(ids, stable=True)
    keys = ids[order].contiguous()
    ends = torch.searchsorted(keys, torch.arange(-1, V, device=ids.device), right=True)
    out = torch.empty(V, D, dtype=torch.float64, device=ids.device)
    step = max(1, (1 << 28) // max(V, len(ids)))
    for j in range(0, D, step):
        part = (s["dout"][:, j:j + step].double() * 2.0 ** 44).round().long()[order]
        run_ = torch.nn.functional.pad(torch.cumsum(part, 0), (0, 0, 1, 0))[ends]
        out[:, j:j + step] = (run_[1:] - run_[:-1]).double() * 2.0 ** -44 * s["scale"]
    return {"dtable": out}
