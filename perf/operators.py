"""The matrix products and the SwiGLU around the MoE layer's experts: cases, plain forms and definitions.

Six operators, forward and backward of three:

  linear            out = act(x W + bias) + residual                 x [R, K], W [K, N]
  grouped_linear    the same with W[g], bias[g] for the rows [offsets[g], offsets[g + 1])
  swiglu            out = scale * silu(min(gate, L)) * clip(up, -L, L)   (L = 0: no clamp)

`run` computes them with elementary torch operations in fp32, rounded once at
the end; with `own` true it calls the library's entry points instead.
"""
import math
import random

import torch

own = False

HIDDEN, EXPERTS, INTERMEDIATE, DENSE = 4096, 288, 1280, 11264  # the layer's configuration
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one new token through a square projection, its residual added on the way out
        dict(name="linear_token", op="linear", rows=1, k=HIDDEN, n=HIDDEN, act="none", bias=False,
             residual=True, dtype="bf16"),
        # a prompt's tokens into the dense layers' intermediate size
        dict(name="linear_prompt", op="linear", rows=4096, k=HIDDEN, n=DENSE, act="gelu",
             bias=True, residual=False, dtype="bf16"),
        # a small ragged training batch: no size is a multiple of anything
        dict(name="linear_backward_odd", op="linear_backward", rows=77, k=1100, n=777,
             act="gelu_tanh", bias=True, dtype="f16"),
        # a training batch through the shared expert's first product
        dict(name="linear_backward_batch", op="linear_backward", rows=4096, k=HIDDEN,
             n=INTERMEDIATE, act="silu", bias=True, dtype="bf16"),
        # 64 decoded tokens, 8 experts each: 512 rows, most experts with a few or none
        dict(name="grouped_decode", op="grouped", rows=512, groups=EXPERTS, used=130, skew=0.5,
             k=HIDDEN, n=INTERMEDIATE, act="none", bias=False, dtype="bf16"),
        # a prompt's pairs on one of eight expert-parallel ranks, down projection
        dict(name="grouped_prompt", op="grouped", rows=32768, groups=EXPERTS // 8, used=36,
             skew=0.4, k=INTERMEDIATE, n=HIDDEN, act="none", bias=True, dtype="bf16"),
        # a small training batch with odd sizes and empty groups
        dict(name="grouped_backward_odd", op="grouped_backward", rows=1003, groups=16, used=11,
             skew=0.7, k=250, n=514, act="silu", bias=True, dtype="f16"),
        # a training batch's pairs on one rank, first projection
        dict(name="grouped_backward_batch", op="grouped_backward", rows=16384,
             groups=EXPERTS // 8, used=34, skew=0.4, k=HIDDEN, n=INTERMEDIATE, act="none",
             bias=False, dtype="bf16"),
        # one decoded token's eight pairs
        dict(name="swiglu_token", op="swiglu", rows=8, n=INTERMEDIATE, limit=0.0, scale=True,
             dtype="bf16"),
        # a prompt's pairs with the clamp
        dict(name="swiglu_prompt", op="swiglu", rows=32768, n=INTERMEDIATE, limit=7.0,
             scale=True, dtype="bf16"),
        # an odd width, no gate weight (a shared expert)
        dict(name="swiglu_backward_odd", op="swiglu_backward", rows=1003, n=777, limit=0.0,
             scale=False, dtype="f16"),
        # a training batch's pairs with gate weights and the clamp
        dict(name="swiglu_backward_batch", op="swiglu_backward", rows=32768, n=INTERMEDIATE,
             limit=7.0, scale=True, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """An integer, uniform over the logarithm; half of the large ones a multiple of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.5:
        v = v // 8 * 8
    return max(lo, min(hi, v))


def draw(rng: random.Random):
    op = rng.choice(["linear", "linear_backward", "grouped", "grouped_backward", "swiglu",
                     "swiglu_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op.startswith("swiglu"):
        return dict(op=op, rows=_spread(rng, 1, 32768), n=_spread(rng, 16, INTERMEDIATE),
                    limit=rng.choice([0.0, 7.0]), scale=rng.random() < 0.6, dtype=dtype)
    case = dict(op=op, k=_spread(rng, 16, HIDDEN), n=_spread(rng, 16, HIDDEN),
                act=rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
                bias=rng.random() < 0.5, dtype=dtype)
    if op.startswith("linear"):
        case["rows"] = _spread(rng, 1, 4096)
    else:
        # as many weights as the listed cases have, at most
        weights = (EXPERTS if op == "grouped" else EXPERTS // 8) * HIDDEN * INTERMEDIATE
        case["groups"] = _spread(rng, 1, min(EXPERTS, weights // (case["k"] * case["n"])))
        case["used"] = rng.randint(max(1, case["groups"] // 3), case["groups"])
        case["skew"] = rng.choice([0.0, 0.3, 0.6])
        # the plain form pads every group to the largest
        most = max(64, min(32768, int(4e11 / (2 * case["k"] * case["n"])) // 4))
        case["rows"] = _spread(rng, 1, most)
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return case


def _sizes(case):
    """Rows per group, largest first: a skewed split of `rows` over `used` groups, zeros after."""
    share = [(i + 1) ** -case["skew"] for i in range(case["used"])]
    total, cum, edges = sum(share), 0.0, [0]
    for s in share:
        cum += s
        edges.append(int(round(case["rows"] * cum / total)))
    edges[-1] = case["rows"]
    return [b - a for a, b in zip(edges, edges[1:])] + [0] * (case["groups"] - case["used"])


# ----------------------------------------------------------------- inputs
def _normal(gen, dtype, std, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _weights(gen, dtype, groups, k, n):
    w = torch.empty(groups, k, n, dtype=dtype, device="cuda")
    w.normal_(0.0, k ** -0.5, generator=gen)
    return w


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt, op, rows = _TYPES[case["dtype"]], case["op"], case["rows"]
    s = dict(case=case, binding=None)
    if own:
        from sparse_moe_layer_gemm_b200 import binding
        s["binding"] = binding
    if op.startswith("swiglu"):
        n = case["n"]
        # gate and up are the halves of one product's rows
        both = _normal(gen, dt, 2.0, rows, 2 * n)
        s["gate"], s["up"] = both[:, :n], both[:, n:]
        s["scale"] = torch.rand(rows, generator=gen, device="cuda") if case["scale"] else None
        if op == "swiglu_backward":
            s["dout"] = _normal(gen, dt, 1.0, rows, n)
        return s
    k, n = case["k"], case["n"]
    s["x"] = _normal(gen, dt, 1.0, rows, k)
    if op.startswith("grouped"):
        sizes = _sizes(case)
        random.Random(seed).shuffle(sizes)
        size = torch.tensor(sizes, device="cuda")
        s["offsets"] = torch.zeros(len(sizes) + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = torch.cumsum(size, 0)
        s["most"] = max(sizes)  # the plain form's padded length
        s["w"] = _weights(gen, dt, case["groups"], k, n)
        s["bias"] = _normal(gen, dt, 0.5, case["groups"], n) if case["bias"] else None
        group = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), size)
    else:
        s["w"] = _weights(gen, dt, 1, k, n)[0]
        s["bias"] = _normal(gen, dt, 0.5, n) if case["bias"] else None
        s["residual"] = _normal(gen, dt, 1.0, rows, n) if case.get("residual") else None
        group = None
    if op.endswith("backward"):
        s["dout"] = _normal(gen, dt, 1.0, rows, n)
        s["preact"] = None
        if case["act"] != "none":
            # what the forward pass kept: about x W + bias, which is N(0, 1) here
            z = _normal(gen, torch.float32, 1.0, rows, n)
            if s["bias"] is not None:
                z += s["bias"].float() if group is None else s["bias"].float()[group]
            s["preact"] = z.to(dt)
    return s


# ----------------------------------------------------------------- plain forms
def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _padded(s):
    """Rows of each group as [G, most], clamped to the last row, with the places that exist."""
    start, end = s["offsets"][:-1].long(), s["offsets"][1:].long()
    place = start[:, None] + torch.arange(s["most"], device="cuda")
    there = place < end[:, None]
    return place.clamp(max=s["case"]["rows"] - 1), there[:, :, None]


def _slots(s):
    """Each row's place in the padded [G * most] layout."""
    row = torch.arange(s["case"]["rows"], device="cuda")
    group = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    return group * s["most"] + row - s["offsets"].long()[group]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op.startswith("swiglu"):
        dt, L = s["gate"].dtype, c["limit"]
        gate, up = s["gate"].float(), s["up"].float()
        a = gate.clamp(max=L) if L > 0 else gate
        u = up.clamp(-L, L) if L > 0 else up
        p = torch.sigmoid(a)
        silu = a * p
        scale = 1.0 if s["scale"] is None else s["scale"][:, None]
        if op == "swiglu":
            return (scale * silu * u).to(dt)
        d = s["dout"].float()
        dgate, dup = d * scale * u * p * (1 + a * (1 - p)), d * scale * silu
        if L > 0:
            dgate = dgate * (gate <= L)
            dup = dup * ((up >= -L) & (up <= L))
        dscale = None if s["scale"] is None else (d * silu * u).sum(1)
        return dgate.to(dt), dup.to(dt), dscale
    dt, act = s["x"].dtype, c["act"]
    x, w = s["x"].float(), s["w"].float()
    if op == "linear":
        z = x @ w
        if s["bias"] is not None:
            z = z + s["bias"].float()
        z = _act(z, act)
        if s["residual"] is not None:
            z = z + s["residual"].float()
        return z.to(dt)
    if op == "linear_backward":
        dz = s["dout"].float()
        if act != "none":
            dz = dz * _act_slope(s["preact"].float(), act)
        return ((dz @ w.t()).to(dt), (x.t() @ dz).to(dt),
                dz.sum(0).to(dt) if c["bias"] else None)
    place, there = _padded(s)
    slot = _slots(s)
    xg = x[place] * there
    if op == "grouped":
        z = torch.bmm(xg, w)
        if s["bias"] is not None:
            z = z + s["bias"].float()[:, None]
        return _act(z, act).reshape(-1, c["n"])[slot].to(dt)
    dz = s["dout"].float()
    if act != "none":
        dz = dz * _act_slope(s["preact"].float(), act)
    dz = dz[place] * there
    dx = torch.bmm(dz, w.transpose(1, 2)).reshape(-1, c["k"])[slot]
    return (dx.to(dt), torch.bmm(xg.transpose(1, 2), dz).to(dt),
            dz.sum(1).to(dt) if c["bias"] else None)


def _library(s):
    c, B = s["case"], s["binding"]
    op = c["op"]
    if op == "linear":
        return B.linear(s["x"], s["w"], s["bias"], residual=s["residual"], activation=c["act"])
    if op == "linear_backward":
        return B.linear_backward(s["dout"], s["x"], s["w"], preact=s["preact"],
                                 activation=c["act"], need_db=c["bias"])
    if op == "grouped":
        return B.grouped_linear(s["x"], s["offsets"], s["w"], s["bias"], activation=c["act"])
    if op == "grouped_backward":
        return B.grouped_linear_backward(s["dout"], s["x"], s["offsets"], s["w"],
                                         preact=s["preact"], activation=c["act"],
                                         need_db=c["bias"])
    if op == "swiglu":
        return B.swiglu(s["gate"], s["up"], s["scale"], limit=c["limit"])
    return B.swiglu_backward(s["dout"], s["gate"], s["up"], s["scale"], limit=c["limit"])


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------------- cost
def work(case):
    op, rows, n = case["op"], case["rows"], case["n"]
    if op == "swiglu":
        return {"bytes": 6 * rows * n + (4 * rows if case["scale"] else 0), "flops": 8 * rows * n}
    if op == "swiglu_backward":
        return {"bytes": 10 * rows * n + (8 * rows if case["scale"] else 0),
                "flops": 16 * rows * n}
    k = case["k"]
    # weights are read for the groups that have rows, gradients of weights written for all
    groups = 1 if op.startswith("linear") else case["groups"]
    read = 1 if op.startswith("linear") else sum(v > 0 for v in _sizes(case))
    bias = 1 if case["bias"] else 0
    if not op.endswith("backward"):
        bytes_ = 2 * (rows * k + read * k * n + rows * n + bias * read * n)
        if case.get("residual"):
            bytes_ += 2 * rows * n
        return {"bytes": bytes_, "flops": 2 * rows * k * n}
    bytes_ = 2 * (2 * rows * k + (read + groups) * k * n + rows * n + bias * groups * n)
    if case["act"] != "none":
        bytes_ += 2 * rows * n
    return {"bytes": bytes_, "flops": 4 * rows * k * n}


# ----------------------------------------------------------------- definitions in 64 bits
def _gelu_tanh_parts(z):
    inner = 0.7978845608028654 * (z + 0.044715 * z * z * z)
    inside = 0.7978845608028654 * (1 + 0.134145 * z * z)
    return torch.sigmoid(2 * inner), 2 * inside  # 0.5 (1 + tanh u) = sigmoid(2 u)


def _exact_act(z, name):
    if name == "gelu_tanh":
        return z * _gelu_tanh_parts(z)[0]
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z.clamp(min=0) if name == "relu" else z


def _exact_slope(z, name):
    if name == "gelu_tanh":
        p, dp = _gelu_tanh_parts(z)
        return p + z * p * (1 - p) * dp
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) * 0.3989422804014327
    if name == "silu":
        e = torch.exp(-z)
        return (1 + e + z * e) / (1 + e) ** 2
    return torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device)) \
        if name == "relu" else torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def f64(t):
        return None if t is None else t.to(torch.float64)

    if op.startswith("swiglu"):
        limit = case["limit"] if case["limit"] > 0 else math.inf
        out, dgate, dup, dscale = [], [], [], []
        # in blocks of rows, so that the 64-bit values fit beside the inputs
        for lo in range(0, case["rows"], 4096):
            rows = slice(lo, min(lo + 4096, case["rows"]))
            g, u = f64(s["gate"][rows]), f64(s["up"][rows])
            a, v = torch.clamp(g, max=limit), torch.clamp(u, min=-limit, max=limit)
            scale = f64(s["scale"][rows])[:, None] if case["scale"] else torch.ones_like(g[:, :1])
            act = _exact_act(a, "silu")
            if op == "swiglu":
                out.append(scale * act * v)
                continue
            d = f64(s["dout"][rows])
            dgate.append(torch.where(g <= limit, d * scale * v * _exact_slope(a, "silu"), 0.0))
            dup.append(torch.where(u.abs() <= limit, d * scale * act, 0.0))
            dscale.append(torch.einsum("rn,rn->r", d, act * v))
        if op == "swiglu":
            return torch.cat(out)
        return torch.cat(dgate), torch.cat(dup), torch.cat(dscale) if case["scale"] else None

    grouped = op.startswith("grouped")
    edges = s["offsets"].tolist() if grouped else [0, case["rows"]]
    out, dx, dw, db = [], [], [], []
    for g, (lo, hi) in enumerate(zip(edges, edges[1:])):
        w = f64(s["w"][g] if grouped else s["w"])
        x = f64(s["x"][lo:hi])
        if not op.endswith("backward"):
            z = torch.matmul(x, w)
            if case["bias"]:
                z += f64(s["bias"][g] if grouped else s["bias"])
            z = _exact_act(z, case["act"])
            if case.get("residual"):
                z += f64(s["residual"])
            out.append(z)
            continue
        dz = f64(s["dout"][lo:hi])
        if case["act"] != "none":
            dz = dz * _exact_slope(f64(s["preact"][lo:hi]), case["act"])
        dx.append(torch.einsum("rn,kn->rk", dz, w))
        dw.append(torch.einsum("rk,rn->kn", x, dz))
        db.append(dz.sum(dim=0))
    if not op.endswith("backward"):
        return torch.cat(out)
    return (torch.cat(dx), torch.stack(dw) if grouped else dw[0],
            (torch.stack(db) if grouped else db[0]) if case["bias"] else None)
