"""Cases for timing and checking the operators around the AllReduce of a tensor-parallel layer.

Four operators: ``linear`` (matrix product with bias, activation and residual
in its epilogue) and its backward pass, ``layer_norm`` and its backward pass.
Where ``own`` is false, ``run`` computes them from elementary torch operations
in binary32; where it is true, it calls the package's operators.  ``exact``
computes them in binary64 from torch's own definitions (autograd for the
gradients).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


def _linear(name, rows, k, n, dtype, act="none", bias=True, residual=False, preact=False):
    return {"name": name, "op": "linear", "rows": rows, "in": k, "out": n, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "preact": preact}


def _linear_bwd(name, rows, k, n, dtype, act="none"):
    return {"name": name, "op": "linear_bwd", "rows": rows, "in": k, "out": n, "dtype": dtype, "act": act}


def _norm(name, rows, width, dtype, params="same", stats=False):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "params": params,
            "stats": stats}


def _norm_bwd(name, rows, width, dtype, params="same"):
    return {"name": name, "op": "norm_bwd", "rows": rows, "width": width, "dtype": dtype, "params": params}


def listed():
    return [
        # One token through a column-parallel projection of a rank (hidden 8192): latency and the weight's bytes.
        _linear("linear_token", 1, 8192, 4096, "bf16", act="gelu"),
        # The decode step's 32 tokens through a row-parallel projection back to hidden 8192, residual on this rank.
        _linear("linear_decode", 32, 4096, 8192, "bf16", residual=True),
        # The 8192-token prompt through the column-parallel projection, training form (pre-activation kept).
        _linear("linear_prompt", 8192, 8192, 4096, "bf16", act="gelu", preact=True),
        # The same prompt through the row-parallel projection: partial sums with a residual, binary16.
        _linear("linear_prompt_row", 8192, 4096, 8192, "fp16", residual=True),
        # Odd sizes in binary32: rows that start at no 16-byte boundary.
        _linear("linear_ragged", 1001, 2047, 1537, "fp32", act="silu", residual=True),
        # Backward pass of the column-parallel projection over the prompt.
        _linear_bwd("linear_bwd_prompt", 8192, 8192, 4096, "bf16", act="gelu"),
        # Odd sizes in binary16: rows that start at no 16-byte boundary.
        _linear_bwd("linear_bwd_ragged", 515, 1025, 770, "fp16", act="relu"),
        # The decode step's 32 tokens behind an AllReduce: latency.
        _norm("norm_decode", 32, 8192, "bf16"),
        # The 8192-token prompt, statistics kept for the backward pass.
        _norm("norm_prompt", 8192, 8192, "bf16", stats=True),
        # Odd width in binary16, parameters in binary32.
        _norm("norm_ragged", 4099, 5001, "fp16", params="fp32"),
        # Backward pass over the prompt: input gradient and both parameter gradients.
        _norm_bwd("norm_bwd_prompt", 8192, 8192, "bf16"),
        # Few long rows in binary32, odd width.
        _norm_bwd("norm_bwd_ragged", 257, 16387, "fp32"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    # half of the sizes are multiples of 64 where they are large enough, as a model's are
    return n // 64 * 64 if n >= 256 and rng.random() < 0.5 else n


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    op = rng.choice(["linear", "linear", "linear_bwd", "norm", "norm_bwd"])
    if op in ("norm", "norm_bwd"):
        rows, width = _log_int(rng, 1, 8192), _log_int(rng, 16, 20000)
        while rows * width * BYTES[dtype] > 8192 * 8192 * 2:
            rows = max(1, rows // 2)
        params = rng.choice(["same", "fp32"])
        if op == "norm":
            case = _norm("", rows, width, dtype, params, rng.random() < 0.5)
        else:
            case = _norm_bwd("", rows, width, dtype, params)
    else:
        rows = _log_int(rng, 1, 8192)
        k, n = _log_int(rng, 16, 8192), _log_int(rng, 16, 8192)
        most = 8192 * 8192 * 4096 // (8 if dtype == "fp32" else 1)
        while rows * k * n > most:
            rows = max(1, rows // 2)
        act = rng.choice(ACTIVATIONS)
        if op == "linear":
            case = _linear("", rows, k, n, dtype, act, rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.3)
        else:
            case = _linear_bwd("", rows, k, n, dtype, act)
    del case["name"]
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)

    s = {"case": case}
    if case["op"] in ("norm", "norm_bwd"):
        rows, width = case["rows"], case["width"]
        p = torch.float32 if case["params"] == "fp32" else t
        # residual-stream rows: a few times unit size, off zero
        s["x"] = (normal(rows, width, scale=2.0, dtype=torch.float32)
                  + normal(rows, 1, scale=0.5, dtype=torch.float32)).to(t)
        s["w"] = (1.0 + normal(width, scale=0.2, dtype=torch.float32)).to(p)
        s["b"] = normal(width, scale=0.2, dtype=p)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, width)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
        return s
    rows, k, n = case["rows"], case["in"], case["out"]
    s["x"] = normal(rows, k)
    s["w"] = normal(n, k, scale=k ** -0.5)
    if case["op"] == "linear":
        s["b"] = normal(n, scale=0.5) if case["bias"] else None
        s["r"] = normal(rows, n) if case["residual"] else None
    else:
        s["dy"] = normal(rows, n)
        # what the forward pass kept: the pre-activation, in the activations' type
        s["z"] = (s["x"] @ s["w"].t() + normal(n, scale=0.5)) if case["act"] != "none" else None
    return s


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        return q * (1.0 + z * (1.0 - q))
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    t = s["x"].dtype
    x = s["x"].float()
    if case["op"] == "linear":
        z = x @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, case["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(t), "z": z.to(t)} if case["preact"] else {"y": y.to(t)}
    if case["op"] == "linear_bwd":
        dz = s["dy"].float()
        if case["act"] != "none":
            dz = dz * _act_slope(s["z"].float(), case["act"])
        return {"dx": (dz @ s["w"].float()).to(t), "dw": (dz.t() @ x).to(t), "db": dz.sum(0).to(t)}
    w = s["w"].float()
    if case["op"] == "norm":
        mean = x.mean(1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
        y = ((x - mean) * rstd * w + s["b"].float()).to(t)
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]} if case["stats"] else {"y": y}
    dy = s["dy"].float()
    h = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return {"dx": dx.to(t), "dw": (dy * h).sum(0).to(s["w"].dtype), "db": dy.sum(0).to(s["w"].dtype)}


def _framework(s):
    from allreduce_emulated_peer_amd import mscl

    case = s["case"]
    if case["op"] == "linear":
        out = mscl.linear_tensors(s["x"], s["w"], bias=s["b"], residual=s["r"], activation=case["act"],
                                  return_preact=case["preact"])
        return {"y": out[0], "z": out[1]} if case["preact"] else {"y": out}
    if case["op"] == "linear_bwd":
        dx, dw, db = mscl.linear_backward_tensors(s["dy"], s["x"], s["w"], preact=s["z"], activation=case["act"])
        return {"dx": dx, "dw": dw, "db": db}
    if case["op"] == "norm":
        out = mscl.layer_norm_tensors(s["x"], s["w"], s["b"], eps=EPS, return_stats=case["stats"])
        return {"y": out[0], "mean": out[1], "rstd": out[2]} if case["stats"] else {"y": out}
    dx, dw, db = mscl.layer_norm_backward_tensors(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    return {"dx": dx, "dw": dw, "db": db}


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("norm", "norm_bwd"):
        rows, width = case["rows"], case["width"]
        p = 4 if case["params"] == "fp32" else e
        if case["op"] == "norm":
            return {"bytes": 2 * rows * width * e + 2 * width * p + (8 * rows if case["stats"] else 0),
                    "flops": 8 * rows * width}
        return {"bytes": 3 * rows * width * e + 8 * rows + 3 * width * p, "flops": 16 * rows * width}
    m, k, n = case["rows"], case["in"], case["out"]
    if case["op"] == "linear":
        moved = m * k + n * k + (n if case["bias"] else 0)
        moved += m * n * (1 + int(case["residual"]) + int(case["preact"]))
        return {"bytes": moved * e, "flops": 2 * m * n * k}
    moved = m * n * (2 if case["act"] != "none" else 1) + 2 * m * k + 2 * n * k + n
    return {"bytes": moved * e, "flops": 4 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    F = torch.nn.functional
    d = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    acts = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}
    if case["op"] == "linear":
        z = F.linear(d["x"], d["w"], d["b"])
        y = acts[case["act"]](z)
        if d["r"] is not None:
            y = y.add_(d["r"]) if case["act"] != "none" else y + d["r"]
        return {"y": y, "z": z} if case["preact"] else {"y": y}
    if case["op"] == "norm":
        y = F.layer_norm(d["x"], (case["width"],), d["w"], d["b"], EPS)
        if not case["stats"]:
            return {"y": y}
        var, mean = torch.var_mean(d["x"], 1, correction=0)
        return {"y": y, "mean": mean, "rstd": (var + EPS).rsqrt()}
    if case["op"] == "linear_bwd":
        dz = d["dy"]
        if case["act"] != "none":
            z = d["z"].requires_grad_()
            (dz,) = torch.autograd.grad(acts[case["act"]](z), z, d["dy"])
        return {"dx": torch.mm(dz, d["w"]), "dw": torch.mm(dz.t().contiguous(), d["x"]), "db": dz.sum(0)}
    # the kept statistics are inputs: they are rounded values of the ones that x has
    h = torch.mul(d["x"] - d["mean"].unsqueeze(1), d["rstd"].unsqueeze(1))
    width = case["width"]
    g = d["dy"] * d["w"]
    along = torch.linalg.vecdot(g, h) / width
    dx = (g - (g.sum(1) / width).unsqueeze(1) - h * along.unsqueeze(1)) * d["rstd"].unsqueeze(1)
    return {"dx": dx, "dw": torch.einsum("ij,ij->j", d["dy"], h), "db": d["dy"].sum(0)}
