"""What is measured of the linear, grouped and SwiGLU operators: inputs, the
plain forms they are compared with, and the bytes and operations they need.

    linear           z = x W^T + b, y = act(z) + r, and its gradients
    grouped_linear   y[i] = x[i] W[e]^T for the rows i of each expert e (rows
                     sorted by expert, offsets as moe_route writes them), and
                     its gradients
    swiglu           h = silu(g) u on rows [g | u], and its gradient

The plain forms compute in fp32 and round once at the end; exact() computes
the same from the definitions in fp64.
"""
import math
import random

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _linear(name, T, K, N, act="none", bias=False, residual=False, save=False):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "act": act, "bias": bias, "residual": residual,
            "save": save}


def listed():
    return [
        # the smallest call: 64 tokens at the widths of the tiny layer, where launch latency is all
        _linear("linear_tiny", 64, 256, 512, "relu", bias=True),
        # one token of a sequence being generated: a square projection at the layer's width, added to the stream
        _linear("linear_token", 1, 5120, 5120, residual=True),
        # a decode batch through an up projection as wide as the dense layer's
        _linear("linear_decode_batch", 16, 5120, 16384, "gelu", bias=True),
        # a whole prompt through the dense layer's down projection, added to the stream
        _linear("linear_prompt", 8192, 16384, 5120, residual=True),
        # a training forward on a ragged batch with widths that are no multiple of 64; z is kept for the backward pass
        _linear("linear_ragged_saved", 1217, 1416, 5640, "gelu", bias=True, save=True),
        # the backward pass of a projection on an odd number of tokens
        {"name": "linear_backward", "op": "linear_backward", "T": 4099, "K": 5120, "N": 5120, "act": "gelu", "bias": True},
        # decode: 16 tokens over 16 experts, most of them with a token or two (bound by the touched weights)
        {"name": "grouped_decode", "op": "grouped", "n": 16, "E": 16, "K": 5120, "N": 8192, "skew": 0.0},
        # a prompt over 16 experts, evenly routed
        {"name": "grouped_prompt", "op": "grouped", "n": 8192, "E": 16, "K": 5120, "N": 8192, "skew": 0.0},
        # eight experts of 128 for each of 4096 tokens: about 256 rows an expert, all of the weights read
        {"name": "grouped_many_experts", "op": "grouped", "n": 32768, "E": 128, "K": 5120, "N": 8192, "skew": 0.0},
        # fine-tuning under a skewed router: half of the rows on one expert, a few rows on the last
        {"name": "grouped_backward_skewed", "op": "grouped_backward", "n": 8191, "E": 16, "K": 5120, "N": 8192, "skew": 1.5},
        # a decode batch between an expert's two products
        {"name": "swiglu_decode", "op": "swiglu", "n": 16, "F": 8192},
        # the gradient of a prompt's hidden rows
        {"name": "swiglu_backward", "op": "swiglu_backward", "n": 8191, "F": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(8, 8 * int(round(_log(rng, lo, hi) / 8)))


def draw(rng: random.Random):
    op = rng.choice(["linear", "linear", "linear_backward", "grouped", "grouped", "grouped_backward", "swiglu",
                     "swiglu_backward"])
    while True:
        K, N = _width(rng, 64, 16384), _width(rng, 64, 16384)
        if op == "linear":
            act = rng.choice(ACTS)
            case = _linear("", _log(rng, 1, 16384), K, N, act, rng.random() < 0.5, rng.random() < 0.5,
                           act != "none" and rng.random() < 0.5)
            del case["name"]
        elif op == "linear_backward":
            case = {"op": op, "T": _log(rng, 1, 16384), "K": K, "N": N, "act": rng.choice(ACTS), "bias": rng.random() < 0.5}
        elif op in ("grouped", "grouped_backward"):
            case = {"op": op, "n": _log(rng, 1, 32768), "E": _log(rng, 2, 128), "K": K, "N": N,
                    "skew": rng.choice([0.0, 0.5, 1.5])}
        else:
            case = {"op": op, "n": _log(rng, 1, 32768), "F": _width(rng, 64, 16384)}
        w = work(case)
        if w["flops"] <= 2.5e12 and w["bytes"] <= 6e9:
            return case


def _counts(case):
    """Rows of each expert: drawn with Zipf-like weights (e + 1)^-skew from the sizes alone; a
    run's seed only decides which expert gets which count."""
    n, E = case["n"], case["E"]
    g = torch.Generator().manual_seed(n * 1009 + E)
    p = torch.arange(1, E + 1, dtype=torch.float64) ** -case["skew"]
    ids = torch.multinomial(p, n, replacement=True, generator=g)
    return torch.bincount(ids, minlength=E)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)

    op = case["op"]
    st = {"case": case}
    if op in ("linear", "linear_backward"):
        T, K, N = case["T"], case["K"], case["N"]
        st["x"], st["w"] = normal(T, K), normal(N, K, std=0.02)
        if op == "linear":
            st["b"] = normal(N, std=0.1) if case["bias"] else None
            st["r"] = normal(T, N) if case["residual"] else None
        else:
            st["dy"] = normal(T, N)
            # the pre-activations the forward pass kept, with the spread that x W^T has
            st["z"] = normal(T, N, std=0.02 * math.sqrt(K)) if case["act"] != "none" else None
    elif op in ("grouped", "grouped_backward"):
        n, E, K, N = case["n"], case["E"], case["K"], case["N"]
        counts = _counts(case)[torch.randperm(E, generator=torch.Generator().manual_seed(seed))]
        ends = torch.cumsum(counts, 0)
        st["sizes"] = counts.tolist()
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).cuda()
        st["x"], st["w"] = normal(n, K), normal(E, N, K, std=0.02)
        if op == "grouped_backward":
            st["dy"] = normal(n, N)
    else:
        st["gu"] = normal(case["n"], 2 * case["F"], std=1.4)
        if op == "swiglu_backward":
            st["dh"] = normal(case["n"], case["F"])
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_linear(st):
    c = st["case"]
    z = st["x"].float() @ st["w"].float().t()
    if st["b"] is not None:
        z = z + st["b"].float()
    y = _act(z, c["act"])
    if st["r"] is not None:
        y = y + st["r"].float()
    y = y.bfloat16()
    return (y, z.bfloat16()) if c["save"] else y


def _plain_linear_backward(st):
    c = st["case"]
    dz = st["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(st["z"].float(), c["act"])
    dx = (dz @ st["w"].float()).bfloat16()
    dw = (dz.t() @ st["x"].float()).bfloat16()
    return (dx, dw, dz.sum(0).bfloat16()) if c["bias"] else (dx, dw)


def _plain_grouped(st):
    x, w = st["x"], st["w"]
    y = torch.empty(x.shape[0], w.shape[1], dtype=torch.bfloat16, device=x.device)
    first = 0
    for e, rows in enumerate(st["sizes"]):
        if rows:
            y[first:first + rows] = x[first:first + rows].float() @ w[e].float().t()
        first += rows
    return y


def _plain_grouped_backward(st):
    x, w, dy = st["x"], st["w"], st["dy"]
    dx, dw = torch.empty_like(x), torch.zeros_like(w)
    first = 0
    for e, rows in enumerate(st["sizes"]):
        if rows:
            d = dy[first:first + rows].float()
            dx[first:first + rows] = d @ w[e].float()
            dw[e] = d.t() @ x[first:first + rows].float()
        first += rows
    return dx, dw


def _plain_swiglu(st):
    g, u = st["gu"].float().chunk(2, dim=1)
    return (_act(g, "silu") * u).bfloat16()


def _plain_swiglu_backward(st):
    g, u = st["gu"].float().chunk(2, dim=1)
    dh = st["dh"].float()
    return torch.cat([dh * u * _act_grad(g, "silu"), dh * _act(g, "silu")], dim=1).bfloat16()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(st):
    import int4_quantized_expert_b200 as moe
    c = st["case"]
    act = ACTS.index(c["act"]) if "act" in c else moe.ACT_NONE
    if c["op"] == "linear":
        return moe.linear(st["x"], st["w"], st["b"], activation=act, residual=st["r"], save_preact=c["save"])
    if c["op"] == "linear_backward":
        dx, dw, db = moe.linear_backward(st["dy"], st["x"], st["w"], activation=act, preact=st["z"],
                                         need_dbias=c["bias"])
        return (dx, dw, db) if c["bias"] else (dx, dw)
    if c["op"] == "grouped":
        return moe.grouped_linear(st["x"], st["w"], st["offsets"])
    if c["op"] == "grouped_backward":
        return moe.grouped_linear_backward(st["dy"], st["x"], st["w"], st["offsets"])
    if c["op"] == "swiglu":
        return moe.swiglu(st["gu"])
    return moe.swiglu_backward(st["dh"], st["gu"])


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "grouped": _plain_grouped,
            "grouped_backward": _plain_grouped_backward, "swiglu": _plain_swiglu,
            "swiglu_backward": _plain_swiglu_backward}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without (bf16 tensors: 2 bytes a value)
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        values = T * K + N * K + T * N * (1 + case["residual"] + case["save"]) + N * case["bias"]
        return {"bytes": 2 * values, "flops": 2 * T * K * N}
    if op == "linear_backward":
        T, K, N = case["T"], case["K"], case["N"]
        values = 2 * (T * K + N * K) + T * N * (1 + (case["act"] != "none")) + N * case["bias"]
        return {"bytes": 2 * values, "flops": 4 * T * K * N}
    if op in ("grouped", "grouped_backward"):
        n, E, K, N = case["n"], case["E"], case["K"], case["N"]
        touched = int((_counts(case) > 0).sum())
        if op == "grouped":
            return {"bytes": 2 * (n * K + touched * N * K + n * N), "flops": 2 * n * K * N}
        # dw is written for every expert
        return {"bytes": 2 * (2 * n * K + n * N + (touched + E) * N * K), "flops": 4 * n * K * N}
    n, F = case["n"], case["F"]
    if op == "swiglu":
        return {"bytes": 2 * 3 * n * F, "flops": 6 * n * F}
    return {"bytes": 2 * 5 * n * F, "flops": 12 * n * F}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _sigma64(t):
    return torch.special.expit(t)


def _phi64(t):   # the normal distribution function
    return torch.special.ndtr(t)


def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() for k, v in st.items() if torch.is_tensor(v) and k not in ("w", "offsets")}
    op = case["op"]
    if op in ("linear", "linear_backward"):
        w = st["w"].double()
    if op == "linear":
        z = torch.einsum("tk,nk->tn", d["x"], w)
        if case["bias"]:
            z += d["b"]
        y = {"none": lambda: z.clone(), "relu": lambda: z.clamp(min=0), "silu": lambda: z * _sigma64(z),
             "gelu": lambda: z * _phi64(z)}[case["act"]]()
        if case["residual"]:
            y += d["r"]
        return (y, z) if case["save"] else y
    if op == "linear_backward":
        dz = d["dy"]
        if case["act"] == "relu":
            dz = torch.where(d["z"] > 0, dz, 0.0)
        elif case["act"] == "silu":
            s = _sigma64(d["z"])
            dz = dz * (s + d["z"] * s * _sigma64(-d["z"]))
        elif case["act"] == "gelu":
            dz = dz * (_phi64(d["z"]) + d["z"] * torch.exp(-d["z"].square() / 2) / math.sqrt(2 * math.pi))
        dx, dw = torch.einsum("tn,nk->tk", dz, w), torch.einsum("tn,tk->nk", dz, d["x"])
        return (dx, dw, torch.einsum("tn->n", dz)) if case["bias"] else (dx, dw)
    if op in ("grouped", "grouped_backward"):
        lo = st["offsets"].tolist()
        spans = [(e, slice(lo[e], lo[e + 1])) for e in range(case["E"])]
        if op == "grouped":
            return torch.cat([torch.einsum("rk,nk->rn", d["x"][s], st["w"][e].double()) for e, s in spans])
        return (torch.cat([torch.einsum("rn,nk->rk", d["dy"][s], st["w"][e].double()) for e, s in spans]),
                torch.stack([torch.einsum("rn,rk->nk", d["dy"][s], d["x"][s]) for _, s in spans]))
    g, u = d["gu"][:, :case["F"]], d["gu"][:, case["F"]:]
    s = _sigma64(g)
    if op == "swiglu":
        return g * s * u
    return torch.cat([d["dh"] * u * (s + g * s * _sigma64(-g)), d["dh"] * g * s], dim=1)
