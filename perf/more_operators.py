"""Cases of the feed-forward block between two boundaries: layer norm with the residual add and its gradient, the gated
feed-forward's projections with activation and product and their gradient, and products in 8-bit floating point
with a scale for each block of 128.

Every case has a plain form (elementary torch operations in 32 bits) and the framework's calls; `own` says which of
the two `run` takes.  Both take the same state.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one token of one sequence: residual add and layer norm, where latency counts
        _norm_case("layer-norm-token", 1, 4096, "bf16", residual=True),
        # a prefill batch's residual add and layer norm: memory
        _norm_case("layer-norm-prefill", 8192, 8192, "bf16", residual=True),
        # odd rows in 32 bits, the norm alone, without a bias
        _norm_case("layer-norm-f32-odd", 1037, 5120, "f32", residual=False, bias=False),
        # a training step's gradient, the residual stream's own gradient added in
        _norm_case("layer-norm-grad-long", 8192, 5120, "bf16", residual=True, grad=True),
        # the same in 32 bits without one, ragged sizes
        _norm_case("layer-norm-grad-f32-odd", 777, 2064, "f32", residual=False, grad=True),
        # one token through a projection in 8 bits: the weights' bytes count
        _fp8_case("fp8-token", 1, 8192, 8192),
        # odd tokens, features and hidden sizes that end inside a tile and inside a block
        _fp8_case("fp8-odd", 777, 4112, 4144),
        # a prefill batch: the product's rate counts
        _fp8_case("fp8-prefill", 8192, 8192, 8192),
        # one token through both projections, the activation and the product: the weights' bytes count
        _ffn_case("ffn-token", 1, 8192, 8192, "silu"),
        # odd sizes and the other activation
        _ffn_case("ffn-odd", 333, 4112, 2064, "gelu"),
        # a prefill batch's
        _ffn_case("ffn-prefill", 4096, 8192, 8192, "silu"),
        # a training step's gradients of the inputs and both weights
        _ffn_case("ffn-grad", 4096, 8192, 4096, "silu", grad=True),
    ]


def _norm_case(name, rows, hidden, dtype, residual, bias=True, grad=False):
    return {"name": name, "kind": "norm-grad" if grad else "norm", "rows": rows, "hidden": hidden, "dtype": dtype,
            "residual": residual, "bias": bias}


def _fp8_case(name, rows, features, hidden):
    return {"name": name, "kind": "fp8", "rows": rows, "features": features, "hidden": hidden}


def _ffn_case(name, rows, features, hidden, activation, grad=False):
    return {"name": name, "kind": "ffn-grad" if grad else "ffn", "rows": rows, "features": features,
            "hidden": hidden, "activation": activation}


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["norm", "norm-grad", "fp8", "ffn", "ffn-grad"])
    if kind in ("norm", "norm-grad"):
        dtype = rng.choice(["bf16", "f32"])
        c = _norm_case("", _log(rng, 1, 8192 // (2 if dtype == "f32" else 1)), _log(rng, 64, 8192, 16), dtype,
                       rng.random() < 0.7, rng.random() < 0.7, kind == "norm-grad")
    elif kind == "fp8":
        c = _fp8_case("", _log(rng, 1, 8192), _log(rng, 64, 8192, 16), _log(rng, 64, 8192, 16))
    else:
        grad = kind == "ffn-grad"
        c = _ffn_case("", _log(rng, 1, 4096), _log(rng, 64, 8192, 16), _log(rng, 64, 4096 if grad else 8192, 16),
                      rng.choice(["silu", "gelu"]), grad)
    del c["name"]
    return c


def work(case):
    t, h, kind = case["rows"], case["hidden"], case["kind"]
    if kind in ("norm", "norm-grad"):
        size = 2 if case["dtype"] == "bf16" else 4
        if kind == "norm":  # x, r in, h, y out; weight and bias
            tensors = 4 if case["residual"] else 2
            return {"bytes": (tensors * t + 1 + int(case["bias"])) * h * size, "flops": 10 * t * h}
        tensors = 4 if case["residual"] else 3  # h, dy and perhaps dh in, dx out; the weights' gradients in 32 bits
        return {"bytes": (tensors * t + 1) * h * size + 8 * t + (1 + int(case["bias"])) * h * 4, "flops": 16 * t * h}
    n = case["features"]
    if kind == "fp8":
        return {"bytes": 2 * t * h + n * h + 2 * t * n, "flops": 2 * t * n * h}
    if kind == "ffn":
        return {"bytes": 2 * (t * h + 2 * n * h + t * n), "flops": 4 * t * n * h}
    # x, both weights, g, u and the output's gradient in; dx and the weights' gradients out
    return {"bytes": 2 * (2 * t * h + 4 * n * h + 3 * t * n), "flops": 8 * t * n * h}


# ----------------------------------------------------------------- inputs ---
def _normal(gen, *shape, dtype=torch.float32, mean=0.0, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)


def _activations(gen, rows, hidden, dtype, mean=0.0):
    """N(mean, 1) with half a percent of the channels twenty times as large, as the boundary's activations are."""
    x = torch.randn(rows, hidden, generator=gen, device="cuda") + mean
    channel = torch.rand(hidden, generator=gen, device="cuda") < 0.005
    return (x * torch.where(channel, 20.0, 1.0)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, h, kind = case["rows"], case["hidden"], case["kind"]
    s = {"case": case}
    if kind in ("norm", "norm-grad"):
        dtype = _TYPES[case["dtype"]]
        s["weight"] = _normal(gen, h, dtype=dtype, mean=1.0, std=0.1)
        s["bias"] = _normal(gen, h, dtype=dtype, std=0.1) if case["bias"] else None
        if kind == "norm":
            s["x"] = _activations(gen, t, h, dtype, mean=0.25)
            s["residual"] = _normal(gen, t, h, dtype=dtype) if case["residual"] else None
        else:  # the forward pass keeps its input and each row's mean and inverse deviation
            s["h"] = _activations(gen, t, h, dtype, mean=0.25)
            s["stats"] = torch.stack(_moments(s["h"].float()), 1).view(t, 2).contiguous()
            s["dy"] = _normal(gen, t, h, dtype=dtype)
            s["dh"] = _normal(gen, t, h, dtype=dtype) if case["residual"] else None
        return s
    n = case["features"]
    s["x"] = _activations(gen, t, h, torch.bfloat16)
    if kind == "fp8":  # the weight in 8 bits: quantised once
        s["weight"] = _fp8_encode(_normal(gen, n, h, std=1 / math.sqrt(h)), 128)
        return s
    s["w_gate"] = _normal(gen, n, h, dtype=torch.bfloat16, std=1 / math.sqrt(h))
    s["w_up"] = _normal(gen, n, h, dtype=torch.bfloat16, std=1 / math.sqrt(h))
    if kind == "ffn-grad":  # both projections are kept by the forward pass
        s["gate"] = (s["x"].float() @ s["w_gate"].float().T).to(torch.bfloat16)
        s["up"] = (s["x"].float() @ s["w_up"].float().T).to(torch.bfloat16)
        s["dout"] = _normal(gen, t, n, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------ plain forms ---
def _moments(h):
    mean = h.mean(1, keepdim=True)
    return mean, 1 / torch.sqrt(((h - mean) * (h - mean)).mean(1, keepdim=True) + _EPS)


def _norm_plain(s):
    dtype, h = s["x"].dtype, s["x"]
    out = {}
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(dtype)
        out["h"] = h
    h = h.float()  # the norm is that of the residual stream as it is kept
    mean, inv = _moments(h)
    y = (h - mean) * inv * s["weight"].float()
    out["y"] = (y if s["bias"] is None else y + s["bias"].float()).to(dtype)
    return out


def _norm_grad_plain(s):
    dy, mean, inv = s["dy"].float(), s["stats"][:, :1], s["stats"][:, 1:]
    hh = (s["h"].float() - mean) * inv
    a = dy * s["weight"].float()
    dx = inv * (a - a.mean(1, keepdim=True) - hh * (a * hh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    out = {"dx": dx.to(s["h"].dtype), "dweight": (dy * hh).sum(0)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _pad128(x, rows):
    """x with zeros up to whole blocks of `rows` by 128."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 128, 0, -x.shape[0] % rows))


def _blocks(x, rows):
    """[row blocks, rows, column blocks, 128] of x."""
    p = _pad128(x, rows)
    return p.view(p.shape[0] // rows, rows, p.shape[1] // 128, 128)


def _fp8_encode(x, rows):
    """Codes (e4m3, one a byte) of x and the scales of its blocks of `rows` by 128."""
    b = _blocks(x.float(), rows)
    most = torch.full((), 448.0, device=x.device)  # by a number of the host torch would multiply with its inverse
    scale = (b.abs().amax((1, 3)) / most).clamp(min=2.0 ** -60)
    codes = (b / scale[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(-1, codes.shape[2] * 128)[:x.shape[0], :x.shape[1]].contiguous(), scale


def _fp8_values(codes, scale, rows):
    b = _blocks(codes, rows).view(torch.float8_e4m3fn).float() * scale[:, None, :, None]
    return b.view(-1, b.shape[2] * 128)[:codes.shape[0], :codes.shape[1]]


def _fp8_plain(s):
    x = _fp8_values(*_fp8_encode(s["x"], 1), 1)
    return (x @ _fp8_values(*s["weight"], 128).T).to(torch.bfloat16)


def _act(name, g):
    """The activation and its slope."""
    if name == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    c, k = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (g + k * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * k * g * g)


def _ffn_plain(s):
    x = s["x"].float()
    a, _ = _act(s["case"]["activation"], x @ s["w_gate"].float().T)
    return (a * (x @ s["w_up"].float().T)).to(torch.bfloat16)


def _ffn_grad_plain(s):
    x, d = s["x"].float(), s["dout"].float()
    a, slope = _act(s["case"]["activation"], s["gate"].float())
    dg, du = d * s["up"].float() * slope, d * a
    dx = dg @ s["w_gate"].float() + du @ s["w_up"].float()
    return {"dx": dx.to(torch.bfloat16), "dw_gate": (dg.T @ x).to(torch.bfloat16),
            "dw_up": (du.T @ x).to(torch.bfloat16)}


# ------------------------------------------------------- the framework's ---
def _bind(s):
    """The pass's calls with their arguments marshalled once (fcomm.Bound), as a serving or training loop with fixed
    buffers keeps them, and the buffers that they write."""
    from quantized_reduce_rmsnorm_gb300 import fcomm as fc
    c = s["case"]
    kind, t, h = c["kind"], c["rows"], c["hidden"]
    if kind == "norm":
        out = {"y": torch.empty_like(s["x"])}
        if c["residual"]:
            out["h"] = torch.empty_like(s["x"])
        return [fc.bind_layer_norm(s["x"], out["y"], weight=s["weight"], bias=s["bias"], residual_in=s["residual"],
                                   residual_out=out.get("h"), eps=_EPS)], out
    if kind == "norm-grad":
        out = {"dx": torch.empty_like(s["h"]), "dweight": torch.empty(h, dtype=torch.float32, device="cuda")}
        if c["bias"]:
            out["dbias"] = torch.empty(h, dtype=torch.float32, device="cuda")
        return [fc.bind_layer_norm_backward(s["h"], s["stats"], s["dy"], dh=s["dh"], weight=s["weight"],
                                            workspace=fc.alloc_layer_norm_workspace(t, h), **out)], out
    out = torch.empty(t, c["features"], dtype=torch.bfloat16, device="cuda")
    if kind == "fp8":
        q = fc.alloc_fp8(t, h)
        return [fc.bind_fp8_quantize(s["x"], q), fc.bind_fp8_matmul(q, s["weight"], out)], out
    act = {"silu": fc.ACT_SILU, "gelu": fc.ACT_GELU_TANH}[c["activation"]]
    if kind == "ffn":
        return [fc.bind_gated_ffn(s["x"], s["w_gate"], s["w_up"], out, activation=act)], out
    out = {"dx": torch.empty_like(s["x"]), "dw_gate": torch.empty_like(s["w_gate"]),
           "dw_up": torch.empty_like(s["w_up"])}
    return [fc.bind_gated_ffn_backward(s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["dout"], activation=act,
                                       workspace=fc.alloc_gated_ffn_workspace(t, c["features"]), **out)], out


_PLAIN = {"norm": _norm_plain, "norm-grad": _norm_grad_plain, "fp8": _fp8_plain, "ffn": _ffn_plain,
          "ffn-grad": _ffn_grad_plain}


def run(state):
    if not own:
        return _PLAIN[state["case"]["kind"]](state)
    if "calls" not in state:
        state["calls"], state["out"] = _bind(state)
    for call in state["calls"]:
        call()
    return state["out"]


# ------------------------------------------------------------------ exact ---
def exact(case, seed):
    s = prepare(case, seed)
    kind, t, h = case["kind"], case["rows"], case["hidden"]
    if kind == "norm":
        out, kept = {}, s["x"].double()
        if s["residual"] is not None:
            out["h"] = kept + s["residual"].double()
            kept = out["h"].to(s["x"].dtype).double()
        c = kept - kept.sum(1, keepdim=True) / h
        y = c * (c.square().sum(1, keepdim=True) / h + _EPS).rsqrt() * s["weight"].double()
        out["y"] = y if s["bias"] is None else y + s["bias"].double()
        return out
    if kind == "norm-grad":
        # y_i = w_i n_i, n = (h - mean) r: dn_i/dh_j = r (1[i = j] - 1/H - n_i n_j / H)
        r = s["stats"][:, 1:].double()
        nrm = (s["h"].double() - s["stats"][:, :1].double()) * r
        dy = s["dy"].double()
        b = dy * s["weight"].double()
        dx = r * (b - b.sum(1, keepdim=True) / h - nrm * (b * nrm).sum(1, keepdim=True) / h)
        out = {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dweight": torch.einsum("th,th->h", dy, nrm)}
        if s["bias"] is not None:
            out["dbias"] = dy.sum(0)
        return out
    x = s["x"].double()
    if kind == "fp8":
        # scales and quotients are binary32 numbers; the code is the quotient's nearest value, spaced 2^(e - 3) for
        # magnitudes in [2^e, 2^(e + 1)), 2^-9 below 2^-6
        kb = torch.arange(h, device="cuda") // 128
        amax = torch.zeros(t, (h + 127) // 128, dtype=torch.float64, device="cuda")
        amax.scatter_reduce_(1, kb.expand(t, h), x.abs(), "amax")
        sx = (amax / 448).float().clamp(min=2.0 ** -60).double()[:, kb]
        q = (x / sx).float().double()
        step = torch.exp2((torch.frexp(q.abs()).exponent - 1).clamp(min=-6).double() - 3)
        v = (torch.round(q / step) * step).clamp(-448, 448) * sx
        codes, scale = s["weight"]
        c = codes.int()
        e, m = (c >> 3) & 15, (c & 7).double()
        w = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10)) * (1 - 2 * (c >> 7)).double()
        rb = torch.arange(case["features"], device="cuda") // 128
        return v @ (w * scale.double()[rb][:, kb]).T
    wg, wu = s["w_gate"].double(), s["w_up"].double()

    def value(z):
        if case["activation"] == "silu":
            return z * torch.sigmoid(z)
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))

    if kind == "ffn":
        return value(x @ wg.T) * (x @ wu.T)
    g, d = s["gate"].double(), s["dout"].double()
    if case["activation"] == "silu":
        slope = torch.sigmoid(g) + value(g) * torch.sigmoid(-g)
    else:  # z sigmoid(p(z)): sigmoid + z p' sigmoid (1 - sigmoid)
        k = 2 * math.sqrt(2 / math.pi)
        p = k * (g + 0.044715 * g ** 3)
        slope = torch.sigmoid(p) + value(g) * k * (1 + 0.134145 * g.square()) * torch.sigmoid(-p)
    dg, du = d * s["up"].double() * slope, d * value(g)
    return {"dx": torch.cat([dg, du], 1) @ torch.cat([wg, wu]), "dw_gate": dg.T @ x, "dw_up": du.T @ x}
