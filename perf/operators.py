"""Cases of the operators around a tensor-parallel layer boundary: the norms before and after a block with its gate
and residual scale, their gradient, microscaled 4-bit quantisation and the product of microscaled tensors.

Every case has a plain form (elementary torch operations in 32 bits) and the framework's calls; `own` says which of
the two `run` takes.  Both take the same state.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one token of one sequence between two blocks: residual add and the next block's norm, where latency counts
        _norm_case("norm-token", 1, 4096, "bf16", post=False, gate_rows=0, pre=True),
        # a decode batch, normed before and after the block, one gate for all tokens
        _norm_case("norm-decode", 64, 8192, "bf16", post=True, gate_rows=1, pre=True, block_scale=0.5),
        # a prefill batch of eight sequences, each with a gate of its own
        _norm_case("norm-prefill", 8192, 8192, "bf16", post=True, gate_rows=8, pre=True, residual_scale=0.75),
        # odd rows in 32 bits, a gate for every token
        _norm_case("norm-f32-odd", 1037, 5120, "f32", post=True, gate_rows=1037, pre=True),
        # a training step's gradient of everything, the gate shared by all tokens
        _norm_case("grad-long", 8192, 5120, "bf16", post=True, gate_rows=1, pre=True, grad=True, block_scale=0.5),
        # the same in 32 bits with seven gates, ragged sizes
        _norm_case("grad-f32-odd", 777, 2064, "f32", post=True, gate_rows=7, pre=True, grad=True,
                   residual_scale=0.75),
        # a decode batch to four bits and back
        {"name": "mx4-decode", "kind": "mx4", "rows": 64, "hidden": 8192, "dtype": "bf16"},
        # a prefill batch to four bits and back
        {"name": "mx4-prefill", "kind": "mx4", "rows": 8192, "hidden": 8192, "dtype": "bf16"},
        # one token's projection: the weights' bytes count
        _project_case("project-token", 1, 8192, 8192),
        # odd tokens, features and hidden sizes that end inside a tile
        _project_case("project-odd", 777, 4112, 4128),
        # a prefill batch's projection: the product's rate counts
        _project_case("project-prefill", 8192, 8192, 8192),
        # norms, gate and residual, the normed rows straight to four bits and through the next projection
        dict(_norm_case("norm-project", 512, 8192, "bf16", post=True, gate_rows=1, pre=True, block_scale=0.5),
             kind="step", features=8192),
    ]


def _norm_case(name, rows, hidden, dtype, post, gate_rows, pre, grad=False, residual_scale=1.0, block_scale=1.0):
    return {"name": name, "kind": "grad" if grad else "norm", "rows": rows, "hidden": hidden, "dtype": dtype,
            "post": post, "gate_rows": gate_rows, "pre": pre, "residual_scale": residual_scale,
            "block_scale": block_scale}


def _project_case(name, rows, features, hidden):
    return {"name": name, "kind": "project", "rows": rows, "features": features, "hidden": hidden}


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["norm", "grad", "mx4", "project", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "mx4":
        return {"kind": kind, "rows": _log(rng, 1, 8192), "hidden": _log(rng, 64, 8192, 32),
                "dtype": rng.choice(["bf16", "f32"])}
    if kind == "project":
        return {"kind": kind, "rows": _log(rng, 1, 8192), "features": _log(rng, 64, 8192, 16),
                "hidden": _log(rng, 64, 8192, 32)}
    form = rng.choice(["none", "shared", "sequence", "token"])
    seqs = rng.randint(2, 9)
    rows = _log(rng, 1, 8192 // (2 if dtype == "f32" else 1))
    if form == "sequence":
        rows = seqs * max(1, rows // seqs)
    c = _norm_case("", rows, _log(rng, 64, 8192, 16), dtype, post=rng.random() < 0.7,
                   gate_rows={"none": 0, "shared": 1, "sequence": seqs, "token": rows}[form], pre=True,
                   grad=kind == "grad", residual_scale=rng.choice([1.0, 0.75]),
                   block_scale=rng.choice([1.0, 0.5]))
    del c["name"]
    if kind == "step":
        c.update(kind="step", dtype="bf16", hidden=_log(rng, 64, 8192, 32), features=_log(rng, 64, 8192, 16),
                 rows=min(rows, 4096 // seqs * seqs))
        if form == "token":
            c["gate_rows"] = c["rows"]
    return c


_EPS = 1e-5


def work(case):
    t, h, kind = case["rows"], case["hidden"], case["kind"]
    if kind == "mx4":  # read, write codes and scales, read them back, write
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": t * h * (2 * size + 2 * (0.5 + 1 / 32)), "flops": 4 * t * h}
    if kind == "project":
        n = case["features"]
        return {"bytes": 2 * t * h + n * h * (0.5 + 1 / 32) + 2 * t * n, "flops": 2 * t * n * h}
    size = 2 if case["dtype"] == "bf16" else 4
    gate = case["gate_rows"] * h * size
    weights = (int(case["post"]) + int(case["pre"])) * h * size
    if kind == "norm":
        return {"bytes": 4 * t * h * size + gate + weights, "flops": 12 * t * h}
    if kind == "grad":  # x, h, dy, dh in; dx, dresidual out; the weights' gradients in 32 bits
        grads = (int(case["post"]) + int(case["pre"])) * h * 4
        return {"bytes": 6 * t * h * size + 2 * gate + weights + grads, "flops": 30 * t * h}
    n = case["features"]
    return {"bytes": 3 * t * h * size + gate + weights + n * h * (0.5 + 1 / 32) + 2 * t * n,
            "flops": 12 * t * h + 2 * t * n * h}


# ----------------------------------------------------------------- inputs ---
def _normal(gen, *shape, dtype=torch.float32, mean=0.0, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)


def _activations(gen, rows, hidden, dtype):
    """N(0, 1) with half a percent of the channels twenty times as large, as the boundary's activations are."""
    x = torch.randn(rows, hidden, generator=gen, device="cuda")
    channel = torch.rand(hidden, generator=gen, device="cuda") < 0.005
    return (x * torch.where(channel, 20.0, 1.0)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, h = case["rows"], case["hidden"]
    s = {"case": case}
    if case["kind"] == "mx4":
        s["x"] = _activations(gen, t, h, _TYPES[case["dtype"]])
        return s
    if case["kind"] in ("project", "step"):
        n = case["features"]
        w = _normal(gen, n, h, std=1 / math.sqrt(h))
        codes, e = _mx4_encode(w)
        s["weight"] = (_pack(codes), _tile(e))  # laid out once, as the framework's scales are kept
    if case["kind"] == "project":
        s["x"] = _activations(gen, t, h, torch.bfloat16)
        return s
    dtype = _TYPES[case["dtype"]]
    s["x"] = _activations(gen, t, h, dtype)
    s["residual"] = _normal(gen, t, h, dtype=dtype)
    s["post_weight"] = _normal(gen, h, dtype=dtype, mean=1.0, std=0.1) if case["post"] else None
    s["pre_weight"] = _normal(gen, h, dtype=dtype, mean=1.0, std=0.1) if case["pre"] else None
    s["gate"] = _normal(gen, case["gate_rows"], h, dtype=dtype, std=0.7) if case["gate_rows"] else None
    if case["kind"] == "grad":
        s["h"], _ = _norm_plain(s)  # kept by the forward pass
        del s["residual"]
        s["dy"] = _normal(gen, t, h, dtype=dtype)
        s["dh"] = _normal(gen, t, h, dtype=dtype)
    return s


# ------------------------------------------------------------ plain forms ---
def _gated(case, u, gate):
    """Each row's values times its gate: rows / gate_rows neighbouring rows share one."""
    if gate is None:
        return u
    return (u.view(case["gate_rows"], -1, case["hidden"]) * gate[:, None]).view_as(u)


def _inv(x):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + _EPS)


def _norm_plain(s):
    c, x = s["case"], s["x"].float()
    u = x * _inv(x) * s["post_weight"].float() if c["post"] else x
    u = _gated(c, u, None if s["gate"] is None else s["gate"].float())
    h = (c["residual_scale"] * s["residual"].float() + c["block_scale"] * u).to(s["x"].dtype)
    hf = h.float()  # the norm before the next block is that of the residual stream as it is kept
    return h, (hf * _inv(hf) * s["pre_weight"].float()).to(s["x"].dtype)


def _grad_plain(s):
    c, dtype, x, h = s["case"], s["x"].dtype, s["x"].float(), s["h"].float()
    inv_h = _inv(h)
    hh, dy = h * inv_h, s["dy"].float()
    dn = dy * s["pre_weight"].float()
    dh = s["dh"].float() + inv_h * (dn - hh * (dn * hh).mean(1, keepdim=True))
    out = {"dpre_weight": (dy * hh).sum(0), "dresidual": (c["residual_scale"] * dh).to(dtype)}
    xh = x * _inv(x) if c["post"] else x
    u = xh * s["post_weight"].float() if c["post"] else x
    db = c["block_scale"] * dh
    du = _gated(c, db, None if s["gate"] is None else s["gate"].float())
    if s["gate"] is not None:
        out["dgate"] = (db * u).view(c["gate_rows"], -1, c["hidden"]).sum(1).to(dtype)
    if c["post"]:
        out["dpost_weight"] = (du * xh).sum(0)
        dxh = du * s["post_weight"].float()
        du = _inv(x) * (dxh - xh * (dxh * xh).mean(1, keepdim=True))
    out["dx"] = du.to(dtype)
    return out


def _mx4_encode(x):
    """Codes (e2m1, one a byte) and scales' exponents (e8m0) of x, in blocks of 32 along its rows."""
    b = x.float().view(x.shape[0], -1, 32)
    e = ((b.abs().amax(2).view(torch.int32) >> 23) - 2).clamp(min=0)  # floor(log2) - 2, with the bias 127
    a = b.abs() * ((254 - e) << 23).view(torch.float32)[..., None]
    codes = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
             + (a >= 3.5).byte() + (a > 5).byte()) + (b < 0).byte() * 8
    return codes.view(x.shape), e.to(torch.uint8)


def _mx4_values(codes, e):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    grid = torch.cat([grid, -grid])
    scale = torch.where(e == 0, 2.0 ** -127, (e.int() << 23).view(torch.float32))
    return (grid[codes.int()].view(codes.shape[0], -1, 32) * scale[..., None]).view(codes.shape)


def _pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous()


def _unpack(packed):
    return torch.stack([packed & 15, packed >> 4], 2).view(packed.shape[0], -1)


def _tile(e):
    """Scales in tiles of 128 rows and 4 blocks: row r, block k at byte (r % 32) * 16 + (r / 32 % 4) * 4 + k % 4."""
    rows, blocks = e.shape
    p = torch.nn.functional.pad(e, (0, -blocks % 4, 0, -rows % 128))
    return p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile(tiled, rows, blocks):
    q = -(-blocks // 4)
    p = tiled.view(-1, q, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * q)
    return p[:rows, :blocks]


def _weight_values(s):
    codes, scales = s["weight"]
    return _mx4_values(_unpack(codes), _untile(scales, codes.shape[0], codes.shape[1] // 16))


def _project_plain(s, x):
    return (_mx4_values(*_mx4_encode(x)) @ _weight_values(s).T).to(torch.bfloat16)


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "mx4":
        return _mx4_values(*_mx4_encode(s["x"])).to(s["x"].dtype)
    if kind == "project":
        return _project_plain(s, s["x"])
    if kind == "grad":
        return _grad_plain(s)
    h, y = _norm_plain(s)
    return {"h": h, "y": y} if kind == "norm" else {"h": h, "out": _project_plain(s, y)}


# ------------------------------------------------------- the framework's ---
def _bind(s):
    """The pass's calls with their arguments marshalled once (fcomm.Bound), as a serving or training loop with fixed
    buffers keeps them, and the buffers that they write."""
    from quantized_reduce_rmsnorm_gb300 import fcomm as fc
    c, x = s["case"], s["x"]
    kind, t, h = c["kind"], c["rows"], c["hidden"]
    if kind in ("mx4", "project", "step"):
        q = fc.alloc_mx4(t, h)
    if kind == "mx4":
        out = torch.empty_like(x)
        return [fc.bind_mx4_quantize(x, q), fc.bind_mx4_dequantize(q, out)], out
    if kind in ("project", "step"):
        out = torch.empty(t, c["features"], dtype=torch.bfloat16, device="cuda")
        product = fc.bind_mx4_matmul(q, s["weight"], out)
    if kind == "project":
        return [fc.bind_mx4_quantize(x, q), product], out
    spec = dict(post_weight=s["post_weight"], gate=s["gate"], pre_weight=s["pre_weight"],
                residual_scale=c["residual_scale"], block_scale=c["block_scale"], post_eps=_EPS, pre_eps=_EPS)
    if kind == "grad":
        out = {"dx": torch.empty_like(x), "dresidual": torch.empty_like(x),
               "dpre_weight": torch.empty(h, dtype=torch.float32, device="cuda")}
        if c["post"]:
            out["dpost_weight"] = torch.empty(h, dtype=torch.float32, device="cuda")
        if s["gate"] is not None:
            out["dgate"] = torch.empty_like(s["gate"])
        ws = fc.alloc_block_norm_workspace(t, h, c["gate_rows"])
        return [fc.bind_block_norm_backward(x, s["h"], s["dy"], s["dh"], workspace=ws, **out, **spec)], out
    hid = torch.empty_like(x)
    if kind == "norm":
        y = torch.empty_like(x)
        return [fc.bind_block_norm(x, s["residual"], hid, y, **spec)], {"h": hid, "y": y}
    return [fc.bind_block_norm(x, s["residual"], hid, None, y_mx4=q, **spec), product], {"h": hid, "out": out}


def run(state):
    if not own:
        return _plain(state)
    if "calls" not in state:
        state["calls"], state["out"] = _bind(state)
    for call in state["calls"]:
        call()
    return state["out"]


# ------------------------------------------------------------------ exact ---
def exact(case, seed):
    s = prepare(case, seed)
    kind, t, h = case["kind"], case["rows"], case["hidden"]

    def quantised(v):
        """Values of v in four bits: spacing 2^(floor(log2 |v|) - 1), 0.5 below 1, at most 6, after the block's scale."""
        b = v.double().reshape(v.shape[0], -1, 32)
        top = torch.frexp(b.abs().amax(2, keepdim=True))
        scale = torch.ldexp(torch.ones_like(top.mantissa), (top.exponent - 3).clamp(min=-127))
        a = b.abs() / scale
        step = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 1).clamp(min=0) - 1)
        a = torch.where(top.mantissa == 0, 0.0, torch.round(a / step) * step).clamp(max=6.0)
        return (torch.copysign(a, b) * scale).reshape(v.shape)

    def product(v):
        packed, tiled = s["weight"]
        values = torch.tensor([0.0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
        k = torch.arange(h, device="cuda")
        nibble = (packed[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
        w = values[(nibble & 7).long()] * (1 - 2 * (nibble >> 3)).double()
        r, b = torch.arange(len(packed), device="cuda")[:, None], (k // 32)[None]
        at = ((r // 128) * -(-h // 128) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
        return quantised(v) @ (w * torch.exp2(tiled[at].double() - 127)).T

    if kind == "mx4":
        return quantised(s["x"])
    if kind == "project":
        return product(s["x"])
    x = s["x"].double()
    group = torch.arange(t, device="cuda") // (t // max(1, case["gate_rows"]))
    g = torch.ones_like(x) if s["gate"] is None else s["gate"].double()[group]
    w1 = s["post_weight"].double() if case["post"] else None
    rx = (x.square().mean(1, keepdim=True) + _EPS).rsqrt() if case["post"] else torch.ones(t, 1, device="cuda").double()
    u = x * rx * w1 if case["post"] else x
    w2 = s["pre_weight"].double()
    if kind != "grad":
        hid = case["residual_scale"] * s["residual"].double() + case["block_scale"] * g * u
        kept = hid.to(s["x"].dtype).double()
        y = w2 * kept / (kept.square().mean(1, keepdim=True) + _EPS).sqrt()
        return {"h": hid, "y": y} if kind == "norm" else {"h": hid, "out": product(y.to(s["x"].dtype))}
    # y = w2 h r with r = (mean h^2 + eps)^(-1/2): dh_j = dh'_j + r w2_j dy_j - r^3 h_j / H sum_i w2_i dy_i h_i
    hid, dy = s["h"].double(), s["dy"].double()
    r = (hid.square().mean(1, keepdim=True) + _EPS).rsqrt()
    dh = s["dh"].double() + r * w2 * dy - r ** 3 * hid * (w2 * dy * hid).sum(1, keepdim=True) / h
    out = {"dpre_weight": (dy * hid * r).sum(0), "dresidual": case["residual_scale"] * dh}
    db = case["block_scale"] * dh
    if s["gate"] is not None:
        zero = torch.zeros(case["gate_rows"], h, dtype=torch.float64, device="cuda")
        out["dgate"] = zero.index_add(0, group, db * u)
    if case["post"]:
        out["dpost_weight"] = (db * g * x * rx).sum(0)
        e = db * g * w1
        out["dx"] = rx * e - rx ** 3 * x * (e * x).sum(1, keepdim=True) / h
    else:
        out["dx"] = db * g
    return out
