"""Plain 64-bit references of layer norm, its gradient, 8-bit floating point with a scale
for each block of 128, the product, and the gated feed-forward with its gradient (torch
float64 on whichever device the inputs are on), each with the size of the terms that
make it up, and inputs whose results are exact."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24                                             # half a step of binary32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TC = 2.0 ** -23  # a step of the tensor core's sum, of the sum of the terms' sizes


# ------------------------------------------------------------ layer norm ---
def layer_norm_reference(h, weight, bias, eps):
    """(y, stats, size of y's error in units of U): see the tests' tolerances."""
    h = h.double()
    mean = h.mean(1, keepdim=True)
    inv = ((h - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    n = (h - mean) * inv
    w = 1.0 if weight is None else weight.double()
    b = torch.zeros_like(h) if bias is None else bias.double().expand_as(h)
    y = n * w + b
    # a normed value is off by its own rounding, by the mean's (26 U of the mean size of the
    # distances to a first mean that is itself off by 26 U of the mean size of the values)
    # and by the inverse deviation's
    first = 26 * U * h.abs().mean(1, keepdim=True) * inv
    size = 64 * (n.abs() + 1 + first) * abs(w) + 2 * b.abs()
    return y, torch.cat([mean, inv], 1), size


def layer_norm_grad_reference(h, stats, dy, dh, weight):
    """{name: (value, size)} by the formula, from the statistics given."""
    m, r = stats[:, :1].double(), stats[:, 1:].double()
    n, dy = (h.double() - m) * r, dy.double()
    a = dy if weight is None else dy * weight.double()
    dx = r * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
    size = r * (a.abs() + a.abs().mean(1, keepdim=True) + n.abs() * (a * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    return {"dx": (dx, size), "dweight": ((dy * n).sum(0), (dy * n).abs().sum(0)), "dbias": (dy.sum(0), dy.abs().sum(0))}


# ------------------------------------------------- 8-bit floating point ----
def grid() -> torch.Tensor:
    """The non-negative e4m3 values by code, 0 to 0x7E."""
    c = torch.arange(127)
    e, m = c >> 3, (c & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))


def values(codes) -> torch.Tensor:
    """float64 values of e4m3 codes."""
    g = torch.cat([grid(), torch.tensor([float("nan")], dtype=torch.float64)]).to(codes.device)
    c = codes.long()
    return g[c & 127] * (1 - 2 * (c >> 7)).double()


def spread(scales, rows: int, hidden: int) -> torch.Tensor:
    """One scale an element, [rows, hidden], of scales for blocks of 1 or 128 rows."""
    br = 1 if scales.shape[0] == rows else 128
    s = scales.double().repeat_interleave(br, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :hidden]


def quantise(x, block_rows: int):
    """(codes, scales) by the definition: the scale and the quotient are binary32 numbers,
    the code's value the nearest of the grid, ties to the even code."""
    rows, hidden = x.shape
    xs = x.float()
    nb, kb = -(-rows // block_rows), -(-hidden // 128)
    scales = torch.empty(nb, kb)
    codes = torch.empty(rows, hidden, dtype=torch.uint8)
    g = grid()
    mid = (g[:-1] + g[1:]) / 2
    for i in range(nb):
        for k in range(kb):
            r, c = slice(i * block_rows, (i + 1) * block_rows), slice(k * 128, (k + 1) * 128)
            b = xs[r, c]
            if not torch.isfinite(b).all():
                scales[i, k] = float("nan")
                codes[r, c] = 0x7F
                continue
            s = (b.abs().max().double() / 448).float().clamp(min=2.0 ** -60)  # one division, rounded once
            scales[i, k] = s
            q = (b.double().abs() / s.double()).float().double()
            below = torch.bucketize(q, mid, right=False)   # ties go down ...
            tie = (below < 126) & (q == mid[below.clamp(max=125)])
            code = torch.where(tie & (below % 2 == 1), below + 1, below)  # ... unless the code is odd
            codes[r, c] = (code + 128 * torch.signbit(b).long()).to(torch.uint8)
    return codes, scales


def exact_pair(g: torch.Generator, rows: int, features: int, hidden: int):
    """Two 8-bit operands whose product is exact in binary32 in any order of its sums: codes
    of 0, 1, 2 and 3 and their negatives, scales of 1, 2 or 4 that differ from block to
    block; the sum of the sizes, below 9 * 16 * hidden, is below 2^24 for hidden up to 65536."""
    pick = torch.tensor([0x00, 0x38, 0x40, 0x44, 0xB8, 0xC0, 0xC4], dtype=torch.uint8)  # 0, 1, 2, 3, -1, -2, -3
    out = []
    for n, br in ((rows, 1), (features, 128)):
        codes = pick[torch.randint(0, 7, (n, hidden), generator=g)]
        scales = torch.exp2(torch.randint(0, 3, (-(-n // br), -(-hidden // 128)), generator=g).float())
        out.append((codes, scales))
    assert 144 * hidden < 2 ** 24
    x, w = (values(c) * spread(s, c.shape[0], hidden) if s.shape[0] == c.shape[0]
            else values(c) * s.double().repeat_interleave(128, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :hidden]
            for c, s in out)
    return out, x @ w.T


# -------------------------------------------------- gated feed-forward -----
def activation(name: str, z):
    """(act, act', p): the activation z sigmoid(p), its slope, and p."""
    if name == "silu":
        p, dp = z, torch.ones_like(z)
    else:
        k = 2 * math.sqrt(2 / math.pi)
        p, dp = k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(p)
    return z * s, s + z * dp * s * torch.sigmoid(-p), p


def gated_reference(x, wg, wu, name):
    """(out, tolerance of its binary32 value, g, u, tolerances of those)."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    K = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = (K * TC * (x.abs() @ w.abs().T) for w in (wg, wu))
    a, _, p = activation(name, g)
    # the slope of either activation is below 1.13; sigmoid(p) is within (5 |p| + 16) U of itself
    # (p's own roundings, the exponential's, the reciprocal's), and below 2^-120 where it is
    # flushed to 0
    tol = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + ((5 * p.abs() + 16) * U * a.abs() + 2.0 ** -110) * u.abs()
    return a * u, tol, g, u, eg, eu


def gated_grad_reference(x, wg, wu, gate, up, dout, name):
    """{name: (value, size of the terms)}, and the relative error of dg and du before their
    rounding, in units of U of their terms."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    z, u, d = gate.double(), up.double(), dout.double()
    a, slope, p = activation(name, z)
    s = torch.sigmoid(p)
    dg, du = d * u * slope, d * a
    # the slope's two terms: s, off by rel of itself, and z p' s t with t = 1 - s, which is off by
    # what s is, sigmoid(-p) rel (the exponential's share) and 4 U of it, and by its rounding
    dp = torch.ones_like(z) if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    rel = (5 * p.abs() + 24) * U
    eg = (d * u).abs() * (s * rel + (z * dp).abs() * s * (2 * torch.sigmoid(-p) * rel + 6 * U)) + 2.0 ** -110 * (d * u).abs()
    eu = rel * (d * a).abs() + 2.0 ** -110 * d.abs()
    # dg and du as the products take them: two bf16 numbers each for few tokens or few values, else one
    terms = 2 if len(z) <= 128 or z.numel() <= 1 << 19 else 1
    half = HALF[torch.bfloat16] ** terms
    tg, tu = eg + half * dg.abs(), eu + half * du.abs()
    R, F = x.shape[0], wg.shape[0]
    return {"dx": (dg @ wg + du @ wu, tg @ wg.abs() + tu @ wu.abs() + 2 * F * terms * TC * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())),
            "dw_gate": (dg.T @ x, tg.T @ x.abs() + R * terms * TC * (dg.abs().T @ x.abs())),
            "dw_up": (du.T @ x, tu.T @ x.abs() + R * terms * TC * (du.abs().T @ x.abs()))}


def two_term_case(g: torch.Generator, rows: int, features: int, hidden: int, device="cpu"):
    """Inputs of the gradient (SiLU) whose factors need two bf16 numbers each and whose sums
    binary32 holds exactly, with their dg and du: where the gate's projection is 65, SiLU is 65
    and its slope 1 (in binary32); dout is odd and up such that dg = dout up is odd and above
    256, as du = 65 dout is.  Weights of -1, 0 and 1: a sum of sizes is below 1430 features."""
    assert 2 * 715 * features < 2 ** 24 and 3 * 715 * rows < 2 ** 24

    def odd(lo, hi, *shape):
        v = 2 * torch.randint(lo // 2, (hi + 1) // 2, shape, generator=g) + 1
        return v * (2 * torch.randint(0, 2, shape, generator=g) - 1)

    def ints(most, *shape):
        return torch.randint(-most, most + 1, shape, generator=g)

    i = dict(x=ints(3, rows, hidden), w_gate=ints(1, features, hidden), w_up=ints(1, features, hidden),
             gate=torch.full((rows, features), 65), up=odd(53, 65, rows, features), dout=odd(5, 11, rows, features))
    i = {k: v.to(torch.bfloat16).to(device) for k, v in i.items()}
    d, u = i["dout"].double(), i["up"].double()
    dg, du = d * u, 65 * d
    assert dg.abs().min() > 256 and max(dg.abs().max(), du.abs().max()) <= 715 and (dg % 2 != 0).all()
    return i, dg, du


def gradients(i, dg, du):
    """bf16 gradients of the factors, of sums that are exact."""
    x, wg, wu = (i[k].double() for k in ("x", "w_gate", "w_up"))
    out = {"dx": dg @ wg + du @ wu, "dw_gate": dg.T @ x, "dw_up": du.T @ x}
    return {k: v.float().to(torch.bfloat16) for k, v in out.items()}
