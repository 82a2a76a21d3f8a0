"""Plain 64-bit references of the block norms, their gradient, microscaled
4-bit quantisation and the product (torch float64 on whichever device the
inputs are on), and the inputs of their tests."""
from __future__ import annotations

import torch

U = 2.0 ** -24                                             # half a step of binary32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx4_reference(x: torch.Tensor):
    """(codes [rows, hidden] one a byte, scale bytes [rows, hidden / 32]) by the
    definition, element by element against the midpoints of the e2m1 grid."""
    rows, hidden = x.shape
    b = x.double().reshape(rows, hidden // 32, 32)
    bad = ~torch.isfinite(b).all(2)
    b = torch.where(torch.isfinite(b), b, 0.0)
    m = b.abs().amax(2)
    e = torch.where(m > 0, torch.frexp(m).exponent - 1 - 2, -127).clamp(min=-127)
    a = b.abs() / torch.ldexp(torch.ones_like(m), e)[..., None]
    code = torch.zeros_like(a, dtype=torch.int64)
    for i in range(1, 8):
        mid = (GRID[i - 1] + GRID[i]) / 2
        # a tie goes to the even code
        code = torch.where((a > mid) | ((a == mid) & (i % 2 == 0)), i, code)
    code = code + 8 * torch.signbit(x.reshape(b.shape)).long()
    byte = torch.where(bad, 255, e + 127)
    return code.reshape(rows, hidden), byte


def scale_offsets(rows: int, hidden: int) -> torch.Tensor:
    """Byte offset of every [row, block] scale in the tiled layout."""
    r = torch.arange(rows)[:, None]
    k = torch.arange(hidden // 32)[None]
    return (r // 128 * -(-hidden // 128) + k // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + k % 4


def unpack(codes: torch.Tensor) -> torch.Tensor:
    """uint8 [rows, hidden / 2] -> one code a byte [rows, hidden]."""
    return torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1).long()


def mx4_values(code: torch.Tensor, byte: torch.Tensor) -> torch.Tensor:
    """The float64 values of codes [rows, hidden] and scale bytes [rows, hidden / 32]."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=code.device)
    v = grid[code & 7] * (1 - 2 * (code >> 3)).double()
    s = torch.where(byte == 255, float("nan"), torch.exp2(byte.double() - 127))
    return v * s.repeat_interleave(32, 1)


def pack_mx4(code: torch.Tensor, byte: torch.Tensor, fill: int = 0):
    """(codes, scales) as the library lays them out; the rows behind the last
    hold `fill`, the blocks past a row's end 0."""
    rows, hidden = code.shape
    tiles = -(-hidden // 128)
    scales = torch.full((-(-rows // 128) * tiles * 512,), fill, dtype=torch.uint8)
    scales[scale_offsets(rows, tiles * 128)] = 0
    scales[scale_offsets(rows, hidden)] = byte.to(torch.uint8).cpu()
    c = code.to(torch.uint8)
    return (c[:, 0::2] | c[:, 1::2] << 4).contiguous(), scales


def gate_rows_of(gate, rows: int) -> torch.Tensor:
    """gate expanded to one row a token."""
    return gate.double().repeat_interleave(rows // gate.shape[0], 0)


def norm_reference(x, r, post_w, gate, alpha, beta, eps):
    """(h, |alpha r| + |beta g u|): h in 64 bits and the size of its two terms."""
    x = x.double()
    u = x if post_w is None else x / (x.square().mean(1, keepdim=True) + eps).sqrt() * post_w.double()
    if gate is not None:
        u = u * gate_rows_of(gate, x.shape[0])
    res = torch.zeros_like(x) if r is None else alpha * r.double()
    return res + beta * u, res.abs() + (beta * u).abs()


def rms_reference(h, w, eps):
    h = h.double()
    return h / (h.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def grad_reference(x, h, dy, dh, post_w, gate, pre_w, alpha, beta, eps):
    """The gradients in 64 bits, and for each the size of the terms that make it
    up: {name: (value, size)}."""
    x, n = x.double(), x.shape[1]
    rows = x.shape[0]
    out = {}
    d = torch.zeros_like(x) if dh is None else dh.double()
    size = d.abs()
    if pre_w is not None:
        h, dy, w2 = h.double(), dy.double(), pre_w.double()
        r = (h.square().mean(1, keepdim=True) + eps).rsqrt()
        dn, hh = dy * w2, h * r
        d = d + r * (dn - hh * (dn * hh).mean(1, keepdim=True))
        size = size + r * (dn.abs() + hh.abs() * (dn * hh).abs().mean(1, keepdim=True))
        out["dpre_weight"] = ((dy * hh).sum(0), (dy * hh).abs().sum(0))
    out["dresidual"] = (alpha * d, abs(alpha) * size)
    rx = torch.ones(rows, 1, dtype=x.dtype, device=x.device)
    w1 = torch.ones(n, dtype=x.dtype, device=x.device)
    if post_w is not None:
        rx, w1 = (x.square().mean(1, keepdim=True) + eps).rsqrt(), post_w.double()
    xh = x * rx
    g = torch.ones_like(x) if gate is None else gate_rows_of(gate, rows)
    if gate is not None:
        def fold(t):
            return t.reshape(gate.shape[0], -1, n).sum(1)
        out["dgate"] = (fold(beta * d * xh * w1), fold(abs(beta) * size * (xh * w1).abs()))
    du, su = beta * g * d, (beta * g).abs() * size
    if post_w is not None:
        out["dpost_weight"] = ((du * xh).sum(0), (su * xh.abs()).sum(0))
        e, se = du * w1, su * w1.abs()
        out["dx"] = (rx * (e - xh * (e * xh).mean(1, keepdim=True)),
                     rx * (se + xh.abs() * (se * xh.abs()).mean(1, keepdim=True)))
    else:
        out["dx"] = (du, su)
    return out


def scaled_pair(g: torch.Generator, rows: int, features: int, hidden: int):
    """Two microscaled operands whose blocks' scales differ, (code, byte) each, and whose
    product is exact in binary32 in any order of its sums: values are multiples of
    0.5, products of 0.25, and the sum of the products' sizes, which bounds every
    partial sum, is below 2^24 of those.  Scales of 1 to 128 where that leaves room,
    else of 1 to 8, of 1 or 2."""
    code = [torch.randint(0, 16, (n, hidden), generator=g) for n in (rows, features)]
    pick = [torch.randint(0, 8, (n, hidden // 32), generator=g) for n in (rows, features)]
    for spread in (8, 4, 2):
        byte = [127 + p % spread for p in pick]
        xv, wv = (mx4_values(c, b) for c, b in zip(code, byte))
        if (xv.abs() @ wv.abs().T).max() * 4 < 2 ** 24:
            return list(zip(code, byte)), xv @ wv.T
    raise AssertionError("no such scales at this size")
