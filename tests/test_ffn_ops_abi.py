"""CPU checks of layer norm, 8-bit floating point and the gated feed-forward: sizes,
references, and every refusal before anything touches a GPU (the pointers given here are
never followed)."""
import pytest
import torch

import ffn_ref as ref
from quantized_reduce_rmsnorm_gb300 import fcomm as fc

A = [1 << 40 | k << 33 for k in range(1, 20)]  # 32-byte aligned, eight gigabytes apart
BF16, F32, INT8 = fc.FMT_BF16, fc.FMT_F32, fc.FMT_INT8_SYM


def refused(name, *args, status=fc.FC_ERR_INVALID, says=""):
    L = fc.load()
    assert getattr(L, name)(*args) == status
    msg = L.fc_last_error().decode()
    assert msg and says in msg, msg


def test_sizes():
    L = fc.load()
    assert fc.fp8_scales(3, 144) == 6 and fc.fp8_scales(129, 144, 128) == 4 and fc.fp8_scales(0, 128) == 0
    assert fc.fp8_scales(3, 24) == 0 and fc.fp8_scales(3, 32, 64) == 0 and fc.fp8_scales(-1, 32) == 0
    ws = L.fc_layer_norm_backward_workspace
    assert ws(5, 64) == 5 * 64 * 8 and ws(10 ** 6, 64) == 608 * 64 * 8 and ws(0, 64) == 0
    ws = L.fc_gated_ffn_backward_workspace
    assert ws(5, 64) == 5 * 64 * 8 and ws(1 << 20, 1 << 14) == 1 << 36 and ws(0, 64) == 0
    assert ws(128, 1 << 14) == 1 << 24 and ws(512, 1024) == 1 << 22 and ws(4096, 8192) == 1 << 27


@pytest.mark.parametrize("name", ["fc_layer_norm_backward_workspace", "fc_gated_ffn_backward_workspace"])
def test_a_workspace_serves_smaller_calls(name):
    """A workspace laid out for the largest call holds what any smaller one takes."""
    ws = getattr(fc.load(), name)
    rows, cols = [1, 16, 64, 127, 128, 129, 511, 512, 513, 1023, 1024, 1025, 4096], [16, 512, 1024, 1040, 4096, 16384]
    for f in cols:
        sizes = [ws(r, f) for r in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for r in rows:
        sizes = [ws(r, f) for f in cols]
        assert sizes == sorted(sizes)
    if name == "fc_gated_ffn_backward_workspace":  # dg and du, in one bf16 number or two
        for r in rows:
            for f in cols:
                assert ws(r, f) >= r * f * (8 if r <= 128 or r * f <= 1 << 19 else 4)


# ------------------------------------------------------------ references ---
def test_grid_and_quantiser_by_hand():
    g = ref.grid()
    assert len(g) == 127 and g[1] == 2.0 ** -9 and g[7] == 7 * 2.0 ** -9 and g[8] == 2.0 ** -6 and g[126] == 448
    assert (g[1:] > g[:-1]).all()
    x = torch.zeros(1, 16)
    x[0, :6] = torch.tensor([448.0, -448.0, 1.0, 17.0, 19.0, -2.0 ** -10])  # scale 1: ties to even
    codes, scales = ref.quantise(x, 1)
    assert scales.tolist() == [[1.0]]
    assert ref.values(codes)[0, :6].tolist() == [448, -448, 1, 16, 20, 0]
    assert codes[0, 5] == 0x80
    codes, scales = ref.quantise(torch.zeros(2, 16), 128)
    assert scales.tolist() == [[2.0 ** -60]] and (codes == 0).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantiser_agrees_with_the_float8_cast(block_rows):
    g = torch.Generator().manual_seed(block_rows)
    x = torch.randn(130, 272, generator=g) * torch.exp2(torch.randint(-20, 20, (130, 1), generator=g).float())
    codes, scales = ref.quantise(x, block_rows)
    s = ref.spread(scales, 130, 272).float()
    assert torch.equal((x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), codes)
    assert ref.values(codes).abs().max() == 448


@pytest.mark.parametrize("hidden", [16, 144, 4096])
def test_exact_product_inputs_show_every_block(hidden):
    """A block left out or two blocks' scales exchanged change the exact inputs' product."""
    g = torch.Generator().manual_seed(hidden)
    ((xc, xs), (wc, ws)), want = ref.exact_pair(g, 5, 144, hidden)
    assert torch.equal(want.float().double(), want)
    full = [ref.values(xc) * ref.spread(xs, 5, hidden), ref.values(wc) * ref.spread(ws, 144, hidden)]
    assert torch.equal(full[0] @ full[1].T, want)
    for k in range(-(-hidden // 128)):
        cut = full[0].clone()
        cut[:, k * 128:(k + 1) * 128] = 0
        assert ((cut @ full[1].T) != want).any(1).all()


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activation_reference(name):
    z = torch.linspace(-30, 30, 1201, dtype=torch.float64, requires_grad=True)
    want = torch.nn.functional.silu(z) if name == "silu" else torch.nn.functional.gelu(z, approximate="tanh")
    want.sum().backward()
    a, slope, _ = ref.activation(name, z.detach())
    assert (a - want.detach()).abs().max() < 1e-13 and (slope - z.grad).abs().max() < 1e-12
    assert slope.abs().max() < 1.13


def test_gated_gradient_reference_is_that_of_the_formula():
    g = torch.Generator().manual_seed(3)
    x, wg, wu, d = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((6, 32), (16, 32), (16, 32), (6, 16)))
    for name in ("silu", "gelu"):
        t = [v.clone().requires_grad_() for v in (x, wg, wu)]
        a = t[0] @ t[1].T
        a = torch.nn.functional.silu(a) if name == "silu" else torch.nn.functional.gelu(a, approximate="tanh")
        (a * (t[0] @ t[2].T) * d).sum().backward()
        got = ref.gated_grad_reference(x, wg, wu, x @ wg.T, x @ wu.T, d, name)
        for k, v in zip(("dx", "dw_gate", "dw_up"), t):
            assert torch.allclose(got[k][0], v.grad, rtol=1e-10, atol=1e-10), k


@pytest.mark.parametrize("rows,features,hidden", [(1, 144, 64), (16, 1040, 272), (65, 4112, 144), (300, 1040, 528)])
def test_two_term_inputs_show_both_second_terms(rows, features, hidden):
    """With the second bf16 number of dg or of du left out, or the two exchanged, every row of dx
    differs, and almost every row of the weights' gradients (of 16 tokens and more: a sum
    of one or two factors is often rounded to that of their first numbers)."""
    i, dg, du = ref.two_term_case(torch.Generator().manual_seed(rows), rows, features, hidden)
    (g1, u1), want = (v.to(torch.bfloat16).double() for v in (dg, du)), ref.gradients(i, dg, du)
    g2, u2 = dg - g1, du - u1
    for v in (g2, u2):
        assert (v != 0).all() and torch.equal(v.to(torch.bfloat16).double(), v)
    for a, b, spoilt in ((g1, du, ("dx", "dw_gate")), (dg, u1, ("dx", "dw_up")), (g1 + u2, u1 + g2, tuple(want))):
        got = ref.gradients(i, a, b)
        assert (got["dx"] != want["dx"]).any(1).all()
        for k in spoilt:
            assert rows < 16 or (got[k] != want[k]).any(1).double().mean() > 0.95, k


def test_layer_norm_gradient_reference_is_that_of_the_formula():
    g = torch.Generator().manual_seed(4)
    h, dy, dh = (torch.randn(5, 48, generator=g, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(48, generator=g, dtype=torch.float64) for _ in range(2))
    t = [v.clone().requires_grad_() for v in (h, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (48,), t[1], t[2], 1e-5)
    ((y * dy).sum() + (t[0] * dh).sum()).backward()
    want, stats, _ = ref.layer_norm_reference(h, w, b, 1e-5)
    assert torch.allclose(want, y.detach(), rtol=1e-12, atol=1e-12)
    got = ref.layer_norm_grad_reference(h, stats, dy, dh, w)
    for k, v in zip(("dx", "dweight", "dbias"), t):
        assert torch.allclose(got[k][0], v.grad, rtol=1e-10, atol=1e-10), k


# -------------------------------------------------------------- refusals ---
def norm(x=A[0], r=A[1], rows=6, hidden=64, dtype=BF16, w=A[2], b=A[3], eps=1e-5, h=A[4], y=A[5], st=A[6]):
    return (x, r, rows, hidden, dtype, w, b, eps, h, y, st, None)


def test_layer_norm_refusals():
    n = "fc_layer_norm"
    refused(n, *norm(rows=-1), says="rows")
    refused(n, *norm(hidden=72), says="multiple of 16")
    refused(n, *norm(hidden=0), says="multiple of 16")
    refused(n, *norm(hidden=16400), status=fc.FC_ERR_UNSUPPORTED)
    refused(n, *norm(rows=1 << 31), status=fc.FC_ERR_UNSUPPORTED)
    refused(n, *norm(dtype=INT8), says="dtype")
    for bad in (-1e-6, 1.5, float("nan")):
        refused(n, *norm(eps=bad), says="eps")
    refused(n, *norm(r=None), says="together")
    refused(n, *norm(h=None), says="together")
    for kw in (dict(x=None), dict(x=A[0] + 16), dict(r=A[1] + 16), dict(w=A[2] + 16), dict(b=A[3] + 16),
               dict(h=A[4] + 16), dict(y=None), dict(y=A[5] + 16), dict(st=A[6] + 4)):
        refused(n, *norm(**kw), says="must")
    refused(n, *norm(y=A[4]), says="overlaps")
    refused(n, *norm(y=A[0] + 64), says="overlaps")
    refused(n, *norm(y=A[2]), says="overlaps")
    refused(n, *norm(h=A[3]), says="overlaps")
    refused(n, *norm(st=A[0] + 64), says="overlaps")
    refused(n, *norm(st=A[5] + 64), says="overlaps")
    assert fc.load().fc_layer_norm(*norm(rows=0, x=None, y=None)) == fc.FC_OK


def back(h=A[0], st=A[1], dy=A[2], dh=A[3], rows=6, hidden=64, dtype=BF16, w=A[4], dx=A[5], dw=A[6], db=A[7], ws=A[8],
         d=None):
    return (h, st, dy, dh, rows, hidden, dtype, w, dx, dw, db, ws, d, None)


def test_layer_norm_backward_refusals():
    n = "fc_layer_norm_backward"
    refused(n, *back(hidden=72), says="multiple of 16")
    refused(n, *back(hidden=16400), status=fc.FC_ERR_UNSUPPORTED)
    refused(n, *back(dtype=INT8), says="dtype")
    for kw in (dict(h=None), dict(h=A[0] + 16), dict(st=None), dict(st=A[1] + 4), dict(dy=None), dict(dy=A[2] + 16),
               dict(dh=A[3] + 16), dict(w=A[4] + 16), dict(dx=None), dict(dx=A[5] + 16), dict(dw=A[6] + 2),
               dict(db=A[7] + 2), dict(ws=None), dict(ws=A[8] + 16), dict(d=A[9] + 2)):
        refused(n, *back(**kw), says="must")
    for kw in (dict(dx=A[0] + 64), dict(dx=A[1]), dict(dw=A[7]), dict(dw=A[2]), dict(db=A[4]), dict(ws=A[5]),
               dict(ws=A[0]), dict(dw=A[8] + 64), dict(d=A[1]), dict(d=A[6])):
        refused(n, *back(**kw), says="overlaps")
    for at in A[:9]:
        refused(n, *back(d=at), says="d_status")


def test_fp8_refusals():
    q = fc.Fp8(A[1], A[2])
    for rows, hidden, dtype, br, status in ((-1, 64, BF16, 1, 1), (4, 72, BF16, 1, 1), (4, 0, BF16, 1, 1),
                                            (4, 64, INT8, 1, 1), (4, 65552, F32, 1, 4), (1 << 31, 64, F32, 1, 4),
                                            (4, 64, BF16, 0, 1), (4, 64, BF16, 64, 1), (1 << 30, 512, F32, 128, 4)):
        refused("fc_fp8_quantize", A[0], dtype, rows, hidden, br, q, None, status=status)
        refused("fc_fp8_dequantize", q, rows, hidden, br, A[0], dtype, None, status=status)
    refused("fc_fp8_quantize", None, BF16, 4, 64, 1, q, None, says="x must not be NULL")
    refused("fc_fp8_quantize", A[0] + 16, BF16, 4, 64, 1, q, None, says="32-byte")
    refused("fc_fp8_quantize", A[0], BF16, 4, 64, 1, fc.Fp8(None, A[2]), None, says="out.codes")
    refused("fc_fp8_quantize", A[0], BF16, 4, 64, 1, fc.Fp8(A[1], A[2] + 2), None, says="out.scales")
    refused("fc_fp8_quantize", A[0], BF16, 4, 64, 1, fc.Fp8(A[0] + 64, A[2]), None, says="overlaps")
    refused("fc_fp8_quantize", A[0], BF16, 4, 64, 1, fc.Fp8(A[1], A[1] + 112), None, says="overlaps")
    refused("fc_fp8_dequantize", q, 4, 64, 1, None, BF16, None, says="out")
    refused("fc_fp8_dequantize", q, 4, 64, 128, A[1], BF16, None, says="overlaps")
    assert fc.load().fc_fp8_quantize(None, BF16, 0, 64, 1, fc.Fp8(), None) == fc.FC_OK
    assert fc.load().fc_fp8_dequantize(fc.Fp8(), 0, 64, 1, None, BF16, None) == fc.FC_OK
    x, w, n = fc.Fp8(A[1], A[2]), fc.Fp8(A[3], A[4]), "fc_fp8_matmul"
    for features in (0, 8, 24, -16):
        refused(n, x, w, 4, features, 64, A[0], BF16, None, None, says="features")
    refused(n, x, w, 4, 1 << 23, 64, A[0], BF16, None, None, status=fc.FC_ERR_UNSUPPORTED)
    refused(n, x, w, 1 << 23, 64, 64, A[0], BF16, None, None, status=fc.FC_ERR_UNSUPPORTED)
    refused(n, x, w, 4, 64, 72, A[0], BF16, None, None, says="multiple of 16")
    refused(n, x, w, 4, 64, 64, A[0], INT8, None, None, says="out_dtype")
    refused(n, x, fc.Fp8(), 4, 64, 64, A[0], BF16, None, None, says="w.codes")
    refused(n, fc.Fp8(A[1], None), w, 4, 64, 64, A[0], BF16, None, None, says="x.scales")
    refused(n, x, w, 4, 64, 64, None, BF16, None, None, says="out")
    refused(n, x, w, 4, 64, 64, A[0], BF16, A[5] + 2, None, says="d_status")
    for at in (A[1], A[2] + 12 - 4, A[3] + 64, A[4]):
        refused(n, x, w, 4, 64, 64, at // 32 * 32, BF16, None, None, says="overlaps")
    for at in (A[0], A[1], A[2], A[3], A[4]):
        refused(n, x, w, 4, 64, 64, A[0], BF16, at, None, says="d_status")
    assert fc.load().fc_fp8_matmul(x, w, 0, 64, 64, None, BF16, None, None) == fc.FC_OK


def ffn(x=A[0], wg=A[1], wu=A[2], rows=6, features=32, hidden=64, act=0, out=A[3], g=A[4], u=A[5], d=None):
    return (x, wg, wu, rows, features, hidden, act, out, g, u, d, None)


def ffn_back(x=A[0], wg=A[1], wu=A[2], g=A[3], u=A[4], dout=A[5], rows=6, features=32, hidden=64, act=0, dx=A[6],
             dwg=A[7], dwu=A[8], ws=A[9], d=None):
    return (x, wg, wu, g, u, dout, rows, features, hidden, act, dx, dwg, dwu, ws, d, None)


@pytest.mark.parametrize("name,args", [("fc_gated_ffn", ffn), ("fc_gated_ffn_backward", ffn_back)])
def test_gated_ffn_shapes(name, args):
    refused(name, *args(rows=-1), says="rows")
    refused(name, *args(rows=1 << 23), status=fc.FC_ERR_UNSUPPORTED)
    refused(name, *args(hidden=72), says="multiple of 16")
    refused(name, *args(hidden=65552), status=fc.FC_ERR_UNSUPPORTED)
    refused(name, *args(features=24), says="features")
    refused(name, *args(features=0), says="features")
    refused(name, *args(features=1 << 23), status=fc.FC_ERR_UNSUPPORTED)
    for act in (-1, 2):
        refused(name, *args(act=act), says="activation")


def test_gated_ffn_refusals():
    n = "fc_gated_ffn"
    refused(n, *ffn(g=None), says="together")
    refused(n, *ffn(u=None), says="together")
    for kw in (dict(x=None), dict(x=A[0] + 16), dict(wg=None), dict(wg=A[1] + 16), dict(wu=None), dict(wu=A[2] + 16),
               dict(out=None), dict(out=A[3] + 16), dict(g=A[4] + 16), dict(u=A[5] + 16), dict(d=A[6] + 2)):
        refused(n, *ffn(**kw), says="must")
    for kw in (dict(out=A[0]), dict(out=A[1] + 64), dict(out=A[2]), dict(g=A[3]), dict(u=A[4] + 32), dict(g=A[0]),
               dict(d=A[0]), dict(d=A[3]), dict(d=A[5])):
        refused(n, *ffn(**kw), says="overlaps")
    assert fc.load().fc_gated_ffn(*ffn(rows=0, x=None, out=None)) == fc.FC_OK


def test_gated_ffn_backward_refusals():
    n = "fc_gated_ffn_backward"
    refused(n, *ffn_back(dwg=None), says="together")
    refused(n, *ffn_back(dwu=None), says="together")
    refused(n, *ffn_back(dx=None, dwg=None, dwu=None), says="asked for")
    for k, name in enumerate(("x", "wg", "wu", "g", "u", "dout")):
        refused(n, *ffn_back(**{name: None}), says="must")
        refused(n, *ffn_back(**{name: A[k] + 16}), says="must")
    for kw in (dict(dx=A[6] + 16), dict(dwg=A[7] + 16), dict(dwu=A[8] + 16), dict(ws=None), dict(ws=A[9] + 16),
               dict(d=A[10] + 2)):
        refused(n, *ffn_back(**kw), says="must")
    for kw in (dict(dx=A[0]), dict(dx=A[3]), dict(dwg=A[1]), dict(dwu=A[7]), dict(ws=A[5]), dict(ws=A[6]), dict(d=A[9])):
        refused(n, *ffn_back(**kw), says="overlaps")


def test_gated_ffn_backward_factor_terms():
    L = fc.load()
    ws, by_size = L.fc_gated_ffn_backward_ex_workspace, L.fc_gated_ffn_backward_workspace
    for rows, features in ((1, 16), (128, 4096), (129, 8192), (4096, 8192), (0, 64)):
        assert ws(rows, features, 0) == by_size(rows, features) and ws(rows, features, 2) == 8 * rows * features
    assert ws(128, 64, 1) == 0 and ws(128, 64, 3) == 0 and ws(-1, 64, 2) == 0

    def args(terms, **kw):
        a = ffn_back(**kw)
        return (*a[:10], terms, *a[10:])

    n = "fc_gated_ffn_backward_ex"
    for terms in (-1, 1, 3):
        refused(n, *args(terms), says="factor_terms")
    refused(n, *args(2, hidden=72), says="multiple of 16")
    refused(n, *args(2, ws=A[9] + 16), says="must")
    far = 256 * 4096 * 4  # past what the call takes by size, not what it takes with two terms
    assert by_size(256, 4096) == far
    refused(n, *args(2, rows=256, features=4096, d=A[9] + far), says="workspace overlaps d_status")
    refused(n, *args(2, rows=256, features=4096, d=A[9] + 2 * far - 4), says="workspace overlaps d_status")
    with pytest.raises(ValueError, match="workspace"):
        fc.gated_ffn_backward(torch.zeros(256, 64), None, None, None, None, torch.zeros(256, 4096),
                              fc.alloc_gated_ffn_workspace(256, 4096, "cpu"), factor_terms=2)


def test_binding_checks_shapes_and_types():
    """The binding's own checks come before any pointer is taken."""
    with pytest.raises(ValueError, match="multiple of 16"):
        fc.alloc_fp8(4, 40, device="cpu")
    with pytest.raises(ValueError, match="block_rows"):
        fc.alloc_fp8(4, 64, 2, device="cpu")
    q = fc.alloc_fp8(4, 144, device="cpu")
    assert q[0].shape == (4, 144) and q[1].shape == (4, 2) and fc._block_rows(q, 4) == 1
    w = fc.alloc_fp8(130, 144, 128, device="cpu")
    assert w[1].shape == (2, 2) and fc._block_rows(w, 130) == 128
    with pytest.raises(ValueError, match="CUDA"):
        fc.fp8_quantize(torch.zeros(4, 144), q)
    with pytest.raises(ValueError, match="codes"):
        fc._fp8(q, 4, 128, 1, "q")
    with pytest.raises(ValueError, match="scales"):
        fc._fp8((q[0], q[1].double()), 4, 144, 1, "q")
    with pytest.raises(ValueError, match="scales"):
        fc._fp8((q[0], q[1][:3]), 4, 144, 1, "q")
    with pytest.raises(ValueError, match="scales"):
        fc._fp8(w, 130, 144, 1, "x")
    with pytest.raises(ValueError, match="x must be"):
        fc.gated_ffn(torch.zeros(4, 64), None, None, torch.zeros(4, 32))
    with pytest.raises(ValueError, match="workspace"):
        fc.gated_ffn_backward(torch.zeros(4, 64), None, None, None, None, torch.zeros(4, 32),
                              torch.zeros(8, dtype=torch.uint8))
