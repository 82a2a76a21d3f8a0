"""GPU tests of the block norms, their gradient, microscaled 4-bit quantisation
and the product, against plain references in 64 bits.

Tolerances (u = 2^-24, half a step of binary32; a bf16 result adds 2^-8 of its
value, an fp32 one u):
* a row's sum of squares: a thread adds 16 terms in sequence, then 5 + 5 steps of
  a tree, each within u of a sum of positive terms: 26 u at most; its root halves
  that, and the mean, the added eps, the root and the products add a few u: a
  normed value is within 32 u.
* h = alpha r + beta g u: 32 u of |beta g u| and 4 u of |alpha r|.
* a gradient: each of its terms is a product of a few factors of at most 32 u
  each, and a row's mean of products is within 32 u of the mean of their sizes:
  128 u of the sum of the terms' sizes.  A sum over R rows adds at most u of
  the running sum for each row: (R + 128) u of the sum of the sizes.
* the product: e2m1 products and their scales are exact; each of the K additions is
  within one step (2^-23, a truncation) of the sum of the sizes: K 2^-23.
"""
import pytest
import torch

import block_ref as ref
from block_ref import HALF, U
from quantized_reduce_rmsnorm_gb300 import fcomm as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def randn(gen, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, dtype=torch.float64) * std + mean).to(dtype).cuda()


def gen_of(*key):
    return torch.Generator().manual_seed(sum((i + 1) * ord(c) for i, c in enumerate("/".join(map(str, key)))))


def within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    off = (got - want).abs()
    worst = (off / tol.clamp(min=1e-300)).max().item()
    assert (off <= tol).all(), f"{what}: {worst:.3g} of the tolerance"


# ------------------------------------------------------- quantisation ------
MX_SHAPES = [(1, 32), (1, 64), (3, 96), (5, 160), (127, 128), (128, 4096), (129, 224), (64, 8192), (333, 2080),
             (2, 65536)]


def check_mx4(x, codes, scales, fill):
    """codes and scales bit for bit, pads included, and what is not written left alone."""
    rows, hidden = x.shape
    code, byte = ref.mx4_reference(x.cpu())
    want_c, want_s = ref.pack_mx4(code, byte, fill)
    nan = byte.repeat_interleave(32, 1) == 255
    got = ref.unpack(codes.cpu())
    assert torch.equal(got[~nan], code[~nan])
    assert torch.equal(scales.cpu(), want_s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden", MX_SHAPES)
def test_mx4_quantize_bit_exact_and_reads_back(rows, hidden, dtype):
    g = gen_of("mx", rows, hidden, dtype)
    x = randn(g, rows, hidden)
    x *= torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float()).cuda()
    x[:, hidden // 2] *= 50
    x = x.to(DT[dtype])
    q = fc.alloc_mx4(rows, hidden)
    q[1].fill_(0xAB)
    fc.mx4_quantize(x, q)
    check_mx4(x, *q, 0xAB)
    code, byte = ref.mx4_reference(x.cpu())
    want = ref.mx4_values(code, byte)
    for d in DT.values():
        back = torch.empty(rows, hidden, dtype=d, device="cuda")
        fc.mx4_dequantize(q, back)
        assert torch.equal(back.cpu().double(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mx4_ties_extremes_and_non_finite_blocks(dtype):
    x = torch.zeros(40, 64, dtype=torch.float64)
    ties = torch.tensor([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 0.125, 0.375])
    for i in range(32):
        x[i, :18] = ties * 2.0 ** (i - 16)
        x[i, 18:36] = -ties * 2.0 ** (i - 16)
    x[32, :32] = 3.3e38                                  # the largest exponent
    x[33, :4] = torch.tensor([2.0 ** -126, -(2.0 ** -127), 2.0 ** -128, 2.0 ** -133])  # scale byte 0
    x[34] = -0.0
    x[35, 40] = float("nan")
    x[36, 3] = float("inf")
    x[37, 3] = -float("inf")
    x[38, 0] = float("nan")
    x[38, 1] = float("inf")
    x = x.to(DT[dtype]).cuda()
    q = fc.alloc_mx4(40, 64)
    q[1].fill_(7)
    fc.mx4_quantize(x, q)
    check_mx4(x, *q, 7)
    back = torch.empty(40, 64, dtype=torch.float32, device="cuda")
    fc.mx4_dequantize(q, back)
    bad = torch.isnan(back.cpu())
    want = torch.zeros(40, 64, dtype=torch.bool)
    want[35, 32:] = want[36, :32] = want[37, :32] = want[38, :32] = True
    assert torch.equal(bad, want)


# --------------------------------------------------------- block norms -----
FORMS = {  # post, gate, pre, residual, alpha, beta
    "pre": (False, None, True, True, 1.0, 1.0),
    "post": (True, None, False, True, 1.0, 1.0),
    "sandwich": (True, None, True, True, 0.75, 0.5),
    "gate": (False, "one", True, True, 1.0, 1.0),
    "gate-seq": (True, "seq", True, True, 1.0, 0.5),
    "gate-token": (True, "token", True, True, 0.75, 1.0),
    "gate-only": (False, "token", False, True, 1.0, -1.0),
    "no-residual": (True, "one", True, False, 1.0, 1.0),
}


def norm_inputs(rows, hidden, dtype, form):
    post, gate, pre, res, alpha, beta = FORMS[form]
    g, d = gen_of("norm", rows, hidden, dtype, form), DT[dtype]
    x = randn(g, rows, hidden)
    x[:, hidden // 3] *= 20
    seqs = next(s for s in (7, 5, 3, 2, 1) if rows % s == 0)
    gr = {None: 0, "one": 1, "seq": seqs, "token": rows}[gate]
    return dict(x=x.to(d), r=randn(g, rows, hidden, dtype=d) if res else None,
                post_weight=randn(g, hidden, dtype=d, std=0.1, mean=1.0) if post else None,
                gate=randn(g, gr, hidden, dtype=d) if gr else None,
                pre_weight=randn(g, hidden, dtype=d, std=0.1, mean=1.0) if pre else None,
                residual_scale=alpha, block_scale=beta)


def spec_of(i):
    return {k: i[k] for k in ("post_weight", "gate", "pre_weight", "residual_scale", "block_scale")}


def check_norm(i, h, y, dtype):
    want, size = ref.norm_reference(i["x"], i["r"], i["post_weight"], i["gate"], i["residual_scale"],
                                    i["block_scale"], EPS)
    within(h, want, HALF[dtype] * want.abs() + 32 * U * size, "h")
    if y is not None:
        want = ref.rms_reference(h, i["pre_weight"], EPS)
        within(y, want, (HALF[dtype] + 32 * U) * want.abs(), "y")


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("rows,hidden", [(1, 16), (1, 4096), (6, 48), (7, 512), (35, 528), (64, 8192), (129, 1040),
                                         (210, 5120), (3, 16384), (14, 8208)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_norm(rows, hidden, dtype, form):
    i = norm_inputs(rows, hidden, dtype, form)
    h = torch.full_like(i["x"], float("nan"))
    y = torch.full_like(i["x"], float("nan")) if i["pre_weight"] is not None else None
    fc.block_norm(i["x"], i["r"], h, y, **spec_of(i))
    check_norm(i, h, y, DT[dtype])


@pytest.mark.parametrize("rows,hidden", [(1, 32), (5, 160), (64, 8192), (131, 1056), (2, 16384), (9, 8224)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_norm_quantised_output_is_that_of_y(rows, hidden, dtype):
    """y_mx4 equals fc_mx4_quantize of the stored y bit for bit, with and without y."""
    i = norm_inputs(rows, hidden, dtype, "gate-seq")
    h, y, h2 = (torch.empty_like(i["x"]) for _ in range(3))
    q, q2, alone = (fc.alloc_mx4(rows, hidden) for _ in range(3))
    for t in (q, q2, alone):
        t[1].fill_(0x5A)
    fc.block_norm(i["x"], i["r"], h, y, y_mx4=q, **spec_of(i))
    fc.block_norm(i["x"], i["r"], h2, None, y_mx4=q2, **spec_of(i))
    fc.mx4_quantize(y, alone)
    check_norm(i, h, y, DT[dtype])
    assert torch.equal(h, h2)
    for t in (q, q2):
        assert torch.equal(t[0], alone[0]) and torch.equal(t[1], alone[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_norm_in_place(dtype):
    i = norm_inputs(33, 2064, dtype, "gate-seq")
    h, y = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    fc.block_norm(i["x"], i["r"], h, y, **spec_of(i))
    x, r = i["x"].clone(), i["r"].clone()
    fc.block_norm(x, r, r, x, **spec_of(i))
    assert torch.equal(r, h) and torch.equal(x, y)


def test_block_norm_rows_of_zeros_and_non_finite_rows_stay_their_own():
    """A row of zeros gives 0 (eps > 0); an infinity or a NaN spoils its own row alone."""
    i = norm_inputs(12, 1024, "bf16", "sandwich")
    h0, y0, h, y = (torch.empty_like(i["x"]) for _ in range(4))
    fc.block_norm(i["x"], i["r"], h0, y0, **spec_of(i))
    i["x"][3] = 0
    i["r"][3] = 0
    i["x"][5, 7] = float("inf")
    i["r"][8, 9] = float("nan")
    fc.block_norm(i["x"], i["r"], h, y, **spec_of(i))
    assert (h[3] == 0).all() and (y[3] == 0).all()
    keep = [k for k in range(12) if k not in (3, 5, 8)]
    assert torch.equal(h[keep], h0[keep]) and torch.equal(y[keep], y0[keep])
    assert not torch.isfinite(y[8]).any()


def test_what_the_binding_refuses():
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    h, q = torch.empty_like(x), fc.alloc_mx4(8, 64)
    with pytest.raises(ValueError, match="contiguous"):
        fc.block_norm(torch.zeros(64, 8, dtype=torch.bfloat16, device="cuda").t(), None, h)
    with pytest.raises(ValueError, match="residual_out"):
        fc.block_norm(x, None, h.float())
    with pytest.raises(ValueError, match="pre_weight"):
        fc.block_norm(x, x, h, h, pre_weight=torch.ones(63, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fc.FcommError, match="gate_rows"):
        fc.block_norm(x, x, h, gate=torch.ones(3, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fc.FcommError, match="overlaps"):
        fc.block_norm(x, x, h, h, pre_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="codes"):
        fc.mx4_quantize(x, fc.alloc_mx4(4, 128))
    with pytest.raises(ValueError, match="workspace"):
        fc.block_norm_backward(x, x, x, x, h, torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="x's codes"):
        fc.mx4_matmul(fc.alloc_mx4(8, 32), fc.alloc_mx4(16, 64), torch.empty(8, 16, device="cuda"))
    with pytest.raises(fc.FcommError, match="features"):
        fc.mx4_matmul(q, fc.alloc_mx4(8, 64), torch.empty(8, 8, device="cuda"))


# ------------------------------------------------------------ gradient -----
def grad_inputs(rows, hidden, dtype, form):
    i = norm_inputs(rows, hidden, dtype, form)
    g, d = gen_of("grad", rows, hidden, dtype, form), DT[dtype]
    i["h"] = ref.norm_reference(i["x"], i["r"], i["post_weight"], i["gate"], i["residual_scale"], i["block_scale"],
                                EPS)[0].to(d)
    i["dy"] = randn(g, rows, hidden, dtype=d) if i["pre_weight"] is not None else None
    i["dh"] = randn(g, rows, hidden, dtype=d) if i["dy"] is None or form != "gate" else None
    return i


def grad_outputs(i):
    x, f32 = i["x"], torch.float32
    hidden = x.shape[1]
    out = {"dx": torch.full_like(x, float("nan")), "dresidual": torch.full_like(x, float("nan"))}
    if i["post_weight"] is not None:
        out["dpost_weight"] = torch.full((hidden,), float("nan"), dtype=f32, device="cuda")
    if i["pre_weight"] is not None:
        out["dpre_weight"] = torch.full((hidden,), float("nan"), dtype=f32, device="cuda")
    if i["gate"] is not None:
        out["dgate"] = torch.full_like(i["gate"], float("nan"))
    return out


def run_grad(i, out, ws=None, stream=None):
    x = i["x"]
    if ws is None:
        ws = fc.alloc_block_norm_workspace(*x.shape, 0 if i["gate"] is None else i["gate"].shape[0])
    fc.block_norm_backward(x, i["h"], i["dy"], i["dh"], workspace=ws, stream=stream, **out, **spec_of(i))


def check_grad(i, out):
    rows = i["x"].shape[0]
    want = ref.grad_reference(i["x"], i["h"] if i["dy"] is not None else None, i["dy"], i["dh"], i["post_weight"],
                              i["gate"], i["pre_weight"], i["residual_scale"], i["block_scale"], EPS)
    for name, got in out.items():
        value, size = want[name]
        summed = rows if name not in ("dx", "dresidual") else 0
        within(got, value, HALF[got.dtype] * value.abs() + (summed + 128) * U * size, name)


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("rows,hidden", [(1, 16), (1, 4096), (6, 48), (35, 528), (64, 8192), (210, 1040),
                                         (1400, 2064), (5, 16384), (14, 8208)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_norm_backward(rows, hidden, dtype, form):
    i = grad_inputs(rows, hidden, dtype, form)
    out = grad_outputs(i)
    run_grad(i, out)
    check_grad(i, out)
    again = grad_outputs(i)
    run_grad(i, again)
    for k in out:
        assert torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("gate_rows", [1, 2, 75, 300, 600, 700, 2100])
def test_gradient_of_a_shared_gate(gate_rows):
    """Gates shared by many rows, by few, and by fewer than a CTA takes."""
    i = grad_inputs(4200, 272, "f32", "sandwich")
    i["gate"] = randn(gen_of("shared", gate_rows), gate_rows, 272)
    out = grad_outputs(i)
    run_grad(i, out)
    check_grad(i, out)


def test_gradient_in_place_and_without_the_optional_outputs():
    i = grad_inputs(45, 1040, "bf16", "gate-seq")
    out = grad_outputs(i)
    run_grad(i, out)
    only = {"dx": torch.empty_like(i["x"])}
    run_grad(i, only)
    assert torch.equal(only["dx"], out["dx"])
    run_grad(i, {"dx": i["dy"], "dresidual": i["dh"]})
    assert torch.equal(i["dy"], out["dx"]) and torch.equal(i["dh"], out["dresidual"])


def test_gradient_matches_differences():
    """d/ds of sum(y * dy + h * dh) along a random direction of every input, by
    central differences of the 64-bit forward pass, against the kernel's gradients."""
    i = grad_inputs(14, 528, "f32", "gate-seq")
    h, _ = ref.norm_reference(i["x"], i["r"], i["post_weight"], i["gate"], i["residual_scale"], i["block_scale"], EPS)
    out = grad_outputs(i)
    run_grad(i, out)
    names = {"x": "dx", "r": "dresidual", "post_weight": "dpost_weight", "gate": "dgate", "pre_weight": "dpre_weight"}
    g = gen_of("differences")

    def loss(j):
        hh, _ = ref.norm_reference(j["x"], j["r"], j["post_weight"], j["gate"], j["residual_scale"],
                                   j["block_scale"], EPS)
        y = ref.rms_reference(hh, j["pre_weight"], EPS)
        return ((y * i["dy"].double()).sum() + (hh * i["dh"].double()).sum()).item()

    for name, grad in names.items():
        d = randn(g, *i[name].shape).double()
        step = 1e-5
        up, down = ({**i, name: i[name].double() + s * step * d} for s in (1, -1))
        want = (loss(up) - loss(down)) / (2 * step)
        got = (out[grad].double() * d).sum().item()
        size = (out[grad].double() * d).abs().sum().item()
        # third-order remainder of the difference (1e-10 times the third derivative) and the
        # gradient's own error, with the forward pass's h rounded to fp32: 1e-5 of the terms' size
        assert abs(got - want) <= 1e-5 * size, (name, got, want, size)


def test_gradient_of_rows_of_zeros_with_a_small_eps():
    """x = h = 0: xh = hh = 0 and inv = eps^-1/2, so dh' = dh + inv dy pre_weight and dx = inv beta post_weight dh';
    inv^3 = 1e45 is past binary32."""
    rows, hidden, eps = 3, 1040, 1e-30
    g = gen_of("zeros")
    x = torch.zeros(rows, hidden, device="cuda")
    dy, dh = randn(g, rows, hidden, std=1e-15), randn(g, rows, hidden)
    w1, w2 = randn(g, hidden, mean=1.0, std=0.1), randn(g, hidden, mean=1.0, std=0.1)
    dx, dr = torch.empty_like(x), torch.empty_like(x)
    fc.block_norm_backward(x, x, dy, dh, dx, fc.alloc_block_norm_workspace(rows, hidden), dresidual=dr,
                           post_weight=w1, pre_weight=w2, post_eps=eps, pre_eps=eps)
    inv = float(torch.tensor(eps, dtype=torch.float32)) ** -0.5
    d, size = dh.double() + inv * dy.double() * w2.double(), dh.double().abs() + inv * (dy.double() * w2.double()).abs()
    within(dr, d, 128 * U * size, "dresidual")
    within(dx, inv * w1.double() * d, 128 * U * inv * w1.double().abs() * size, "dx")


def test_gradient_of_no_rows_is_zero():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((64,), float("nan"), device="cuda")
    dg = torch.full((2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    fc.block_norm_backward(x, x, x, x, torch.empty_like(x), fc.alloc_block_norm_workspace(0, 64),
                           dpre_weight=dw, dgate=dg, pre_weight=w, gate=torch.ones_like(dg))
    assert (dw == 0).all() and (dg == 0).all()


# ------------------------------------------------------------- product -----
def mx4_random(g, rows, hidden, scales=(127, 128)):
    code = torch.randint(0, 16, (rows, hidden), generator=g)
    byte = torch.randint(*scales, (rows, hidden // 32), generator=g)
    codes, sc = ref.pack_mx4(code, byte, fill=0xFF)  # the rows behind the last hold NaN scales
    return (codes.cuda(), sc.cuda()), ref.mx4_values(code, byte)


SHAPES = [(1, 16, 32), (1, 128, 64), (2, 144, 96), (3, 256, 128), (16, 128, 160), (17, 272, 224), (31, 128, 256),
          (33, 400, 288), (64, 512, 1024), (65, 128, 512), (127, 144, 320), (129, 272, 2080), (200, 1040, 544),
          (256, 256, 4096), (257, 400, 352), (300, 2064, 1056), (513, 640, 8192), (1, 8192, 4096), (64, 4096, 8192),
          (3, 32, 65536), (5000, 16, 64), (130, 48, 8192), (1, 16, 16384)]


@pytest.mark.parametrize("rows,features,hidden", SHAPES)
def test_product_of_small_numbers_is_exact(rows, features, hidden):
    """With all scales 1 every partial sum is a multiple of 0.25 below 36 * 8192: exact
    in binary32 in any order, so the fp32 output equals the sum and bf16 is its rounding."""
    g = gen_of("exact", rows, features, hidden)
    x, xv = mx4_random(g, rows, hidden)
    w, wv = mx4_random(g, features, hidden)
    want = xv @ wv.T
    status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    for d in (torch.float32, torch.bfloat16):
        out = torch.full((rows, features), float("nan"), dtype=d, device="cuda")
        fc.mx4_matmul(x, w, out, d_status=status)
        assert status.tolist() == [0, fc.STATUS_NO_INDEX]
        assert torch.equal(out.cpu(), want.to(d))


@pytest.mark.parametrize("rows,features,hidden", SHAPES)
def test_product_with_scales(rows, features, hidden):
    g = gen_of("scales", rows, features, hidden)
    x, xv = mx4_random(g, rows, hidden, (117, 137))
    w, wv = mx4_random(g, features, hidden, (112, 133))
    want, size = xv @ wv.T, xv.abs() @ wv.abs().T
    out = torch.full((rows, features), float("nan"), device="cuda")
    fc.mx4_matmul(x, w, out)
    within(out.cpu(), want, hidden * 2.0 ** -23 * size, "out")


@pytest.mark.parametrize("rows", [5, 200])
@pytest.mark.parametrize("ex,ew", [(-120, 110), (120, -110), (100, 20), (-127, 127), (-60, -60)])
def test_product_with_far_scales(rows, ex, ew):
    """The blocks' scales multiply exactly over their whole range.  Every partial sum,
    in any order, is at most the sum of the terms' sizes: where that is below
    binary32's largest number nothing overflows, and the result is exact; at 2^120
    it reaches 160 * 36 * 2^120 = 7.7e39, past 3.4e38, and there a sum on the way may
    overflow although the last one does not."""
    g = gen_of("far scales", rows, ex, ew)
    x, xv = mx4_random(g, rows, 160, (127 + ex, 128 + ex))
    w, wv = mx4_random(g, 272, 160, (127 + ew, 128 + ew))
    out = torch.empty(rows, 272, device="cuda")
    fc.mx4_matmul(x, w, out)
    safe = xv.abs() @ wv.abs().T < torch.finfo(torch.float32).max
    assert safe.all() or ex + ew == 120
    out, want = out.cpu(), (xv @ wv.T).float()
    assert ((out == want) | (~safe & ~torch.isfinite(out))).all()


def test_product_leaves_what_is_behind_the_output_alone():
    g = gen_of("behind")
    x, xv = mx4_random(g, 35, 288)
    w, wv = mx4_random(g, 144, 288)
    buf = torch.full((64 * 144,), 7.0, dtype=torch.bfloat16, device="cuda")
    fc.mx4_matmul(x, w, buf[16 * 144:51 * 144].view(35, 144))
    got = buf.cpu().view(64, 144)
    assert (got[:16] == 7).all() and (got[51:] == 7).all()
    assert torch.equal(got[16:51], (xv @ wv.T).bfloat16())


def test_nan_scales_spoil_their_own_rows_and_columns():
    g = gen_of("nan")
    x, xv = mx4_random(g, 40, 512)
    w, wv = mx4_random(g, 256, 512)
    x[1][ref.scale_offsets(40, 512)[7, 3]] = 255
    w[1][ref.scale_offsets(256, 512)[130, 15]] = 255
    out = torch.empty(40, 256, device="cuda")
    fc.mx4_matmul(x, w, out)
    bad = torch.zeros(40, 256, dtype=torch.bool)
    bad[7] = bad[:, 130] = True
    out = out.cpu()
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad].double(), (xv @ wv.T)[~bad])


@pytest.mark.parametrize("rows,features,hidden", [(2100, 4368, 288), (1100, 9232, 1568), (4099, 1552, 96)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product_over_many_tiles(rows, features, hidden, dtype):
    """More tiles than the GPU holds at once, the last of them ragged; exact as above."""
    g = gen_of("tiles", rows, features, hidden)
    x, xv = mx4_random(g, rows, hidden)
    w, wv = mx4_random(g, features, hidden)
    out = torch.full((rows, features), float("nan"), dtype=DT[dtype], device="cuda")
    fc.mx4_matmul(x, w, out)
    assert torch.equal(out, (xv.cuda() @ wv.cuda().T).to(DT[dtype]))


# ------------------------------------------ sizes that take other kernels --
@pytest.mark.parametrize("rows,hidden", [(1300, 1040), (700, 8192)])
def test_block_norm_of_many_rows(rows, hidden):
    i = norm_inputs(rows, hidden, "bf16", "gate-seq")
    h, y = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    fc.block_norm(i["x"], i["r"], h, y, **spec_of(i))
    check_norm(i, h, y, torch.bfloat16)


@pytest.mark.parametrize("form", ["sandwich", "gate-seq", "gate-token", "pre", "post"])
@pytest.mark.parametrize("rows,hidden,dtype", [(1260, 3600, "bf16"), (330, 6160, "bf16"), (315, 5136, "f32"),
                                               (40, 12304, "bf16"), (20, 12304, "f32"), (700, 2576, "f32")])
def test_gradient_of_every_plan(rows, hidden, dtype, form):
    i = grad_inputs(rows, hidden, dtype, form)
    out = grad_outputs(i)
    status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    ws = fc.alloc_block_norm_workspace(rows, hidden, 0 if i["gate"] is None else i["gate"].shape[0])
    fc.block_norm_backward(i["x"], i["h"], i["dy"], i["dh"], workspace=ws, d_status=status, **out, **spec_of(i))
    check_grad(i, out)
    assert status.tolist() == [0, fc.STATUS_NO_INDEX]


# ------------------------------------------------- offsets past 32 bits ----
def test_rows_past_the_32_bit_offsets():
    """More than 2^32 elements: the first and the last rows as when they are alone."""
    rows, hidden, k = 66000, 65536, 3
    x = torch.randn(rows, hidden, device="cuda", dtype=torch.bfloat16)
    q = fc.alloc_mx4(rows, hidden)
    fc.mx4_quantize(x, q)
    for r in (slice(0, k), slice(rows - k, rows)):
        code, byte = ref.mx4_reference(x[r].cpu())
        assert torch.equal(ref.unpack(q[0][r].cpu()), code)
        off = ref.scale_offsets(rows, hidden)[r].cuda()
        assert torch.equal(q[1][off.flatten()].cpu().long(), byte.flatten())
    want = x[rows - k:].clone()
    fc.mx4_dequantize(q, x)
    assert torch.equal(x[rows - k:].cpu().double(), ref.mx4_values(*ref.mx4_reference(want.cpu())))


def test_norm_and_gradient_past_the_32_bit_offsets():
    rows, hidden, k = 530000, 8192, 5
    w = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(rows, hidden, device="cuda", dtype=torch.bfloat16)
    h, y = torch.empty_like(x), torch.empty_like(x)
    fc.block_norm(x, x, h, y, post_weight=w, pre_weight=w)
    small = x[rows - k:].contiguous()
    h2, y2 = torch.empty_like(small), torch.empty_like(small)
    fc.block_norm(small, small, h2, y2, post_weight=w, pre_weight=w)
    assert torch.equal(h[rows - k:], h2) and torch.equal(y[rows - k:], y2)
    dx, dx2 = torch.empty_like(x), torch.empty_like(small)
    dw = torch.empty(hidden, device="cuda")
    for a, b, c, n in ((x, h, dx, rows), (small, h2, dx2, k)):
        fc.block_norm_backward(a, b, a, b, c, fc.alloc_block_norm_workspace(n, hidden), dpost_weight=dw,
                               post_weight=w, pre_weight=w)
    assert torch.equal(dx[rows - k:], dx2)


@pytest.mark.parametrize("rows,features", [(140000, 16384), (100, 4190000)])
def test_product_past_the_32_bit_offsets(rows, features):
    hidden = 64
    x, xv = mx4_random(gen_of("far", rows), rows, hidden)
    w, wv = mx4_random(gen_of("wide", features), features, hidden)
    out = torch.empty(rows, features, dtype=torch.bfloat16 if rows > 100 else torch.float32, device="cuda")
    fc.mx4_matmul(x, w, out)
    for r, c in ((slice(0, 3), slice(0, 40)), (slice(rows - 3, rows), slice(features - 40, features))):
        assert torch.equal(out[r, c].cpu(), (xv[r] @ wv[c].T).to(out.dtype))


# ------------------------------------------------------- used together -----
def test_two_gradients_at_once():
    """Two calls on two streams, each with a workspace of its own, as one after the other."""
    jobs = []
    for k, (rows, hidden) in enumerate([(900, 2064), (700, 4096)]):
        i = grad_inputs(rows, hidden, "bf16", "gate-seq")
        want, out = grad_outputs(i), grad_outputs(i)
        run_grad(i, want)
        ws = fc.alloc_block_norm_workspace(rows, hidden, i["gate"].shape[0])
        jobs.append((i, want, out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for i, _, out, ws, st in jobs:
            run_grad(i, out, ws, st)
    torch.cuda.synchronize()
    for _, want, out, _, _ in jobs:
        for name in want:
            assert torch.equal(want[name], out[name]), name


@pytest.mark.parametrize("name", ["decode", "prefill", "token-split", "decode-qtagged"])
def test_pipeline_into_the_next_projection(name):
    """The boundary's step with a projection: h, y and the payload as without it, and
    the product of the quantised y with the quantised weight."""
    from quantized_reduce_rmsnorm_gb300 import synth
    from quantized_reduce_rmsnorm_gb300.pipeline import Pipeline
    w = synth.Workload(**{**synth.WORKLOADS[name].__dict__, "T": 48})
    inp = synth.make_inputs(w, seed=3)
    weight = randn(gen_of("projection", name), 1040, w.H, std=w.H ** -0.5, dtype=torch.bfloat16)
    plain, pipe = Pipeline(w, inp), Pipeline(w, inp, projection=weight)
    assert pipe.launches_per_step == plain.launches_per_step + 3
    assert set(pipe.alg_bytes()) == set(plain.alg_bytes()) | {"projection"}
    plain.step()
    pipe.step()
    want, got = plain.outputs(), pipe.outputs()
    for k in want:
        assert want[k] is None and got[k] is None or (want[k] == got[k]).all(), k
    assert got["projection_status"].tolist() == [0, fc.STATUS_NO_INDEX]
    xv = ref.mx4_values(*ref.mx4_reference(pipe.y.cpu()))
    wv = ref.mx4_values(*ref.mx4_reference(weight.cpu()))
    value, size = xv @ wv.T, xv.abs() @ wv.abs().T
    within(pipe.out.cpu(), value, HALF[torch.bfloat16] * value.abs() + w.H * 2.0 ** -23 * size, "out")
    if name in ("decode", "prefill"):
        pipe.capture()
        pipe.out.zero_()
        pipe.replay()
        assert (pipe.outputs()["out"] == got["out"]).all()
    with pytest.raises(ValueError, match="projection"):
        Pipeline(w, inp, projection=weight[:, :64])


def test_norm_quantise_project_streams_and_graph():
    """Norms to four bits and through a projection: launched on a side stream, and
    captured and replayed on new inputs, the same bits as one call after another."""
    rows, hidden, features = 96, 2048, 1040
    i = norm_inputs(rows, hidden, "bf16", "gate-seq")
    w, _ = mx4_random(gen_of("w"), features, hidden, (115, 122))
    h, y = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    q = fc.alloc_mx4(rows, hidden)
    out = torch.empty(rows, features, dtype=torch.bfloat16, device="cuda")
    calls = [fc.bind_block_norm(i["x"], i["r"], h, None, y_mx4=q, **spec_of(i)), fc.bind_mx4_matmul(q, w, out)]

    def plain():
        hh, yy, qq, oo = torch.empty_like(h), torch.empty_like(y), fc.alloc_mx4(rows, hidden), torch.empty_like(out)
        fc.block_norm(i["x"], i["r"], hh, yy, **spec_of(i))
        fc.mx4_quantize(yy, qq)
        torch.cuda.synchronize()
        fc.mx4_matmul(qq, w, oo)
        torch.cuda.synchronize()
        return hh, oo

    want = plain()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c in calls:
        c(side)
    side.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(out, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            c(side)
    for k in range(3):
        i["x"].mul_(1.25)
        i["r"].add_(0.5)
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = plain()
        assert torch.equal(h, want[0]) and torch.equal(out, want[1])


def test_products_on_two_streams():
    """Both kernels of the product at once, many times over: the bits of one after the other."""
    jobs = []
    for k, (rows, features, hidden) in enumerate([(700, 2064, 4096), (9, 4096, 4096), (64, 2048, 8192)]):
        g = gen_of("streams", k)
        x, _ = mx4_random(g, rows, hidden, (117, 137))
        w, _ = mx4_random(g, features, hidden, (112, 133))
        want, out = (torch.empty(rows, features, device="cuda") for _ in range(2))
        fc.mx4_matmul(x, w, want)
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        jobs.append((fc.bind_mx4_matmul(x, w, out, status), torch.cuda.Stream(), want, out, status))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, st, _, _, _ in jobs:
            call(st)
    torch.cuda.synchronize()
    for _, _, want, out, status in jobs:
        assert torch.equal(want, out) and status.tolist() == [0, fc.STATUS_NO_INDEX]


def test_training_step_captured():
    """Forward and gradient captured into one graph and replayed: the bits of the calls."""
    i = grad_inputs(150, 2064, "bf16", "gate-seq")
    h, y = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    i["h"] = h
    out, want = grad_outputs(i), grad_outputs(i)
    ws = fc.alloc_block_norm_workspace(150, 2064, i["gate"].shape[0])
    side = torch.cuda.Stream()
    fc.block_norm(i["x"], i["r"], h, y, **spec_of(i))
    run_grad(i, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fc.block_norm(i["x"], i["r"], h, y, stream=side, **spec_of(i))
        run_grad(i, out, ws, side)
    for _ in range(2):
        h.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], want[k]), k


# ------------------------------------------------------- ends of the range --
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hidden", [272, 1040, 8208])
@pytest.mark.parametrize("eps", [1e-36, 1e-39, 1e-42, 1.4e-45])
def test_gradient_of_rows_of_zeros_with_the_smallest_eps(eps, hidden, dtype):
    """As above for the smallest eps: inv = eps^-1/2 is up to 2.7e22, its square past
    binary32, and the result 0 times neither."""
    rows, d = 3, DT[dtype]
    g = gen_of("zeros", eps, hidden, dtype)
    x = torch.zeros(rows, hidden, dtype=d, device="cuda")
    dy, dh = randn(g, rows, hidden, std=1e-15, dtype=d), randn(g, rows, hidden, dtype=d)
    w1, w2 = (randn(g, hidden, mean=1.0, std=0.1, dtype=d) for _ in range(2))
    gate = randn(g, 1, hidden, dtype=d)
    dx, dr, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gate)
    dw1, dw2 = (torch.full((hidden,), float("nan"), device="cuda") for _ in range(2))
    fc.block_norm_backward(x, x, dy, dh, dx, fc.alloc_block_norm_workspace(rows, hidden, 1), dresidual=dr,
                           dpost_weight=dw1, dpre_weight=dw2, dgate=dg, post_weight=w1, gate=gate, pre_weight=w2,
                           post_eps=eps, pre_eps=eps)
    inv = float(torch.tensor(eps, dtype=torch.float32)) ** -0.5
    a = inv * dy.double() * w2.double()
    want, size = dh.double() + a, dh.double().abs() + a.abs()
    f = inv * w1.double() * gate.double()
    within(dr, want, HALF[d] * want.abs() + 128 * U * size, "dresidual")
    within(dx, f * want, HALF[d] * (f * want).abs() + 128 * U * f.abs() * size, "dx")
    assert all((t == 0).all() for t in (dw1, dw2, dg))


@pytest.mark.parametrize("hidden", [272, 1040, 8208])
@pytest.mark.parametrize("std", [3e-19, 3e-20])
def test_gradient_of_very_small_rows_without_eps(std, hidden):
    """Rows whose mean of squares nears the end of binary32, or is past its normal
    numbers (3e-20: 9e-40, held to half a step of 2^-149, 13 u of it).  That error is
    in each row's two sums of squares (6.5 u in each inverse root) and, as x h, in
    the last of the row's sums (13 u): with at most four inverse roots in a term, 40 u
    beside the 128."""
    rows = 5
    g = gen_of("small rows", std, hidden)
    i = dict(x=randn(g, rows, hidden, std=std), h=randn(g, rows, hidden, std=std), gate=randn(g, 1, hidden),
             dy=randn(g, rows, hidden, std=1e-3), dh=randn(g, rows, hidden),
             post_weight=randn(g, hidden, mean=1.0, std=0.1), pre_weight=randn(g, hidden, mean=1.0, std=0.1))
    out = grad_outputs(i)
    fc.block_norm_backward(i["x"], i["h"], i["dy"], i["dh"], workspace=fc.alloc_block_norm_workspace(rows, hidden, 1),
                           post_weight=i["post_weight"], gate=i["gate"], pre_weight=i["pre_weight"], post_eps=0.0,
                           pre_eps=0.0, **out)
    want = ref.grad_reference(i["x"], i["h"], i["dy"], i["dh"], i["post_weight"], i["gate"], i["pre_weight"], 1.0, 1.0,
                              0.0)
    for name, got in out.items():
        value, size = want[name]
        summed = rows if name not in ("dx", "dresidual") else 0
        within(got, value, U * value.abs() + (summed + 168) * U * size, name)


# ------------------------------------------- blocks of different scales ----
@pytest.mark.parametrize("rows,features,hidden", SHAPES + [(2100, 4368, 288), (1100, 9232, 1568), (700, 528, 16384)])
def test_product_with_scales_is_exact(rows, features, hidden):
    """Every block has its scale and no other's: bit for bit, in fp32 and in bf16."""
    pair, want = ref.scaled_pair(gen_of("scaled", rows, features, hidden), rows, features, hidden)
    x, w = (tuple(t.cuda() for t in ref.pack_mx4(*p, fill=0xFF)) for p in pair)
    for d in (torch.float32, torch.bfloat16):
        out = torch.full((rows, features), float("nan"), dtype=d, device="cuda")
        fc.mx4_matmul(x, w, out)
        assert torch.equal(out.cpu(), want.to(d))


@pytest.mark.parametrize("hidden", [272, 4096, 12288])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_block_scale_of_small_rows(dtype, hidden):
    """block_scale times an inverse root may be past binary32 where block_scale times the
    normed row is not: rows of zeros with the smallest eps, and rows of 1e-15 without."""
    d = DT[dtype]
    g = gen_of("large scale", dtype, hidden)
    x, r = randn(g, 4, hidden, std=1e-15, dtype=d), randn(g, 4, hidden, dtype=d)
    w, gate = randn(g, hidden, mean=1.0, std=0.1, dtype=d), randn(g, 1, hidden, dtype=d)
    h = torch.empty_like(x)
    fc.block_norm(x, r, h, post_weight=w, gate=gate, block_scale=1e25, post_eps=0.0)
    beta = float(torch.tensor(1e25))
    want, size = ref.norm_reference(x, r, w, gate, 1.0, beta, 0.0)
    within(h, want, HALF[d] * want.abs() + 32 * U * size, "h")
    for res in (r, None):
        fc.block_norm(torch.zeros_like(x), res, h, post_weight=w, gate=gate, block_scale=1e25, post_eps=1.4e-45)
        assert torch.equal(h, torch.zeros_like(h) if res is None else r)
