"""GPU tests of layer norm and its gradient, 8-bit floating point with a scale for each
block of 128 and its product, and the gated feed-forward and its gradient, against plain
references in 64 bits.

Tolerances (u = 2^-24, half a step of binary32; a bf16 result adds 2^-8 of its
value, an fp32 one u; a step of the tensor core's sum 2^-23 of the sum of the sizes):
* layer norm: a sum over a row is within 26 u of the sum of its terms' sizes (16 terms in
  sequence, then 5 + 5 steps of a tree).  The first mean is off by 26 u of the mean size
  of the values, m; the second sum's mean of distances to it by 26 u of their mean size,
  which is at most the deviation plus what the first mean is off by: with the
  distance's own rounding a normed value is off by 30 u (|n| + 1 + 26 u m inv), the
  inverse deviation by 16 u: 64 u of (|n| + 1 + 26 u m inv) in all, times the weight.
* its gradient, from the statistics given: each term is a product of a few factors, a
  row's mean of products within 32 u of the mean of their sizes: 128 u of the sum of
  the sizes.  A sum over R rows adds u of the running sum for each: (R + 128) u.
* 8-bit product: codes' products are exact; a block's sum is off by 128 steps of 2^-23,
  the two scales' product by u, its product with the sum and the addition by u for each
  of the blocks and the eight parts: (128 * 2 + blocks + 10) u of the sum of the sizes.
* gated feed-forward: K steps of 2^-23 for each projection, carried through the activation
  (ffn_ref.gated_reference); its gradient with dg and du rounded to bf16, 2^-8 of each
  of their terms, or, for up to 128 tokens or 2^19 values, to two bf16 numbers, 2^-16, then R,
  or twice the features, steps of 2^-23, for each of the one or two.
"""
import pytest
import torch

import ffn_ref as ref
from ffn_ref import HALF, U
from quantized_reduce_rmsnorm_gb300 import fcomm as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
B16 = torch.bfloat16
EPS = 1e-5
ACT = {"silu": fc.ACT_SILU, "gelu": fc.ACT_GELU_TANH}


def gen_of(*key):
    return torch.Generator().manual_seed(sum((i + 1) * ord(c) for i, c in enumerate("/".join(map(str, key)))))


def randn(gen, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, dtype=torch.float64) * std + mean).to(dtype).cuda()


def within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    off = (got - want).abs()
    worst = (off / tol.clamp(min=1e-300)).max().item()
    assert (off <= tol).all(), f"{what}: {worst:.3g} of the tolerance"


def guarded(*shape, dtype=B16):
    """A tensor to write to, and the memory behind its last row, which stays as it is."""
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + 4096,), 7, dtype=dtype, device="cuda")
    whole[:n] = 0 if dtype == torch.uint8 else float("nan")
    return whole[:n].view(*shape), whole[n:]


# ---------------------------------------------------------- layer norm -----
NORM_SHAPES = [(1, 16), (1, 4096), (3, 48), (7, 512), (35, 528), (64, 8192), (129, 1040), (2, 16384), (9, 8208),
               (300, 272), (700, 2064)]


def run_norm(x, r, w, b, stats=True, **kw):
    y = torch.empty_like(x)
    h = None if r is None else torch.empty_like(x)
    st = torch.empty(len(x), 2, device="cuda") if stats else None
    fc.layer_norm(x, y, weight=w, bias=b, residual_in=r, residual_out=h, eps=EPS, stats=st, **kw)
    return h, y, st


def check_norm(h, y, st, w, b):
    want, stats, size = ref.layer_norm_reference(h, w, b, EPS)
    within(y, want, HALF[y.dtype] * want.abs() + U * size, "y")
    if st is not None:
        h = h.double()
        dist = (h - stats[:, :1]).abs().mean(1) + 26 * U * h.abs().mean(1)
        within(st[:, 0], stats[:, 0], 2 * U * stats[:, 0].abs() + 30 * U * dist, "mean")
        # squares within 30 u, and the correction's square is far below
        within(st[:, 1], stats[:, 1], 32 * U * stats[:, 1], "inverse deviation")


@pytest.mark.parametrize("form", ["plain", "residual", "no-bias", "bare"])
@pytest.mark.parametrize("rows,hidden", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm(rows, hidden, dtype, form):
    g, d = gen_of("ln", rows, hidden, dtype, form), DT[dtype]
    x = randn(g, rows, hidden, dtype=d, mean=0.5, std=2.0)
    r = randn(g, rows, hidden, dtype=d) if form != "plain" else None
    w = randn(g, hidden, dtype=d, mean=1.0, std=0.1) if form != "bare" else None
    b = randn(g, hidden, dtype=d) if form in ("plain", "residual") else None
    h, y, st = run_norm(x, r, w, b)
    if r is not None:
        assert torch.equal(h, (x.float() + r.float()).to(d))
    check_norm(x if r is None else h, y, st, w, b)


@pytest.mark.parametrize("hidden", [272, 2064, 12288])
@pytest.mark.parametrize("mean", [300.0, 1e4])
def test_layer_norm_far_from_zero(mean, hidden):
    """A mean far above the deviation: the variance is of distances, not of a difference of sums."""
    x = randn(gen_of("far", mean, hidden), 9, hidden, mean=mean)
    _, y, st = run_norm(x, None, None, None)
    check_norm(x, y, st, None, None)


def test_layer_norm_rows_of_one_value_and_non_finite_rows_stay_their_own():
    x = randn(gen_of("rows"), 12, 1040)
    x[3] = 0.0
    x[4] = 5.0
    _, y0, st0 = run_norm(x, None, None, None)
    assert (y0[3] == 0).all() and st0[3, 0] == 0
    # the mean of equal values is off by 26 u of them at most; what is left is within that of 0
    assert y0[4].abs().max() <= 30 * U * 5 * EPS ** -0.5
    x[5, 7] = float("nan")
    x[8, 3] = float("inf")
    x[9, 1] = -float("inf")
    _, y, st = run_norm(x, None, None, None)
    keep = [k for k in range(12) if k not in (5, 8, 9)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(st[keep], st0[keep])
    assert torch.isnan(y[[5, 8, 9]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_in_place_and_nothing_behind_the_rows(dtype):
    g, d = gen_of("in place", dtype), DT[dtype]
    x, r = randn(g, 37, 1040, dtype=d), randn(g, 37, 1040, dtype=d)
    w = randn(g, 1040, dtype=d)
    h, y, _ = run_norm(x, r, w, w)
    for swap in (False, True):
        a, c = x.clone(), r.clone()
        ho, yo = (c, a) if swap else (a, c)
        fc.layer_norm(a, yo, weight=w, bias=w, residual_in=c, residual_out=ho, eps=EPS)
        assert torch.equal(ho, h) and torch.equal(yo, y)
    yg, behind = guarded(37, 1040, dtype=d)
    sg, behind_stats = guarded(37, 2, dtype=torch.float32)
    fc.layer_norm(x, yg, eps=EPS, stats=sg)
    assert (behind == 7).all() and (behind_stats == 7).all() and torch.isfinite(sg).all()


def grad_case(rows, hidden, dtype, dh=True, weight=True):
    g, d = gen_of("lng", rows, hidden, dtype), DT[dtype]
    i = dict(h=randn(g, rows, hidden, dtype=d, mean=0.3, std=1.5), dy=randn(g, rows, hidden, dtype=d),
             dh=randn(g, rows, hidden, dtype=d) if dh else None,
             weight=randn(g, hidden, dtype=d, mean=1.0, std=0.1) if weight else None)
    _, _, i["stats"] = run_norm(i["h"], None, None, None)
    return i


def norm_grad_outputs(i):
    hidden = i["h"].shape[1]
    return {"dx": torch.full_like(i["h"], float("nan")),
            "dweight": torch.full((hidden,), float("nan"), device="cuda"),
            "dbias": torch.full((hidden,), float("nan"), device="cuda")}


def run_norm_grad(i, out, ws=None, stream=None, **kw):
    fc.layer_norm_backward(i["h"], i["stats"], i["dy"], workspace=ws if ws is not None else
                           fc.alloc_layer_norm_workspace(*i["h"].shape), dh=i["dh"], weight=i["weight"], stream=stream,
                           **out, **kw)


def check_norm_grad(i, out):
    want = ref.layer_norm_grad_reference(i["h"], i["stats"], i["dy"], i["dh"], i["weight"])
    rows = len(i["h"])
    for k, (v, size) in want.items():
        if k in out:
            n = 128 if k == "dx" else rows + 128
            within(out[k], v, HALF[out[k].dtype] * v.abs() + n * U * size, k)


@pytest.mark.parametrize("dh", [True, False])
@pytest.mark.parametrize("rows,hidden", NORM_SHAPES + [(1400, 3600), (333, 6160), (210, 16384), (40, 12288), (350, 5136)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_backward(rows, hidden, dtype, dh):
    i = grad_case(rows, hidden, dtype, dh, weight=dh or hidden % 32 == 0)
    out = norm_grad_outputs(i)
    run_norm_grad(i, out)
    check_norm_grad(i, out)
    again = norm_grad_outputs(i)
    run_norm_grad(i, again)
    assert all(torch.equal(out[k], again[k]) for k in out)


def test_layer_norm_gradient_in_place_and_without_the_optional_outputs():
    i = grad_case(75, 1040, "bf16")
    out = norm_grad_outputs(i)
    run_norm_grad(i, out)
    for only in (["dx"], ["dx", "dweight"], ["dx", "dbias"]):
        got = {k: v for k, v in norm_grad_outputs(i).items() if k in only}
        run_norm_grad(i, got)
        assert all(torch.equal(got[k], out[k]) for k in only)
    for name in ("h", "dy", "dh"):
        j = {**i, name: i[name].clone()}
        run_norm_grad(j, {"dx": j[name]})
        assert torch.equal(j[name], out["dx"])
    dx, behind = guarded(75, 1040)
    run_norm_grad(i, {"dx": dx})
    assert torch.equal(dx, out["dx"]) and (behind == 7).all()


def test_layer_norm_gradient_matches_differences():
    """d/ds of sum(y * dy + h * dh) along a random direction of x, the weight and the bias,
    by central differences of the 64-bit forward pass, against the kernel's gradients
    with the kernel's own statistics."""
    i = grad_case(14, 528, "f32")
    b = randn(gen_of("bias"), 528)
    out = norm_grad_outputs(i)
    run_norm_grad(i, out)
    g = gen_of("differences")

    def loss(h, w, bias):
        y, _, _ = ref.layer_norm_reference(h, w, bias, EPS)
        return ((y * i["dy"].double()).sum() + (h.double() * i["dh"].double()).sum()).item()

    at = {"dx": i["h"].double(), "dweight": i["weight"].double(), "dbias": b.double()}
    for name in at:
        d = randn(g, *at[name].shape).double()
        step = 1e-5
        up, down = ([v + (s * step * d if k == name else 0) for k, v in at.items()] for s in (1, -1))
        want = (loss(*up) - loss(*down)) / (2 * step)
        got, size = ((out[name].double() * d).sum().item(), (out[name].double() * d).abs().sum().item())
        # the difference's third-order remainder (1e-10 of the third derivative), and the
        # gradient's and the statistics' own errors: 1e-5 of the terms' size
        assert abs(got - want) <= 1e-5 * size, (name, got, want, size)


def test_layer_norm_gradient_of_no_rows_is_zero():
    x = torch.empty(0, 64, dtype=B16, device="cuda")
    dw, db = (torch.full((64,), float("nan"), device="cuda") for _ in range(2))
    st = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    fc.layer_norm_backward(x, torch.empty(0, 2, device="cuda"), x, torch.empty_like(x),
                           fc.alloc_layer_norm_workspace(0, 64), dweight=dw, dbias=db, d_status=st)
    assert (dw == 0).all() and (db == 0).all() and st.tolist() == [0, fc.STATUS_NO_INDEX]


# ------------------------------------------------- 8-bit floating point ----
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,hidden", [(1, 16), (1, 128), (3, 144), (5, 272), (127, 128), (128, 4096), (129, 1040),
                                         (300, 2064), (2, 65536)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fp8_quantize_bit_exact_and_reads_back(rows, hidden, dtype, block_rows):
    g = gen_of("fp8", rows, hidden, dtype)
    x = randn(g, rows, hidden)
    x *= torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float()).cuda()
    x[:, hidden // 2] *= 50
    x = x.to(DT[dtype])
    codes, behind = guarded(rows, hidden, dtype=torch.uint8)
    scales, behind_scales = guarded(*fc.alloc_fp8(rows, hidden, block_rows)[1].shape, dtype=torch.float32)
    fc.fp8_quantize(x, (codes, scales))
    want_c, want_s = ref.quantise(x.cpu(), block_rows)
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)
    assert (behind == 7).all() and (behind_scales == 7).all()
    want = ref.values(want_c) * (ref.spread(want_s, rows, hidden) if rows > 1 else
                                 want_s.double().repeat_interleave(128, 1)[:, :hidden])
    for d in DT.values():
        back, behind = guarded(rows, hidden, dtype=d)
        fc.fp8_dequantize((codes, scales), back)
        assert torch.equal(back.cpu(), want.float().to(d))  # one rounding to binary32, one to the type
        assert (behind == 7).all()


def test_fp8_many_rows():
    """Three turns a lane, and a last CTA that is not full."""
    x = randn(gen_of("many"), 800, 8016, dtype=B16)
    q = fc.alloc_fp8(800, 8016)
    fc.fp8_quantize(x, q)
    want = ref.quantise(x[790:].cpu(), 1)
    assert torch.equal(q[0][790:].cpu(), want[0]) and torch.equal(q[1][790:].cpu(), want[1])
    s = q[1].repeat_interleave(128, 1)[:, :8016]
    assert torch.equal((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), q[0])
    back = torch.empty_like(x)
    fc.fp8_dequantize(q, back)
    assert torch.equal(back, (q[0].view(torch.float8_e4m3fn).float() * s).to(B16))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fp8_ties_extremes_and_non_finite_blocks(dtype, block_rows):
    grid = ref.grid()
    ties = torch.cat([(grid[:-1] + grid[1:]) / 2, grid])[:252]
    x = torch.zeros(40 * block_rows, 384, dtype=torch.float64)
    at = torch.arange(40) * block_rows
    for i in range(30):  # scale exactly 2^(i - 15): the largest is 448 of it
        x[at[i], :252] = torch.where(torch.arange(252) % 3 == 0, -1.0, 1.0) * ties * 2.0 ** (i - 15)
        x[at[i], [0, 128]] = 448.0 * 2.0 ** (i - 15)
    x[at[30], :128] = 3.3e38                              # near the largest
    x[at[31], :3] = torch.tensor([2.0 ** -70, -(2.0 ** -64), 2.0 ** -55])  # below the least scale's range
    x[at[32]] = -0.0
    for i, v in ((33, float("nan")), (34, float("inf")), (35, -float("inf"))):
        x[at[i], 200] = v
    # quotients next to ties: a scale with every bit in use, values about its multiples
    x[at[36], :252] = ties * (1.0 + 3 * 2.0 ** -7)
    x[at[37], :252] = ties * (2.0 ** -9 / 7)
    x = x.to(DT[dtype])
    q = fc.alloc_fp8(len(x), 384, block_rows)
    fc.fp8_quantize(x.cuda(), q)
    want_c, want_s = ref.quantise(x, block_rows)
    bad = torch.isnan(want_s)
    assert bad.sum() == 3 and torch.equal(torch.isnan(q[1].cpu()), bad)
    assert torch.equal(q[1].cpu()[~bad], want_s[~bad])
    keep = ~torch.isnan(ref.spread(want_s, len(x), 384))
    assert torch.equal(q[0].cpu()[keep], want_c[keep])
    back = torch.empty(len(x), 384, device="cuda")
    fc.fp8_dequantize(q, back)
    assert torch.equal(torch.isnan(back.cpu()), ~keep)


FP8_SHAPES = [(1, 16, 16), (1, 144, 128), (3, 528, 400), (16, 128, 4096), (17, 272, 144), (40, 4112, 2064),
              (64, 512, 8192), (100, 272, 1040), (128, 128, 128), (129, 144, 272), (257, 1040, 528), (300, 8192, 256),
              (777, 528, 1168), (2100, 4368, 288)]


@pytest.mark.parametrize("rows,features,hidden", FP8_SHAPES)
def test_fp8_product_is_exact(rows, features, hidden):
    """Sums that binary32 holds exactly in any order: bit for bit, in both output types."""
    (x, w), want = ref.exact_pair(gen_of("exact", rows, features, hidden), rows, features, hidden)
    x, w = (tuple(t.cuda() for t in q) for q in (x, w))
    for d in DT.values():
        out, behind = guarded(rows, features, dtype=d)
        st = torch.full((2,), 9, dtype=torch.int32, device="cuda")
        fc.fp8_matmul(x, w, out, d_status=st)
        assert torch.equal(out.cpu(), want.float().to(d))
        assert (behind == 7).all() and st.tolist() == [0, fc.STATUS_NO_INDEX]


@pytest.mark.parametrize("rows,features,hidden", FP8_SHAPES)
def test_fp8_product_of_quantised_tensors(rows, features, hidden):
    g = gen_of("product", rows, features, hidden)
    q, w = fc.alloc_fp8(rows, hidden), fc.alloc_fp8(features, hidden, 128)
    xs = randn(g, rows, hidden) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float()).cuda()
    xs[:, ::5] *= 8
    fc.fp8_quantize(xs, q)
    fc.fp8_quantize(randn(g, features, hidden, std=0.02), w)
    xv = ref.values(q[0]) * q[1].double().repeat_interleave(128, 1)[:, :hidden]
    wv = ref.values(w[0]) * w[1].double().repeat_interleave(128, 0)[:features].repeat_interleave(128, 1)[:, :hidden]
    want, size = xv @ wv.T, xv.abs() @ wv.abs().T
    for d in DT.values():
        out = torch.empty(rows, features, dtype=d, device="cuda")
        fc.fp8_matmul(q, w, out)
        within(out, want, HALF[d] * want.abs() + (256 + -(-hidden // 128) + 10) * U * size, d)


@pytest.mark.parametrize("rows", [5, 200])
def test_fp8_nan_scales_spoil_their_own_rows_and_columns(rows):
    (x, w), want = ref.exact_pair(gen_of("nan", rows), rows, 400, 272)
    x[1][3, 1] = float("nan")
    w[1][1, 0] = float("nan")
    out = torch.empty(rows, 400, device="cuda")
    fc.fp8_matmul(tuple(t.cuda() for t in x), tuple(t.cuda() for t in w), out)
    bad = torch.zeros(rows, 400, dtype=torch.bool)
    bad[3] = True
    bad[:, 128:256] = True
    assert torch.equal(torch.isnan(out.cpu()), bad)
    assert torch.equal(out.cpu()[~bad], want.float()[~bad])


@pytest.mark.parametrize("rows", [4, 300])
def test_fp8_product_with_far_scales(rows):
    """Scales of one operand far up, the other's far down: their product is what counts."""
    (x, w), want = ref.exact_pair(gen_of("far", rows), rows, 272, 400)
    for e in (60, 100, -60):
        out = torch.empty(rows, 272, device="cuda")
        fc.fp8_matmul((x[0].cuda(), (x[1] * 2.0 ** e).cuda()), (w[0].cuda(), (w[1] * 2.0 ** -e).cuda()), out)
        assert torch.equal(out.cpu(), want.float())


# --------------------------------------------------- gated feed-forward ----
FFN_SHAPES = [(1, 16, 16), (1, 144, 64), (3, 528, 400), (16, 128, 4096), (17, 272, 144), (40, 4112, 2064),
              (64, 512, 8192), (100, 272, 1040), (128, 128, 128), (129, 144, 272), (257, 1040, 528), (300, 4112, 256),
              (777, 528, 1168), (1300, 2576, 80)]
# the gradient with k in parts, and next to where it is not
FEW_SHAPES = [(16, 1040, 272), (30, 528, 1040), (33, 80, 8208), (65, 4112, 144), (128, 1040, 528), (127, 2064, 16),
              (128, 496, 272), (129, 4112, 144), (300, 1040, 528), (161, 3216, 272)]


def ffn_case(g, rows, features, hidden):
    return (randn(g, rows, hidden, dtype=B16), randn(g, features, hidden, dtype=B16, std=hidden ** -0.5),
            randn(g, features, hidden, dtype=B16, std=hidden ** -0.5))


@pytest.mark.parametrize("name", list(ACT))
@pytest.mark.parametrize("rows,features,hidden", FFN_SHAPES)
def test_gated_ffn(rows, features, hidden, name):
    x, wg, wu = ffn_case(gen_of("ffn", rows, features, hidden), rows, features, hidden)
    out, behind = guarded(rows, features)
    fc.gated_ffn(x, wg, wu, out, activation=ACT[name])
    want, tol, g, u, eg, eu = ref.gated_reference(x, wg, wu, name)
    half = HALF[B16]
    within(out, want, half * want.abs() + tol, "out")
    assert (behind == 7).all()
    again, gate, up = (guarded(rows, features) for _ in range(3))
    st = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    fc.gated_ffn(x, wg, wu, again[0], activation=ACT[name], gate=gate[0], up=up[0], d_status=st)
    assert torch.equal(again[0], out) and st.tolist() == [0, fc.STATUS_NO_INDEX]
    within(gate[0], g, half * g.abs() + eg, "gate")
    within(up[0], u, half * u.abs() + eu, "up")
    assert all((t[1] == 7).all() for t in (again, gate, up))


def small_ints(g, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=g).to(B16).cuda()


@pytest.mark.parametrize("rows,features,hidden", FFN_SHAPES)
def test_gated_ffn_projections_are_exact(rows, features, hidden):
    """Projections of small whole numbers, bit for bit: every element of k in its place."""
    g = gen_of("ints", rows, features, hidden)
    x, wg, wu = (small_ints(g, *s) for s in ((rows, hidden), (features, hidden), (features, hidden)))
    out, gate, up = (torch.empty(rows, features, dtype=B16, device="cuda") for _ in range(3))
    fc.gated_ffn(x, wg, wu, out, gate=gate, up=up)
    assert torch.equal(gate, (x.double() @ wg.double().T).to(B16))
    assert torch.equal(up, (x.double() @ wu.double().T).to(B16))


@pytest.mark.parametrize("name", list(ACT))
@pytest.mark.parametrize("rows", [3, 140])
def test_gated_ffn_of_far_projections(rows, name):
    """Projections from far below the activation's range to far above, an infinity and a NaN."""
    hidden, features = 64, 208
    x = torch.zeros(rows, hidden, dtype=B16, device="cuda")
    x[:, 0] = 1
    wg, wu = (torch.zeros(features, hidden, dtype=B16, device="cuda") for _ in range(2))
    z = torch.cat([torch.linspace(-104, 104, 105), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 200, -200, 3e4, -3e4]),
                   torch.linspace(-8, 8, 95)]).to(B16)
    assert len(z) == features
    wg[:, 0], wu[:, 0] = z.cuda(), torch.linspace(-2, 2, features).to(B16).cuda()
    out = torch.empty(rows, features, dtype=B16, device="cuda")
    fc.gated_ffn(x, wg, wu, out, activation=ACT[name])
    want, tol, *_ = ref.gated_reference(x, wg, wu, name)
    within(out, want, HALF[B16] * want.abs() + tol, "out")
    x[1, 0] = float("nan")
    x[2, 0] = float("inf")
    again = torch.empty_like(out)
    fc.gated_ffn(x, wg, wu, again, activation=ACT[name])
    assert torch.equal(again[3:], out[3:]) and torch.equal(again[0], out[0])
    assert torch.isnan(again[1]).all() and not torch.isfinite(again[2]).any()


def ffn_grad_case(g, rows, features, hidden):
    x, wg, wu = ffn_case(g, rows, features, hidden)
    return dict(x=x, w_gate=wg, w_up=wu, gate=randn(g, rows, features, dtype=B16, std=2.0),
                up=randn(g, rows, features, dtype=B16), dout=randn(g, rows, features, dtype=B16))


def ffn_grad_outputs(i):
    return {"dx": torch.full_like(i["x"], float("nan")), "dw_gate": torch.full_like(i["w_gate"], float("nan")),
            "dw_up": torch.full_like(i["w_up"], float("nan"))}


def run_ffn_grad(i, out, name="silu", ws=None, stream=None, **kw):
    fc.gated_ffn_backward(i["x"], i["w_gate"], i["w_up"], i["gate"], i["up"], i["dout"],
                          ws if ws is not None else fc.alloc_gated_ffn_workspace(*i["gate"].shape), stream=stream,
                          activation=ACT[name], **out, **kw)


@pytest.mark.parametrize("name", list(ACT))
@pytest.mark.parametrize("rows,features,hidden", FFN_SHAPES + FEW_SHAPES)
def test_gated_ffn_backward(rows, features, hidden, name):
    i = ffn_grad_case(gen_of("ffng", rows, features, hidden, name), rows, features, hidden)
    out = ffn_grad_outputs(i)
    st = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    run_ffn_grad(i, out, name, d_status=st)
    assert st.tolist() == [0, fc.STATUS_NO_INDEX]
    want = ref.gated_grad_reference(*i.values(), name)
    for k, (v, tol) in want.items():
        within(out[k], v, HALF[B16] * v.abs() + tol, k)
    again = ffn_grad_outputs(i)
    run_ffn_grad(i, again, name)
    assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("z", [0.0, 64.0])
@pytest.mark.parametrize("rows,features,hidden", FFN_SHAPES + FEW_SHAPES)
def test_gated_ffn_gradient_is_exact(rows, features, hidden, z):
    """Where the gate's projection is 0, SiLU is 0 and its slope 1/2; where it is 64, SiLU is 64
    and its slope 1 (in binary32).  With small whole numbers the gradients are exact."""
    g = gen_of("exact", rows, features, hidden, z)
    i = dict(x=small_ints(g, rows, hidden), w_gate=small_ints(g, features, hidden), w_up=small_ints(g, features, hidden),
             gate=torch.full((rows, features), z, dtype=B16, device="cuda"), up=small_ints(g, rows, features),
             dout=2 * small_ints(g, rows, features, most=2))
    out = {k: guarded(*v.shape) for k, v in ffn_grad_outputs(i).items()}
    run_ffn_grad(i, {k: v[0] for k, v in out.items()})
    d, u = i["dout"].double(), i["up"].double()
    dg, du = (d * u / 2, 0 * d) if z == 0 else (d * u, 64 * d)
    x, wg, wu = (i[k].double() for k in ("x", "w_gate", "w_up"))
    want = {"dx": dg @ wg + du @ wu, "dw_gate": dg.T @ x, "dw_up": du.T @ x}
    for k in want:
        assert want[k].abs().max() < 2 ** 24 and torch.equal(out[k][0], want[k].float().to(B16)), k
        assert (out[k][1] == 7).all(), k


@pytest.mark.parametrize("rows,features,hidden", [s for s in FFN_SHAPES + FEW_SHAPES if s[0] <= 128 or s[0] * s[1] <= 1 << 19])
def test_gated_ffn_gradient_of_two_term_factors_is_exact(rows, features, hidden):
    """Factors that need both of their bf16 numbers, for few tokens or few factors: bit for bit."""
    i, dg, du = ref.two_term_case(gen_of("two terms", rows, features, hidden), rows, features, hidden, "cuda")
    want, out = ref.gradients(i, dg, du), {k: guarded(*v.shape) for k, v in ffn_grad_outputs(i).items()}
    run_ffn_grad(i, {k: v[0] for k, v in out.items()})
    for k in want:
        assert torch.equal(out[k][0], want[k]) and (out[k][1] == 7).all(), k
    dx = {"dx": torch.full_like(i["x"], float("nan"))}
    run_ffn_grad(i, dx)
    assert torch.equal(dx["dx"], want["dx"])


# above 128 tokens and 2^19 factors: with k of dx in parts, and with every product in one launch
@pytest.mark.parametrize("rows,features,hidden", [(129, 4112, 144), (300, 4112, 256), (140, 4112, 1040), (1300, 2576, 80),
                                                  (777, 1040, 1168), (64, 528, 400)])
def test_gated_ffn_gradient_of_two_terms_asked_for_is_exact(rows, features, hidden):
    """factor_terms=2 at every size: factors that need both of their bf16 numbers, bit for bit;
    with the terms by size the results are off."""
    i, dg, du = ref.two_term_case(gen_of("asked", rows, features, hidden), rows, features, hidden, "cuda")
    want, out = ref.gradients(i, dg, du), {k: guarded(*v.shape) for k, v in ffn_grad_outputs(i).items()}
    ws, behind = guarded(fc.load().fc_gated_ffn_backward_ex_workspace(rows, features, 2), dtype=torch.uint8)
    st = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    run_ffn_grad(i, {k: v[0] for k, v in out.items()}, ws=ws, factor_terms=2, d_status=st)
    assert st.tolist() == [0, fc.STATUS_NO_INDEX] and (behind == 7).all()
    for k in want:
        assert torch.equal(out[k][0], want[k]) and (out[k][1] == 7).all(), k
    by_size = ffn_grad_outputs(i)
    run_ffn_grad(i, by_size)
    assert all(torch.equal(by_size[k], want[k]) == (rows == 64) for k in want)


def rms(v):
    return v.square().mean().sqrt().item()


@pytest.mark.parametrize("rows,features,hidden", [(300, 4112, 256), (777, 2064, 1040), (2100, 1040, 528)])
def test_gated_ffn_gradient_error_beside_its_rounding(rows, features, hidden):
    """The root mean square of the results' distance to the 64-bit ones, in that of their own
    rounding.  Two terms: a factor is off by 2^-16, and sums by a few 2^-23 of their terms'
    sizes: 1.02.  One term: the factors' errors are independent of one another and of the
    result's, so the squares add up; with as many values at each place between two powers of
    two the two are alike, and the ratio is the root of 2.  A rounding's mean square is 1 / 12
    of a step's, a step between 2^-8 and 2^-7 of its value, so that whatever the places the
    factors' share is at most four times the result's: below the root of 5."""
    i = ffn_grad_case(gen_of("rms", rows, features, hidden), rows, features, hidden)
    want = ref.gated_grad_reference(*i.values(), "silu")
    for terms, most in ((0, 5 ** 0.5), (2, 1.02)):
        out = ffn_grad_outputs(i)
        run_ffn_grad(i, out, ws=fc.alloc_gated_ffn_workspace(rows, features, factor_terms=terms), factor_terms=terms)
        for k, (v, _) in want.items():
            ratio = rms(out[k].double() - v) / rms(v.to(B16).double() - v)
            print(f"{k}, factor_terms={terms}: {ratio:.3f} of its rounding")
            assert ratio <= most, (k, terms)


@pytest.mark.parametrize("name", list(ACT))
@pytest.mark.parametrize("rows,features", [(1, 208), (140, 4112)])
def test_gated_ffn_gradient_of_far_projections(rows, features, name):
    """Projections from the lowest number of the type to the highest: the activation and its
    slope have their limits there.  One column of x is 1, one feature's weights are 1."""
    hidden = 32
    z = torch.cat([torch.linspace(-104, 104, 105), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38, 1e19, -1e19]),
                   torch.linspace(-8, 8, 95)]).to(B16).cuda()
    i = dict(x=torch.zeros(rows, hidden, dtype=B16, device="cuda"),
             w_gate=torch.zeros(features, hidden, dtype=B16, device="cuda"),
             w_up=torch.zeros(features, hidden, dtype=B16, device="cuda"),
             gate=torch.zeros(rows, features, dtype=B16, device="cuda"),
             up=torch.full((rows, features), 0.75, dtype=B16, device="cuda"),
             dout=torch.zeros(rows, features, dtype=B16, device="cuda"))
    i["gate"][0, :208], i["dout"][0, :208] = z, 0.5
    i["x"][0, 0] = 1
    i["w_gate"][:100, 1], i["w_up"][:105, 2] = 1, 1
    out = ffn_grad_outputs(i)
    run_ffn_grad(i, out, name)
    want = ref.gated_grad_reference(*i.values(), name)
    for k, (v, tol) in want.items():
        within(out[k], v, HALF[B16] * v.abs() + tol, k)


@pytest.mark.parametrize("name", list(ACT))
@pytest.mark.parametrize("rows,features,hidden", [(16, 1040, 272), (65, 4112, 144), (161, 3216, 272), (300, 4112, 256)])
def test_gated_ffn_gradient_of_infinities_and_nans(rows, features, hidden, name):
    """An infinity or a NaN of the gate's projection, the other's or the gradient spoils the
    sums that it is in, as by the formula in 64 bits, and no others."""
    i = ffn_grad_case(gen_of("spoilt", rows, features, name), rows, features, hidden)
    clean = ffn_grad_outputs(i)
    run_ffn_grad(i, clean, name)
    inf, nan = float("inf"), float("nan")
    at = [("gate", inf), ("gate", -inf), ("gate", nan), ("up", inf), ("up", -inf), ("up", nan), ("dout", inf), ("dout", nan)]
    for k, (which, v) in enumerate(at):
        i[which][rows - 1 - k, 5 + k * (features // 8)] = v
    out = ffn_grad_outputs(i)
    run_ffn_grad(i, out, name)
    want = ref.gated_grad_reference(*i.values(), name)
    for k, (v, _) in want.items():
        spoilt = ~torch.isfinite(v)
        lines = spoilt.any(1)
        assert torch.equal(spoilt, lines[:, None].expand_as(spoilt)) and 0 < lines.sum() <= 8
        assert torch.equal(~torch.isfinite(out[k]), spoilt), (k, (torch.isfinite(out[k]) & spoilt).any(1).nonzero())
        assert torch.equal(out[k][~lines], clean[k][~lines]), k


def test_gated_ffn_gradient_without_the_optional_outputs():
    i = ffn_grad_case(gen_of("optional"), 150, 272, 400)
    out = ffn_grad_outputs(i)
    run_ffn_grad(i, out)
    for only in (["dx"], ["dw_gate", "dw_up"]):
        got = {k: v for k, v in ffn_grad_outputs(i).items() if k in only}
        run_ffn_grad(i, got)
        assert all(torch.equal(got[k], out[k]) for k in only)
    st = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    e = {k: v[:0] for k, v in i.items() if k not in ("w_gate", "w_up")}
    run_ffn_grad({**i, **e}, {"dw_gate": out["dw_gate"], "dw_up": out["dw_up"]}, ws=torch.empty(32, device="cuda"),
                 d_status=st)
    assert (out["dw_gate"] == 0).all() and (out["dw_up"] == 0).all() and st.tolist() == [0, fc.STATUS_NO_INDEX]


@pytest.mark.parametrize("name", list(ACT))
def test_gated_ffn_gradient_matches_differences(name):
    """Along a random direction of every input, by central differences of the 64-bit forward
    pass.  dg = dout u act'(z), at most G = 1.13 |dout u|, is off by 2^-8 of that for u's
    rounding to bf16, for its own, and (|z act''(z)| is below 0.6) for z's; du = dout
    act(z), at most D = |dout z|, by 2^-8 for its own and 1.13 times that for z's: 3 * 2^-8 of G
    and D.  A result's own rounding adds 2^-8."""
    g = gen_of("differences", name)
    x, wg, wu = ffn_case(g, 40, 96, 64)
    dout = randn(g, 40, 96, dtype=B16)
    out, gate, up = (torch.empty_like(dout) for _ in range(3))
    fc.gated_ffn(x, wg, wu, out, activation=ACT[name], gate=gate, up=up)
    i = dict(x=x, w_gate=wg, w_up=wu, gate=gate, up=up, dout=dout)
    got = ffn_grad_outputs(i)
    run_ffn_grad(i, got, name)
    at = {"dx": x.double(), "dw_gate": wg.double(), "dw_up": wu.double()}
    G = 1.13 * (dout.double() * (at["dx"] @ at["dw_up"].T)).abs()
    D = (dout.double() * (at["dx"] @ at["dw_gate"].T)).abs()

    def loss(*v):
        return (ref.gated_reference(*v, name)[0] * dout.double()).sum().item()

    for k in at:
        d = randn(g, *at[k].shape).double()
        up_, down = ([v + (s * 1e-5 * d if n == k else 0) for n, v in at.items()] for s in (1, -1))
        want = (loss(*up_) - loss(*down)) / 2e-5
        if k == "dx":
            size = (G * (d @ at["dw_gate"].T).abs()).sum() + (D * (d @ at["dw_up"].T).abs()).sum()
        else:
            size = ((G if k == "dw_gate" else D) * (at["dx"] @ d.T).abs()).sum()
        terms = got[k].double() * d
        tol = HALF[B16] * (3 * size + terms.abs().sum()).item() + 1e-6 * abs(want)
        assert abs(terms.sum().item() - want) <= tol, (k, terms.sum().item(), want, tol)


# ------------------------------------------------- offsets past 32 bits ----
def test_fp8_rows_past_the_32_bit_offsets():
    rows, hidden, k = 66000, 65536, 3
    x = torch.randn(rows, hidden, device="cuda", dtype=B16)
    q = fc.alloc_fp8(rows, hidden)
    fc.fp8_quantize(x, q)
    for r in (slice(0, k), slice(rows - k, rows)):
        want = ref.quantise(x[r].cpu(), 1)
        assert torch.equal(q[0][r].cpu(), want[0]) and torch.equal(q[1][r].cpu(), want[1])
    fc.fp8_dequantize(q, x)
    want = ref.values(q[0][rows - k:].cpu()) * ref.spread(q[1][rows - k:].cpu(), k, hidden)
    assert torch.equal(x[rows - k:].cpu(), want.float().to(B16))
    w = fc.alloc_fp8(rows, hidden, 128)
    fc.fp8_quantize(x, w)
    last = rows - rows % 128
    want = ref.quantise(x[last:].cpu(), 128)
    assert torch.equal(w[0][last:].cpu(), want[0]) and torch.equal(w[1][-1:].cpu(), want[1])


def test_layer_norm_past_the_32_bit_offsets():
    rows, hidden, k = 530000, 8192, 5
    w = torch.ones(hidden, device="cuda", dtype=B16)
    x = torch.randn(rows, hidden, device="cuda", dtype=B16)
    h, y, st = run_norm(x, x, w, w)
    small = x[rows - k:].contiguous()
    h2, y2, st2 = run_norm(small, small, w, w)
    assert torch.equal(h[rows - k:], h2) and torch.equal(y[rows - k:], y2) and torch.equal(st[rows - k:], st2)
    dx, dx2 = torch.empty_like(x), torch.empty_like(small)
    for a, s, c in ((h, st, dx), (h2, st2, dx2)):
        fc.layer_norm_backward(a, s, a, c, fc.alloc_layer_norm_workspace(*a.shape), dh=a, weight=w)
    assert torch.equal(dx[rows - k:], dx2)


def test_layer_norm_of_the_most_rows():
    """2^31 - 1 rows, in place: the last ones are as those of a small call."""
    rows, hidden, k = 2 ** 31 - 1, 16, 9
    x, w = torch.zeros(rows, hidden, dtype=B16, device="cuda"), randn(gen_of("w"), hidden, dtype=B16)
    st = torch.zeros(rows, 2, device="cuda")
    ends = (slice(0, k), slice(rows - k, rows))
    for r in ends:
        x[r] = randn(gen_of("most rows", r.start), k, hidden, dtype=B16)
    want = [run_norm(x[r].clone(), None, w, w) for r in ends]
    fc.layer_norm(x, x, weight=w, bias=w, eps=EPS, stats=st)
    for r, (_, y, s) in zip(ends, want):
        assert torch.equal(x[r], y) and torch.equal(st[r], s)
    assert torch.equal(x[1 << 30], w) and st[1 << 30, 0] == 0


def test_layer_norm_gradient_of_the_most_rows():
    """2^31 - 1 rows: the rows that a CTA stages ahead of its last ones would pass 2^31.  Whole
    numbers at both ends, with mean 0 and deviation 1 given: the result is exact."""
    rows, hidden, k = 2 ** 31 - 1, 16, 9
    h, dy = (torch.zeros(rows, hidden, dtype=B16, device="cuda") for _ in range(2))
    stats = torch.zeros(rows, 2, device="cuda")
    stats[:, 1] = 1
    g, ends = gen_of("most rows"), (slice(0, k), slice(rows - k, rows))
    want, dw, db = [], 0, 0
    for r in ends:
        h[r], dy[r] = small_ints(g, k, hidden), small_ints(g, k, hidden)
        n, e = h[r].double(), dy[r].double()
        want.append((e - e.mean(1, keepdim=True) - n * (e * n).mean(1, keepdim=True)).float().to(B16))
        dw, db = dw + (e * n).sum(0).float(), db + e.sum(0).float()
    got_w, got_b = (torch.full((hidden,), float("nan"), device="cuda") for _ in range(2))
    st = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    fc.layer_norm_backward(h, stats, dy, dy, fc.alloc_layer_norm_workspace(rows, hidden), dweight=got_w, dbias=got_b,
                           d_status=st)
    assert st.tolist() == [0, fc.STATUS_NO_INDEX]
    for r, v in zip(ends, want):
        assert torch.equal(dy[r], v)
    assert (dy[1 << 30:(1 << 30) + 4096] == 0).all()
    assert torch.equal(got_w, dw) and torch.equal(got_b, db)


@pytest.mark.parametrize("rows,features", [(140000, 32768), (100, 4190000)])
def test_products_past_the_32_bit_offsets(rows, features):
    (x, w), _ = ref.exact_pair(gen_of("far", rows), 64, 128, 64)
    x = tuple(t.cuda().repeat(-(-rows // 64), 1)[:rows].contiguous() for t in x)
    w = (w[0].cuda().repeat(-(-features // 128), 1)[:features].contiguous(),
         w[1].cuda().repeat(-(-features // 128), 1).contiguous())
    out = torch.empty(rows, features, dtype=B16 if rows > 100 else torch.float32, device="cuda")
    fc.fp8_matmul(x, w, out)
    ints = [t[0].view(torch.float8_e4m3fn).to(B16) for t in (x, w)]
    ends = [(slice(0, 3), slice(0, 40)), (slice(rows - 3, rows), slice(features - 40, features))]
    for r, c in ends:
        want = (x[0][r].cpu(), x[1][r].cpu()), (w[0][c].cpu(), w[1][c.start // 128:c.start // 128 + 1].cpu())
        v = ref.values(want[0][0]) * want[0][1].double()
        block = torch.arange(c.start, c.stop) // 128 - c.start // 128
        sw = w[1].cpu()[c.start // 128 + block].double()
        assert torch.equal(out[r, c].cpu(), (v @ (ref.values(want[1][0]) * sw).T).float().to(out.dtype))
    if rows > 100:
        fc.gated_ffn(ints[0], ints[1], ints[1], out)
        for r, c in ends:
            want, tol, *_ = ref.gated_reference(ints[0][r], ints[1][c], ints[1][c], "silu")
            within(out[r, c], want, HALF[B16] * want.abs() + tol, "out")


# -------------------------------------------------------- used together ----
def layer(rows, hidden, features, seed):
    """A feed-forward block between two boundaries: norm, gated projections, the way down in
    8 bits; its buffers and calls."""
    g = gen_of("layer", seed)
    s = dict(x=randn(g, rows, hidden, dtype=B16), r=randn(g, rows, hidden, dtype=B16),
             w=randn(g, hidden, dtype=B16, mean=1.0, std=0.1), b=randn(g, hidden, dtype=B16, std=0.1),
             wg=randn(g, features, hidden, dtype=B16, std=hidden ** -0.5),
             wu=randn(g, features, hidden, dtype=B16, std=hidden ** -0.5), down=fc.alloc_fp8(hidden, features, 128))
    fc.fp8_quantize(randn(g, hidden, features, std=features ** -0.5), s["down"])
    for k, shape in (("h", (rows, hidden)), ("y", (rows, hidden)), ("a", (rows, features)), ("g", (rows, features)),
                     ("u", (rows, features)), ("out", (rows, hidden))):
        s[k] = torch.empty(*shape, dtype=B16, device="cuda")
    s["stats"] = torch.empty(rows, 2, device="cuda")
    s["q"] = fc.alloc_fp8(rows, features)
    s["calls"] = [
        fc.bind_layer_norm(s["x"], s["y"], weight=s["w"], bias=s["b"], residual_in=s["r"], residual_out=s["h"],
                           stats=s["stats"]),
        fc.bind_gated_ffn(s["y"], s["wg"], s["wu"], s["a"], gate=s["g"], up=s["u"]),
        fc.bind_fp8_quantize(s["a"], s["q"]), fc.bind_fp8_matmul(s["q"], s["down"], s["out"])]
    return s


@pytest.mark.parametrize("rows", [3, 200])
def test_feed_forward_between_boundaries(rows):
    """One token batch from a boundary's output through the feed-forward to the next one's
    partial sums, which the fused boundary reduces: each step against its reference."""
    hidden, features = 512, 1040
    s = layer(rows, hidden, features, rows)
    for c in s["calls"]:
        c()
    assert torch.equal(s["h"], (s["x"].float() + s["r"].float()).to(B16))
    check_norm(s["h"], s["y"], s["stats"], s["w"], s["b"])
    want, tol, *_ = ref.gated_reference(s["y"], s["wg"], s["wu"], "silu")
    within(s["a"], want, HALF[B16] * want.abs() + tol, "a")
    codes, scales = ref.quantise(s["a"].cpu(), 1)
    assert torch.equal(s["q"][0].cpu(), codes) and torch.equal(s["q"][1].cpu(), scales)
    xv = ref.values(s["q"][0]) * ref.spread(s["q"][1], rows, features)
    wv = ref.values(s["down"][0]) * ref.spread(s["down"][1], hidden, features)
    want = xv @ wv.T
    within(s["out"], want, HALF[B16] * want.abs() + 300 * U * (xv.abs() @ wv.abs().T), "out")
    y, h = torch.empty_like(s["h"]), torch.empty_like(s["h"])
    gamma = torch.ones(hidden, dtype=B16, device="cuda")
    fc.allreduce_residual_rmsnorm([s["out"], s["x"]], fc.BF16, rows, hidden, s["h"], h, gamma, EPS, y)
    assert torch.equal(h, ((s["out"].float() + s["x"].float()) + s["h"].float()).to(B16))


@pytest.mark.parametrize("rows", [5, 300])
def test_training_step_captured_and_replayed(rows):
    """Forward and gradients of norm and feed-forward captured into one graph, replayed on new
    inputs on a side stream: the bits of the calls one after another."""
    hidden, features = 400, 528
    s = layer(rows, hidden, features, 7)
    s2 = layer(rows, hidden, features, 7)

    def back(t):
        da = t["da"] = torch.ones(rows, features, dtype=B16, device="cuda")
        t["dy"], t["dx"] = (torch.empty(rows, hidden, dtype=B16, device="cuda") for _ in range(2))
        t["dwg"], t["dwu"] = torch.empty_like(t["wg"]), torch.empty_like(t["wu"])
        t["dw"], t["db"] = (torch.empty(hidden, device="cuda") for _ in range(2))
        t["calls"] = t["calls"][:2] + [
            fc.bind_gated_ffn_backward(t["y"], t["wg"], t["wu"], t["g"], t["u"], da,
                                       fc.alloc_gated_ffn_workspace(rows, features), dx=t["dy"], dw_gate=t["dwg"],
                                       dw_up=t["dwu"]),
            fc.bind_layer_norm_backward(t["h"], t["stats"], t["dy"], t["dx"], fc.alloc_layer_norm_workspace(rows, hidden),
                                        dh=t["x"], weight=t["w"], dweight=t["dw"], dbias=t["db"])]

    back(s), back(s2)
    for c in s["calls"]:
        c()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in s["calls"]:
            c(side)
    for k in range(3):
        for t in (s, s2):
            t["x"].copy_(randn(gen_of("new", k), rows, hidden, dtype=B16))
            t["da"].copy_(randn(gen_of("grad", k), rows, features, dtype=B16))
        for name in ("dx", "dwg", "dwu", "dw", "db"):
            s[name].fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        for c in s2["calls"]:
            c()
        torch.cuda.synchronize()
        for name in ("y", "g", "u", "dy", "dx", "dwg", "dwu", "dw", "db"):
            assert torch.isfinite(s[name]).all() and torch.equal(s[name], s2[name]), name


def test_calls_on_several_streams_at_once():
    """Every kind of call on a stream of its own, many times over: the bits of one after another."""
    jobs = []
    for k, (rows, hidden, features) in enumerate([(3, 2048, 1040), (300, 528, 2064), (90, 4096, 512)]):
        s = layer(rows, hidden, features, 20 + k)
        for c in s["calls"]:
            c()
        i = ffn_grad_case(gen_of("streams", k), rows, features, hidden)
        out = ffn_grad_outputs(i)
        ws = fc.alloc_gated_ffn_workspace(rows, features)
        call = fc.bind_gated_ffn_backward(i["x"], i["w_gate"], i["w_up"], i["gate"], i["up"], i["dout"], ws, **out)
        call()
        j = grad_case(rows, hidden, "f32")
        nout = norm_grad_outputs(j)
        ncall = fc.bind_layer_norm_backward(j["h"], j["stats"], j["dy"], workspace=fc.alloc_layer_norm_workspace(rows, hidden),
                                            dh=j["dh"], weight=j["weight"], **nout)
        ncall()
        torch.cuda.synchronize()
        got = [s["y"], s["a"], s["g"], s["u"], s["out"], *out.values(), *nout.values()]
        jobs.append((s["calls"], call, ncall, got, [t.clone() for t in got], [torch.cuda.Stream() for _ in range(3)]))
    torch.cuda.synchronize()
    for _ in range(10):
        for calls, call, ncall, _, _, st in jobs:
            for c in calls:
                c(st[0])
            call(st[1])
            ncall(st[2])
    torch.cuda.synchronize()
    for _, _, _, got, want, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_what_the_binding_refuses():
    x = torch.zeros(8, 64, dtype=B16, device="cuda")
    y = torch.empty_like(x)
    with pytest.raises(ValueError, match="contiguous"):
        fc.layer_norm(torch.zeros(64, 8, dtype=B16, device="cuda").t(), y)
    with pytest.raises(ValueError, match="weight"):
        fc.layer_norm(x, y, weight=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError, match="stats"):
        fc.layer_norm(x, y, stats=torch.empty(8, device="cuda"))
    with pytest.raises(fc.FcommError, match="together"):
        fc.layer_norm(x, y, residual_in=x)
    with pytest.raises(ValueError, match="workspace"):
        fc.layer_norm_backward(x, torch.empty(8, 2, device="cuda"), x, y, torch.empty(64, dtype=torch.uint8, device="cuda"))
    q = fc.alloc_fp8(8, 64)
    with pytest.raises(ValueError, match="codes"):
        fc.fp8_quantize(x, fc.alloc_fp8(4, 128))
    with pytest.raises(ValueError, match="w's scales"):
        fc.fp8_matmul(q, fc.alloc_fp8(16, 64), torch.empty(8, 16, device="cuda"))
    with pytest.raises(fc.FcommError, match="features"):
        fc.fp8_matmul(q, fc.alloc_fp8(8, 64, 128), torch.empty(8, 8, device="cuda"))
    w = torch.zeros(16, 64, dtype=B16, device="cuda")
    out = torch.empty(8, 16, dtype=B16, device="cuda")
    with pytest.raises(ValueError, match="w_up"):
        fc.gated_ffn(x, w, w[:8], out)
    with pytest.raises(ValueError, match="x must be"):
        fc.gated_ffn(x.float(), w, w, out)
    with pytest.raises(fc.FcommError, match="activation"):
        fc.gated_ffn(x, w, w, out, activation=5)
    with pytest.raises(fc.FcommError, match="together"):
        fc.gated_ffn(x, w, w, out, gate=torch.empty_like(out))
    with pytest.raises(fc.FcommError, match="asked for"):
        fc.gated_ffn_backward(x, w, w, out, out, out, fc.alloc_gated_ffn_workspace(8, 16))


@pytest.mark.parametrize("rows", [1, 70, 300])
def test_serving_step_captured_and_replayed(rows):
    """Norm, projections, quantisation and product captured into one graph and replayed on new
    inputs, launches without a wait between them: the bits of the calls one after another."""
    s, s2 = layer(rows, 528, 1040, 9), layer(rows, 528, 1040, 9)
    for c in s["calls"]:
        c()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in s["calls"]:
            c(side)
    for k in range(3):
        for t in (s, s2):
            t["x"].copy_(randn(gen_of("serve", k), rows, 528, dtype=B16))
        s["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        for c in s2["calls"]:
            c()
            torch.cuda.synchronize()
        for name in ("h", "y", "a", "g", "u", "out"):
            assert torch.isfinite(s[name]).all() and torch.equal(s[name], s2[name]), name


def test_two_graphs_at_once():
    """Two captured gradients, each with a workspace of its own, replayed on two streams at once."""
    jobs = []
    for k, (rows, features, hidden) in enumerate([(300, 528, 400), (130, 1040, 272)]):
        i = ffn_grad_case(gen_of("graphs", k), rows, features, hidden)
        want, out = ffn_grad_outputs(i), ffn_grad_outputs(i)
        run_ffn_grad(i, want)
        ws = fc.alloc_gated_ffn_workspace(rows, features)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            run_ffn_grad(i, out, ws=ws, stream=st)
        jobs.append((i, want, out, ws, st, graph))
    for _ in range(5):
        for *_, st, graph in jobs:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, want, out, *_ in jobs:
        assert all(torch.equal(want[k], out[k]) for k in want)


@pytest.mark.parametrize("name", ["decode", "prefill", "decode-qtagged"])
def test_pipeline_into_an_8_bit_projection(name):
    """The boundary's step with an 8-bit projection: h, y and the payload as without it, and
    the product of the quantised y with the quantised weight."""
    from quantized_reduce_rmsnorm_gb300 import synth
    from quantized_reduce_rmsnorm_gb300.pipeline import Pipeline
    w = synth.Workload(**{**synth.WORKLOADS[name].__dict__, "T": 48})
    inp = synth.make_inputs(w, seed=3)
    weight = randn(gen_of("projection", name), 1040, w.H, std=w.H ** -0.5, dtype=B16)
    plain, pipe = Pipeline(w, inp), Pipeline(w, inp, projection=weight, projection_format="fp8")
    assert pipe.launches_per_step == plain.launches_per_step + 3
    assert set(pipe.alg_bytes()) == set(plain.alg_bytes()) | {"projection"}
    plain.step()
    pipe.step()
    want, got = plain.outputs(), pipe.outputs()
    for k in want:
        assert want[k] is None and got[k] is None or (want[k] == got[k]).all(), k
    assert got["projection_status"].tolist() == [0, fc.STATUS_NO_INDEX]
    q = ref.quantise(pipe.y.cpu(), 1)
    assert torch.equal(pipe.y_fp8[0].cpu(), q[0]) and torch.equal(pipe.y_fp8[1].cpu(), q[1])
    xv = ref.values(q[0]) * ref.spread(q[1], 48, w.H)
    wv = ref.values(pipe.weight[0]) * ref.spread(pipe.weight[1], 1040, w.H)
    value, size = xv.cuda() @ wv.T, xv.abs().cuda() @ wv.abs().T
    within(pipe.out, value, HALF[B16] * value.abs() + (256 + w.H // 128 + 10) * U * size, "out")
    if name != "decode-qtagged":
        pipe.capture()
        pipe.out.zero_()
        pipe.replay()
        assert (pipe.outputs()["out"] == got["out"]).all()
    with pytest.raises(ValueError, match="projection_format"):
        Pipeline(w, inp, projection=weight, projection_format="fp4")
