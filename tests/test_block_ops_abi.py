"""CPU checks of the block norms, their gradient and the microscaled 4-bit entry
points: sizes, and every refusal before anything touches a GPU (the pointers
given here are never followed)."""
import ctypes

import pytest
import torch

import block_ref as ref
from quantized_reduce_rmsnorm_gb300 import fcomm as fc

A = [1 << 40 | k << 30 for k in range(1, 16)]  # 32-byte aligned, a gigabyte apart
BF16, F32, INT8 = fc.FMT_BF16, fc.FMT_F32, fc.FMT_INT8_SYM


def refused(name, *args, status=fc.FC_ERR_INVALID, says=""):
    L = fc.load()
    assert getattr(L, name)(*args) == status
    msg = L.fc_last_error().decode()
    assert msg and says in msg, msg


def test_sizes():
    assert fc.mx4_codes_bytes(3, 64) == 96 and fc.mx4_codes_bytes(3, 48) == 0
    assert fc.mx4_scales_bytes(1, 32) == 512 and fc.mx4_scales_bytes(129, 160) == 4 * 512
    assert fc.mx4_scales_bytes(0, 128) == 0 and fc.mx4_scales_bytes(-1, 128) == 0
    ws = fc.load().fc_block_norm_backward_workspace
    assert ws(5, 64, 0) == 5 * 64 * 4 * 2 and ws(5, 64, 1) == 5 * 64 * 4 * 3 and ws(5, 64, 5) == 5 * 64 * 4 * 2
    assert ws(10 ** 6, 64, 0) == 608 * 64 * 4 * 2 and ws(0, 64, 0) == 0
    # rows * hidden past 32 bits
    assert fc.mx4_codes_bytes(1 << 20, 16384) == 1 << 33


def test_scale_tiles_hold_every_scale_once():
    for rows, hidden in ((1, 32), (129, 160), (300, 1056)):
        off = ref.scale_offsets(rows, hidden).flatten()
        assert len(off.unique()) == len(off) and int(off.max()) < fc.mx4_scales_bytes(rows, hidden)


def test_reference_codec_by_hand():
    x = torch.tensor([[6.0, 0.25, 0.75, -2.5, 5.0, 7.9, -0.3] + [0.0] * 25])
    code, byte = ref.mx4_reference(x)  # largest 7.9: e = 2 - 2 = 0
    assert byte.tolist() == [[127]]
    assert code[0, :8].tolist() == [7, 0, 2, 12, 6, 7, 9, 0]
    codes, scales = ref.pack_mx4(code, byte, fill=9)
    assert codes[0, :4].tolist() == [0x07, 0xC2, 0x76, 0x09]
    assert scales[:4].tolist() == [127, 0, 0, 0] and (scales[4:] == 9).all()


@pytest.mark.parametrize("rows,hidden,dtype,status", [
    (-1, 64, BF16, 1), (4, 48, BF16, 1), (4, 0, BF16, 1), (4, 64, INT8, 1), (4, 65568, F32, 4), (1 << 31, 64, F32, 4)])
def test_mx4_shapes(rows, hidden, dtype, status):
    q = fc.Mx4(A[1], A[2])
    refused("fc_mx4_quantize", A[0], dtype, rows, hidden, q, None, status=status)
    refused("fc_mx4_dequantize", q, rows, hidden, A[0], dtype, None, status=status)
    refused("fc_mx4_matmul", q, fc.Mx4(A[3], A[4]), rows, 64, hidden, A[0], dtype, None, None, status=status)


def test_mx4_pointers_and_overlaps():
    q = fc.Mx4(A[1], A[2])
    refused("fc_mx4_quantize", None, BF16, 4, 64, q, None, says="x must not be NULL")
    refused("fc_mx4_quantize", A[0] + 16, BF16, 4, 64, q, None, says="32-byte")
    refused("fc_mx4_quantize", A[0], BF16, 4, 64, fc.Mx4(None, A[2]), None, says="out.codes")
    refused("fc_mx4_quantize", A[0], BF16, 4, 64, fc.Mx4(A[1], A[2] + 8), None, says="out.scales")
    refused("fc_mx4_quantize", A[0], BF16, 4, 64, fc.Mx4(A[0] + 64, A[2]), None, says="overlaps")
    refused("fc_mx4_quantize", A[0], BF16, 4, 64, fc.Mx4(A[1], A[1] + 112), None, says="overlaps")
    refused("fc_mx4_dequantize", q, 4, 64, None, BF16, None, says="out")
    refused("fc_mx4_dequantize", q, 4, 64, A[1], BF16, None, says="overlaps")
    assert fc.load().fc_mx4_quantize(None, BF16, 0, 64, fc.Mx4(), None) == fc.FC_OK
    assert fc.load().fc_mx4_dequantize(fc.Mx4(), 0, 64, None, BF16, None) == fc.FC_OK


def test_matmul_refusals():
    x, w = fc.Mx4(A[1], A[2]), fc.Mx4(A[3], A[4])
    for features in (0, 8, 24, -16):
        refused("fc_mx4_matmul", x, w, 4, features, 64, A[0], BF16, None, None, says="features")
    refused("fc_mx4_matmul", x, w, 4, 1 << 23, 64, A[0], BF16, None, None, status=fc.FC_ERR_UNSUPPORTED)
    refused("fc_mx4_matmul", x, w, 1 << 23, 64, 64, A[0], BF16, None, None, status=fc.FC_ERR_UNSUPPORTED)
    refused("fc_mx4_matmul", x, fc.Mx4(), 4, 64, 64, A[0], BF16, None, None, says="w.codes")
    refused("fc_mx4_matmul", x, w, 4, 64, 64, A[0], BF16, A[5] + 2, None, says="d_status")
    refused("fc_mx4_matmul", x, w, 4, 64, 64, A[1], BF16, None, None, says="overlaps")
    assert fc.load().fc_mx4_matmul(x, w, 0, 64, 64, None, BF16, None, None) == fc.FC_OK


def spec(post=None, gate=None, pre=None, gate_rows=0, alpha=1.0, beta=1.0, eps1=1e-5, eps2=1e-5):
    return fc.BlockNormSpec(post, gate, pre, gate_rows, alpha, beta, eps1, eps2)


def norm(sp, x=A[0], r=A[1], rows=6, hidden=64, dtype=BF16, h=A[2], y=None, q=None):
    return (x, r, rows, hidden, dtype, None if sp is None else ctypes.byref(sp), h, y, q or fc.Mx4(), None)


def test_block_norm_refusals():
    n = "fc_block_norm"
    pre = spec(pre=A[5])
    refused(n, *norm(None), says="spec")
    refused(n, *norm(spec(), rows=-1), says="rows")
    refused(n, *norm(spec(), hidden=72), says="multiple of 16")
    refused(n, *norm(spec(), hidden=16400), status=fc.FC_ERR_UNSUPPORTED)
    refused(n, *norm(spec(), dtype=INT8), says="dtype")
    refused(n, *norm(pre), says="pre_weight needs")
    refused(n, *norm(spec(), y=A[3]), says="need pre_weight")
    refused(n, *norm(pre, hidden=48, q=fc.Mx4(A[3], A[4])), says="multiple of 32")
    refused(n, *norm(pre, q=fc.Mx4(A[3], None)), says="y_mx4.scales")
    for rows in (0, 4, 7, -1):
        refused(n, *norm(spec(gate=A[6], gate_rows=rows)), says="gate_rows")
    refused(n, *norm(spec(gate_rows=2)), says="gate_rows")
    for bad in (-1e-6, 1.5, float("nan")):
        refused(n, *norm(spec(eps1=bad)), says="eps")
        refused(n, *norm(spec(eps2=bad)), says="eps")
    for bad in (float("nan"), float("inf")):
        refused(n, *norm(spec(alpha=bad)), says="finite")
        refused(n, *norm(spec(beta=bad)), says="finite")
    for kw in (dict(x=None), dict(x=A[0] + 16), dict(r=A[1] + 16), dict(h=None), dict(h=A[2] + 2)):
        refused(n, *norm(spec(), **kw))
    refused(n, *norm(spec(pre=A[5] + 16), y=A[3]), says="pre_weight")
    refused(n, *norm(pre, y=A[2]), says="overlaps")            # y and residual_out
    refused(n, *norm(spec(), h=A[0] + 64), says="overlaps")    # part of x
    refused(n, *norm(spec(gate=A[6], gate_rows=6), h=A[6]), says="overlaps")
    refused(n, *norm(spec(post=A[6]), h=A[6]), says="overlaps")
    refused(n, *norm(pre, q=fc.Mx4(A[0], A[4])), says="overlaps")
    assert fc.load().fc_block_norm(*norm(pre, rows=0, y=A[3])) == fc.FC_OK


def back(sp, g, x=A[0], h=A[1], dy=A[2], dh=A[3], rows=6, hidden=64, dtype=BF16, ws=A[4], st=None):
    return (x, h, dy, dh, rows, hidden, dtype, ctypes.byref(sp), None if g is None else ctypes.byref(g), ws, st, None)


def test_block_norm_backward_refusals():
    n = "fc_block_norm_backward"
    full = spec(post=A[5], gate=A[6], pre=A[7], gate_rows=2)
    g = fc.BlockNormGrads(A[8], A[9], A[10], A[11], A[12])
    refused(n, *back(full, None), says="grads")
    refused(n, *back(spec(pre=A[7]), g), says="asked for")
    refused(n, *back(spec(), fc.BlockNormGrads(A[8], None, None, None, A[12])), says="asked for")
    refused(n, *back(full, g, dy=None), says="dy")
    refused(n, *back(full, g, h=None), says="h must")
    refused(n, *back(spec(), fc.BlockNormGrads(A[8])), says="dy needs pre_weight")
    refused(n, *back(spec(), fc.BlockNormGrads(A[8]), dy=None, dh=None), says="dh")
    refused(n, *back(full, fc.BlockNormGrads(None, A[9])), says="dx")
    refused(n, *back(full, g, ws=None), says="workspace")
    refused(n, *back(full, g, ws=A[4] + 16), says="workspace")
    refused(n, *back(full, g, st=A[13] + 2), says="d_status")
    refused(n, *back(full, fc.BlockNormGrads(A[8], A[8])), says="overlaps")
    refused(n, *back(full, fc.BlockNormGrads(A[8], None, None, A[6])), says="overlaps")
    refused(n, *back(full, g, ws=A[12]), says="overlaps")
    refused(n, *back(full, fc.BlockNormGrads(A[2] + 32)), says="overlaps")
    refused(n, *back(full, g, hidden=16400), status=fc.FC_ERR_UNSUPPORTED)
    for k in (2, 4):
        bad = fc.BlockNormGrads(A[8], A[9], A[10], A[11], A[12])
        setattr(bad, fc.BlockNormGrads._fields_[k][0], A[10] + 2)
        refused(n, *back(full, bad), says="4-byte")


def test_binding_checks_shapes_and_types():
    """The binding's own checks come before any pointer is taken."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fc.mx4_quantize(x, (torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        fc._dtype(x.half(), "x")
    with pytest.raises(ValueError, match="y must be"):
        fc._want(x[:2], x.shape, x.dtype, "y")
    with pytest.raises(ValueError, match="y must be"):
        fc._want(x.float(), x.shape, x.dtype, "y")
    with pytest.raises(ValueError, match="scales"):
        fc._mx4((torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(511, dtype=torch.uint8)), 4, 64, "q")
    with pytest.raises(ValueError, match="codes"):
        fc._mx4((torch.zeros(4, 31, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)), 4, 64, "q")
    with pytest.raises(ValueError, match="multiple of 32"):
        fc.alloc_mx4(4, 48, device="cpu")
    with pytest.raises(ValueError, match="one device"):
        fc._one_device(x, torch.zeros(1, device="meta"))


def test_device_bound_call_passes_exact_arguments(monkeypatch):
    """A device-bound call hands the entry point the values it was bound to, in its
    own types, on the stream asked for or the device's current one."""
    seen = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + d, raising=False)
    L = fc.load()
    q = fc.Mx4(A[1], A[2])
    b = fc.DeviceBound(L.fc_mx4_quantize, [A[0], BF16, 0, 1 << 33, q, None], 5, keep=(), device=0)
    assert b._fn.argtypes is None and b._fn(*b._args) == fc.FC_ERR_UNSUPPORTED  # hidden 2^33 arrives whole
    b._fn = lambda *a: seen.append([v.value if hasattr(v, "value") else v for v in a]) or 0
    for stream in (None, 5, None, 5):
        b(stream)
    assert [a[5] for a in seen] == [70, 5, 70, 5]
    assert all(a[:4] == [A[0], BF16, 0, 1 << 33] and a[4] is q for a in seen)
    b._fn = lambda *a: fc.FC_ERR_INVALID
    with pytest.raises(fc.FcommError):
        b()


@pytest.mark.parametrize("kind", ["Bound", "DeviceBound"])
def test_bound_call_shared_by_threads_keeps_each_call_on_its_stream(kind, monkeypatch):
    """Another thread's whole call on another stream, put between any two lines of a
    call: both launch on their own streams, and so do the calls after them."""
    import sys
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    cls = getattr(fc, kind)
    code = cls.__call__.__code__
    lines, at = 0, 0
    while at <= lines:
        fn, args = fc.load().fc_mx4_quantize, [A[0], BF16, 0, 64, fc.Mx4(A[1], A[2]), None]
        b = cls(fn, args, 5, keep=(), device=0) if kind == "DeviceBound" else cls(fn, args, 5)
        launched = []
        b._fn = lambda *a: launched.append(getattr(a[5], "value", a[5])) or 0
        seen = 0

        def trace(frame, event, arg):
            nonlocal seen
            if frame.f_code is not code:
                return None
            if event == "line":
                seen += 1
                if seen == at:  # the other thread runs here
                    sys.settrace(None)
                    b(22)
                    sys.settrace(trace)
            return trace

        b(33)
        before = sys.gettrace()
        sys.settrace(trace)
        try:
            b(11)
        finally:
            sys.settrace(before)
        lines = max(lines, seen)
        assert sorted(launched[1:]) == ([11, 22] if at else [11]), (at, launched)
        for s in (11, 22, 11):
            b(s)
            assert launched[-1] == s, (at, launched)
        at += 1
    assert lines >= 3


def test_status_word_overlaps_no_tensor_of_its_call():
    """d_status is an output: reset before the kernel runs, it would spoil an input that holds it."""
    x, w, E = fc.Mx4(A[1], A[2]), fc.Mx4(A[3], A[4]), A[5]
    for at in (A[0], A[0] + 4 * 64 * 2 - 4, A[1], A[2] + 508, A[3] + 64, A[4]):
        refused("fc_mx4_matmul", x, w, 4, 64, 64, A[0], BF16, at, None, says="d_status")
    full = spec(post=A[5], gate=A[6], pre=A[7], gate_rows=2)
    g = fc.BlockNormGrads(A[8], A[9], A[10], A[11], A[12])
    for at in A[:13]:
        refused("fc_block_norm_backward", *back(full, g, st=at), says="d_status")
    refused("fc_block_norm_backward", *back(full, g, st=A[0] - 4), says="d_status")


@pytest.mark.parametrize("rows,features,hidden", [(3, 32, 65536), (1, 16, 16384), (1, 512, 4096), (5, 16, 64)])
def test_exact_product_inputs_show_every_block(rows, features, hidden):
    """The inputs of the exact test of the product see a block's scale doubled, a stage of
    256 elements left out and two neighbouring blocks' scales exchanged, at any k."""
    g = torch.Generator().manual_seed(rows + features + hidden)
    ((xc, xb), (wc, wb)), want = ref.scaled_pair(g, rows, features, hidden)
    assert torch.equal(want.float().double(), want) and len(xb.unique()) > 1 and len(wb.unique()) > 1
    blocks = hidden // 32
    xv, wv = (ref.mx4_values(c, b).reshape(len(c), blocks, 32) for c, b in ((xc, xb), (wc, wb)))
    part = torch.einsum("tbk,nbk->btn", xv, wv)  # each block's share of the result
    assert (part.sum(0) == want).all()
    assert (part != 0).any(2).float().mean() > 0.99     # a block of x doubled: seen in some feature
    assert (part != 0).any(1).float().mean() > 0.85     # a block of w: few tokens see it
    stages = torch.stack([p.sum(0) for p in part.split(8)])
    assert (stages != 0).flatten(1).any(1).all()
    f = torch.exp2((xb[:, 1:] - xb[:, :-1]).double()).T[..., None]  # [block, token, 1]
    moved = part[:-1] * f + part[1:] / f - part[:-1] - part[1:]
    assert (moved != 0).any(2)[(f != 1)[..., 0]].float().mean() > 0.97
