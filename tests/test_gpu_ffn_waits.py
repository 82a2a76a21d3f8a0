"""GPU tests of waits that run out in layer norm's gradient, the 8-bit product and the gated
feed-forward: a call gives up on a copy or a product that is on its way, reports
FC_ERR_CUDA in its status and lets what is in flight end; the calls after it are as ever."""
import pytest
import torch

import ffn_ref as ref
from quantized_reduce_rmsnorm_gb300 import fcomm as fc
from test_gpu_bounded_waits import run_out

pytestmark = pytest.mark.gpu
B16 = torch.bfloat16
FEW = [0, 600, 1500, 3000, 7000, 20000, 1 << 19]  # where a call that gives up takes a second


def give_up(call, outs, limits=None, times=3, rest=None):
    """run_out() of a call whose outputs are `outs`: whole they are those of a call that is
    let run; what is there of them after one that gives up is right."""
    status = call[1]
    call[0]()
    want = [t.clone() for t in outs]
    assert not any(torch.isnan(t).any() for t in want)

    def run():
        for t in outs:
            t.fill_(float("nan"))
        call[0]()

    def check():
        assert all(torch.equal(a, b) for a, b in zip(outs, want))

    def check_rest():
        for a, b in zip(outs, want):
            there = ~torch.isnan(a)
            assert torch.equal(a[there], b[there])

    kw = {} if limits is None else {"limits": limits, "times": times}
    run_out(run, status, check, rest or check_rest, **kw)


def status_word():
    return torch.zeros(2, dtype=torch.int32, device="cuda")


# one CTA a tile; k over four and eight CTAs of a cluster; each width of the tile
@pytest.mark.parametrize("rows,features,hidden", [(5, 272, 160), (30, 512, 4096), (64, 512, 1024), (1, 8192, 4096),
                                                  (130, 48, 8192)])
def test_fp8_product_that_gives_up(rows, features, hidden):
    pair, _ = ref.exact_pair(torch.Generator().manual_seed(rows), rows, features, hidden)
    x, w = (tuple(t.cuda() for t in q) for q in pair)
    out, st = torch.empty(rows, features, device="cuda"), status_word()
    give_up((fc.bind_fp8_matmul(x, w, out, d_status=st), st), [out])


# fewer tiles than pairs of CTAs, and several tiles a pair
@pytest.mark.parametrize("rows,features,hidden,dtype", [(200, 1040, 544, B16), (2100, 4368, 288, torch.float32)])
def test_wide_fp8_product_that_gives_up(rows, features, hidden, dtype):
    pair, _ = ref.exact_pair(torch.Generator().manual_seed(rows), rows, features, hidden)
    x, w = (tuple(t.cuda() for t in q) for q in pair)
    out, st = torch.empty(rows, features, dtype=dtype, device="cuda"), status_word()
    give_up((fc.bind_fp8_matmul(x, w, out, d_status=st), st), [out], limits=FEW, times=1)


def ffn_tensors(rows, features, hidden):
    g = torch.Generator(device="cuda").manual_seed(rows + features)
    return [torch.randn(*s, generator=g, device="cuda").to(B16)
            for s in ((rows, hidden), (features, hidden), (features, hidden), (rows, features))]


@pytest.mark.parametrize("rows,features,hidden", [(5, 272, 160), (30, 512, 4096), (64, 512, 1024), (1, 8192, 4096),
                                                  (130, 48, 4096)])
def test_gated_ffn_that_gives_up(rows, features, hidden):
    x, wg, wu, out = ffn_tensors(rows, features, hidden)
    gate, up, st = torch.empty_like(out), torch.empty_like(out), status_word()
    give_up((fc.bind_gated_ffn(x, wg, wu, out, gate=gate, up=up, d_status=st), st), [out, gate, up])


@pytest.mark.parametrize("rows,features,hidden", [(200, 1040, 544), (2100, 4368, 144)])
def test_wide_gated_ffn_that_gives_up(rows, features, hidden):
    x, wg, wu, out = ffn_tensors(rows, features, hidden)
    gate, up, st = torch.empty_like(out), torch.empty_like(out), status_word()
    give_up((fc.bind_gated_ffn(x, wg, wu, out, gate=gate, up=up, d_status=st), st), [out, gate, up], limits=FEW, times=1)


@pytest.mark.parametrize("rows,features,hidden", [(5, 528, 160), (30, 512, 272), (64, 4112, 1040), (100, 1040, 528)])
def test_gated_ffn_gradient_of_few_tokens_that_gives_up(rows, features, hidden):
    x, wg, wu, d = ffn_tensors(rows, features, hidden)
    dx, st = torch.empty_like(x), status_word()
    call = fc.bind_gated_ffn_backward(x, wg, wu, d, d, d, fc.alloc_gated_ffn_workspace(rows, features), dx=dx, d_status=st)
    give_up((call, st), [dx])


@pytest.mark.parametrize("rows,features,hidden", [(20, 272, 528), (200, 528, 272), (1100, 4368, 144)])
def test_gated_ffn_gradient_that_gives_up(rows, features, hidden):
    x, wg, wu, d = ffn_tensors(rows, features, hidden)
    outs, st = [torch.empty_like(t) for t in (x, wg, wu)], status_word()
    call = fc.bind_gated_ffn_backward(x, wg, wu, d, d, d, fc.alloc_gated_ffn_workspace(rows, features), dx=outs[0],
                                      dw_gate=outs[1], dw_up=outs[2], d_status=st)
    give_up((call, st), outs, limits=FEW, times=1)


# one CTA a row of each size, and a cluster of two
@pytest.mark.parametrize("rows,hidden,dtype", [(1, 1040, B16), (700, 1040, B16), (300, 4112, torch.float32),
                                               (300, 16384, B16), (200, 12288, torch.float32)])
def test_layer_norm_gradient_that_gives_up(rows, hidden, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + hidden)
    h, dy, dh = (torch.randn(rows, hidden, generator=g, device="cuda").to(dtype) for _ in range(3))
    stats = torch.tensor([[0.0, 1.0]], device="cuda").repeat(rows, 1)
    dx, st = torch.empty_like(h), status_word()
    dw, db = (torch.empty(hidden, device="cuda") for _ in range(2))
    call = fc.bind_layer_norm_backward(h, stats, dy, dx, fc.alloc_layer_norm_workspace(rows, hidden), dh=dh, dweight=dw,
                                       dbias=db, d_status=st)

    def rest():  # every row counts as late, none is written; the sums over rows are of no use
        assert torch.isnan(dx).all()

    give_up((call, st), [dx, dw, db], limits=[0, 1 << 19], times=3, rest=rest)
