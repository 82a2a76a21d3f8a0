"""GPU tests of waits that run out: with the limit of the kernels' waits made short, a
call gives up on a copy or a product that is on its way, reports FC_ERR_CUDA in
its status and lets what is in flight end; the calls after it are as ever."""
import contextlib
import ctypes

import pytest
import torch

import block_ref as ref
from quantized_reduce_rmsnorm_gb300 import fcomm as fc

pytestmark = pytest.mark.gpu

# Clock cycles: none at all, where the first copy is always given up on, to more than
# these calls take.
LIMITS = [0, 300, 600, 1000, 1500, 2000, 3000, 4500, 7000, 12000, 1 << 19]


@contextlib.contextmanager
def wait_cycles(n: int):
    limit = ctypes.c_int64.in_dll(fc.load(), "_ZN2fc11wait_cyclesE")
    whole = limit.value
    limit.value = n
    try:
        yield
    finally:
        limit.value = whole


def product_case(rows, features, hidden):
    g = torch.Generator().manual_seed(rows + 3 * features + 5 * hidden)
    q, v = [], []
    for n in (rows, features):
        code = torch.randint(0, 16, (n, hidden), generator=g)
        byte = torch.full((n, hidden // 32), 127)
        q.append(tuple(t.cuda() for t in ref.pack_mx4(code, byte, fill=0xFF)))
        v.append(ref.mx4_values(code, byte).cuda())
    return q, (v[0] @ v[1].T).float()  # exact: multiples of 0.25 below 2^24 of them


def run_out(call, status, check, check_rest, limits=LIMITS, times=3):
    """call() under each limit: FC_OK and check(), or FC_ERR_CUDA, which it is without any
    waiting, and check_rest(); between them, with the whole limit, FC_OK and check()."""
    seen = set()
    for n in limits:
        for _ in range(times):
            with wait_cycles(n):
                call()
            torch.cuda.synchronize()
            got = status.tolist()
            assert got[0] in (fc.FC_OK, fc.FC_ERR_CUDA) and got[1] == fc.STATUS_NO_INDEX, got
            assert n > 0 or got[0] == fc.FC_ERR_CUDA
            seen.add(got[0])
            (check if got[0] == fc.FC_OK else check_rest)()
        call()
        assert status.tolist() == [fc.FC_OK, fc.STATUS_NO_INDEX]
        check()
    assert seen == {fc.FC_OK, fc.FC_ERR_CUDA}


# one CTA a tile, of one and of four stages; k over four and over eight CTAs of a cluster
@pytest.mark.parametrize("rows,features,hidden", [(5, 272, 160), (64, 512, 1024), (1, 8192, 4096), (40, 1024, 8192),
                                                  (130, 48, 8192)])
def test_product_that_gives_up(rows, features, hidden):
    (x, w), want = product_case(rows, features, hidden)
    out = torch.empty(rows, features, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    call = fc.bind_mx4_matmul(x, w, out, d_status=status)

    def run():
        out.fill_(float("nan"))
        call()

    def check():
        assert torch.equal(out, want)

    def check_rest():  # what is there is right
        there = ~torch.isnan(out)
        assert torch.equal(out[there], want[there])

    run_out(run, status, check, check_rest)


# fewer tiles than pairs of CTAs, and several tiles a pair; a call that gives up takes a second
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,features,hidden", [(200, 1040, 544), (2100, 4368, 288)])
def test_wide_product_that_gives_up(rows, features, hidden, dtype):
    (x, w), want = product_case(rows, features, hidden)
    want = want.to(dtype)
    out = torch.empty(rows, features, dtype=dtype, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    call = fc.bind_mx4_matmul(x, w, out, d_status=status)

    def run():
        out.fill_(float("nan"))
        call()

    def check():
        assert torch.equal(out, want)

    def check_rest():
        there = ~torch.isnan(out)
        assert torch.equal(out[there], want[there])

    run_out(run, status, check, check_rest,
            limits=[0, 600, 1500, 3000, 7000, 20000, 1 << 19], times=1)


# one CTA a row, and clusters of two and of four
@pytest.mark.parametrize("rows,hidden,dtype", [(1, 1040, torch.bfloat16), (700, 1040, torch.bfloat16),
                                               (300, 2064, torch.float32), (300, 16384, torch.bfloat16),
                                               (200, 12288, torch.float32)])
def test_gradient_that_gives_up(rows, hidden, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + hidden)
    x, h, dy, dh = (torch.randn(rows, hidden, generator=g, device="cuda").to(dtype) for _ in range(4))
    w = torch.ones(hidden, dtype=dtype, device="cuda")
    dx, dr = torch.empty_like(x), torch.empty_like(x)
    dw1, dw2 = (torch.empty(hidden, device="cuda") for _ in range(2))
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    call = fc.bind_block_norm_backward(x, h, dy, dh, dx, fc.alloc_block_norm_workspace(rows, hidden), dresidual=dr,
                                       dpost_weight=dw1, dpre_weight=dw2, post_weight=w, pre_weight=w, d_status=status)
    outs = (dx, dr, dw1, dw2)

    def run():
        for t in outs:
            t.fill_(float("nan"))
        call()

    run()
    want = [t.clone() for t in outs]
    assert not any(torch.isnan(t).any() for t in want)

    def check():
        assert all(torch.equal(a, b) for a, b in zip(outs, want))

    def check_rest():  # every row counts as late, none is written; the sums over rows are of no use
        assert torch.isnan(dx).all() and torch.isnan(dr).all()

    run_out(run, status, check, check_rest, limits=[0, 1 << 19])
