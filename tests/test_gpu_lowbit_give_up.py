"""4-bit products whose bounded waits run out: a test hook lets some of the
threads that load operands stop early, and a short limit ends the waits for
what they would have brought. The kernel records it in the workspace's status
word and ends in order: what it wrote is right, the rest is as it was, and what
follows on the same device is right again."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TIMEOUT = 8


@pytest.fixture(scope="module")
def mb():
    import muon_newton_schulz_05_b200 as m
    torch.cuda.set_device(0)
    return m


def _ones(mb, rows, k, gen):
    """+1 and -1, which 4 bits hold exactly, quantised; sums of up to 2^24 of their products are exact in fp32."""
    x = torch.randint(0, 2, (rows, k), generator=gen, device="cuda").mul_(2).sub_(1).float()
    q = mb.alloc_mxfp4((rows, k))
    mb.mxfp4_quantize(x, q)
    return q, x.double()


def _give_up(mb, m, n, k, dtype, add, modes, split):
    gen = torch.Generator(device="cuda").manual_seed(5)
    (qa, a), (qb, b) = _ones(mb, m, k, gen), _ones(mb, n, k, gen)
    ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
    assert (ws.numel() > 4096) == split
    addend = torch.randint(-8, 9, (m, n), generator=gen, device="cuda").to(dtype) if add else None
    want = a @ b.T
    want = (want + addend.double() if add else want).float().to(dtype)
    out = torch.empty(m, n, dtype=dtype, device="cuda")
    left = torch.full_like(out, 12345.0)
    for mode in modes * 2:
        out.copy_(left)
        mb.set_debug(mode, 0.02)
        try:
            mb.mxfp4_matmul(qa, qb, out, ws, add=addend)
        finally:
            mb.set_debug(0, 0.0)
        assert mb.device_status(ws) == TIMEOUT
        assert bool(((out == want) | (out == left)).all()) and bool((out == left).any())
        if split:
            assert torch.equal(out, left)
            # and so they do, as documented, until the word is cleared
            mb.mxfp4_matmul(qa, qb, out, ws, add=addend)
            assert torch.equal(out, left)
        assert mb.device_status(ws, clear=True) == TIMEOUT and mb.device_status(ws) == 0
        mb.mxfp4_matmul(qa, qb, out, ws, add=addend)
        assert torch.equal(out, want) and mb.device_status(ws) == 0


# five or four stages in flight, one or many tiles per pair, results by TMA or by the warps, split along k
@pytest.mark.parametrize("m,n,k,modes,split", [(2600, 2600, 160, [1], False), (1024, 2048, 2560, [1, 2], False),
                                               (300, 1001, 2200, [1, 2], False), (768, 768, 32768, [1, 2], True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("add", [False, True])
def test_large_products_give_up_in_order(mb, m, n, k, dtype, add, modes, split):
    _give_up(mb, m, n, k, dtype, add, modes, split)


# K whole or split over a cluster, more stages than the ring holds, right rows that some CTAs have none of
@pytest.mark.parametrize("m,n,k", [(1, 50304, 768), (16, 2560, 2560), (1, 768, 768), (3, 300, 40000), (50, 640, 1024),
                                   (20, 384, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("add", [False, True])
def test_few_row_products_give_up_in_order(mb, m, n, k, dtype, add):
    _give_up(mb, m, n, k, dtype, add, [1, 2], False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_set_status_word_holds_split_products_back(mb, dtype):
    """The word set from the host on a healthy GPU: split products leave out as it was, others do not look."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    for m, n, k, split in ((200, 200, 16384, True), (600, 600, 512, False), (5, 600, 4096, False)):
        (qa, a), (qb, b) = _ones(mb, m, k, gen), _ones(mb, n, k, gen)
        ws = mb.alloc_matmul_workspace(qa.shape, qb.shape)
        assert (ws.numel() > 4096) == split
        want = (a @ b.T).float().to(dtype)
        out = torch.full((m, n), 12345.0, dtype=dtype, device="cuda")
        ws[:4] = torch.tensor([TIMEOUT, 0, 0, 0], dtype=torch.uint8, device="cuda")
        mb.mxfp4_matmul(qa, qb, out, ws)
        assert torch.equal(out, torch.full_like(out, 12345.0) if split else want)
        assert mb.device_status(ws, clear=True) == TIMEOUT
        mb.mxfp4_matmul(qa, qb, out, ws)
        assert torch.equal(out, want) and mb.device_status(ws) == 0


def test_a_layer_reports_and_clears_all_its_products(mb):
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear
    lin = Mxfp4Linear((1, 200, 320), 16384)
    gen = torch.Generator(device="cuda").manual_seed(7)
    w, x, dy = (torch.randn(s, generator=gen, device="cuda") for s in ((1, 200, 320), (16384, 320), (16384, 200)))
    rng = torch.tensor([1, 0], dtype=torch.int64, device="cuda")
    y, want, grad = torch.empty_like(dy), torch.empty_like(w), torch.full_like(w, 12345.0)
    lin.refresh(w)
    lin.forward(x, y)
    lin.backward(dy, want, rng=rng)
    assert lin.device_status() == 0 and lin.ws_dw.numel() > 4096     # the weight gradient is split
    for ws in (lin.ws_y, lin.ws_dw):
        ws[0] = TIMEOUT
    lin.backward(dy, grad, rng=rng)
    assert bool((grad == 12345.0).all())
    assert lin.device_status() == TIMEOUT == lin.device_status(clear=True)
    assert lin.device_status() == 0
    lin.backward(dy, grad, rng=rng)
    assert torch.equal(grad, want)
