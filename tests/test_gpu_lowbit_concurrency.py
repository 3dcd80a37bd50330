"""4-bit products that run beside one another on the GPU: many few-row products
whose CTAs share SMs (and their tensor-memory columns) on many streams."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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
    return q, x


@pytest.mark.parametrize("m,n,k", [(1, 768, 768), (20, 768, 768), (4, 2560, 512), (50, 640, 1024)])
def test_split_few_row_products_on_many_streams(mb, m, n, k):
    """24 streams of split products at once, eager and as one graph with as many branches."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    work = []
    for i in range(24):
        (qa, a), (qb, b) = _ones(mb, m, k, gen), _ones(mb, n, k, gen)
        out = torch.zeros(m, n, device="cuda")
        work.append((qa, qb, out, mb.alloc_matmul_workspace(qa.shape, qb.shape), (a.double() @ b.double().T).float()))
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()

    def fork_and_join():
        main = torch.cuda.current_stream()
        for s, (qa, qb, out, ws, _) in zip(streams, work):
            s.wait_stream(main)
            with torch.cuda.stream(s):
                for _ in range(6):
                    mb.mxfp4_matmul(qa, qb, out, ws)
        for s in streams:
            main.wait_stream(s)

    def check():
        torch.cuda.synchronize()
        for _, _, out, ws, want in work:
            assert torch.equal(out, want) and mb.device_status(ws) == 0
            out.zero_()
    fork_and_join()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fork_and_join()
    for _ in range(10):
        graph.replay()
    check()
