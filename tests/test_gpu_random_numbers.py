"""Dropout masks and roundings of layers and steps on the GPU, eager and replayed:
no two passes of a run share them."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_masks_and_roundings_of_a_run_differ(captured):
    import muon_newton_schulz_05_b200 as mb
    from muon_newton_schulz_05_b200.fourbit import Mxfp4Linear, advance
    torch.cuda.set_device(0)
    T, N, p = 256, 512, 0.5
    layers = [Mxfp4Linear((1, N, N), T, p=p, site=s) for s in range(3)]
    rng = torch.tensor([3, 2 ** 40], dtype=torch.int64, device="cuda")
    w = torch.zeros(1, N, N, device="cuda")
    x = torch.ones(T, N, device="cuda")
    dy = torch.full((T, N), 1.25, device="cuda")     # half way between two levels of its block's scale
    dy[:, ::32] = 6.0
    y, grad, dx = torch.empty(T, N, device="cuda"), torch.empty_like(w), torch.empty_like(x)
    seen = torch.empty(len(layers), 2, T, N, device="cuda")
    for lin in layers:
        lin.refresh(w)

    def step():
        for i, lin in enumerate(layers):
            lin.forward(x, y, rng)
            lin.backward(dy, grad, dx, rng)
            mb.mxfp4_dequantize(lin.x, seen[i, 0])
            mb.mxfp4_dequantize(lin.dy, seen[i, 1])
        advance(rng, layers)
    run = step
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    drawn = []
    for _ in range(4):
        run()
        drawn += [v.clone() for v in seen]
    assert rng.tolist() == [3, 2 ** 40 + 4 * 3]
    free = torch.ones(N, dtype=torch.bool, device="cuda")
    free[::32] = False                               # the columns that hold the sixes
    for a, b in itertools.combinations(drawn, 2):
        # fair coins: equal in half of the places, give or take six standard deviations
        for k, n in ((0, T * N), (1, T * int(free.sum()))):
            same = (a[k] == b[k])[:, free].double().mean() if k else (a[k] == b[k]).double().mean()
            assert abs(float(same) - 0.5) < 6 * 0.5 / n ** 0.5
    assert all(lin.device_status() == 0 for lin in layers)
