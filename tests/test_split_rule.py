"""Which products are split along K (seen in the workspace they ask for): where
splitting and not splitting were measured to differ by more than 4 %, the
faster one."""
import pytest

import muon_newton_schulz_05_b200 as mb

# (m, n, k), us unsplit, us split
MEASURED = [((200, 200, 4096), 9.7, 9.3), ((200, 200, 8192), 14.7, 9.8), ((500, 500, 5120), 12.8, 10.3),
            ((768, 768, 3328), 10.7, 11.0), ((768, 768, 5120), 12.7, 11.6), ((768, 768, 8192), 16.2, 12.8),
            ((700, 1000, 4096), 10.9, 12.1), ((700, 1000, 8192), 15.5, 13.6), ((1000, 1000, 5120), 12.1, 12.9),
            ((1000, 1000, 8192), 15.6, 14.1), ((1000, 1500, 6144), 14.2, 15.4), ((1000, 1500, 10240), 18.9, 17.6),
            ((1500, 1500, 8192), 16.6, 19.8), ((1500, 1500, 10240), 18.9, 21.2), ((1500, 1500, 12288), 21.2, 22.7)]


@pytest.mark.parametrize("shape,whole,split", MEASURED, ids=str)
def test_the_faster_form_is_taken(shape, whole, split):
    m, n, k = shape
    if abs(whole - split) > 0.04 * min(whole, split):
        assert (mb.matmul_workspace_size((1, m, k), (1, n, k)) > 4096) == (split < whole)
