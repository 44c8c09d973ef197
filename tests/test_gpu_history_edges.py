"""Blocks that go on, at the edges: values that are not finite."""
import math

import pytest
import torch

from test_gpu_history import E4M3, Cache, _done, _gen, _wave

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("sizes", [(-60, 0, 40, 100), (40, 0), (20, 100), (120,)])
def test_values_that_are_not_finite_in_a_block_that_goes_on(block, frame, sizes):
    """NaN stays NaN whatever the block's scale becomes; an infinity is held as 448 times the scale that the block has
    when it comes, and goes along with the scale from there as any value does."""
    H, D, T = 2, 64, 128
    w = _wave(H, D, S=1, T=T)
    got = Cache(1, H, T, D, block)
    want = got.clone()
    first = torch.zeros(1, 3, H, D, device="cuda")
    first[0, 1, 0, 3], first[0, 2, 1, 63], first[0, 2, 0, 5], first[0, 1, 1, 7] = math.nan, math.nan, math.inf, -math.inf
    then = [torch.randn(1, 3, H, D, generator=_gen(k), device="cuda") * 2.0 ** e for k, e in enumerate(sizes)]
    for t, x in enumerate([first] + then):
        if frame:
            w.history_append_frame(0, torch.tensor([t], dtype=torch.int32, device="cuda"), x.reshape(1, -1), got.kv, got.sc, H, block)
        else:
            w.history_append(0, [0, 1], [0], [t], x.reshape(1, -1), got.kv, got.sc, H, block)
        want.write(0, t, x[:, 1], x[:, 2])
        gk, wk = (a.kv.view(E4M3).float() for a in (got, want))
        assert torch.equal(gk.isnan(), wk.isnan()), t
        assert torch.equal(gk.nan_to_num(), wk.nan_to_num()), t
        assert bool(gk[0, 0, 0, 0, 0, 3].isnan()) and bool(gk[0, 1, 0, 1, 0, 63].isnan())
        assert torch.equal(got.sc.nan_to_num(nan=-7.0), want.sc.nan_to_num(nan=-7.0))
    _done(w)
