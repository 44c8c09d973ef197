"""Sessions from prompts at the edges: rows and parameters that the calls allow
and that the other tests' shapes do not reach."""
import pytest
import torch

import frame_step_decode_gb300 as fsd
from test_gpu_prompt import _check_state, _hybrid, _state_case, _weights

pytestmark = pytest.mark.gpu


def _run_state(hs, case, slots, starts, S, heads=1, dim=64):
    """One call on a handle of its own; the new state (9 where nothing is written)."""
    cu, zx, prm, h0, out = case
    cfg, w = _hybrid(hs, S=S, heads=heads, dim=dim)
    new = torch.full_like(h0, 9.0)
    try:
        w.prompt_state(0, _weights(cfg, prm), cu, slots, starts, zx, h0, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    return new


@pytest.mark.parametrize("lens", [[129], [700], [64, 0, 1, 200], [1500, 3]])
@pytest.mark.parametrize("hs", [4, 12, 20])
def test_state_rows_padded_to_16_bytes(hs, lens):
    """Rows of a width that is no multiple of 16 bytes, padded to one: the
    stride is what a tensor map describes, whatever the width is."""
    n = len(lens)
    starts, slots = [i % 2 for i in range(n)], list(range(n))
    case = _state_case(lens, hs, starts, seed=hs + n, first=2, tail=3, S=n, pad=4)
    cu, zx, prm, h0, out = case
    assert zx.stride(0) % 8 == 0 and zx.shape[1] % 8 == 4
    new = _run_state(hs, case, slots, starts, n)
    _check_state(cu, zx, prm, h0, slots, starts, hs, out, new, n)
    assert bool((out[:2] == 7).all()) and bool((out[cu[-1]:] == 7).all())
