"""Sessions from prompts at the edges: rows and parameters that the calls allow
and that the other tests' shapes do not reach."""
import pytest
import torch

import frame_step_decode_gb300 as fsd
from test_gpu_prompt import _attention, _check_attention, _check_state, _hybrid, _state_case, _wave, _weights

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


@pytest.mark.parametrize("a_log", [88.0, 89.0, 3e38])
@pytest.mark.parametrize("lens", [[25, 28], [129, 384, 200], [1300]])
def test_state_decays_beyond_fp32(a_log, lens):
    """exp(A_log) near the end of fp32's range and beyond it: a token with a
    step forgets all before it, one whose step is zero nothing, and what is not
    there (the rest of the last chunk) does neither."""
    hs, n = 4, len(lens)
    case = _state_case(lens, hs, [3] * n, seed=7, S=n)
    cu, zx, prm, h0, out = case
    prm[:hs], prm[hs:2 * hs] = a_log, 3.0
    if a_log < 1e3:  # softplus(-197) is zero in fp32, and 1e38 of it no decay
        for b in cu[1:]:
            zx[b - 7:b:2, -hs:] = -200.0
    slots, starts = list(range(n)), [3] * n
    new = _run_state(hs, case, slots, starts, n)
    _check_state(cu, zx, prm, h0, slots, starts, hs, out, new, n)


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("lens", [[25], [129], [1300]])
def test_state_parameters_that_are_not_a_number(lens, which):
    """NaN as a head's A_log, dt_bias or D: that head's outputs (and, but for
    D, its state) are NaN, the other heads of the call are exact."""
    hs = 4
    case = _state_case(lens, hs, [3], seed=8, S=1)
    cu, zx, prm, h0, out = case
    clean = prm.clone()
    prm[which * hs + 1] = float("nan")
    new = _run_state(hs, case, [0], [3], 1)
    P = h0.shape[3]
    assert bool(torch.isnan(out[:, P:2 * P]).all())
    if which < 2:
        assert bool(torch.isnan(new[0, 0, 1]).all())
    exact = torch.full_like(out, 7.0)
    want = _run_state(hs, (cu, zx, clean, h0, exact), [0], [3], 1)
    rest = [h for h in range(hs) if h != 1 or which == 2]
    assert torch.equal(new[0, 0, rest], want[0, 0, rest])
    assert torch.equal(out[:, :P], exact[:, :P]) and torch.equal(out[:, 2 * P:], exact[:, 2 * P:])
    if which == 0:  # also where no token has a step: NaN times zero
        zx[:, -hs:] = -200.0
        new = _run_state(hs, case, [0], [3], 1)
        assert bool(torch.isnan(out[:, P:2 * P]).all()) and bool(torch.isnan(new[0, 0, 1]).all())


@pytest.mark.parametrize("hs,lens", [(4, [25, 2048]), (64, [1, 300]), (64, [28] + [500] * 12), (32, [7, 300, 20, 129, 600, 40, 260]),
                                     (64, [1, 600] + [1] * 30), (8, [17, 3000, 5])])
def test_state_of_a_short_sequence_whoever_else_is_in_the_call(hs, lens):
    """Sequences of up to 28 tokens, alone and beside long ones: the same bits,
    of outputs and of the state; in place and called again at once, each call
    goes on from what the one before left."""
    n = len(lens)
    starts, slots = [3] * n, list(range(n))
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=hs, S=n)
    cfg, w = _hybrid(hs, S=n)
    wt = _weights(cfg, prm)
    together, alone, alone_out = h0.clone(), h0.clone(), torch.full_like(out, 7.0)
    try:
        for _ in range(3):
            w.prompt_state(0, wt, cu, slots, starts, zx, together, together, out)
        for i in range(n):
            for _ in range(3 if lens[i] <= 28 else 0):
                w.prompt_state(0, wt, cu[i:i + 2], [i], [3], zx, alone, alone, alone_out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    for i in range(n):
        if lens[i] <= 28:
            assert torch.equal(together[0, i], alone[0, i])
            assert torch.equal(out[cu[i]:cu[i + 1]], alone_out[cu[i]:cu[i + 1]])


def _timed(run):
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    run()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("ms", [2, 20])
def test_limits_take_the_time_they_say(ms):
    """A wait that nothing ends, in the attention and in the chunked state:
    near its limit (a try is 7920 cycles, counted as 4 us; 2.07 GHz at most)."""
    cu, q, k, v, out = _attention([300, 1, 700], 2, 2, 128, torch.bfloat16, seed=1)
    cs, zx, prm, h0, so = _state_case([300], 8, [0], seed=1)
    cfg, w = _hybrid(8, S=1, heads=2, dim=128)
    wt = _weights(cfg, prm)
    new = torch.zeros_like(h0)
    calls = [(9, lambda: w.prompt_attention(cu, q, k, v, out)), (10, lambda: w.prompt_state(0, wt, cs, [0], [0], zx, h0, new, so))]
    try:
        for which, run in calls:
            run()
            w.set_timeout_ns(ms * 1_000_000)
            w.debug_skip_signal(which, 0)
            took = _timed(run)
            assert w.status() == fsd.WAVE_ETIMEOUT
            assert 0.5 * ms < took < 2.5 * ms, took
            w.debug_skip_signal(which, -1)
            run()
            assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_attention(cu, q, k, v, out)
    _check_state(cs, zx, prm, h0, [0], [0], 8, so, new, 1)


LIMIT_MS = 20  # of a wait


@pytest.mark.parametrize("lens,H,Hkv", [([300] * 96, 8, 2), ([300, 1, 700], 2, 2), ([4100, 300], 4, 1)])  # more items than SMs, fewer, divided keys
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_attention_that_is_stuck_ends_after_one_limit(lens, H, Hkv, tile):
    """Copies that end before a tile: every role's wait runs out, CTAs that
    begin afterwards leave at once, and the handle goes on."""
    cu, q, k, v, out = _attention(lens, H, Hkv, 128, torch.bfloat16, seed=tile)
    w = _wave(H, 128)
    try:
        w.prompt_attention(cu, q, k, v, out)
        w.set_timeout_ns(LIMIT_MS * 1_000_000)
        w.debug_skip_signal(9, tile)
        ms = _timed(lambda: w.prompt_attention(cu, q, k, v, out))
        assert w.status() == fsd.WAVE_ETIMEOUT
        assert 0.5 * LIMIT_MS < ms < 2.5 * LIMIT_MS, ms
        w.debug_skip_signal(9, -1)
        w.prompt_attention(cu, q, k, v, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_attention(cu, q, k, v, out)


@pytest.mark.parametrize("hs,lens,pad", [(64, [200] * 40, 0), (64, [500] * 6, 0), (8, [600, 129], 0), (8, [2600, 700], 0), (4, [600, 129], 0),
                                         (4, [600, 20], 4)])
@pytest.mark.parametrize("chunk", [0, 1])
def test_state_that_is_stuck_ends_after_one_limit(hs, lens, pad, chunk):
    """The same of the chunked state, with and without a tensor map, in more
    units than SMs, fewer, and segments (of one chunk: there is no second)."""
    n = len(lens)
    starts, slots = [i % 2 for i in range(n)], list(range(n))
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=chunk, S=n, pad=pad)
    cfg, w = _hybrid(hs, S=n)
    wt = _weights(cfg, prm)
    new = torch.full_like(h0, 9.0)
    run = lambda: w.prompt_state(0, wt, cu, slots, starts, zx, h0, new, out)  # noqa: E731
    try:
        run()
        w.set_timeout_ns(LIMIT_MS * 1_000_000)
        w.debug_skip_signal(10, chunk)
        ms = _timed(run)
        if chunk == 0 or hs == 64:
            assert w.status() == fsd.WAVE_ETIMEOUT
            assert 0.5 * LIMIT_MS < ms < 2.5 * LIMIT_MS, ms
        else:
            assert w.status() in (fsd.WAVE_ETIMEOUT, fsd.WAVE_OK) and ms < 2.5 * LIMIT_MS
        w.debug_skip_signal(10, -1)
        run()
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_state(cu, zx, prm, h0, slots, starts, hs, out, new, n)


@pytest.mark.parametrize("ns", [4_000, 12_000])
def test_attention_gives_up_in_the_middle_of_an_item(ns):
    """A limit of a few tries, with items of 64 blocks: what waits for an item's
    end runs out while copies and products are under way.  Launches behind it
    give up too until the status has been read, and the next one is right."""
    cu, q, k, v, out = _attention([8192], 8, 1, 128, torch.bfloat16, seed=4)
    w = _wave(8, 128)
    try:
        w.set_timeout_ns(ns)
        w.prompt_attention(cu, q, k, v, out)
        w.set_timeout_ns(2_000_000_000)
        out.fill_(7)
        w.prompt_attention(cu, q, k, v, out)
        assert w.status() == fsd.WAVE_ETIMEOUT
        assert bool((out == 7).all()), "a launch behind one that gave up finds no work"
        w.prompt_attention(cu, q, k, v, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_attention(cu, q, k, v, out)


def test_attention_scales_at_the_ends_of_fp32():
    """Scores of zero are zero at every scale that is taken; one whose
    logarithm to base 2 leaves fp32 is refused."""
    cu, q, k, v, out = _attention([300], 2, 1, 64, torch.bfloat16, seed=1)
    q.zero_()
    w = _wave(2, 64)
    try:
        for scale in (2.3e38, 1e-45):
            out.fill_(7)
            w.prompt_attention(cu, q, k, v, out, scale=scale)
            assert w.status() == fsd.WAVE_OK
            _check_attention(cu, q, k, v, out, scale=scale)
        out.fill_(7)
        assert w.prompt_attention(cu, q, k, v, out, scale=3e38, check=False) == fsd.WAVE_EINVAL
        assert w.status() == fsd.WAVE_OK and bool((out == 7).all())
    finally:
        w.close()


@pytest.mark.parametrize("name", ["TINY", "MID"])
def test_append_of_a_steps_own_qkv_equals_its_append(name):
    """The q, k and v that a step dumps before the rotation (fp32), appended as
    prompts of one token at the sessions' positions: the codes and scales that
    the step wrote, bit for bit, of K and of V."""
    import synth
    from gpu_case import DeviceCase, dump_acts
    work = getattr(synth, name)
    case = DeviceCase(work)
    L, H, D, S, d = work.n_layers, work.n_heads, work.head_dim, case.S, work.d_model
    w = fsd.Wave(case.cfg, case.S_max, work.T_max)
    kv, sc = torch.zeros_like(case.kv), torch.zeros_like(case.sc)
    pos = case.pos_h.tolist()
    try:
        acts = torch.from_numpy(dump_acts(w, S, 1, lambda: case.step(w)))[0].cuda()  # [layers][S][record]
        for l in range(L):
            w.prompt_append(l, list(range(S + 1)), list(range(S)), pos, acts[l, :, 2 * d:2 * d + 3 * H * D].contiguous(), kv, sc)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    for s, p in enumerate(pos):
        assert torch.equal(kv[:, :, s, :, p], case.kv[:, :, s, :, p])
        assert torch.equal(sc[:, :, s, :, p], case.sc[:, :, s, :, p])


@pytest.mark.parametrize("lens,H,Hkv,D", [([3000], 2, 1, 128), ([900, 40], 4, 4, 64)])
def test_attention_alone_and_in_a_batch(lens, H, Hkv, D):
    """Prompts whose keys are divided when they come alone and are not in a
    larger batch: both within the bound of the definition."""
    more = lens + [700] * 60
    cu, q, k, v, out = _attention(more, H, Hkv, D, torch.bfloat16, seed=5)
    n = sum(lens)
    mine = cu[:len(lens) + 1]
    alone = torch.full_like(out, 7.0)
    w = _wave(H, D)
    try:
        w.prompt_attention(cu, q, k, v, out)
        w.prompt_attention(mine, q, k, v, alone)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    assert bool((alone[n:] == 7).all())
    for got in (out, alone):
        _check_attention(mine, q[:n], k[:n], v[:n], got[:n])


@pytest.mark.parametrize("hs,lens", [(128, [1, 40, 130]), (100, [300, 28]), (768, [2, 129])])
def test_state_of_many_heads(hs, lens):
    n = len(lens)
    starts, slots = [i % 2 for i in range(n)], list(range(n))
    case = _state_case(lens, hs, starts, seed=hs, S=n)
    cu, zx, prm, h0, out = case
    new = _run_state(hs, case, slots, starts, n)
    _check_state(cu, zx, prm, h0, slots, starts, hs, out, new, n)
