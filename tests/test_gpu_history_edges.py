"""Attention over the history, and blocks that go on, at the edges: scales that
lie far apart, of tokens that a row sees and of tokens that it does not, tiles
of zeros, the ends of fp32's range, and values that are not finite.  The bound
on a row's error comes from the slots that the row sees alone."""
import math

import pytest
import torch

from test_gpu_history import BF, E4M3, F16, HALF, TINY, U, Cache, _cu, _done, _far, _gen, _queries, _wave

pytestmark = pytest.mark.gpu


def seen_reference(c, q, lens, slots, starts, cu, scale):
    """(out, the bound on |got - out|) in 64 bits.  With w the normalised weights, A = sum w |v| and s the scores: weights are
    rounded to fp16 (2^-11 A); scores carry at most (D + 8) fp32 roundings of their absolute sum, which enter a weight
    as a factor exp(2 ds); exponentials and sums 2^-18; a product's sums are cut to fp32 after each 16 keys (2^-23 of A
    each); the result is rounded once.  Weights below fp16's normal range are off by 2^-25 where 2^7 stands for the
    largest weight times the largest V scale of its 128 slots, brought up to a power of two; of slots that the row does not
    see at most 2^4 times the least that it does: 2^-28 of 448 times that a key.  Scales are powers of two (or one a
    token), so that codes are exact."""
    H, D = q.shape[1], q.shape[2]
    g = H // c.Hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for i, (n, slot, s0) in enumerate(zip(lens, slots, starts)):
        t = s0 + n
        kd, vd = (c.values(which, slot, 0, t).repeat_interleave(g, 0) for which in (0, 1))
        vs = c.sc[c.layer, 1, slot][:, torch.arange(t, device=q.device) // c.block].double().repeat_interleave(g, 0)[:, None]
        qd = q[cu[i]:cu[i + 1]].double().transpose(0, 1)
        mask = torch.arange(t, device=q.device)[None] > s0 + torch.arange(n, device=q.device)[:, None]
        s = ((qd @ kd.transpose(1, 2)) * scale).masked_fill(mask, -math.inf)
        w = torch.softmax(s, -1)
        A = w @ vd.abs()
        # the largest seen scale of each 128 slots times the largest seen weight of them
        per_tile = lambda x: torch.nn.functional.pad(x, (0, -t % 128)).unflatten(-1, (-1, 128)).amax(-1)  # noqa: E731
        top = (per_tile(w) * 2 * per_tile(vs.expand_as(w).masked_fill(mask, 0.0))).amax(-1, keepdim=True)
        ds = ((D + 8) * U * scale * (qd.abs() @ kd.abs().transpose(1, 2))).masked_fill(mask, 0.0).amax(-1, keepdim=True)
        out[cu[i]:cu[i + 1]] = (w @ vd).transpose(0, 1)
        tol[cu[i]:cu[i + 1]] = (HALF[q.dtype] * (w @ vd).abs() + (2.0 ** -11 + 2.0 * ds + 2.0 ** -18 + t / 16 * 2.0 ** -23) * A * 1.01
                                + 2.0 ** -28 * 448 * top * t + TINY[q.dtype]).transpose(0, 1)
    return out, tol


def _run(c, q, lens, starts, H, D, frame=False, scale=None):
    """One call; its output, which is within the bound."""
    slots, cu, Hkv = list(range(len(lens))), _cu(lens), c.Hkv
    out = torch.full_like(q, 7.0)
    w = _wave(H, D, S=len(lens), T=c.T)
    if frame:
        w.history_attention_frame(0, torch.tensor(starts, dtype=torch.int32, device="cuda"), q, c.kv, c.sc, Hkv, c.block, out, scale=scale)
    else:
        w.history_attention(0, cu, slots, starts, q, c.kv, c.sc, Hkv, c.block, out, scale=scale)
    _done(w)
    ref, tol = seen_reference(c, q, lens, slots, starts, cu, D ** -0.5 if scale is None else scale)
    worst = float(((out.double() - ref).abs() / tol).max())
    assert worst <= 1.0, worst
    return out


def _rows(n, Hkv, D, seed):
    return [torch.randn(n, Hkv, D, generator=_gen(seed + j), device="cuda") * (1.5, 1.0)[j] for j in (0, 1)]


# a prompt of few rows, one of many that begins the history, one that goes on, one whose rows lie in two tiles of 128 slots
PROMPTS = [([12], [70]), ([200], [0]), ([150], [300]), ([90], [1000])]


@pytest.mark.parametrize("lens,starts", PROMPTS)
@pytest.mark.parametrize("block", [1, 16, 64, 128])
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("large", [1e3, 1e6, 1e12, 1e30])
def test_later_tokens_do_not_reach_earlier_rows(lens, starts, block, which, large):
    """Keys and values of the tokens from the middle of a prompt on that are finite and large: the rows before them stay
    within a bound that knows nothing of them."""
    H, Hkv, D = 4, 2, 64
    n, s0 = lens[0], starts[0]
    k, v = _rows(s0 + n, Hkv, D, 3)
    at = s0 + n // 2
    if which in ("k", "both"):
        k[at:] *= large
    if which in ("v", "both"):
        v[at:] *= large
    c = Cache(1, Hkv, (s0 + n + 3) // 4 * 4, D, block)
    c.write(0, 0, k, v)
    q, _ = _queries(n, H, D, BF)
    # large keys give the rows that see them scores that fp32 does not hold to a part of a unit: rows before them are checked
    rows = n // 2 if which != "v" else n
    out = torch.full_like(q, 7.0)
    w = _wave(H, D, S=1, T=c.T)
    w.history_attention(0, [0, n], [0], [s0], q, c.kv, c.sc, Hkv, block, out)
    _done(w)
    ref, tol = seen_reference(c, q[:rows], [rows], [0], [s0], [0, rows], D ** -0.5)
    worst = float(((out[:rows].double() - ref).abs() / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("block", [1, 16, 32, 128])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, BF), (128, F16)])
def test_one_later_value_far_from_the_others(block, D, dtype):
    """A single V token 2^30 above (fp16: 2^12) or a run of small ones 2^30 below the others, in and before the prompt."""
    H, Hkv, n, s0 = 3, 3, 300, 77
    far = 2.0 ** (30 if dtype is BF else 12)
    for change in ("later", "earlier", "small"):
        k, v = _rows(s0 + n, Hkv, D, 8)
        if change == "later":
            v[s0 + 140] *= far
        elif change == "earlier":
            v[30] *= far
        else:
            v[:s0 + 100] /= far
        c = Cache(1, Hkv, 380, D, block)
        c.write(0, 0, k, v)
        _run(c, _queries(n, H, D, dtype)[0], [n], [s0], H, D)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [1, 16, 128])
@pytest.mark.parametrize("lo,hi", [(-6, 6), (-40, 40), (-100, -60), (60, 90), (-60, 60)])
def test_values_of_many_magnitudes(frame, block, lo, hi):
    """V scales that differ by many powers of two, and runs of zeros, within a bound from the slots that a row sees."""
    lens, starts = ([1, 1, 1], [500, 39, 1100]) if frame else ([150, 1, 30], [300, 39, 1100])
    c = Cache(3, 2, 1132, 64, block)
    for i, (n, s0) in enumerate(zip(lens, starts)):
        k, v = _rows(n + s0, 2, 64, 20 + i)
        c.write(i, 0, k, v * _far(lo, hi)(n + s0))
    _run(c, _queries(sum(lens), 4, 64, BF)[0], lens, starts, 4, 64, frame=frame)


@pytest.mark.parametrize("block", [1, 16, 64])
@pytest.mark.parametrize("D,dtype,lo,hi", [(128, BF, -30, 30), (64, BF, -30, 30), (128, F16, -20, 6), (64, F16, -20, 6)])
def test_scales_far_apart_in_a_history_that_many_ctas_share(block, D, dtype, lo, hi):
    """Units whose keys are divided among CTAs, shared heads, two tiles of rows to a unit, K's scales far apart too; and NaN in
    V behind a row's end, which reaches the rows that attend to it alone."""
    H, Hkv, lens, starts = 6, 2, [300, 70, 33], [2500, 1100, 0]
    c, cu = Cache(3, Hkv, 2800, D, block), _cu(lens)
    for i, (n, s0) in enumerate(zip(lens, starts)):
        k, v = _rows(n + s0, Hkv, D, 40 + i)
        c.write(i, 0, k * _far(-12, 1)(n + s0).roll(17, 0), v * _far(lo, hi)(n + s0))
    q = _queries(cu[-1], H, D, dtype)[0]
    out = _run(c, q, lens, starts, H, D)
    c.kv[0, 1, 0, 1, 2500 + 150, 5] = 0x7F
    c.kv[0, 1, 2, 0, 20, D - 1] = 0xFF
    again, w = torch.full_like(q, 7.0), _wave(H, D, S=3, T=c.T)
    w.history_attention(0, cu, [0, 1, 2], starts, q, c.kv, c.sc, Hkv, block, again)
    _done(w)
    nan = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    nan[150:300, 3:, 5] = True
    nan[cu[2] + 20:, :3, D - 1] = True
    assert torch.equal(again.isnan(), nan)
    assert torch.equal(again[~nan], out[~nan])


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [1, 16, 128])
@pytest.mark.parametrize("small,large", [(0.0, 2.0 ** 60), (0.0, 1.0), (2.0 ** -100, 2.0 ** 60)])
@pytest.mark.parametrize("order", ["small first", "large first", "in turns"])
def test_a_tile_of_values_far_below_anothers(frame, block, small, large, order):
    """All 128 values of a tile zero, or 2^160 below the next tile's: their weights still count in the sum."""
    H, D, n, s0 = 2, 64, 1 if frame else 70, 511
    k, v = _rows(s0 + n, H, D, 5)
    tile = torch.arange(s0 + n, device="cuda") // 128
    low = {"small first": tile < 2, "large first": tile >= 2, "in turns": tile % 2 == 0}[order]
    v = v * torch.where(low, small, large)[:, None, None]
    c = Cache(1, H, 584, D, block)
    c.write(0, 0, k, v)
    for q in (torch.zeros(n, H, D, dtype=BF, device="cuda"), _queries(n, H, D, BF)[0]):
        _run(c, q, [n], [s0], H, D, frame=frame)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [1, 16, 128])
@pytest.mark.parametrize("gap", [60.0, 300.0])
def test_scores_that_rise_and_fall_far(frame, block, gap):
    """Scores of whole tiles that differ by hundreds, rising, falling and in turns, with values that do not make up for it."""
    H, D, n, s0 = 2, 64, 1 if frame else 70, 640
    base_k, base_v = _rows(s0 + n, H, D, 6)
    q = _queries(n, H, D, BF)[0]
    q[..., 0] = 4.0
    tile = torch.arange(s0 + n, device="cuda") // 128
    for level in (tile, 5 - tile, tile % 2, (tile * 3) % 5):
        k, v = base_k.clone(), base_v * 2.0 ** (-9.0 * level.float())[:, None, None]
        k[..., 0] = level[:, None] * gap * D ** 0.5 / 4.0
        c = Cache(1, H, 712, D, block)
        c.write(0, 0, k, v)
        _run(c, q, [n], [s0], H, D, frame=frame)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [1, 16, 128])
def test_values_at_the_lower_end_of_fp32(frame, block):
    """V scales of 2^-120 and less, down to the least ordinary number."""
    H, D, n, s0 = 4, 64, 1 if frame else 100, 300
    for e in (-108, -114):
        k, v = _rows(s0 + n, 2, D, 9)
        c = Cache(1, 2, 400 + 4, D, block)
        c.write(0, 0, k, v * 2.0 ** e)
        out = _run(c, _queries(n, H, D, BF)[0], [n], [s0], H, D, frame=frame)
        assert bool((out != 0).any())


@pytest.mark.parametrize("n,s0", [(1, 9000), (5, 9000), (100, 4000), (300, 0)])
@pytest.mark.parametrize("block", [1, 16, 128])
def test_values_at_the_upper_end_of_fp32(n, s0, block):
    """Thousands of values of one sign near fp32's largest, whose sum leaves it, where warps and CTAs share a row's keys."""
    H, Hkv, D = 2, 2, 64
    for big in (2.0 ** 116, 2.0 ** 124):
        k, v = _rows(s0 + n, Hkv, D, 11)
        c = Cache(1, Hkv, (s0 + n + 3) // 4 * 4, D, block)
        c.write(0, 0, k, (1.0 + v.abs()).clamp(max=3.0) * big)
        for q in (torch.zeros(n, H, D, dtype=BF, device="cuda"), _queries(n, H, D, BF)[0]):
            out = _run(c, q, [n], [s0], H, D, frame=n == 1)
            assert bool(out.isfinite().all())


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [1, 16, 128])
def test_the_largest_scale_of_scores(frame, block):
    """scale near its limit with keys that keep the scores moderate: no factor between leaves fp32."""
    H, D, n, s0 = 4, 64, 1 if frame else 100, 300
    k, v = _rows(s0 + n, 2, D, 10)
    c = Cache(1, 2, 404, D, block)
    q = _queries(n, H, D, BF)[0].float()
    q = q.sign() * (2.0 + q.abs() / 4)
    for key, query, scale in ((2.0 ** -130, 1.0, 2.0e38), (2.0 ** -124, 2.0 ** 125, 0.25 / 64)):
        c.write(0, 0, k * key, v)
        _run(c, (q * query).to(BF), [n], [s0], H, D, frame=frame, scale=scale)


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
