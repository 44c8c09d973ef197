"""Rotary positions and the block-scaled history on the GPU: append, read back
and attention, each against a plain 64-bit restatement, with bounds derived
from the roundings each one makes."""
import math

import pytest
import torch

import frame_step_decode_gb300 as fsd

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half a step below the normal range
U = 2.0 ** -24
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn


def _cu(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _wave(heads, dim, S=8, T=64, layers=1):
    return fsd.Wave(fsd.WaveConfig(layers, 64, heads, dim, 64, 1e-5, 1e4), S, T)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _done(w):
    try:
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()


# ------------------------------------------------------------------- rotation
ROPES = {"whole": dict(dims=1.0), "half turned": dict(dims=0.5), "48": dict(dims=48), "one group": dict(dims=16),
         "linear": dict(dims=1.0, scaling="linear", factor=4.0),
         "parts": dict(dims=1.0, scaling="parts", factor=8.0, original=4096.0, amplitude=1.2)}


def _plan(name, layout, D, base=1e4):
    kw = dict(ROPES[name])
    dims = kw.pop("dims")
    return fsd.rope_plan(int(dims * D) if isinstance(dims, float) else dims, base, layout=layout, **kw)


def turned(plan, pos, x):
    """(rotated rows, the bound on the fp32 arithmetic) in 64 bits: angles from the
    plan's turns by exact integers modulo a turn."""
    n = plan.dims
    turns = [plan.turns[i] for i in range(n // 2)]
    frac = torch.tensor([[(t * int(p)) % 2 ** 64 / 2.0 ** 64 for t in turns] for p in pos], dtype=torch.float64, device=x.device)
    ang = 2 * math.pi * frac
    c, s = plan.amplitude * ang.cos()[:, None], plan.amplitude * ang.sin()[:, None]
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    lo, hi = (slice(0, n // 2), slice(n // 2, n)) if plan.layout == 0 else (slice(0, n, 2), slice(1, n, 2))
    a, b = x[..., lo].double(), x[..., hi].double()
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    # the angle is held to pi/4 2^-24 of fp32, sine and cosine to 2 units in the last place, times the amplitude
    # (half a unit), two products and a sum (half a unit each): under 8 U of |a| + |b|
    e = 8 * U * plan.amplitude * (a.abs() + b.abs())
    tol[..., lo], tol[..., hi] = e, e
    return y, tol


@pytest.mark.parametrize("name", sorted(ROPES))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("types", [(BF, BF), (F32, F32), (F16, F32), (F32, F16), (BF, F16)])
def test_rotation_of_packed_rows(name, layout, D, types):
    plan = _plan(name, layout, D)
    lens, starts = [3, 0, 17, 1], [0, 5, 1000, 2 ** 31 - 2]
    cu, H = _cu(lens, first=2), 3
    x = (2 * torch.randn(cu[-1] + 3, H, D, generator=_gen(1), device="cuda")).to(types[0])
    out = torch.full(x.shape, 7.0, dtype=types[1], device="cuda")
    fsd.rope_apply(plan, x, out, cu_seqlens=cu, starts=starts)
    pos = [p + i for n, p in zip(lens, starts) for i in range(n)]
    ref, tol = turned(plan, pos, x[cu[0]:cu[-1]])
    tol = tol + HALF[types[1]] * (ref.abs() + tol) + TINY[types[1]]
    assert bool(((out[cu[0]:cu[-1]].double() - ref).abs() <= tol).all())
    assert bool((out[:cu[0]] == 7).all()) and bool((out[cu[-1]:] == 7).all())
    assert torch.equal(out[cu[0]:cu[-1], :, plan.dims:], x[cu[0]:cu[-1], :, plan.dims:].to(types[1]))


@pytest.mark.parametrize("rows,H", [(1, 1), (1, 40), (7, 5), (300, 2), (33, 80)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_at_positions_on_the_device(rows, H, layout):
    plan, D = _plan("whole", layout, 64, base=5e5), 64
    x = torch.randn(rows + 2, H, D, generator=_gen(rows), device="cuda").to(BF)
    pos = torch.randint(0, 2 ** 20, (rows,), generator=_gen(2), device="cuda", dtype=torch.int32)
    pos[rows // 2] = -1 - rows
    before = x.clone()
    fsd.rope_apply(plan, x, positions=pos)  # in place
    ref, tol = turned(plan, pos.clamp(min=0).tolist(), before[:rows])
    tol = tol + HALF[BF] * (ref.abs() + tol) + TINY[BF]
    on = pos >= 0
    assert bool(((x[:rows].double() - ref).abs() <= tol)[on].all())
    assert torch.equal(x[:rows][~on], before[:rows][~on]) and torch.equal(x[rows:], before[rows:])


def test_rotation_of_a_slice_of_a_wider_row():
    """The q and k of a qkv row at once, in place; v as it was."""
    H, Hkv, D, n = 4, 2, 64, 50
    qkv = torch.randn(n, (H + 2 * Hkv), D, generator=_gen(4), device="cuda")
    before, plan = qkv.clone(), _plan("parts", "half", D)
    fsd.rope_apply(plan, qkv[:, :H + Hkv], cu_seqlens=[0, n], starts=[7])
    ref, tol = turned(plan, range(7, 7 + n), before[:, :H + Hkv])
    assert bool(((qkv[:, :H + Hkv].double() - ref).abs() <= tol + U * ref.abs()).all())
    assert torch.equal(qkv[:, H + Hkv:], before[:, H + Hkv:])


def test_rotation_agrees_with_the_steps():
    """The half layout over whole heads is the step's rotation: prompt_append's q, within roundings."""
    H, D, n = 2, 128, 40
    qkv = torch.randn(n, 3 * H * D, generator=_gen(5), device="cuda")
    q, kv, sc = torch.zeros(n, H, D, dtype=F16, device="cuda"), torch.zeros(2 * H * 64 * D, dtype=torch.uint8, device="cuda"), torch.zeros(2 * H * 64, device="cuda")
    w = _wave(H, D, S=1)
    w.prompt_append(0, [0, n], [0], [3], qkv, kv, sc, q)
    _done(w)
    got = torch.zeros_like(q)
    x = qkv[:, :H * D].reshape(n, H, D)
    fsd.rope_apply(fsd.rope_plan(D), x, got, cu_seqlens=[0, n], starts=[3])
    assert bool(((got.double() - q.double()).abs() <= 2 * HALF[F16] * q.double().abs() + 16 * U * 6 + TINY[F16]).all())


# --------------------------------------------------------------------- history
def power_of_two(amax):
    """The least power of two s with amax <= 448 s, from 2^-126 on; 0 for 0."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
    return torch.where(amax == 0, torch.zeros_like(s), s)


def finite_amax(v):
    """Values that are not finite count as the least ordinary number."""
    return torch.where(v.isfinite(), v.abs(), torch.full_like(v, 2.0 ** -126)).amax(-1)


def encode(v, scale):
    q = torch.where(scale == 0, torch.zeros_like(v), v / torch.where(scale == 0, torch.ones_like(scale), scale))
    q = torch.where(q.isnan(), q, q.clamp(-448, 448))  # infinities saturate
    return q.to(E4M3).view(torch.uint8)


class Cache:
    """A history of one layer on the device, and the plain rules beside it."""

    def __init__(self, S, Hkv, T, D, block, layers=1, layer=0):
        self.S, self.Hkv, self.T, self.D, self.block, self.layer = S, Hkv, T, D, block, layer
        self.nb = -(-T // block)
        self.kv = torch.full((layers, 2, S, Hkv, T, D), 0x7F, dtype=torch.uint8, device="cuda")  # NaN where nothing was written
        self.sc = torch.full((layers, 2, S, Hkv, self.nb), math.nan, device="cuda")

    def clone(self):
        c = Cache.__new__(Cache)
        c.__dict__.update(self.__dict__)
        c.kv, c.sc = self.kv.clone(), self.sc.clone()
        return c

    def write(self, slot, start, k, v):
        """The append's rule on rows [n][Hkv][D] in fp32."""
        for which, rows in enumerate((k, v)):
            x = rows.transpose(0, 1).contiguous()  # [Hkv][n][D]
            n, b = x.shape[1], self.block
            codes, sc = self.kv[self.layer, which, slot], self.sc[self.layer, which, slot]
            if b == 1:
                s = x.abs().amax(-1)
                s = s / torch.full_like(s, 448.0)  # by a number, torch multiplies with its reciprocal
                sc[:, start:start + n] = s
                codes[:, start:start + n] = encode(x, s[..., None])
                continue
            for blk in range(start // b, (start + n - 1) // b + 1):
                lo, hi = max(start, blk * b), min(start + n, (blk + 1) * b)
                part = x[:, lo - start:hi - start]
                s = power_of_two(finite_amax(part).amax(-1))
                if lo > blk * b:
                    old = sc[:, blk].clone()
                    s = torch.maximum(s, old)
                    held = codes[:, blk * b:lo].view(E4M3).float()
                    ratio = torch.where(s == old, torch.ones_like(s), old / s)[:, None, None]
                    codes[:, blk * b:lo] = torch.where(ratio == 1, codes[:, blk * b:lo].int(), (held * ratio).to(E4M3).view(torch.uint8).int()).to(torch.uint8)
                sc[:, blk] = s
                codes[:, lo:hi] = encode(part, s[:, None, None])

    def values(self, which, slot, lo, hi, dtype=torch.float64):
        """[Hkv][hi - lo][D]"""
        per = torch.arange(lo, hi, device="cuda") // self.block
        return self.kv[self.layer, which, slot, :, lo:hi].view(E4M3).to(dtype) * self.sc[self.layer, which, slot][:, per, None].to(dtype)

    def same(self, other):
        return torch.equal(self.kv, other.kv) and torch.equal(self.sc.nan_to_num(nan=-7.0), other.sc.nan_to_num(nan=-7.0))


def _split(qkv, H, Hkv, D):
    x = qkv.float().reshape(qkv.shape[0], H + 2 * Hkv, D)
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


@pytest.mark.parametrize("block", [1, 16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,types", [(2, 2, (F32, BF)), (6, 2, (BF, F16)), (12, 3, (BF, BF)), (1, 1, (F32, F16))])
def test_append_codes_and_scales(block, D, H, Hkv, types):
    """Without a rotation the codes and scales are the rule's on the inputs, bit for bit: fresh blocks, blocks that go
    on with a larger, a smaller and an equal scale, blocks cut at either end, empty sequences, rows around them."""
    T, S = 404, 5
    w = _wave(H, D, S=S, T=T, layers=2)
    got = Cache(S, Hkv, T, D, block, layers=2, layer=1)
    want = got.clone()
    size = 0
    for k, (lens, slots, starts) in enumerate([([130, 0, 17, 1], [3, 1, 0, 4], [0, 0, 0, 0]), ([200, 47, 300], [3, 0, 4], [130, 17, 1]),
                                               ([1, 5, 60, 3], [3, 0, -1, 4], [330, 64, 0, 301]), ([403], [2], [1])]):
        cu = _cu(lens, first=k)
        # magnitudes that grow, shrink and reach over many powers of two; a few heads all zero
        mag = 2.0 ** torch.randint(-8, 9, (cu[-1] + 2, (H + 2 * Hkv), 1), generator=_gen(k), device="cuda").float()
        x = torch.randn(cu[-1] + 2, H + 2 * Hkv, D, generator=_gen(10 + k), device="cuda") * mag * 4.0 ** ((k + 1) % 3)
        if k == 0:
            x[:, H] = 0.0
        qkv = x.reshape(cu[-1] + 2, -1).to(types[0])
        q = torch.full((cu[-1] + 2, H, D), 7.0, dtype=types[1], device="cuda")
        if k == 3:
            want.write(2, 0, torch.zeros(1, Hkv, D, device="cuda"), torch.zeros(1, Hkv, D, device="cuda"))
            got = want.clone()
        w.history_append(1, cu, slots, starts, qkv, got.kv, got.sc, Hkv, block, q=q)
        xq, xk, xv = _split(qkv, H, Hkv, D)
        for i, (n, slot, s0) in enumerate(zip(lens, slots, starts)):
            r = slice(cu[i], cu[i + 1])
            if slot >= 0 and n:
                want.write(slot, s0, xk[r], xv[r])
                assert torch.equal(q[r], xq[r].to(types[1]))
            else:
                assert bool((q[r] == 7).all())
        assert bool((q[:cu[0]] == 7).all()) and bool((q[cu[-1]:] == 7).all())
        assert got.same(want), (k, block)
    _done(w)


@pytest.mark.parametrize("block", [1, 16, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_append_of_frames(block, D):
    """One token of each session at positions on the device: block starts, blocks that go on, the last slot, empty slots."""
    H, Hkv, S, T = 4, 2, 6, 132
    w = _wave(H, D, S=8, T=T)
    got = Cache(8, Hkv, T, D, block)
    for s, n in enumerate((40, 0, 64, 131, 7, 100)):
        if n:
            got.write(s, 0, torch.randn(n, Hkv, D, generator=_gen(s), device="cuda"), torch.randn(n, Hkv, D, generator=_gen(9 + s), device="cuda"))
    want = got.clone()
    pos = [40, 0, 64, 131, -1, 100]
    qkv = (torch.randn(S, H + 2 * Hkv, D, generator=_gen(77), device="cuda") * torch.tensor([64.0, 1, 2, 9, 1, 0.1], device="cuda")[:, None, None])
    qkv = qkv.reshape(S, -1)
    q = torch.full((S, H, D), 7.0, dtype=BF, device="cuda")
    w.history_append_frame(0, torch.tensor(pos, dtype=torch.int32, device="cuda"), qkv, got.kv, got.sc, Hkv, block, q=q)
    xq, xk, xv = _split(qkv, H, Hkv, D)
    for s, p in enumerate(pos):
        if p >= 0:
            want.write(s, p, xk[s:s + 1], xv[s:s + 1])
            assert torch.equal(q[s], xq[s].to(BF))
        else:
            assert bool((q[s] == 7).all())
    assert got.same(want)
    _done(w)


@pytest.mark.parametrize("block", [1, 32])
def test_a_frames_position_beyond_the_history(block):
    H, D, T = 2, 64, 64
    w = _wave(H, D, S=3, T=T)
    got = Cache(3, H, T, D, block)
    got.write(0, 0, torch.ones(9, H, D, device="cuda"), torch.ones(9, H, D, device="cuda"))
    before = got.clone()
    pos = torch.tensor([T, 2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    w.history_append_frame(0, pos, torch.ones(3, 3 * H * D, device="cuda"), got.kv, got.sc, H, block)
    assert w.status() == fsd.WAVE_EPOS and w.status() == fsd.WAVE_OK
    assert got.same(before)
    q = torch.ones(3, H, D, dtype=BF, device="cuda")
    out = torch.full_like(q, 7.0)
    w.history_attention_frame(0, pos, q, got.kv, got.sc, H, block, out)
    assert w.status() == fsd.WAVE_EPOS
    assert bool((out[:2] == 0).all()) and bool((out[2] == 7).all())
    pos[:2] = torch.tensor([8, -1])
    w.history_attention_frame(0, pos, q, got.kv, got.sc, H, block, out)
    assert bool((out[0] == 1).all()) and bool((out[1] == 0).all())
    _done(w)


@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("frame", [False, True])
def test_append_of_values_that_are_not_finite(block, frame):
    """They take no part in the scale: infinities saturate, NaN stays, the rest of the block keeps its precision."""
    H, D, T = 2, 64, 128
    w = _wave(H, D, S=1, T=T)
    n = 1 if frame else 40
    x = torch.randn(n, 3, H, D, generator=_gen(3), device="cuda")
    x[0, 1, 0, 3], x[0, 1, 0, 9], x[0, 2, 1, 63] = math.inf, -math.inf, math.nan
    if frame:
        x[0, 2, 0] = math.inf  # nothing finite at all
    else:
        x[17, 2, 0, 5], x[39, 1, 1] = math.nan, math.nan
    got = Cache(1, H, T, D, block)
    want = got.clone()
    if frame:
        w.history_append_frame(0, torch.zeros(1, dtype=torch.int32, device="cuda"), x.reshape(n, -1), got.kv, got.sc, H, block)
    else:
        w.history_append(0, [0, n], [0], [0], x.reshape(n, -1), got.kv, got.sc, H, block)
    want.write(0, 0, x[:, 1], x[:, 2])
    gk, wk = (c.kv.view(E4M3).float() for c in (got, want))
    assert torch.equal(gk.isnan(), wk.isnan()) and torch.equal(gk.nan_to_num(), wk.nan_to_num())
    assert torch.equal(got.sc.nan_to_num(nan=-7.0), want.sc.nan_to_num(nan=-7.0)) and bool((got.sc[..., 0] > 0).all())
    _done(w)


@pytest.mark.parametrize("block", [16, 64])
def test_scales_at_the_ends_of_fp32(block):
    """Largest magnitudes at and around 448 times a power of two, from the least numbers to the largest."""
    D = H = 64
    amax = torch.cat([(torch.tensor([448.0, 448.0 * (1 + 2.0 ** -23), 448.0 * (1 - 2.0 ** -24), 256.0, 447.9])[None] *
                       2.0 ** torch.tensor([-149.0, -135, -134, -126, -30, 0, 57, 100, 118])[:, None].double()).float().flatten(),
                      torch.tensor([3.4e38, 2.0 ** -149, 0.0])]).cuda()
    n = -(-amax.numel() // H) * H
    amax = torch.cat([amax, torch.ones(n - amax.numel(), device="cuda")]).reshape(-1, H)
    for row in amax:
        w = _wave(H, D, S=1, T=64)
        x = torch.rand(block, H, D, generator=_gen(1), device="cuda") * row[None, :, None]
        x[block // 2, :, 7] = -row
        got = Cache(1, H, 64, D, block)
        want = got.clone()
        w.history_append(0, [0, block], [0], [0], torch.stack([x, x, x], 1).reshape(block, -1), got.kv, got.sc, H, block)
        want.write(0, 0, x, x)
        assert got.same(want)
        _done(w)


@pytest.mark.parametrize("block", [1, 64])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("name", ["whole", "half turned", "parts"])
@pytest.mark.parametrize("frame", [False, True])
def test_append_of_rotated_rows(block, layout, name, frame):
    """The rotation's bound, and then the code's half step: 2^-4 relative, or 2^-10 of the scale below the normal range."""
    H, Hkv, D, T = 6, 3, 128, 256
    plan = _plan(name, layout, D)
    w = _wave(H, D, S=4, T=T)
    got = Cache(4, Hkv, T, D, block)
    if frame:
        starts, lens, slots = [0, 100, 255], [1, 1, 1], [0, 1, 2]
    else:
        starts, lens, slots = [5, 0, 99], [100, 1, 129], [2, 0, 1]
    for s, p in zip(slots, starts):
        if p:
            got.write(s, 0, 0.01 * torch.ones(p, Hkv, D, device="cuda"), 0.01 * torch.ones(p, Hkv, D, device="cuda"))
    cu = _cu(lens)
    qkv = (2 * torch.randn(cu[-1], (H + 2 * Hkv) * D, generator=_gen(6), device="cuda")).to(BF)
    q = torch.zeros(cu[-1], H, D, dtype=BF, device="cuda")
    if frame:
        w.history_append_frame(0, torch.tensor(starts, dtype=torch.int32, device="cuda"), qkv, got.kv, got.sc, Hkv, block, rope=plan, q=q)
    else:
        w.history_append(0, cu, slots, starts, qkv, got.kv, got.sc, Hkv, block, rope=plan, q=q)
    _done(w)
    x = qkv.reshape(cu[-1], H + 2 * Hkv, D)
    pos = [p + i for n, p in zip(lens, starts) for i in range(n)]
    ref, tol = turned(plan, pos, x[:, :H + Hkv])
    assert bool(((q.double() - ref[:, :H]).abs() <= tol[:, :H] + HALF[BF] * (ref[:, :H].abs() + tol[:, :H]) + TINY[BF]).all())
    for i, (n, slot, s0) in enumerate(zip(lens, slots, starts)):
        for which, rows, t in ((0, ref[:, H:], tol[:, H:]), (1, x[:, H + Hkv:].double(), torch.zeros_like(tol[:, H:]))):
            r, t = rows[cu[i]:cu[i + 1]].transpose(0, 1), t[cu[i]:cu[i + 1]].transpose(0, 1)
            back = got.values(which, slot, s0, s0 + n)
            per = torch.arange(s0, s0 + n, device="cuda") // block
            s = got.sc[0, which, slot][:, per, None].double()
            assert bool(((back - r).abs() <= t + 2.0 ** -4 * (r.abs() + t) + 2.0 ** -10 * s).all())
            # the scale: no larger than twice what the values need, no smaller than that
            most = torch.stack([r.abs()[:, per == b].amax((1, 2)) for b in per.unique()], -1)
            have = got.sc[0, which, slot][:, per.unique()].double()
            assert bool((most <= 448 * have * (1 + 2.0 ** -20)).all())
            assert bool((448 * have * (0.5 if block > 1 else 1.0) <= most.clamp(min=0.01) * (1 + 2.0 ** -20)).all())


@pytest.mark.parametrize("block", [16, 128])
def test_frames_leave_what_a_prompt_leaves(block):
    """Token by token and all at once: the same scales, and the same values but for codes that were encoded anew below the
    normal range (off by half a step there, 2^-10 of the scale, for each time)."""
    H, D, T, n = 2, 64, 128, 70
    x = torch.randn(n, 3 * H * D, generator=_gen(8), device="cuda") * 2.0 ** torch.linspace(-3, 3, n, device="cuda")[:, None]
    w = _wave(H, D, S=1, T=T)
    once, steps = Cache(1, H, T, D, block), Cache(1, H, T, D, block)
    plan = fsd.rope_plan(D)
    w.history_append(0, [0, n], [0], [0], x, once.kv, once.sc, H, block, rope=plan)
    for t in range(n):
        w.history_append_frame(0, torch.tensor([t], dtype=torch.int32, device="cuda"), x[t:t + 1], steps.kv, steps.sc, H, block, rope=plan)
    _done(w)
    assert torch.equal(once.sc.nan_to_num(nan=-7.0), steps.sc.nan_to_num(nan=-7.0))
    for which in (0, 1):
        a, b = once.values(which, 0, 0, n), steps.values(which, 0, 0, n)
        s = once.sc[0, which, 0].double()[:, torch.arange(n, device="cuda") // block, None]
        assert bool(((a - b).abs() <= 2.0 ** -9 * s).all()) and float((a != b).double().mean()) < 0.05


def test_append_of_blocks_of_one_is_the_steps():
    """V (not rotated) bit for bit as wave_prompt_append writes it; K within the two rotations' roundings."""
    H, D, T, n = 4, 128, 256, 200
    qkv = (3 * torch.randn(n, 3 * H * D, generator=_gen(11), device="cuda")).to(BF)
    w = _wave(H, D, S=2, T=T)
    a, b = Cache(2, H, T, D, 1), Cache(2, H, T, D, 1)
    w.prompt_append(0, [0, n], [1], [30], qkv, a.kv, a.sc)
    w.history_append(0, [0, n], [1], [30], qkv, b.kv, b.sc, H, 1, rope=fsd.rope_plan(D))
    _done(w)
    assert torch.equal(a.kv[:, 1], b.kv[:, 1]) and torch.equal(a.sc[:, 1].nan_to_num(nan=-7), b.sc[:, 1].nan_to_num(nan=-7))
    x, y = a.values(0, 1, 30, 30 + n), b.values(0, 1, 30, 30 + n)
    s = a.sc[0, 0, 1, :, 30:30 + n, None].double()
    assert bool(((x - y).abs() <= 2.0 ** -3 * x.abs() * (1 + 2.0 ** -10) + 2.0 ** -9 * s).all())  # a step of the code at most
    assert float((a.kv[0, 0, 1, :, 30:30 + n] != b.kv[0, 0, 1, :, 30:30 + n]).double().mean()) < 1e-3


@pytest.mark.parametrize("block", [1, 16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_read_back(block, D, dtype):
    Hkv, T, S = 3, 300, 4
    w = _wave(6, D, S=S, T=T, layers=2)
    c = Cache(S, Hkv, T, D, block, layers=2, layer=1)
    for s in range(S):
        c.write(s, 0, torch.randn(T, Hkv, D, generator=_gen(s), device="cuda"), torch.randn(T, Hkv, D, generator=_gen(9 + s), device="cuda"))
    lens, slots, starts = [1, 0, 150, 299], [2, 1, 0, 3], [299, 0, 70, 1]
    cu = _cu(lens, first=3)
    k, v = (torch.full((cu[-1] + 2, Hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    w.history_read(1, cu, slots, starts, c.kv, c.sc, Hkv, block, k, v)
    only = torch.zeros_like(v)
    w.history_read(1, cu, slots, starts, c.kv, c.sc, Hkv, block, v=only)
    for i, (n, slot, s0) in enumerate(zip(lens, slots, starts)):
        for which, got in ((0, k), (1, v)):
            assert torch.equal(got[cu[i]:cu[i + 1]], c.values(which, slot, s0, s0 + n, torch.float32).transpose(0, 1).to(dtype))
    assert torch.equal(only[cu[0]:cu[-1]], v[cu[0]:cu[-1]])
    for got in (k, v):
        assert bool((got[:cu[0]] == 7).all()) and bool((got[cu[-1]:] == 7).all())
    _done(w)


# ------------------------------------------------------------------- attention
def attention_reference(c, q, lens, slots, starts, cu, scale):
    """(out, the bound on |got - out|) in 64 bits.  With w the normalised weights, A = sum w |v| and s the scores: weights are
    rounded to fp16 (2^-11 A); scores carry at most (D + 8) fp32 roundings of their absolute sum, which enter a weight
    as a factor exp(2 ds); exponentials and sums 2^-18; a product's sums are cut to fp32 after each 16 keys (2^-23 of A
    each); the result is rounded once.  Weights below fp16's normal range are off by 2^-25 where the largest weight,
    times the largest V scale of its 128 slots, is 2^7 at least: 2^-32 of 448 times that a key.  Keys are brought to the
    largest scale of their 128 slots in fp16: off by 2^-25 2^-6 of it at most."""
    H, D = q.shape[1], q.shape[2]
    g = H // c.Hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for i, (n, slot, s0) in enumerate(zip(lens, slots, starts)):
        if not n or slot < 0:
            continue
        t = s0 + n
        kd, vd = (c.values(which, slot, 0, t).repeat_interleave(g, 0) for which in (0, 1))
        per = torch.arange(t, device=q.device)
        tops = []
        for which in (0, 1):
            sc = c.sc[c.layer, which, slot][:, per // c.block].double()
            pad = torch.nn.functional.pad(sc, (0, -t % 128)).reshape(c.Hkv, -1, 128).amax(-1)
            tops.append((2 * pad[:, per // 128]).repeat_interleave(g, 0)[:, None])  # a power of two above it
        qd = q[cu[i]:cu[i + 1]].double().transpose(0, 1)
        mask = per[None] > s0 + torch.arange(n, device=q.device)[:, None]
        s = ((qd @ kd.transpose(1, 2)) * scale).masked_fill(mask, -math.inf)
        w = torch.softmax(s, -1)
        o, A = w @ vd, w @ vd.abs()
        ds = (D + 8) * U * scale * (qd.abs() @ kd.abs().transpose(1, 2)) + 2.0 ** -31 * scale * qd.abs().sum(-1, keepdim=True) * tops[0]
        ds = ds.masked_fill(mask, 0.0).amax(-1, keepdim=True)
        lost = 2.0 ** -32 * 448 * (w * tops[1]).amax(-1, keepdim=True) * t
        out[cu[i]:cu[i + 1]] = o.transpose(0, 1)
        tol[cu[i]:cu[i + 1]] = (HALF[q.dtype] * o.abs() + (2.0 ** -11 + 2.0 * ds + 2.0 ** -18 + t / 16 * 2.0 ** -23) * A * 1.01 + lost
                                + TINY[q.dtype]).transpose(0, 1)
    return out, tol


def _history(lens, slots, starts, S, Hkv, D, block, seed=0, T=None, mag=None):
    """Sessions that hold their tokens and nothing behind them (NaN codes, and NaN scales of blocks that begin there)."""
    T = T or (max(n + s for n, s in zip(lens, starts)) + 3) // 4 * 4
    c = Cache(S, Hkv, T, D, block)
    for i, (n, slot, s0) in enumerate(zip(lens, slots, starts)):
        if slot < 0 or n + s0 == 0:
            continue
        k, v = (torch.randn(n + s0, Hkv, D, generator=_gen(seed * 1000 + 2 * i + j), device="cuda") for j in (0, 1))
        if mag is not None:
            v = v * mag(n + s0)
        c.write(slot, 0, 1.5 * k, v)
    return c


def _queries(n, H, D, dtype, seed=0):
    return (1.5 * torch.randn(n, H, D, generator=_gen(500 + seed), device="cuda")).to(dtype), torch.full((n, H, D), 7.0, dtype=dtype, device="cuda")


def _check(c, q, out, lens, slots, starts, cu, scale=None):
    ref, tol = attention_reference(c, q, lens, slots, starts, cu, q.shape[2] ** -0.5 if scale is None else scale)
    on = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for i, (n, slot) in enumerate(zip(lens, slots)):
        if slot >= 0:
            on[cu[i]:cu[i + 1]] = True
    worst = float(((out.double() - ref).abs() / tol)[on].max()) if bool(on.any()) else 0.0
    assert worst <= 1.0, worst
    assert bool((out[~on] == 7).all()), "rows outside every sequence are left as they were"


def _attend(lens, starts, H, Hkv, D, block, dtype, slots=None, seed=0, first=0, tail=0, scale=None, mag=None, frame=False):
    S = max(len(lens), 1)
    slots = [(3 * i + 1) % S if S % 3 else i for i in range(S)] if slots is None else slots
    if frame:
        slots = list(range(S))
    c = _history(lens, slots, starts, max(S, max(slots) + 1), Hkv, D, block, seed, mag=mag)
    cu = _cu(lens, first)
    q, out = _queries(cu[-1] + tail, H, D, dtype, seed)
    w = _wave(H, D, S=c.S, T=c.T)
    if frame:
        pos = torch.tensor(starts, dtype=torch.int32, device="cuda")
        w.history_attention_frame(0, pos, q, c.kv, c.sc, Hkv, block, out, scale=scale)
    else:
        w.history_attention(0, cu, slots, starts, q, c.kv, c.sc, Hkv, block, out, scale=scale)
    _done(w)
    _check(c, q, out, lens, slots, starts, cu, scale)
    return c, q, out


@pytest.mark.parametrize("lens,starts", [([1], [0]), ([1], [127]), ([1], [128]), ([2, 1], [126, 1000]), ([127], [1]), ([128], [128]), ([129], [127]),
                                         ([255, 256, 257], [1, 0, 255]), ([0, 5, 0, 64], [7, 300, 0, 77]), ([300, 1, 77, 13], [500, 900, 3, 130]),
                                         ([600], [1500]), ([33], [2100]), ([1] * 128, list(range(128))), ([20 + i for i in range(20)], [41 * i for i in range(20)])])
@pytest.mark.parametrize("D,dtype,block", [(128, BF, 64), (64, BF, 1), (128, F16, 1), (64, F16, 128), (128, BF, 16)])
def test_attention_lengths(lens, starts, D, dtype, block):
    _attend(lens, starts, 2, 2, D, block, dtype, seed=sum(lens), first=3, tail=2)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (6, 3), (8, 2), (5, 5), (32, 8), (7, 1), (48, 2), (16, 1), (24, 3)])
@pytest.mark.parametrize("D,block", [(64, 32), (128, 1)])
def test_attention_grouped_heads(H, Hkv, D, block):
    _attend([260, 3, 1, 131], [100, 400, 259, 0], H, Hkv, D, block, BF, seed=H)


@pytest.mark.parametrize("S", [1, 5, 80, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (12, 1), (40, 2)])
@pytest.mark.parametrize("D,block,dtype", [(128, 64, BF), (64, 16, F16), (128, 1, F16), (64, 1, BF), (64, 128, BF)])
def test_attention_of_frames(S, H, Hkv, D, block, dtype):
    """Single tokens: from an empty history to one that many CTAs share."""
    starts = [(i * 7919 + 3) % 900 for i in range(S)]
    starts[0] = 5000 if S < 80 else 1301
    if S > 4:
        starts[1:5] = [0, 15, 16, 127]
    _attend([1] * S, starts, H, Hkv, D, block, dtype, seed=S, frame=True)


@pytest.mark.parametrize("frame", [False, True])
def test_attention_of_a_long_history(frame):
    _attend([1] if frame else [40], [20000], 4, 2, 128, 128, BF, frame=frame)


def test_attention_empty_slots():
    """Frames: rows of empty slots are left as they were; prompts: sequences of no session."""
    H, Hkv, D, block = 4, 2, 128, 16
    starts = [40, -1, 0, -3, 200]
    c = _history([1] * 5, [0, -1, 2, -1, 4], starts, 5, Hkv, D, block)
    q, out = _queries(5, H, D, BF)
    w = _wave(H, D, S=5, T=c.T)
    w.history_attention_frame(0, torch.tensor(starts, dtype=torch.int32, device="cuda"), q, c.kv, c.sc, Hkv, block, out)
    _check(c, q, out, [1] * 5, [0, -1, 2, -1, 4], starts, _cu([1] * 5))
    out.fill_(7)
    w.history_attention_frame(0, torch.full((5,), -1, dtype=torch.int32, device="cuda"), q, c.kv, c.sc, Hkv, block, out)
    w.history_attention(0, [0, 5], [-1], [0], q, c.kv, c.sc, Hkv, block, out)
    w.history_attention(0, [0, 0, 0], [0, 1], [4, 9], q, c.kv, c.sc, Hkv, block, out)
    assert bool((out == 7).all())
    _done(w)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_slices_of_a_wider_row(frame, D):
    H, Hkv, block = 4, 2, 32
    lens, starts = ([1, 1], [70, 300]) if frame else ([200, 7], [77, 300])
    c, cu = _history(lens, [0, 1], starts, 2, Hkv, D, block), _cu(lens)
    wide = torch.randn(cu[-1] + 4, 3 * H, D, generator=_gen(1), device="cuda").to(BF)
    q, out = wide[:, :H], wide[:, H:2 * H]
    out.fill_(7)
    before = wide.clone()
    w = _wave(H, D, S=2, T=c.T)
    if frame:
        w.history_attention_frame(0, torch.tensor(starts, dtype=torch.int32, device="cuda"), q, c.kv, c.sc, Hkv, block, out)
    else:
        w.history_attention(0, cu, [0, 1], starts, q, c.kv, c.sc, Hkv, block, out)
    _done(w)
    _check(c, q, out, lens, [0, 1], starts, cu)
    assert torch.equal(wide[:, :H], before[:, :H]) and torch.equal(wide[:, 2 * H:], before[:, 2 * H:])


def _far(lo, hi):
    """V magnitudes from 2^lo to 2^hi, by runs of 40 tokens, with runs of zeros."""
    def mag(n):
        g = torch.Generator().manual_seed(n)
        e = torch.randint(lo, hi + 1, (n // 40 + 1,), generator=g).repeat_interleave(40)[:n]
        m = torch.ldexp(torch.ones(n), e)
        m[(torch.arange(n) // 40) % 5 == 2] = 0.0
        return m.cuda()[:, None, None]
    return mag


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [1, 16, 128])
@pytest.mark.parametrize("lo,hi", [(-6, 6), (-40, 40), (-100, -60), (60, 90)])
def test_attention_values_of_many_magnitudes(frame, block, lo, hi):
    """V scales that differ by many powers of two, and blocks of zeros.  The output type is bf16: fp16 ends before 2^40."""
    _attend([1, 1, 1] if frame else [150, 1, 30], [500, 39, 1100] if frame else [300, 39, 1100], 4, 2, 64, block, BF, mag=_far(lo, hi), frame=frame)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [1, 32])
@pytest.mark.parametrize("scale", [1e-6, 3.0])
def test_attention_scales(frame, block, scale):
    _attend([1, 1] if frame else [130, 9], [300, 5], 4, 4, 64, block, BF, scale=scale, frame=frame)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("mag", [1e-30, 1e-7, 1e4, 1e30])
def test_attention_queries_of_any_magnitude(frame, mag):
    """bf16 queries far outside fp16's range, with a scale that keeps the scores moderate; one row of zeros."""
    H, Hkv, D, block = 4, 2, 128, 64
    lens, starts = ([1, 1, 1], [300, 17, 900]) if frame else ([100, 1, 3], [300, 17, 900])
    c, cu = _history(lens, [0, 1, 2], starts, 3, Hkv, D, block), _cu(lens)
    q, out = _queries(cu[-1], H, D, BF)
    q = (q.float() * mag).to(BF)
    q[1] = 0
    q[0, :, 7] *= 2.0 ** -12
    w = _wave(H, D, S=3, T=c.T)
    scale = D ** -0.5 / mag
    if frame:
        w.history_attention_frame(0, torch.tensor(starts, dtype=torch.int32, device="cuda"), q, c.kv, c.sc, Hkv, block, out, scale=scale)
    else:
        w.history_attention(0, cu, [0, 1, 2], starts, q, c.kv, c.sc, Hkv, block, out, scale=scale)
    _done(w)
    _check(c, q, out, lens, [0, 1, 2], starts, cu, scale)


@pytest.mark.parametrize("block", [1, 16, 128])
@pytest.mark.parametrize("D,group", [(128, 1), (64, 4), (128, 3)])
@pytest.mark.parametrize("lens", [[150, 1, 300], [4, 2, 3]])
def test_attention_of_values_that_are_not_finite(block, D, group, lens):
    """NaN codes reach exactly the rows that attend to them: in K every head of the group and value, in V the value."""
    Hkv = 2
    H, starts = Hkv * group, [130, 700, 40]
    c = _history(lens, [0, 1, 2], starts, 3, Hkv, D, block, seed=4)
    cu = _cu(lens)
    q, out = _queries(cu[-1], H, D, BF)
    ref, tol = attention_reference(c, q, lens, [0, 1, 2], starts, cu, D ** -0.5)
    nan = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    # session 0: a V value of head 0 at its second new token; session 1: one of head 1 long ago; session 2: a K row of
    # head 1 and V values of head 0 at its last token but one
    c.kv[0, 1, 0, 0, starts[0] + 1, 5] = 0xFF
    nan[cu[0] + 1:cu[1], :group, 5] = True
    c.kv[0, 1, 1, 1, 300, D - 1] = 0x7F
    nan[cu[1]:cu[2], group:, D - 1] = True
    c.kv[0, 0, 2, 1, starts[2] + lens[2] - 2, 3] = 0x7F
    nan[cu[3] - 2:cu[3], group:] = True
    c.kv[0, 1, 2, 0, starts[2] + lens[2] - 2, ::7] = 0x7F
    nan[cu[3] - 2:cu[3], :group, ::7] = True
    w = _wave(H, D, S=3, T=c.T)
    w.history_attention(0, cu, [0, 1, 2], starts, q, c.kv, c.sc, Hkv, block, out)
    _done(w)
    assert torch.equal(out.isnan(), nan)
    assert bool(((out.double() - ref).abs() <= tol)[~nan].all())


def test_attention_of_a_history_beyond_32_bits():
    """Codes beyond 2^32 bytes and scales beyond 2^31 of them."""
    H, D, T, S = 32, 128, 9000, 64
    c = Cache(S, H, T, D, 1)
    assert c.kv.numel() > 2 ** 32
    lens, slots, starts = [3, 1], [63, 62], [8990, 8000]
    for slot, n in zip(slots, (8993, 8001)):
        c.write(slot, 0, *(torch.randn(n, H, D, generator=_gen(slot + j), device="cuda") for j in (0, 1)))
    cu = _cu(lens)
    q, out = _queries(cu[-1], H, D, BF)
    w = _wave(H, D, S=S, T=T)
    w.history_attention(0, cu, slots, starts, q, c.kv, c.sc, H, 1, out)
    _check(c, q, out, lens, slots, starts, cu)
    pos = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    pos[63] = 8992
    qf, of = _queries(S, H, D, BF)
    qf[63] = q[2]
    w.history_attention_frame(0, pos, qf, c.kv, c.sc, H, 1, of)
    _check(c, qf, of, [1], [63], [8992], [63, 64])
    # append and read at the far end
    x = torch.randn(2, 3 * H * D, generator=_gen(5), device="cuda")
    w.history_append(0, [0, 2], [63], [8996], x, c.kv, c.sc, H, 1)
    k = torch.zeros(2, H, D, device="cuda")
    w.history_read(0, [0, 2], [63], [8996], c.kv, c.sc, H, 1, k)
    assert torch.equal(k, c.values(0, 63, 8996, 8998, torch.float32).transpose(0, 1))
    want = x.reshape(2, 3, H, D)[:, 1].double()
    assert bool(((k.double() - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * want.abs().amax(-1, keepdim=True) / 448).all())
    _done(w)


@pytest.mark.parametrize("block,Hkv", [(1, 4), (64, 2)])
def test_a_session_from_prompt_to_frames(block, Hkv):
    """A prompt, a second one that goes on, then frames replayed from one captured graph: the history holds what appending
    all at once leaves, and each attention is the formula's over it."""
    H, D, T, n1, n2, frames = 4, 128, 256, 90, 70, 9
    plan = fsd.rope_plan(D, layout="interleaved", scaling="parts", factor=4.0, original=64.0)
    x = torch.randn(n1 + n2 + frames, (H + 2 * Hkv) * D, generator=_gen(2), device="cuda")
    w = _wave(H, D, S=2, T=T)
    c, whole = Cache(2, Hkv, T, D, block), Cache(2, Hkv, T, D, block)
    q, out = torch.zeros(len(x), H, D, dtype=BF, device="cuda"), torch.full((len(x), H, D), 7.0, dtype=BF, device="cuda")
    for a, n in ((0, n1), (n1, n2)):
        cu = [a, a + n]
        w.history_append(0, cu, [1], [a], x, c.kv, c.sc, Hkv, block, rope=plan, q=q)
        w.history_attention(0, cu, [1], [a], q, c.kv, c.sc, Hkv, block, out)
        _check(c, q[a:a + n], out[a:a + n], [n], [1], [a], [0, n])
    # the frames: slot 0 is empty, slot 1 goes on
    fx, fq, fo = torch.zeros(2, x.shape[1], device="cuda"), torch.zeros(2, H, D, dtype=BF, device="cuda"), torch.full((2, H, D), 7.0, dtype=BF, device="cuda")
    pos = torch.tensor([-1, n1 + n2], dtype=torch.int32, device="cuda")
    spare = c.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # once outside the graph, on a copy
        w.history_append_frame(0, pos, fx, spare.kv, spare.sc, Hkv, block, rope=plan, q=fq)
        w.history_attention_frame(0, pos, fq, spare.kv, spare.sc, Hkv, block, fo)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.history_append_frame(0, pos, fx, c.kv, c.sc, Hkv, block, rope=plan, q=fq)
        w.history_attention_frame(0, pos, fq, c.kv, c.sc, Hkv, block, fo)
    for f in range(frames):
        fx[1] = x[n1 + n2 + f]
        g.replay()
        p = n1 + n2 + f
        _check(c, fq, fo, [1], [1], [p], [1, 2])
        pos[1] += 1
    w.history_append(0, [0, len(x)], [1], [0], x, whole.kv, whole.sc, Hkv, block, rope=plan)
    assert torch.equal(whole.sc.nan_to_num(nan=-7), c.sc.nan_to_num(nan=-7))
    for which in (0, 1):
        a, b = whole.values(which, 1, 0, len(x)), c.values(which, 1, 0, len(x))
        s = whole.sc[0, which, 1].double()[:, torch.arange(len(x), device="cuda") // block, None]
        assert bool(((a - b).abs() <= 2.0 ** -9 * s).all())
    _done(w)


def test_a_prompt_that_goes_on_over_the_steps_history():
    """History written by wave_prompt_append, read by the block calls: the second half of a prompt attends as the whole does."""
    H, D, T, n = 4, 64, 512, 400
    qkv = torch.randn(n, 3 * H * D, generator=_gen(12), device="cuda")
    q, k, v, whole = (torch.zeros(n, H, D, dtype=F16, device="cuda") for _ in range(4))
    w = _wave(H, D, S=2, T=T)
    c = Cache(2, H, T, D, 1)
    w.prompt_append(0, [0, n], [1], [0], qkv, c.kv, c.sc, q, k, v)
    w.prompt_attention([0, n], q, k, v, whole)
    out = torch.full((n, H, D), 7.0, dtype=F16, device="cuda")
    w.history_attention(0, [150, n], [1], [150], q, c.kv, c.sc, H, 1, out)
    _done(w)
    ref, tol = attention_reference(c, q, [n - 150], [1], [150], [150, n], D ** -0.5)
    assert bool(((out.double() - ref).abs() <= tol)[150:].all()) and bool((out[:150] == 7).all())
    # prompt_attention takes k and v rounded to 16 bits: 2^-11 of each more
    qd, kd = q.double(), k.double()
    ds = 2.0 ** -11 * D ** -0.5 * float((qd.abs().amax((0, 1)) * kd.abs().amax((0, 1))).sum())
    assert bool(((out.double() - whole.double()).abs() <= 2 * tol + (2.0 ** -11 + 2 * ds) * v.double().abs().amax())[150:].all())


def test_attention_is_the_same_every_time():
    """Bit for bit, alone on the GPU and beside other work."""
    for frame, lens, starts in ((False, [300, 2, 77], [900, 2000, 0]), (True, [1] * 30, [(i * 7919) % 3000 for i in range(30)])):
        slots = list(range(len(lens)))
        c, cu = _history(lens, slots, starts, len(lens), 2, 128, 64), _cu(lens)
        q, out = _queries(cu[-1], 8, 128, BF)
        w = _wave(8, 128, S=len(lens), T=c.T)
        pos = torch.tensor(starts, dtype=torch.int32, device="cuda")
        busy = torch.randn(4096, 4096, device="cuda")
        side, first = torch.cuda.Stream(), None
        for k in range(6):
            if k % 2:
                with torch.cuda.stream(side):
                    busy @ busy
            o = torch.full_like(out, 7.0)
            if frame:
                w.history_attention_frame(0, pos, q, c.kv, c.sc, 2, 64, o)
            else:
                w.history_attention(0, cu, slots, starts, q, c.kv, c.sc, 2, 64, o)
            torch.cuda.synchronize()
            first = o if first is None else first
            assert torch.equal(first, o)
        _done(w)


def test_work_on_another_stream():
    """Calls follow the stream that they are given: appended and attended to on a side stream, behind its own work."""
    H, Hkv, D, n = 8, 2, 64, 300
    w = _wave(H, D, S=1, T=n + 4)
    c, want = Cache(1, Hkv, n + 4, D, 32), Cache(1, Hkv, n + 4, D, 32)
    src = torch.randn(n, (H + 2 * Hkv) * D, generator=_gen(1), device="cuda")
    x, q = torch.zeros_like(src), torch.zeros(n, H, D, dtype=BF, device="cuda")
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.copy_(src)
        w.history_append(0, [0, n], [0], [0], x, c.kv, c.sc, Hkv, 32, q=q)
        w.history_attention(0, [0, n], [0], [0], q, c.kv, c.sc, Hkv, 32, out)
    torch.cuda.synchronize()
    _, k, v = _split(src, H, Hkv, D)
    want.write(0, 0, k, v)
    assert c.same(want)
    _check(c, q, out, [n], [0], [0], [0, n])
    _done(w)


def test_refusals():
    H, Hkv, D, T, S, block = 4, 2, 64, 64, 4, 16
    w = _wave(H, D, S=S, T=T)
    c = Cache(S, Hkv, T, D, block)
    q, out = _queries(8, H, D, BF)
    x, k = torch.zeros(8, (H + 2 * Hkv) * D, device="cuda"), torch.zeros(8, Hkv, D, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    rc = lambda f, *a, **kw: f(*a, check=False, **kw)  # noqa: E731
    for args, code in (((0, [0, 8], [4], [0]), fsd.WAVE_EINVAL), ((0, [0, 8], [0], [-1]), fsd.WAVE_EINVAL), ((1, [0, 8], [0], [0]), fsd.WAVE_EINVAL),
                       ((-1, [0, 8], [0], [0]), fsd.WAVE_EINVAL), ((0, [0, 4, 8], [1, 1], [0, 4]), fsd.WAVE_EINVAL), ((0, [0, 8], [0], [57]), fsd.WAVE_EPOS),
                       ((0, [8, 0], [0], [0]), fsd.WAVE_EINVAL), ((0, [0] * 130, [0] * 129, [0] * 129), fsd.WAVE_EINVAL)):
        assert rc(w.history_append, *args, x, c.kv, c.sc, Hkv, block) == code
        assert rc(w.history_read, *args, c.kv, c.sc, Hkv, block, k) == code
        assert rc(w.history_attention, *args, q, c.kv, c.sc, Hkv, block, out) == code
    assert rc(w.history_read, 0, [0, 8], [0], [0], c.kv, c.sc, Hkv, block) == fsd.WAVE_EINVAL
    for scale in (0.0, -1.0, math.nan, math.inf, 3e38):
        assert rc(w.history_attention, 0, [0, 8], [0], [0], q, c.kv, c.sc, Hkv, block, out, scale=scale) == fsd.WAVE_EINVAL
        assert rc(w.history_attention_frame, 0, pos, q, c.kv, c.sc, Hkv, block, out, scale=scale) == fsd.WAVE_EINVAL
    assert rc(w.history_append, 0, [0, 8], [0], [0], x.half(), c.kv, c.sc, Hkv, block) == fsd.WAVE_EINVAL
    assert rc(w.history_append, 0, [0, 8], [0], [0], x, c.kv, c.sc, Hkv, block, q=q.float()) == fsd.WAVE_EINVAL
    assert rc(w.history_append, 0, [0, 8], [0], [0], x, c.kv, c.sc, Hkv, block, rope=fsd.rope_plan(128)) == fsd.WAVE_EINVAL
    assert rc(w.history_attention, 0, [0, 8], [0], [0], q.float(), c.kv, c.sc, Hkv, block, out.float()) == fsd.WAVE_EINVAL
    wide = torch.zeros(8, H * D + 4, dtype=BF, device="cuda")
    assert rc(w.history_attention, 0, [0, 8], [0], [0], wide[:, :H * D].unflatten(1, (H, D)), c.kv, c.sc, Hkv, block, out) == fsd.WAVE_EINVAL
    off = torch.zeros(8 * H * D + 8, dtype=BF, device="cuda")[1:1 + 8 * H * D].view(8, H, D)
    assert rc(w.history_attention, 0, [0, 8], [0], [0], off, c.kv, c.sc, Hkv, block, out) == fsd.WAVE_EINVAL
    five = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert rc(w.history_attention_frame, 0, five, q, c.kv, c.sc, Hkv, block, out) == fsd.WAVE_EINVAL
    assert rc(w.history_append_frame, 0, five, x, c.kv, c.sc, Hkv, block) == fsd.WAVE_EINVAL
    for bad in (lambda: w.history_attention(0, [0, 8], [0], [0], q, c.kv[:, :, :3], c.sc, Hkv, block, out),
                lambda: w.history_attention(0, [0, 8], [0], [0], q, c.kv, c.sc[..., :3], Hkv, block, out),
                lambda: w.history_attention(0, [0, 8], [0], [0], q, c.kv, c.sc.double(), Hkv, block, out),
                lambda: w.history_attention(0, [0, 8], [0], [0], q, c.kv.cpu(), c.sc, Hkv, block, out),
                lambda: w.history_attention(0, [0, 8], [0], [0], q.cpu(), c.kv, c.sc, Hkv, block, out),
                lambda: w.history_attention_frame(0, pos.long(), q, c.kv, c.sc, Hkv, block, out),
                lambda: w.history_append_frame(0, pos.cpu(), x, c.kv, c.sc, Hkv, block)):
        with pytest.raises(ValueError):
            bad()
    assert bool((out == 7).all()) and bool((c.kv == 0x7F).all())
    _done(w)


@pytest.mark.parametrize("lens,starts,H,Hkv", [([300] * 20, [40 * i for i in range(20)], 8, 8), ([200, 1, 40, 3, 16, 33, 900], [0, 5, 700, 90, 300, 2, 1], 8, 4),
                                               ([5, 6, 7, 8, 9, 1], [300] * 6, 16, 4)])
@pytest.mark.parametrize("D,block", [(128, 1), (64, 64)])
def test_attention_of_few_and_many_rows_together(lens, starts, H, Hkv, D, block):
    """More units than SMs; prompts of few rows, of two tiles of them and of many in one call; and each alone, within the bounds."""
    c, q, out = _attend(lens, starts, H, Hkv, D, block, F16, seed=7, first=1, tail=1)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("block", [16, 128])
def test_attention_of_scales_that_are_no_powers_of_two(frame, block):
    """A history filled by other means: K's and V's scales are then taken to fp16's 11 bits, and so are their products with a
    code (2^-11 of a key or a value each)."""
    H, Hkv, D = 4, 2, 64
    lens, starts = ([1, 1], [300, 1000]) if frame else ([150, 40], [300, 1000])
    c, cu = _history(lens, [0, 1], starts, 2, Hkv, D, block), _cu(lens)
    c.sc *= 0.5 + torch.rand(c.sc.shape, generator=_gen(1), device="cuda")
    q, out = _queries(cu[-1], H, D, BF)
    w = _wave(H, D, S=2, T=c.T)
    if frame:
        w.history_attention_frame(0, torch.tensor(starts, dtype=torch.int32, device="cuda"), q, c.kv, c.sc, Hkv, block, out)
    else:
        w.history_attention(0, cu, [0, 1], starts, q, c.kv, c.sc, Hkv, block, out)
    _done(w)
    ref, tol = attention_reference(c, q, lens, [0, 1], starts, cu, D ** -0.5)
    g = H // Hkv
    for i, (n, s0) in enumerate(zip(lens, starts)):
        kd, vd = (c.values(which, i, 0, s0 + n).repeat_interleave(g, 0) for which in (0, 1))
        qd = q[cu[i]:cu[i + 1]].double().transpose(0, 1)
        later = torch.arange(s0 + n, device="cuda")[None] > s0 + torch.arange(n, device="cuda")[:, None]
        s = ((qd @ kd.transpose(1, 2)) * D ** -0.5).masked_fill(later, -math.inf)
        A = torch.softmax(s, -1) @ vd.abs()
        ds = 2 * 2.0 ** -11 * D ** -0.5 * (qd.abs() @ kd.abs().transpose(1, 2)).masked_fill(later, 0.0).amax(-1, keepdim=True)
        tol[cu[i]:cu[i + 1]] += ((2 * ds + 2 * 2.0 ** -11) * A * 1.02).transpose(0, 1)
    assert bool(((out.double() - ref).abs() <= tol).all())


def test_history_of_a_hybrid_handle():
    """The layer is the model's: an attention block's; others are refused."""
    cfg = fsd.WaveHybridConfig(6, 64, 3, 2, 64, 4, 64, 128, 1e-5, 1e4)
    w = fsd.HybridWave(cfg, 2, 64)
    H, D, n, block = 2, 64, 20, 16
    got = Cache(2, H, 64, D, block, layers=2, layer=1)
    want = got.clone()
    x = torch.randn(n, 3 * H * D, generator=_gen(1), device="cuda")
    for layer in (0, 1, 3, 4, 6):
        assert w.history_append(layer, [0, n], [1], [0], x, got.kv, got.sc, H, block, check=False) == fsd.WAVE_EINVAL
    q = torch.zeros(n, H, D, dtype=BF, device="cuda")
    w.history_append(5, [0, n], [1], [0], x, got.kv, got.sc, H, block, q=q)
    _, k, v = _split(x, H, H, D)
    want.write(1, 0, k, v)
    assert got.same(want)
    out = torch.zeros_like(q)
    w.history_attention(5, [0, n], [1], [0], q, got.kv, got.sc, H, block, out)
    _check(got, q, out, [n], [1], [0], [0, n])
    _done(w)


def test_append_of_128_sequences():
    H, Hkv, D, T, block = 2, 1, 64, 64, 16
    lens, starts, slots = [1 + i % 23 for i in range(128)], [(7 * i) % 30 for i in range(128)], [(i * 37) % 128 for i in range(128)]
    w = _wave(H, D, S=128, T=T)
    got = Cache(128, Hkv, T, D, block)
    for s, p in zip(slots, starts):
        if p:
            got.write(s, 0, torch.ones(p, Hkv, D, device="cuda"), torch.ones(p, Hkv, D, device="cuda"))
    want, cu = got.clone(), _cu(lens)
    x = (4 * torch.randn(cu[-1], (H + 2 * Hkv) * D, generator=_gen(3), device="cuda")).to(BF)
    w.history_append(0, cu, slots, starts, x, got.kv, got.sc, Hkv, block)
    _, k, v = _split(x, H, Hkv, D)
    for i, (n, s, p) in enumerate(zip(lens, slots, starts)):
        want.write(s, p, k[cu[i]:cu[i + 1]], v[cu[i]:cu[i + 1]])
    assert got.same(want)
    _done(w)


@pytest.mark.parametrize("index", [0, 1, 5])
@pytest.mark.parametrize("block", [1, 128])
def test_attention_whose_tiles_do_not_come(index, block):
    """The conversion ends before a tile: the waits run out, the launch ends, the status says so once, and the next call on
    the handle is right."""
    H, Hkv, D = 4, 2, 128
    lens, starts = [300, 200], [500, 0]
    c, cu = _history(lens, [0, 1], starts, 2, Hkv, D, block), _cu(lens)
    q, out = _queries(cu[-1], H, D, BF)
    w = _wave(H, D, S=2, T=c.T)
    call = lambda: w.history_attention(0, cu, [0, 1], starts, q, c.kv, c.sc, Hkv, block, out)  # noqa: E731
    call()
    assert w.status() == fsd.WAVE_OK
    w.set_timeout_ns(20_000_000)
    w.debug_skip_signal(11, index)
    call()
    assert w.status() == fsd.WAVE_ETIMEOUT and w.status() == fsd.WAVE_OK
    w.debug_skip_signal(11, -1)
    out.fill_(7)
    call()
    _check(c, q, out, lens, [0, 1], starts, cu)
    w.set_timeout_ns(1)  # no wait gets any time
    call()
    assert w.status() == fsd.WAVE_ETIMEOUT
    w.set_timeout_ns(2_000_000_000)
    out.fill_(7)
    call()
    _check(c, q, out, lens, [0, 1], starts, cu)
    _done(w)


def test_calls_replayed_from_graphs_that_share_a_handle():
    """Two captured calls of one handle, of few and of many rows, replayed one after another and in either order."""
    H, Hkv, D, block = 8, 2, 128, 64
    lens, starts = [[1] * 3, [200, 3, 60]], [[700, 5, 2000], [300, 900, 0]]
    cs = [_history(n, [0, 1, 2], s, 3, Hkv, D, block, seed=i, T=2004) for i, (n, s) in enumerate(zip(lens, starts))]
    w = _wave(H, D, S=3, T=2004)
    qs = [_queries(sum(n), H, D, BF, seed=i) for i, n in enumerate(lens)]
    graphs = []
    for (q, out), c, n, s in zip(qs, cs, lens, starts):
        call = lambda: w.history_attention(0, _cu(n), [0, 1, 2], s, q, c.kv, c.sc, Hkv, block, out)  # noqa: E731
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1, 0)):
        for q, out in qs:
            out.fill_(7)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            _check(cs[i], qs[i][0], qs[i][1], lens[i], [0, 1, 2], starts[i], _cu(lens[i]))
    _done(w)


@pytest.mark.parametrize("frame", [False, True])
@pytest.mark.parametrize("D,block", [(64, 128), (128, 1), (128, 16)])
def test_attention_of_one_head_shared_by_128(frame, D, block):
    """The largest group: a tile of 128 rows is one token; a frame has 8 row tiles to a head."""
    if frame:
        _attend([1] * 5, [0, 700, 127, 16, 1300], 128, 1, D, block, BF, seed=5, frame=True)
    else:
        _attend([3, 1, 70], [300, 0, 129], 128, 1, D, block, BF, seed=6)


@pytest.mark.parametrize("D,block", [(128, 128), (64, 128), (128, 1)])
def test_a_captured_prompt(D, block):
    """Append, attention and read back of packed prompts captured into one graph, the first use of the handle, and
    replayed with other inputs: the history, the outputs and what is read back follow them."""
    H, Hkv, lens, slots, starts = 4, 2, [200, 3], [1, 0], [0, 0]
    cu, T = _cu(lens), 204
    w = _wave(H, D, S=2, T=T)
    plan = fsd.rope_plan(D)
    c = Cache(2, Hkv, T, D, block)
    x = torch.zeros(cu[-1], (H + 2 * Hkv) * D, device="cuda")
    q, out = torch.zeros(cu[-1], H, D, dtype=F16, device="cuda"), torch.zeros(cu[-1], H, D, dtype=F16, device="cuda")
    k = torch.zeros(cu[-1], Hkv, D, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.history_append(0, cu, slots, starts, x, c.kv, c.sc, Hkv, block, rope=plan, q=q)
        w.history_attention(0, cu, slots, starts, q, c.kv, c.sc, Hkv, block, out)
        w.history_read(0, cu, slots, starts, c.kv, c.sc, Hkv, block, k)
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=_gen(seed), device="cuda"))
        want = Cache(2, Hkv, T, D, block)
        w.history_append(0, cu, slots, starts, x, want.kv, want.sc, Hkv, block, rope=plan)
        g.replay()
        torch.cuda.synchronize()
        assert c.same(want)
        _check(c, q, out, lens, slots, starts, cu)
        for i, (n, slot) in enumerate(zip(lens, slots)):
            assert torch.equal(k[cu[i]:cu[i + 1]].transpose(0, 1), c.values(0, slot, 0, n, torch.float32))
    _done(w)
