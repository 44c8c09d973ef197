"""Sessions from prompts on the GPU: prompt append, prompt attention, the
selective-state block over prompts and session copies, each against a plain
64-bit restatement, with bounds derived from the roundings each one makes."""
import math

import numpy as np
import pytest
import torch

import frame_step_decode_gb300 as fsd

pytestmark = pytest.mark.gpu

P, N = 64, 128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
U = 2.0 ** -24                                                 # the same of fp32
# half a step below the normal range, absolute: fp16's spacing there is 2^-24, bf16's is under 2^-130
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def _cu(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _wave(heads, dim, S=8, T=64, layers=1):
    return fsd.Wave(fsd.WaveConfig(layers, 64, heads, dim, 64, 1e-5, 1e4), S, T)


def _hybrid(state_heads, S=8, T=64, layers=2, every=2, heads=1, dim=64):
    cfg = fsd.WaveHybridConfig(layers, 64, every, heads, dim, state_heads, P, N, 1e-5, 1e4)
    return cfg, fsd.HybridWave(cfg, S, T)


# ------------------------------------------------------------------ attention
def attention_reference(q, k, v, cu, scale):
    """(out, the bound on |got - out|) in 64 bits.  With w the normalised
    weights, A = sum w |v| and s the scores: the weights are rounded to the
    16-bit type (half a step each: half * A), scores carry at most (D + 8)
    fp32 roundings of their absolute sum, which enter a weight as a factor
    exp(2 ds), the exponential and the two running sums a few more, and the
    result is rounded once (half * |out|).  A weight or result below the
    type's normal range is off by up to TINY instead of half a relative step:
    the largest weight is at least 1 before it is divided by the sum, so
    TINY * (1 + sum |v|) covers them."""
    D, half = q.shape[2], HALF[q.dtype]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    g = q.shape[1] // k.shape[1]
    for a, b in zip(cu, cu[1:]):
        if a == b:
            continue
        qd = q[a:b].double().transpose(0, 1)
        kd = k[a:b].double().transpose(0, 1).repeat_interleave(g, 0)
        vd = v[a:b].double().transpose(0, 1).repeat_interleave(g, 0)
        mask = torch.ones(b - a, b - a, dtype=torch.bool, device=q.device).triu(1)
        s = ((qd @ kd.transpose(1, 2)) * scale).masked_fill(mask, -math.inf)
        w = torch.softmax(s, -1)
        o = w @ vd
        A = w @ vd.abs()
        ds = (D + 8) * U * scale * (qd.abs() @ kd.abs().transpose(1, 2)).masked_fill(mask, 0.0).amax(-1, keepdim=True)
        out[a:b] = o.transpose(0, 1)
        # 2^-18: the exponential (2^-22) and (b - a)-term fp32 sums (random walks of U-sized errors)
        tol[a:b] = (half * o.abs() + (half + 2.0 * ds + 2.0 ** -18) * A * 1.01
                    + TINY[q.dtype] * (1 + (~mask).double() @ vd.abs())).transpose(0, 1)
    return out, tol


def _attention(lens, H, Hkv, D, dtype, seed=0, first=0, tail=0, scale=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu = _cu(lens, first)
    n = cu[-1] + tail
    mk = lambda h: torch.randn(n, h, D, generator=g, device="cuda")  # noqa: E731
    q, k, v = (1.5 * mk(H)).to(dtype), (1.5 * mk(Hkv)).to(dtype), mk(Hkv).to(dtype)
    return cu, q, k, v, torch.full((n, H, D), 7.0, dtype=dtype, device="cuda")


def _attend(cu, q, k, v, out, scale=None, **kw):
    w = _wave(q.shape[1], q.shape[2])
    try:
        w.prompt_attention(cu, q, k, v, out, scale=scale, **kw)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()


def _check_attention(cu, q, k, v, out, scale=None):
    ref, tol = attention_reference(q, k, v, cu, q.shape[2] ** -0.5 if scale is None else scale)
    a, b = cu[0], cu[-1]
    err = (out.double() - ref).abs()[a:b]
    worst = float((err / tol[a:b]).max()) if b > a else 0.0
    assert worst <= 1.0, worst
    assert bool((out[:a] == 7).all()) and bool((out[b:] == 7).all()), "rows outside every sequence are left as they were"


@pytest.mark.parametrize("lens", [[1], [2, 1], [127], [128], [129], [255, 256, 257], [0, 5, 0, 0, 64, 0], [300, 1, 1, 77, 513],
                                  [1025], [1] * 128, [40 + i for i in range(20)]])
@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.bfloat16), (128, torch.float16), (64, torch.float16)])
def test_attention_lengths(lens, D, dtype):
    case = _attention(lens, 2, 2, D, dtype, seed=sum(lens))
    _attend(*case)
    _check_attention(*case)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (6, 3), (8, 2), (5, 5), (32, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_grouped_heads(H, Hkv, D):
    case = _attention([260, 3, 131], H, Hkv, D, torch.bfloat16, seed=H)
    _attend(*case)
    _check_attention(*case)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_slices_of_a_wider_row(D):
    H, cu = 3, _cu([200, 77], first=5)
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(cu[-1] + 9, 4 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v, out = (wide[:, i * H:(i + 1) * H] for i in range(4))
    out.fill_(7)
    before = wide.clone()
    _attend(cu, q, k, v, out)
    _check_attention(cu, q, k, v, out)
    assert torch.equal(wide[:, :3 * H], before[:, :3 * H])


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_never_reads_what_a_row_does_not_attend_to(D, dtype, bad):
    """Non-finite rows before, between and behind the sequences and at later
    tokens of a sequence: the rows that do not attend to them stay exact."""
    lens = [150, 1, 300]
    cu, q, k, v, out = _attention(lens, 4, 2, D, dtype, seed=3, first=11, tail=13)
    for t in (q, k, v):
        t[:11] = bad
        t[cu[-1]:] = bad
    # the last token of sequence 0, tokens 130.. of sequence 2 (in K and V alike)
    k[cu[1] - 1], v[cu[1] - 1] = bad, bad
    k[cu[2] + 130:cu[3]], v[cu[2] + 130:cu[3], :, ::3] = bad, bad
    _attend(cu, q, k, v, out)
    fine = torch.zeros(out.shape[0], dtype=torch.bool)
    fine[cu[0]:cu[1] - 1] = True
    fine[cu[1]:cu[2] + 130] = True
    ref, tol = attention_reference(q[:cu[2] + 130], k[:cu[2] + 130], v[:cu[2] + 130],
                                   [cu[0], cu[1] - 1, cu[1], cu[2], cu[2] + 130][0:2], D ** -0.5)
    got = out.double()
    for a, b in ((cu[0], cu[1] - 1), (cu[1], cu[2]), (cu[2], cu[2] + 130)):
        ref, tol = attention_reference(q, k, v, [a, b], D ** -0.5)
        assert bool(((got - ref).abs()[a:b] <= tol[a:b]).all())
    assert not bool(torch.isfinite(out[cu[1] - 1]).all()), "the row that attends to them is not finite"
    assert not bool(torch.isfinite(out[cu[2] + 131]).all())
    assert bool((out[:11] == 7).all()) and bool((out[cu[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_non_finite_values_reach_the_rows_that_see_them(dtype):
    """V alone non-finite at one token (K finite): every later row of that
    head carries it, every other column and row is exact."""
    for at in (5, 130, 257, 299):
        cu, q, k, v, out = _attention([300], 2, 2, 128, dtype, seed=at)
        v[at, 1, 17], v[at, 1, 18] = float("inf"), float("nan")
        _attend(cu, q, k, v, out)
        clean = v.clone()
        clean[at] = 0
        ref, tol = attention_reference(q, k, clean, cu, 128 ** -0.5)
        ok = (out.double() - ref).abs() <= tol
        assert bool(ok[:at].all())
        assert bool(torch.isinf(out[at:, 1, 17]).all()) and bool((out[at:, 1, 17] > 0).all())
        assert bool(torch.isnan(out[at:, 1, 18]).all())
        assert bool(torch.isfinite(out[:, 0]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_wide_scores_and_scales(dtype):
    """Scores hundreds wide (one-hot rows), rising along the keys so that the
    running maximum moves in every block, and a large and a small scale."""
    cu, q, k, v, out = _attention([700], 2, 1, 64, dtype, seed=9)
    k *= torch.linspace(0.1, 8, 700, device="cuda")[:, None, None].to(dtype)
    for scale in (1.0, 0.125, 1e-3):
        out.fill_(7)
        _attend(cu, q, k, v, out, scale=scale)
        _check_attention(cu, q, k, v, out, scale=scale)


def test_attention_is_deterministic_and_replays():
    cu, q, k, v, out = _attention([513, 40, 1300], 4, 4, 128, torch.bfloat16, seed=2)
    w = _wave(4, 128)
    try:
        w.prompt_attention(cu, q, k, v, out)
        once = out.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            w.prompt_attention(cu, q, k, v, out)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.prompt_attention(cu, q, k, v, out)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, once)
        q.copy_(q.flip(0))  # the replay reads the buffers, not what they held
        graph.replay()
        assert w.status() == fsd.WAVE_OK
        _check_attention(cu, q, k, v, out)
    finally:
        w.close()


def test_attention_batches_of_every_size():
    """As many sequences as a call takes, and the last of them alone."""
    g = np.random.default_rng(3)
    lens = [int(n) for n in g.integers(0, 300, fsd.WAVE_MAX_SEQS)]
    cu, q, k, v, out = _attention(lens, 4, 2, 64, torch.bfloat16, seed=1, first=2, tail=3)
    _attend(cu, q, k, v, out)
    _check_attention(cu, q, k, v, out)
    one = torch.full_like(out, 7.0)
    _attend(cu[-2:], q, k, v, one)
    assert torch.equal(one[cu[-2]:cu[-1]], out[cu[-2]:cu[-1]])


@pytest.mark.parametrize("H,Hkv,D", [(16, 4, 64), (12, 12, 128)])
def test_attention_of_more_items_than_sms(H, Hkv, D):
    """Items beyond the SMs, eager, on two streams at once and replayed: the
    same bits whoever takes whose place."""
    lens = [int(n) for n in np.random.default_rng(H).integers(1, 700, 24)]
    cu, q, k, v, out = _attention(lens, H, Hkv, D, torch.bfloat16, seed=3)
    ws = [_wave(H, D) for _ in range(2)]
    outs = [torch.full_like(out, 7.0) for _ in range(2)]
    try:
        ws[0].prompt_attention(cu, q, k, v, out)
        graph, streams = torch.cuda.CUDAGraph(), [torch.cuda.Stream() for _ in range(2)]
        with torch.cuda.graph(graph, stream=streams[0]):
            ws[0].prompt_attention(cu, q, k, v, outs[0], stream=streams[0])
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            with torch.cuda.stream(streams[0]):
                graph.replay()
            ws[1].prompt_attention(cu, q, k, v, outs[1], stream=streams[1])
        torch.cuda.synchronize()
        assert ws[0].status() == fsd.WAVE_OK and ws[1].status() == fsd.WAVE_OK
    finally:
        for w in ws:
            w.close()
    _check_attention(cu, q, k, v, out)
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)


@pytest.mark.parametrize("lens,H,Hkv,D,dtype", [([2000], 1, 1, 128, torch.bfloat16), ([1500, 3, 900], 2, 1, 64, torch.float16),
                                                ([1281, 1, 640], 4, 4, 64, torch.bfloat16), ([3000, 129], 3, 1, 128, torch.float16),
                                                ([896, 897], 6, 2, 128, torch.bfloat16)])
def test_attention_of_few_rows_divides_the_keys(lens, H, Hkv, D, dtype):
    """Long prompts of few heads, whose keys are divided among CTAs and joined:
    strided, with rows outside, values that are not finite where no row may see
    them and where some do, eager and replayed."""
    cu, q, k, v, out = _attention(lens, H, Hkv, D, dtype, seed=7, first=3, tail=5)
    wide = torch.full((q.shape[0], H * D + 8), 7.0, dtype=dtype, device="cuda")
    out = wide[:, :H * D].unflatten(1, (H, D))
    k[:3], v[:3], k[cu[-1]:], v[cu[-1]:] = float("nan"), float("inf"), float("nan"), float("nan")
    w = _wave(H, D)
    try:
        w.prompt_attention(cu, q, k, v, out)
        assert w.status() == fsd.WAVE_OK
        _check_attention(cu, q, k, v, out)
        assert bool((wide[:, H * D:] == 7).all())
        once = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.prompt_attention(cu, q, k, v, out)
        wide[3:cu[-1]].fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, once)
        t = cu[0] + lens[0] * 2 // 3  # from this token on, not before
        v[t, 0, 5] = float("inf")
        w.prompt_attention(cu, q, k, v, out)
        assert w.status() == fsd.WAVE_OK
        own = out[:, :H // Hkv]
        assert torch.equal(own[:t], once[:t, :H // Hkv]) and not bool(torch.isfinite(own[t:cu[1], :, 5]).any())
        assert torch.equal(out[cu[1]:], once[cu[1]:]) and torch.equal(out[:, H // Hkv:], once[:, H // Hkv:])
        keep = [i for i in range(D) if i != 5]
        assert torch.equal(own[t:cu[1]][..., keep], once[t:cu[1], :H // Hkv][..., keep])
    finally:
        w.close()


def test_attention_offsets_beyond_32_bits():
    """Rows whose offsets in elements pass 2^31 (slices of a wide buffer)."""
    H, D, n = 32, 128, 176000
    cu = [n - 300, n - 170, n - 2]
    wide = torch.empty(n, 3 * H * D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(n, 2 * H * D, dtype=torch.bfloat16, device="cuda")[:, H * D:].unflatten(1, (H, D))
    g = torch.Generator(device="cuda").manual_seed(1)
    wide[cu[0]:] = torch.randn(300, 3 * H * D, generator=g, device="cuda").to(torch.bfloat16)
    out[cu[0]:] = 7
    q, k, v = (wide[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
    assert cu[0] * wide.stride(0) > 2 ** 31
    _attend(cu, q, k, v, out)
    tail = lambda t: t[cu[0]:].contiguous()  # noqa: E731
    _check_attention([0, 130, 298], tail(q), tail(k), tail(v), tail(out))


# --------------------------------------------------------------------- append
def rope64(x, pos, base=1e4):
    D = x.shape[-1]
    ang = pos.double()[:, None] * base ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=x.device) / D)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[..., :D // 2].double(), x[..., D // 2:].double()
    return torch.cat([a * c - b * s, a * s + b * c], -1)


@pytest.mark.parametrize("D,H", [(64, 1), (64, 6), (128, 5), (128, 32)])
@pytest.mark.parametrize("dtype,out_type", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float16)])
def test_append(D, H, dtype, out_type):
    lens, slots, starts = [37, 0, 1, 130, 5], [3, 1, 0, -1, 6], [0, 4, 171, 2, 9]
    S, T, L, layer = 7, 172, 2, 1
    cu = _cu(lens, first=3)
    g = torch.Generator(device="cuda").manual_seed(H)
    n = cu[-1] + 4
    wide = (2 * torch.randn(n, 3 * H * D + 8, generator=g, device="cuda")).to(dtype)
    qkv = wide[:, :3 * H * D]
    qkv[cu[0] + 1] = 0  # a zero row: zero codes, scale 0
    kv = torch.full((L, 2, S, H, T, D), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((L, 2, S, H, T), -3.0, device="cuda")
    q, k, v = (torch.full((n, H, D), 7.0, dtype=out_type, device="cuda") for _ in range(3))
    w = _wave(H, D, S, T, L)
    try:
        w.prompt_append(layer, cu, slots, starts, qkv, kv, sc, q, k, v)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    want_kv, want_sc = torch.full_like(kv, 0x55), torch.full_like(sc, -3.0)
    named = torch.zeros(n, dtype=torch.bool, device="cuda")
    for i, ln in enumerate(lens):
        if slots[i] < 0 or ln == 0:
            continue
        r = slice(cu[i], cu[i + 1])
        named[r] = True
        x = qkv[r].float().reshape(ln, 3, H, D)
        pos = starts[i] + torch.arange(ln, device="cuda")
        # V: bit for bit the library's own quantiser
        codes = torch.empty(ln, H, D, dtype=torch.uint8, device="cuda")
        scales = torch.empty(ln, H, device="cuda")
        fsd.kv_quantize(x[:, 2].contiguous(), codes, scales)
        want_kv[layer, 1, slots[i], :, pos] = codes.transpose(0, 1)
        want_sc[layer, 1, slots[i], :, pos] = scales.t()
        # K: the rotation carries three fp32 roundings of its two products
        # (and of the table's cos and sin), then the quantiser's half step
        k64 = rope64(x[:, 1], pos)
        mag = x[:, 1].double().abs().amax(-1, keepdim=True) * 2
        got_sc = sc[layer, 0, slots[i], :, pos].t().double()
        got = kv[layer, 0, slots[i], :, pos].transpose(0, 1).contiguous().view(torch.float8_e4m3fn).double() * got_sc[..., None]
        amax = k64.abs().amax(-1)
        assert bool(((got_sc * 448 - amax).abs() <= 6 * U * mag[..., 0] + 2 * U * amax).all())
        # half a step of e4m3: 2^-4 relative, 2^-10 of the scale below the normal range
        assert bool(((got - k64).abs() <= k64.abs() * 2.0 ** -4 * 1.001 + got_sc[..., None] * 2.0 ** -10 + 8 * U * mag).all())
        want_kv[layer, 0, slots[i], :, pos] = kv[layer, 0, slots[i], :, pos]
        want_sc[layer, 0, slots[i], :, pos] = sc[layer, 0, slots[i], :, pos]
        q64 = rope64(x[:, 0], pos)
        qmag = x[:, 0].double().abs().amax(-1, keepdim=True) * 2
        assert bool(((q[r].double() - q64).abs() <= HALF[out_type] * q64.abs() + 8 * U * qmag).all())
        # k, v read back: code * scale (one fp32 product) rounded once to the type, exactly
        for got16, plane in ((k, 0), (v, 1)):
            c = kv[layer, plane, slots[i], :, pos].transpose(0, 1).contiguous().view(torch.float8_e4m3fn).float()
            assert torch.equal(got16[r], (c * sc[layer, plane, slots[i], :, pos].t()[..., None]).to(out_type))
    assert torch.equal(kv, want_kv) and torch.equal(sc, want_sc), "only the named slots are written"
    for t in (q, k, v):
        assert bool((t[~named] == 7).all())


@pytest.mark.parametrize("D,H", [(64, 3), (64, 13), (128, 6), (128, 9)])
def test_append_of_many_tokens_equals_parts(D, H):
    """Heads that are no multiple of four, in one call of many tokens and in
    calls of few: the same bits."""
    S, T, L = 3, 1600, 1
    lens, starts = [1500, 1, 1203], [7, 1599, 0]
    cu = _cu(lens, first=2)
    g = torch.Generator(device="cuda").manual_seed(H)
    qkv = torch.randn(cu[-1], 3 * H * D, generator=g, device="cuda")
    got = []
    w = _wave(H, D, S, T, L)
    try:
        for parts in (1, 20):
            kv = torch.zeros(L, 2, S, H, T, D, dtype=torch.uint8, device="cuda")
            sc = torch.zeros(L, 2, S, H, T, device="cuda")
            q, k, v = (torch.zeros(cu[-1], H, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
            if parts == 1:
                w.prompt_append(0, cu, [0, 1, 2], starts, qkv, kv, sc, q, k, v)
            else:
                for s in range(3):
                    for a in range(0, lens[s], 100):
                        b = min(lens[s], a + 100)
                        w.prompt_append(0, [cu[s] + a, cu[s] + b], [s], [starts[s] + a], qkv, kv, sc, q, k, v)
            got.append((kv, sc, q, k, v))
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_append_rounds_its_quotients_as_a_division_does():
    """Values a few units in the last place around every midpoint of two codes
    (where a quotient that is not rounded as the division rounds it would give
    the other code), at scales from tiny to huge, zeros, infinities and NaN:
    V's codes and scales are the library's quantiser's, bit for bit."""
    H, D, S = 2, 128, 1
    codes = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2
    g = np.random.default_rng(4)
    rows = []
    for top in np.concatenate([g.uniform(0.5, 2.0, 60) * 2.0 ** g.integers(-20, 20, 60), 2.0 ** np.arange(-148.0, 125.0, 3.0)]):
        scale = np.float32(np.float32(top) / np.float32(448.0))
        v = (mid.numpy() * float(scale)).astype(np.float32)  # 126 midpoints
        v = (v.view(np.int32) + g.integers(-4, 5, v.shape).astype(np.int32) * (v != 0)).view(np.float32)
        v = np.concatenate([v, [np.float32(top), 0.0]]).astype(np.float32) * np.where(g.random(128) < 0.5, -1, 1).astype(np.float32)
        rows.append(np.clip(np.nan_to_num(v), -abs(np.float32(top)), abs(np.float32(top))))
    rows += [np.zeros(128, np.float32), -np.zeros(128, np.float32)]
    for bad in (np.inf, -np.inf, np.nan):
        r = rows[3].copy()
        r[5] = bad
        rows.append(r)
    v = torch.from_numpy(np.stack(rows + rows[:len(rows) % 2])).cuda().reshape(-1, H, D)
    n = v.shape[0]
    T = (n + 3) // 4 * 4
    qkv = torch.cat([torch.zeros(n, 2 * H * D, device="cuda"), v.reshape(n, H * D)], 1)
    kv = torch.zeros(1, 2, S, H, T, D, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(1, 2, S, H, T, device="cuda")
    w = _wave(H, D, S, T)
    try:
        w.prompt_append(0, [0, n], [0], [0], qkv, kv, sc)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    want, want_sc = torch.empty(n, H, D, dtype=torch.uint8, device="cuda"), torch.empty(n, H, device="cuda")
    fsd.kv_quantize(v.contiguous(), want, want_sc)
    assert torch.equal(kv[0, 1, 0, :, :n].transpose(0, 1), want)
    assert torch.equal(sc[0, 1, 0, :, :n].t().contiguous().view(torch.int32), want_sc.view(torch.int32))


def test_append_equals_the_steps_own_append():
    """The rows that a step quantises (its pre-quantisation dump: k rotated,
    v) give, appended as a prompt's v rows, the codes the step wrote."""
    from gpu_case import DeviceCase
    import synth
    w = synth.TINY
    case = DeviceCase(w)
    wave = fsd.Wave(case.cfg, case.S_max, w.T_max)
    L, H, D, S = w.n_layers, w.n_heads, w.head_dim, case.S
    dump = torch.zeros((L, 2, S, H, D), device="cuda")
    try:
        wave.debug_dump_kv(dump)
        case.step(wave)
        assert wave.status() == fsd.WAVE_OK
        kv, sc = torch.zeros_like(case.kv), torch.zeros_like(case.sc)
        for l in range(L):
            rows = torch.cat([torch.zeros(S, H * D, device="cuda"), torch.zeros(S, H * D, device="cuda"),
                              dump[l, 1].reshape(S, H * D)], 1)
            wave.prompt_append(l, list(range(S + 1)), list(range(S)), case.pos_h.tolist(), rows, kv, sc)
        assert wave.status() == fsd.WAVE_OK
    finally:
        wave.close()
    for s, pos in enumerate(case.pos_h.tolist()):
        assert torch.equal(kv[:, 1, s, :, pos], case.kv[:, 1, s, :, pos])
        assert torch.equal(sc[:, 1, s, :, pos], case.sc[:, 1, s, :, pos])


@pytest.mark.parametrize("D", [64, 128])
def test_append_many_sessions_far_into_the_history(D):
    """A batch of 128 sessions, replayed from a graph on a stream of its own,
    into a history whose offsets pass 32 bits: equal to a session at a time."""
    S, H, T = 128, 32, 4100 * 128 // D
    g = torch.Generator(device="cuda").manual_seed(D)
    lens = [int(n) for n in np.random.default_rng(D).integers(0, 9, S)]
    starts = [T - n for n in lens]
    cu = _cu(lens)
    qkv = torch.randn(cu[-1], 3 * H * D, generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.empty(1, 2, S, H, T, D, dtype=torch.uint8, device="cuda")
    assert kv.numel() > 2 ** 32
    sc = torch.empty(1, 2, S, H, T, device="cuda")
    last = (kv[..., T - 12:, :], sc[..., T - 12:])
    for t in last:
        t.fill_(3)
    q, k = (torch.empty(cu[-1], H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = _wave(H, D, S, T)
    try:
        for i in range(S):
            if lens[i]:
                w.prompt_append(0, cu[i:i + 2], [i], [starts[i]], qkv, kv, sc, q, k)
        want = [t.clone() for t in (*last, q, k)]
        for t in (*last, q, k):
            t.fill_(3)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            w.prompt_append(0, cu, list(range(S)), starts, qkv, kv, sc, q, k, stream=s)
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        assert w.status() == fsd.WAVE_OK
        for a, b in zip((*last, q, k), want):
            assert torch.equal(a, b)
        for i in range(S):
            assert bool((last[0][0, :, i, :, :12 - lens[i]] == 3).all()) and bool((last[1][0, :, i, :, :12 - lens[i]] == 3).all())
    finally:
        w.close()


# ---------------------------------------------------------------------- state
def state_reference(zx, prm, h0, cu, hs):
    """(out, its bound, states, their bound) in 64 bits, by the recurrence.
    With T the sums of the absolute values of the terms (the recurrence of
    |x|, |B|, |C|): the products' factors may be rounded to bf16 once each
    (half a step; two of them in a term of y), the state's to 16 bits
    (2^-17) with fp32 sums, and the gate's factors a few fp32 roundings; the
    decay is the exponential of a sum of at most len terms, each with a few
    fp32 roundings of its size."""
    di = hs * P
    z, x = zx[:, :di].double().reshape(-1, hs, P), zx[:, di:2 * di].double().reshape(-1, hs, P)
    B, C = zx[:, 2 * di:2 * di + N].double(), zx[:, 2 * di + N:2 * di + 2 * N].double()
    a_log, bias, skip = (prm[i * hs:(i + 1) * hs].double() for i in range(3))
    dt = torch.nn.functional.softplus(zx[:, 2 * di + 2 * N:].double() + bias)
    lam = torch.exp(a_log) * dt
    out = torch.zeros(zx.shape[0], hs, P, dtype=torch.float64, device=zx.device)
    tol = torch.zeros_like(out)
    states, st_tol = [], []
    half = HALF[torch.bfloat16]
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        h, T = h0[i].double().clone(), h0[i].double().abs()
        # an entry that has been carried over n tokens: its decay's exponent
        # carries (n + 4) roundings of the decays' logarithms; the weight of
        # an old entry falls as exp(-total), so x exp(-x) <= 0.37 bounds it
        R = 4.0 * U * T
        for t in range(a, b):
            dec = torch.exp(-lam[t])[:, None, None]
            new = (dt[t][:, None] * x[t])[:, :, None] * B[t][None, None]
            h, T = dec * h + new, dec * T + new.abs()
            R = dec * R + U * (8 + 8 * lam[t].clamp(max=40.0))[:, None, None] * T
            y = h @ C[t] + skip[:, None] * x[t]
            mag = T @ C[t].abs() + (skip[:, None] * x[t]).abs()
            gate = torch.nn.functional.silu(z[t])
            out[t] = y * gate
            tol[t] = half * out[t].abs() * 1.01 + gate.abs() * (2.02 * half * mag + R @ C[t].abs()) + 1e-30
        states.append(h)
        st_tol.append(2.0 ** -16 * T + 8 * R + 1e-30)
    return out.reshape(-1, di), tol.reshape(-1, di), states, st_tol


def _state_case(lens, hs, starts, seed=0, first=0, tail=0, S=None, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu = _cu(lens, first)
    n = cu[-1] + tail
    width = 2 * hs * P + 2 * N + hs
    zx = torch.randn(n, width + pad, generator=g, device="cuda").to(torch.bfloat16)[:, :width]
    prm = torch.cat([torch.randn(hs, generator=g, device="cuda"), torch.randn(hs, generator=g, device="cuda") - 2,
                     torch.randn(hs, generator=g, device="cuda")]).to(torch.bfloat16)
    S = len(lens) if S is None else S
    state = torch.randn(1, S, hs, P, N, generator=g, device="cuda")
    out = torch.full((n, hs * P), 7.0, dtype=torch.bfloat16, device="cuda")
    return cu, zx, prm, state, out


def _weights(cfg, prm, layer=0):
    blob = torch.zeros(fsd.hybrid_weights_bytes(cfg) // 2, dtype=torch.bfloat16, device="cuda")
    hs = cfg.ssm_heads
    end = fsd.hybrid_layer_offset(cfg, layer + 1) // 2
    at = end - (3 * hs + 7) // 8 * 8
    blob[at:at + 3 * hs] = prm
    return fsd.hybrid_pack_weights(cfg, blob)


def _check_state(cu, zx, prm, h0, slots, starts, hs, out, got_state, S):
    zero = torch.zeros(hs, P, N, device="cuda")
    ref, tol, states, st_tol = state_reference(zx, prm, [h0[0, s] if s0 > 0 else zero for s, s0 in zip(slots, starts)], cu, hs)
    worst = (((out.double() - ref).abs() / tol.clamp(min=1e-30))[cu[0]:cu[-1]]).max() if cu[-1] > cu[0] else 0
    assert float(worst) <= 1.0, float(worst)
    for i, s in enumerate(slots):
        if cu[i] == cu[i + 1]:
            continue
        w = float(((got_state[0, s].double() - states[i]).abs() / st_tol[i]).max())
        assert w <= 1.0, (i, w)


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [64, 0, 1, 200], [385, 16, 15, 17], [700], [1] * 20])
@pytest.mark.parametrize("hs", [4, 12])
def test_state_lengths(lens, hs):
    n = len(lens)
    starts = [(0 if i % 2 == 0 else 5) for i in range(n)]
    slots = list(reversed(range(n)))
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=sum(lens), first=3, tail=2, S=n + 1, pad=8)
    cfg, w = _hybrid(hs, S=n + 1)
    new = torch.full_like(h0, 9.0)
    try:
        w.prompt_state(0, _weights(cfg, prm), cu, slots, starts, zx, h0, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_state(cu, zx, prm, h0, slots, starts, hs, out, new, n + 1)
    assert bool((out[:3] == 7).all()) and bool((out[cu[-1]:] == 7).all())
    assert bool((new[0, n] == 9).all()), "a session that the call does not name"
    for i, s in enumerate(slots):
        if lens[i] == 0:
            assert bool((new[0, s] == 9).all())


@pytest.mark.parametrize("hs,lens,starts", [(4, [2600], [0]), (4, [1281], [3]), (8, [1500, 9, 900, 640], [0, 2, 5, 0]),
                                            (12, [700, 700], [1, 0]), (64, [2048], [0])])
def test_state_long_sequences_of_few_heads(hs, lens, starts):
    """Sequences cut into segments over the SMs: the state passes from one to
    the next, from zero and from an earlier one."""
    n = len(lens)
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=hs, S=n)
    cfg, w = _hybrid(hs, S=n)
    new = torch.full_like(h0, 9.0)
    try:
        for _ in range(2):  # the scratch of one call is no part of the next
            w.prompt_state(0, _weights(cfg, prm), cu, list(range(n)), starts, zx, h0, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_state(cu, zx, prm, h0, list(range(n)), starts, hs, out, new, n)


@pytest.mark.parametrize("hs,lens", [(64, [130, 129, 300, 64, 50, 257, 1, 17]), (24, [49 + 5 * i for i in range(30)] + [3]),
                                     (12, [50 + i % 9 for i in range(64)])])
def test_state_of_more_sequences_than_sms(hs, lens):
    """Head pairs of sequences beyond the SMs, a few short sequences among
    them: the CTAs that run take the others' places."""
    n = len(lens)
    starts = [i % 2 for i in range(n)]
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=hs, S=n)
    cfg, w = _hybrid(hs, S=n)
    wt = _weights(cfg, prm)
    new, again, out2 = torch.full_like(h0, 9.0), h0.clone(), torch.zeros_like(out)
    try:
        w.prompt_state(0, wt, cu, list(range(n)), starts, zx, h0, new, out)
        w.prompt_state(0, wt, cu, list(range(n)), starts, zx, again, again, out2)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    assert torch.equal(new, again) and torch.equal(out, out2), "in place, and whoever takes whose place"
    _check_state(cu, zx, prm, h0, list(range(n)), starts, hs, out, new, n)


@pytest.mark.parametrize("lens", [[16], [25], [129], [2048]])
def test_state_is_carried_in_fp32(lens):
    """The 2-norm of the state's error, relative to the state: a weight is a
    product of some six factors and exponentials of 1 to 4 roundings each
    (10 U in quadrature), and the sums add a rounding a step, those of old
    tokens decayed (6 U): far below one part of 2^-16, two bf16 of a weight."""
    hs = 16
    cu, zx, prm, h0, out = _state_case(lens, hs, [0], seed=lens[0])
    cfg, w = _hybrid(hs, S=1)
    new = torch.zeros_like(h0)
    try:
        w.prompt_state(0, _weights(cfg, prm), cu, [0], [0], zx, None, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _, _, states, _ = state_reference(zx, prm, [torch.zeros(hs, P, N, device="cuda")], cu, hs)
    assert float((new[0, 0].double() - states[0]).norm() / states[0].norm()) <= 16 * U


def test_state_in_place_in_parts_and_left_out():
    """A prompt in one call, and in three calls on the same buffer, each going
    on from the state of the last; a left-out sequence keeps its state."""
    hs, lens = 8, [300, 40]
    cu, zx, prm, h0, out = _state_case(lens, hs, [0, 0], seed=4)
    cfg, w = _hybrid(hs, S=2)
    wt = _weights(cfg, prm)
    try:
        whole = torch.zeros_like(h0)
        w.prompt_state(0, wt, cu, [0, 1], [0, 0], zx, None, whole, out)
        parts, kept = h0.clone(), h0[0, 1].clone()
        out2 = torch.zeros_like(out)
        at = 0
        for n in (129, 1, 170):
            w.prompt_state(0, wt, [at, at + n, at + n + 5], [0, -1], [at, 0], zx, parts, parts, out2)
            at += n
        assert w.status() == fsd.WAVE_OK
        assert torch.equal(parts[0, 1], kept)
    finally:
        w.close()
    zero = [torch.zeros(hs, P, N, device="cuda")]
    ref, tol, states, st_tol = state_reference(zx[:300], prm, zero, [0, 300], hs)
    for o in (out, out2):
        assert bool(((o[:300].double() - ref).abs() <= tol).all())
    for st in (whole, parts):
        assert bool(((st[0, 0].double() - states[0]).abs() <= st_tol[0]).all())


@pytest.mark.parametrize("a_log", [4.0, -12.0])
def test_state_extreme_decays(a_log):
    """A head that forgets at once (the decay of a token underflows), and one
    that keeps everything."""
    hs, lens = 4, [260, 5]
    cu, zx, prm, h0, out = _state_case(lens, hs, [3, 3], seed=5)
    prm[:hs] = a_log
    prm[hs:2 * hs] = 3.0
    cfg, w = _hybrid(hs, S=2)
    new = torch.zeros_like(h0)
    try:
        w.prompt_state(0, _weights(cfg, prm), cu, [0, 1], [3, 3], zx, h0, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_state(cu, zx, prm, h0, [0, 1], [3, 3], hs, out, new, 2)


def test_state_non_finite_tokens_do_not_reach_earlier_ones():
    """NaN and infinities at a token (its x, B, C, z and dt), and in rows
    outside every sequence: earlier tokens and other sequences are exact."""
    hs, lens = 4, [200, 150]
    cu, zx, prm, h0, out = _state_case(lens, hs, [0, 0], seed=6, first=5, tail=70)
    zx[:5], zx[cu[-1]:] = float("nan"), float("inf")
    zx[cu[0] + 140] = float("nan")
    cfg, w = _hybrid(hs, S=2)
    new = torch.zeros_like(h0)
    try:
        w.prompt_state(0, _weights(cfg, prm), cu, [0, 1], [0, 0], zx, None, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    zero = [torch.zeros(hs, P, N, device="cuda")]
    for a, b in ((cu[0], cu[0] + 140), (cu[1], cu[2])):
        ref, tol, states, st_tol = state_reference(zx, prm, zero, [a, b], hs)
        assert bool(((out.double() - ref).abs() <= tol)[a:b].all())
    assert bool(((new[0, 1].double() - states[0]).abs() <= st_tol[0]).all())
    assert bool(torch.isnan(out[cu[0] + 140:cu[1]]).all()) and bool(torch.isnan(new[0, 0]).all())


@pytest.mark.parametrize("lens", [[17], [127], [128], [129], [64, 0, 1, 200], [385, 16, 15, 18], [255, 257]])
@pytest.mark.parametrize("hs", [8, 24])
def test_state_lengths_of_aligned_rows(lens, hs):
    """Rows of a multiple of 16 bytes, which a tensor map describes."""
    n = len(lens)
    starts, slots = [(4 if i % 2 == 0 else 0) for i in range(n)], list(range(n))
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=sum(lens), first=1, tail=3, S=n)
    assert zx.stride(0) % 8 == 0
    cfg, w = _hybrid(hs, S=n)
    new = torch.full_like(h0, 9.0)
    try:
        w.prompt_state(0, _weights(cfg, prm), cu, slots, starts, zx, h0, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_state(cu, zx, prm, h0, slots, starts, hs, out, new, n)
    assert bool((out[:1] == 7).all()) and bool((out[cu[-1]:] == 7).all())


@pytest.mark.parametrize("hs,lens", [(8, [1500, 700]), (4, [1300]), (64, [200, 40, 9])])
def test_state_in_place_beside_other_work(hs, lens):
    """In place and elsewhere are the same, with the SMs kept busy by another
    stream (the CTAs of a sequence's segments do not all run at once)."""
    n = len(lens)
    cu, zx, prm, h0, out = _state_case(lens, hs, [1] * n, seed=hs, S=n)
    cfg, w = _hybrid(hs, S=n)
    wt = _weights(cfg, prm)
    a = torch.randn(4096, 4096, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    try:
        new, out2 = torch.zeros_like(h0), torch.zeros_like(out)
        w.prompt_state(0, wt, cu, list(range(n)), [1] * n, zx, h0, new, out)
        for _ in range(8):
            state = h0.clone()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(4):
                    a @ a
            w.prompt_state(0, wt, cu, list(range(n)), [1] * n, zx, state, state, out2)
            assert torch.equal(state, new) and torch.equal(out2, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()


def test_state_batch_replays_from_a_graph():
    """128 sessions, short and long, captured and replayed with new tokens on
    a stream of its own."""
    hs, n = 4, fsd.WAVE_MAX_SEQS
    lens = [int(x) for x in np.random.default_rng(9).integers(0, 40, n)]
    lens[5], lens[77] = 300, 129
    starts = [i % 3 for i in range(n)]
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=9, S=n)
    cfg, w = _hybrid(hs, S=n)
    wt = _weights(cfg, prm)
    new = torch.full_like(h0, 9.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            w.prompt_state(0, wt, cu, list(range(n)), starts, zx, h0, new, out, stream=s)
        zx.copy_(zx.flip(0))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
            graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_state(cu, zx, prm, h0, list(range(n)), starts, hs, out, new, n)


@pytest.mark.parametrize("hs,lens,starts", [(4, [1300, 20], [2, 0]), (8, [900], [0]), (24, [1000, 3, 640], [1, 4, 0])])
def test_state_segments_replay(hs, lens, starts):
    """Segmented sequences from a graph, in place, again and again: each replay
    goes on from the state of the one before, as eager calls do."""
    n = len(lens)
    cu, zx, prm, h0, out = _state_case(lens, hs, starts, seed=hs + 1, S=n)
    cfg, w = _hybrid(hs, S=n)
    wt = _weights(cfg, prm)
    a, b = h0.clone(), h0.clone()
    out2 = torch.zeros_like(out)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.prompt_state(0, wt, cu, list(range(n)), starts, zx, b, b, out2)
        w.prompt_state(0, wt, cu, list(range(n)), starts, zx, a, a, out)
        _check_state(cu, zx, prm, h0, list(range(n)), starts, hs, out, a, n)
        for _ in range(2):
            w.prompt_state(0, wt, cu, list(range(n)), starts, zx, a, a, out)
        for _ in range(3):
            graph.replay()
        assert w.status() == fsd.WAVE_OK
        assert torch.equal(a, b) and torch.equal(out, out2)
    finally:
        w.close()


@pytest.mark.parametrize("pad", [0, 4])
def test_state_offsets_beyond_32_bits(pad):
    """Rows whose offsets in elements pass 2^31."""
    hs, n = 64, 254000
    lens, starts = [140, 9], [2, 0]
    width = 2 * hs * P + 2 * N + hs
    zx = torch.empty(n, width + pad, dtype=torch.bfloat16, device="cuda")[:, :width]
    out = torch.empty(n, hs * P, dtype=torch.bfloat16, device="cuda")
    _, small, prm, h0, _ = _state_case(lens, hs, starts, seed=pad)
    zx[n - 149:] = small
    cu = [n - 149, n - 9, n]
    assert cu[0] * zx.stride(0) > 2 ** 31
    cfg, w = _hybrid(hs, S=2)
    new = torch.zeros_like(h0)
    try:
        w.prompt_state(0, _weights(cfg, prm), cu, [0, 1], starts, zx, h0, new, out)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_state([0, 140, 149], small, prm, h0, [0, 1], starts, hs, out[n - 149:], new, 2)


# --------------------------------------------------------------------- copies
def _sessions(hybrid, S=9, T=72, H=3, D=64, hs=4):
    g = torch.Generator(device="cuda").manual_seed(S)
    if hybrid:
        _, w = _hybrid(hs, S=S, T=T, layers=6, every=3, heads=H, dim=D)
        la, lm = 2, 4
    else:
        w, la, lm = _wave(H, D, S, T, 3), 3, 0
    kv = torch.randint(0, 256, (la, 2, S, H, T, D), dtype=torch.uint8, device="cuda", generator=g)
    sc = torch.rand((la, 2, S, H, T), device="cuda", generator=g)
    st = torch.randn(lm, S, hs, P, N, generator=g, device="cuda") if hybrid else None
    return w, kv, sc, st


@pytest.mark.parametrize("hybrid", [False, True])
@pytest.mark.parametrize("move", [False, True])
@pytest.mark.parametrize("src,dst", [([0], [8]), ([4, 4, 4], [1, 2, 3]), ([8, 7, 8, 0], [3, 1, 2, 5]), ([5, 6, 7], [0, 1, 2])])
def test_sessions_copy(hybrid, move, src, dst):
    w, kv, sc, st = _sessions(hybrid)
    pos_h = [37, 9, -1, 72, 71, 1, 0, -1, 33]
    pos = torch.tensor(pos_h, dtype=torch.int32, device="cuda")
    want_kv, want_sc, want_st = kv.clone(), sc.clone(), None if st is None else st.clone()
    want_pos = list(pos_h)
    for a, b in zip(src, dst):
        n = max(0, pos_h[a])
        want_kv[:, :, b, :, :n], want_sc[:, :, b, :, :n] = kv[:, :, a, :, :n], sc[:, :, a, :, :n]
        if st is not None and pos_h[a] >= 0:
            want_st[:, b] = st[:, a]
        want_pos[b] = pos_h[a]
    if move:
        for a in src:
            want_pos[a] = -1
    try:
        w.sessions_copy(src, dst, kv, sc, pos, state=st, move=move)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    assert torch.equal(kv, want_kv) and torch.equal(sc, want_sc) and pos.tolist() == want_pos
    assert st is None or torch.equal(st, want_st)


@pytest.mark.parametrize("T,D,pos", [(20000, 64, 19999), (5000, 128, 4999)])
def test_sessions_copy_long(T, D, pos):
    """Rows of many pieces, the last one ragged in codes and scales."""
    w, kv, sc, _ = _sessions(False, S=3, T=T, H=2, D=D)
    p = torch.tensor([-1, pos, 5], dtype=torch.int32, device="cuda")
    want_kv, want_sc = kv.clone(), sc.clone()
    for b in (0, 2):
        want_kv[:, :, b, :, :pos], want_sc[:, :, b, :, :pos] = kv[:, :, 1, :, :pos], sc[:, :, 1, :, :pos]
    try:
        w.sessions_copy([1, 1], [0, 2], kv, sc, p)
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    assert torch.equal(kv, want_kv) and torch.equal(sc, want_sc) and p.tolist() == [pos] * 3


def test_sessions_copy_beyond_32_bits_and_replayed():
    """The last session of a large history to the first slots, from a graph
    that reads the positions when it runs."""
    S, H, T, D = 128, 32, 4100, 128
    kv = torch.empty(1, 2, S, H, T, D, dtype=torch.uint8, device="cuda")
    sc = torch.empty(1, 2, S, H, T, device="cuda")
    assert kv.numel() > 2 ** 32
    for s in (0, 1, 127):
        kv[:, :, s], sc[:, :, s] = s + 1, s + 1
    pos = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    w = _wave(H, D, S, T)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.sessions_copy([127, 127], [0, 1], kv, sc, pos)
        pos[127] = 4001
        graph.replay()
        assert w.status() == fsd.WAVE_OK
        for s in (0, 1):
            assert bool((kv[:, :, s, :, :4001] == 128).all()) and bool((kv[:, :, s, :, 4001:] == s + 1).all())
            assert bool((sc[:, :, s, :, :4001] == 128).all()) and bool((sc[:, :, s, :, 4001:] == s + 1).all())
        assert pos[:2].tolist() == [4001, 4001]
    finally:
        w.close()


# ------------------------------------------------------------------- refusals
def test_waits_that_run_out_are_reported():
    """With a limit far below what the kernels take, their waits give up: the
    launch ends by itself, the status says so once, and the handle goes on."""
    cu, q, k, v, out = _attention([4100, 300], 4, 4, 128, torch.bfloat16, seed=2)
    lens, starts = [2600, 700], [0, 3]
    cs, zx, prm, h0, so = _state_case(lens, 8, starts, seed=1)
    cfg, w = _hybrid(8, S=2, heads=4, dim=128)
    wt = _weights(cfg, prm)
    new = torch.zeros_like(h0)
    calls = [lambda: w.prompt_attention(cu, q, k, v, out), lambda: w.prompt_state(0, wt, cs, [0, 1], starts, zx, h0, new, so)]
    try:
        for c in calls:
            w.set_timeout_ns(1)
            c()
            assert w.status() == fsd.WAVE_ETIMEOUT
            assert w.status() == fsd.WAVE_OK
        w.set_timeout_ns(2_000_000_000)
        for c in calls:
            c()
        assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_attention(cu, q, k, v, out)
    _check_state(cs, zx, prm, h0, [0, 1], starts, 8, so, new, 2)


def test_refusals_before_any_launch():
    """Every bad argument is answered on the host, and nothing is written."""
    L = fsd.lib()
    H, D, S, T = 2, 64, 4, 64
    w = _wave(H, D, S, T, 2)
    cfg, hw = _hybrid(4, S=S, T=T)
    E, OK = fsd.WAVE_EINVAL, fsd.WAVE_OK
    ints = lambda v: fsd._ints(v)[0]  # noqa: E731
    buf = torch.zeros(1 << 20, device="cuda")
    b = buf.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    try:
        def append(h=w.h, layer=0, cu=(0, 3, 5), slots=(0, 1), starts=(0, 0), qkv=b, t=1, stride=384, kv=b, sc=b, q=b, k=b, v=b, o=1):
            return L.wave_prompt_append(h, layer, len(cu) - 1, ints(cu), ints(slots), ints(starts), qkv, t, stride, kv, sc, q, k, v, o, st)

        def attend(h=w.h, cu=(0, 3, 5), hkv=1, t=1, q=b, qs=128, k=b + 4096, ks=64, v=b + 8192, vs=64, scale=0.125, out=b + 16384, os=128):
            return L.wave_prompt_attention(h, len(cu) - 1, ints(cu), hkv, t, q, qs, k, ks, v, vs, scale, out, os, st)

        def state(h=hw.h, layer=0, wt=b, cu=(0, 3, 5), slots=(0, 1), starts=(0, 0), zx=b, zs=776, si=None, so=b, out=b, os=256):
            return L.wave_hybrid_prompt_state(h, layer, wt, len(cu) - 1, ints(cu), ints(slots), ints(starts), zx, zs, si, so, out, os, st)

        def copy(h=w.h, src=(0,), dst=(1,), move=0, kv=b, sc=b, ss=None, pos=b):
            return L.wave_sessions_copy(h, len(src), ints(src), ints(dst), move, kv, sc, ss, pos, st)

        many = dict(cu=range(130), slots=range(129), starts=[0] * 129)
        for kw in [dict(h=None), dict(layer=-1), dict(layer=2), dict(cu=(0,)), dict(cu=(0, 5, 3)), dict(cu=(-1, 3, 5)),
                   dict(slots=(0, 4)), dict(slots=(1, 1)), dict(starts=(0, -1)), dict(qkv=None), dict(qkv=b + 8), dict(t=2), dict(t=9),
                   dict(stride=376), dict(stride=388), dict(kv=None), dict(kv=b + 4), dict(sc=None), dict(sc=b + 4), dict(q=b + 2),
                   dict(k=b + 8), dict(v=b + 8), dict(o=0), dict(o=3), dict(stride=2 ** 31), many]:
            assert append(**kw) == E, kw
        assert append(starts=(62, 0)) == fsd.WAVE_EPOS and append(starts=(0, 2 ** 31 - 2)) == fsd.WAVE_EPOS
        assert append(h=hw.h, layer=0, stride=192) == E  # a selective-state block has no history
        assert append(slots=(-1, -1)) == OK and append(cu=(7, 7, 7)) == OK  # nothing to do
        for kw in [dict(h=None), dict(cu=(0,)), dict(cu=(4, 3)), dict(cu=(-1, 2)), dict(cu=range(130)), dict(hkv=0), dict(hkv=3), dict(t=0),
                   dict(t=3), dict(q=None), dict(q=b + 2), dict(qs=120), dict(qs=132), dict(k=None), dict(k=b + 8), dict(ks=56),
                   dict(v=None), dict(vs=68), dict(out=None), dict(out=b + 4), dict(os=64), dict(scale=0.0), dict(scale=-1.0),
                   dict(scale=float("inf")), dict(scale=float("nan")), dict(qs=2 ** 31)]:
            assert attend(**kw) == E, kw
        assert attend(cu=(3, 3)) == OK
        for kw in [dict(h=None), dict(h=w.h), dict(layer=1), dict(layer=-1), dict(layer=2), dict(wt=None), dict(wt=b + 8), dict(cu=(0,)),
                   dict(cu=(2, 1)), dict(slots=(0, 4)), dict(slots=(2, 2)), dict(starts=(-1, 0)), dict(starts=(1, 0)), dict(zx=None),
                   dict(zx=b + 8), dict(zs=768), dict(zs=774), dict(so=None), dict(so=b + 8), dict(si=b + 4), dict(out=None),
                   dict(out=b + 8), dict(os=248), dict(os=260), dict(zs=2 ** 31), dict(os=2 ** 31), many]:
            assert state(**kw) == E, kw
        assert state(slots=(-1, -1)) == OK
        for kw in [dict(h=None), dict(src=()), dict(src=(4,)), dict(src=(-1,)), dict(dst=(4,)), dict(dst=(-1,)), dict(dst=(0,)),
                   dict(src=(0, 1), dst=(2, 2)), dict(src=(0, 1), dst=(1, 2)), dict(src=(0,) * 5, dst=(1, 2, 3, 1, 2)), dict(kv=None),
                   dict(kv=b + 8), dict(sc=None), dict(sc=b + 4), dict(pos=None), dict(pos=b + 2), dict(ss=b), dict(h=hw.h)]:
            assert copy(**kw) == E, kw
        torch.cuda.synchronize()
        assert not bool(buf.any())
        assert w.status() == OK and hw.status() == OK
    finally:
        w.close()
        hw.close()


def test_waits_that_run_out_with_more_work_than_sms():
    """The same where CTAs take the places of others."""
    cu, q, k, v, out = _attention([600] * 24, 8, 8, 128, torch.bfloat16, seed=2)
    lens, starts, n = [200] * 6, [0, 3] * 3, 6
    cs, zx, prm, h0, so = _state_case(lens, 64, starts, seed=1)
    cfg, w = _hybrid(64, S=n, heads=8, dim=128)
    wt = _weights(cfg, prm)
    new = torch.zeros_like(h0)
    calls = [lambda: w.prompt_attention(cu, q, k, v, out),
             lambda: w.prompt_state(0, wt, cs, list(range(n)), starts, zx, h0, new, so)]
    try:
        for c in calls:
            w.set_timeout_ns(1)
            c()
            assert w.status() == fsd.WAVE_ETIMEOUT
            w.set_timeout_ns(1000)  # a try each: some run out in the middle of the work
            c()
            assert w.status() in (fsd.WAVE_ETIMEOUT, fsd.WAVE_OK)
            w.set_timeout_ns(2_000_000_000)
            c()
            assert w.status() == fsd.WAVE_OK
    finally:
        w.close()
    _check_attention(cu, q, k, v, out)
    _check_state(cs, zx, prm, h0, list(range(n)), starts, 64, so, new, n)


# ------------------------------------------------------- the operators together
def test_a_prompt_leaves_what_stepping_through_it_leaves():
    """The small hybrid model: prompts of two sessions run through the prompt
    calls (projections in 64 bits, rounded to bf16 where the step rounds) leave the history and
    state that stepping token by token leaves, up to bf16 flips; one is then
    forked into a third slot and the next frame of both is bit-identical."""
    import synth
    w = synth.HYBRID_SMALL
    cfg = fsd.WaveHybridConfig.of(w)
    S, lens, slots = 4, [21, 9], [2, 0]
    cu = _cu(lens)
    W = torch.from_numpy(synth.hybrid_weights_host(w).view(np.int16)).cuda().view(torch.bfloat16)
    wt = fsd.hybrid_pack_weights(cfg, W)
    d, H, D, hs = w.d_model, w.n_heads, w.head_dim, w.ssm_heads
    di, La, Lm = hs * P, w.n_layers // w.attn_every, w.n_layers - w.n_layers // w.attn_every
    kv = [torch.zeros((La, 2, S, H, w.T_max, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((La, 2, S, H, w.T_max), device="cuda") for _ in range(2)]
    state = [torch.zeros((Lm, S, hs, P, N), device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(cu[-1], d, generator=g, device="cuda").to(torch.bfloat16)
    wave = fsd.HybridWave(cfg, S, w.T_max)
    try:
        # token by token
        for t in range(max(lens)):
            pos = torch.full((S,), -1, dtype=torch.int32)
            xs = torch.zeros(S, d, dtype=torch.bfloat16, device="cuda")
            for i, s in enumerate(slots):
                if t < lens[i]:
                    pos[s] = t
                    xs[s] = x[cu[i] + t]
            ys = torch.zeros_like(xs)
            wave.hybrid_step(S, wt, kv[0], sc[0], state[0], pos.cuda(), xs, ys)
        # the prompts at once
        r = x.double()
        for l in range(w.n_layers):
            o = fsd.hybrid_layer_offset(cfg, l) // 2
            gain = W[o:o + d].double()
            xn = (r / torch.sqrt((r * r).mean(-1, keepdim=True) + w.rms_eps) * gain).to(torch.bfloat16).double()
            o += d
            if l % w.attn_every == w.attn_every - 1:
                wqkv = W[o:o + 3 * H * D * d].view(3 * H * D, d).double()
                wo = W[o + 3 * H * D * d:o + 4 * H * D * d].view(d, H * D).double()
                q, k, v, att = (torch.zeros(cu[-1], H, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
                wave.prompt_append(l, cu, slots, [0, 0], (xn @ wqkv.t()).float(), kv[1], sc[1], q, k, v)
                wave.prompt_attention(cu, q, k, v, att)
                r = r + att.reshape(-1, H * D).double() @ wo.t()
            else:
                rows = 2 * di + 2 * N + hs
                w_in = W[o:o + rows * d].view(rows, d).double()
                w_out = W[o + rows * d:o + rows * d + d * di].view(d, di).double()
                out = torch.zeros(cu[-1], di, dtype=torch.bfloat16, device="cuda")
                lm = l - l // w.attn_every
                wave.prompt_state(l, wt, cu, slots, [0, 0], (xn @ w_in.t()).to(torch.bfloat16), None, state[1], out)
                r = r + out.double() @ w_out.t()
        assert wave.status() == fsd.WAVE_OK
        # bf16 roundings of q, k, v and zxbcdt stand where the step keeps fp32: half a step (2^-8) each
        # per block, relative to the rows' size; the state of the first block sees one such rounding
        # of its inputs only (three factors: dt, x, B), later ones their cascade through the layers
        a, b = state[0][:, slots].double(), state[1][:, slots].double()
        rel = [float((a[m] - b[m]).norm() / a[m].norm()) for m in range(Lm)]
        print("state, normwise, by block:", rel)
        assert rel[0] <= 3 * 2.0 ** -8 and max(rel) <= 5e-2
        for i, s in enumerate(slots):
            va = kv[0][:, :, s, :, :lens[i]].view(torch.float8_e4m3fn).double() * sc[0][:, :, s, :, :lens[i], None].double()
            vb = kv[1][:, :, s, :, :lens[i]].view(torch.float8_e4m3fn).double() * sc[1][:, :, s, :, :lens[i], None].double()
            assert float((va - vb).norm() / va.norm()) <= 2.0 ** -4  # e4m3 codes of nearby values: a step at most
        # fork the session in slot 2 into slot 1, then one frame of both
        pos = torch.tensor([lens[1], -1, lens[0], -1], dtype=torch.int32, device="cuda")
        wave.sessions_copy([2], [1], kv[1], sc[1], pos, state=state[1])
        assert pos.tolist() == [lens[1], lens[0], lens[0], -1]
        xs = torch.randn(S, d, generator=g, device="cuda").to(torch.bfloat16)
        xs[1] = xs[2]
        ys = torch.zeros_like(xs)
        wave.hybrid_step(S, wt, kv[1], sc[1], state[1], pos, xs, ys)
        assert wave.status() == fsd.WAVE_OK
        assert torch.equal(ys[1], ys[2]) and torch.equal(state[1][:, 1], state[1][:, 2])
        assert torch.equal(kv[1][:, :, 1, :, :lens[0] + 1], kv[1][:, :, 2, :, :lens[0] + 1])
    finally:
        wave.close()
