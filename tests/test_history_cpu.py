"""CPU: rotary plans against the formula, and what the calls on rotary
positions and on the block-scaled history refuse without touching a device."""
import ctypes
import math

import numpy as np
import pytest
import torch

import frame_step_decode_gb300 as fsd


def _b(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _decoder(heads=4, dim=64):
    w = fsd.Wave.__new__(fsd.Wave)  # a binding object whose handle is NULL (no device here to create one)
    w.cfg, w.h = fsd.WaveConfig(1, 64, heads, dim, 64, 1e-5, 1e4), None
    return w


@pytest.mark.parametrize("dims", [16, 48, 64, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "parts"])
def test_a_plan_holds_the_formulas_turns(dims, scaling):
    p = fsd.rope_plan(dims, 1e4, layout="interleaved", scaling=scaling, factor=8.0, original=4096.0, fast=32.0, slow=1.0, amplitude=1.25)
    assert (p.layout, p.dims, p.amplitude) == (1, dims, 1.25)
    for i in range(64):
        f = 0.0
        if i < dims // 2:
            f = 1e4 ** (-2.0 * i / dims)
            if scaling == "linear":
                f /= 8.0
            if scaling == "parts":
                keep = min(1.0, max(0.0, (4096.0 * f / (2 * math.pi) - 1.0) / 31.0))
                f = keep * f + (1 - keep) * f / 8.0
        # a few roundings of a double, relative to the frequency; a fraction of 64 bits is off by half of 2^-64
        assert abs(p.turns[i] / 2.0 ** 64 - f / (2 * math.pi)) <= 2.0 ** -50 * f + 2.0 ** -65


def test_angles_modulo_a_turn():
    """turns * position in 64 bits is the angle of far positions, by exact integers."""
    p = fsd.rope_plan(128, 5e5)
    for i in (0, 1, 17, 63):
        for pos in (0, 1, 4095, 10 ** 6 + 3, 2 ** 31 - 1):
            frac = (p.turns[i] * pos) % 2 ** 64 / 2.0 ** 64
            want = 5e5 ** (-2.0 * i / 128) / (2 * math.pi) * pos % 1.0
            d = abs(frac - want)
            # pos times a double's half step, and that of 64 bits; the wanted value's own product rounds to 2^-53 of it
            assert min(d, 1 - d) <= pos * 2.0 ** -52 + 2.0 ** -50


@pytest.mark.parametrize("bad", [dict(dims=8), dict(dims=24), dict(dims=144), dict(base=0.0), dict(base=-1.0), dict(base=math.nan),
                                 dict(base=math.inf), dict(amplitude=math.inf), dict(scaling="linear", factor=0.0),
                                 dict(scaling="linear", factor=math.nan), dict(scaling="parts", factor=2.0, original=0.0),
                                 dict(scaling="parts", factor=2.0, original=math.inf),
                                 dict(scaling="parts", factor=2.0, original=4096.0, fast=1.0, slow=1.0),
                                 dict(scaling="parts", factor=2.0, original=4096.0, fast=4.0, slow=-1.0),
                                 dict(scaling="parts", factor=2.0, original=4096.0, fast=math.inf)])
def test_bad_plans_are_refused(bad):
    with pytest.raises(fsd.WaveError) as e:
        fsd.rope_plan(**{"dims": 64, **bad})
    assert e.value.code == fsd.WAVE_EINVAL


def test_unknown_names_and_null_plans_are_refused():
    for bad in (dict(layout="neox"), dict(scaling="dynamic")):
        with pytest.raises(ValueError):
            fsd.rope_plan(64, **bad)
    L = fsd.lib()
    c, r = fsd.WaveRopeConfig(0, 64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, 1.0), fsd.WaveRope()
    assert L.wave_rope_plan(None, ctypes.addressof(r)) == fsd.WAVE_EINVAL
    assert L.wave_rope_plan(ctypes.byref(c), None) == fsd.WAVE_EINVAL
    c.layout = 2
    assert L.wave_rope_plan(ctypes.byref(c), ctypes.addressof(r)) == fsd.WAVE_EINVAL


def test_rows_that_do_not_fit_a_rotation_are_refused():
    p, x = fsd.rope_plan(64), _b(3, 2, 64)
    bad = [lambda: fsd.rope_apply(p, x, cu_seqlens=[0, 4], starts=[0], stream=0),
           lambda: fsd.rope_apply(p, x, cu_seqlens=[0, 3], starts=[0, 0], stream=0),
           lambda: fsd.rope_apply(p, x, cu_seqlens=[0, 3], stream=0),
           lambda: fsd.rope_apply(p, x, stream=0),
           lambda: fsd.rope_apply(p, x, cu_seqlens=[0, 3], starts=[0], positions=_b(3, dtype=torch.int32), stream=0),
           lambda: fsd.rope_apply(p, x, positions=_b(4, dtype=torch.int32), stream=0),
           lambda: fsd.rope_apply(p, x, _b(3, 1, 64), cu_seqlens=[0, 3], starts=[0], stream=0),
           lambda: fsd.rope_apply(p, x.transpose(1, 2), cu_seqlens=[0, 3], starts=[0], stream=0),
           lambda: fsd.rope_apply(None, x, cu_seqlens=[0, 3], starts=[0], stream=0) or (_ for _ in ()).throw(ValueError()),
           lambda: fsd.rope_apply(object(), x, cu_seqlens=[0, 3], starts=[0], stream=0)]
    for i, c in enumerate(bad):
        with pytest.raises((ValueError, fsd.WaveError)):
            c()


class _NothingIsCalled:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was reached")


@pytest.mark.parametrize("types", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16)])
def test_a_rotation_of_the_hosts_tensors_is_refused(types, monkeypatch):
    """Rows, outputs and positions that fit in all but where they are: no call of the library is made with their addresses."""
    monkeypatch.setattr(fsd, "_lib", _NothingIsCalled())
    p, x, out = fsd.WaveRope(0, 64), _b(3, 2, 64, dtype=types[0]), _b(3, 2, 64, dtype=types[1])
    with pytest.raises(AssertionError):
        fsd.lib().wave_rope_apply  # the stub stands in for the library
    pos = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: fsd.rope_apply(p, x, out, cu_seqlens=[0, 3], starts=[0], stream=0),
                 lambda: fsd.rope_apply(p, out, cu_seqlens=[0, 3], starts=[0], stream=0),
                 lambda: fsd.rope_apply(p, x, out, positions=pos, stream=0),
                 lambda: fsd.rope_apply(p, x, out, positions=pos.long(), stream=0)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("change", [dict(n_heads=0), dict(head_dim=96), dict(head_dim=64, dims=128), dict(type=7), dict(out_type=-1),
                                    dict(x_stride=120), dict(x_stride=132), dict(x_stride=2 ** 31), dict(out_stride=64), dict(x=0), dict(out=0),
                                    dict(x=4104), dict(starts=[-1]), dict(starts=[2 ** 31 - 3]), dict(cu=[3, 0]), dict(cu=[-1, 3]),
                                    dict(x=8192, out=8192, out_type=0)])
def test_what_the_c_call_refuses(change):
    """Each before anything is enqueued: the addresses are made up."""
    a = dict(n_heads=2, head_dim=64, dims=64, type=1, out_type=1, x_stride=128, out_stride=128, x=4096, out=8192, starts=[0], cu=[0, 3]) | change
    p = fsd.rope_plan(a["dims"])
    rc = fsd.lib().wave_rope_apply(ctypes.addressof(p), 1, np.array(a["cu"], np.int32).tobytes(), np.array(a["starts"], np.int32).tobytes(),
                                   a["n_heads"], a["head_dim"], a["x"], a["type"], a["x_stride"], a["out"], a["out_type"], a["out_stride"], None)
    assert rc == fsd.WAVE_EINVAL


def test_a_spoilt_plan_is_refused():
    for field, value in (("dims", 24), ("dims", 0), ("dims", 256), ("layout", 5)):
        p = fsd.rope_plan(64)
        setattr(p, field, value)
        rc = fsd.lib().wave_rope_apply(ctypes.addressof(p), 1, np.array([0, 3], np.int32).tobytes(), np.array([0], np.int32).tobytes(),
                                       2, 64, 4096, 1, 128, 8192, 1, 128, None)
        assert rc == fsd.WAVE_EINVAL


def test_a_missing_handle_is_refused():
    w = _decoder()
    kv, sc, pos = _b(8, dtype=torch.uint8), _b(8, dtype=torch.float32), _b(3, dtype=torch.int32)
    q = _b(3, 4, 64)
    calls = [lambda: w.history_append(0, [0, 3], [0], [0], _b(3, 512), kv, sc, 2, 16, stream=0),
             lambda: w.history_append_frame(0, pos, _b(3, 512), kv, sc, 2, 16, stream=0),
             lambda: w.history_read(0, [0, 3], [0], [0], kv, sc, 2, 16, _b(3, 2, 64), stream=0),
             lambda: w.history_attention(0, [0, 3], [0], [0], q, kv, sc, 2, 16, q, stream=0),
             lambda: w.history_attention_frame(0, pos, q, kv, sc, 2, 16, q, stream=0)]
    for c in calls:
        with pytest.raises(fsd.WaveError) as e:
            c()
        assert e.value.code == fsd.WAVE_EINVAL


def test_shapes_that_do_not_fit_are_refused():
    w = _decoder()
    kv, sc, pos = _b(8, dtype=torch.uint8), _b(8, dtype=torch.float32), _b(3, dtype=torch.int32)
    q, x = _b(3, 4, 64), _b(3, 512)
    bad = [lambda: w.history_append(0, [0, 3], [0, 1], [0], x, kv, sc, 2, 16, stream=0),
           lambda: w.history_append(0, [0, 4], [0], [0], x, kv, sc, 2, 16, stream=0),
           lambda: w.history_append(0, [0, 3], [0], [0], x, kv, sc, 4, 16, stream=0),
           lambda: w.history_append(0, [0, 3], [0], [0], x, kv, sc, 3, 16, stream=0),
           lambda: w.history_append(0, [0, 3], [0], [0], x, kv, sc, 2, 8, stream=0),
           lambda: w.history_append(0, [0, 3], [0], [0], x, kv, sc, 2, 256, stream=0),
           lambda: w.history_append(0, [0, 3], [0], [0], x, kv, sc, 2, 16, q=_b(3, 2, 64), stream=0),
           lambda: w.history_append(0, [0, 3], [0], [0], x, kv, sc, 2, 16, rope=1e4, stream=0),
           lambda: w.history_append(0, [0, 3], [0], [2 ** 31], x, kv, sc, 2, 16, stream=0),
           lambda: w.history_append_frame(0, _b(4, dtype=torch.int32), x, kv, sc, 2, 16, stream=0),
           lambda: w.history_read(0, [0, 3], [0], [0], kv, sc, 2, 16, _b(3, 4, 64), stream=0),
           lambda: w.history_read(0, [0, 3], [0], [0], kv, sc, 2, 16, _b(3, 2, 64), _b(3, 2, 64, dtype=torch.float16), stream=0),
           lambda: w.history_read(0, [0, 3], [0], [0], kv, sc, 0, 16, stream=0),
           lambda: w.history_attention(0, [0, 4], [0], [0], q, kv, sc, 2, 16, q, stream=0),
           lambda: w.history_attention(0, [0, 3], [0], [0], q, kv, sc, 2, 16, q.half(), stream=0),
           lambda: w.history_attention(0, [0, 3], [0], [0], q.transpose(1, 2), kv, sc, 2, 16, q, stream=0),
           lambda: w.history_attention_frame(0, _b(4, dtype=torch.int32), q, kv, sc, 2, 16, q, stream=0)]
    for i, c in enumerate(bad):
        with pytest.raises(ValueError):
            c()
