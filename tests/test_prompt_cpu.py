"""CPU: the calls on packed prompts and sessions refuse a missing handle and
badly shaped tensors without touching a device."""
import numpy as np
import pytest
import torch

import frame_step_decode_gb300 as fsd


def _unbound(cls, cfg):
    """A binding object whose handle is NULL (no device here to create one)."""
    w = cls.__new__(cls)
    w.cfg, w.h = cfg, None
    return w


def _decoder():
    return _unbound(fsd.Wave, fsd.WaveConfig(1, 64, 2, 64, 64, 1e-5, 1e4))


def _hybrid():
    return _unbound(fsd.HybridWave, fsd.WaveHybridConfig(2, 64, 2, 1, 64, 4, 64, 128, 1e-5, 1e4))


def _b(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_a_missing_handle_is_refused():
    w, h = _decoder(), _hybrid()
    kv, sc, pos = _b(8, dtype=torch.uint8), _b(8, dtype=torch.float32), _b(4, dtype=torch.int32)
    calls = [lambda: w.prompt_append(0, [0, 3], [0], [0], _b(3, 384), kv, sc, stream=0),
             lambda: w.prompt_attention([0, 3], _b(3, 2, 64), _b(3, 1, 64), _b(3, 1, 64), _b(3, 2, 64), stream=0),
             lambda: h.prompt_state(0, kv, [0, 3], [0], [0], _b(3, 772), None, sc, _b(3, 256), stream=0),
             lambda: w.sessions_copy([0], [1], kv, sc, pos, stream=0)]
    for c in calls:
        with pytest.raises(fsd.WaveError) as e:
            c()
        assert e.value.code == fsd.WAVE_EINVAL


def test_shapes_that_do_not_fit_are_refused():
    w, h = _decoder(), _hybrid()
    kv, sc, pos = _b(8, dtype=torch.uint8), _b(8, dtype=torch.float32), _b(4, dtype=torch.int32)
    q, k, out = _b(3, 2, 64), _b(3, 1, 64), _b(3, 2, 64)
    bad = [lambda: w.prompt_append(0, [0, 3], [0, 1], [0], _b(3, 384), kv, sc, stream=0),
           lambda: w.prompt_append(0, [0, 3], [0], [0], _b(3, 380), kv, sc, stream=0),
           lambda: w.prompt_append(0, [0, 4], [0], [0], _b(3, 384), kv, sc, stream=0),
           lambda: w.prompt_append(0, [0, 3], [0], [0], _b(3, 384), kv, sc, q=_b(3, 2, 32), stream=0),
           lambda: w.prompt_append(0, [0, 3], [0], [0], _b(3, 384), kv, sc, q=_b(3, 2, 64), k=_b(3, 2, 64, dtype=torch.float16), stream=0),
           lambda: w.prompt_attention([0, 4], q, k, k, out, stream=0),
           lambda: w.prompt_attention([0, 3], q, k, k, out.float(), stream=0),
           lambda: w.prompt_attention([0, 3], q, k, _b(3, 2, 64), out, stream=0),
           lambda: w.prompt_attention([0, 3], _b(3, 64, 2).transpose(1, 2), k, k, out, stream=0),
           lambda: w.prompt_attention([0, 3], _b(3, 4, 64), k, k, out, stream=0),
           lambda: h.prompt_state(0, kv, [0, 3], [0], [0], _b(3, 771), None, sc, _b(3, 256), stream=0),
           lambda: h.prompt_state(0, kv, [0, 3], [0], [0], _b(3, 772, dtype=torch.float32), None, sc, _b(3, 256), stream=0),
           lambda: h.prompt_state(0, kv, [0, 3], [0, 1], [0], _b(3, 772), None, sc, _b(3, 256), stream=0),
           lambda: h.prompt_state(0, kv, [0, 3], [0], [0], _b(3, 772), None, sc, _b(3, 255), stream=0),
           lambda: w.sessions_copy([0], [1, 2], kv, sc, pos, stream=0)]
    for i, c in enumerate(bad):
        with pytest.raises(ValueError):
            c()


def test_integers_beyond_32_bits_are_refused():
    w = _decoder()
    kv, sc, pos = _b(8, dtype=torch.uint8), _b(8, dtype=torch.float32), _b(4, dtype=torch.int32)
    q, k = _b(3, 2, 64), _b(3, 1, 64)
    bad = [lambda: w.prompt_append(0, [0, 3], [2 ** 32], [0], _b(3, 384), kv, sc, stream=0),
           lambda: w.prompt_append(0, [0, 3], [0], [-2 ** 31 - 1], _b(3, 384), kv, sc, stream=0),
           lambda: w.prompt_attention([2 ** 32, 2 ** 32 + 3], q, k, k, q, stream=0),
           lambda: w.sessions_copy([0.5], [1], kv, sc, pos, stream=0)]
    for c in bad:
        with pytest.raises(ValueError):
            c()
    for values in (torch.tensor([3, -1]), np.array([3, -1]), (3, -1)):
        assert fsd._ints(values) == (np.array([3, -1], dtype=np.int32).tobytes(), 2)


class _Accepts:
    """A library whose calls all succeed: what reaches it has passed the binding's checks."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


def _bound(w, S_max, T_max, monkeypatch):
    """w as if it had a handle, for buffers on the CPU (device -1), and its calls counted."""
    fake = _Accepts()
    w.S_max, w.T_max = S_max, T_max
    w._sizes()  # of the packed weights by the library itself
    w.device = -1
    monkeypatch.setattr(fsd, "lib", lambda: fake)
    monkeypatch.setattr(type(w), "close", lambda self: None)
    w.h = 1
    return w, fake


def test_buffers_of_another_size_or_type_are_refused(monkeypatch):
    """History, scales, state, weights and positions are read and written by
    slot: too few values, another type, gaps or another device would be out of
    range or the wrong bytes on the device."""
    S, T = 4, 64
    w, fake = _bound(_decoder(), S, T, monkeypatch)
    kv, sc = _b(1, 2, S, 2, T, 64, dtype=torch.uint8), _b(1, 2, S, 2, T, dtype=torch.float32)
    pos = _b(S, dtype=torch.int32)
    qkv, q = _b(3, 384), _b(3, 2, 64)
    append = lambda kv=kv, sc=sc, **kw: w.prompt_append(0, [0, 3], [0], [0], qkv, kv, sc, stream=0, **kw)  # noqa: E731
    copy = lambda kv=kv, sc=sc, pos=pos, **kw: w.sessions_copy([0], [1], kv, sc, pos, stream=0, **kw)  # noqa: E731
    attend = lambda: w.prompt_attention([0, 3], q, q, q, q, stream=0)  # noqa: E731
    append(), append(q=q), copy(), attend()
    append(kv=kv.view(torch.float8_e4m3fn), sc=4096)  # codes of any one-byte type; an address is the caller's
    assert fake.calls == 5
    bad = [lambda f=f, kw=kw: f(**kw) for f in (append, copy) for kw in
           (dict(kv=kv.flatten()[:-1]), dict(kv=kv.to(torch.float16)), dict(kv=kv.transpose(3, 4)), dict(sc=sc.flatten()[:-1]),
            dict(sc=sc.to(torch.bfloat16)), dict(sc=sc.double()), dict(sc=sc.transpose(3, 4)))]
    bad += [lambda: copy(pos=pos.long()), lambda: copy(pos=pos[:3]), lambda: copy(pos=_b(8, dtype=torch.int32)[::2]),
            lambda: copy(pos=pos.float())]
    for c in bad:
        with pytest.raises(ValueError):
            c()
    w.device = 0  # the tensors are elsewhere
    for c in (append, copy, attend, lambda: append(kv=4096, sc=4096)):
        with pytest.raises(ValueError):
            c()
    assert fake.calls == 5



def test_state_buffers_of_another_size_or_type_are_refused(monkeypatch):
    S, T = 4, 64
    n = fsd.hybrid_packed_weights_bytes(_hybrid().cfg)
    h, fake = _bound(_hybrid(), S, T, monkeypatch)
    pos = _b(S, dtype=torch.int32)
    wt, st, zx, out = _b(n // 2), _b(1, S, 4, 64, 128, dtype=torch.float32), _b(3, 772), _b(3, 256)
    state = lambda wt=wt, si=st, so=st: h.prompt_state(0, wt, [0, 3], [0], [2], zx, si, so, out, stream=0)  # noqa: E731
    state(), state(si=None)
    for kw in (dict(wt=wt[:-1]), dict(wt=wt.float()), dict(si=st.half()), dict(si=st[:, :3]), dict(so=st.to(torch.bfloat16)),
               dict(so=st.flatten()[:-4]), dict(so=st.transpose(3, 4)), dict(so=st.double())):
        with pytest.raises(ValueError):
            state(**kw)
    for kw in (dict(state=st.half()), dict(state=st.flatten()[1:])):
        with pytest.raises(ValueError):
            h.sessions_copy([0], [1], _b(1, 2, S, 1, T, 64, dtype=torch.uint8), _b(1, 2, S, 1, T, dtype=torch.float32), pos, stream=0, **kw)
    assert fake.calls == 2


@pytest.mark.parametrize("raw", [True, False])
def test_the_current_stream_with_and_without_the_raw_getter(monkeypatch, raw):
    """The handle of torch's current stream, also where torch does not export
    the function that gives it without a Stream object."""
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(fsd, "_CURRENT", [])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream if device == 3 else None)
    if raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 77 if device == 3 else 0, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert fsd._stream(None) == 77 and fsd._stream(None) == 77
    assert fsd._stream(5) == 5 and fsd._stream(Stream) == 77
