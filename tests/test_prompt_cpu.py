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
