"""Sessions that are appended to, attended and stepped in turns: the history in
blocks of one token, with as many K/V heads as query heads, is the step's own."""
import numpy as np
import pytest
import torch

import frame_step_decode_gb300 as fsd
import synth
from gpu_case import DeviceCase
from test_gpu_history import BF, Cache, _cu, _gen
from test_gpu_history_edges import seen_reference
from test_gpu_step import _y_within_sensitivity

pytestmark = pytest.mark.gpu


def _layer(case, layer):
    """Layer `layer` of the case's history, as the references of attention take it."""
    c = Cache.__new__(Cache)
    c.__dict__.update(kv=case.kv, sc=case.sc, layer=layer, block=1, Hkv=case.w.n_heads, S=case.S, T=case.w.T_max, D=case.w.head_dim)
    return c


def _near(c, q, out, lens, slots, starts, cu):
    ref, tol = seen_reference(c, q, lens, slots, starts, cu, q.shape[2] ** -0.5)
    for a, b in zip(cu, cu[1:]):
        assert bool(((out.double() - ref).abs() <= tol)[a:b].all())


@pytest.mark.parametrize("w", [synth.TINY, synth.MID], ids=lambda w: w.name)
def test_sessions_appended_attended_and_stepped_in_turns(w):
    """Prompts of every length, none among them, that begin sessions and go on after steps, of few rows and of many: each
    attention is the formula's over what appends and steps have left; each step is the oracle's over the same history, writes one
    token of it and moves nothing else; what it wrote is read back and attended to as the rest."""
    S, H, D, L, T = 4, w.n_heads, w.head_dim, w.n_layers, w.T_max
    case = DeviceCase(w, S=S, pos=[0] * S)
    wave = fsd.Wave(case.cfg, S, T)
    plan = fsd.rope_plan(D, w.rope_base)
    W = synth.weights_host(w)
    pos = np.zeros(S, np.int32)
    small = T < 100
    rounds = [([20, 1, 9, 33], 1), ([0, 12, 1, 2], 2), ([3, 0, 17, 1], 1)] if small else [([90, 1, 40, 128], 1), ([0, 50, 33, 2], 2), ([3, 0, 70, 100], 1)]
    try:
        for r, (lens, steps) in enumerate(rounds):
            slots, cu = [2, 0, 3, 1], _cu(lens)
            starts = [int(pos[s]) for s in slots]
            for layer in range(L):
                qkv = torch.randn(cu[-1], 3 * H * D, generator=_gen(100 * r + layer), device="cuda").to(BF)
                q, out = (torch.zeros(cu[-1], H, D, dtype=BF, device="cuda") for _ in range(2))
                wave.history_append(layer, cu, slots, starts, qkv, case.kv, case.sc, H, 1, rope=plan, q=q)
                wave.history_attention(layer, cu, slots, starts, q, case.kv, case.sc, H, 1, out)
                _near(_layer(case, layer), q, out, lens, slots, starts, cu)
            for s, n in zip(slots, lens):
                pos[s] += n
            for k in range(steps):
                case.pos.copy_(torch.from_numpy(pos))
                kv, sc = case.kv.clone(), case.sc.clone()
                case.step(wave)
                assert wave.status() == fsd.WAVE_OK
                _y_within_sensitivity(w, W, pos, case.x_h, case.y_bits(), kv.cpu().numpy(), sc.cpu().numpy())
                for s in range(S):  # but for the token that it wrote
                    kv[:, :, s, :, pos[s]], sc[:, :, s, :, pos[s]] = case.kv[:, :, s, :, pos[s]], case.sc[:, :, s, :, pos[s]]
                assert torch.equal(kv, case.kv) and torch.equal(sc.nan_to_num(nan=-7.0), case.sc.nan_to_num(nan=-7.0))
                for layer in range(L):
                    c = _layer(case, layer)
                    q = torch.randn(S, H, D, generator=_gen(7000 + 100 * r + 10 * k + layer), device="cuda").to(BF)
                    out = torch.zeros_like(q)
                    wave.history_attention_frame(layer, case.pos, q, case.kv, case.sc, H, 1, out)
                    _near(c, q, out, [1] * S, list(range(S)), pos.tolist(), _cu([1] * S))
                    new = [torch.zeros(S, H, D, device="cuda") for _ in range(2)]
                    wave.history_read(layer, _cu([1] * S), list(range(S)), pos.tolist(), case.kv, case.sc, H, 1, *new)
                    for which in (0, 1):
                        for s in range(S):
                            assert torch.equal(new[which][s], c.values(which, s, int(pos[s]), int(pos[s]) + 1, torch.float32)[:, 0])
                        assert bool(new[which].isfinite().all()) and bool((new[which] != 0).any())
                pos += 1
        assert wave.status() == fsd.WAVE_OK
    finally:
        wave.close()
