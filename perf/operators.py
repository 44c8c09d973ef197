"""What is measured of the operators that bring a session into the batch.

A case names one of four operators:

  append   the rotary embedding, FP8 quantisation and append of packed prompts to the sessions' history
  attend   causal attention over packed prompts of different lengths, with grouped heads
  state    the selective-state block over packed prompts: a recurrence with a decay for each head
  copy     a session's history, state and position copied to other slots of the batch (a fork, or a
           compaction into free slots)

Lengths, slots and positions are lists written as texts.  `run` is either the plain form (elementary torch
operations in 32 bits) or, with `own`, the call that a user of the library makes.
"""
import math

import numpy as np
import torch

own = False

P, N = 64, 128  # head dim and state size of a selective-state head
ROPE_BASE = 10000.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# Sixteen sessions that join at the same frame, each with its own prompt: from a single token to two minutes of
# 12.5 Hz frames, on, below and above a multiple of 128.
ADMIT = "1500,37,613,250,1,980,128,129,444,77,1201,325,25,760,511,1024"


def listed():
    return [
        # one persona prompt of 25 frames (two seconds) on the small 16 x 64 shape: latency
        {"name": "attend 25, 16x64", "op": "attend", "lens": "25", "heads": 16, "kv_heads": 16, "dim": 64, "type": "bf16"},
        # sixteen sessions joining together on the 32 x 128 shape
        {"name": "attend 16 prompts, 32x128", "op": "attend", "lens": ADMIT, "heads": 32, "kv_heads": 32, "dim": 128, "type": "bf16"},
        # grouped heads, half precision, one long prompt with short ones beside it
        {"name": "attend grouped 32/8x128 f16", "op": "attend", "lens": "4096,1,2001", "heads": 32, "kv_heads": 8, "dim": 128,
         "type": "f16"},
        # a long context prompt: bound by the tensor cores
        {"name": "attend 8192, 32x128", "op": "attend", "lens": "8192", "heads": 32, "kv_heads": 32, "dim": 128, "type": "bf16"},
        # the same prompts' K and V into the history (qkv as a projection leaves it in 32 bits)
        {"name": "append 25, 16x64", "op": "append", "lens": "25", "starts": "0", "heads": 16, "dim": 64, "type": "bf16",
         "out": "bf16", "t_max": 64},
        {"name": "append 16 prompts, 32x128", "op": "append", "lens": ADMIT, "starts": ",".join(["0"] * 16), "heads": 32, "dim": 128,
         "type": "f32", "out": "bf16", "t_max": 1500},
        # a prompt of 25 tokens on the small hybrid shape: latency
        {"name": "state 25, 4 heads", "op": "state", "lens": "25", "starts": "0", "heads": 4},
        # one token for each of 56 sessions: the recurrent form, bound by the state's bytes
        {"name": "state 56 x 1, 64 heads", "op": "state", "lens": ",".join(["1"] * 56), "starts": ",".join(["9"] * 56), "heads": 64},
        # one prompt of 2048 tokens: few rows, a long axis
        {"name": "state 2048, 64 heads", "op": "state", "lens": "2048", "starts": "0", "heads": 64},
        # sixteen sessions joining, four of them going on from an earlier state
        {"name": "state 16 prompts, 64 heads", "op": "state", "lens": ADMIT,
         "starts": ",".join(str(9 * (i % 4 == 1)) for i in range(16)), "heads": 64},
        # one prepared persona forked into eight sessions (eight layers of the 32 x 128 shape)
        {"name": "copy 1 to 8, 32x128", "op": "copy", "src": ",".join(["0"] * 8), "dst": "1,2,3,4,5,6,7,8", "pos": "1500,-1,-1,-1,-1,-1,-1,-1,-1",
         "layers": 8, "attn_every": 0, "heads": 32, "dim": 128, "state_heads": 0, "t_max": 2000},
        # four sessions of the hybrid moved into the holes that others left (history and recurrent state)
        {"name": "copy 4 hybrid sessions", "op": "copy", "src": "12,13,14,15", "dst": "1,4,7,9",
         "pos": "310,-1,1200,45,-1,801,77,-1,640,-1,222,1499,1100,37,803,1", "layers": 12, "attn_every": 6, "heads": 32, "dim": 128,
         "state_heads": 64, "t_max": 1500},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "state", "state", "copy"])
    n = _log(rng, 1, 24)
    if op == "attend":
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8, 16])
        heads = kv * rng.choice([g for g in (1, 2, 3, 4, 8) if kv * g <= 32])
        lens = [_log(rng, 1, 5500 if n <= 2 else 1700) for _ in range(n)]
        return {"op": op, "lens": ",".join(map(str, lens)), "heads": heads, "kv_heads": kv, "dim": dim, "type": rng.choice(["bf16", "bf16", "f16"])}
    if op == "append":
        dim, heads = rng.choice([(64, 4), (64, 16), (128, 8), (128, 32)])
        lens = [_log(rng, 1, 2500 if n <= 4 else 1200) for _ in range(n)]
        starts = [rng.choice([0, 0, _log(rng, 1, 500)]) for _ in range(n)]
        t_max = (max(a + b for a, b in zip(lens, starts)) + 3) // 4 * 4
        return {"op": op, "lens": ",".join(map(str, lens)), "starts": ",".join(map(str, starts)), "heads": heads, "dim": dim,
                "type": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f16"]), "t_max": t_max}
    if op == "state":
        heads = 4 * _log(rng, 1, 16)
        lens = [_log(rng, 1, 2500 if n <= 2 else 1200) for _ in range(n)]
        starts = [rng.choice([0, 7]) for _ in range(n)]
        return {"op": op, "lens": ",".join(map(str, lens)), "starts": ",".join(map(str, starts)), "heads": heads}
    s = rng.randint(4, 16)
    order = rng.sample(range(s), s)
    k = rng.randint(1, s // 2)
    hybrid = rng.random() < 0.5
    t_max = 4 * _log(rng, 16, 375)
    dst = order[:k]
    src = [rng.choice(order[k:]) for _ in dst]
    pos = [rng.randint(0, t_max) if i in src else rng.choice([-1, rng.randint(0, t_max)]) for i in range(s)]
    dim, heads = rng.choice([(64, 16), (128, 8), (128, 32)])
    return {"op": "copy", "src": ",".join(map(str, src)), "dst": ",".join(map(str, dst)), "pos": ",".join(map(str, pos)),
            "layers": 6 if hybrid else rng.randint(1, 6), "attn_every": 3 if hybrid else 0, "heads": heads, "dim": dim,
            "state_heads": 4 * rng.randint(1, 12) if hybrid else 0, "t_max": t_max}


def _ints(text):
    return [int(v) for v in text.split(",")]


def _cu(lens):
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    return cu


def _padding(lens, device):
    """[sequences][longest] row numbers of the packed tokens, and which of them are there."""
    at = torch.arange(max(lens), device=device)
    first = torch.tensor(_cu(lens)[:-1], device=device)
    return first[:, None] + at[None, :], at[None, :] < torch.tensor(lens, device=device)[:, None]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    c, st = case, {"case": case}
    if c["op"] in ("append", "attend", "state"):
        st["lens"] = _ints(c["lens"])
        st["cu"] = _cu(st["lens"])
        n = st["cu"][-1]
        st["rows"], st["there"] = _padding(st["lens"], "cuda")
        # the sessions' slots, in another order than the prompts
        st["slots"] = [(5 * i + 2) % len(st["lens"]) if len(st["lens"]) % 5 else i for i in range(len(st["lens"]))]
    if c["op"] == "attend":
        t = TYPES[c["type"]]
        # q and k after a norm and the rotary embedding: a few units wide, so that a softmax has a peak
        st["q"] = (1.5 * randn(n, c["heads"], c["dim"])).to(t)
        st["k"] = (1.5 * randn(n, c["kv_heads"], c["dim"])).to(t)
        st["v"] = randn(n, c["kv_heads"], c["dim"]).to(t)
        st["out"] = torch.zeros_like(st["q"])
    elif c["op"] == "append":
        hd = c["heads"] * c["dim"]
        st["starts"] = _ints(c["starts"])
        st["qkv"] = (2.0 * randn(n, 3 * hd)).to(TYPES[c["type"]])
        s, t = len(st["lens"]), c["t_max"]
        st["kv"] = torch.zeros((1, 2, s, c["heads"], t, c["dim"]), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros((1, 2, s, c["heads"], t), device="cuda")
        for x in "qkv":
            st[x] = torch.zeros((n, c["heads"], c["dim"]), dtype=TYPES[c["out"]], device="cuda")
        st["pos"] = torch.cat([torch.arange(v, device="cuda") + s0 for v, s0 in zip(st["lens"], st["starts"])])
        st["slot_of"] = torch.cat([torch.full((v,), s0, device="cuda") for v, s0 in zip(st["lens"], st["slots"])])
    elif c["op"] == "state":
        hs = c["heads"]
        st["starts"] = _ints(c["starts"])
        st["zx"] = randn(n, 2 * hs * P + 2 * N + hs).to(torch.bfloat16)
        # A = -exp(A_log): from a head that forgets at once to one that hardly forgets, as the model draws it
        st["a_log"], st["dt_bias"], st["d"] = randn(hs).to(torch.bfloat16), (randn(hs) - 2).to(torch.bfloat16), randn(hs).to(torch.bfloat16)
        st["state_in"] = randn(1, len(st["lens"]), hs, P, N)
        st["state_out"] = torch.zeros_like(st["state_in"])
        st["out"] = torch.zeros((n, hs * P), dtype=torch.bfloat16, device="cuda")
        st["slots_d"] = torch.tensor(st["slots"], device="cuda")
        st["goes_on"] = torch.tensor([v > 0 for v in st["starts"]], device="cuda")
    else:
        st["src"], st["dst"], pos = _ints(c["src"]), _ints(c["dst"]), _ints(c["pos"])
        s, t = len(pos), c["t_max"]
        la = c["layers"] // c["attn_every"] if c["attn_every"] else c["layers"]
        st["positions"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        st["kv"] = torch.randint(0, 127, (la, 2, s, c["heads"], t, c["dim"]), dtype=torch.uint8, device="cuda", generator=g)
        st["scales"] = torch.rand((la, 2, s, c["heads"], t), device="cuda", generator=g)
        st["state"] = randn(c["layers"] - la, s, c["state_heads"], P, N) if c["state_heads"] else None
        st["src_d"], st["dst_d"] = torch.tensor(st["src"], device="cuda"), torch.tensor(st["dst"], device="cuda")
    if own:
        import frame_step_decode_gb300 as fsd
        st["wave"] = _handle(fsd, c, st)
    return st


def _handle(fsd, c, st):
    """The handle that a user's program made when it loaded the model, and the packed weights beside it."""
    if c["op"] == "attend":
        return fsd.Wave(fsd.WaveConfig(1, 64, c["heads"], c["dim"], 64, 1e-5, ROPE_BASE), 1, 64)
    if c["op"] == "append":
        return fsd.Wave(fsd.WaveConfig(1, 64, c["heads"], c["dim"], 64, 1e-5, ROPE_BASE), len(st["lens"]), c["t_max"])
    if c["op"] == "state":
        cfg = fsd.WaveHybridConfig(2, 64, 2, 1, 64, c["heads"], P, N, 1e-5, ROPE_BASE)
        blob = torch.zeros(fsd.hybrid_weights_bytes(cfg) // 2, dtype=torch.bfloat16, device="cuda")
        block = (3 * c["heads"] + 7) // 8 * 8
        first = fsd.hybrid_layer_offset(cfg, 1) // 2 - block  # the end of the first block: A_log, dt_bias, D
        blob[first:first + 3 * c["heads"]] = torch.cat([st["a_log"], st["dt_bias"], st["d"]])
        st["weights"] = fsd.hybrid_pack_weights(cfg, blob)
        return fsd.HybridWave(cfg, len(st["lens"]), 64)
    s = st["positions"].numel()
    if c["attn_every"]:
        return fsd.HybridWave(fsd.WaveHybridConfig(c["layers"], 64, c["attn_every"], c["heads"], c["dim"], c["state_heads"], P, N, 1e-5,
                                                   ROPE_BASE), s, c["t_max"])
    return fsd.Wave(fsd.WaveConfig(c["layers"], 64, c["heads"], c["dim"], 64, 1e-5, ROPE_BASE), s, c["t_max"])


def _outputs(st):
    """The buffers that a case's operator fills; 8-bit codes as the numbers that they stand for."""
    op = st["case"]["op"]
    if op == "attend":
        return st["out"]
    if op == "append":
        return {"q": st["q"], "k": st["k"], "v": st["v"], "codes": st["kv"].view(torch.float8_e4m3fn), "scales": st["scales"]}
    if op == "state":
        return {"out": st["out"], "state": st["state_out"]}
    got = {"codes": st["kv"].view(torch.float8_e4m3fn), "scales": st["scales"], "positions": st["positions"]}
    return got if st["state"] is None else got | {"state": st["state"]}


def run(st):
    op = st["case"]["op"]
    if own:
        w = st["wave"]
        if op == "attend":
            w.prompt_attention(st["cu"], st["q"], st["k"], st["v"], st["out"])
        elif op == "append":
            w.prompt_append(0, st["cu"], st["slots"], st["starts"], st["qkv"], st["kv"], st["scales"], st["q"], st["k"], st["v"])
        elif op == "state":
            w.prompt_state(0, st["weights"], st["cu"], st["slots"], st["starts"], st["zx"], st["state_in"], st["state_out"], st["out"])
        else:
            w.sessions_copy(st["src"], st["dst"], st["kv"], st["scales"], st["positions"], state=st["state"])
        return _outputs(st)
    {"attend": _attend, "append": _append, "state": _state, "copy": _copy}[op](st)
    return _outputs(st)


def _attend(st):
    q, k, v = st["q"], st["k"], st["v"]
    rows, there = st["rows"].clamp(max=q.shape[0] - 1), st["there"]
    group = q.shape[1] // k.shape[1]
    b, m = rows.shape
    pad = lambda x: x[rows].float().permute(0, 2, 1, 3)  # noqa: E731  [b][heads][m][d]
    qp = pad(q).reshape(b, k.shape[1], group * m, -1)
    s = (qp @ pad(k).transpose(-1, -2)).reshape(b, k.shape[1], group, m, m) / math.sqrt(q.shape[2])
    at = torch.arange(m, device=q.device)
    s.masked_fill_(at[None, :] > at[:, None], -math.inf)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    s /= s.sum(-1, keepdim=True)
    o = (s.reshape(b, k.shape[1], group * m, m) @ pad(v)).reshape(b, q.shape[1], m, -1).permute(0, 2, 1, 3)
    st["out"][st["rows"][there]] = o[there].to(q.dtype)


def _append(st):
    c = st["case"]
    h, d = c["heads"], c["dim"]
    x = st["qkv"].float().reshape(-1, 3, h, d)
    freq = ROPE_BASE ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    ang = st["pos"].double()[:, None] * freq
    cos, sin = ang.cos().float()[:, None, None], ang.sin().float()[:, None, None]
    a, b = x[:, :2, :, :d // 2], x[:, :2, :, d // 2:]
    qk = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    kv = torch.stack([qk[:, 1], x[:, 2]], 1)  # [tokens][K|V][heads][d]
    scale = kv.abs().amax(-1) / 448.0
    codes = torch.where(scale[..., None] == 0, 0.0, kv / scale[..., None]).to(torch.float8_e4m3fn)
    back = codes.float() * scale[..., None]
    # the history is [K|V][slot][heads][t][d]
    st["kv"][0].permute(1, 3, 0, 2, 4)[st["slot_of"], st["pos"]] = codes.view(torch.uint8)
    st["scales"][0].permute(1, 3, 0, 2)[st["slot_of"], st["pos"]] = scale
    st["q"].copy_(qk[:, 0])
    st["k"].copy_(back[:, 0])
    st["v"].copy_(back[:, 1])


def _state(st):
    hs = st["case"]["heads"]
    di = hs * P
    rows, there = st["rows"].clamp(max=st["zx"].shape[0] - 1), st["there"]
    zx = st["zx"][rows].float()  # [b][m][...]
    b, m = rows.shape
    z, x = zx[..., :di].reshape(b, m, hs, P), zx[..., di:2 * di].reshape(b, m, hs, P)
    bb, cc = zx[..., 2 * di:2 * di + N], zx[..., 2 * di + N:2 * di + 2 * N]
    raw = zx[..., 2 * di + 2 * N:] + st["dt_bias"].float()
    dt = (torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)) * there[..., None]  # a token that is not there changes nothing
    cum = (-torch.exp(st["a_log"].float()) * dt).double().cumsum(1).permute(0, 2, 1)  # [b][hs][m]: the log of the decay so far
    at = torch.arange(m, device=zx.device)
    decay = (cum[:, :, :, None] - cum[:, :, None, :]).float()
    decay.masked_fill_(at[None, :] > at[:, None], -math.inf).exp_()
    decay *= (cc @ bb.transpose(-1, -2))[:, None]
    u = (x * dt[..., None]).permute(0, 2, 1, 3)  # [b][hs][m][P]
    h0 = torch.where(st["goes_on"][:, None, None, None], st["state_in"][0][st["slots_d"]], 0.0)
    y = decay @ u + cum.float().exp()[..., None] * (cc[:, None] @ h0.transpose(-1, -2))
    y = y.permute(0, 2, 1, 3) + st["d"].float()[:, None] * x
    out = (y * (z / (1 + torch.exp(-z)))).reshape(b, m, di)
    st["out"][st["rows"][there]] = out[there].to(torch.bfloat16)
    last = (cum[:, :, -1:] - cum).float().exp()
    h = cum[:, :, -1].float().exp()[..., None, None] * h0 + (u * last[..., None]).transpose(-1, -2) @ bb[:, None]
    st["state_out"][0][st["slots_d"]] = h


def _copy(st):
    src, dst = st["src_d"], st["dst_d"]
    pos = st["positions"][src]
    held = torch.arange(st["kv"].shape[4], device="cuda")[None, :] < pos[:, None]  # [pairs][t]
    st["kv"][:, :, dst] = torch.where(held[:, None, :, None], st["kv"][:, :, src], st["kv"][:, :, dst])
    st["scales"][:, :, dst] = torch.where(held[:, None, :], st["scales"][:, :, src], st["scales"][:, :, dst])
    if st["state"] is not None:
        st["state"][:, dst] = torch.where(pos[:, None, None, None] >= 0, st["state"][:, src], st["state"][:, dst])
    st["positions"][dst] = pos


def work(case):
    c = case
    if c["op"] == "copy":
        src, dst, pos = _ints(c["src"]), _ints(c["dst"]), _ints(c["pos"])
        la = c["layers"] // c["attn_every"] if c["attn_every"] else c["layers"]
        held = lambda s: la * 2 * c["heads"] * max(0, pos[s]) * (c["dim"] + 4) + (pos[s] >= 0) * (  # noqa: E731
            (c["layers"] - la) * c["state_heads"] * P * N * 4) + 4
        return {"bytes": sum(held(s) for s in set(src)) + sum(held(s) for s in src), "flops": 0}
    lens = _ints(c["lens"])
    n = sum(lens)
    if c["op"] == "attend":
        return {"bytes": 2 * n * c["dim"] * 2 * (c["heads"] + c["kv_heads"]),
                "flops": sum(4 * c["dim"] * v * (v + 1) // 2 for v in lens) * c["heads"]}
    if c["op"] == "append":
        hd = c["heads"] * c["dim"]
        size = 4 if c["type"] == "f32" else 2
        return {"bytes": n * (3 * hd * size + 3 * hd * 2 + 2 * hd + 2 * c["heads"] * 4), "flops": n * hd * 14}
    hs = c["heads"]
    states = len(lens) + sum(v > 0 for v in _ints(c["starts"]))
    return {"bytes": n * 2 * (2 * hs * P + 2 * N + hs) + n * 2 * hs * P + states * hs * P * N * 4, "flops": n * hs * P * N * 5}


# ---- the definitions in 64 bits, sequence by sequence


def exact(case, seed):
    if case["op"] == "copy":
        return None
    st = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "state": _exact_state}[case["op"]](case, st)


def _exact_attend(c, st):
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for a, b in zip(st["cu"], st["cu"][1:]):
        for h in range(c["heads"]):
            g = h // (c["heads"] // c["kv_heads"])
            s = torch.mm(st["q"][a:b, h].double(), st["k"][a:b, g].double().t()) * c["dim"] ** -0.5
            s = torch.softmax(s + torch.full_like(s, -math.inf).triu(1), dim=1)
            out[a:b, h] = torch.mm(s, st["v"][a:b, g].double())
    return out


def _exact_append(c, st):
    h, d = c["heads"], c["dim"]
    x = st["qkv"].double().cpu().numpy().reshape(-1, 3, h, d)
    pos = np.concatenate([s + np.arange(n) for n, s in zip(st["lens"], st["starts"])])
    turn = np.exp(1j * pos[:, None] * ROPE_BASE ** (-np.arange(0, d, 2) / d))[:, None]  # a rotation of each pair (i, i + d/2)
    rot = [(x[:, i, :, :d // 2] + 1j * x[:, i, :, d // 2:]) * turn for i in (0, 1)]
    q, k = (np.concatenate([r.real, r.imag], -1) for r in rot)
    scales = np.zeros((1, 2, len(st["lens"]), h, c["t_max"]))
    slot = np.concatenate([np.full(n, s) for n, s in zip(st["lens"], st["slots"])])
    for i, rows in enumerate((k, x[:, 2])):
        scales[0, i, slot, :, pos] = np.abs(rows).max(-1) / 448
    return {"q": q, "k": None, "v": None, "codes": None, "scales": scales}


def _exact_state(c, st):
    hs, di = c["heads"], c["heads"] * P
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    states = torch.zeros(st["state_out"].shape, dtype=torch.float64, device="cuda")
    a_neg, skip = -torch.exp(st["a_log"].double()), st["d"].double()
    # the recurrence, one token of every sequence that is that long at a time
    order = sorted(range(len(st["lens"])), key=lambda i: -st["lens"][i])
    lens = [st["lens"][i] for i in order]
    first = torch.tensor([st["cu"][i] for i in order], device="cuda")
    slot = torch.tensor([st["slots"][i] for i in order], device="cuda")
    on = torch.tensor([float(st["starts"][i] > 0) for i in order], device="cuda", dtype=torch.float64)
    h = st["state_in"][0][slot].double() * on[:, None, None, None]
    dts = torch.nn.functional.softplus(st["zx"][:, 2 * di + 2 * N:].double() + st["dt_bias"].double())
    for t in range(lens[0]):
        k = sum(v > t for v in lens)
        row = first[:k] + t
        r, dt = st["zx"][row].double(), dts[row]
        x = r[:, di:2 * di].reshape(k, hs, P)
        h[:k] = h[:k] * torch.exp(a_neg * dt)[..., None, None] + (dt[..., None] * x)[..., None] * r[:, None, None, 2 * di:2 * di + N]
        y = torch.einsum("shpn,sn->shp", h[:k], r[:, 2 * di + N:2 * di + 2 * N]) + skip[:, None] * x
        out[row] = y.reshape(k, di) * torch.nn.functional.silu(r[:, :di])
    states[0][slot] = h
    return {"out": out, "state": states}
