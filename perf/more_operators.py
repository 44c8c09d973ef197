"""What is measured of the block-scaled history, the attention that reads it and the rotary positions of its keys.

A case names one of four operators:

  rotate   rotary positions on packed rows: half or interleaved pairs, part of a head, frequencies scaled for long contexts
  append   the rotation, 8-bit quantisation and append of packed tokens, or of a frame of single ones, to the history;
           one scale for each block of tokens and head (a block of 1 is the history that the step reads)
  read     the history's keys and values back in 16 or 32 bits
  attend   attention over the history: of prompts that go on from what a session holds, and of a frame of single tokens

Lengths and positions are lists written as texts.  `run` is either the plain form (elementary torch operations in 32
bits) or, with `own`, the call that a user of the library makes.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCKS = [1, 16, 32, 64, 128]

# Sixteen sessions that join at the same frame, each with its own prompt: from a single token to two minutes of
# 12.5 Hz frames, on, below and above a multiple of 128.
ADMIT = "1500,37,613,250,1,980,128,129,444,77,1201,325,25,760,511,1024"

# Rotary forms: the step's; half of each head in interleaved pairs; contexts eight times longer than trained on, by
# slower turns for all pairs or only for those that turn seldom.
ROPES = {
    "step": {"layout": "half", "part": 1.0, "scaling": "none"},
    "part": {"layout": "interleaved", "part": 0.5, "scaling": "none"},
    "linear": {"layout": "half", "part": 1.0, "scaling": "linear"},
    "parts": {"layout": "interleaved", "part": 1.0, "scaling": "parts"},
}
FACTOR, ORIGINAL, FAST, SLOW = 8.0, 4096.0, 32.0, 1.0
AMPLITUDE = {"none": 1.0, "linear": 1.0, "parts": 0.1 * math.log(FACTOR) + 1.0}
BASE = 10000.0


def _spread(n, most):
    """n positions spread over [0, most), in no order."""
    return ",".join(str((i * 7919 + 211) % most) for i in range(n))


def listed():
    return [
        # the queries and keys of one persona prompt of 25 frames on the small 16 x 64 shape: latency
        {"name": "rotate 25, 16x64", "op": "rotate", "lens": "25", "starts": "0", "heads": 32, "dim": 64, "rope": "step", "type": "bf16", "out": "bf16"},
        # sixteen sessions joining, 32 query and 8 key heads, a long-context model
        {"name": "rotate 16 prompts, 40x128", "op": "rotate", "lens": ADMIT, "starts": ",".join(["0"] * 16), "heads": 40, "dim": 128,
         "rope": "parts", "type": "bf16", "out": "bf16"},
        # the same prompt of 25 frames into blocks of 16: latency
        {"name": "append 25, 16x64", "op": "append", "lens": "25", "starts": "0", "heads": 16, "kv_heads": 16, "dim": 64, "block": 16,
         "rope": "step", "type": "bf16", "out": "bf16", "frame": False},
        # sixteen sessions, some going on in the middle of a block (qkv as a projection leaves it in 32 bits)
        {"name": "append 16 prompts, 32/8x128", "op": "append", "lens": ADMIT, "starts": ",".join(str(37 * (i % 4 == 1)) for i in range(16)),
         "heads": 32, "kv_heads": 8, "dim": 128, "block": 64, "rope": "parts", "type": "f32", "out": "bf16", "frame": False},
        # one frame of the whole batch: a token of each of 80 sessions
        {"name": "append a frame of 80, 32/8x128", "op": "append", "lens": ",".join(["1"] * 80), "starts": _spread(80, 3000), "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 64, "rope": "part", "type": "bf16", "out": "bf16", "frame": True},
        # one session's history read back
        {"name": "read 37, 4x64", "op": "read", "lens": "37", "starts": "0", "kv_heads": 4, "dim": 64, "block": 16, "out": "bf16"},
        # sixteen sessions' (to hand them to another engine, or to a layer that wants 16 bits)
        {"name": "read 16 sessions, 32x128", "op": "read", "lens": ADMIT, "starts": ",".join(["0"] * 16), "kv_heads": 32, "dim": 128,
         "block": 1, "out": "bf16"},
        # one frame of 80 sessions with up to 3000 tokens, grouped heads: bound by the history's bytes
        {"name": "attend a frame of 80, 32/8x128", "op": "attend", "lens": ",".join(["1"] * 80), "starts": _spread(80, 3000), "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 64, "type": "bf16", "frame": True},
        # one session with a long context: few rows, a long axis
        {"name": "attend 1 after 32000, 32/8x128", "op": "attend", "lens": "1", "starts": "32000", "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 128, "type": "bf16", "frame": True},
        # a second prompt of 25 frames to a session of two minutes, over the step's own history
        {"name": "attend 25 after 1475, 16x64", "op": "attend", "lens": "25", "starts": "1475", "heads": 16, "kv_heads": 16, "dim": 64,
         "block": 1, "type": "bf16", "frame": False},
        # a document that goes on: bound by the tensor cores
        {"name": "attend 1024 after 7168, 32x128", "op": "attend", "lens": "1024", "starts": "7168", "heads": 32, "kv_heads": 32, "dim": 128,
         "block": 128, "type": "f16", "frame": False},
        # sessions that go on, long and short together
        {"name": "attend 4 going on, 32/8x128", "op": "attend", "lens": "2001,300,17,1", "starts": "4096,1200,2900,801", "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 32, "type": "bf16", "frame": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _join(values):
    return ",".join(map(str, values))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "read", "attend", "attend", "attend"])
    n = _log(rng, 1, 24)
    some = lambda most: [rng.randint(1, most) for _ in range(n)]  # noqa: E731
    after = lambda most: [rng.choice([0, rng.randint(1, most)]) for _ in range(n)]  # noqa: E731
    dim = rng.choice([64, 128])
    if op == "rotate":
        return {"op": op, "lens": _join(some(_log(rng, 1, 10000 // n))), "starts": _join(after(_log(rng, 1, 500000))), "heads": _log(rng, 1, 40),
                "dim": dim, "rope": rng.choice(sorted(ROPES)), "type": rng.choice(["bf16", "f16"]), "out": rng.choice(["bf16", "f16"])}
    kv = rng.choice([1, 2, 4, 8, 16])
    heads = kv * rng.choice([g for g in (1, 2, 3, 4, 8) if kv * g <= 32])
    block = rng.choice(BLOCKS)
    if op == "append":
        frame = rng.random() < 0.4
        if frame:
            n = _log(rng, 1, 128)
        lens = [1] * n if frame else some(_log(rng, 1, 12000 // n))
        return {"op": op, "lens": _join(lens), "starts": _join(after(_log(rng, 1, 2000))), "heads": heads, "kv_heads": kv, "dim": dim,
                "block": block, "rope": rng.choice(sorted(ROPES)), "type": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f16"]),
                "frame": frame}
    if op == "read":
        return {"op": op, "lens": _join(some(_log(rng, 1, 12000 // n))), "starts": _join(after(_log(rng, 1, 900))), "kv_heads": kv, "dim": dim,
                "block": block, "out": rng.choice(["bf16", "f16"])}
    frame = rng.random() < 0.5
    if frame:
        n = _log(rng, 1, 128)
        lens, starts = [1] * n, [v - 1 for v in some(_log(rng, 16, max(16, min(32000, 300_000_000 // (n * kv * dim * 2)))))]
    else:
        n = _log(rng, 1, 6)
        lens, starts = some(_log(rng, 1, 2200 // n)), after(_log(rng, 1, 8000 // n))
    return {"op": op, "lens": _join(lens), "starts": _join(starts), "heads": heads, "kv_heads": kv, "dim": dim, "block": block,
            "type": rng.choice(["bf16", "f16"]), "frame": frame}


def _ints(text):
    return [int(v) for v in text.split(",")]


def _cu(lens):
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    return cu


def _frequencies(name, dim):
    """The pairs' angles for one position, in 64 bits."""
    r = ROPES[name]
    turned = int(dim * r["part"])
    f = BASE ** (-torch.arange(0, turned, 2, dtype=torch.float64) / turned)
    if r["scaling"] == "linear":
        f = f / FACTOR
    elif r["scaling"] == "parts":
        keep = ((ORIGINAL * f / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / FACTOR
    return f


def _power_of_two(amax):
    """The least power of two s with amax <= 448 s (0 for 0)."""
    m, e = torch.frexp(amax)
    return torch.where(amax == 0, 0.0, torch.ldexp(torch.ones_like(amax), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)))


def _encode(v, scale):
    q = torch.where(scale == 0, 0.0, v / torch.where(scale == 0, 1.0, scale))
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _fill(g, kv, scales, block):
    """A history in which every slot was written before (16 sessions' heads at a time)."""
    t = kv.shape[-2]
    for k in range(2):
        for s in range(kv.shape[2]):
            rows = torch.randn(kv.shape[3:], generator=g, device="cuda") * (1.5 if k == 0 else 1.0)
            amax = rows.abs().amax(-1)
            if block > 1:
                pad = -t % block
                amax = torch.nn.functional.pad(amax, (0, pad)).reshape(amax.shape[0], -1, block).amax(-1)
            sc = _power_of_two(amax) if block > 1 else amax / 448.0
            scales[0, k, s] = sc
            kv[0, k, s] = _encode(rows, sc.repeat_interleave(block, -1)[:, :t, None]).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    c, st = case, {"case": case}
    st["lens"], st["starts"] = _ints(c["lens"]), _ints(c["starts"])
    st["cu"] = _cu(st["lens"])
    n, ns, d = st["cu"][-1], len(st["lens"]), c["dim"]
    # the sessions' slots, in another order than the prompts; a frame has row s for slot s
    st["slots"] = list(range(ns)) if c.get("frame") or ns % 5 == 0 else [(5 * i + 2) % ns for i in range(ns)]
    st["pos"] = torch.cat([torch.arange(v, device="cuda") + s0 for v, s0 in zip(st["lens"], st["starts"])])
    st["slot_of"] = torch.cat([torch.full((v,), s, device="cuda") for v, s in zip(st["lens"], st["slots"])])
    st["positions"] = torch.tensor(st["starts"], dtype=torch.int32, device="cuda")
    st["slots_d"], st["lens_d"] = torch.tensor(st["slots"], device="cuda"), torch.tensor(st["lens"], device="cuda")
    if "rope" in c:
        st["freq"] = _frequencies(c["rope"], d).cuda()
    if c["op"] == "rotate":
        st["x"] = (2.0 * randn(n, c["heads"], d)).to(TYPES[c["type"]])
        st["out"] = torch.zeros((n, c["heads"], d), dtype=TYPES[c["out"]], device="cuda")
    else:
        st["t_max"] = (max(a + b for a, b in zip(st["lens"], st["starts"])) + 3) // 4 * 4
        st["kv"] = torch.zeros((1, 2, ns, c["kv_heads"], st["t_max"], d), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros((1, 2, ns, c["kv_heads"], -(-st["t_max"] // c["block"])), device="cuda")
        _fill(g, st["kv"], st["scales"], c["block"])
        if c["op"] == "append":
            st["qkv"] = (2.0 * randn(n, (c["heads"] + 2 * c["kv_heads"]) * d)).to(TYPES[c["type"]])
            st["q"] = torch.zeros((n, c["heads"], d), dtype=TYPES[c["out"]], device="cuda")
        elif c["op"] == "read":
            for x in "kv":
                st["out_" + x] = torch.zeros((n, c["kv_heads"], d), dtype=TYPES[c["out"]], device="cuda")
        else:
            # after a norm and the rotary embedding: a few units wide, so that a softmax has a peak
            st["q"] = (1.5 * randn(n, c["heads"], d)).to(TYPES[c["type"]])
            st["out"] = torch.zeros_like(st["q"])
    if own:
        import frame_step_decode_gb300 as fsd
        if "rope" in c:
            r = ROPES[c["rope"]]
            st["plan"] = fsd.rope_plan(int(d * r["part"]), BASE, layout=r["layout"], scaling=r["scaling"], factor=FACTOR, original=ORIGINAL,
                                       fast=FAST, slow=SLOW, amplitude=AMPLITUDE[r["scaling"]])
        if c["op"] != "rotate":
            heads = c.get("heads", c["kv_heads"])
            st["wave"] = fsd.Wave(fsd.WaveConfig(1, 64, heads, d, 64, 1e-5, BASE), ns, st["t_max"])
    return st


def _outputs(st):
    """The buffers that a case's operator fills; 8-bit codes as the numbers that they stand for."""
    op = st["case"]["op"]
    if op == "append":
        return {"q": st["q"], "codes": st["kv"].view(torch.float8_e4m3fn), "scales": st["scales"]}
    return {"k": st["out_k"], "v": st["out_v"]} if op == "read" else st["out"]


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import frame_step_decode_gb300 as fsd
        if op == "rotate":
            fsd.rope_apply(st["plan"], st["x"], st["out"], cu_seqlens=st["cu"], starts=st["starts"])
        elif op == "append" and c["frame"]:
            st["wave"].history_append_frame(0, st["positions"], st["qkv"], st["kv"], st["scales"], c["kv_heads"], c["block"], rope=st["plan"], q=st["q"])
        elif op == "append":
            st["wave"].history_append(0, st["cu"], st["slots"], st["starts"], st["qkv"], st["kv"], st["scales"], c["kv_heads"], c["block"],
                                      rope=st["plan"], q=st["q"])
        elif op == "read":
            st["wave"].history_read(0, st["cu"], st["slots"], st["starts"], st["kv"], st["scales"], c["kv_heads"], c["block"], st["out_k"], st["out_v"])
        elif c["frame"]:
            st["wave"].history_attention_frame(0, st["positions"], st["q"], st["kv"], st["scales"], c["kv_heads"], c["block"], st["out"])
        else:
            st["wave"].history_attention(0, st["cu"], st["slots"], st["starts"], st["q"], st["kv"], st["scales"], c["kv_heads"], c["block"], st["out"])
        return _outputs(st)
    {"rotate": _rotate, "append": _append, "read": _read, "attend": _attend}[op](st)
    return _outputs(st)


def _turn(st, x):
    """The rotation of rows [tokens][heads][dim] in 32 bits; the angles in 64."""
    r = ROPES[st["case"]["rope"]]
    n = 2 * st["freq"].numel()
    ang = st["pos"].double()[:, None] * st["freq"]
    amp = AMPLITUDE[r["scaling"]]
    cos, sin = (amp * ang.cos()).float()[:, None], (amp * ang.sin()).float()[:, None]
    a, b = (x[..., :n // 2], x[..., n // 2:n]) if r["layout"] == "half" else (x[..., :n:2], x[..., 1:n:2])
    y, z = a * cos - b * sin, a * sin + b * cos
    both = torch.cat([y, z], -1) if r["layout"] == "half" else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([both, x[..., n:]], -1)


def _rotate(st):
    st["out"].copy_(_turn(st, st["x"].float()))


def _append(st):
    c = st["case"]
    h, hkv, d, b = c["heads"], c["kv_heads"], c["dim"], c["block"]
    x = st["qkv"].float().reshape(-1, h + 2 * hkv, d)
    turned = _turn(st, x[:, :h + hkv])
    st["q"].copy_(turned[:, :h])
    rows = torch.stack([turned[:, h:], x[:, h + hkv:]], 1)  # [tokens][K|V][heads][d]
    amax = rows.abs().amax(-1)
    pos, slot = st["pos"], st["slot_of"]
    scales = st["scales"][0].permute(1, 3, 0, 2)            # [slot][block][K|V][heads]
    codes = st["kv"][0].permute(1, 3, 0, 2, 4)              # [slot][t][K|V][heads][d]
    if b == 1:
        scale = amax / 448.0
        scales[slot, pos] = scale
    else:
        nb = scales.shape[1]
        most = torch.zeros((scales.shape[0] * nb,) + amax.shape[1:], device="cuda").index_reduce_(0, slot * nb + pos // b, amax, "amax")
        # blocks that go on: the one that holds a sequence's first token, where that is not the block's first
        first = st["positions"].long()
        at, goes_on = first // b, first % b > 0
        old = scales[st["slots_d"], at].clone()
        fresh = _power_of_two(most).reshape(scales.shape)
        fresh[st["slots_d"], at] = torch.maximum(fresh[st["slots_d"], at], torch.where(goes_on[:, None, None], old, 0.0))
        scales[slot, pos // b] = fresh[slot, pos // b]
        # what those blocks held before, under the new scale
        new = fresh[st["slots_d"], at]
        t = at[:, None] * b + torch.arange(b, device="cuda")
        held = t < first[:, None]
        who = st["slots_d"][:, None].expand_as(t)[held]
        ratio = torch.where(new == 0, 0.0, old / torch.where(new == 0, 1.0, new))[:, None].expand(-1, b, -1, -1)[held]
        before = codes[who, t[held]].view(torch.float8_e4m3fn).float()
        codes[who, t[held]] = (before * ratio[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = scales[slot, pos // b]
    codes[slot, pos] = _encode(rows, scale[..., None]).view(torch.uint8)


def _read(st):
    b = st["case"]["block"]
    codes = st["kv"][0].permute(1, 3, 0, 2, 4)[st["slot_of"], st["pos"]].view(torch.float8_e4m3fn).float()
    x = codes * st["scales"][0].permute(1, 3, 0, 2)[st["slot_of"], st["pos"] // b][..., None]
    st["out_k"].copy_(x[:, 0])
    st["out_v"].copy_(x[:, 1])


def _attend(st):
    c = st["case"]
    hkv, d, b = c["kv_heads"], c["dim"], c["block"]
    group = c["heads"] // hkv
    m, t = max(st["lens"]), max(p + n for p, n in zip(st["starts"], st["lens"]))
    first = st["lens_d"].cumsum(0) - st["lens_d"]
    at = torch.arange(m, device="cuda")
    rows, there = first[:, None] + at, at < st["lens_d"][:, None]
    q = st["q"][rows.clamp(max=st["q"].shape[0] - 1)].float()          # [b][m][heads][d]
    ns = q.shape[0]
    q = q.reshape(ns, m, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(ns, hkv, group * m, d)
    scale = st["scales"][0][:, st["slots_d"]].repeat_interleave(b, -1)[..., :t, None]
    k, v = st["kv"][0][:, st["slots_d"], :, :t].view(torch.float8_e4m3fn).float() * scale
    s = (q @ k.transpose(-1, -2)).reshape(ns, hkv, group, m, t) / math.sqrt(d)
    seen = st["positions"].long()[:, None] + at                         # [b][m]: the last position of a row
    s.masked_fill_((torch.arange(t, device="cuda") > seen[..., None])[:, None, None], -math.inf)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    s /= s.sum(-1, keepdim=True)
    o = (s.reshape(ns, hkv, group * m, t) @ v).reshape(ns, hkv, group, m, d).permute(0, 3, 1, 2, 4).reshape(ns, m, -1, d)
    st["out"][rows[there]] = o[there].to(st["out"].dtype)


def work(case):
    c = case
    lens, starts, d = _ints(c["lens"]), _ints(c["starts"]), c["dim"]
    n = sum(lens)
    size = lambda t: 4 if t == "f32" else 2  # noqa: E731
    if c["op"] == "rotate":
        return {"bytes": n * c["heads"] * d * (size(c["type"]) + size(c["out"])), "flops": n * c["heads"] * d * 3}
    hkv, b = c["kv_heads"], c["block"]
    blocks = lambda lo, hi: -(-hi // b) - lo // b  # noqa: E731
    held = sum(2 * hkv * (v * d + 4 * blocks(s, s + v)) for s, v in zip(starts, lens))  # codes and scales of the call's tokens
    if c["op"] == "append":
        return {"bytes": n * d * ((c["heads"] + 2 * hkv) * size(c["type"]) + c["heads"] * size(c["out"])) + held,
                "flops": n * d * (c["heads"] * 3 + hkv * 9)}
    if c["op"] == "read":
        return {"bytes": held + 2 * n * hkv * d * size(c["out"]), "flops": 2 * n * hkv * d}
    pairs = sum(v * s + v * (v + 1) // 2 for s, v in zip(starts, lens))
    return {"bytes": sum(2 * hkv * ((s + v) * d + 4 * blocks(0, s + v)) for s, v in zip(starts, lens)) + 2 * n * c["heads"] * d * size(c["type"]),
            "flops": 4 * d * c["heads"] * pairs}


# ---- the definitions in 64 bits, sequence by sequence


def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, st)


def _exact_turn(c, st, x):
    """x [tokens][heads][dim], numpy, in place: a rotation of each pair as a complex number."""
    r = ROPES[c["rope"]]
    n = int(c["dim"] * r["part"])
    f = np.array([BASE ** (-2.0 * i / n) for i in range(n // 2)])
    for i in range(n // 2):
        if r["scaling"] == "linear":
            f[i] /= FACTOR
        elif r["scaling"] == "parts":
            turns = ORIGINAL * f[i] / (2 * np.pi)
            keep = min(1.0, max(0.0, (turns - SLOW) / (FAST - SLOW)))
            f[i] *= keep + (1 - keep) / FACTOR
    pos = np.concatenate([s + np.arange(v) for s, v in zip(st["starts"], st["lens"])])
    z = AMPLITUDE[r["scaling"]] * np.exp(1j * pos[:, None] * f)[:, None]
    lo, hi = (slice(0, n // 2), slice(n // 2, n)) if r["layout"] == "half" else (slice(0, n, 2), slice(1, n, 2))
    w = (x[..., lo] + 1j * x[..., hi]) * z
    x[..., lo], x[..., hi] = w.real, w.imag
    return x


def _exact_rotate(c, st):
    return _exact_turn(c, st, st["x"].double().cpu().numpy())


def _exact_append(c, st):
    h, hkv, d, b = c["heads"], c["kv_heads"], c["dim"], c["block"]
    x = st["qkv"].double().cpu().numpy().reshape(-1, h + 2 * hkv, d)
    x[:, :h + hkv] = _exact_turn(c, st, x[:, :h + hkv].copy())
    scales = st["scales"].double().cpu().numpy()
    for i, slot in enumerate(st["slots"]):
        rows = x[st["cu"][i]:st["cu"][i + 1], h:].reshape(-1, 2, hkv, d)
        pos = st["starts"][i] + np.arange(len(rows))
        amax = np.abs(rows).max(-1)
        for blk in np.unique(pos // b):
            a = amax[pos // b == blk].max(0)
            if b == 1:
                scales[0, :, slot, :, blk] = a / 448
            else:
                s = 2.0 ** np.ceil(np.log2(a) - np.log2(448.0))
                s = np.where(s / 2 * 448 >= a, s / 2, np.where(s * 448 < a, s * 2, s))  # log2's rounding
                goes_on = blk == st["starts"][i] // b and st["starts"][i] % b
                scales[0, :, slot, :, blk] = np.maximum(s, scales[0, :, slot, :, blk]) if goes_on else s
    return {"q": x[:, :h], "codes": None, "scales": scales}


def _history(c, st, i, kind):
    """Session i's keys (0) or values (1), [heads][t][d]."""
    slot, t = st["slots"][i], st["starts"][i] + st["lens"][i]
    per = torch.arange(t, device="cuda") // c["block"]
    return st["kv"][0, kind, slot, :, :t].view(torch.float8_e4m3fn).double() * st["scales"][0, kind, slot][:, per, None].double()


def _exact_read(c, st):
    got = {}
    for kind, name in enumerate("kv"):
        got[name] = torch.cat([_history(c, st, i, kind)[:, s0:].transpose(0, 1) for i, s0 in enumerate(st["starts"])])
    return got


def _exact_attend(c, st):
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    group = c["heads"] // c["kv_heads"]
    for i, (a, e) in enumerate(zip(st["cu"], st["cu"][1:])):
        k, v = _history(c, st, i, 0), _history(c, st, i, 1)
        later = torch.full((e - a, k.shape[1]), -math.inf, dtype=torch.float64, device="cuda").triu(st["starts"][i] + 1)
        for h in range(c["heads"]):
            s = torch.mm(st["q"][a:e, h].double(), k[h // group].t()) * c["dim"] ** -0.5 + later
            out[a:e, h] = torch.mm(torch.softmax(s, dim=1), v[h // group])
    return out
