"""Python binding of libwave.so (include/wave.h): argument marshalling only.

Every step of the frame runs in the library's CUDA kernels; PyTorch is used
only to own device memory and streams.  There is no fallback: if the library
is not built, importing the binding's entry points raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libwave.so")

WAVE_OK, WAVE_EINVAL, WAVE_ECUDA, WAVE_ELAUNCH = 0, -1, -2, -3
WAVE_ETIMEOUT, WAVE_EPOS, WAVE_EDEVICE, WAVE_ENOMEM = -4, -5, -6, -7
WAVE_F32, WAVE_BF16, WAVE_F16 = 0, 1, 2
WAVE_MAX_SEQS = 128
_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "parts": 2}


class WaveConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("rope_base", ctypes.c_float)]

    @classmethod
    def of(cls, w) -> "WaveConfig":
        """From any object with the decoder-shape attributes."""
        return cls(w.n_layers, w.d_model, w.n_heads, w.head_dim, w.ffn, w.rms_eps, w.rope_base)


class WaveHybridConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("d_model", ctypes.c_int), ("attn_every", ctypes.c_int),
                ("n_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ssm_heads", ctypes.c_int),
                ("ssm_head_dim", ctypes.c_int), ("ssm_state", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("rope_base", ctypes.c_float)]

    @classmethod
    def of(cls, w) -> "WaveHybridConfig":
        """From any object with the hybrid-shape attributes."""
        return cls(w.n_layers, w.d_model, w.attn_every, w.n_heads, w.head_dim, w.ssm_heads, w.ssm_head_dim,
                   w.ssm_state, w.rms_eps, w.rope_base)


class WaveRopeConfig(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int), ("dims", ctypes.c_int), ("base", ctypes.c_float), ("scaling", ctypes.c_int),
                ("factor", ctypes.c_float), ("original", ctypes.c_float), ("fast", ctypes.c_float), ("slow", ctypes.c_float),
                ("amplitude", ctypes.c_float)]


class WaveRope(ctypes.Structure):
    """A plan of rotary positions (rope_plan)."""
    _fields_ = [("layout", ctypes.c_int32), ("dims", ctypes.c_int32), ("amplitude", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turns", ctypes.c_uint64 * 64)]


class WaveError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


_lib = None
EXPORTS = ("wave_create", "wave_destroy", "wave_weights_bytes", "wave_weight_offset", "wave_packed_weights_bytes",
           "wave_pack_weights", "wave_hybrid_packed_weights_bytes", "wave_hybrid_pack_weights",
           "wave_step", "wave_beat", "wave_depth",
           "wave_status", "wave_strerror", "wave_kv_quantize", "wave_fp8_encode", "wave_step_static",
           "wave_set_timeout_ns", "wave_debug_skip_barrier", "wave_debug_skip_signal", "wave_debug_dump_kv", "wave_debug_dump_acts",
           "wave_debug_act_record_floats", "wave_debug_phase_times", "wave_debug_arrival_times",
           "wave_grid_size", "wave_barriers_per_step", "wave_phases_per_step", "wave_hybrid_create", "wave_hybrid_step",
           "wave_hybrid_weights_bytes", "wave_hybrid_layer_offset",
           "wave_prompt_append", "wave_prompt_attention", "wave_hybrid_prompt_state", "wave_sessions_copy",
           "wave_rope_plan", "wave_rope_apply", "wave_rope_apply_at", "wave_history_append", "wave_history_append_frame",
           "wave_history_read", "wave_history_attention", "wave_history_attention_frame")


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run frame_step_decode_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        cfgp = ctypes.POINTER(WaveConfig)
        L.wave_create.argtypes = [cfgp, i32, i32, ctypes.POINTER(vp)]
        L.wave_create.restype = i32
        L.wave_destroy.argtypes = [vp]
        L.wave_destroy.restype = None
        L.wave_weights_bytes.argtypes = [cfgp]
        L.wave_weights_bytes.restype = sz
        L.wave_weight_offset.argtypes = [cfgp, i32, i32]
        L.wave_weight_offset.restype = sz
        L.wave_packed_weights_bytes.argtypes = [cfgp]
        L.wave_packed_weights_bytes.restype = sz
        L.wave_pack_weights.argtypes = [cfgp, vp, vp, vp]
        L.wave_pack_weights.restype = i32
        L.wave_hybrid_packed_weights_bytes.argtypes = [ctypes.POINTER(WaveHybridConfig)]
        L.wave_hybrid_packed_weights_bytes.restype = sz
        L.wave_hybrid_pack_weights.argtypes = [ctypes.POINTER(WaveHybridConfig), vp, vp, vp]
        L.wave_hybrid_pack_weights.restype = i32
        L.wave_step.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp]
        L.wave_step.restype = i32
        L.wave_beat.argtypes = [vp, i32, i32, vp, vp, vp, vp, i32, vp, vp, vp]
        L.wave_beat.restype = i32
        L.wave_depth.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.wave_depth.restype = i32
        L.wave_hybrid_create.argtypes = [ctypes.POINTER(WaveHybridConfig), i32, i32, ctypes.POINTER(vp)]
        L.wave_hybrid_create.restype = i32
        L.wave_hybrid_step.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.wave_hybrid_step.restype = i32
        L.wave_hybrid_weights_bytes.argtypes = [ctypes.POINTER(WaveHybridConfig)]
        L.wave_hybrid_weights_bytes.restype = ctypes.c_size_t
        L.wave_hybrid_layer_offset.argtypes = [ctypes.POINTER(WaveHybridConfig), i32]
        L.wave_hybrid_layer_offset.restype = ctypes.c_size_t
        L.wave_status.argtypes = [vp]
        L.wave_status.restype = i32
        L.wave_strerror.argtypes = [i32]
        L.wave_strerror.restype = ctypes.c_char_p
        L.wave_kv_quantize.argtypes = [vp, i64, i32, vp, vp, vp]
        L.wave_kv_quantize.restype = i32
        L.wave_fp8_encode.argtypes = [vp, i64, vp, vp]
        L.wave_fp8_encode.restype = i32
        L.wave_step_static.argtypes = [cfgp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
        L.wave_step_static.restype = i32
        L.wave_set_timeout_ns.argtypes = [vp, ctypes.c_longlong]
        L.wave_set_timeout_ns.restype = i32
        L.wave_debug_skip_barrier.argtypes = [vp, i32, i32]
        L.wave_debug_skip_barrier.restype = i32
        L.wave_debug_skip_signal.argtypes = [vp, i32, i32]
        L.wave_debug_skip_signal.restype = i32
        L.wave_debug_dump_kv.argtypes = [vp, vp]
        L.wave_debug_dump_kv.restype = i32
        L.wave_debug_dump_acts.argtypes = [vp, vp, i32]
        L.wave_debug_dump_acts.restype = i32
        L.wave_debug_act_record_floats.argtypes = [vp]
        L.wave_debug_act_record_floats.restype = ctypes.c_longlong
        L.wave_debug_phase_times.argtypes = [vp, vp]
        L.wave_debug_phase_times.restype = i32
        L.wave_debug_arrival_times.argtypes = [vp, vp]
        L.wave_debug_arrival_times.restype = i32
        L.wave_grid_size.argtypes = [vp]
        L.wave_grid_size.restype = i32
        L.wave_barriers_per_step.argtypes = [vp]
        L.wave_barriers_per_step.restype = i32
        L.wave_phases_per_step.argtypes = [vp]
        L.wave_phases_per_step.restype = i32
        # the host arrays of int32 come as bytes
        L.wave_prompt_append.argtypes = [vp, i32, i32, vp, vp, vp, vp, i32, i64, vp, vp, vp, vp, vp, i32, vp]
        L.wave_prompt_append.restype = i32
        L.wave_prompt_attention.argtypes = [vp, i32, vp, i32, i32, vp, i64, vp, i64, vp, i64, ctypes.c_float, vp, i64, vp]
        L.wave_prompt_attention.restype = i32
        L.wave_hybrid_prompt_state.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, i64, vp, vp, vp, i64, vp]
        L.wave_hybrid_prompt_state.restype = i32
        L.wave_sessions_copy.argtypes = [vp, i32, vp, vp, i32, vp, vp, vp, vp, vp]
        L.wave_sessions_copy.restype = i32
        L.wave_rope_plan.argtypes = [ctypes.POINTER(WaveRopeConfig), vp]
        L.wave_rope_plan.restype = i32
        L.wave_rope_apply.argtypes = [vp, i32, vp, vp, i32, i32, vp, i32, i64, vp, i32, i64, vp]
        L.wave_rope_apply.restype = i32
        L.wave_rope_apply_at.argtypes = [vp, i64, vp, i32, i32, vp, i32, i64, vp, i32, i64, vp]
        L.wave_rope_apply_at.restype = i32
        L.wave_history_append.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, i32, i64, vp, vp, i32, i32, vp, i32, vp]
        L.wave_history_append.restype = i32
        L.wave_history_append_frame.argtypes = [vp, i32, i32, vp, vp, vp, i32, i64, vp, vp, i32, i32, vp, i32, vp]
        L.wave_history_append_frame.restype = i32
        L.wave_history_read.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, i32, i32, vp, vp, i32, vp]
        L.wave_history_read.restype = i32
        L.wave_history_attention.argtypes = [vp, i32, i32, vp, vp, vp, i32, vp, i64, vp, vp, i32, i32, ctypes.c_float, vp, i64, vp]
        L.wave_history_attention.restype = i32
        L.wave_history_attention_frame.argtypes = [vp, i32, i32, vp, i32, vp, i64, vp, vp, i32, i32, ctypes.c_float, vp, i64, vp]
        L.wave_history_attention_frame.restype = i32
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().wave_strerror(code).decode()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_PACKS: dict = {}  # packers of n int32 by n


def _ints(values):
    """A host array of int32 (any sequence of integers that fit) as bytes, and its length."""
    n = len(values)
    p = _PACKS.get(n)
    if p is None:
        p = _PACKS[n] = struct.Struct(f"{n}i")
    try:
        return p.pack(*values), n
    except (struct.error, TypeError) as e:
        raise ValueError("a sequence of 32-bit integers is wanted") from e


def _types() -> dict:
    import torch
    return {torch.float32: WAVE_F32, torch.bfloat16: WAVE_BF16, torch.float16: WAVE_F16}


_TYPES: dict = {}


def _type_of(t) -> int:
    if not _TYPES:
        _TYPES.update(_types())
    return _TYPES.get(t.dtype, -1)


def _rows(t, what: str) -> int:
    """The row stride in elements of a packed tensor [rows][H][D] or
    [rows][values]; what lies inside a row has to be contiguous."""
    shape = t.shape
    n = len(shape)
    if n == 3 and t.is_contiguous():
        return shape[1] * shape[2]
    stride = t.stride()
    width = shape[-1]
    fits = 2 <= n <= 3 and (stride[-1] == 1 or width == 1)
    if n == 3:
        fits = fits and (stride[1] == width or shape[1] == 1)
        width *= shape[1]
    if not fits:
        raise ValueError(f"{what}: a packed tensor of rows, contiguous inside a row, is wanted")
    return stride[0] if shape[0] > 1 else width


def _is_rows(t, rows: int, H: int, D: int) -> bool:
    """Whether t is [rows or more][H][D]."""
    shape = t.shape
    return len(shape) == 3 and shape[2] == D and shape[1] == H and shape[0] >= rows


_DTYPES: dict = {}  # float32 and int32 by name


def _held(t, kind, count: int, device: int, what: str) -> None:
    """Refuse a buffer of the handle's layout (history, state, positions,
    weights) that a call would read or write beyond its end, as another type
    (kind: a name in _DTYPES, or the bytes of a value) or on another device.
    An address (int) or None is the caller's."""
    if t is None or isinstance(t, int):
        return
    fits = t.element_size() == kind if isinstance(kind, int) else t.dtype is _DTYPES[kind]
    if not fits or t.numel() < count or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: {count} contiguous values ({kind if isinstance(kind, str) else f'{kind} bytes each'}) on device {device} "
                         f"are wanted, not {t.numel()} of {t.dtype} on device {t.get_device()}")


def _here(device: int, what: str, *tensors) -> None:
    """Refuse tensors that are not on the handle's device."""
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{what}: a tensor on device {t.get_device()}, the handle's is {device}")


_CURRENT: list = []  # torch's current device, and the current stream's handle on it


def _stream(stream) -> int:
    if stream is None:  # without a Stream object around the handle (4 of a call's 12 us)
        if not _CURRENT:
            import torch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # not a public name
            _CURRENT.extend((torch.cuda.current_device, raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)))
        return _CURRENT[1](_CURRENT[0]())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def weights_bytes(cfg: WaveConfig) -> int:
    return lib().wave_weights_bytes(ctypes.byref(cfg))


def weight_offset(cfg: WaveConfig, layer: int, which: int) -> int:
    return lib().wave_weight_offset(ctypes.byref(cfg), layer, which)


def packed_weights_bytes(cfg: WaveConfig) -> int:
    return lib().wave_packed_weights_bytes(ctypes.byref(cfg))


def pack_weights(cfg: WaveConfig, src, dst=None, stream=None):
    """wave_pack_weights: the packed blob the step reads, from the row-major
    blob src (a device tensor).  Returns dst (a new bf16 device tensor when
    not given)."""
    import torch
    if dst is None:
        dst = torch.empty(packed_weights_bytes(cfg) // 2, dtype=torch.bfloat16, device=src.device)
    rc = lib().wave_pack_weights(ctypes.byref(cfg), _ptr(src), _ptr(dst), _stream(stream))
    if rc != WAVE_OK:
        raise WaveError(rc, "wave_pack_weights")
    return dst


def hybrid_packed_weights_bytes(cfg: "WaveHybridConfig") -> int:
    return lib().wave_hybrid_packed_weights_bytes(ctypes.byref(cfg))


def hybrid_pack_weights(cfg: "WaveHybridConfig", src, dst=None, stream=None):
    """wave_hybrid_pack_weights (as pack_weights, for the hybrid blob)."""
    import torch
    if dst is None:
        dst = torch.empty(hybrid_packed_weights_bytes(cfg) // 2, dtype=torch.bfloat16, device=src.device)
    rc = lib().wave_hybrid_pack_weights(ctypes.byref(cfg), _ptr(src), _ptr(dst), _stream(stream))
    if rc != WAVE_OK:
        raise WaveError(rc, "wave_hybrid_pack_weights")
    return dst


class Wave:
    """A step context: wave_create / wave_step / wave_status / wave_destroy."""

    def __init__(self, cfg: WaveConfig, S_max: int, T_max: int):
        self.cfg = cfg
        self.S_max, self.T_max = S_max, T_max
        h = ctypes.c_void_p()
        rc = lib().wave_create(ctypes.byref(cfg), S_max, T_max, ctypes.byref(h))
        if rc != WAVE_OK:
            raise WaveError(rc, "wave_create")
        self.h = h
        self._sizes()

    def _sizes(self) -> None:
        """What the calls on prompts and sessions compare buffers with: the
        handle's device, and how many values history, scales, state and packed
        weights have."""
        import torch
        _DTYPES.update(float32=torch.float32, int32=torch.int32)
        c, hybrid = self.cfg, isinstance(self.cfg, WaveHybridConfig)
        layers = c.n_layers // c.attn_every if hybrid else c.n_layers
        self._n_scales = layers * 2 * self.S_max * c.n_heads * self.T_max
        self._n_codes = self._n_scales * c.head_dim
        self._n_state = (c.n_layers - layers) * self.S_max * c.ssm_heads * c.ssm_head_dim * c.ssm_state if hybrid else 0
        self._n_weights = hybrid_packed_weights_bytes(c) // 2 if hybrid else 0
        self.device = torch.cuda.current_device() if torch.cuda.is_available() else -1

    def step(self, S, weights, kv, kv_scales, positions, x, y, stream=None, check=True) -> int:
        rc = lib().wave_step(self.h, S, _ptr(weights), _ptr(kv), _ptr(kv_scales), _ptr(positions),
                             _ptr(x), _ptr(y), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, "wave_step")
        return rc

    def depth(self, S, steps, weights, w_proj, kv, kv_scales, x0, xs, y, stream=None, check=True) -> int:
        """The inner depth loop: `steps` dependent steps, x_k = bf16(W_p y_{k-1})
        (xs [steps][S][d] scratch, y [steps][S][d])."""
        rc = lib().wave_depth(self.h, S, steps, _ptr(weights), _ptr(w_proj), _ptr(kv), _ptr(kv_scales),
                              _ptr(x0), _ptr(xs), _ptr(y), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, "wave_depth")
        return rc

    def beat(self, S, frames, weights, kv, kv_scales, positions, x, y, advance=True, stream=None,
             check=True) -> int:
        """`frames` frames in one launch (x, y [frames][S][d]); frame f at
        positions + f; positions advanced by `frames` on the device when
        `advance` is set."""
        rc = lib().wave_beat(self.h, S, frames, _ptr(weights), _ptr(kv), _ptr(kv_scales), _ptr(positions),
                             int(bool(advance)), _ptr(x), _ptr(y), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, "wave_beat")
        return rc

    def prompt_append(self, layer, cu_seqlens, slots, starts, qkv, kv, kv_scales, q=None, k=None, v=None,
                      stream=None, check=True) -> int:
        """wave_prompt_append: RoPE, FP8 quantisation and append of packed
        prompts to layer `layer`'s history.  cu_seqlens, slots and starts are
        host integers; qkv is [rows][3*H*D] (fp32 or bf16, rows may be
        strided); q, k, v (each optional) are contiguous [rows][H][D] outputs
        of one 16-bit type: the rotated q and the k, v that the history now
        holds."""
        (cu, n_cu), (sl, n_sl), (s0, n_s0) = _ints(cu_seqlens), _ints(slots), _ints(starts)
        if n_cu < 2 or n_sl != n_cu - 1 or n_s0 != n_sl:
            raise ValueError("wave_prompt_append: one slot and one start for each sequence")
        H, D = self.cfg.n_heads, self.cfg.head_dim
        rows, out_type = int(cu_seqlens[n_sl]), -1
        for t in (q, k, v):
            if t is None:
                continue
            kind = _type_of(t)
            if not _is_rows(t, rows, H, D) or out_type not in (-1, kind) or not t.is_contiguous():
                raise ValueError("wave_prompt_append: q, k and v are contiguous [rows][H][D], of one type")
            out_type = kind
        shape = qkv.shape
        if len(shape) != 2 or shape[1] != 3 * H * D or shape[0] < rows:
            raise ValueError("wave_prompt_append: qkv is [rows][3*H*D], with the rows that cu_seqlens names")
        if self.h:
            _here(self.device, "wave_prompt_append", qkv, q, k, v)
            _held(kv, 1, self._n_codes, self.device, "wave_prompt_append: kv")
            _held(kv_scales, "float32", self._n_scales, self.device, "wave_prompt_append: kv_scales")
        rc = lib().wave_prompt_append(self.h, layer, n_sl, cu, sl, s0, _ptr(qkv), _type_of(qkv), _rows(qkv, "qkv"),
                                      _ptr(kv), _ptr(kv_scales), _ptr(q), _ptr(k), _ptr(v),
                                      WAVE_BF16 if out_type < 0 else out_type, _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, "wave_prompt_append")
        return rc

    def prompt_attention(self, cu_seqlens, q, k, v, out, scale=None, stream=None, check=True) -> int:
        """wave_prompt_attention: causal attention over packed prompts.  q and
        out are [rows][n_heads][D], k and v [rows][n_kv_heads][D], all bf16 or
        all fp16, rows may be strided; scale defaults to 1/sqrt(D)."""
        cu, n_cu = _ints(cu_seqlens)
        H, D = self.cfg.n_heads, self.cfg.head_dim
        what, dtype = "wave_prompt_attention", q.dtype
        if n_cu < 2:
            raise ValueError(f"{what}: cu_seqlens has one entry more than there are sequences")
        rows, Hkv = int(cu_seqlens[n_cu - 1]), k.shape[1] if len(k.shape) == 3 else 0
        if k.dtype != dtype or v.dtype != dtype or out.dtype != dtype or not _is_rows(q, rows, H, D) \
                or not _is_rows(out, rows, H, D) or not _is_rows(k, rows, Hkv, D) or not _is_rows(v, rows, Hkv, D):
            raise ValueError(f"{what}: q, out [rows][n_heads][D] and k, v [rows][n_kv_heads][D] of one type, with the rows "
                             "that cu_seqlens names")
        if self.h:
            _here(self.device, what, q, k, v, out)
        rc = lib().wave_prompt_attention(self.h, n_cu - 1, cu, Hkv, _type_of(q), _ptr(q), _rows(q, what), _ptr(k),
                                         _rows(k, what), _ptr(v), _rows(v, what), D ** -0.5 if scale is None else scale,
                                         _ptr(out), _rows(out, what), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, what)
        return rc

    def sessions_copy(self, src, dst, kv, kv_scales, positions, state=None, move=False, stream=None,
                      check=True) -> int:
        """wave_sessions_copy: sessions src (host integers) copied to slots dst:
        history, position and, for a hybrid handle, the recurrent state.  With
        move the sources are freed (position -1)."""
        (s, n), (d, n_d) = _ints(src), _ints(dst)
        if n != n_d:
            raise ValueError("wave_sessions_copy: one destination for each source")
        if self.h:
            _held(kv, 1, self._n_codes, self.device, "wave_sessions_copy: kv")
            _held(kv_scales, "float32", self._n_scales, self.device, "wave_sessions_copy: kv_scales")
            _held(state, "float32", self._n_state, self.device, "wave_sessions_copy: state")
            _held(positions, "int32", self.S_max, self.device, "wave_sessions_copy: positions")
        rc = lib().wave_sessions_copy(self.h, n, s, d, int(bool(move)), _ptr(kv), _ptr(kv_scales), _ptr(state),
                                      _ptr(positions), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, "wave_sessions_copy")
        return rc

    def _history(self, what, kv, kv_scales, n_kv_heads, block) -> None:
        """Refuse buffers that are no history of n_kv_heads heads with a scale for each `block` tokens."""
        c = self.cfg
        if n_kv_heads < 1 or c.n_heads % n_kv_heads or block not in (1, 16, 32, 64, 128):
            raise ValueError(f"{what}: n_kv_heads divides n_heads, and a block is 1, 16, 32, 64 or 128 tokens")
        if self.h:
            rows = self._n_scales // (c.n_heads * self.T_max) * n_kv_heads
            _held(kv, 1, rows * self.T_max * c.head_dim, self.device, f"{what}: kv")
            _held(kv_scales, "float32", rows * -(-self.T_max // block), self.device, f"{what}: kv_scales")

    def _append_rows(self, what, rows, qkv, n_kv_heads, q) -> None:
        """Refuse a qkv or a q that does not have the call's rows."""
        H, D = self.cfg.n_heads, self.cfg.head_dim
        if len(qkv.shape) != 2 or qkv.shape[1] != (H + 2 * n_kv_heads) * D or qkv.shape[0] < rows:
            raise ValueError(f"{what}: qkv is [rows][(n_heads + 2 n_kv_heads) * D], with the rows that the call names")
        if q is not None and (not _is_rows(q, rows, H, D) or not q.is_contiguous()):
            raise ValueError(f"{what}: q is contiguous [rows][n_heads][D]")
        if self.h:
            _here(self.device, what, qkv, q)

    def history_append(self, layer, cu_seqlens, slots, starts, qkv, kv, kv_scales, n_kv_heads, block, rope=None, q=None,
                       stream=None, check=True) -> int:
        """wave_history_append: rotary positions (rope: a rope_plan or None),
        8-bit quantisation and append of packed prompts to layer `layer`'s
        history of n_kv_heads heads with one scale for each `block` tokens.
        qkv is [rows][(n_heads + 2 n_kv_heads) * D] (fp32 or bf16, rows may be
        strided); q, optional, the rotated q, contiguous [rows][n_heads][D]."""
        what = "wave_history_append"
        (cu, n_cu), (sl, n_sl), (s0, n_s0) = _ints(cu_seqlens), _ints(slots), _ints(starts)
        if n_cu < 2 or n_sl != n_cu - 1 or n_s0 != n_sl:
            raise ValueError(f"{what}: one slot and one start for each sequence")
        self._append_rows(what, int(cu_seqlens[n_sl]), qkv, n_kv_heads, q)
        self._history(what, kv, kv_scales, n_kv_heads, block)
        rc = lib().wave_history_append(self.h, layer, n_sl, cu, sl, s0, _plan(rope), _ptr(qkv), _type_of(qkv), _rows(qkv, what),
                                       _ptr(kv), _ptr(kv_scales), n_kv_heads, block, _ptr(q),
                                       WAVE_BF16 if q is None else _type_of(q), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, what)
        return rc

    def history_append_frame(self, layer, positions, qkv, kv, kv_scales, n_kv_heads, block, rope=None, q=None, stream=None,
                             check=True) -> int:
        """wave_history_append_frame: the same for one token of each session,
        row s in slot s at positions[s] (int32 on the device; negative: an
        empty slot)."""
        what, S = "wave_history_append_frame", positions.numel()
        self._append_rows(what, S, qkv, n_kv_heads, q)
        self._history(what, kv, kv_scales, n_kv_heads, block)
        if self.h:
            _held(positions, "int32", S, self.device, f"{what}: positions")
        rc = lib().wave_history_append_frame(self.h, layer, S, _ptr(positions), _plan(rope), _ptr(qkv), _type_of(qkv),
                                             _rows(qkv, what), _ptr(kv), _ptr(kv_scales), n_kv_heads, block, _ptr(q),
                                             WAVE_BF16 if q is None else _type_of(q), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, what)
        return rc

    def history_read(self, layer, cu_seqlens, slots, starts, kv, kv_scales, n_kv_heads, block, k=None, v=None, stream=None,
                     check=True) -> int:
        """wave_history_read: positions starts[i] .. of session slots[i] back
        as contiguous k and v [rows][n_kv_heads][D] (either optional, of one
        type: fp32, bf16 or fp16)."""
        what = "wave_history_read"
        (cu, n_cu), (sl, n_sl), (s0, n_s0) = _ints(cu_seqlens), _ints(slots), _ints(starts)
        if n_cu < 2 or n_sl != n_cu - 1 or n_s0 != n_sl:
            raise ValueError(f"{what}: one slot and one start for each sequence")
        rows, out_type = int(cu_seqlens[n_sl]), -1
        for t in (k, v):
            if t is None:
                continue
            kind = _type_of(t)
            if not _is_rows(t, rows, n_kv_heads, self.cfg.head_dim) or out_type not in (-1, kind) or not t.is_contiguous():
                raise ValueError(f"{what}: k and v are contiguous [rows][n_kv_heads][D], of one type")
            out_type = kind
        self._history(what, kv, kv_scales, n_kv_heads, block)
        if self.h:
            _here(self.device, what, k, v)
        rc = lib().wave_history_read(self.h, layer, n_sl, cu, sl, s0, _ptr(kv), _ptr(kv_scales), n_kv_heads, block, _ptr(k), _ptr(v),
                                     out_type, _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, what)
        return rc

    def _attention_rows(self, what, rows, q, out) -> None:
        """Refuse q and out that do not have the call's rows."""
        H, D = self.cfg.n_heads, self.cfg.head_dim
        if out.dtype != q.dtype or not _is_rows(q, rows, H, D) or not _is_rows(out, rows, H, D):
            raise ValueError(f"{what}: q and out are [rows][n_heads][D] of one type, with the rows that the call names")
        if self.h:
            _here(self.device, what, q, out)

    def history_attention(self, layer, cu_seqlens, slots, starts, q, kv, kv_scales, n_kv_heads, block, out, scale=None,
                          stream=None, check=True) -> int:
        """wave_history_attention: attention of packed prompts that go on from
        their sessions' history (append them first).  q and out are
        [rows][n_heads][D], bf16 or fp16, rows may be strided; scale defaults
        to 1/sqrt(D)."""
        what = "wave_history_attention"
        (cu, n_cu), (sl, n_sl), (s0, n_s0) = _ints(cu_seqlens), _ints(slots), _ints(starts)
        if n_cu < 2 or n_sl != n_cu - 1 or n_s0 != n_sl:
            raise ValueError(f"{what}: one slot and one start for each sequence")
        self._attention_rows(what, int(cu_seqlens[n_sl]), q, out)
        self._history(what, kv, kv_scales, n_kv_heads, block)
        rc = lib().wave_history_attention(self.h, layer, n_sl, cu, sl, s0, _type_of(q), _ptr(q), _rows(q, what), _ptr(kv),
                                          _ptr(kv_scales), n_kv_heads, block, self.cfg.head_dim ** -0.5 if scale is None else scale,
                                          _ptr(out), _rows(out, what), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, what)
        return rc

    def history_attention_frame(self, layer, positions, q, kv, kv_scales, n_kv_heads, block, out, scale=None, stream=None,
                                check=True) -> int:
        """wave_history_attention_frame: the same for one token of each
        session, row s in slot s at positions[s] (int32 on the device;
        negative: an empty slot, whose row is left as it is)."""
        what, S = "wave_history_attention_frame", positions.numel()
        self._attention_rows(what, S, q, out)
        self._history(what, kv, kv_scales, n_kv_heads, block)
        if self.h:
            _held(positions, "int32", S, self.device, f"{what}: positions")
        rc = lib().wave_history_attention_frame(self.h, layer, S, _ptr(positions), _type_of(q), _ptr(q), _rows(q, what), _ptr(kv),
                                                _ptr(kv_scales), n_kv_heads, block,
                                                self.cfg.head_dim ** -0.5 if scale is None else scale, _ptr(out),
                                                _rows(out, what), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, what)
        return rc

    def status(self, sync: bool = True) -> int:
        """wave_status.  The C call synchronises nothing and reports the
        launches already finished; with sync (the default) the device is
        synchronised first, so that it reports every launch made so far."""
        if sync:
            import torch
            torch.cuda.synchronize()
        return lib().wave_status(self.h)

    def set_timeout_ns(self, ns: int) -> None:
        rc = lib().wave_set_timeout_ns(self.h, ns)
        if rc != WAVE_OK:
            raise WaveError(rc, "wave_set_timeout_ns")

    def debug_skip_barrier(self, cta: int, barrier: int) -> None:
        lib().wave_debug_skip_barrier(self.h, cta, barrier)

    def debug_skip_signal(self, which: int, index: int) -> None:
        """Testing hook: later steps never publish item `index` of kind
        `which` (0 QKV tile, 1 gate/up tile, 2 a head's attention rows, 3 O
        tile, 4 down tile, 5 norm row; hybrid: 6 selective-state
        in-projection tile, 7 a CTA's finished state items, 8 selective-state
        out-projection tile; prompts: 9 a CTA's K/V tile of the attention, 10
        a CTA's chunk of the selective state, 11 a CTA's K/V tile of the
        attention over the history); index < 0 disables."""
        rc = lib().wave_debug_skip_signal(self.h, which, index)
        if rc != WAVE_OK:
            raise WaveError(rc, "wave_debug_skip_signal")

    def debug_dump_kv(self, dst) -> None:
        """Testing hook: later steps write their pre-quantisation K/V rows
        into dst ([L][2][S_max][H][D] fp32 on the device); None disables."""
        lib().wave_debug_dump_kv(self.h, _ptr(dst))

    def debug_dump_acts(self, dst, n_sessions: int = 0) -> None:
        """Testing hook: later launches record every phase's input and output
        for sessions 0..n_sessions-1 into dst ([frames][layers][n][R] fp32 on
        the device, R = act_record_floats); None disables."""
        rc = lib().wave_debug_dump_acts(self.h, _ptr(dst), n_sessions if dst is not None else 0)
        if rc != WAVE_OK:
            raise WaveError(rc, "wave_debug_dump_acts")

    @property
    def act_record_floats(self) -> int:
        return lib().wave_debug_act_record_floats(self.h)

    def debug_phase_times(self, dst) -> None:
        """Profiling hook: later steps write globaltimer stamps (int64) at
        entry, after every grid barrier and at exit into dst; None disables."""
        lib().wave_debug_phase_times(self.h, _ptr(dst))

    def debug_arrival_times(self, dst) -> None:
        """Profiling hook: later steps write the globaltimer stamp at which
        each CTA finished each phase into dst ([phases][grid] int64); None
        disables."""
        lib().wave_debug_arrival_times(self.h, _ptr(dst))

    @property
    def grid(self) -> int:
        return lib().wave_grid_size(self.h)

    @property
    def barriers_per_step(self) -> int:
        return lib().wave_barriers_per_step(self.h)

    @property
    def phases_per_step(self) -> int:
        return lib().wave_phases_per_step(self.h)

    def close(self) -> None:
        if getattr(self, "h", None):
            lib().wave_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def step_static(cfg: WaveConfig, S_max: int, T_max: int, S: int, weights, kv, kv_scales, positions,
                x, y, stream=None) -> int:
    """wave_step_static: one frame with the library's fixed scratch instead
    of an allocated workspace, for callers that cannot allocate device memory.
    Waits for the step and returns its status code."""
    return lib().wave_step_static(ctypes.byref(cfg), S_max, T_max, S, _ptr(weights), _ptr(kv),
                                  _ptr(kv_scales), _ptr(positions), _ptr(x), _ptr(y),
                                  _stream(stream))


def kv_quantize(v, codes, scales, stream=None) -> None:
    """FP8 quantiser of the K/V append on rows of v (last dim D)."""
    D = v.shape[-1]
    rows = v.numel() // D
    rc = lib().wave_kv_quantize(_ptr(v), rows, D, _ptr(codes), _ptr(scales), _stream(stream))
    if rc != WAVE_OK:
        raise WaveError(rc, "wave_kv_quantize")


def fp8_encode(inp, out, stream=None, n: int | None = None) -> None:
    n = inp.numel() if n is None else n
    rc = lib().wave_fp8_encode(_ptr(inp), n, _ptr(out), _stream(stream))
    if rc != WAVE_OK:
        raise WaveError(rc, "wave_fp8_encode")


def rope_plan(dims: int, base: float = 10000.0, layout: str = "half", scaling: str = "none", factor: float = 1.0,
              original: float = 0.0, fast: float = 32.0, slow: float = 1.0, amplitude: float = 1.0) -> WaveRope:
    """wave_rope_plan: rotary positions of the leading `dims` values of a head.
    layout "half" (pairs (i, i + dims/2)) or "interleaved" ((2i, 2i + 1));
    scaling "none", "linear" (frequencies / factor) or "parts" (only those of
    few turns over `original` positions)."""
    if layout not in _ROPE_LAYOUTS or scaling not in _ROPE_SCALINGS:
        raise ValueError('wave_rope_plan: layout is "half" or "interleaved", scaling "none", "linear" or "parts"')
    c = WaveRopeConfig(_ROPE_LAYOUTS[layout], dims, base, _ROPE_SCALINGS[scaling], factor, original, fast, slow, amplitude)
    plan = WaveRope()
    rc = lib().wave_rope_plan(ctypes.byref(c), ctypes.addressof(plan))
    if rc != WAVE_OK:
        raise WaveError(rc, "wave_rope_plan")
    return plan


def _plan(rope) -> int | None:
    if rope is None:
        return None
    if not isinstance(rope, WaveRope):
        raise ValueError("a plan made by rope_plan is wanted")
    return ctypes.addressof(rope)


def rope_apply(plan, x, out=None, cu_seqlens=None, starts=None, positions=None, stream=None) -> None:
    """wave_rope_apply (cu_seqlens and starts: host integers, rows of packed
    prompts) or wave_rope_apply_at (positions: int32 on the device, one for each
    row).  x and out are [rows][heads][D] of fp32, bf16 or fp16 on the current
    device, rows may be strided; out defaults to x itself."""
    out = x if out is None else out
    what = "wave_rope_apply"
    if len(x.shape) != 3 or x.shape[1:] != out.shape[1:] or (positions is None) == (cu_seqlens is None or starts is None):
        raise ValueError(f"{what}: x and out are [rows][heads][D]; either cu_seqlens and starts or positions are given")
    if positions is None:
        (cu, n_cu), (s0, n_s0) = _ints(cu_seqlens), _ints(starts)
        if n_cu < 2 or n_s0 != n_cu - 1:
            raise ValueError(f"{what}: one start for each sequence")
        rows = int(cu_seqlens[n_s0])
    else:
        rows = positions.numel()
    if x.shape[0] < rows or out.shape[0] < rows:
        raise ValueError(f"{what}: x and out have the rows that the call names")
    if not x.is_cuda:
        raise ValueError(f"{what}: tensors on the current device are wanted, not on {x.device}")
    import torch
    device = torch.cuda.current_device()
    _here(device, what, x, out)
    if positions is not None:
        _DTYPES.setdefault("int32", torch.int32)
        _held(positions, "int32", rows, device, f"{what}: positions")
    heads, D = x.shape[1], x.shape[2]
    xs = (_ptr(x), _type_of(x), _rows(x, what), _ptr(out), _type_of(out), _rows(out, what), _stream(stream))
    if positions is None:
        rc = lib().wave_rope_apply(_plan(plan), n_s0, cu, s0, heads, D, *xs)
    else:
        rc = lib().wave_rope_apply_at(_plan(plan), rows, _ptr(positions), heads, D, *xs)
    if rc != WAVE_OK:
        raise WaveError(rc, what)


class HybridWave(Wave):
    """A hybrid-step context: wave_hybrid_create / wave_hybrid_step (status,
    hooks and close as Wave)."""

    def __init__(self, cfg: WaveHybridConfig, S_max: int, T_max: int):
        self.cfg = cfg
        self.S_max, self.T_max = S_max, T_max
        h = ctypes.c_void_p()
        rc = lib().wave_hybrid_create(ctypes.byref(cfg), S_max, T_max, ctypes.byref(h))
        if rc != WAVE_OK:
            raise WaveError(rc, "wave_hybrid_create")
        self.h = h
        self._sizes()

    def hybrid_step(self, S, weights, kv, kv_scales, ssm_state, positions, x, y, stream=None,
                    check=True) -> int:
        rc = lib().wave_hybrid_step(self.h, S, _ptr(weights), _ptr(kv), _ptr(kv_scales), _ptr(ssm_state),
                                    _ptr(positions), _ptr(x), _ptr(y), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, "wave_hybrid_step")
        return rc

    def prompt_state(self, layer, weights, cu_seqlens, slots, starts, zxbcdt, state_in, state_out, out, stream=None,
                     check=True) -> int:
        """wave_hybrid_prompt_state: the selective-state block `layer` over
        packed prompts.  zxbcdt is bf16 [rows][in_rows] and out bf16
        [rows][d_inner], rows may be strided; state_in (None when every start
        is 0) and state_out are the fp32 state, which may be one buffer."""
        (cu, n_cu), (sl, n_sl), (s0, n_s0) = _ints(cu_seqlens), _ints(slots), _ints(starts)
        if n_cu < 2 or n_sl != n_cu - 1 or n_s0 != n_sl:
            raise ValueError("wave_hybrid_prompt_state: one slot and one start for each sequence")
        c = self.cfg
        di = c.ssm_heads * c.ssm_head_dim
        zs, ys = zxbcdt.shape, out.shape
        if len(zs) != 2 or len(ys) != 2 or zs[1] != 2 * di + 2 * c.ssm_state + c.ssm_heads or ys[1] != di \
                or _type_of(zxbcdt) != WAVE_BF16 or _type_of(out) != WAVE_BF16:
            raise ValueError("wave_hybrid_prompt_state: zxbcdt is bf16 [rows][in_rows], out bf16 [rows][d_inner]")
        if min(zs[0], ys[0]) < int(cu_seqlens[n_sl]):
            raise ValueError("wave_hybrid_prompt_state: cu_seqlens names more rows than a buffer has")
        if self.h:
            _here(self.device, "wave_hybrid_prompt_state", zxbcdt, out)
            _held(weights, 2, self._n_weights, self.device, "wave_hybrid_prompt_state: weights")
            _held(state_in, "float32", self._n_state, self.device, "wave_hybrid_prompt_state: state_in")
            _held(state_out, "float32", self._n_state, self.device, "wave_hybrid_prompt_state: state_out")
        rc = lib().wave_hybrid_prompt_state(self.h, layer, _ptr(weights), n_sl, cu, sl, s0, _ptr(zxbcdt),
                                            _rows(zxbcdt, "zxbcdt"), _ptr(state_in), _ptr(state_out), _ptr(out),
                                            _rows(out, "out"), _stream(stream))
        if check and rc != WAVE_OK:
            raise WaveError(rc, "wave_hybrid_prompt_state")
        return rc


def hybrid_weights_bytes(cfg: WaveHybridConfig) -> int:
    return lib().wave_hybrid_weights_bytes(ctypes.byref(cfg))


def hybrid_layer_offset(cfg: WaveHybridConfig, layer: int) -> int:
    return lib().wave_hybrid_layer_offset(ctypes.byref(cfg), layer)
