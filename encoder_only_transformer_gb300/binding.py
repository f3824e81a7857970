"""Thin ctypes binding of libmbert_attn.so (argument marshalling only).

Every step of the attention block runs in the library's CUDA kernels; this
module checks torch dtypes, devices and shapes, passes raw device pointers
and the current CUDA stream, and turns status codes into exceptions.  There
is no fallback: if the library is missing, every call raises.
"""
import ctypes
import os
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libmbert_attn.so"

GLOBAL = 0
LOCAL = 1
_KINDS = {"global": GLOBAL, "local": LOCAL, GLOBAL: GLOBAL, LOCAL: LOCAL}

HEADS, HEAD_DIM = 12, 64
QKV_WIDTH, OUT_WIDTH = 3 * HEADS * HEAD_DIM, HEADS * HEAD_DIM
MLP_INNER = 1152  # the GeGLU MLP's inner width (teardown, "What Does the GeGLU MLP Do?")
NORM_EPS = 1e-5   # LayerNorm eps of ModernBERT-base (teardown, "What Does LayerNorm Do?")

# Every symbol the public header declares, with its ctypes signature.
_c_int, _c_i64, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p


class Config(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("half_window", ctypes.c_int), ("max_seqlen", ctypes.c_int),
                ("theta_global", ctypes.c_double), ("theta_local", ctypes.c_double)]


class Scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("original", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("amplitude", ctypes.c_double)]


class RotarySpec(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int), ("layout", ctypes.c_int), ("amplitude", ctypes.c_double),
                ("freq", ctypes.c_double * 128)]


class Heads(ctypes.Structure):
    _fields_ = [("src", _vp), ("dst", _vp), ("weight", _vp), ("heads", ctypes.c_int),
                ("src_row", _c_i64), ("src_head", _c_i64), ("dst_row", _c_i64), ("dst_head", _c_i64)]


class CrossArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("out", _vp),
                ("q_row", _c_i64), ("k_row", _c_i64), ("v_row", _c_i64), ("out_row", _c_i64),
                ("rows_q", _c_i64), ("rows_k", _c_i64),
                ("heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("n_seqs", ctypes.c_int),
                ("cu_q", _vp), ("cu_k", _vp), ("max_seqlen_q", ctypes.c_int), ("key_mask", _vp)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("weight", _vp), ("bias", _vp), ("residual", _vp), ("out", _vp),
                ("x_row", _c_i64), ("weight_row", _c_i64), ("weight_expert", _c_i64), ("residual_row", _c_i64),
                ("out_row", _c_i64), ("rows", _c_i64), ("inner", _c_int), ("outer", _c_int), ("dtype", _c_int),
                ("activation", _c_int), ("gated", _c_int), ("experts", _c_int), ("cu_experts", _vp),
                ("row_scale", _vp)]


class ResidualNormArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("branch", _vp), ("gate", _vp), ("weight", _vp), ("bias", _vp),
                ("branch_weight", _vp), ("branch_bias", _vp), ("h", _vp), ("y", _vp),
                ("x_row", _c_i64), ("branch_row", _c_i64), ("gate_row", _c_i64), ("h_row", _c_i64), ("y_row", _c_i64),
                ("rows", _c_i64), ("width", _c_int), ("dtype", _c_int), ("norm", _c_int), ("gate_kind", _c_int),
                ("cu_seqlens", _vp), ("n_seqs", _c_int), ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)]


_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3, "yarn": 4}
_NORMS = {"rms": 1, "layer": 2}
_ACTIVATIONS = {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3, "relu": 4}

SIGNATURES = {
    "mbert_attn_default_config": (_c_int, [ctypes.POINTER(Config)]),
    "mbert_attn_create": (_c_int, [ctypes.POINTER(_vp), ctypes.POINTER(Config), _c_int]),
    "mbert_attn_reserve": (_c_int, [_vp, _c_i64, _c_i64]),
    "mbert_attn_forward": (_c_int, [_vp, _vp, _vp, _c_int, _c_i64, _c_int, _c_int, _vp, _vp]),
    "mbert_attn_forward_padded": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp]),
    "mbert_attn_key_counts": (_c_int, [_vp, _vp, _c_int, _c_i64, _c_int, _c_int, _vp, _vp]),
    "mbert_attn_out_proj": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _vp, _vp]),
    "mbert_attn_ln_qkv": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, ctypes.c_float, _vp, _vp]),
    "mbert_attn_mlp": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_i64, ctypes.c_float, _vp, _vp]),
    "mbert_attn_rotary_init": (_c_int, [ctypes.POINTER(RotarySpec), _c_int, _c_int, ctypes.c_double,
                                        ctypes.POINTER(Scaling)]),
    "mbert_attn_rotary": (_c_int, [_vp, ctypes.POINTER(Heads), _c_i64, _c_int, _c_int,
                                   ctypes.POINTER(RotarySpec), _vp, _c_int, _vp, _c_int, _c_int, _vp]),
    "mbert_attn_qk_norm_rotary": (_c_int, [_vp, ctypes.POINTER(Heads), ctypes.POINTER(Heads), _c_i64,
                                           _c_int, _c_int, _c_int, ctypes.c_float,
                                           ctypes.POINTER(RotarySpec), _vp, _c_int, _vp, _c_int, _vp]),
    "mbert_attn_cross_workspace": (_c_int, [_vp, ctypes.POINTER(CrossArgs), ctypes.POINTER(_c_i64)]),
    "mbert_attn_cross": (_c_int, [_vp, ctypes.POINTER(CrossArgs), _vp, _c_i64, _vp]),
    "mbert_attn_linear": (_c_int, [_vp, ctypes.POINTER(LinearArgs), _vp]),
    "mbert_attn_linear_plan": (_c_int, [_vp, ctypes.POINTER(LinearArgs), ctypes.POINTER(ctypes.c_int32)]),
    "mbert_attn_residual_norm": (_c_int, [_vp, ctypes.POINTER(ResidualNormArgs), _vp]),
    "mbert_attn_get_error": (_c_int, [_vp]),
    "mbert_attn_selftest_timeout": (_c_int, [_vp, _c_i64, _vp]),
    "mbert_attn_forward_noalloc": (_c_int, [_vp, _vp, _c_int, _c_i64, _c_int, _c_int, _vp, _vp,
                                            _vp]),
    "mbert_attn_profile_enable": (_c_int, [_vp, _c_int]),
    "mbert_attn_profile_read": (_c_int, [_vp, ctypes.POINTER(ctypes.c_double),
                                         ctypes.POINTER(ctypes.c_int64),
                                         ctypes.POINTER(ctypes.c_int64)]),
    "mbert_attn_destroy": (None, [_vp]),
    "mbert_attn_strerror": (ctypes.c_char_p, [_c_int]),
}

_lib = None
_lib_lock = threading.Lock()


class MbertAttnError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        msg = strerror(status) if _lib is not None else str(status)
        super().__init__(f"{what}: {msg} (status {status})" if what else f"{msg} (status {status})")


def library_path() -> str:
    return os.path.join(PKG, "_build", LIB_NAME)


def load_library(path: str = None):
    """Load the CUDA library (once).  Raises OSError if it is not built."""
    global _lib
    with _lib_lock:
        if _lib is None:
            p = path or library_path()
            if not os.path.exists(p):
                raise OSError(f"{p} is missing: build it with "
                              f"`python -c 'import __graft_entry__ as g; g.build()'`")
            lib = ctypes.CDLL(p)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def strerror(status: int) -> str:
    return load_library().mbert_attn_strerror(int(status)).decode()


def _check(status, what):
    if status != 0:
        raise MbertAttnError(status, what)


def _kind(layer_kind) -> int:
    try:
        return _KINDS[layer_kind]
    except KeyError:
        raise ValueError(f"layer_kind must be 'global', 'local', 0 or 1, not {layer_kind!r}")


def _stream_ptr(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the current stream's handle without a Stream object around it (a tenth of
# the time, which single-token calls feel), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device) -> int:
    return _raw_stream(device.index) if _raw_stream is not None else _stream_ptr(device)


def _layout(*tensors):
    """What the checks of a call look at besides the pointers."""
    return tuple([(t.shape, t.stride(), t.dtype, t.device) for t in tensors])


def _key(t):
    """One tensor's part of such a look, with the device as a number (-1 for the
    host): cheaper to make and to compare."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


_INT_MAX = 2 ** 31 - 1


class Rotary:
    """How a head is rotated: its first `dim` numbers (even, up to 256) in
    pairs, `layout` "half" (x[m], x[m + dim/2]) or "interleaved" (x[2m],
    x[2m+1]), pair m by position * base^(-2m/dim).  `scaling` stretches the
    frequencies for contexts longer than the trained one, a dict with "kind":

      "linear"    factor: f / factor
      "ntk"       factor: base * factor^(dim/(dim-2))
      "by_parts"  factor, original, low=1, high=32: with r = original f / 2 pi
                  turns over the original context, f where r >= high, f/factor
                  where r <= low, linear in r between
      "yarn"      factor, original, low=1, high=32, amplitude=None: the same
                  borders as rounded pair numbers and a ramp over the pair
                  numbers between; rows times 0.1 ln(factor) + 1 unless given

    Host data only: made once, usable on every device."""

    def __init__(self, dim: int, base: float = 10000.0, layout: str = "half", scaling: dict = None):
        if dim != int(dim):
            raise ValueError(f"dim must be a whole number, not {dim!r}")
        # (ctypes would cut a larger number to its lower 32 bits)
        if abs(int(dim)) > _INT_MAX:
            raise MbertAttnError(-1, "rotary_init")
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
        sc = None
        if scaling is not None:
            given = dict(scaling)
            kind = given.pop("kind", None)
            if kind not in _SCALINGS:
                raise ValueError(f"scaling kind must be one of {sorted(_SCALINGS)}, not {kind!r}")
            takes = {"none": (), "linear": ("factor",), "ntk": ("factor",),
                     "by_parts": ("factor", "original", "low", "high"),
                     "yarn": ("factor", "original", "low", "high", "amplitude")}[kind]
            extra = sorted(set(given) - set(takes))
            missing = sorted(({"factor", "original"} & set(takes)) - set(given))
            if extra or missing:
                raise ValueError(f"scaling {kind!r}: unknown {extra}, missing {missing}")
            amplitude = given.get("amplitude")
            if amplitude is not None and not amplitude > 0:
                raise ValueError("scaling amplitude must be positive")
            sc = Scaling(_SCALINGS[kind], float(given.get("factor", 1.0)),
                         float(given.get("original", 1.0)), float(given.get("low", 1.0)),
                         float(given.get("high", 32.0)), float(amplitude or 0.0))
        self.spec = RotarySpec()
        _check(load_library().mbert_attn_rotary_init(
            ctypes.byref(self.spec), int(dim), _LAYOUTS[layout], float(base),
            None if sc is None else ctypes.byref(sc)), "rotary_init")
        self._ref = ctypes.byref(self.spec)

    @property
    def dim(self) -> int:
        return self.spec.dim

    @property
    def frequencies(self):
        """Radians per position of each pair."""
        return list(self.spec.freq[:self.spec.dim // 2])

    @property
    def amplitude(self) -> float:
        return self.spec.amplitude


class Attention:
    """A library handle on one CUDA device (owns the RoPE tables, the work
    list, the rotated-operand scratch and the device error word)."""

    def __init__(self, device=None, half_window: int = 64, max_seqlen: int = 8192,
                 theta_global: float = 160000.0, theta_local: float = 10000.0):
        lib = load_library()
        if device is None:
            idx = torch.cuda.current_device()
        elif isinstance(device, int):
            idx = device
        else:
            d = torch.device(device)
            idx = d.index if d.index is not None else torch.cuda.current_device()
        self.device = torch.device("cuda", idx)
        cfg = Config()
        _check(lib.mbert_attn_default_config(ctypes.byref(cfg)), "default_config")
        cfg.half_window = half_window
        cfg.max_seqlen = max_seqlen
        cfg.theta_global = theta_global
        cfg.theta_local = theta_local
        self.config = cfg
        h = _vp()
        _check(lib.mbert_attn_create(ctypes.byref(h), ctypes.byref(cfg), self.device.index), "create")
        self._h = h
        # layouts that have passed a call's checks, and what follows from them
        # (no data, no addresses): a call like an earlier one skips the checks
        self._known = {}

    def _remember(self, key, value):
        if len(self._known) >= 1024:
            self._known.clear()
        self._known[key] = value
        return value

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            load_library().mbert_attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check_cu(self, cu_seqlens):
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1:
            raise TypeError("cu_seqlens must be a 1-D int32 tensor")
        if cu_seqlens.device != self.device:
            raise ValueError(f"cu_seqlens must be on {self.device}")
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")

    def reserve(self, max_tokens: int, max_seqs: int):
        _check(load_library().mbert_attn_reserve(self._h, int(max_tokens), int(max_seqs)), "reserve")

    def forward(self, qkv: torch.Tensor, cu_seqlens: torch.Tensor, layer_kind,
                max_seqlen: int = 0, out: torch.Tensor = None) -> torch.Tensor:
        """out[T, 768] bf16 = the attention block of one layer over qkv[T, 2304]."""
        kind = _kind(layer_kind)
        if qkv.dtype != torch.bfloat16 or qkv.dim() != 2 or qkv.shape[1] != QKV_WIDTH:
            raise TypeError("qkv must be a bf16 tensor of shape [T, 2304]")
        if qkv.device != self.device:
            raise ValueError(f"qkv must be on {self.device}")
        if not qkv.is_contiguous():
            raise ValueError("qkv must be contiguous")
        self._check_cu(cu_seqlens)
        T = qkv.shape[0]
        if out is None:
            out = torch.empty(T, OUT_WIDTH, dtype=torch.bfloat16, device=self.device)
        elif (out.dtype != torch.bfloat16 or tuple(out.shape) != (T, OUT_WIDTH)
              or out.device != self.device or not out.is_contiguous()):
            raise TypeError("out must be a contiguous bf16 [T, 768] tensor on the same device")
        st = load_library().mbert_attn_forward(
            self._h, qkv.data_ptr(), cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, T,
            int(max_seqlen), kind, out.data_ptr(), _stream_ptr(self.device))
        _check(st, "forward")
        return out

    def out_proj(self, a: torch.Tensor, wo: torch.Tensor, x: torch.Tensor,
                 out: torch.Tensor = None) -> torch.Tensor:
        """y[T, 768] bf16 = x + a Wo^T: the output projection (Wo [768, 768],
        stored [out, in]) with the residual add.  `out` may be `x` itself."""
        def check(t, name, shape):
            if (t.dtype != torch.bfloat16 or tuple(t.shape) != shape or t.device != self.device
                    or not t.is_contiguous()):
                raise TypeError(f"{name} must be a contiguous bf16 {list(shape)} tensor on {self.device}")
        T = a.shape[0] if a.dim() == 2 else -1
        check(a, "a", (T, OUT_WIDTH))
        check(wo, "wo", (OUT_WIDTH, OUT_WIDTH))
        check(x, "x", (T, OUT_WIDTH))
        if out is None:
            out = torch.empty(T, OUT_WIDTH, dtype=torch.bfloat16, device=self.device)
        check(out, "out", (T, OUT_WIDTH))
        st = load_library().mbert_attn_out_proj(self._h, a.data_ptr(), wo.data_ptr(), x.data_ptr(),
                                                T, out.data_ptr(), _stream_ptr(self.device))
        _check(st, "out_proj")
        return out

    def forward_padded(self, qkv: torch.Tensor, attention_mask: torch.Tensor, layer_kind,
                       out: torch.Tensor = None) -> torch.Tensor:
        """out[B, S, 768] bf16 for a padded batch: qkv [B, S, 2304] bf16 and
        attention_mask [B, S] int32 (1 = real token, 0 = pad) on this device;
        pad rows of out are zeros."""
        kind = _kind(layer_kind)
        if qkv.dim() != 3 or qkv.shape[2] != QKV_WIDTH or qkv.dtype != torch.bfloat16 \
                or qkv.device != self.device or not qkv.is_contiguous():
            raise TypeError(f"qkv must be a contiguous bf16 [B, S, {QKV_WIDTH}] tensor on {self.device}")
        B, S = qkv.shape[0], qkv.shape[1]
        if (attention_mask.dtype != torch.int32 or tuple(attention_mask.shape) != (B, S)
                or attention_mask.device != self.device or not attention_mask.is_contiguous()):
            raise TypeError(f"attention_mask must be a contiguous int32 [{B}, {S}] tensor on {self.device}")
        if out is None:
            out = torch.empty(B, S, OUT_WIDTH, dtype=torch.bfloat16, device=self.device)
        if (out.dtype != torch.bfloat16 or tuple(out.shape) != (B, S, OUT_WIDTH)
                or out.device != self.device or not out.is_contiguous()):
            raise TypeError(f"out must be a contiguous bf16 [{B}, {S}, {OUT_WIDTH}] tensor")
        st = load_library().mbert_attn_forward_padded(self._h, qkv.data_ptr(),
                                                      attention_mask.data_ptr(), B, S, kind,
                                                      out.data_ptr(), _stream_ptr(self.device))
        _check(st, "forward_padded")
        return out

    def ln_qkv(self, x: torch.Tensor, norm_w, wqkv: torch.Tensor, eps: float = NORM_EPS,
               out: torch.Tensor = None) -> torch.Tensor:
        """qkv[T, 2304] bf16 = LayerNorm(x) Wqkv^T: the bias-free pre-attention
        norm (weight norm_w [768], or None for layer 0's identity) and the
        fused Wqkv projection (Wqkv [2304, 768], stored [out, in])."""
        def check(t, name, shape):
            if (t.dtype != torch.bfloat16 or tuple(t.shape) != shape or t.device != self.device
                    or not t.is_contiguous()):
                raise TypeError(f"{name} must be a contiguous bf16 {list(shape)} tensor on {self.device}")
        T = x.shape[0] if x.dim() == 2 else -1
        check(x, "x", (T, OUT_WIDTH))
        if norm_w is not None:
            check(norm_w, "norm_w", (OUT_WIDTH,))
        check(wqkv, "wqkv", (QKV_WIDTH, OUT_WIDTH))
        if out is None:
            out = torch.empty(T, QKV_WIDTH, dtype=torch.bfloat16, device=self.device)
        check(out, "out", (T, QKV_WIDTH))
        st = load_library().mbert_attn_ln_qkv(
            self._h, x.data_ptr(), None if norm_w is None else norm_w.data_ptr(), wqkv.data_ptr(),
            T, float(eps), out.data_ptr(), _stream_ptr(self.device))
        _check(st, "ln_qkv")
        return out

    def mlp(self, x: torch.Tensor, norm_w: torch.Tensor, wi: torch.Tensor, wo: torch.Tensor,
            eps: float = NORM_EPS, out: torch.Tensor = None) -> torch.Tensor:
        """y[T, 768] bf16 = x + (GELU(g) * u) Wo^T, g and u the halves of
        LayerNorm(x) Wi^T (norm_w [768], Wi [2304, 768], Wo [768, 1152], stored
        [out, in]).  `out` may be `x` itself."""
        def check(t, name, shape):
            if (t.dtype != torch.bfloat16 or tuple(t.shape) != shape or t.device != self.device
                    or not t.is_contiguous()):
                raise TypeError(f"{name} must be a contiguous bf16 {list(shape)} tensor on {self.device}")
        T = x.shape[0] if x.dim() == 2 else -1
        check(x, "x", (T, OUT_WIDTH))
        check(norm_w, "norm_w", (OUT_WIDTH,))
        check(wi, "wi", (2 * MLP_INNER, OUT_WIDTH))
        check(wo, "wo", (OUT_WIDTH, MLP_INNER))
        if out is None:
            out = torch.empty(T, OUT_WIDTH, dtype=torch.bfloat16, device=self.device)
        check(out, "out", (T, OUT_WIDTH))
        st = load_library().mbert_attn_mlp(self._h, x.data_ptr(), norm_w.data_ptr(), wi.data_ptr(),
                                           wo.data_ptr(), T, float(eps), out.data_ptr(),
                                           _stream_ptr(self.device))
        _check(st, "mlp")
        return out

    def _check_heads(self, t, name, like=None):
        """A [T, H, D] tensor on this device whose last dimension is contiguous."""
        if t.dim() != 3 or t.dtype not in _DTYPES or t.device != self.device:
            raise TypeError(f"{name} must be a bf16, fp16 or fp32 [T, heads, head_dim] tensor on {self.device}")
        if t.shape[2] > 1 and t.stride(2) != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")
        if like is not None and (t.shape[0] != like.shape[0] or t.shape[2] != like.shape[2]
                                 or t.dtype != like.dtype):
            raise TypeError(f"{name} must have the rows, head size and type of the other tensor")

    def _heads_template(self, src, dst):
        """The Heads of a [T, H, D] tensor and its result (None: a new one)
        without the pointers."""
        T, H, D = src.shape
        (a, b, _), (c, d, _) = src.stride(), (H * D, D, 1) if dst is None else dst.stride()
        if T <= 1 or H <= 1:
            # a dimension of one element has no stride that matters
            a, c = (a, c) if T > 1 else (H * D, H * D)
            b, d = (b, d) if H > 1 else (D, D)
        return bytes(Heads(None, None, None, H, a, b, c, d))

    def _check_out(self, out, name, like):
        self._check_heads(out, name, like)
        if out.shape != like.shape:
            raise TypeError(f"{name} must have the shape {list(like.shape)}")

    def _positions(self, positions, cu_seqlens, tokens):
        """-> (positions pointer, bits, cu_seqlens pointer, sequences)"""
        if (positions is None) == (cu_seqlens is None):
            raise ValueError("give either positions or cu_seqlens")
        if positions is None:
            self._check_cu(cu_seqlens)
            return None, 0, cu_seqlens.data_ptr(), cu_seqlens.shape[0] - 1
        if (positions.dtype not in (torch.int32, torch.int64) or positions.shape != (tokens,)
                or positions.device != self.device or not positions.is_contiguous()):
            raise TypeError(f"positions must be a contiguous int32 or int64 [{tokens}] tensor on {self.device}")
        return positions.data_ptr(), 8 * positions.element_size(), None, 0

    def rotary(self, x: torch.Tensor, rope: Rotary, positions: torch.Tensor = None,
               cu_seqlens: torch.Tensor = None, inverse: bool = False,
               out: torch.Tensor = None) -> torch.Tensor:
        """out[T, H, D] = x with every head turned by its row's position (bf16,
        fp16 or fp32, fp32 arithmetic).  Positions: int32 or int64 [T], or from
        cu_seqlens (int32 [n+1]; a row's place in its sequence; rows behind the
        last sequence are left as they were).  x may be strided (a view of fused
        rows); out may be x.  inverse=True turns the other way (the transpose:
        the gradient of a turned tensor goes back through it)."""
        key = ("rotary", _layout(x)) if out is None else ("rotary", _layout(x), _layout(out))
        known = self._known.get(key)
        if known is None:
            self._check_heads(x, "x")
            if out is not None:
                self._check_out(out, "out", x)
            known = self._remember(key, (x.shape[0], x.shape[2], _DTYPES[x.dtype], self._heads_template(x, out)))
        T, D, dtype, template = known
        pos, bits, cu, n = self._positions(positions, cu_seqlens, T)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=self.device)
        heads = Heads.from_buffer_copy(template)
        heads.src, heads.dst = x.data_ptr(), out.data_ptr()
        st = _lib.mbert_attn_rotary(self._h, ctypes.byref(heads), T, D, dtype, rope._ref, pos, bits, cu, n,
                                    1 if inverse else 0, _stream_of(self.device))
        if st != 0:
            _check(st, "rotary")
        return out

    def qk_norm_rotary(self, q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor,
                       k_weight: torch.Tensor, rope: Rotary = None, positions: torch.Tensor = None,
                       cu_seqlens: torch.Tensor = None, norm: str = "rms", eps: float = 1e-6,
                       q_out: torch.Tensor = None, k_out: torch.Tensor = None):
        """(q_out, k_out) = every query and key head normed over its D numbers
        ("rms" or bias-free "layer", weight [D]) and then turned, in one kernel.
        q [T, Hq, D] and k [T, Hk, D] share rows and type; either may be None.
        rope None: the norm alone.  Positions, strides and in-place use as in
        rotary."""
        if norm not in _NORMS:
            raise ValueError(f"norm must be 'rms' or 'layer', not {norm!r}")
        first = q if q is not None else k
        if first is None:
            raise ValueError("give q, k or both")
        sides = []
        for t, w, o, name in ((q, q_weight, q_out, "q"), (k, k_weight, k_out, "k")):
            if t is None:
                sides.append(None)
            elif w is None:
                raise TypeError(f"{name}_weight is missing")
            else:
                sides.append(_layout(t, w) if o is None else _layout(t, w, o))
        key = ("qk_norm_rotary", sides[0], sides[1])
        known = self._known.get(key)
        if known is None:
            templates = []
            for t, w, o, name in ((q, q_weight, q_out, "q"), (k, k_weight, k_out, "k")):
                if t is None:
                    templates.append(None)
                    continue
                self._check_heads(t, name, first)
                if (w.dtype != t.dtype or tuple(w.shape) != (t.shape[2],)
                        or w.device != self.device or not w.is_contiguous()):
                    raise TypeError(f"{name}_weight must be a contiguous [{t.shape[2]}] tensor of {name}'s type")
                if o is not None:
                    self._check_out(o, f"{name}_out", t)
                templates.append(self._heads_template(t, o))
            known = self._remember(key, (first.shape[0], first.shape[2], _DTYPES[first.dtype], *templates))
        T, D, dtype, q_template, k_template = known
        if rope is None or rope.dim == 0:
            if positions is not None or cu_seqlens is not None:
                raise ValueError("positions or cu_seqlens without a rotation")
            pos, bits, cu, n = None, 0, None, 0
        else:
            pos, bits, cu, n = self._positions(positions, cu_seqlens, T)
        q_ref = k_ref = None
        if q is None:
            q_out = None
        else:
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
            heads = Heads.from_buffer_copy(q_template)
            heads.src, heads.dst, heads.weight = q.data_ptr(), q_out.data_ptr(), q_weight.data_ptr()
            q_ref = ctypes.byref(heads)
        if k is None:
            k_out = None
        else:
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=self.device)
            heads = Heads.from_buffer_copy(k_template)
            heads.src, heads.dst, heads.weight = k.data_ptr(), k_out.data_ptr(), k_weight.data_ptr()
            k_ref = ctypes.byref(heads)
        st = _lib.mbert_attn_qk_norm_rotary(
            self._h, q_ref, k_ref, T, D, dtype, _NORMS[norm], float(eps), None if rope is None else rope._ref,
            pos, bits, cu, n, _stream_of(self.device))
        if st != 0:
            _check(st, "qk_norm_rotary")
        return q_out, k_out

    def _check_cross(self, t, name, dims):
        """A [..., heads, head_dim] tensor whose heads lie side by side."""
        if (t.dim() != dims or t.dtype not in (torch.bfloat16, torch.float16) or t.device != self.device
                or t.shape[-1] not in (64, 128) or t.shape[-2] < 1):
            raise TypeError(f"{name} must be a bf16 or fp16 tensor of {dims} dimensions "
                            f"[..., heads, 64 or 128] on {self.device}")
        if t.stride(-1) != 1 or (t.shape[-2] > 1 and t.stride(-2) != t.shape[-1]):
            raise ValueError(f"the heads of {name} must lie side by side in each row")

    def _cross(self, known, q, k, v, out, cu_q, cu_k, key_mask):
        """Enqueue a call whose layouts have been checked; known: the arguments
        without their pointers, and the workspace's size."""
        template, need = known
        args = CrossArgs.from_buffer_copy(template)
        args.q, args.k, args.v, args.out = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr()
        if cu_q is not None:
            args.cu_q, args.cu_k = cu_q.data_ptr(), cu_k.data_ptr()
        if key_mask is not None:
            args.key_mask = key_mask.data_ptr()
        # of the call's own, from torch's allocator: calls on other streams and
        # captured ones never share it
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        st = _lib.mbert_attn_cross(self._h, ctypes.byref(args), None if ws is None else ws.data_ptr(), need,
                                   _stream_of(self.device))
        if st != 0:
            _check(st, "cross_attention")
        return out

    def _cross_known(self, key, q, k, v, out, rows_q, rows_k, pitches, n_seqs, packed, max_seqlen_q, key_mask, scale):
        """Remember the arguments (without pointers) and the workspace's size."""
        if scale is None:
            scale = 0.0
        elif not 0.0 < ctypes.c_float(scale).value < float("inf"):
            raise ValueError("scale must be positive and finite (in fp32)")
        # the size depends on which pointers there are, not on where they point
        there = ctypes.addressof(ctypes.c_int(0))
        args = CrossArgs(None, None, None, None, *pitches, rows_q, rows_k, q.shape[-2], k.shape[-2], q.shape[-1],
                         _DTYPES[q.dtype], scale, n_seqs, there if packed else None, there if packed else None,
                         max_seqlen_q, None if key_mask is None else there)
        need = _c_i64()
        _check(load_library().mbert_attn_cross_workspace(self._h, ctypes.byref(args), ctypes.byref(need)),
               "cross_attention")
        args.cu_q = args.cu_k = args.key_mask = None
        return self._remember(key, (bytes(args), need.value))

    def cross_attention(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_seqlen_q: int = 0,
                        key_mask: torch.Tensor = None, scale: float = None,
                        out: torch.Tensor = None) -> torch.Tensor:
        """out[Tq, Hq, D] = attention of packed queries over keys and values of
        another length: q [Tq, Hq, D], k and v [Tk, Hk, D] (bf16 or fp16, D 64 or
        128, Hq a multiple of Hk), sequence s the rows cu_seqlens_q[s] ..
        cu_seqlens_q[s+1] over cu_seqlens_k[s] .. cu_seqlens_k[s+1] (int32 [n+1]).
        No rotation and no causal mask; key_mask (int32 [Tk], non-zero = visible)
        hides keys; a row without a visible key is 0; rows of out behind the
        last sequence are left as they were.  max_seqlen_q is the caller's bound
        on the longest query sequence: give it for single tokens (at most
        16 / (Hq / Hk) rows a sequence), which then have a kernel of their own, and
        for short ones (128 / (Hq / Hk)): without it the call counts on one sequence
        of Tq rows (a token of 200 sequences over 500 keys, 12 heads of 64: 125 us
        instead of 61; of 64 over 2000: 81 instead of 76).  scale None: 1 / sqrt(D).
        Rows may be strided (views of fused rows)."""
        # (a bound beyond 32 bits is none; ctypes would cut it to its lower bits)
        max_seqlen_q = max(-1, min(int(max_seqlen_q), _INT_MAX))
        scale = None if scale is None else float(scale)
        key = ("cross", _layout(q, k, v, cu_seqlens_q, cu_seqlens_k), None if out is None else _layout(out),
               None if key_mask is None else _layout(key_mask), max_seqlen_q, scale)
        known = self._known.get(key)
        if known is None:
            for t, name in ((q, "q"), (k, "k"), (v, "v")):
                self._check_cross(t, name, 3)
            if k.shape != v.shape or k.shape[2] != q.shape[2] or not q.dtype == k.dtype == v.dtype:
                raise TypeError("q, k and v must agree in type and head size, k and v in shape")
            self._check_cu(cu_seqlens_q)
            self._check_cu(cu_seqlens_k)
            if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 1:
                raise ValueError("cu_seqlens_q and cu_seqlens_k must name the same number of sequences")
            if out is not None:
                self._check_cross(out, "out", 3)
                if out.shape != q.shape or out.dtype != q.dtype:
                    raise TypeError(f"out must be a {q.dtype} tensor of shape {list(q.shape)}")
            if key_mask is not None and (key_mask.dtype != torch.int32 or tuple(key_mask.shape) != (k.shape[0],)
                                         or key_mask.device != self.device or not key_mask.is_contiguous()):
                raise TypeError(f"key_mask must be a contiguous int32 [{k.shape[0]}] tensor on {self.device}")
            # one row has no pitch that matters, and a new result is contiguous
            width = q.shape[1] * q.shape[2]
            pitches = [t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2] for t in (q, k, v)]
            pitches.append(out.stride(0) if out is not None and out.shape[0] > 1 else width)
            known = self._cross_known(key, q, k, v, out, q.shape[0], k.shape[0], pitches,
                                      cu_seqlens_q.numel() - 1, True, max_seqlen_q, key_mask, scale)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        return self._cross(known, q, k, v, out, cu_seqlens_q, cu_seqlens_k, key_mask)

    def cross_attention_padded(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                               key_mask: torch.Tensor = None, scale: float = None,
                               out: torch.Tensor = None) -> torch.Tensor:
        """The padded form: q [B, Sq, Hq, D] over k and v [B, Sk, Hk, D] with
        key_mask int32 [B, Sk] (1 = real token, 0 = pad; None: all real) ->
        out [B, Sq, Hq, D].  Every query row is computed; one whose keys are all
        pads is 0.  Rows may be strided, with the batch rows one pitch apart
        (views of fused rows).  Else as cross_attention."""
        scale = None if scale is None else float(scale)
        key = ("cross_padded", _layout(q, k, v), None if out is None else _layout(out),
               None if key_mask is None else _layout(key_mask), scale)
        known = self._known.get(key)
        if known is None:
            for t, name in ((q, "q"), (k, "k"), (v, "v")):
                self._check_cross(t, name, 4)
            if (k.shape != v.shape or k.shape[3] != q.shape[3] or k.shape[0] != q.shape[0]
                    or not q.dtype == k.dtype == v.dtype):
                raise TypeError("q, k and v must agree in type, batch and head size, k and v in shape")
            B, Sq, Sk = q.shape[0], q.shape[1], k.shape[1]
            if out is not None:
                self._check_cross(out, "out", 4)
                if out.shape != q.shape or out.dtype != q.dtype:
                    raise TypeError(f"out must be a {q.dtype} tensor of shape {list(q.shape)}")
            if key_mask is not None and (key_mask.dtype != torch.int32 or tuple(key_mask.shape) != (B, Sk)
                                         or key_mask.device != self.device or not key_mask.is_contiguous()):
                raise TypeError(f"key_mask must be a contiguous int32 [{B}, {Sk}] tensor on {self.device}")
            pitches = []
            for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
                if t is None:
                    pitches.append(q.shape[2] * q.shape[3])
                    continue
                pitch = t.stride(1) if t.shape[1] > 1 else t.stride(0) if B > 1 else t.shape[2] * t.shape[3]
                if B > 1 and t.shape[1] > 0 and t.stride(0) != t.shape[1] * pitch:
                    raise ValueError(f"the rows of {name} must be one pitch apart throughout the batch")
                pitches.append(pitch)
            known = self._cross_known(key, q, k, v, out, B * Sq, B * Sk, pitches, B, False, 0, key_mask, scale)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        return self._cross(known, q, k, v, out, None, None, key_mask)

    def _check_rows(self, t, name, dtype, shape):
        """A tensor of that type and shape on this device whose last dimension is contiguous."""
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != self.device:
            raise TypeError(f"{name} must be a {dtype} {list(shape)} tensor on {self.device}")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")

    @staticmethod
    def _pitch(t):
        """Elements from row to row of a [T, D] tensor (one row has no pitch that matters)."""
        return t.stride(0) if t.shape[0] > 1 else t.shape[1]

    def _linear_known(self, key, x, weight, experts, bias, activation, gated, residual, row_scale, out):
        """Check a call's layouts and remember its arguments without pointers."""
        if activation not in _ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, not {activation!r}")
        if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.float16) or x.device != self.device:
            raise TypeError(f"x must be a bf16 or fp16 [T, K] tensor on {self.device}")
        T, K = x.shape
        lead = () if experts is None else (experts,)
        if weight.dim() != 2 + len(lead):
            raise TypeError(f"weight must have the shape {'[N, K]' if experts is None else '[experts, N, K]'}")
        W = weight.shape[-2]
        if gated and W % 2:
            raise ValueError("a gated product's weight has an even number of rows")
        N = W // 2 if gated else W
        if K < 1 or N < 1:
            raise ValueError("weight must have rows and columns")
        self._check_rows(x, "x", x.dtype, (T, K))
        self._check_rows(weight, "weight", x.dtype, lead + (W, K))
        if bias is not None:
            self._check_rows(bias, "bias", x.dtype, lead + (W,))
            if not bias.is_contiguous():
                raise ValueError("bias must be contiguous")
        if residual is not None:
            self._check_rows(residual, "residual", x.dtype, (T, N))
        if row_scale is not None and (row_scale.dtype != torch.float32 or tuple(row_scale.shape) != (T,)
                                      or row_scale.device != self.device or not row_scale.is_contiguous()):
            raise TypeError(f"row_scale must be a contiguous fp32 [{T}] tensor on {self.device}")
        if out is not None:
            self._check_rows(out, "out", x.dtype, (T, N))
        for t, name in ((x, "x"), (weight, "weight")):
            if any(n > 1 and st % 8 for n, st in zip(t.shape[:-1], t.stride()[:-1])):
                raise ValueError(f"the rows of {name} must lie a multiple of 8 elements apart")
        args = LinearArgs(None, None, None, None, None, self._pitch(x), weight.stride(-2) if W > 1 else K,
                          weight.stride(0) if experts is not None and experts > 1 else 0,
                          self._pitch(residual) if residual is not None else 0,
                          self._pitch(out) if out is not None else N, T, K, N, _DTYPES[x.dtype],
                          _ACTIVATIONS[activation], 1 if gated else 0, experts or 0, None, None)
        return self._remember(key, (bytes(args), (T, N)))

    def _linear(self, known, what, x, weight, bias, residual, out, cu=None, row_scale=None):
        template, shape = known
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=self.device)
        args = LinearArgs.from_buffer_copy(template)
        args.x, args.weight, args.out = x.data_ptr(), weight.data_ptr(), out.data_ptr()
        if bias is not None:
            args.bias = bias.data_ptr()
        if residual is not None:
            args.residual = residual.data_ptr()
        if cu is not None:
            args.cu_experts = cu.data_ptr()
        if row_scale is not None:
            args.row_scale = row_scale.data_ptr()
        st = _lib.mbert_attn_linear(self._h, ctypes.byref(args), _stream_of(self.device))
        if st != 0:
            _check(st, what)
        return out

    def linear(self, x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor = None, activation: str = "none",
               gated: bool = False, residual: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
        """out[T, N] = residual + act(x weight^T + bias), for x [T, K] and weight
        [N, K] (bf16 or fp16) of any width; fp32 sums and epilogue, one rounding.
        activation: "none", "gelu" (the erf form), "gelu_tanh", "silu" or "relu".
        gated: weight [2N, K] and bias [2N] hold the activated half first, and
        out = residual + act(x Wg^T + bg) * (x Wu^T + bu).  `out` may be
        `residual` itself.  Rows may be strided; those of x and weight start at
        16-byte boundaries (K a multiple of 8 where they are contiguous)."""
        key = ("linear", activation, bool(gated), _key(x), _key(weight), _key(bias), _key(residual), _key(out))
        known = self._known.get(key)
        if known is None:
            known = self._linear_known(key, x, weight, None, bias, activation, bool(gated), residual, None, out)
        return self._linear(known, "linear", x, weight, bias, residual, out)

    def linear_plan(self, rows: int, inner: int, outer: int, activation: str = "none", gated: bool = False,
                    experts: int = 0):
        """How a product of these sizes runs (experts: of that many groups), for profiles
        and tests: ("many", columns) for the kernel for many rows, in units of 256 rows
        and that many accumulator columns, or ("few", rows of a tile, pieces of that many
        times 32 output columns, CTAs that share the inner dimension)."""
        args = LinearArgs(rows=rows, inner=inner, outer=outer, activation=_ACTIVATIONS[activation],
                          gated=1 if gated else 0, experts=experts)
        plan = (ctypes.c_int32 * 4)()
        _check(load_library().mbert_attn_linear_plan(self._h, ctypes.byref(args), plan), "linear_plan")
        return ("few", *plan[1:]) if plan[0] else ("many", plan[1])

    def expert_linear(self, x: torch.Tensor, weight: torch.Tensor, cu_experts: torch.Tensor,
                      bias: torch.Tensor = None, activation: str = "none", gated: bool = False,
                      row_scale: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
        """linear with a weight for each group of rows: rows cu_experts[e] ..
        cu_experts[e+1] (int32 [E+1]) of x take weight[e] and bias[e] of weight
        [E, N, K] and bias [E, N] ([E, 2N, K] and [E, 2N] gated), and row t's
        result is multiplied by row_scale[t] (fp32, a router's weight).  Empty
        groups are allowed; rows of out behind the last group are left as they
        were.  Experts' weights lie one behind another (padding between them is
        fine, rows of several interleaved are refused)."""
        key = ("expert_linear", activation, bool(gated), _key(x), _key(weight), _key(cu_experts), _key(bias),
               _key(row_scale), _key(out))
        known = self._known.get(key)
        if known is None:
            self._check_cu(cu_experts)
            experts = cu_experts.numel() - 1
            if experts < 1:
                raise ValueError("cu_experts must name at least one expert")
            known = self._linear_known(key, x, weight, experts, bias, activation, bool(gated), None, row_scale, out)
        return self._linear(known, "expert_linear", x, weight, bias, None, out, cu_experts, row_scale)

    def residual_norm(self, x: torch.Tensor, branch: torch.Tensor = None, weight: torch.Tensor = None,
                      bias: torch.Tensor = None, branch_weight: torch.Tensor = None, branch_bias: torch.Tensor = None,
                      gate: torch.Tensor = None, cu_seqlens: torch.Tensor = None, norm: str = "layer",
                      residual_scale: float = 1.0, eps: float = NORM_EPS, h_out: torch.Tensor = None,
                      y_out: torch.Tensor = None):
        """(h, y) = the residual stream behind a block and its norm for the next:
        h = residual_scale x + gate P(branch), y = N(h), over rows of x [T, D]
        (bf16, fp16 or fp32; D up to 16384) in one kernel.  P is the norm with
        branch_weight [D] (None: none) and branch_bias, N that with weight (None:
        no y, None is returned for it) and bias, both "layer" or "rms".  gate:
        [D], [T, D], or with cu_seqlens (int32 [n+1]) [n, D], of the row's
        sequence; rows behind the last sequence are left as they were.  branch
        None: (x, N(x)).  h_out and y_out may each be x or branch.  y is of the
        h that has not been rounded.  Rows may be strided.  A row's bits do not go
        by the rows beside it or by how many there are."""
        if norm not in _NORMS:
            raise ValueError(f"norm must be 'rms' or 'layer', not {norm!r}")
        residual_scale, eps = float(residual_scale), float(eps)
        key = ("residual_norm", norm, residual_scale, eps, _key(x), _key(branch), _key(weight), _key(bias),
               _key(branch_weight), _key(branch_bias), _key(gate), _key(cu_seqlens), _key(h_out), _key(y_out))
        known = self._known.get(key)
        if known is None:
            known = self._residual_norm_known(key, x, branch, weight, bias, branch_weight, branch_bias, gate, cu_seqlens,
                                              h_out, y_out, norm, residual_scale, eps)
        args = ResidualNormArgs.from_buffer_copy(known)
        args.x = x.data_ptr()
        h, y = x, None
        if branch is not None:
            h = torch.empty(x.shape, dtype=x.dtype, device=self.device) if h_out is None else h_out
            args.branch, args.h = branch.data_ptr(), h.data_ptr()
        if weight is not None:
            y = torch.empty(x.shape, dtype=x.dtype, device=self.device) if y_out is None else y_out
            args.weight, args.y = weight.data_ptr(), y.data_ptr()
        if bias is not None:
            args.bias = bias.data_ptr()
        if branch_weight is not None:
            args.branch_weight = branch_weight.data_ptr()
        if branch_bias is not None:
            args.branch_bias = branch_bias.data_ptr()
        if gate is not None:
            args.gate = gate.data_ptr()
        if cu_seqlens is not None:
            args.cu_seqlens = cu_seqlens.data_ptr()
        st = _lib.mbert_attn_residual_norm(self._h, ctypes.byref(args), _stream_of(self.device))
        if st != 0:
            _check(st, "residual_norm")
        return h, y

    def _residual_norm_known(self, key, x, branch, weight, bias, branch_weight, branch_bias, gate, cu_seqlens, h_out,
                             y_out, norm, residual_scale, eps):
        if x.dim() != 2 or x.dtype not in _DTYPES or x.device != self.device:
            raise TypeError(f"x must be a bf16, fp16 or fp32 [T, D] tensor on {self.device}")
        T, D = x.shape
        if branch is None and weight is None:
            raise ValueError("give branch, weight or both")
        if branch is None and (branch_weight is not None or gate is not None or h_out is not None
                               or residual_scale != 1.0):
            raise ValueError("branch_weight, gate, residual_scale and h_out go with a branch")
        for w, b, name in ((weight, bias, "bias"), (branch_weight, branch_bias, "branch_bias")):
            if b is not None and w is None:
                raise ValueError(f"{name} goes with its norm's weight")
        if y_out is not None and weight is None:
            raise ValueError("y_out goes with weight")
        if cu_seqlens is not None and gate is None:
            raise ValueError("cu_seqlens goes with a gate for each sequence")
        for t, name in ((x, "x"), (branch, "branch"), (h_out, "h_out"), (y_out, "y_out")):
            if t is not None:
                self._check_rows(t, name, x.dtype, (T, D))
        for t, name in ((weight, "weight"), (bias, "bias"), (branch_weight, "branch_weight"),
                        (branch_bias, "branch_bias")):
            if t is not None:
                self._check_rows(t, name, x.dtype, (D,))
        kind, n, gate_row = 0, 0, 0
        if gate is not None:
            if cu_seqlens is not None:
                self._check_cu(cu_seqlens)
                n = cu_seqlens.numel() - 1
                if n < 1:
                    raise ValueError("cu_seqlens must name at least one sequence")
                kind, shape = 3, (n, D)
            else:
                kind, shape = (1, (D,)) if gate.dim() == 1 else (2, (T, D))
            self._check_rows(gate, "gate", x.dtype, shape)
            gate_row = self._pitch(gate) if gate.dim() == 2 else D
        args = ResidualNormArgs(*[None] * 9, self._pitch(x), 0 if branch is None else self._pitch(branch), gate_row,
                                D if h_out is None else self._pitch(h_out), D if y_out is None else self._pitch(y_out),
                                T, D, _DTYPES[x.dtype], _NORMS[norm], kind, None, n, residual_scale, eps)
        return self._remember(key, bytes(args))

    def key_counts(self, cu_seqlens: torch.Tensor, total_tokens: int, layer_kind,
                   max_seqlen: int = 0) -> torch.Tensor:
        """int32 [T]: keys the kernels' schedule and mask admit per query row."""
        kind = _kind(layer_kind)
        self._check_cu(cu_seqlens)
        counts = torch.full((int(total_tokens),), -1, dtype=torch.int32, device=self.device)
        st = load_library().mbert_attn_key_counts(
            self._h, cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, int(total_tokens),
            int(max_seqlen), kind, counts.data_ptr(), _stream_ptr(self.device))
        _check(st, "key_counts")
        return counts

    def selftest_timeout(self, limit_us: int = 20000):
        """Enqueue the bounded-wait self-test (sets the timeout status)."""
        _check(load_library().mbert_attn_selftest_timeout(self._h, int(limit_us),
                                                          _stream_ptr(self.device)),
               "selftest_timeout")

    def profile(self, enable: bool = True):
        """Record a CUDA event pair around every attention, projection and norm kernel."""
        _check(load_library().mbert_attn_profile_enable(self._h, 1 if enable else 0), "profile")

    def profile_read(self):
        """-> ({'global', 'local', 'out_proj', 'qkv_proj', 'layernorm', 'mlp_up',
        'mlp_down'} -> summed kernel ms, the same keys -> kernel count,
        total_launches); synchronises and clears the record."""
        keys = ("global", "local", "out_proj", "qkv_proj", "layernorm", "mlp_up", "mlp_down")
        ms = (ctypes.c_double * len(keys))()
        n = (ctypes.c_int64 * len(keys))()
        tot = ctypes.c_int64()
        _check(load_library().mbert_attn_profile_read(self._h, ms, n, ctypes.byref(tot)),
               "profile_read")
        return ({k: ms[i] for i, k in enumerate(keys)}, {k: n[i] for i, k in enumerate(keys)},
                int(tot.value))

    def get_error(self) -> int:
        """Wait for the device (every stream, replayed graphs too), then return
        and clear the device-side status."""
        return int(load_library().mbert_attn_get_error(self._h))


_handles = {}


def _default(device) -> Attention:
    idx = device.index if device.index is not None else torch.cuda.current_device()
    h = _handles.get(idx)
    if h is None:
        h = _handles[idx] = Attention(idx)
    return h


def _of(x) -> Attention:
    """The handle of a tensor's device."""
    idx = x.get_device()
    h = _handles.get(idx)
    if h is None:
        if not x.is_cuda:
            raise ValueError("x must be a CUDA tensor")
        h = _default(x.device)
    return h


def attention(qkv: torch.Tensor, cu_seqlens: torch.Tensor, layer_kind, max_seqlen: int = 0,
              out: torch.Tensor = None) -> torch.Tensor:
    """ModernBERT-base attention for one layer: qkv[T,2304] bf16 (CUDA),
    cu_seqlens int32 [n+1] (CUDA), layer_kind 'global' | 'local' ->
    out[T,768] bf16, enqueued on the current stream."""
    if not qkv.is_cuda:
        raise ValueError("qkv must be a CUDA tensor")
    return _default(qkv.device).forward(qkv, cu_seqlens, layer_kind, max_seqlen, out)


def attention_padded(qkv: torch.Tensor, attention_mask: torch.Tensor, layer_kind,
                     out: torch.Tensor = None) -> torch.Tensor:
    """The attention block for a padded batch: qkv [B, S, 2304] bf16 and
    attention_mask [B, S] int32 (CUDA) -> out [B, S, 768], zeros at pads."""
    if not qkv.is_cuda:
        raise ValueError("qkv must be a CUDA tensor")
    return _default(qkv.device).forward_padded(qkv, attention_mask, layer_kind, out)


def ln_qkv(x: torch.Tensor, norm_w, wqkv: torch.Tensor, eps: float = NORM_EPS,
           out: torch.Tensor = None) -> torch.Tensor:
    """qkv = LayerNorm(x) Wqkv^T (bf16, CUDA tensors; norm_w None on layer 0):
    the step before the attention block."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    return _default(x.device).ln_qkv(x, norm_w, wqkv, eps, out)


def mlp(x: torch.Tensor, norm_w: torch.Tensor, wi: torch.Tensor, wo: torch.Tensor,
        eps: float = NORM_EPS, out: torch.Tensor = None) -> torch.Tensor:
    """y = x + (GELU(g) * u) Wo^T after the MLP's LayerNorm (bf16, CUDA tensors)."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    return _default(x.device).mlp(x, norm_w, wi, wo, eps, out)


def out_proj(a: torch.Tensor, wo: torch.Tensor, x: torch.Tensor, out: torch.Tensor = None) -> torch.Tensor:
    """y = x + a Wo^T (bf16, CUDA tensors): the step after the attention block."""
    if not a.is_cuda:
        raise ValueError("a must be a CUDA tensor")
    return _default(a.device).out_proj(a, wo, x, out=out)


def key_counts(cu_seqlens: torch.Tensor, total_tokens: int, layer_kind) -> torch.Tensor:
    if not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be a CUDA tensor")
    return _default(cu_seqlens.device).key_counts(cu_seqlens, total_tokens, layer_kind)


def rotary(x: torch.Tensor, rope: Rotary, positions: torch.Tensor = None, cu_seqlens: torch.Tensor = None,
           inverse: bool = False, out: torch.Tensor = None) -> torch.Tensor:
    """Rotary positions on x [T, H, D] (CUDA; bf16, fp16 or fp32), positions
    given or from cu_seqlens: Attention.rotary on the device's handle."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    return _default(x.device).rotary(x, rope, positions, cu_seqlens, inverse, out)


def qk_norm_rotary(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                   rope: Rotary = None, positions: torch.Tensor = None, cu_seqlens: torch.Tensor = None,
                   norm: str = "rms", eps: float = 1e-6, q_out: torch.Tensor = None,
                   k_out: torch.Tensor = None):
    """Norm of every query and key head and its rotation in one kernel:
    Attention.qk_norm_rotary on the device's handle."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("give q, k or both")
    if not first.is_cuda:
        raise ValueError("q and k must be CUDA tensors")
    return _default(first.device).qk_norm_rotary(q, k, q_weight, k_weight, rope, positions, cu_seqlens,
                                                 norm, eps, q_out, k_out)


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    cu_seqlens_k: torch.Tensor, max_seqlen_q: int = 0, key_mask: torch.Tensor = None,
                    scale: float = None, out: torch.Tensor = None) -> torch.Tensor:
    """Attention of packed queries over keys and values of another length
    (CUDA, bf16 or fp16): Attention.cross_attention on the device's handle."""
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    return _default(q.device).cross_attention(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, key_mask,
                                              scale, out)


def cross_attention_padded(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, key_mask: torch.Tensor = None,
                           scale: float = None, out: torch.Tensor = None) -> torch.Tensor:
    """The padded form, q [B, Sq, Hq, D] over k and v [B, Sk, Hk, D] with a mask
    [B, Sk]: Attention.cross_attention_padded on the device's handle."""
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    return _default(q.device).cross_attention_padded(q, k, v, key_mask, scale, out)


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor = None, activation: str = "none",
           gated: bool = False, residual: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
    """out = residual + act(x weight^T + bias), or gated, of any width (CUDA, bf16
    or fp16): Attention.linear on the device's handle."""
    return _of(x).linear(x, weight, bias, activation, gated, residual, out)


def expert_linear(x: torch.Tensor, weight: torch.Tensor, cu_experts: torch.Tensor, bias: torch.Tensor = None,
                  activation: str = "none", gated: bool = False, row_scale: torch.Tensor = None,
                  out: torch.Tensor = None) -> torch.Tensor:
    """linear with a weight for each group of rows: Attention.expert_linear on the
    device's handle."""
    return _of(x).expert_linear(x, weight, cu_experts, bias, activation, gated, row_scale, out)


def residual_norm(x: torch.Tensor, branch: torch.Tensor = None, weight: torch.Tensor = None,
                  bias: torch.Tensor = None, branch_weight: torch.Tensor = None, branch_bias: torch.Tensor = None,
                  gate: torch.Tensor = None, cu_seqlens: torch.Tensor = None, norm: str = "layer",
                  residual_scale: float = 1.0, eps: float = NORM_EPS, h_out: torch.Tensor = None,
                  y_out: torch.Tensor = None):
    """(h, y): the residual stream behind a block and its norm for the next one:
    Attention.residual_norm on the device's handle."""
    return _of(x).residual_norm(x, branch, weight, bias, branch_weight, branch_bias, gate, cu_seqlens,
                                norm, residual_scale, eps, h_out, y_out)
