"""Thin ctypes binding of the C ABI in include/esm_encoder.h.

Argument marshalling only: every step of the forward runs in the CUDA library.  torch is
used for device memory and streams.  Loading fails loudly when the library has not been
built; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Sequence

import numpy as np


class _Torch:
    """Stands for torch until its first use, which imports it: the ctypes side needs none."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libesm_encoder.so")

ESM_OK = 0
STATUS_NAMES = {0: "ESM_OK", 1: "ESM_ERR_INVALID_ARG", 2: "ESM_ERR_UNSUPPORTED", 3: "ESM_ERR_BAD_CU_SEQLENS",
                4: "ESM_ERR_TOKEN_RANGE", 5: "ESM_ERR_WORKSPACE", 6: "ESM_ERR_CUDA", 7: "ESM_ERR_TIMEOUT"}
PRECISIONS = {"fp32": 0, "bf16": 1, "fp8": 2, "fp4": 3}
EPILOGUES = {"bias_f32": 0, "qkv_rope": 1, "residual": 2, "gelu": 3}

# Every symbol the header declares (checked by the tests).
EXPORTS = ("esm_encoder_create", "esm_encoder_destroy", "esm_encoder_workspace_size", "esm_encoder_forward",
           "esm_encoder_forward_host", "esm_encoder_forward_padded", "esm_encoder_check",
           "esm_encoder_debug_pack_index", "esm_op_layernorm", "esm_op_gemm", "esm_op_attention",
           "esm_encoder_get_fp8_state", "esm_encoder_set_fp8_state", "esm_encoder_set_profiling",
           "esm_encoder_get_profile", "esm_op_attention_noalloc", "esm_op_layernorm_e4m3", "esm_op_gemm_fp8",
           "esm_encoder_debug_wait_timeout", "esm_encoder_lm_head_workspace_size", "esm_encoder_lm_head",
           "esm_encoder_set_layer_precision",
           "esm_encoder_train_buffer_size", "esm_encoder_forward_train", "esm_encoder_backward",
           "esm_op_gemm_dgrad", "esm_op_gemm_wgrad_workspace_size", "esm_op_gemm_wgrad",
           "esm_op_layernorm_backward_workspace_size", "esm_op_layernorm_backward", "esm_op_attention_train",
           "esm_op_attention_backward_workspace_size", "esm_op_attention_backward",
           "esm_encoder_lm_head_backward_workspace_size", "esm_encoder_lm_head_backward",
           "esm_op_quantize_nvfp4", "esm_op_gemm_nvfp4", "esm_encoder_get_fp4_scales", "esm_status_string",
           "esm_encoder_set_attention_window", "esm_op_attention_window_workspace_size", "esm_op_attention_window",
           "esm_op_attention_window_backward", "esm_op_distill_loss_workspace_size", "esm_op_distill_loss",
           "esm_op_distill_loss_backward", "esm_encoder_lm_head_distill_backward", "esm_op_dropout", "esm_op_embed",
           "esm_op_embed_backward_workspace_size", "esm_op_embed_backward", "esm_op_block_norm",
           "esm_op_block_norm_backward_workspace_size", "esm_op_block_norm_backward", "esm_encoder_set_dropout")
STREAM_MAX = 1 << 30  # ESM_STREAM_MAX
DISTILL_MAX = 1 << 30  # ESM_DISTILL_MAX
PROFILE_CLASSES = ("gemm_qkv", "attention", "gemm_oproj", "gemm_fc1", "gemm_fc2", "layernorm", "other",
                   "gemm_backward")


class EsmError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class EsmConfig(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int), ("hidden", ctypes.c_int), ("heads", ctypes.c_int),
                ("ffn", ctypes.c_int), ("vocab", ctypes.c_int), ("max_positions", ctypes.c_int),
                ("ln_eps", ctypes.c_float), ("rope_base", ctypes.c_float), ("emb_scale", ctypes.c_float),
                ("final_ln", ctypes.c_int), ("precision", ctypes.c_int), ("amax_history_len", ctypes.c_int)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class EsmProfile(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * 8), ("launches", ctypes.c_longlong * 8), ("total_launches", ctypes.c_longlong)]


class EsmWeights(ctypes.Structure):
    _fields_ = [("emb", ctypes.c_void_p)] + \
        [(n, _PP) for n in ("ln1_g", "ln1_b", "w_qkv", "b_qkv", "w_o", "b_o", "ln2_g", "ln2_b",
                            "w_1", "b_1", "w_2", "b_2")] + \
        [("lnf_g", ctypes.c_void_p), ("lnf_b", ctypes.c_void_p)]


_PF = ctypes.POINTER(ctypes.c_void_p)
GRAD_NAMES = ("ln1_g", "ln1_b", "w_qkv", "b_qkv", "w_o", "b_o", "ln2_g", "ln2_b", "w_1", "b_1", "w_2", "b_2")


class EsmGrads(ctypes.Structure):
    _fields_ = [("emb", ctypes.c_void_p)] + [(n, _PF) for n in GRAD_NAMES] + \
        [("lnf_g", ctypes.c_void_p), ("lnf_b", ctypes.c_void_p)]


class EsmAttnWindow(ctypes.Structure):
    _fields_ = [("left", ctypes.c_int), ("right", ctypes.c_int), ("sinks", ctypes.c_int)]


LM_HEAD_NAMES = ("dense_w", "dense_b", "ln_g", "ln_b", "emb", "bias")


class EsmLmHead(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LM_HEAD_NAMES]


class EsmLmHeadGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LM_HEAD_NAMES]


class EsmDropout(ctypes.Structure):
    _fields_ = [("rng", ctypes.c_void_p), ("offset", ctypes.c_int64), ("p", ctypes.c_double)]


_PD = ctypes.POINTER(EsmDropout)
NORM_KINDS = {"layer": 0, "rms": 1}
BLOCK_NORM_PARAMS = ("post_gamma", "post_beta", "pre_gamma", "pre_beta")


class EsmBlockNorm(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("residual_scale", ctypes.c_float)] + \
        [(n, ctypes.c_void_p) for n in BLOCK_NORM_PARAMS]


class EsmBlockNormGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in BLOCK_NORM_PARAMS + ("gate",)]


_lib = None


def load_library() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run python -m transformer_esm_layer_gb300.build)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    i64, f32 = ctypes.c_longlong, ctypes.c_float
    sig = {
        "esm_encoder_create": (i32, [ctypes.POINTER(EsmConfig), ctypes.POINTER(vp)]),
        "esm_encoder_destroy": (None, [vp]),
        "esm_encoder_workspace_size": (i32, [vp, i32, i32, ctypes.POINTER(sz)]),
        "esm_encoder_forward": (i32, [vp, ctypes.POINTER(EsmWeights), vp, vp, i32, i32, i32, vp, vp, sz, vp]),
        "esm_encoder_forward_host": (i32, [vp, ctypes.POINTER(EsmWeights), vp, vp, i32, i32, i32, vp, vp, sz, vp]),
        "esm_encoder_forward_padded": (i32, [vp, ctypes.POINTER(EsmWeights), vp, vp, i32, i32, vp, vp, sz, vp]),
        "esm_encoder_check": (i32, [vp, vp]),
        "esm_encoder_set_layer_precision": (i32, [vp, ctypes.POINTER(ctypes.c_int), i32]),
        "esm_encoder_lm_head_workspace_size": (i32, [vp, i32, ctypes.POINTER(sz)]),
        "esm_encoder_lm_head": (i32, [vp, ctypes.POINTER(EsmLmHead), vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "esm_encoder_debug_pack_index": (i32, [vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]),
        "esm_op_layernorm": (i32, [vp, vp, vp, vp, vp, i32, i32, vp]),
        "esm_op_gemm": (i32, [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, vp]),
        "esm_op_attention": (i32, [vp, vp, vp, i32, i32, i32, vp, vp, sz, vp]),
        "esm_encoder_get_fp8_state": (i32, [vp, ctypes.POINTER(ctypes.c_float), sz]),
        "esm_encoder_set_fp8_state": (i32, [vp, ctypes.POINTER(ctypes.c_float), sz]),
        "esm_encoder_set_profiling": (i32, [vp, i32]),
        "esm_encoder_get_profile": (i32, [vp, ctypes.POINTER(EsmProfile), i32]),
        "esm_op_attention_noalloc": (i32, [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]),
        "esm_op_quantize_nvfp4": (i32, [vp, vp, i32, i32, vp, vp, vp, vp, vp]),
        "esm_encoder_get_fp4_scales": (i32, [vp, ctypes.POINTER(ctypes.c_float), sz]),
        "esm_op_gemm_nvfp4": (i32, [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp]),
        "esm_op_layernorm_e4m3": (i32, [vp, vp, vp, vp, vp, i32, i32, vp, vp, vp]),
        "esm_encoder_debug_wait_timeout": (i32, [vp, i32, vp]),
        "esm_op_gemm_fp8": (i32, [vp, i32, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp]),
        "esm_status_string": (ctypes.c_char_p, [i32]),
        "esm_encoder_train_buffer_size": (i32, [vp, i32, ctypes.POINTER(sz)]),
        "esm_encoder_forward_train": (i32, [vp, ctypes.POINTER(EsmWeights), vp, vp, i32, i32, i32, vp, vp, sz, vp, sz,
                                            vp]),
        "esm_encoder_backward": (i32, [vp, ctypes.POINTER(EsmWeights), vp, ctypes.POINTER(EsmGrads), vp, sz, vp, sz,
                                       vp]),
        "esm_op_gemm_dgrad": (i32, [vp, vp, vp, vp, i32, i32, i32, i32, vp]),
        "esm_op_gemm_wgrad_workspace_size": (i32, [vp, i32, i32, ctypes.POINTER(sz)]),
        "esm_op_gemm_wgrad": (i32, [vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]),
        "esm_op_layernorm_backward_workspace_size": (i32, [vp, i32, i32, ctypes.POINTER(sz)]),
        "esm_op_layernorm_backward": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, sz, vp]),
        "esm_op_attention_train": (i32, [vp, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]),
        "esm_op_attention_backward_workspace_size": (i32, [vp, i32, i32, ctypes.POINTER(sz)]),
        "esm_op_attention_backward": (i32, [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, sz, vp]),
        "esm_encoder_lm_head_backward_workspace_size": (i32, [vp, i32, ctypes.POINTER(sz)]),
        "esm_encoder_lm_head_backward": (i32, [vp, ctypes.POINTER(EsmLmHead), vp, i32, vp, vp,
                                               ctypes.POINTER(EsmLmHeadGrads), vp, vp, vp, vp, sz, vp]),
        "esm_encoder_lm_head_distill_backward": (i32, [vp, ctypes.POINTER(EsmLmHead), vp, i32, vp, vp, i32, f32, vp,
                                                       ctypes.POINTER(EsmLmHeadGrads), vp, vp, vp, vp, sz, vp]),
        "esm_encoder_set_attention_window": (i32, [vp, ctypes.POINTER(EsmAttnWindow)]),
        "esm_op_attention_window_workspace_size": (i32, [vp, i32, i32, ctypes.POINTER(EsmAttnWindow), i32,
                                                         ctypes.POINTER(sz)]),
        "esm_op_attention_window": (i32, [vp, vp, vp, i32, i32, i32, ctypes.POINTER(EsmAttnWindow), vp, vp, vp, sz,
                                          vp]),
        "esm_op_attention_window_backward": (i32, [vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                                   ctypes.POINTER(EsmAttnWindow), vp, vp, sz, vp]),
        "esm_op_distill_loss_workspace_size": (i32, [vp, i32, i32, ctypes.POINTER(sz)]),
        "esm_op_distill_loss": (i32, [vp, vp, i32, i64, vp, vp, i32, i32, i32, f32, vp, vp, vp, vp, vp, sz, vp]),
        "esm_op_distill_loss_backward": (i32, [vp, vp, i32, i64, vp, vp, i32, i32, i32, f32, vp, vp, vp, i64, vp]),
        "esm_encoder_set_dropout": (i32, [vp, _PD]),
        "esm_op_dropout": (i32, [vp, vp, i32, i64, vp, i64, vp, i32, i64, i32, i32, _PD, vp]),
        "esm_op_embed": (i32, [vp, vp, i32, vp, i32, i32, i32, f32, vp, _PD, vp, i32, i64, vp]),
        "esm_op_embed_backward_workspace_size": (i32, [vp, i32, i32, i32, ctypes.POINTER(sz)]),
        "esm_op_embed_backward": (i32, [vp, vp, i32, vp, i32, i64, f32, vp, _PD, vp, i32, i32, i32, vp, sz, vp]),
        "esm_op_block_norm": (i32, [vp, ctypes.POINTER(EsmBlockNorm), vp, i32, _PD, vp, vp, vp, vp, vp, i32, i32, vp]),
        "esm_op_block_norm_backward_workspace_size": (i32, [vp, i32, i32, ctypes.POINTER(sz)]),
        "esm_op_block_norm_backward": (i32, [vp, ctypes.POINTER(EsmBlockNorm), vp, i32, _PD, vp, vp, vp, vp, vp, vp,
                                             vp, ctypes.POINTER(EsmBlockNormGrads), i32, i32, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


def _refuse(where: str, what: str):
    raise ValueError(f"{where}: {what}")


def _need(ok, where: str, what: str):
    """Arguments the C side cannot check (it sees only addresses)."""
    if not ok:
        _refuse(where, what)


def _check_tensor(t, where: str, name: str, dtype, shape, device):
    """A contiguous tensor of this type and shape (a tuple, or None for any) on this CUDA device.

    One expression decides and the message is put together only for a refusal: an operator of a
    few microseconds has several tensors to check in every call."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_cuda
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return
    _need(isinstance(t, torch.Tensor) and t.is_cuda, where, f"{name} must be a CUDA tensor")
    _need(t.device == device, where, f"{name} must be on {device}")
    _need(t.dtype == dtype, where, f"{name} must be {dtype}")
    _need(shape is None or t.shape == shape, where, f"{name} must be {shape and list(shape)}")
    _refuse(where, f"{name} must be contiguous")


def _check_scalar(t, where: str, name: str, dtype, device):
    _check_tensor(t, where, name, dtype, None, device)
    if t.numel() != 1:
        _refuse(where, f"{name} must hold one value")


def _launch_stream(where: str, stream, device) -> Optional[int]:
    """The stream of a launch on `device`'s tensors: the current one unless given.  The kernels run
    on the current device, so that must be the tensors'."""
    if torch.cuda.current_device() != device.index:
        _refuse(where, f"the tensors' device {device} must be the current one")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index) or None
    _need(stream.device == device, where, "stream must be on the tensors' device")
    return stream.cuda_stream or None


def _allocating(stream):
    """Context for what a call allocates itself: memory of the launch stream, so that neither its
    last use (on another stream, perhaps still running) nor its next one overlaps this call's."""
    return torch.cuda.stream(stream)


def _check_workspace(t, where: str, device):
    if not (isinstance(t, torch.Tensor) and t.device == device and t.is_contiguous()):
        _refuse(where, f"workspace must be a contiguous tensor on {device}")


def _c_int(where: str, name: str, value) -> int:
    """A whole number that fits the library's int (ctypes keeps the low 32 bits of any other)."""
    if type(value) is int and -2 ** 31 <= value < 2 ** 31:
        return value
    n = int(value)
    if n != value or not -2 ** 31 <= n < 2 ** 31:
        _refuse(where, f"{name} must be a 32-bit whole number, not {value}")
    return n


def _window_struct(window) -> EsmAttnWindow:
    left, right, sinks = window
    return EsmAttnWindow(_c_int("window", "left", left), _c_int("window", "right", right),
                         _c_int("window", "sinks", sinks))


class DeviceWeights:
    """Weights on the device in the handle's parameter dtype, plus the esm_weights struct.

    ``w`` is the dict returned by synth.model_weights (float32 arrays)."""

    def __init__(self, w: Dict, precision: str, device="cuda"):
        dt = torch.float32 if precision == "fp32" else torch.bfloat16
        to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device=device, dtype=dt)
        self.emb = to(w["emb"])
        self.layers = [{k: to(v) for k, v in wl.items()} for wl in w["layers"]]
        self.lnf_g = to(w["lnf_g"])
        self.lnf_b = to(w["lnf_b"])
        self._keep = []
        n = len(self.layers)
        st = EsmWeights()
        st.emb = self.emb.data_ptr()
        for name in ("ln1_g", "ln1_b", "w_qkv", "b_qkv", "w_o", "b_o", "ln2_g", "ln2_b", "w_1", "b_1", "w_2", "b_2"):
            arr = (ctypes.c_void_p * max(n, 1))(*[l[name].data_ptr() for l in self.layers])
            self._keep.append(arr)
            setattr(st, name, ctypes.cast(arr, _PP))
        st.lnf_g = self.lnf_g.data_ptr()
        st.lnf_b = self.lnf_b.data_ptr()
        self.struct = st


class DeviceGrads:
    """float32 gradient buffers on the device, shaped like the weights, plus the esm_grads
    struct (esm_encoder_backward overwrites them)."""

    def __init__(self, g, num_layers: int, device="cuda"):
        z = lambda *shape: torch.empty(*shape, dtype=torch.float32, device=device)
        d, f = g.hidden, g.ffn
        shapes = {"ln1_g": (d,), "ln1_b": (d,), "w_qkv": (3 * d, d), "b_qkv": (3 * d,), "w_o": (d, d), "b_o": (d,),
                  "ln2_g": (d,), "ln2_b": (d,), "w_1": (f, d), "b_1": (f,), "w_2": (d, f), "b_2": (d,)}
        self.emb = z(g.vocab, d)
        self.layers = [{k: z(*s) for k, s in shapes.items()} for _ in range(num_layers)]
        self.lnf_g = z(d)
        self.lnf_b = z(d)
        self._keep = []
        st = EsmGrads()
        st.emb = self.emb.data_ptr()
        for name in GRAD_NAMES:
            arr = (ctypes.c_void_p * max(num_layers, 1))(*[l[name].data_ptr() for l in self.layers])
            self._keep.append(arr)
            setattr(st, name, ctypes.cast(arr, _PF))
        st.lnf_g = self.lnf_g.data_ptr()
        st.lnf_b = self.lnf_b.data_ptr()
        self.struct = st

    def tensors(self):
        """Every gradient tensor in a fixed order (embedding, layers, final LayerNorm)."""
        return [self.emb] + [l[n] for l in self.layers for n in GRAD_NAMES] + [self.lnf_g, self.lnf_b]


class DeviceLmHead:
    """Masked-LM head weights on the device (handle's parameter dtype) plus the esm_lm_head
    struct; ``w`` is the dict of synth.lm_head_weights (its "emb" is the tied embedding)."""

    def __init__(self, w: Dict, precision: str, device="cuda"):
        dt = torch.float32 if precision == "fp32" else torch.bfloat16
        to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device=device, dtype=dt)
        self.t = {k: to(w[k]) for k in ("dense_w", "dense_b", "ln_g", "ln_b", "emb", "bias")}
        self.struct = EsmLmHead(*[self.t[k].data_ptr() for k in ("dense_w", "dense_b", "ln_g", "ln_b", "emb", "bias")])


class _Frozen:
    """Objects whose C struct is made once: a later change of an attribute would not reach it."""

    __slots__ = ()

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__} cannot be changed: make another")

    def _set(self, **values):
        for name, value in values.items():
            object.__setattr__(self, name, value)


class Dropout(_Frozen):
    """A dropout of probability p whose mask is drawn from (seed, base + offset) and never stored.

    ``rng``: int64 CUDA tensor (seed, base), read when a kernel runs: a training program adds to the
    base every step (in place, on the device), and captured graphs see it.  ``offset`` tells the
    dropouts of one step apart: give the same object to a forward call and its backward, another one
    to every other dropout, and let the base move past all offsets of a step."""

    __slots__ = ("p", "rng", "offset", "device", "struct")

    def __init__(self, p: float, rng, offset: int = 0):
        where = "Dropout"
        _need(isinstance(rng, torch.Tensor) and rng.is_cuda, where, "rng must be a CUDA tensor")
        _check_tensor(rng, where, "rng", torch.int64, (2,), rng.device)
        p, offset = float(p), int(offset)
        _need(0.0 <= p <= 1.0, where, f"p must be in [0, 1], not {p}")
        _need(-2 ** 63 <= offset < 2 ** 63, where, "offset must be a 64-bit whole number")
        self._set(p=p, rng=rng, offset=offset, device=rng.device, struct=EsmDropout(rng.data_ptr(), offset, p))


class BlockNorm(_Frozen):
    """The norms on both sides of a block and the scale of the residual they are added to (the
    arguments of EsmEncoder.op_block_norm that a model keeps): kind "layer" or "rms"; gammas and betas
    [cols] of the handle's parameter dtype, a gamma of None for no norm, a beta of None for none."""

    __slots__ = ("kind", "residual_scale", "cols", "dtype", "device", "struct") + BLOCK_NORM_PARAMS

    def __init__(self, kind: str = "layer", post_gamma=None, post_beta=None, pre_gamma=None, pre_beta=None,
                 residual_scale: float = 1.0):
        where = "BlockNorm"
        _need(kind in NORM_KINDS, where, f"kind must be one of {sorted(NORM_KINDS)}")
        given = dict(post_gamma=post_gamma, post_beta=post_beta, pre_gamma=pre_gamma, pre_beta=pre_beta)
        for norm in ("post", "pre"):
            _need(given[norm + "_gamma"] is not None or given[norm + "_beta"] is None, where,
                  f"{norm}_beta needs {norm}_gamma")
        first = next((t for t in given.values() if t is not None), None)
        cols = dtype = device = None
        if first is not None:
            _need(isinstance(first, torch.Tensor) and first.dim() == 1, where, "parameters must be 1-D tensors")
            _need(first.dtype in (torch.float32, torch.bfloat16), where, "parameters must be float32 or bfloat16")
            cols, dtype, device = first.shape[0], first.dtype, first.device
            for name, t in given.items():
                if t is not None:
                    _check_tensor(t, where, name, dtype, (cols,), device)
        scale = float(residual_scale)
        self._set(kind=kind, residual_scale=scale, cols=cols, dtype=dtype, device=device,
                  struct=EsmBlockNorm(NORM_KINDS[kind], scale, *[_ptr(given[n]) for n in BLOCK_NORM_PARAMS]), **given)


class EsmEncoder:
    """One esm_encoder handle (the esm_encoder_* calls with their own names)."""

    def __init__(self, num_layers: int, hidden: int, heads: int, ffn: int, vocab: int = 33,
                 max_positions: int = 1026, precision: str = "bf16", final_ln: bool = True,
                 ln_eps: float = 1e-5, rope_base: float = 10000.0, emb_scale: float = 1.0,
                 amax_history_len: int = 16):
        self.lib = load_library()
        self.cfg = EsmConfig(num_layers, hidden, heads, ffn, vocab, max_positions, ln_eps, rope_base, emb_scale,
                             int(final_ln), PRECISIONS[precision], amax_history_len)
        self.precision = precision
        self.hidden = hidden
        self.num_layers = num_layers
        self.amax_history_len = amax_history_len
        h = ctypes.c_void_p()
        self._raise(self.lib.esm_encoder_create(ctypes.byref(self.cfg), ctypes.byref(h)), "esm_encoder_create")
        self.handle = h

    @classmethod
    def from_geometry(cls, g, precision: str, final_ln: bool = True, **kw):
        return cls(g.num_layers, g.hidden, g.heads, g.ffn, g.vocab, g.max_positions, precision, final_ln, **kw)

    @staticmethod
    def _raise(st: int, where: str):
        if st != ESM_OK:
            raise EsmError(st, where)

    def close(self):
        if getattr(self, "handle", None):
            self.lib.esm_encoder_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ buffers
    @property
    def out_dtype(self):
        return torch.float32 if self.precision == "fp32" else torch.bfloat16

    def workspace_size(self, max_tokens: int, max_seqs: int) -> int:
        n = ctypes.c_size_t()
        self._raise(self.lib.esm_encoder_workspace_size(self.handle, max_tokens, max_seqs, ctypes.byref(n)),
                    "esm_encoder_workspace_size")
        return n.value

    def workspace(self, max_tokens: int, max_seqs: int, device="cuda"):
        return torch.empty(self.workspace_size(max_tokens, max_seqs), dtype=torch.uint8, device=device)

    # ------------------------------------------------------------------ calls
    def forward(self, weights: DeviceWeights, token_ids, cu_seqlens, max_seqlen: int, out=None, workspace=None,
                stream=None, check: bool = False):
        T = token_ids.numel()
        B = cu_seqlens.numel() - 1
        if out is None:
            out = torch.empty(T, self.hidden, dtype=self.out_dtype, device=token_ids.device)
        if workspace is None:
            workspace = self.workspace(T, B, token_ids.device)
        st = self.lib.esm_encoder_forward(self.handle, ctypes.byref(weights.struct), _ptr(token_ids),
                                          _ptr(cu_seqlens), B, T, int(max_seqlen), _ptr(out), _ptr(workspace),
                                          workspace.numel(), _stream_ptr(stream))
        self._raise(st, "esm_encoder_forward")
        if check:
            self.check(stream)
        return out

    def forward_host(self, weights: DeviceWeights, token_ids: np.ndarray, cu_seqlens: np.ndarray, max_seqlen: int,
                     out: np.ndarray, workspace, stream=None):
        """Host buffers in and out (numpy arrays, or pinned torch CPU tensors via .numpy())."""
        T = int(token_ids.size)
        B = int(cu_seqlens.size) - 1
        st = self.lib.esm_encoder_forward_host(self.handle, ctypes.byref(weights.struct),
                                               token_ids.ctypes.data, cu_seqlens.ctypes.data, B, T, int(max_seqlen),
                                               out.ctypes.data, _ptr(workspace), workspace.numel(),
                                               _stream_ptr(stream))
        self._raise(st, "esm_encoder_forward_host")
        return out

    def forward_padded(self, weights: DeviceWeights, token_ids, seq_lens, out=None, workspace=None, stream=None,
                       check: bool = False):
        B, S = token_ids.shape
        if out is None:
            out = torch.empty(B, S, self.hidden, dtype=self.out_dtype, device=token_ids.device)
        if workspace is None:
            workspace = self.workspace(B * S, B, token_ids.device)
        st = self.lib.esm_encoder_forward_padded(self.handle, ctypes.byref(weights.struct), _ptr(token_ids),
                                                 _ptr(seq_lens), B, S, _ptr(out), _ptr(workspace), workspace.numel(),
                                                 _stream_ptr(stream))
        self._raise(st, "esm_encoder_forward_padded")
        if check:
            self.check(stream)
        return out

    def check(self, stream=None) -> int:
        st = self.lib.esm_encoder_check(self.handle, _stream_ptr(stream))
        self._raise(st, "esm_encoder_check")
        return st

    def check_status(self, stream=None) -> int:
        """Like check() but returns the status instead of raising."""
        return self.lib.esm_encoder_check(self.handle, _stream_ptr(stream))

    def debug_pack_index(self, cu_seqlens, total_tokens: int, max_seqlen: int, workspace=None, stream=None):
        B = cu_seqlens.numel() - 1
        pos = torch.empty(max(total_tokens, 1), dtype=torch.int32, device=cu_seqlens.device)
        seg = torch.empty_like(pos)
        if workspace is None:
            workspace = self.workspace(total_tokens, B, cu_seqlens.device)
        st = self.lib.esm_encoder_debug_pack_index(self.handle, _ptr(cu_seqlens), B, total_tokens, int(max_seqlen),
                                                   _ptr(pos), _ptr(seg), _ptr(workspace), workspace.numel(),
                                                   _stream_ptr(stream))
        self._raise(st, "esm_encoder_debug_pack_index")
        return pos[:total_tokens], seg[:total_tokens]

    def debug_wait_timeout(self, timeout_us: int, stream=None):
        self._raise(self.lib.esm_encoder_debug_wait_timeout(self.handle, int(timeout_us), _stream_ptr(stream)),
                    "esm_encoder_debug_wait_timeout")

    def op_layernorm(self, x, gamma, beta, y, stream=None):
        rows, cols = x.shape
        self._raise(self.lib.esm_op_layernorm(self.handle, _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), rows, cols,
                                              _stream_ptr(stream)), "esm_op_layernorm")
        return y

    def op_gemm(self, epi: str, A, B, bias, out, pos_id=None, stream=None):
        M, K = A.shape
        N = B.shape[0]
        self._raise(self.lib.esm_op_gemm(self.handle, EPILOGUES[epi], _ptr(A), _ptr(B), _ptr(bias), _ptr(out),
                                         _ptr(pos_id), M, N, K, _stream_ptr(stream)), "esm_op_gemm")
        return out

    def op_layernorm_e4m3(self, x, gamma, beta, y, scale, amax, stream=None):
        rows, cols = x.shape
        self._raise(self.lib.esm_op_layernorm_e4m3(self.handle, _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), rows, cols,
                                                   _ptr(scale), _ptr(amax), _stream_ptr(stream)),
                    "esm_op_layernorm_e4m3")
        return y

    def op_gemm_fp8(self, epi: str, A, B, a_scale, b_scale, bias, out, pos_id=None, stream=None):
        M, K = A.shape
        N = B.shape[0]
        self._raise(self.lib.esm_op_gemm_fp8(self.handle, EPILOGUES[epi], _ptr(A), _ptr(B), _ptr(a_scale),
                                             _ptr(b_scale), _ptr(bias), _ptr(out), _ptr(pos_id), M, N, K,
                                             _stream_ptr(stream)), "esm_op_gemm_fp8")
        return out

    def op_attention(self, qkv, cu_seqlens, max_seqlen: int, o, workspace=None, stream=None):
        T = qkv.shape[0]
        B = cu_seqlens.numel() - 1
        if workspace is None:
            workspace = self.workspace(T, B, qkv.device)
        self._raise(self.lib.esm_op_attention(self.handle, _ptr(qkv), _ptr(cu_seqlens), B, T, int(max_seqlen),
                                              _ptr(o), _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
                    "esm_op_attention")
        return o

    # ------------------------------------------------------------------ windowed attention
    def set_attention_window(self, window=None):
        """esm_encoder_set_attention_window: (left, right, sinks) for every layer, -1 = unlimited;
        None restores full attention.  Set it before train_buffer()."""
        w = None if window is None else ctypes.byref(_window_struct(window))
        self._raise(self.lib.esm_encoder_set_attention_window(self.handle, w), "esm_encoder_set_attention_window")

    def op_attention_window_workspace(self, T: int, B: int, window, backward: bool = False, device="cuda"):
        n = ctypes.c_size_t()
        self._raise(self.lib.esm_op_attention_window_workspace_size(self.handle, T, B,
                                                                    ctypes.byref(_window_struct(window)),
                                                                    int(backward), ctypes.byref(n)),
                    "esm_op_attention_window_workspace_size")
        return torch.empty(int(n.value), dtype=torch.uint8, device=device)

    def _check_packed(self, where: str, qkv, cu_seqlens):
        """q | k | v and offsets of a packed batch; returns its tokens and sequences."""
        _need(isinstance(qkv, torch.Tensor) and qkv.dim() == 2, where, "qkv must be a 2-D tensor")
        T = qkv.shape[0]
        _check_tensor(qkv, where, "qkv", self.out_dtype, (T, 3 * self.hidden), qkv.device)
        _check_tensor(cu_seqlens, where, "cu_seqlens", torch.int32, None, qkv.device)
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2, where, "cu_seqlens must hold at least two offsets")
        return T, cu_seqlens.numel() - 1

    def op_attention_window(self, qkv, cu_seqlens, max_seqlen: int, window, o, lse=None, workspace=None, stream=None):
        """esm_op_attention_window: attention of packed q | k | v [T, 3*hidden] under a window
        (left, right, sinks), -1 = unlimited: query i sees key j of its sequence if j <= i + right
        and (j >= i - left or j < sinks).  Writes o [T, hidden] and, if given, lse float32 [heads, T]."""
        where = "op_attention_window"
        T, B = self._check_packed(where, qkv, cu_seqlens)
        dev = qkv.device
        _check_tensor(o, where, "o", qkv.dtype, (T, self.hidden), dev)
        if lse is not None:
            _check_tensor(lse, where, "lse", torch.float32, (self.cfg.heads, T), dev)
        st = _launch_stream(where, stream, dev)
        if workspace is None:
            with _allocating(stream):
                workspace = self.op_attention_window_workspace(T, B, window, device=dev)
        _check_workspace(workspace, where, dev)
        self._raise(self.lib.esm_op_attention_window(self.handle, qkv.data_ptr(), cu_seqlens.data_ptr(), B, T,
                                                     _c_int(where, "max_seqlen", max_seqlen),
                                                     ctypes.byref(_window_struct(window)), o.data_ptr(), _ptr(lse),
                                                     workspace.data_ptr(), workspace.nbytes, st),
                    "esm_op_attention_window")
        return o

    def op_attention_window_backward(self, qkv, o, lse, d_o, cu_seqlens, max_seqlen: int, window, dqkv,
                                     workspace=None, stream=None):
        """esm_op_attention_window_backward: dqkv [T, 3*hidden] (bf16) from the forward's qkv, o and
        lse under the same window and d_o = dL/do."""
        where = "op_attention_window_backward"
        T, B = self._check_packed(where, qkv, cu_seqlens)
        dev, hidden = qkv.device, (T, self.hidden)
        _check_tensor(o, where, "o", torch.bfloat16, hidden, dev)
        _check_tensor(d_o, where, "d_o", torch.bfloat16, hidden, dev)
        _check_tensor(lse, where, "lse", torch.float32, (self.cfg.heads, T), dev)
        _check_tensor(dqkv, where, "dqkv", torch.bfloat16, (T, 3 * self.hidden), dev)
        st = _launch_stream(where, stream, dev)
        if workspace is None:
            with _allocating(stream):
                workspace = self.op_attention_window_workspace(T, B, window, backward=True, device=dev)
        _check_workspace(workspace, where, dev)
        self._raise(self.lib.esm_op_attention_window_backward(self.handle, qkv.data_ptr(), o.data_ptr(),
                                                              lse.data_ptr(), d_o.data_ptr(), cu_seqlens.data_ptr(),
                                                              B, T, _c_int(where, "max_seqlen", max_seqlen),
                                                              ctypes.byref(_window_struct(window)), dqkv.data_ptr(),
                                                              workspace.data_ptr(), workspace.nbytes, st),
                    "esm_op_attention_window_backward")
        return dqkv

    # ------------------------------------------------------------------ distillation
    def op_distill_loss_workspace(self, T: int, vocab: int, device="cuda"):
        n = ctypes.c_size_t()
        self._raise(self.lib.esm_op_distill_loss_workspace_size(self.handle, T, vocab, ctypes.byref(n)),
                    "esm_op_distill_loss_workspace_size")
        return torch.empty(int(n.value), dtype=torch.uint8, device=device)

    @staticmethod
    def _check_distill(where: str, logits, teacher_ids, teacher_logits):
        """Logits and teacher entries; returns the logits' esm_precision, rows, columns, row stride
        (a single row may report any stride) and the entries per row."""
        _need(isinstance(logits, torch.Tensor) and logits.is_cuda, where, "logits must be a CUDA tensor")
        f32 = logits.dtype is torch.float32
        _need(f32 or logits.dtype is torch.bfloat16, where, "logits must be float32 or bfloat16")
        shape, stride = logits.shape, logits.stride()
        _need(len(shape) == 2 and (stride[1] == 1 or shape[1] == 1), where,
              "logits must be 2-D with contiguous rows")
        T, V = shape
        if T > DISTILL_MAX or V > DISTILL_MAX:
            _refuse(where, "logits must have at most 2^30 rows and columns")
        _need(isinstance(teacher_ids, torch.Tensor) and teacher_ids.dim() == 2, where, "teacher_ids must be [T, K]")
        K, dev = teacher_ids.shape[1], logits.device
        _check_tensor(teacher_ids, where, "teacher_ids", torch.int32, (T, K), dev)
        _check_tensor(teacher_logits, where, "teacher_logits", torch.float32, (T, K), dev)
        return PRECISIONS["fp32" if f32 else "bf16"], T, V, stride[0] if T > 1 else max(stride[0], V), K

    @staticmethod
    def _row_stride(t) -> int:
        """Elements between rows (a single row may report any stride)."""
        return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])

    def op_distill_loss(self, logits, teacher_ids, teacher_logits, temperature: float, token_loss, lse=None,
                        loss_sum=None, count=None, workspace=None, stream=None):
        """esm_op_distill_loss: t^2 KL(teacher's top logits || student) per row of logits [T, vocab]
        (float32 or bf16, rows may be strided), into token_loss [T]; optionally the rows' lse [T]
        (for the backward) and the sum and number of scored rows (device scalars).  teacher_ids
        int32, teacher_logits float32 [T, K]; id -1: unused entry."""
        where = "op_distill_loss"
        kind, T, V, stride, K = self._check_distill(where, logits, teacher_ids, teacher_logits)
        dev = logits.device
        _check_tensor(token_loss, where, "token_loss", torch.float32, (T,), dev)
        if lse is not None:
            _check_tensor(lse, where, "lse", torch.float32, (T,), dev)
        if loss_sum is not None:
            _check_scalar(loss_sum, where, "loss_sum", torch.float32, dev)
        if count is not None:
            _check_scalar(count, where, "count", torch.int32, dev)
        st = _launch_stream(where, stream, dev)
        if workspace is None and (loss_sum is not None or count is not None):
            with _allocating(stream):
                workspace = self.op_distill_loss_workspace(T, V, dev)
        if workspace is not None:
            _check_workspace(workspace, where, dev)
        self._raise(self.lib.esm_op_distill_loss(self.handle, logits.data_ptr(), kind, stride, teacher_ids.data_ptr(),
                                                 teacher_logits.data_ptr(), K, T, V, float(temperature),
                                                 token_loss.data_ptr(), _ptr(lse), _ptr(loss_sum), _ptr(count),
                                                 _ptr(workspace), 0 if workspace is None else workspace.nbytes, st),
                    "esm_op_distill_loss")
        return token_loss

    def op_distill_loss_backward(self, logits, teacher_ids, teacher_logits, temperature: float, lse, d_logits,
                                 loss_count=None, stream=None):
        """esm_op_distill_loss_backward: d_logits (the logits' type; may be logits itself) of the
        sum of token_loss divided by loss_count (device int32 scalar; None: of the sum)."""
        where = "op_distill_loss_backward"
        kind, T, V, stride, K = self._check_distill(where, logits, teacher_ids, teacher_logits)
        dev = logits.device
        _check_tensor(lse, where, "lse", torch.float32, (T,), dev)
        _need(isinstance(d_logits, torch.Tensor) and d_logits.device == dev and d_logits.dtype is logits.dtype
              and d_logits.shape == logits.shape and (d_logits.stride(1) == 1 or V == 1), where,
              "d_logits must have the type, device and shape of logits, and contiguous rows")
        if loss_count is not None:
            _check_scalar(loss_count, where, "loss_count", torch.int32, dev)
        self._raise(self.lib.esm_op_distill_loss_backward(self.handle, logits.data_ptr(), kind, stride,
                                                          teacher_ids.data_ptr(), teacher_logits.data_ptr(), K, T, V,
                                                          float(temperature), lse.data_ptr(), _ptr(loss_count),
                                                          d_logits.data_ptr(), self._row_stride(d_logits),
                                                          _launch_stream(where, stream, dev)),
                    "esm_op_distill_loss_backward")
        return d_logits

    # ------------------------------------------------------------------ the residual stream
    @staticmethod
    def _check_rows(t, where: str, name: str, device):
        """A 2-D float32 or bfloat16 CUDA tensor with contiguous rows; returns its esm_precision, shape and
        row stride (attributes are read once: an operator of a few microseconds has several tensors)."""
        if isinstance(t, torch.Tensor) and t.device == device and t.is_cuda:
            dtype, shape, strides = t.dtype, t.shape, t.stride()
            kind = 0 if dtype is torch.float32 else 1 if dtype is torch.bfloat16 else -1
            if kind >= 0 and len(shape) == 2:
                rows, cols = shape
                if (strides[1] == 1 or cols == 1) and rows <= STREAM_MAX and cols <= STREAM_MAX:
                    return kind, shape, strides[0] if rows > 1 else max(strides[0], cols)
        _need(isinstance(t, torch.Tensor) and t.is_cuda, where, f"{name} must be a CUDA tensor")
        _need(t.device == device, where, f"{name} must be on {device}")
        _need(t.dtype in (torch.float32, torch.bfloat16), where, f"{name} must be float32 or bfloat16")
        _need(t.dim() == 2, where, f"{name} must be 2-D")
        _need(t.stride(1) == 1 or t.shape[1] == 1, where, f"{name} must have contiguous rows")
        _refuse(where, f"{name} must have at most 2^30 rows and columns")

    @staticmethod
    def _dropout_struct(dropout, where: str, device):
        if dropout is None:
            return None
        if not (isinstance(dropout, Dropout) and dropout.device == device):
            _refuse(where, f"dropout must be a Dropout with its rng on {device}")
        return dropout.struct

    def op_dropout(self, x, y, dropout: Optional[Dropout], residual=None, stream=None):
        """esm_op_dropout: y = dropout(x), or residual + dropout(x); float32 or bf16 [rows, cols], rows
        may be strided.  y may be x or the residual.  The gradient: the same call on dy."""
        where = "op_dropout"
        _need(isinstance(x, torch.Tensor) and x.is_cuda, where, "x must be a CUDA tensor")
        dev = x.device
        kx, shape, sx = self._check_rows(x, where, "x", dev)
        ky, y_shape, sy = self._check_rows(y, where, "y", dev)
        if y_shape != shape:
            _refuse(where, "y must have the shape of x")
        sr = 0
        if residual is not None:
            kr, r_shape, sr = self._check_rows(residual, where, "residual", dev)
            _need(kr == ky and r_shape == shape, where, "residual must have the type and shape of y")
        d = self._dropout_struct(dropout, where, dev)
        self._raise(self.lib.esm_op_dropout(self.handle, x.data_ptr(), kx, sx, _ptr(residual), sr, y.data_ptr(), ky, sy,
                                            shape[0], shape[1], d, _launch_stream(where, stream, dev)),
                    "esm_op_dropout")
        return y

    @staticmethod
    def _check_ids(where: str, ids, row_scale):
        _need(isinstance(ids, torch.Tensor) and ids.is_cuda and ids.dim() == 1, where, "ids must be a 1-D CUDA tensor")
        T, dev = ids.shape[0], ids.device
        _check_tensor(ids, where, "ids", torch.int32, (T,), dev)
        _need(T <= STREAM_MAX, where, "ids must hold at most 2^30 tokens")
        if row_scale is not None:
            _check_tensor(row_scale, where, "row_scale", torch.float32, (T,), dev)
        return T, dev

    def op_embed(self, ids, table, out, scale: float = 1.0, row_scale=None, dropout: Optional[Dropout] = None,
                 stream=None):
        """esm_op_embed: out[t] = dropout(scale * row_scale[t] * table[ids[t]]), a row of zeros for id -1.
        ids int32 [T], table [vocab, cols] and out [T, cols] float32 or bf16 (out's rows may be strided),
        row_scale float32 [T]."""
        where = "op_embed"
        T, dev = self._check_ids(where, ids, row_scale)
        kt, (V, cols), _ = self._check_rows(table, where, "table", dev)
        ko, shape, so = self._check_rows(out, where, "out", dev)
        if not table.is_contiguous():
            _refuse(where, "table must be contiguous")
        if shape != (T, cols):
            _refuse(where, f"out must be {[T, cols]}")
        d = self._dropout_struct(dropout, where, dev)
        self._raise(self.lib.esm_op_embed(self.handle, ids.data_ptr(), T, table.data_ptr(), kt, V, cols, float(scale),
                                          _ptr(row_scale), d, out.data_ptr(), ko, so,
                                          _launch_stream(where, stream, dev)), "esm_op_embed")
        return out

    def op_embed_backward_workspace(self, T: int, vocab: int, cols: int, device="cuda"):
        where, n = "op_embed_backward_workspace", ctypes.c_size_t()
        T, vocab, cols = _c_int(where, "T", T), _c_int(where, "vocab", vocab), _c_int(where, "cols", cols)
        self._raise(self.lib.esm_op_embed_backward_workspace_size(self.handle, T, vocab, cols, ctypes.byref(n)),
                    "esm_op_embed_backward_workspace_size")
        return torch.empty(int(n.value), dtype=torch.uint8, device=device)

    def op_embed_backward(self, ids, d_out, d_table, scale: float = 1.0, row_scale=None,
                          dropout: Optional[Dropout] = None, accumulate: bool = False, workspace=None, stream=None):
        """esm_op_embed_backward: d_table (float32 [vocab, cols]) = or, with accumulate, += the sum over each
        id's tokens of scale * row_scale[t] * dropout(d_out[t]); d_out float32 or bf16 [T, cols]."""
        where = "op_embed_backward"
        T, dev = self._check_ids(where, ids, row_scale)
        kd, shape, sd = self._check_rows(d_out, where, "d_out", dev)
        kt, (V, cols), _ = self._check_rows(d_table, where, "d_table", dev)
        if kt or not d_table.is_contiguous():
            _refuse(where, "d_table must be contiguous float32")
        if shape != (T, cols):
            _refuse(where, f"d_out must be {[T, cols]}")
        d = self._dropout_struct(dropout, where, dev)
        st = _launch_stream(where, stream, dev)
        if workspace is None:
            with _allocating(stream):
                workspace = self.op_embed_backward_workspace(T, V, cols, dev)
        _check_workspace(workspace, where, dev)
        self._raise(self.lib.esm_op_embed_backward(self.handle, ids.data_ptr(), T, d_out.data_ptr(), kd, sd,
                                                   float(scale), _ptr(row_scale), d, d_table.data_ptr(), V, cols,
                                                   int(bool(accumulate)), workspace.data_ptr(), workspace.nbytes, st),
                    "esm_op_embed_backward")
        return d_table

    def _check_block_norm(self, where: str, norm, y, gate):
        """The block's output, norms and gate; returns rows, cols, the device and whether the gate has rows."""
        _need(isinstance(norm, BlockNorm), where, "norm must be a BlockNorm")
        _need(isinstance(y, torch.Tensor) and y.is_cuda and y.dim() == 2, where, "y must be a 2-D CUDA tensor")
        rows, cols = y.shape
        dev, act = y.device, self.out_dtype
        _check_tensor(y, where, "y", act, (rows, cols), dev)
        _need(rows <= STREAM_MAX and cols <= STREAM_MAX, where, "y must have at most 2^30 rows and columns")
        if norm.cols is not None and not (norm.cols == cols and norm.dtype is act and norm.device == dev):
            _refuse(where, f"norm's parameters must be {act} [{cols}] on {dev}")
        gate_rows = 0
        if gate is not None:
            gate_rows = int(isinstance(gate, torch.Tensor) and gate.dim() == 2)
            _check_tensor(gate, where, "gate", act, (rows, cols) if gate_rows else (cols,), dev)
        return rows, cols, dev, gate_rows

    def op_block_norm(self, norm: BlockNorm, x, y, x_out, h=None, gate=None, dropout: Optional[Dropout] = None,
                      stats=None, stream=None):
        """esm_op_block_norm: x_out = residual_scale * x + gate * dropout(post(y)), h = pre(x_out), with
        norm's post and pre.  x, x_out float32 [rows, cols] (x_out may be x); y, h of the activation dtype (h may
        be y; None without a pre); gate [cols] or [rows, cols]; stats float32 [rows, 4] for the backward."""
        where = "op_block_norm"
        rows, cols, dev, gate_rows = self._check_block_norm(where, norm, y, gate)
        _check_tensor(x, where, "x", torch.float32, (rows, cols), dev)
        _check_tensor(x_out, where, "x_out", torch.float32, (rows, cols), dev)
        _need((h is not None) == (norm.pre_gamma is not None), where, "h goes with a norm before the next block")
        if h is not None:
            _check_tensor(h, where, "h", self.out_dtype, (rows, cols), dev)
        if stats is not None:
            _check_tensor(stats, where, "stats", torch.float32, (rows, 4), dev)
        d = self._dropout_struct(dropout, where, dev)
        self._raise(self.lib.esm_op_block_norm(self.handle, norm.struct, _ptr(gate), gate_rows, d, x.data_ptr(),
                                               y.data_ptr(), x_out.data_ptr(), _ptr(h), _ptr(stats), rows, cols,
                                               _launch_stream(where, stream, dev)), "esm_op_block_norm")
        return x_out, h

    def op_block_norm_backward_workspace(self, rows: int, cols: int, device="cuda"):
        where, n = "op_block_norm_backward_workspace", ctypes.c_size_t()
        rows, cols = _c_int(where, "rows", rows), _c_int(where, "cols", cols)
        self._raise(self.lib.esm_op_block_norm_backward_workspace_size(self.handle, rows, cols, ctypes.byref(n)),
                    "esm_op_block_norm_backward_workspace_size")
        return torch.empty(int(n.value), dtype=torch.uint8, device=device)

    def op_block_norm_backward(self, norm: BlockNorm, x_out, y, stats, d_x_out, d_h, dx, dy, grads: Dict, gate=None,
                               dropout: Optional[Dropout] = None, workspace=None, stream=None):
        """esm_op_block_norm_backward: dx (float32; may be d_x_out), dy (the activation dtype; may be d_h or
        y) and the gradients named in grads ("post_gamma", "post_beta", "pre_gamma", "pre_beta", "gate":
        float32 [cols]; the gradient of a gate [rows, cols] like the gate) from x_out, y and stats of the forward,
        d_x_out float32 (None: 0) and d_h (None exactly without a pre)."""
        where = "op_block_norm_backward"
        rows, cols, dev, gate_rows = self._check_block_norm(where, norm, y, gate)
        act, full = self.out_dtype, (rows, cols)
        pre = norm.pre_gamma is not None
        _need((d_h is not None) == pre, where, "d_h goes with a norm before the next block")
        for name, t, dt in (("x_out", x_out, torch.float32), ("d_x_out", d_x_out, torch.float32), ("d_h", d_h, act),
                            ("dx", dx, torch.float32), ("dy", dy, act)):
            if t is not None or name in ("dx", "dy") or (pre and name == "x_out"):
                _check_tensor(t, where, name, dt, full, dev)
        if pre or norm.post_gamma is not None:
            _check_tensor(stats, where, "stats", torch.float32, (rows, 4), dev)
        g = EsmBlockNormGrads()
        for name, t in grads.items():
            has = gate if name == "gate" else getattr(norm, name) if name in BLOCK_NORM_PARAMS else None
            _need(has is not None, where, f"there is no {name!r} to take a gradient of")
            if name == "gate" and gate_rows:
                _check_tensor(t, where, "grads['gate']", act, full, dev)
            else:
                _check_tensor(t, where, f"grads[{name!r}]", torch.float32, (cols,), dev)
            setattr(g, name, t.data_ptr())
        d = self._dropout_struct(dropout, where, dev)
        st = _launch_stream(where, stream, dev)
        if workspace is None:
            with _allocating(stream):
                workspace = self.op_block_norm_backward_workspace(rows, cols, dev)
        _check_workspace(workspace, where, dev)
        self._raise(self.lib.esm_op_block_norm_backward(self.handle, norm.struct, _ptr(gate), gate_rows, d, _ptr(x_out),
                                                        y.data_ptr(), _ptr(stats), _ptr(d_x_out), _ptr(d_h),
                                                        dx.data_ptr(), dy.data_ptr(), g, rows, cols,
                                                        workspace.data_ptr(), workspace.nbytes, st),
                    "esm_op_block_norm_backward")
        return dx, dy, grads

    def set_layer_precision(self, per_layer):
        """esm_encoder_set_layer_precision: one of "fp32", "bf16", "fp8", "fp4" per layer."""
        arr = (ctypes.c_int * max(1, len(per_layer)))(*[PRECISIONS[p] for p in per_layer])
        self._raise(self.lib.esm_encoder_set_layer_precision(self.handle, arr, len(per_layer)),
                    "esm_encoder_set_layer_precision")

    def lm_head_workspace(self, T: int, device="cuda"):
        n = ctypes.c_size_t()
        self._raise(self.lib.esm_encoder_lm_head_workspace_size(self.handle, T, ctypes.byref(n)),
                    "esm_encoder_lm_head_workspace_size")
        return torch.empty(max(int(n.value), 256), dtype=torch.uint8, device=device)

    def lm_head(self, head: "DeviceLmHead", hidden, targets=None, logits=None, token_loss=None, loss_sum=None,
                count=None, workspace=None, stream=None):
        """esm_encoder_lm_head: logits [T, vocab] / per-token masked cross-entropy / its sum and
        the number of scored tokens, into the given device tensors (any may be None)."""
        T = hidden.shape[0]
        if workspace is None:
            workspace = self.lm_head_workspace(T, hidden.device)
        self._raise(self.lib.esm_encoder_lm_head(self.handle, ctypes.byref(head.struct), _ptr(hidden), T, _ptr(targets),
                                                 _ptr(logits), _ptr(token_loss), _ptr(loss_sum), _ptr(count),
                                                 _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
                    "esm_encoder_lm_head")

    # ------------------------------------------------------------------ training
    def set_dropout(self, dropout: Optional[Dropout] = None):
        """esm_encoder_set_dropout: dropout of the embedding and of every block's output in forward_train
        (and its backward); None for none.  A step uses 2 * num_layers + 1 offsets from dropout's on."""
        where = "set_dropout"
        _need(dropout is None or isinstance(dropout, Dropout), where, "dropout must be a Dropout or None")
        self._raise(self.lib.esm_encoder_set_dropout(self.handle, None if dropout is None else dropout.struct),
                    "esm_encoder_set_dropout")
        self._dropout = dropout  # keeps rng's memory

    def train_buffer(self, max_tokens: int, device="cuda"):
        n = ctypes.c_size_t()
        self._raise(self.lib.esm_encoder_train_buffer_size(self.handle, max_tokens, ctypes.byref(n)),
                    "esm_encoder_train_buffer_size")
        return torch.empty(int(n.value), dtype=torch.uint8, device=device)

    def forward_train(self, weights: DeviceWeights, token_ids, cu_seqlens, max_seqlen: int, train_buf, workspace,
                      out=None, stream=None):
        """esm_encoder_forward_train: the forward, keeping its activations in train_buf."""
        T = token_ids.numel()
        B = cu_seqlens.numel() - 1
        drop = getattr(self, "_dropout", None)
        _need(drop is None or drop.device == token_ids.device, "forward_train",
              f"the dropout's rng must be on {token_ids.device}")
        if out is None:
            out = torch.empty(T, self.hidden, dtype=self.out_dtype, device=token_ids.device)
        self._raise(self.lib.esm_encoder_forward_train(self.handle, ctypes.byref(weights.struct), _ptr(token_ids),
                                                       _ptr(cu_seqlens), B, T, int(max_seqlen), _ptr(out),
                                                       _ptr(train_buf), train_buf.numel(), _ptr(workspace),
                                                       workspace.numel(), _stream_ptr(stream)),
                    "esm_encoder_forward_train")
        self._train_dropout = drop  # the backward reads its rng
        return out

    def backward(self, weights: DeviceWeights, d_out, grads: "DeviceGrads", train_buf, workspace, stream=None):
        """esm_encoder_backward: parameter gradients of the last forward_train, given dL/d(out)."""
        self._raise(self.lib.esm_encoder_backward(self.handle, ctypes.byref(weights.struct), _ptr(d_out),
                                                  ctypes.byref(grads.struct), _ptr(train_buf), train_buf.numel(),
                                                  _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
                    "esm_encoder_backward")
        return grads

    def op_gemm_dgrad(self, dY, W, out, stream=None):
        M, N = dY.shape
        K = W.shape[1]
        self._raise(self.lib.esm_op_gemm_dgrad(self.handle, _ptr(dY), _ptr(W), _ptr(out),
                                               int(out.dtype == torch.bfloat16), M, N, K, _stream_ptr(stream)),
                    "esm_op_gemm_dgrad")
        return out

    def op_gemm_wgrad(self, dY, X, dW, workspace=None, stream=None):
        M, N = dY.shape
        K = X.shape[1]
        if workspace is None:
            n = ctypes.c_size_t()
            self._raise(self.lib.esm_op_gemm_wgrad_workspace_size(self.handle, N, K, ctypes.byref(n)),
                        "esm_op_gemm_wgrad_workspace_size")
            workspace = torch.empty(int(n.value), dtype=torch.uint8, device=dY.device)
        self._raise(self.lib.esm_op_gemm_wgrad(self.handle, _ptr(dY), _ptr(X), _ptr(dW), M, N, K, _ptr(workspace),
                                               0 if workspace is None else workspace.numel(), _stream_ptr(stream)),
                    "esm_op_gemm_wgrad")
        return dW

    def op_layernorm_backward(self, x, gamma, dy, dres, dx, dgamma, dbeta, stream=None):
        rows, cols = x.shape
        n = ctypes.c_size_t()
        self._raise(self.lib.esm_op_layernorm_backward_workspace_size(self.handle, rows, cols, ctypes.byref(n)),
                    "esm_op_layernorm_backward_workspace_size")
        ws = torch.empty(int(n.value), dtype=torch.uint8, device=x.device)
        self._raise(self.lib.esm_op_layernorm_backward(self.handle, _ptr(x), _ptr(gamma), _ptr(dy), _ptr(dres),
                                                       _ptr(dx), _ptr(dgamma), _ptr(dbeta), rows, cols, _ptr(ws),
                                                       ws.numel(), _stream_ptr(stream)), "esm_op_layernorm_backward")
        return dx, dgamma, dbeta

    def op_attention_train(self, qkv, cu_seqlens, max_seqlen: int, o, lse, workspace=None, stream=None):
        T = qkv.shape[0]
        B = cu_seqlens.numel() - 1
        if workspace is None:
            workspace = self.workspace(T, B, qkv.device)
        self._raise(self.lib.esm_op_attention_train(self.handle, _ptr(qkv), _ptr(cu_seqlens), B, T, int(max_seqlen),
                                                    _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                                                    _stream_ptr(stream)), "esm_op_attention_train")
        return o, lse

    def op_attention_backward(self, qkv, o, lse, d_o, cu_seqlens, max_seqlen: int, dqkv, workspace=None,
                              stream=None):
        T = qkv.shape[0]
        B = cu_seqlens.numel() - 1
        if workspace is None:
            n = ctypes.c_size_t()
            self._raise(self.lib.esm_op_attention_backward_workspace_size(self.handle, T, B, ctypes.byref(n)),
                        "esm_op_attention_backward_workspace_size")
            workspace = torch.empty(int(n.value), dtype=torch.uint8, device=qkv.device)
        self._raise(self.lib.esm_op_attention_backward(self.handle, _ptr(qkv), _ptr(o), _ptr(lse), _ptr(d_o),
                                                       _ptr(cu_seqlens), B, T, int(max_seqlen), _ptr(dqkv),
                                                       _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
                    "esm_op_attention_backward")
        return dqkv

    def lm_head_backward_workspace(self, T: int, device="cuda"):
        n = ctypes.c_size_t()
        self._raise(self.lib.esm_encoder_lm_head_backward_workspace_size(self.handle, T, ctypes.byref(n)),
                    "esm_encoder_lm_head_backward_workspace_size")
        return torch.empty(int(n.value), dtype=torch.uint8, device=device)

    def lm_head_backward(self, head: "DeviceLmHead", hidden, targets, d_hidden=None, grads=None, loss_sum=None,
                         count=None, workspace=None, stream=None, loss_count=None):
        """esm_encoder_lm_head_backward: dL/d(hidden) (float32 [T, hidden]) and the head's
        gradients (dict of float32 device tensors shaped like the head's parameters) of the
        mean masked-LM loss.  ``loss_count`` (device int32 scalar): the scored-token count the
        mean divides by, e.g. the global batch's in data-parallel training (None: this call's)."""
        T = hidden.shape[0]
        dev = hidden.device
        if d_hidden is None:
            d_hidden = torch.empty(T, self.hidden, dtype=torch.float32, device=dev)
        if grads is None:
            grads = {k: torch.empty(tuple(head.t[k].shape), dtype=torch.float32, device=dev) for k in LM_HEAD_NAMES}
        if workspace is None:
            workspace = self.lm_head_backward_workspace(T, dev)
        gs = EsmLmHeadGrads(*[grads[k].data_ptr() for k in LM_HEAD_NAMES])
        self._raise(self.lib.esm_encoder_lm_head_backward(self.handle, ctypes.byref(head.struct), _ptr(hidden), T,
                                                          _ptr(targets), _ptr(d_hidden), ctypes.byref(gs),
                                                          _ptr(loss_sum), _ptr(count), _ptr(loss_count),
                                                          _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
                    "esm_encoder_lm_head_backward")
        return d_hidden, grads

    def lm_head_distill_backward(self, head: "DeviceLmHead", hidden, teacher_ids, teacher_logits, temperature: float,
                                 d_hidden=None, grads=None, loss_sum=None, count=None, workspace=None, stream=None,
                                 loss_count=None):
        """esm_encoder_lm_head_distill_backward: as lm_head_backward, for the distillation loss
        against a teacher's top logits (teacher_ids int32, teacher_logits float32 [T, K])."""
        where = "lm_head_distill_backward"
        _need(isinstance(hidden, torch.Tensor) and hidden.dim() == 2, where, "hidden must be a 2-D tensor")
        T, dev = hidden.shape[0], hidden.device
        _check_tensor(hidden, where, "hidden", self.out_dtype, (T, self.hidden), dev)
        _need(isinstance(teacher_ids, torch.Tensor) and teacher_ids.dim() == 2, where, "teacher_ids must be [T, K]")
        K = teacher_ids.shape[1]
        _check_tensor(teacher_ids, where, "teacher_ids", torch.int32, (T, K), dev)
        _check_tensor(teacher_logits, where, "teacher_logits", torch.float32, (T, K), dev)
        for name, t, dt in (("loss_sum", loss_sum, torch.float32), ("count", count, torch.int32),
                            ("loss_count", loss_count, torch.int32)):
            if t is not None:
                _check_scalar(t, where, name, dt, dev)
        st = _launch_stream(where, stream, dev)
        with _allocating(stream):
            if d_hidden is None:
                d_hidden = torch.empty(T, self.hidden, dtype=torch.float32, device=dev)
            if grads is None:
                grads = {k: torch.empty_like(head.t[k], dtype=torch.float32) for k in LM_HEAD_NAMES}
            if workspace is None:
                workspace = self.lm_head_backward_workspace(T, dev)
        _check_tensor(d_hidden, where, "d_hidden", torch.float32, (T, self.hidden), dev)
        for k in LM_HEAD_NAMES:
            _check_tensor(grads[k], where, f"grads[{k!r}]", torch.float32, head.t[k].shape, dev)
        _check_workspace(workspace, where, dev)
        gs = EsmLmHeadGrads(*[grads[k].data_ptr() for k in LM_HEAD_NAMES])
        self._raise(self.lib.esm_encoder_lm_head_distill_backward(
            self.handle, ctypes.byref(head.struct), hidden.data_ptr(), T, teacher_ids.data_ptr(),
            teacher_logits.data_ptr(), K, float(temperature), d_hidden.data_ptr(), ctypes.byref(gs), _ptr(loss_sum),
            _ptr(count), _ptr(loss_count), workspace.data_ptr(), workspace.nbytes, st),
            "esm_encoder_lm_head_distill_backward")
        return d_hidden, grads

    def op_quantize_nvfp4(self, x, stream=None):
        """esm_op_quantize_nvfp4 of a contiguous bf16 [rows, cols] CUDA tensor: returns (codes uint8
        [rows, cols/2], scales uint8 [rows * cols / 16] in the tensor-core atom order, amax and
        scale as float32 one-element tensors)."""
        rows, cols = x.shape
        codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(rows * cols // 16, dtype=torch.uint8, device=x.device)
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
        self._raise(self.lib.esm_op_quantize_nvfp4(self.handle, _ptr(x), rows, cols, _ptr(codes), _ptr(scales),
                                                   _ptr(amax), _ptr(scale), _stream_ptr(stream)), "esm_op_quantize_nvfp4")
        return codes, scales, amax, scale

    def op_gemm_nvfp4(self, a, b, bias=None, out=None, epi="bias_f32", pos_id=None, stream=None):
        """esm_op_gemm_nvfp4 of two operands returned by op_quantize_nvfp4 (A [M, K], B [N, K]):
        v = (A B^T) / (S_A S_B) + bias, then the epilogue `epi` ("bias_f32": float32 out = v;
        "residual": float32 out += v; "gelu": bf16 out = GELU(v); "qkv_rope": bf16 out = v with
        RoPE at the rows' positions pos_id)."""
        (ac, asf, _, asc), (bc, bsf, _, bsc) = a, b
        M, N, K = ac.shape[0], bc.shape[0], 2 * ac.shape[1]
        if out is None:
            dt = torch.float32 if epi in ("bias_f32", "residual") else torch.bfloat16
            out = torch.zeros(M, N, dtype=dt, device=ac.device)
        self._raise(self.lib.esm_op_gemm_nvfp4(self.handle, EPILOGUES[epi], _ptr(ac), _ptr(asf), _ptr(asc), _ptr(bc),
                                               _ptr(bsf), _ptr(bsc), _ptr(bias), _ptr(pos_id), _ptr(out), M, N, K,
                                               _stream_ptr(stream)), "esm_op_gemm_nvfp4")
        return out

    def set_profiling(self, enable: bool):
        self._raise(self.lib.esm_encoder_set_profiling(self.handle, int(enable)), "esm_encoder_set_profiling")

    def get_profile(self, reset: bool = True) -> Dict:
        """{class: {"ms": summed device ms, "launches": n}} plus "total_launches"."""
        p = EsmProfile()
        self._raise(self.lib.esm_encoder_get_profile(self.handle, ctypes.byref(p), int(reset)),
                    "esm_encoder_get_profile")
        out = {name: {"ms": p.ms[i], "launches": int(p.launches[i])} for i, name in enumerate(PROFILE_CLASSES)}
        out["total_launches"] = int(p.total_launches)
        return out

    def fp8_state_size(self) -> int:
        return self.num_layers * 8 * (1 + self.amax_history_len)

    def get_fp8_state(self) -> np.ndarray:
        buf = np.zeros(self.fp8_state_size(), dtype=np.float32)
        self._raise(self.lib.esm_encoder_get_fp8_state(self.handle, buf.ctypes.data_as(ctypes.POINTER(ctypes.c_float)),
                                                       buf.size), "esm_encoder_get_fp8_state")
        return buf

    def set_fp8_state(self, buf: np.ndarray):
        buf = np.ascontiguousarray(buf, dtype=np.float32)
        self._raise(self.lib.esm_encoder_set_fp8_state(self.handle, buf.ctypes.data_as(ctypes.POINTER(ctypes.c_float)),
                                                       buf.size), "esm_encoder_set_fp8_state")

    def fp4_scales(self) -> np.ndarray:
        """[num_layers, 8] NVFP4 tensor scales of the last forward's FP4 layers (tensor order
        x_qkv, w_qkv, x_o, w_o, x_1, w_1, x_2, w_2; zero for other layers)."""
        buf = np.zeros(self.num_layers * 8, dtype=np.float32)
        self._raise(self.lib.esm_encoder_get_fp4_scales(self.handle, buf.ctypes.data_as(ctypes.POINTER(ctypes.c_float)),
                                                        buf.size), "esm_encoder_get_fp4_scales")
        return buf.reshape(self.num_layers, 8)

    def fp8_scales(self, buf: Optional[np.ndarray] = None) -> np.ndarray:
        """[num_layers, 8] scales from a state buffer (tensor order x_qkv, w_qkv, x_o, w_o, x_1, w_1, x_2, w_2)."""
        buf = self.get_fp8_state() if buf is None else buf
        return buf[:self.num_layers * 8].reshape(self.num_layers, 8)

    def fp8_history(self, buf: Optional[np.ndarray] = None) -> np.ndarray:
        buf = self.get_fp8_state() if buf is None else buf
        return buf[self.num_layers * 8:].reshape(self.num_layers, 8, self.amax_history_len)


def op_attention_noalloc(qkv, cu_seqlens, max_seqlen: int, hidden: int, heads: int, o, status=None,
                         stream=None) -> int:
    """esm_op_attention_noalloc: attention with no handle, no workspace and no allocation.

    qkv: contiguous CUDA bf16 [T, 3*hidden]; o: contiguous CUDA bf16 [T, hidden];
    cu_seqlens: contiguous int32 [B + 1] on the same device; status: optional int32 device
    tensor of one element that receives the call's device-side outcome (ESM_OK,
    ESM_ERR_BAD_CU_SEQLENS or ESM_ERR_TIMEOUT).  Raises ValueError on tensors the C side
    cannot check (wrong dtype, device, layout or shape); returns the call's status code."""

    def need(ok, what):
        if not ok:
            raise ValueError(f"op_attention_noalloc: {what}")

    for name, t in (("qkv", qkv), ("o", o), ("cu_seqlens", cu_seqlens)):
        need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name} must be a CUDA tensor")
        need(t.is_contiguous(), f"{name} must be contiguous")
        need(t.device == qkv.device, f"{name} must be on {qkv.device}")
    need(qkv.dtype == torch.bfloat16 and o.dtype == torch.bfloat16, "qkv and o must be bfloat16")
    need(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2,
         "cu_seqlens must be a 1-D int32 tensor of at least two offsets")
    need(qkv.dim() == 2 and qkv.shape[1] == 3 * hidden, f"qkv must be [T, {3 * hidden}]")
    need(o.dim() == 2 and tuple(o.shape) == (qkv.shape[0], hidden), f"o must be [{qkv.shape[0]}, {hidden}]")
    if status is not None:
        need(isinstance(status, torch.Tensor) and status.device == qkv.device and status.dtype == torch.int32
             and status.numel() >= 1, "status must be an int32 tensor on the device of qkv")
    lib = load_library()
    return lib.esm_op_attention_noalloc(_ptr(qkv), _ptr(cu_seqlens), cu_seqlens.numel() - 1, qkv.shape[0],
                                        int(max_seqlen), hidden, heads, _ptr(o), _ptr(status), _stream_ptr(stream))


def packed_inputs(tokens: np.ndarray, lengths: Sequence[int], device="cuda"):
    """Device token ids and cu_seqlens (int32) for a packed batch."""
    from .synth import cu_seqlens_from_lengths
    tok = torch.from_numpy(np.ascontiguousarray(tokens, dtype=np.int32)).to(device)
    cu = torch.from_numpy(cu_seqlens_from_lengths(lengths)).to(device)
    return tok, cu
