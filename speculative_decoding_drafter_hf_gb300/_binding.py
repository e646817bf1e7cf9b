"""ctypes binding of libhyflash.so (include/hyflash.h): argument marshalling only.

Every computation happens in the library's CUDA kernels. PyTorch is used here
only to hand over device pointers and streams. If the shared library has not
been built, importing this module raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import enum
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhyflash.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python -m speculative_decoding_drafter_hf_gb300.build` (nvcc, sm_103a)")

lib = ctypes.CDLL(LIB_PATH)


class Status(enum.IntEnum):
    OK = 0
    EINVAL = 1
    ENOMEM = 2
    ECUDA = 3
    ETIMEOUT = 4
    EDEVICE = 5


class Tensor(enum.IntEnum):
    STATE = 0
    RING_K = 1
    RING_V = 2
    RING_TAG = 3
    POS = 4
    OFFSETS = 5
    DRAFT_PROJ = 6
    DRAFT_MIX = 7
    MEM_X = 8
    MEM_B = 9
    MEM_DT = 10
    CONV = 11
    LOGITS = 12


class Family(enum.IntEnum):
    DRAFT_PROJ = 0
    ATTN_MEM = 1
    OUT_PROJ = 2
    ROUND_PROJ = 3
    COMMIT_PROJ = 4
    COMMIT_STATE = 5
    PREFILL = 6
    OTHER = 7
    MLP = 8
    HEAD = 9


HF_F32, HF_BF16, HF_E4M3 = 0, 1, 2


class HfConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "d_model", "n_q_heads", "n_kv_heads", "head_dim", "window", "block",
        "ssm_heads", "ssm_headdim", "d_state", "n_groups", "n_layers",
        "max_batch", "chunk", "dtype")] + [("prefill_tokens_max", ctypes.c_int64),
                                           ("cross_slot_off", ctypes.c_int32),
                                           ("mem_horizon", ctypes.c_int32),
                                           ("memory_kind", ctypes.c_int32),
                                           ("weight_bits", ctypes.c_int32),
                                           ("block_kind", ctypes.c_int32),
                                           ("mlp_dim", ctypes.c_int32),
                                           ("vocab", ctypes.c_int32)]


WEIGHT_FIELDS = ("w_q", "w_k", "w_v", "w_o", "w_x", "w_B", "w_C", "w_dt", "w_mo",
                 "dt_bias", "A_log", "w_beta")
MEMORY_KINDS = {"mamba2": 0, "gdn": 1}


class HfLayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_FIELDS]


BLOCK_FIELDS = ("g_mix", "g_mlp", "w_z", "d_skip", "conv_w", "conv_b", "w_gate", "w_up", "w_down")
BLOCK_F32 = ("g_mix", "g_mlp", "d_skip", "conv_w", "conv_b")


class HfBlockWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in BLOCK_FIELDS]


class HfQ4Matrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


Q4_MATRICES = ("w_q", "w_k", "w_v", "w_o", "w_x", "w_B", "w_C", "w_dt", "w_mo", "w_beta")


class HfLayerWeightsQ4(ctypes.Structure):
    _fields_ = [(n, HfQ4Matrix) for n in Q4_MATRICES] + [
        ("dt_bias", ctypes.c_void_p), ("A_log", ctypes.c_void_p)]


_h = ctypes.c_void_p
_st = ctypes.c_int
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32


def _sig(name, res, *args):
    f = getattr(lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


hf_create = _sig("hf_create", _st, ctypes.POINTER(HfConfig), _i32, ctypes.POINTER(_h))
hf_destroy = _sig("hf_destroy", None, _h)
hf_set_weights = _sig("hf_set_weights", _st, _h, _i32, ctypes.POINTER(HfLayerWeights))
hf_set_weights_q4 = _sig("hf_set_weights_q4", _st, _h, _i32, ctypes.POINTER(HfLayerWeightsQ4))
hf_prefill = _sig("hf_prefill", _st, _h, _vp, ctypes.POINTER(_i32), ctypes.POINTER(_i32), _i32, _vp)
hf_commit = _sig("hf_commit", _st, _h, _vp, _vp, _i32, _vp)
hf_draft = _sig("hf_draft", _st, _h, _vp, _vp, _i32, _vp)
hf_round = _sig("hf_round", _st, _h, _vp, _vp, _vp, _vp, _i32, _vp)
hf_sync = _sig("hf_sync", _st, _h, _vp)
hf_last_error = _sig("hf_last_error", ctypes.c_char_p, _h)
hf_status_string = _sig("hf_status_string", ctypes.c_char_p, _st)
hf_tensor_bytes = _sig("hf_tensor_bytes", _st, _h, _i32, ctypes.POINTER(ctypes.c_size_t))
hf_read_tensor = _sig("hf_read_tensor", _st, _h, _i32, _vp, ctypes.c_size_t)
hf_context_bytes = _sig("hf_context_bytes", ctypes.c_size_t, _h)
hf_export_context = _sig("hf_export_context", _st, _h, _vp, ctypes.c_size_t)
hf_import_context = _sig("hf_import_context", _st, _h, _vp, ctypes.c_size_t)
hf_profile_enable = _sig("hf_profile_enable", _st, _h, _i32)
hf_profile_collect = _sig("hf_profile_collect", _st, _h)
hf_profile_read = _sig("hf_profile_read", _st, _h, _i32, ctypes.POINTER(ctypes.c_double),
                       ctypes.POINTER(ctypes.c_int64), _i32)
hf_launch_count = _sig("hf_launch_count", ctypes.c_int64, _h)
hf_attention_noalloc = _sig("hf_attention_noalloc", _st, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                            _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp)
hf_set_block_weights = _sig("hf_set_block_weights", _st, _h, _i32, ctypes.POINTER(HfLayerWeights),
                            ctypes.POINTER(HfBlockWeights))
hf_set_head_weights = _sig("hf_set_head_weights", _st, _h, _vp, _vp)
hf_draft_tokens = _sig("hf_draft_tokens", _st, _h, _vp, _vp, _vp, _i32, _vp)


class HfPages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "table", "lens", "refs", "work", "status")] + [
        (n, ctypes.c_int32) for n in ("dtype", "n_layers", "n_pages", "n_kv_heads", "page", "head_dim",
                                      "n_requests", "table_ld")]


class HfPages8(ctypes.Structure):
    _fields_ = [("pages", HfPages), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class HfRotaryScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("original", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("factor", "fast", "slow", "attention")]


ROTARY_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}

_i64, _f32, _sz = ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_pp = ctypes.POINTER(HfPages)
_p8 = ctypes.POINTER(HfPages8)
hf_attention_prompt = _sig("hf_attention_prompt", _st, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _i64,
                           _vp, _i64, _vp, _f32, _vp, _i64, _vp, _vp)
hf_attention_pages = _sig("hf_attention_pages", _st, _pp, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _i32, _f32,
                          _vp, _i64, _vp, _sz, _vp)
hf_attention_pages_workspace = _sig("hf_attention_pages_workspace", _sz, _pp, _i32, _i32, _i32, _i32)
hf_pages_work_ints = _sig("hf_pages_work_ints", _sz, _pp)
hf_pages_extend = _sig("hf_pages_extend", _st, _pp, _vp, _vp, _i32, _vp)
hf_pages_write = _sig("hf_pages_write", _st, _pp, _i32, _i32, _vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _vp)
hf_pages_fork = _sig("hf_pages_fork", _st, _pp, _vp, _vp, _i32, _vp)
hf_pages_truncate = _sig("hf_pages_truncate", _st, _pp, _vp, _vp, _i32, _vp)
hf_pages_compact = _sig("hf_pages_compact", _st, _pp, _vp, _vp)
hf_attention_pages8 = _sig("hf_attention_pages8", _st, _p8, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _i32, _f32,
                           _vp, _i64, _vp, _sz, _vp)
hf_attention_pages8_workspace = _sig("hf_attention_pages8_workspace", _sz, _p8, _i32, _i32, _i32, _i32)
hf_pages8_work_ints = _sig("hf_pages8_work_ints", _sz, _p8)
hf_pages8_extend = _sig("hf_pages8_extend", _st, _p8, _vp, _vp, _i32, _vp)
hf_pages8_fork = _sig("hf_pages8_fork", _st, _p8, _vp, _vp, _i32, _vp)
hf_pages8_truncate = _sig("hf_pages8_truncate", _st, _p8, _vp, _vp, _i32, _vp)
hf_pages8_compact = _sig("hf_pages8_compact", _st, _p8, _vp, _vp)
hf_pages8_write = _sig("hf_pages8_write", _st, _p8, _i32, _i32, _vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _vp)
hf_pages8_read = _sig("hf_pages8_read", _st, _p8, _i32, _i32, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32, _vp)
hf_rotary_table = _sig("hf_rotary_table", _st, _i32, ctypes.c_double, ctypes.POINTER(HfRotaryScaling), _vp,
                       ctypes.POINTER(_f32))
hf_rotary = _sig("hf_rotary", _st, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _f32, _vp, _vp, _i64, _vp, _i64,
                 _vp, _i64, _vp, _i64, _vp)
hf_verify_tokens = _sig("hf_verify_tokens", _st, _i32, _vp, _i64, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp,
                        _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp, _vp)
hf_verify_workspace = _sig("hf_verify_workspace", _sz, _i32, _i32, _i32)
hf_debug_set_wait_limit = _sig("hf_debug_set_wait_limit", _st, _h, ctypes.c_int64)
hf_debug_fail_alloc = _sig("hf_debug_fail_alloc", _st, ctypes.c_int64)
hf_debug_check_guards = _sig("hf_debug_check_guards", _st, _h)

EXPORTED = ("hf_create", "hf_destroy", "hf_set_weights", "hf_set_weights_q4", "hf_prefill", "hf_commit", "hf_draft",
            "hf_round", "hf_sync", "hf_last_error", "hf_status_string", "hf_tensor_bytes", "hf_read_tensor",
            "hf_context_bytes", "hf_export_context", "hf_import_context", "hf_profile_enable",
            "hf_profile_collect", "hf_profile_read", "hf_launch_count", "hf_attention_noalloc",
            "hf_debug_set_wait_limit", "hf_debug_fail_alloc", "hf_debug_check_guards",
            "hf_set_block_weights", "hf_set_head_weights", "hf_draft_tokens",
            "hf_attention_prompt", "hf_attention_pages", "hf_attention_pages_workspace", "hf_pages_work_ints",
            "hf_pages_extend", "hf_pages_write", "hf_pages_fork", "hf_pages_truncate", "hf_pages_compact",
            "hf_verify_tokens", "hf_verify_workspace",
            "hf_attention_pages8", "hf_attention_pages8_workspace", "hf_pages8_work_ints", "hf_pages8_extend",
            "hf_pages8_fork", "hf_pages8_truncate", "hf_pages8_compact", "hf_pages8_write", "hf_pages8_read",
            "hf_rotary_table", "hf_rotary")


class HyflashError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = Status(status)
        super().__init__(f"{self.status.name}: {message}")


def make_config(shape, max_batch: int, prefill_tokens_max: int = 0) -> HfConfig:
    """HfConfig from any object with the drafter shape attributes."""
    return HfConfig(
        d_model=shape.d_model, n_q_heads=shape.n_q_heads, n_kv_heads=shape.n_kv_heads,
        head_dim=shape.head_dim, window=shape.window, block=shape.block,
        ssm_heads=shape.ssm_heads, ssm_headdim=shape.ssm_headdim, d_state=shape.d_state,
        n_groups=getattr(shape, "n_groups", 1), n_layers=shape.n_layers, max_batch=max_batch,
        chunk=getattr(shape, "chunk", 128),
        dtype=HF_F32 if shape.dtype in ("f32", "fp32", "float32") else HF_BF16,
        prefill_tokens_max=prefill_tokens_max,
        cross_slot_off=0 if getattr(shape, "cross_slot", True) else 1,
        mem_horizon=int(getattr(shape, "mem_horizon", 0) or 0),
        memory_kind=MEMORY_KINDS[getattr(shape, "memory", "mamba2") or "mamba2"],
        weight_bits=int(getattr(shape, "weight_bits", 16) or 16),
        block_kind=1 if getattr(shape, "full_block", False) else 0,
        mlp_dim=int(getattr(shape, "mlp_dim", 0) or 0) if getattr(shape, "full_block", False) else 0,
        vocab=int(getattr(shape, "vocab", 0) or 0) if getattr(shape, "full_block", False) else 0)


def _stream_ptr(stream) -> Optional[int]:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dev_ptr(t, dtype=None, shape=None, name="tensor"):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


class Drafter:
    """One library handle: windows, memories and weights of ``max_batch``
    requests on one GPU. Methods map one-to-one onto the C calls."""

    def __init__(self, shape, max_batch: int, device: int = 0, prefill_tokens_max: int = 0):
        import torch
        self.shape = shape
        self.max_batch = max_batch
        self.device = device
        self.cfg = make_config(shape, max_batch, prefill_tokens_max)
        self.torch_dtype = torch.float32 if self.cfg.dtype == HF_F32 else torch.bfloat16
        self.np_elem = 4 if self.cfg.dtype == HF_F32 else 2
        h = _h()
        s = hf_create(ctypes.byref(self.cfg), device, ctypes.byref(h))
        if s != 0:
            raise HyflashError(s, hf_last_error(None).decode())
        self._h = h

    # -- lifecycle
    def close(self):
        if getattr(self, "_h", None):
            hf_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, s):
        if s != 0:
            raise HyflashError(s, hf_last_error(self._h).decode())

    # -- weights
    def set_weights(self, layer: int, w):
        import torch
        keep = []
        lw = HfLayerWeights()
        for name in WEIGHT_FIELDS:
            t = getattr(w, name, None)
            if t is None:  # optional (w_beta outside the gated-delta memory)
                continue
            want = torch.float32 if name in ("dt_bias", "A_log") else self.torch_dtype
            t = t.detach().to("cpu", want).contiguous()
            keep.append(t)
            setattr(lw, name, t.data_ptr())
        self._check(hf_set_weights(self._h, layer, ctypes.byref(lw)))

    def _layer_struct(self, w, keep):
        import torch
        lw = HfLayerWeights()
        for name in WEIGHT_FIELDS:
            t = getattr(w, name, None)
            if t is None:  # optional (w_beta outside the gated-delta memory)
                continue
            want = torch.float32 if name in ("dt_bias", "A_log") else self.torch_dtype
            t = t.detach().to("cpu", want).contiguous()
            keep.append(t)
            setattr(lw, name, t.data_ptr())
        return lw

    def set_block_weights(self, layer: int, bw):
        """Full block: the layer's weights (bw.layer) and the parts around it."""
        import torch
        keep = []
        lw = self._layer_struct(bw.layer, keep)
        b = HfBlockWeights()
        for name in BLOCK_FIELDS:
            want = torch.float32 if name in BLOCK_F32 else self.torch_dtype
            t = getattr(bw, name).detach().to("cpu", want).contiguous()
            keep.append(t)
            setattr(b, name, t.data_ptr())
        self._check(hf_set_block_weights(self._h, layer, ctypes.byref(lw), ctypes.byref(b)))

    def set_head_weights(self, hw):
        import torch
        g = hw.g_final.detach().to("cpu", torch.float32).contiguous()
        w = hw.w_lm.detach().to("cpu", self.torch_dtype).contiguous()
        self._check(hf_set_head_weights(self._h, g.data_ptr(), w.data_ptr()))

    def draft_tokens(self, slot_emb, out=None, tokens=None, stream=None):
        """hf_draft_tokens: (hidden out [B, S, D], tokens int32 [B, S])."""
        import torch
        B = int(slot_emb.shape[0])
        shp = (B, self.shape.block, self.shape.d_model)
        sp = _dev_ptr(slot_emb, self.torch_dtype, shp, "slot_emb")
        if out is None:
            out = torch.empty(shp, dtype=self.torch_dtype, device=slot_emb.device)
        if tokens is None:
            tokens = torch.empty((B, self.shape.block), dtype=torch.int32, device=slot_emb.device)
        op = _dev_ptr(out, self.torch_dtype, shp, "out")
        tp = _dev_ptr(tokens, torch.int32, (B, self.shape.block), "tokens")
        self._check(hf_draft_tokens(self._h, sp, op, tp, B, _stream_ptr(stream)))
        return out, tokens

    def set_weights_q4(self, layer: int, w):
        """4-bit weights (weight_bits = 4): each matrix as codes uint8 [in, out],
        scales bf16 [in/128, out], zeros uint8 [in/128, out]."""
        import torch
        keep = []
        lw = HfLayerWeightsQ4()

        def host(t, dtype):
            t = t.detach().to("cpu", dtype).contiguous()
            keep.append(t)
            return t.data_ptr()

        for name in Q4_MATRICES:
            m = getattr(w, name, None)
            if m is None:
                continue
            q = getattr(lw, name)
            q.codes = host(m.codes, torch.uint8)
            q.scales = host(m.scales, torch.bfloat16)
            q.zeros = host(m.zeros, torch.uint8)
        lw.dt_bias = host(w.dt_bias, torch.float32)
        lw.A_log = host(w.A_log, torch.float32)
        self._check(hf_set_weights_q4(self._h, layer, ctypes.byref(lw)))

    # -- the three operations of the method
    def prefill(self, feats, lens: Sequence[int], requests: Optional[Sequence[int]] = None,
                stream=None):
        n = len(lens)
        la = (_i32 * max(n, 1))(*[int(x) for x in lens])
        ra = None
        if requests is not None:
            ra = (_i32 * max(n, 1))(*[int(x) for x in requests])
        total = int(sum(int(x) for x in lens))
        fp = _dev_ptr(feats, self.torch_dtype, (total, self.shape.d_model), "feats") if total else None
        self._check(hf_prefill(self._h, fp, la, ra, n, _stream_ptr(stream)))

    def commit(self, feats, n_accepted, stream=None):
        import torch
        B = int(n_accepted.shape[0])
        fp = _dev_ptr(feats, self.torch_dtype, (B, self.shape.block + 1, self.shape.d_model), "feats")
        npp = _dev_ptr(n_accepted, torch.int32, (B,), "n_accepted")
        self._check(hf_commit(self._h, fp, npp, B, _stream_ptr(stream)))

    def draft(self, slot_emb, out=None, stream=None):
        import torch
        B = int(slot_emb.shape[0])
        shp = (B, self.shape.block, self.shape.d_model)
        sp = _dev_ptr(slot_emb, self.torch_dtype, shp, "slot_emb")
        if out is None:
            out = torch.empty(shp, dtype=self.torch_dtype, device=slot_emb.device)
        op = _dev_ptr(out, self.torch_dtype, shp, "out")
        self._check(hf_draft(self._h, sp, op, B, _stream_ptr(stream)))
        return out

    def round(self, feats, n_accepted, slot_emb, out=None, stream=None):
        """hf_round: commit (feats, n_accepted), then draft slot_emb -> out."""
        import torch
        B = int(n_accepted.shape[0])
        if int(slot_emb.shape[0]) != B:
            raise ValueError("feats, n_accepted and slot_emb must have the same batch")
        fp = _dev_ptr(feats, self.torch_dtype, (B, self.shape.block + 1, self.shape.d_model), "feats")
        npp = _dev_ptr(n_accepted, torch.int32, (B,), "n_accepted")
        shp = (B, self.shape.block, self.shape.d_model)
        sp = _dev_ptr(slot_emb, self.torch_dtype, shp, "slot_emb")
        if out is None:
            out = torch.empty(shp, dtype=self.torch_dtype, device=slot_emb.device)
        op = _dev_ptr(out, self.torch_dtype, shp, "out")
        self._check(hf_round(self._h, fp, npp, sp, op, B, _stream_ptr(stream)))
        return out

    def sync(self, stream=None):
        self._check(hf_sync(self._h, _stream_ptr(stream)))

    def sync_status(self, stream=None):
        """hf_sync's status without raising: (status, message)."""
        s = hf_sync(self._h, _stream_ptr(stream))
        return Status(s), hf_last_error(self._h).decode()

    # -- inspection
    def tensor_bytes(self, which: int) -> int:
        n = ctypes.c_size_t()
        self._check(hf_tensor_bytes(self._h, int(which), ctypes.byref(n)))
        return n.value

    def read(self, which: int) -> np.ndarray:
        """Whole inspectable tensor as a NumPy array (bf16 returned as float32)."""
        nb = self.tensor_bytes(which)
        if nb == 0:  # memory-horizon rows of a handle without them
            return np.zeros((0,), dtype=np.float32)
        buf = np.empty(nb, dtype=np.uint8)
        self._check(hf_read_tensor(self._h, int(which), buf.ctypes.data, nb))
        sh, L, Bm = self.shape, self.shape.n_layers, self.max_batch
        which = Tensor(which)
        if which == Tensor.STATE:
            return buf.view(np.float32).reshape(L, Bm, sh.ssm_heads, sh.ssm_headdim, sh.d_state)
        if which in (Tensor.RING_K, Tensor.RING_V):
            a = self._model_to_f32(buf)
            return a.reshape(L, Bm, sh.n_kv_heads, sh.window, sh.head_dim)
        if which == Tensor.RING_TAG:
            return buf.view(np.int32).reshape(Bm, sh.window)
        if which == Tensor.POS:
            return buf.view(np.int64).copy()
        if which == Tensor.OFFSETS:
            return buf.view(np.int32).copy()
        if which == Tensor.DRAFT_PROJ:
            return buf.view(np.float32).reshape(Bm * sh.block, -1)
        if which == Tensor.CONV:
            return buf.view(np.float32).reshape(L, Bm, 3, -1)
        if which == Tensor.LOGITS:
            return buf.view(np.float32).reshape(Bm * sh.block, -1)
        if which in (Tensor.MEM_X, Tensor.MEM_B, Tensor.MEM_DT):
            R = int(getattr(sh, "mem_horizon", 0)) + sh.block + 1
            a = buf.view(np.float32)
            if which == Tensor.MEM_DT:
                return a.reshape(L, Bm, sh.ssm_heads, R)
            return a.reshape(L, Bm, R, -1)
        return self._model_to_f32(buf).reshape(Bm * sh.block, -1)

    def _model_to_f32(self, buf: np.ndarray) -> np.ndarray:
        if self.np_elem == 4:
            return buf.view(np.float32).copy()
        u = buf.view(np.uint16).astype(np.uint32) << 16
        return u.view(np.float32)

    def context_bytes(self) -> int:
        return int(hf_context_bytes(self._h))

    def export_context(self) -> bytes:
        n = self.context_bytes()
        buf = np.empty(n, dtype=np.uint8)
        self._check(hf_export_context(self._h, buf.ctypes.data, n))
        return buf.tobytes()

    def import_context(self, blob: bytes):
        buf = np.frombuffer(blob, dtype=np.uint8).copy()
        self._check(hf_import_context(self._h, buf.ctypes.data, buf.size))

    # -- measurement
    def profile(self, mode):
        """0 off, 1 (or True) per-call records, 2 records kept for graph replays."""
        self._check(hf_profile_enable(self._h, int(mode)))

    def profile_collect(self):
        self._check(hf_profile_collect(self._h))

    def profile_read(self, family: int, reset: bool = False):
        ms = ctypes.c_double()
        n = ctypes.c_int64()
        self._check(hf_profile_read(self._h, int(family), ctypes.byref(ms), ctypes.byref(n),
                                    1 if reset else 0))
        return ms.value, n.value

    def launch_count(self) -> int:
        return int(hf_launch_count(self._h))

    # -- failure detection (tests)
    def set_wait_limit(self, cycles: int):
        """Limit of the CUDA-core attention's ring-tile wait (-1: default)."""
        self._check(hf_debug_set_wait_limit(self._h, int(cycles)))

    def check_guards(self):
        """Raise if a guard region around one of the handle's buffers changed."""
        self._check(hf_debug_check_guards(self._h))


# ---------------------------------------------------------------- the target model's half of a round
class CallStatus(enum.IntFlag):
    """Bits that device checks set in a call's status word."""
    BAD = 1
    TIMEOUT = 2
    FULL = 4


_CODES = {}  # torch dtypes -> hf_dtype, filled at the first call


def _dtype_code(t, name):
    c = _CODES.get(t.dtype)
    if c is None:
        import torch
        _CODES.update({torch.float32: HF_F32, torch.bfloat16: HF_BF16})
        c = _CODES.get(t.dtype)
        if c is None:
            raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return c


class _On:
    """The device and stream of one call: every tensor lies on the first one's
    device; the call is made with that device current, on `stream` or the
    device's current stream. New outputs belong to the call's stream."""
    __slots__ = ("index", "first", "given", "ptr")

    def __init__(self, first, stream):
        import torch
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise TypeError("expected CUDA tensors")
        self.index = first.get_device()
        self.first = first
        self.given = stream
        if stream is None:
            self.ptr = torch._C._cuda_getCurrentRawStream(self.index)
        else:
            self.ptr = stream if isinstance(stream, int) else stream.cuda_stream

    def arg(self, t, name, dtype=None, shape=None, contiguous=True):
        # (one test for the tensors that are right: a small call is bound by these checks)
        if (t.get_device() == self.index and (dtype is None or t.dtype is dtype)
                and (shape is None or t.shape == shape) and (not contiguous or t.is_contiguous())):
            return t.data_ptr()
        if t.get_device() != self.index:
            raise TypeError(f"{name} must be a CUDA tensor on cuda:{self.index}")
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")

    def zeros(self, shape, dtype):
        return self.empty(shape, dtype, "zeros")

    def empty(self, shape, dtype, kind="empty"):
        if self.given is None:
            return getattr(self.first, "new_" + kind)(shape, dtype=dtype)
        import torch
        s = self.given
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=self.index)
        with torch.cuda.stream(s):
            return getattr(torch, kind)(shape, dtype=dtype, device=self.index)

    def call(self, f, *args):
        import torch
        if torch._C._cuda_getDevice() == self.index:
            s = f(*args, self.ptr)
        else:
            with torch.cuda.device(self.index):
                s = f(*args, self.ptr)
        if s != 0:
            raise HyflashError(s, hf_last_error(None).decode())


def _heads_ld(t, n, h, d, name):
    """Row stride of [..., n, h heads, d] whose heads follow each other."""
    s = t.stride()
    if (s[-1] != 1 and d > 1) or (s[-2] != d and h > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return s[-3] if n > 1 else h * d


def attention_prompt(q, k, v, offsets, *, scale=0.0, out=None, status=None, stream=None):
    """hf_attention_prompt: causal attention over packed prompts. q [T, Hq, dh],
    k and v [T, Hkv, dh] (row strides are free: parts of one projection will do),
    offsets int32 [n + 1]. Returns out [T, Hq, dh]; rows outside every sequence keep
    what `out` held."""
    import torch
    on = _On(q, stream)
    if q.dim() != 3 or k.dim() != 3 or offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("q, k and v must be [tokens, heads, head_dim], offsets [sequences + 1]")
    T, hq, dh = q.shape
    hkv = k.shape[1]
    dt, kv = q.dtype, (T, hkv, dh)
    code = _dtype_code(q, "q")
    kp = on.arg(k, "k", dt, kv, False)
    vp = on.arg(v, "v", dt, kv, False)
    op = on.arg(offsets, "offsets", torch.int32)
    if out is None:
        out = on.empty((T, hq, dh), dt)
    rp = on.arg(out, "out", dt, q.shape, False)
    sp = None if status is None else on.arg(status, "status", torch.int32)
    on.call(hf_attention_prompt, code, offsets.shape[0] - 1, T, hq, hkv, dh, q.data_ptr(), _heads_ld(q, T, hq, dh, "q"),
            kp, _heads_ld(k, T, hkv, dh, "k"), vp, _heads_ld(v, T, hkv, dh, "v"), op, scale or 0.0, rp,
            _heads_ld(out, T, hq, dh, "out"), sp)
    return out


def verify_workspace(target_logits, draft_logits=None):
    """A workspace for verify_tokens with logits of these sizes."""
    import torch
    B, S1, V = target_logits.shape
    n = hf_verify_workspace(B, S1 - 1, V)
    if n == 0:
        raise ValueError("verify_workspace: sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=target_logits.device)


def verify_tokens(target_logits, draft_tokens, u, noise, *, draft_logits=None, temperature=None, n_draft=None,
                  n_accepted=None, tokens=None, workspace=None, status=None, stream=None):
    """hf_verify_tokens: (n_accepted int32 [B], tokens int32 [B, S + 1]) from the
    target's logits [B, S + 1, V] and the drafts int32 [B, S]; u [B, S] uniform and
    noise [B, V] exponential random numbers. n_accepted is what Drafter.commit takes."""
    import torch
    on = _On(target_logits, stream)
    if target_logits.dim() != 3 or target_logits.shape[1] < 2:
        raise ValueError("target_logits must be [batch, block + 1, vocab]")
    B, S, V = target_logits.shape
    S -= 1

    def rows(t, name, n):
        if t.is_contiguous():
            return V
        s = t.stride()
        if (s[2] != 1 and V > 1) or (B > 1 and n > 1 and s[0] != n * s[1]):
            raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
        ld = s[1] if n > 1 else s[0] if B > 1 else V
        if B and ld < V:
            raise ValueError(f"{name}: rows must not overlap")
        return max(ld, V)

    f32, i32 = torch.float32, torch.int32
    batch, slots, drafts = (B,), (B, S + 1), (B, S)
    t_ld = rows(target_logits, "target_logits", S + 1)
    dp, d_ld, d_code = None, 0, 0
    if draft_logits is not None:
        dp = on.arg(draft_logits, "draft_logits", None, (B, S, V), False)
        d_ld = rows(draft_logits, "draft_logits", S)
        d_code = _dtype_code(draft_logits, "draft_logits")
    kp = on.arg(draft_tokens, "draft_tokens", i32, drafts)
    up = on.arg(u, "u", f32, drafts)
    ep = on.arg(noise, "noise", f32, (B, V))
    np_ = None if n_draft is None else on.arg(n_draft, "n_draft", i32, batch)
    hp = None if temperature is None else on.arg(temperature, "temperature", f32, batch)
    if n_accepted is None:
        n_accepted = on.empty(batch, i32)
    if tokens is None:
        tokens = on.empty(slots, i32)
    if workspace is None:
        workspace = on.empty((max(hf_verify_workspace(B, S, V), 16),), torch.uint8)
    on.call(hf_verify_tokens, _dtype_code(target_logits, "target_logits"), target_logits.data_ptr(), t_ld, d_code, dp,
            d_ld, kp, np_, up, ep, V, hp, B, S, V, on.arg(n_accepted, "n_accepted", i32, batch),
            on.arg(tokens, "tokens", i32, slots), on.arg(workspace, "workspace", torch.uint8), workspace.shape[0],
            None if status is None else on.arg(status, "status", i32))
    return n_accepted, tokens


class Pages:
    """A paged key/value cache of the target over the caller's tensors (hf_pages):
    k and v [layers, pages, kv heads, page, head_dim], table int32 [requests,
    columns], lens int32 [requests], refs int32 [pages]. Methods map one-to-one
    onto the C calls; ``status`` is the word their device checks write to."""

    _C = dict(work=hf_pages_work_ints, extend=hf_pages_extend, truncate=hf_pages_truncate, fork=hf_pages_fork,
              compact=hf_pages_compact, write=hf_pages_write, attend=hf_attention_pages,
              attend_workspace=hf_attention_pages_workspace)

    def __init__(self, k, v, table, lens, refs):
        self._setup(k, v, table, lens, refs, HfPages(dtype=_dtype_code(k, "k")), k.dtype)

    def _setup(self, k, v, table, lens, refs, d, rows, wrap=lambda on, d: d):
        """Fill the descriptor d in; rows: the type of rows, q and out; wrap(on, d): what the calls take."""
        import torch
        on = _On(k, None)
        if k.dim() != 5 or table.dim() != 2:
            raise ValueError("k must be [layers, pages, kv heads, page, head_dim], table [requests, columns]")
        L, n, hkv, page, dh = k.shape
        R, ld = table.shape
        i32 = torch.int32
        d.n_layers, d.n_pages, d.n_kv_heads, d.page, d.head_dim, d.n_requests, d.table_ld = L, n, hkv, page, dh, R, ld
        d.k = on.arg(k, "k")
        d.v = on.arg(v, "v", k.dtype, tuple(k.shape))
        d.table = on.arg(table, "table", i32)
        d.lens = on.arg(lens, "lens", i32, (R,))
        d.refs = on.arg(refs, "refs", i32, (n,))
        call = wrap(on, d)
        ints = self._C["work"](ctypes.byref(call))
        self.k, self.v, self.table, self.lens, self.refs = k, v, table, lens, refs
        # scratch of the page calls, and the status word
        self._work = torch.zeros(max(ints, 1), dtype=i32, device=k.device)
        self.status = torch.zeros(1, dtype=i32, device=k.device)
        base = call if call is d else call.pages
        base.work, base.status = self._work.data_ptr(), self.status.data_ptr()
        self._d, self._keep, self._ref = base, call, ctypes.byref(call)
        self._i32, self._index, self._dtype, self._layers, self._row = i32, k.get_device(), rows, L, (hkv, dh)
        self._u8 = torch.uint8
        self._raw_stream, self._current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        with torch.cuda.device(self._index):
            if not torch.cuda.is_current_stream_capturing():  # calls may come on any stream: both are zero by now
                torch.cuda.current_stream().synchronize()
        if ints == 0:  # let a call say what is wrong with the descriptor
            on.call(self._C["compact"], self._ref, None)

    @classmethod
    def empty(cls, n_layers, n_pages, n_kv_heads, page, head_dim, n_requests, columns, dtype=None, device="cuda"):
        """A new cache that holds no request."""
        import torch
        shape = (n_layers, n_pages, n_kv_heads, page, head_dim)
        k = torch.empty(shape, dtype=dtype or torch.bfloat16, device=device)
        ints = dict(dtype=torch.int32, device=device)
        return cls(k, torch.empty_like(k), torch.full((n_requests, columns), -1, **ints),
                   torch.zeros(n_requests, **ints), torch.zeros(n_pages, **ints))

    def check(self):
        """Read and clear the status word. Waits for the device: for calls on every stream."""
        import torch
        torch.cuda.synchronize(self._index)
        s = CallStatus(int(self.status.item()))
        if s:
            self.status.zero_()
            torch.cuda.synchronize(self._index)  # before a call on another stream writes to it
        return s

    def _ints(self, t, n, name):
        """Pointer of an int32 list of n entries on the cache's device."""
        if t is None:
            return None
        if t.dtype is not self._i32 or t.get_device() != self._index or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on cuda:{self._index}")
        return t.data_ptr()

    def _call(self, f, stream, *args):
        if stream is None:
            stream = self._raw_stream(self._index)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        if self._current() == self._index:
            s = f(self._ref, *args, stream)
        else:
            import torch
            with torch.cuda.device(self._index):
                s = f(self._ref, *args, stream)
        if s != 0:
            raise HyflashError(s, hf_last_error(None).decode())

    def extend(self, counts, requests=None, stream=None):
        """Room for counts[i] more tokens of requests[i] (default: request i)."""
        n = counts.shape[0]
        self._call(self._C["extend"], stream, self._ints(requests, n, "requests"), self._ints(counts, n, "counts"), n)

    def truncate(self, keep, requests=None, stream=None):
        """Cut requests[i] to keep[i] tokens; 0 frees it."""
        n = keep.shape[0]
        self._call(self._C["truncate"], stream, self._ints(requests, n, "requests"), self._ints(keep, n, "keep"), n)

    def fork(self, source, into, stream=None):
        """Requests into[i] (empty) share all tokens of source[i]."""
        n = into.shape[0]
        self._call(self._C["fork"], stream, self._ints(source, n, "source"), self._ints(into, n, "into"), n)

    def compact(self, n_used=None, stream=None):
        """Move the pages in use to the front of the pool; n_used int32 [1] receives
        their number."""
        self._call(self._C["compact"], stream, self._ints(n_used, 1, "n_used"))

    def _rows(self, k, v, layer):
        """Layers, tokens, row and layer stride of rows k and v."""
        shape, ks, vs = k.shape, k.stride(), v.stride()
        if (len(shape) != (4 if layer is None else 3) or shape[-2:] != self._row
                or (layer is None and shape[0] > self._layers)):
            raise ValueError("k must be [layers, tokens, kv heads, head_dim], or [tokens, kv heads, head_dim] with layer")
        i, dt = self._index, self._dtype
        if k.dtype is not dt or v.dtype is not dt or k.get_device() != i or v.get_device() != i:
            raise TypeError(f"k and v must be {dt} on cuda:{i}")
        T, (hkv, dh) = shape[-3], self._row
        ld = ks[-3] if T > 1 and ks[-1] == 1 and ks[-2] == dh else _heads_ld(k, T, hkv, dh, "k")
        layers = shape[0] if layer is None else 1
        step = ks[0] if layers > 1 else 0
        if v.shape != shape or (T and vs != ks and (_heads_ld(v, T, hkv, dh, "v") != ld or (layers > 1 and vs[0] != step))):
            raise ValueError("k and v must have the same shape and strides")
        return layers, T, ld, step

    def write(self, k, v, offsets, requests=None, layer=None, stream=None):
        """The newest rows of the requests: k and v [layers, T, kv heads, head_dim]
        for layers 0 .. layers - 1, or [T, kv heads, head_dim] with `layer`; entry i's
        rows are offsets[i] .. offsets[i + 1] - 1."""
        layers, T, ld, step = self._rows(k, v, layer)
        n = offsets.shape[0] - 1
        self._call(self._C["write"], stream, layer or 0, layers, k.data_ptr(), v.data_ptr(),
                   ld, step, self._ints(requests, n, "requests"), self._ints(offsets, n + 1, "offsets"), n, T)

    def attend_workspace(self, q, shared=0):
        """A workspace for attend with queries of this shape."""
        import torch
        n, rows, hq, _ = q.shape
        b = self._C["attend_workspace"](self._ref, n, rows, hq, shared)
        if b == 0:
            raise ValueError("attend_workspace: sizes out of range")
        return torch.empty(b, dtype=torch.uint8, device=self.k.device)

    def attend(self, q, requests=None, *, layer=0, shared=0, scale=0.0, out=None, workspace=None, stream=None):
        """hf_attention_pages: q [n, rows, Hq, dh] are the newest `rows` tokens of the
        requests; returns out of the same shape."""
        shape = q.shape
        if len(shape) != 4 or shape[3] != self._row[1]:
            raise ValueError("q must be [requests, rows, heads, head_dim]")
        n, rows, hq, dh = shape
        dt, i = self._dtype, self._index
        if out is None or workspace is None:
            on = _On(self.k, stream)
            if out is None:
                out = on.empty(tuple(shape), dt)
            if workspace is None:
                workspace = on.empty((max(self._C["attend_workspace"](self._ref, n, rows, hq, shared), 16),), self._u8)
        # (one test for the tensors that are right: a small call is bound by these checks)
        if (q.dtype is not dt or out.dtype is not dt or q.get_device() != i or out.get_device() != i or out.shape != shape
                or workspace.dtype is not self._u8 or workspace.get_device() != i or not workspace.is_contiguous()):
            on = _On(self.k, stream)
            for t, name in ((q, "q"), (out, "out")):
                on.arg(t, name, dt, shape, False)
            on.arg(workspace, "workspace", self._u8)

        def ld(t, name):
            s = t.stride()
            if s[3] == 1 and s[2] == dh and (n == 1 or rows == 1 or s[0] == rows * s[1]):
                return s[1] if rows > 1 else s[0] if n > 1 else hq * dh
            r = _heads_ld(t, rows, hq, dh, name)
            if rows == 1 and n > 1:
                r = s[0]
            elif n > 1 and s[0] != rows * r:
                raise ValueError(f"{name}: its rows must be evenly spaced")
            return r

        self._call(self._C["attend"], stream, layer, n, rows, hq, q.data_ptr(), ld(q, "q"), self._ints(requests, n, "requests"),
                   shared, scale or 0.0, out.data_ptr(), ld(out, "out"), workspace.data_ptr(), workspace.shape[0])
        return out


class Pages8(Pages):
    """The cache in 8 bits (hf_pages8): k and v float8_e4m3fn [layers, pages, kv heads,
    page, head_dim], k_scale and v_scale float32 [layers, pages, kv heads], rows, queries
    and outputs of `dtype`. The methods of Pages; `write` quantises."""

    _C = dict(work=hf_pages8_work_ints, extend=hf_pages8_extend, truncate=hf_pages8_truncate, fork=hf_pages8_fork,
              compact=hf_pages8_compact, write=hf_pages8_write, attend=hf_attention_pages8,
              attend_workspace=hf_attention_pages8_workspace)

    def __init__(self, k, v, k_scale, v_scale, table, lens, refs, dtype=None):
        import torch
        dtype = dtype or torch.bfloat16
        if k.dtype is not torch.float8_e4m3fn:
            raise TypeError(f"k must be float8_e4m3fn, got {k.dtype}")
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")

        def wrap(on, d):
            f32, shape = torch.float32, tuple(k.shape[:3])
            return HfPages8(pages=d, k_scale=on.arg(k_scale, "k_scale", f32, shape),
                            v_scale=on.arg(v_scale, "v_scale", f32, shape),
                            rows=HF_F32 if dtype is f32 else HF_BF16)

        self.k_scale, self.v_scale = k_scale, v_scale
        self._setup(k, v, table, lens, refs, HfPages(dtype=HF_E4M3), dtype, wrap)

    @classmethod
    def empty(cls, n_layers, n_pages, n_kv_heads, page, head_dim, n_requests, columns, dtype=None, device="cuda"):
        """A new cache that holds no request; dtype: of the rows."""
        import torch
        shape = (n_layers, n_pages, n_kv_heads, page, head_dim)
        k = torch.empty(shape, dtype=torch.float8_e4m3fn, device=device)
        scale = torch.ones(shape[:3], dtype=torch.float32, device=device)
        ints = dict(dtype=torch.int32, device=device)
        return cls(k, torch.empty_like(k), scale, torch.ones_like(scale),
                   torch.full((n_requests, columns), -1, **ints), torch.zeros(n_requests, **ints),
                   torch.zeros(n_pages, **ints), dtype)

    def read(self, first, offsets, requests=None, layer=None, *, total=None, k=None, v=None, stream=None):
        """Tokens as rows: entry i's rows offsets[i] .. offsets[i + 1] - 1 of k and v become the
        tokens of requests[i] from first[i] on, in all layers, or in `layer`. k and v (or
        `total`, the rows of new ones, zeros where no entry writes) [layers, T, kv heads, head_dim],
        without the first dim if `layer` is given. Returns them."""
        if (k is None) != (v is None) or (k is None) == (total is None):
            raise ValueError("give k and v, or total")
        if k is None:
            shape = (total, *self._row) if layer is not None else (self._layers, total, *self._row)
            on = _On(self.k, stream)
            k, v = on.zeros(shape, self._dtype), on.zeros(shape, self._dtype)
        layers, T, ld, step = self._rows(k, v, layer)
        n = offsets.shape[0] - 1
        self._call(hf_pages8_read, stream, layer or 0, layers, k.data_ptr(), v.data_ptr(), ld, step,
                   self._ints(requests, n, "requests"), self._ints(first, n, "first"),
                   self._ints(offsets, n + 1, "offsets"), n, T)
        return k, v


class Rotary:
    """Rotary positions of queries and keys (hf_rotary): the table of a head of `head_dim`
    columns, the first `dim` of them turned (default: all), pairs (i, i + dim/2) or, interleaved,
    (2i, 2i + 1). scaling: "none", "linear", "ntk", "yarn" or "bands" with their factor, original,
    fast, slow and attention (hf_rotary_table)."""

    def __init__(self, head_dim, base=1e6, dim=None, interleaved=False, scaling="none", factor=1.0, original=0, fast=0.0,
                 slow=0.0, attention=0.0, device="cuda"):
        import torch
        if scaling not in ROTARY_SCALING:
            raise ValueError(f"scaling must be one of {', '.join(ROTARY_SCALING)}")
        self.head_dim, self.dim, self.interleaved = head_dim, dim if dim is not None else head_dim, bool(interleaved)
        if self.dim > head_dim:
            raise ValueError("dim must be at most head_dim")
        host = np.zeros(max(self.dim // 2, 1), dtype=np.uint64)
        s = HfRotaryScaling(kind=ROTARY_SCALING[scaling], original=original, factor=factor, fast=fast, slow=slow,
                            attention=attention)
        f = ctypes.c_float()
        e = hf_rotary_table(self.dim, base, ctypes.byref(s), host.ctypes.data, ctypes.byref(f))
        if e != 0:
            raise HyflashError(e, hf_last_error(None).decode())
        self.attention = f.value
        self.turns = torch.from_numpy(host.view(np.int64)).to(device)  # w_i / (2 pi) in 2^-64 turns, unsigned
        if self.turns.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.turns.device).synchronize()  # calls may come on any stream
        self._index, self._turns, self._inter, self._i32 = self.turns.get_device(), self.turns.data_ptr(), int(self.interleaved), torch.int32
        self._raw_stream, self._current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

    def __call__(self, q, k, positions, *, q_out=None, k_out=None, stream=None):
        """q [T, Hq, dh] and k [T, Hkv, dh] (or None) turned by positions int32 [T]: into q_out and
        k_out, which may be q and k, or new tensors. Row strides are free. Returns (q_out, k_out)."""
        shape, i, dt = q.shape, q.get_device(), q.dtype
        if i < 0 or i != self._index:
            raise TypeError(f"q must be a CUDA tensor on the table's device ({self.turns.device})")
        if len(shape) != 3 or shape[2] != self.head_dim or (k is not None and k.dim() != 3):
            raise ValueError("q and k must be [tokens, heads, head_dim]")
        T, hq, dh = shape
        code = _dtype_code(q, "q")
        if (positions.dtype is not self._i32 or positions.get_device() != i or positions.shape != (T,)
                or not positions.is_contiguous()):
            raise ValueError(f"positions must be a contiguous int32 tensor of {T} entries on cuda:{i}")

        def ld(t, name, shape):
            # (one test for the tensors that are right: a small call is bound by these checks)
            s = t.stride()
            if t.dtype is dt and t.get_device() == i and t.shape == shape and s[2] == 1 and s[1] == dh:
                return s[0] if T > 1 else shape[1] * dh
            if t.dtype is not dt or t.get_device() != i:
                raise TypeError(f"{name} must be {dt} on cuda:{i}")
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
            return _heads_ld(t, T, shape[1], dh, name)

        if q_out is None or (k is not None and k_out is None):
            on = _On(q, stream)
            q_out = on.empty(tuple(shape), dt) if q_out is None else q_out
            k_out = on.empty((T, k.shape[1], dh), dt) if k is not None and k_out is None else k_out
        if k is None:
            hkv, kp, k_ld, ko, ko_ld = 0, None, 0, None, 0
        else:
            hkv = k.shape[1]
            kv = (T, hkv, dh)
            kp, k_ld, ko, ko_ld = k.data_ptr(), ld(k, "k", kv), k_out.data_ptr(), ld(k_out, "k_out", kv)
        args = (code, self._inter, T, hq, hkv, dh, self.dim, self._turns, self.attention, positions.data_ptr(), q.data_ptr(),
                ld(q, "q", shape), kp, k_ld, q_out.data_ptr(), ld(q_out, "q_out", shape), ko, ko_ld)
        if stream is None:
            stream = self._raw_stream(i)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        if self._current() == i:
            e = hf_rotary(*args, stream)
        else:
            import torch
            with torch.cuda.device(i):
                e = hf_rotary(*args, stream)
        if e != 0:
            raise HyflashError(e, hf_last_error(None).decode())
        return q_out, k_out
