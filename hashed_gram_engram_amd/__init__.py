"""Python binding of libengram.so, the MI355X (gfx950) Engram forward library.

The functions here carry the C ABI's names (include/engram.h) and only marshal arguments:
torch tensors provide device memory, the current torch stream provides the HIP stream, and
every step of the computation runs in the library's HIP kernels.  If the shared library is
missing, importing the binding raises: there is no fallback path.
"""
from __future__ import annotations

import atexit
import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libengram.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                      "(hipcc --offload-arch=gfx950)")

_lib = ctypes.CDLL(LIB_PATH)

ENGRAM_OK = 0
ENGRAM_E_TIMEOUT = -8
ENGRAM_E_WORKSPACE = -5
STATUS = {0: "ok", -1: "null pointer", -2: "layout", -3: "shape", -4: "alignment",
          -5: "workspace", -6: "hip", -7: "device", -8: "timeout"}


class EngramLayout(ctypes.Structure):
    _fields_ = [("hc", ctypes.c_int32), ("dim", ctypes.c_int32), ("n_cols", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("scale_block", ctypes.c_int32),
                ("scale_format", ctypes.c_int32), ("wkv_format", ctypes.c_int32),
                ("n_rows", ctypes.c_int64), ("eps", ctypes.c_float), ("clamp", ctypes.c_float)]


class HashLayout(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("max_ngram", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("pad_id", ctypes.c_int32), ("vocab", ctypes.c_int64),
                ("history_len", ctypes.c_int64)]


class PageLayout(ctypes.Structure):
    _fields_ = [("block_size", ctypes.c_int32), ("max_blocks", ctypes.c_int32), ("n_blocks", ctypes.c_int64)]


class _PlanOut(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("token_start", "start_pos", "seq_lens", "status", "free_left", "slots",
                                                     "positions", "requests", "live")]


class NormLayout(ctypes.Structure):
    _fields_ = [("hc", ctypes.c_int32), ("dim", ctypes.c_int32), ("y_streams", ctypes.c_int32),
                ("stream_format", ctypes.c_int32), ("gate", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("pre_norm", ctypes.c_int32), ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("post_eps", ctypes.c_float), ("pre_eps", ctypes.c_float)]


class LinearLayout(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("glu", ctypes.c_int32), ("stream_format", ctypes.c_int32)]


class LatentLayout(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("cache_format", ctypes.c_int32), ("window", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class EngramError(RuntimeError):
    def __init__(self, where: str, status: int):
        msg = _lib.engram_status_str(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_LP = ctypes.POINTER(EngramLayout)
_lib.engram_status_str.restype = ctypes.c_char_p
_lib.engram_status_str.argtypes = [ctypes.c_int]
_lib.engram_layout_check.argtypes = [_LP]
_lib.engram_param_counts.argtypes = [_LP, ctypes.POINTER(ctypes.c_int64)]
_lib.engram_forward_workspace_bytes.argtypes = [_LP, _i64, _i64]
_lib.engram_forward_workspace_bytes.restype = _sz
_lib.engram_forward_staging_bytes.argtypes = [_LP, _i64, _i64]
_lib.engram_forward_staging_bytes.restype = _sz
_lib.engram_gather_dequant.argtypes = [_LP, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp]
_lib.engram_kv_proj.argtypes = [_LP, _vp, _vp, _i64, _i64, _vp, _vp]
_lib.engram_gate_apply.argtypes = [_LP, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp]
_lib.engram_forward.argtypes = [_LP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp,
                                _sz, _vp, _vp]
_lib.engram_hash_ids.argtypes = [ctypes.POINTER(HashLayout), _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                 _i64, _i64, _vp, _vp, _vp, _vp]
_lib.engram_forward_noalloc.argtypes = [_LP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp]
_lib.engram_forward_noalloc.restype = ctypes.c_int
_lib.engram_forward_check.argtypes = [_vp, _sz, _vp]
_lib.engram_set_spin_budget.argtypes = [ctypes.c_uint32]
_lib.engram_set_spin_budget.restype = ctypes.c_uint32
_lib.engram_batch_plan.argtypes = [ctypes.POINTER(PageLayout), _vp, _vp, _i64, _vp, _vp, _vp, _i64,
                                   ctypes.POINTER(_PlanOut), _vp, _vp]
_lib.engram_hash_ids_paged.argtypes = [ctypes.POINTER(HashLayout), ctypes.POINTER(PageLayout), _vp, _vp, _vp, _vp, _vp, _vp,
                                       _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp]
_lib.engram_residual_norm.argtypes = [ctypes.POINTER(NormLayout), _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp,
                                      _vp, _vp]
_lib.engram_linear.argtypes = [ctypes.POINTER(LinearLayout), _vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _sz, _vp]
_lib.engram_linear_workspace_bytes.argtypes = [ctypes.POINTER(LinearLayout), _i64]
_lib.engram_linear_workspace_bytes.restype = _sz
_lib.engram_linear_workspace_bytes_up_to.argtypes = [ctypes.POINTER(LinearLayout), _i64]
_lib.engram_linear_workspace_bytes_up_to.restype = _sz
_lib.engram_page_layout_check.argtypes = [ctypes.POINTER(PageLayout)]
_lib.engram_norm_layout_check.argtypes = [ctypes.POINTER(NormLayout)]
_lib.engram_linear_layout_check.argtypes = [ctypes.POINTER(LinearLayout)]
_LL = ctypes.POINTER(LatentLayout)
_lib.engram_latent_layout_check.argtypes = [_LL]
_lib.engram_latent_row_bytes.argtypes = [_LL]
_lib.engram_latent_write.argtypes = [_LL, ctypes.POINTER(PageLayout), _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp]
_lib.engram_latent_read.argtypes = [_LL, ctypes.POINTER(PageLayout), _vp, _vp, _vp, _i64, _vp, _i64, _i32, _i64, _vp, _vp, _vp, _vp,
                                    _vp]
_lib.engram_latent_attention.argtypes = [_LL, ctypes.POINTER(PageLayout), _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _i32, _vp, _i64,
                                         _vp, _vp, _sz, _vp, _vp]
_lib.engram_latent_attention_expanded.argtypes = [_LL, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i32, _vp,
                                                  _i64, _vp, _vp, _sz, _vp]
_lib.engram_latent_attention_workspace_bytes.argtypes = [_LL]
_lib.engram_latent_attention_expanded_workspace_bytes.argtypes = [_LL, _i64, _i64, _i64]
_lib.engram_latent_attention_expanded_workspace_bytes_up_to.argtypes = [_LL, _i64, _i64]
for _f in (_lib.engram_latent_row_bytes, _lib.engram_latent_attention_workspace_bytes,
           _lib.engram_latent_attention_expanded_workspace_bytes, _lib.engram_latent_attention_expanded_workspace_bytes_up_to):
    _f.restype = _sz
for _f in (_lib.engram_latent_layout_check, _lib.engram_latent_write, _lib.engram_latent_read, _lib.engram_latent_attention,
           _lib.engram_latent_attention_expanded):
    _f.restype = ctypes.c_int
for _f in (_lib.engram_batch_plan, _lib.engram_hash_ids_paged, _lib.engram_residual_norm, _lib.engram_linear,
           _lib.engram_page_layout_check, _lib.engram_norm_layout_check, _lib.engram_linear_layout_check):
    _f.restype = ctypes.c_int
for _f in (_lib.engram_layout_check, _lib.engram_param_counts, _lib.engram_gather_dequant,
           _lib.engram_kv_proj, _lib.engram_gate_apply, _lib.engram_forward, _lib.engram_hash_ids,
           _lib.engram_forward_check):
    _f.restype = ctypes.c_int

EXPORTED = ["engram_layout_check", "engram_param_counts", "engram_forward_workspace_bytes",
            "engram_forward_staging_bytes",
            "engram_gather_dequant", "engram_kv_proj", "engram_gate_apply", "engram_forward",
            "engram_hash_ids", "engram_status_str", "engram_forward_check", "engram_set_spin_budget",
            "engram_forward_noalloc", "engram_batch_plan", "engram_hash_ids_paged", "engram_residual_norm",
            "engram_linear", "engram_linear_workspace_bytes", "engram_linear_workspace_bytes_up_to",
            "engram_page_layout_check", "engram_norm_layout_check", "engram_linear_layout_check",
            "engram_latent_layout_check", "engram_latent_row_bytes", "engram_latent_write", "engram_latent_read",
            "engram_latent_attention", "engram_latent_attention_workspace_bytes", "engram_latent_attention_expanded",
            "engram_latent_attention_expanded_workspace_bytes", "engram_latent_attention_expanded_workspace_bytes_up_to"]


SCALE_FP32, SCALE_E8M0 = 0, 1  # engram_scale_format
WKV_BF16, WKV_MXFP8 = 0, 1     # engram_wkv_format


def make_layout(hc: int, dim: int, n_cols: int, head_dim: int, scale_block: int, n_rows: int,
                eps: float = 1e-20, clamp: float = 1e-6, scale_format: int = SCALE_FP32,
                wkv_format: int = WKV_BF16) -> EngramLayout:
    return EngramLayout(hc, dim, n_cols, head_dim, scale_block, scale_format, wkv_format, n_rows,
                        eps, clamp)


def wkv_bytes(layout: EngramLayout) -> int:
    """Bytes of the wkv argument: N x K bf16, or for MXFP8 the codes [N, K] followed by the
    E8M0 scales [N, K / 32] in one uint8 buffer."""
    n, k = (layout.hc + 1) * layout.dim, layout.n_cols * layout.head_dim
    return n * k + n * (k // 32) if layout.wkv_format == WKV_MXFP8 else 2 * n * k


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(where: str, st: int):
    if st != ENGRAM_OK:
        raise EngramError(where, st)


def _contig(name: str, t: torch.Tensor, dtype=None) -> torch.Tensor:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t


_BF16 = (torch.bfloat16, torch.int16)


# The library takes plain pointers and cannot see buffer sizes: every tensor's shape (or size) is
# checked here against the layout, so that a mismatch raises instead of reading or writing past
# a buffer on the device.
def _shape(name: str, t: torch.Tensor, shape: tuple):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _numel(name: str, t: torch.Tensor, shape: tuple):
    """t holds exactly the elements of `shape` (in any shape: the library sees a flat buffer)."""
    need = math.prod(shape)
    if t.numel() != need:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {need} elements {tuple(shape)}")


def _nbytes(name: str, t: torch.Tensor, need: int, exact: bool = True):
    have = t.numel() * t.element_size()
    if (have != need) if exact else (have < need):
        raise ValueError(f"{name} holds {have} bytes, expected {'' if exact else 'at least '}{need}")


def _same_device(ref: torch.Tensor, **ts):
    dev = ref.device
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {dev}")
    for name, t in ts.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _dims(layout: EngramLayout):
    """(K, N, scale bytes per table row) of a layout."""
    k, n = layout.n_cols * layout.head_dim, (layout.hc + 1) * layout.dim
    nb = layout.head_dim // layout.scale_block if layout.scale_block > 0 else 0
    return k, n, nb * (1 if layout.scale_format == SCALE_E8M0 else 4)


def _check_table(layout: EngramLayout, table: torch.Tensor, scales: torch.Tensor):
    _, _, sbytes = _dims(layout)
    _nbytes("table", table, layout.n_rows * layout.head_dim, exact=False)
    _nbytes("scales", scales, layout.n_rows * sbytes, exact=False)


def _check_err(err_count: Optional[torch.Tensor]):
    if err_count is not None:
        _contig("err_count", err_count, torch.int32)
        if err_count.numel() < 1:
            raise ValueError("err_count needs one int32")


def _check_wkv(layout: EngramLayout, wkv: torch.Tensor):
    _contig("wkv", wkv, torch.uint8 if layout.wkv_format == WKV_MXFP8 else _BF16)
    if wkv.numel() * wkv.element_size() != wkv_bytes(layout):
        raise ValueError(f"wkv holds {wkv.numel() * wkv.element_size()} bytes, the layout needs "
                         f"{wkv_bytes(layout)}")


def engram_layout_check(layout: EngramLayout) -> int:
    return _lib.engram_layout_check(ctypes.byref(layout))


def engram_param_counts(layout: EngramLayout):
    out = (ctypes.c_int64 * 3)()
    _check("engram_param_counts", _lib.engram_param_counts(ctypes.byref(layout), out))
    return int(out[0]), int(out[1]), int(out[2])


def engram_forward_workspace_bytes(layout: EngramLayout, B: int, T: int) -> int:
    return int(_lib.engram_forward_workspace_bytes(ctypes.byref(layout), B, T))


def engram_forward_staging_bytes(layout: EngramLayout, B: int, T: int) -> int:
    return int(_lib.engram_forward_staging_bytes(ctypes.byref(layout), B, T))


def engram_gather_dequant(layout: EngramLayout, table: torch.Tensor, scales: torch.Tensor,
                          hash_ids: torch.Tensor, emb: Optional[torch.Tensor] = None,
                          err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """emb [B, T, n_cols * head_dim] bf16 from hash_ids [B, T, n_cols] int64."""
    if hash_ids.dim() != 3:
        raise ValueError(f"hash_ids has shape {tuple(hash_ids.shape)}, expected [B, T, n_cols]")
    B, T, C = hash_ids.shape
    _shape("hash_ids", hash_ids, (B, T, layout.n_cols))
    _contig("hash_ids", hash_ids, torch.int64)
    _contig("table", table, torch.uint8)
    _contig("scales", scales, torch.uint8 if layout.scale_format == SCALE_E8M0 else torch.float32)
    _check_table(layout, table, scales)
    _check_err(err_count)
    if emb is None:
        emb = torch.empty((B, T, C * layout.head_dim), dtype=torch.bfloat16, device=hash_ids.device)
    _numel("emb", emb, (B, T, C * layout.head_dim))
    _contig("emb", emb, _BF16)
    _same_device(hash_ids, table=table, scales=scales, emb=emb, err_count=err_count)
    _check("engram_gather_dequant", _lib.engram_gather_dequant(
        ctypes.byref(layout), _ptr(table), _ptr(scales), _ptr(hash_ids), B, T, _ptr(emb),
        _ptr(err_count), _stream()))
    return emb


def engram_kv_proj(layout: EngramLayout, emb: torch.Tensor, wkv: torch.Tensor,
                   kv: Optional[torch.Tensor] = None) -> torch.Tensor:
    """kv [B, T, (hc + 1) * dim] bf16 = emb @ wkv^T (wkv in the layout's wkv_format)."""
    if emb.dim() != 3:
        raise ValueError(f"emb has shape {tuple(emb.shape)}, expected [B, T, n_cols * head_dim]")
    B, T, _ = emb.shape
    K, N, _ = _dims(layout)
    _shape("emb", emb, (B, T, K))
    _contig("emb", emb, _BF16)
    _check_wkv(layout, wkv)
    if kv is None:
        kv = torch.empty((B, T, N), dtype=torch.bfloat16, device=emb.device)
    _numel("kv", kv, (B, T, N))
    _contig("kv", kv, _BF16)
    _same_device(emb, wkv=wkv, kv=kv)
    _check("engram_kv_proj", _lib.engram_kv_proj(ctypes.byref(layout), _ptr(emb), _ptr(wkv), B, T,
                                                 _ptr(kv), _stream()))
    return kv


def make_hash_layout(n_layers: int, max_ngram: int, n_heads: int, pad_id: int, vocab: int,
                     history_len: int) -> HashLayout:
    return HashLayout(n_layers, max_ngram, n_heads, pad_id, vocab, history_len)


def engram_hash_ids(layout: HashLayout, token_map: torch.Tensor, multipliers: torch.Tensor,
                    primes: torch.Tensor, offsets: torch.Tensor, input_ids: torch.Tensor,
                    history: torch.Tensor, start_pos: int = 0,
                    token_mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Row ids [n_layers, B, L, (max_ngram - 1) * n_heads] int64 of tokens input_ids [B, L] at
    positions start_pos.. (engram_hash_ids in include/engram.h); history [B, history_len] int64
    is read and updated in place."""
    if input_ids.dim() != 2:
        raise ValueError(f"input_ids has shape {tuple(input_ids.shape)}, expected [B, L]")
    B, L = input_ids.shape
    _contig("token_map", token_map, (torch.int32, torch.uint32) if hasattr(torch, "uint32") else torch.int32)
    for name, t in (("multipliers", multipliers), ("primes", primes), ("offsets", offsets),
                    ("input_ids", input_ids), ("history", history)):
        _contig(name, t, torch.int64)
    n_cols = (layout.max_ngram - 1) * layout.n_heads
    _numel("token_map", token_map, (layout.vocab,))
    _numel("multipliers", multipliers, (layout.n_layers, layout.max_ngram))
    _numel("primes", primes, (layout.n_layers, layout.max_ngram - 1, layout.n_heads))
    _numel("offsets", offsets, (layout.n_layers, n_cols))
    _numel("history", history, (B, layout.history_len))
    if token_mask is not None:
        _contig("token_mask", token_mask, (torch.uint8, torch.bool))
        _numel("token_mask", token_mask, (B, L))
    _check_err(err_count)
    if out is None:
        out = torch.empty((layout.n_layers, B, L, n_cols), dtype=torch.int64, device=input_ids.device)
    _numel("out", out, (layout.n_layers, B, L, n_cols))
    _contig("out", out, torch.int64)
    _same_device(input_ids, token_map=token_map, multipliers=multipliers, primes=primes,
                 offsets=offsets, history=history, token_mask=token_mask, out=out, err_count=err_count)
    _check("engram_hash_ids", _lib.engram_hash_ids(
        ctypes.byref(layout), _ptr(token_map), _ptr(multipliers), _ptr(primes), _ptr(offsets),
        _ptr(input_ids), _ptr(token_mask), B, L, start_pos, _ptr(history), _ptr(out),
        _ptr(err_count), _stream()))
    return out


def engram_gate_apply(layout: EngramLayout, x: torch.Tensor, kv: torch.Tensor,
                      q_weight: torch.Tensor, k_weight: torch.Tensor,
                      token_mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [B, T, hc, dim] bf16 = x + gate * value (gate per token and stream)."""
    if x.dim() != 4:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [B, T, hc, dim]")
    B, T = x.shape[0], x.shape[1]
    _, N, _ = _dims(layout)
    _shape("x", x, (B, T, layout.hc, layout.dim))
    _contig("x", x, _BF16)
    _numel("kv", kv, (B, T, N))
    _contig("kv", kv, _BF16)
    _contig("q_weight", q_weight, torch.float32)
    _contig("k_weight", k_weight, torch.float32)
    _numel("q_weight", q_weight, (layout.hc, layout.dim))
    _numel("k_weight", k_weight, (layout.hc, layout.dim))
    if token_mask is not None:
        _contig("token_mask", token_mask, (torch.uint8, torch.bool))
        _numel("token_mask", token_mask, (B, T))
    if out is None:
        out = torch.empty_like(x)
    _numel("out", out, tuple(x.shape))
    _contig("out", out, _BF16)
    if gate is not None:
        _numel("gate", gate, (B, T, layout.hc))
        _contig("gate", gate, torch.float32)
    _same_device(x, kv=kv, q_weight=q_weight, k_weight=k_weight, token_mask=token_mask, out=out,
                 gate=gate)
    _check("engram_gate_apply", _lib.engram_gate_apply(
        ctypes.byref(layout), _ptr(x), _ptr(kv), _ptr(q_weight), _ptr(k_weight), _ptr(token_mask),
        B, T, _ptr(out), _ptr(gate), _stream()))
    return out


def _layout_key(layout: EngramLayout) -> tuple:
    # the fields that place control words and staging data (not n_rows, eps, clamp: the two
    # Engram modules of the model differ only in n_rows and share a workspace without clearing)
    return (layout.hc, layout.dim, layout.n_cols, layout.head_dim, layout.scale_block,
            layout.scale_format, layout.wkv_format)


class Workspace:
    """Zero-filled device workspace for engram_forward, grown on demand.

    The library leaves its control words zero after every call (except the time-out counter
    in word 0), and the staging area at the buffer's end holds scratch data; calls with one
    layout never place control words where another call's staging lies.  Calls with another
    layout may, so when the layout changes the buffer is cleared again (a fill kernel on the
    current stream), keeping word 0."""

    def __init__(self, device=None):
        self.device = device
        self.buf: Optional[torch.Tensor] = None
        self.layout = None

    def get(self, layout: EngramLayout, B: int, T: int) -> torch.Tensor:
        need = max(256, engram_forward_workspace_bytes(layout, B, T))
        key = _layout_key(layout)
        if self.buf is None or self.buf.numel() < need:
            old = self.buf
            self.buf = torch.zeros(need, dtype=torch.uint8, device=self.device or "cuda")
            if old is not None:  # keep the time-out counter across growth
                self.buf[:4].copy_(old[:4])
        elif self.layout is not None and key != self.layout:
            self.buf[4:].zero_()
        self.layout = key
        return self.buf


# One default workspace per (device, stream): calls that overlap in time must not share one, and
# calls on different streams may overlap.
_default_ws: dict = {}


def workspace_for(dev: int, stream_handle: int) -> "Workspace":
    """The default Workspace of a (device index, HIP stream handle): one each, made on first use
    (it allocates nothing until its first get())."""
    key = (int(dev), int(stream_handle))
    if key not in _default_ws:
        _default_ws[key] = Workspace(torch.device("cuda", int(dev)))
    return _default_ws[key]


def default_workspace(layout: EngramLayout, B: int, T: int, device: torch.device) -> torch.Tensor:
    """The workspace engram_forward uses when the caller passes none: the one of x's device and
    the current stream, grown on demand."""
    dev = device.index if device.index is not None else torch.cuda.current_device()
    return workspace_for(dev, torch.cuda.current_stream(dev).cuda_stream).get(layout, B, T)


def release_default_workspaces() -> None:
    """Frees the default workspaces (after the work on them has finished).  Registered to run at
    interpreter exit, so that no device buffer of this module outlives the program's own
    teardown of the HIP runtime or of a profiler attached to it."""
    if _default_ws and torch.cuda.is_initialized():
        torch.cuda.synchronize()
    _default_ws.clear()


atexit.register(release_default_workspaces)


def engram_forward_check(workspace: torch.Tensor) -> None:
    """Waits for the current stream and raises EngramError (status ENGRAM_E_TIMEOUT) if a
    cross-workgroup wait of an engram_forward call on `workspace` gave up since the last check;
    the library then zero-fills the workspace, so it can be used again."""
    _contig("workspace", workspace)
    _check("engram_forward_check", _lib.engram_forward_check(
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream()))


def engram_set_spin_budget(polls: int) -> int:
    """Bound of the cross-workgroup waits in polls (0 restores the default); returns the old one."""
    return int(_lib.engram_set_spin_budget(polls))


def engram_forward(layout: EngramLayout, x: torch.Tensor, hash_ids: torch.Tensor,
                   token_mask: Optional[torch.Tensor], table: torch.Tensor, scales: torch.Tensor,
                   wkv: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   err_count: Optional[torch.Tensor] = None, check: bool = False) -> torch.Tensor:
    """The whole Engram forward: out [B, T, hc, dim] bf16 (may be x itself).  With ``check`` the
    call waits for its stream and raises if a cross-workgroup wait timed out
    (engram_forward_check); without it the caller checks when it chooses to."""
    if out is None:
        out = torch.empty_like(x)
    B, T = _check_forward_args(layout, x, hash_ids, token_mask, table, scales, wkv, q_weight,
                               k_weight, out, err_count)
    if workspace is not None:
        _contig("workspace", workspace)
    _same_device(x, workspace=workspace)
    if workspace is None:
        workspace = default_workspace(layout, B, T, x.device)
    _check("engram_forward", _lib.engram_forward(
        ctypes.byref(layout), _ptr(x), _ptr(hash_ids), _ptr(token_mask), _ptr(table), _ptr(scales),
        _ptr(wkv), _ptr(q_weight), _ptr(k_weight), B, T, _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(err_count), _stream()))
    if check:
        engram_forward_check(workspace)
    return out


class PreparedForward:
    """engram_forward with its arguments checked once (prepare_forward): each call passes the same
    tensors' pointers to the C entry point on the current stream, with no per-call Python checks,
    so that back-to-back calls queue faster than the kernels run.  The tensors must stay alive and
    keep their storage while the object is used."""

    def __init__(self, layout, x, hash_ids, token_mask, table, scales, wkv, q_weight, k_weight,
                 out, workspace, err_count):
        B, T = _check_forward_args(layout, x, hash_ids, token_mask, table, scales, wkv, q_weight,
                                   k_weight, out, err_count)
        _contig("workspace", workspace)
        _same_device(x, workspace=workspace)
        need = engram_forward_workspace_bytes(layout, B, T)
        if workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace has {workspace.numel() * workspace.element_size()} bytes, "
                             f"the call needs {need}")
        self._keep = (layout, x, hash_ids, token_mask, table, scales, wkv, q_weight, k_weight, out,
                      workspace, err_count)
        self._args = (ctypes.byref(layout), _ptr(x), _ptr(hash_ids), _ptr(token_mask), _ptr(table),
                      _ptr(scales), _ptr(wkv), _ptr(q_weight), _ptr(k_weight), B, T, _ptr(out),
                      _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err_count))
        self._fn = _lib.engram_forward
        self.out = out
        self.workspace = workspace

    def __call__(self) -> torch.Tensor:
        st = self._fn(*self._args, _stream())
        if st != ENGRAM_OK:
            raise EngramError("engram_forward", st)
        return self.out


def prepare_forward(layout: EngramLayout, x: torch.Tensor, hash_ids: torch.Tensor,
                    token_mask: Optional[torch.Tensor], table: torch.Tensor, scales: torch.Tensor,
                    wkv: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                    out: torch.Tensor, workspace: torch.Tensor,
                    err_count: Optional[torch.Tensor] = None) -> PreparedForward:
    """A repeatable engram_forward on fixed tensors (checked here, once): returns a callable."""
    return PreparedForward(layout, x, hash_ids, token_mask, table, scales, wkv, q_weight, k_weight,
                           out, workspace, err_count)


def engram_forward_noalloc(layout: EngramLayout, x: torch.Tensor, hash_ids: torch.Tensor,
                           token_mask: Optional[torch.Tensor], table: torch.Tensor,
                           scales: torch.Tensor, wkv: torch.Tensor, q_weight: torch.Tensor,
                           k_weight: torch.Tensor, out: torch.Tensor,
                           err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """engram_forward without a workspace argument and without any allocation: the library's
    fixed per-GPU scratch array serves as the workspace (at most 4 MiB of it: up to 128 tokens at
    the model's layout; larger calls raise with status ENGRAM_E_WORKSPACE).  `out` must be
    given; calls on one GPU that overlap in time race on the scratch."""
    B, T = _check_forward_args(layout, x, hash_ids, token_mask, table, scales, wkv, q_weight,
                               k_weight, out, err_count)
    _check("engram_forward_noalloc", _lib.engram_forward_noalloc(
        ctypes.byref(layout), _ptr(x), _ptr(hash_ids), _ptr(token_mask), _ptr(table), _ptr(scales),
        _ptr(wkv), _ptr(q_weight), _ptr(k_weight), B, T, _ptr(out), _ptr(err_count), _stream()))
    return out


def _check_forward_args(layout: EngramLayout, x, hash_ids, token_mask, table, scales, wkv,
                        q_weight, k_weight, out, err_count):
    """Checks the tensors of a whole forward against the layout; returns (B, T)."""
    if x.dim() != 4:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [B, T, hc, dim]")
    B, T = x.shape[0], x.shape[1]
    _shape("x", x, (B, T, layout.hc, layout.dim))
    _contig("x", x, _BF16)
    _numel("hash_ids", hash_ids, (B, T, layout.n_cols))
    _contig("hash_ids", hash_ids, torch.int64)
    _contig("table", table, torch.uint8)
    _contig("scales", scales, torch.uint8 if layout.scale_format == SCALE_E8M0 else torch.float32)
    _check_table(layout, table, scales)
    _check_wkv(layout, wkv)
    _contig("q_weight", q_weight, torch.float32)
    _contig("k_weight", k_weight, torch.float32)
    _numel("q_weight", q_weight, (layout.hc, layout.dim))
    _numel("k_weight", k_weight, (layout.hc, layout.dim))
    if token_mask is not None:
        _contig("token_mask", token_mask, (torch.uint8, torch.bool))
        _numel("token_mask", token_mask, (B, T))
    _check_err(err_count)
    _numel("out", out, tuple(x.shape))
    _contig("out", out, _BF16)
    _same_device(x, hash_ids=hash_ids, table=table, scales=scales, wkv=wkv, q_weight=q_weight,
                 k_weight=k_weight, token_mask=token_mask, out=out, err_count=err_count)
    return B, T


# ----------------------------------------------------------------------------------------
# The serving operators around the forward: a plan of ragged requests, their row ids, the norms
# around a block, a projection with its epilogue.  They launch on the current stream of their
# tensors' device.  As in the forward, a bf16 tensor may be given as its int16 view; bf16 outputs that
# a call makes then have x's type.
# ----------------------------------------------------------------------------------------

STREAM_BF16, STREAM_FP32 = 0, 1                    # engram_stream_format
GATE_NONE, GATE_TOKEN, GATE_FEATURE = 0, 1, 2      # engram_gate_kind
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU, ACT_SIGMOID = range(6)  # engram_activation


_U32 = getattr(torch, "uint32", torch.int32)  # (torch versions without unsigned types hold such maps as int32)

# the HIP stream handle of a device's current stream (torch.cuda.current_stream, without the object)
_raw_stream = torch._C._cuda_getCurrentRawStream
# the current device (torch.cuda.current_device, without its check that the GPU is initialised: tensors on one exist)
_current_device = torch._C._cuda_getDevice


def _launch(where: str, device: int, fn, *args) -> None:
    """Calls a C entry point on the current stream of the device (as its last argument), with that
    device current for the call.  device: the tensors' index, -1 for host memory."""
    if device < 0:
        raise ValueError("tensors must be on a GPU, got cpu")
    if device == _current_device():
        st = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device))
    if st != ENGRAM_OK:
        raise EngramError(where, st)


def _type(name: str, t: torch.Tensor, dtype) -> None:
    if t.dtype not in (_BF16 if dtype is torch.bfloat16 else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _tensor(name: str, t: torch.Tensor, shape: tuple, dtype, device: int) -> int:
    """The address of a contiguous tensor of this shape and dtype (for bf16 also its int16 view) on the
    device."""
    if t.dtype is not dtype:
        _type(name, t, dtype)
    if t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} is on {t.device}, not with the other tensors")
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor, lead: tuple, row: tuple, dtype, device: int) -> int:
    """The stride in elements between the rows of a tensor [*lead, *row] of this dtype whose rows are
    contiguous and evenly spaced."""
    if t.dtype is not dtype:
        _type(name, t, dtype)
    if t.shape != lead + row:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {lead + row}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not with the other tensors")
    size = row[0] if len(row) == 1 else row[0] * row[1]
    if t.is_contiguous():
        return size
    n, want, step = len(lead), 1, t.stride()
    for d in range(len(row) - 1, -1, -1):
        if row[d] != 1 and step[n + d] != want:
            raise ValueError(f"{name}: the last {len(row)} dimensions must be contiguous")
        want *= row[d]
    stride = None
    for d in range(n - 1, -1, -1):
        if lead[d] == 1:
            continue
        if stride is None:
            stride, want = step[d], step[d]
        elif step[d] != want:
            raise ValueError(f"{name}: the rows must be evenly spaced")
        want *= lead[d]
    return size if stride is None else stride


def _refuse_grad(where: str, **tensors) -> None:
    name = next(k for k, t in tensors.items() if t is not None and t.requires_grad)
    raise ValueError(f"{name} requires grad, and {where} has no backward pass: call it under torch.no_grad()")


def _counter(err_count: Optional[torch.Tensor], device: int):
    if err_count is None:
        return None
    _check_err(err_count)
    if err_count.get_device() != device:
        raise ValueError(f"err_count is on {err_count.device}, not with the other tensors")
    return err_count.data_ptr()


def make_page_layout(block_size: int, max_blocks: int, n_blocks: int) -> PageLayout:
    """A pool of n_blocks pages of block_size positions, at most max_blocks of them per request."""
    return PageLayout(block_size, max_blocks, n_blocks)


class BatchPlan:
    """The buffers engram_batch_plan writes (engram_batch_plan_out in include/engram.h), made once by the
    caller and kept from step to step.  They are read, and may be filled, through the attributes named
    in FIELDS, but not replaced or resized.  seq_lens and free_left are the next step's cached_lens and
    free_count: use two plans in turn, or copy them (a call never writes what it reads)."""

    FIELDS = ("token_start", "start_pos", "seq_lens", "status", "free_left", "slots", "positions", "requests", "live")

    def __init__(self, n_requests: int, max_tokens: int, device="cuda"):
        sizes = (n_requests + 1, n_requests, n_requests, n_requests, 1, max_tokens, max_tokens, max_tokens, max_tokens)
        types = [{"slots": torch.int64, "live": torch.uint8}.get(f, torch.int32) for f in self.FIELDS]
        self._buffers = tuple(torch.zeros(n, dtype=t, device=device) for n, t in zip(sizes, types))
        self._out = _PlanOut(*[t.data_ptr() for t in self._buffers])
        self._index = self._buffers[0].get_device()
        self._sizes = (n_requests, max_tokens)

    n_requests = property(lambda self: self._sizes[0])
    max_tokens = property(lambda self: self._sizes[1])
    device = property(lambda self: self._buffers[0].device)


for _i, _f in enumerate(BatchPlan.FIELDS):
    setattr(BatchPlan, _f, property(lambda self, i=_i: self._buffers[i]))


def _plan_on(plan: BatchPlan, device: int) -> BatchPlan:
    if plan._index != device:
        raise ValueError(f"plan is on {plan.device}, not with the other tensors")
    return plan


def engram_batch_plan(layout: PageLayout, new_lens: torch.Tensor, cached_lens: torch.Tensor, block_table: torch.Tensor,
                      free_list: torch.Tensor, free_count: torch.Tensor, plan: BatchPlan,
                      err_count: Optional[torch.Tensor] = None) -> BatchPlan:
    """Plans a step of ragged requests into `plan` (engram_batch_plan in include/engram.h): admits
    requests by tokens and pages, takes and gives back pages (block_table [R, max_blocks] and
    free_list [n_blocks] are updated in place), and lays out the admitted tokens."""
    (R, T), i32, dev = plan._sizes, torch.int32, free_list.get_device()
    new = _tensor("new_lens", new_lens, (R,), i32, dev)
    held = _tensor("cached_lens", cached_lens, (R,), i32, dev)
    table = _tensor("block_table", block_table, (R, layout.max_blocks), i32, dev)
    pool = _tensor("free_list", free_list, (layout.n_blocks,), i32, dev)
    count = _tensor("free_count", free_count, (1,), i32, dev)
    _launch("engram_batch_plan", dev, _lib.engram_batch_plan, layout, new, held, R, table, pool, count, T,
            _plan_on(plan, dev)._out, _counter(err_count, dev))
    return plan


def engram_hash_ids_paged(layout: HashLayout, pages: PageLayout, token_map: torch.Tensor, multipliers: torch.Tensor,
                          primes: torch.Tensor, offsets: torch.Tensor, input_ids: torch.Tensor, plan: BatchPlan,
                          block_table: torch.Tensor, history: torch.Tensor, token_mask: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Row ids [n_layers, n_tokens, (max_ngram - 1) * n_heads] int64 of a plan's flat tokens input_ids
    [plan.max_tokens] (engram_hash_ids_paged in include/engram.h); history [n_blocks, block_size]
    int64, addressed through the plan and block_table, is read and updated in place."""
    (R, n), i64, i32, dev = plan._sizes, torch.int64, torch.int32, input_ids.get_device()
    at = _plan_on(plan, dev)._out
    layers, heads, orders = layout.n_layers, layout.n_heads, layout.max_ngram - 1
    tmap = _tensor("token_map", token_map, (layout.vocab,), i32 if token_map.dtype is i32 else _U32, dev)
    mult = _tensor("multipliers", multipliers, (layers, orders + 1), i64, dev)
    prime = _tensor("primes", primes, (layers, orders, heads), i64, dev)
    offs = _tensor("offsets", offsets, (layers, orders * heads), i64, dev)
    ids = _tensor("input_ids", input_ids, (n,), i64, dev)
    mask = None
    if token_mask is not None:
        mask = _tensor("token_mask", token_mask, (n,), torch.bool if token_mask.dtype is torch.bool else torch.uint8, dev)
    table = _tensor("block_table", block_table, (R, pages.max_blocks), i32, dev)
    hist = _tensor("history", history, (pages.n_blocks, pages.block_size), i64, dev)
    if out is None:
        out = input_ids.new_empty((layers, n, orders * heads))
        to = out.data_ptr()
    else:
        to = _tensor("out", out, (layers, n, orders * heads), i64, dev)
    _launch("engram_hash_ids_paged", dev, _lib.engram_hash_ids_paged, layout, pages, tmap, mult, prime, offs, ids, mask, n, at.slots,
            at.positions, at.requests, at.start_pos, R, table, hist, to, _counter(err_count, dev))
    return out


def make_norm_layout(hc: int, dim: int, y_streams: Optional[int] = None, gate: int = GATE_NONE, post_norm: bool = True,
                     pre_norm: bool = True, alpha: float = 1.0, beta: float = 1.0, post_eps: float = 1e-20,
                     pre_eps: float = 1e-20, stream_format: int = STREAM_BF16) -> NormLayout:
    """Layout of engram_residual_norm; y_streams: hc (the default), or 1 for a block output shared by
    every stream."""
    return NormLayout(hc, dim, hc if y_streams is None else y_streams, stream_format, gate, bool(post_norm), bool(pre_norm),
                      alpha, beta, post_eps, pre_eps)


def engram_residual_norm(layout: NormLayout, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                         gate: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                         pre_weight: Optional[torch.Tensor] = None, token_mask: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None):
    """Closes a block and opens the next (engram_residual_norm in include/engram.h): returns
    (out, h) with out = alpha * x + beta * gate * norm(y) and h = norm(out).  x [B, T, hc, dim]
    contiguous; y and a gate per feature [B, T, y_streams, dim] may be slices of wider rows; out may
    be x.  Without y, h = norm(x) and out is x; without pre_norm, h is None.  Forward only: with autograd on, a
    tensor that requires grad is refused."""
    if (x.requires_grad or (y is not None and y.requires_grad) or (gate is not None and gate.requires_grad) or
            (post_weight is not None and post_weight.requires_grad) or (pre_weight is not None and pre_weight.requires_grad) or
            (out is not None and out.requires_grad) or (h is not None and h.requires_grad)) and torch.is_grad_enabled():
        _refuse_grad("engram_residual_norm", x=x, y=y, gate=gate, post_weight=post_weight, pre_weight=pre_weight, out=out, h=h)
    if x.dim() != 4:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [B, T, hc, dim]")
    B, T, hc, dim = x.shape
    dev, bf16 = x.get_device(), torch.bfloat16
    if (hc, dim) != (layout.hc, layout.dim):
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [B, T, {layout.hc}, {layout.dim}]")
    full = (B, T, hc, dim)
    stream = torch.float32 if layout.stream_format == STREAM_FP32 else bf16
    xp = _tensor("x", x, full, stream, dev)
    yp = gp = op = hp = mp = None
    y_stride = gate_stride = 0
    if y is not None:
        rows = (layout.y_streams, dim)
        y_stride = _rows("y", y, (B, T), rows, bf16, dev)
        yp = y.data_ptr()
        if out is None:
            out = torch.empty_like(x)
            op = out.data_ptr()
        else:
            op = _tensor("out", out, full, stream, dev)
        if (gate is None) != (layout.gate == GATE_NONE):
            raise ValueError("gate does not match the layout's gate kind")
        if layout.gate == GATE_TOKEN:
            gp = _tensor("gate", gate, (B, T, hc), torch.float32, dev)
        elif gate is not None:
            gate_stride = _rows("gate", gate, (B, T), rows, bf16, dev)
            gp = gate.data_ptr()
    elif gate is not None or out is not None:
        raise ValueError("gate and out need y")
    if layout.pre_norm:
        if h is None:
            h = torch.empty_like(x, dtype=x.dtype if stream is bf16 else bf16)
            hp = h.data_ptr()
        else:
            hp = _tensor("h", h, full, bf16, dev)
    elif h is not None:
        raise ValueError("h needs pre_norm")
    post = None if post_weight is None else _tensor("post_weight", post_weight, (hc, dim), torch.float32, dev)
    pre = None if pre_weight is None else _tensor("pre_weight", pre_weight, (hc, dim), torch.float32, dev)
    if token_mask is not None:
        mp = _tensor("token_mask", token_mask, (B, T), torch.bool if token_mask.dtype is torch.bool else torch.uint8, dev)
    _launch("engram_residual_norm", dev, _lib.engram_residual_norm, layout, xp, yp, y_stride, gp, gate_stride, post, pre, mp, B, T,
            op, hp)
    return (x if y is None else out), h


def make_linear_layout(in_features: int, out_features: int, activation: int = ACT_NONE, glu: bool = False,
                       stream_format: int = STREAM_BF16) -> LinearLayout:
    return LinearLayout(in_features, out_features, activation, bool(glu), stream_format)


def engram_linear_workspace_bytes(layout: LinearLayout, M: int) -> int:
    """For exactly M rows on the current device; fewer rows may need more."""
    return int(_lib.engram_linear_workspace_bytes(ctypes.byref(layout), M))


def engram_linear_workspace_bytes_up_to(layout: LinearLayout, M: int) -> int:
    """Enough for every call of 1 .. M rows on the current device: one buffer for steps of different lengths."""
    return int(_lib.engram_linear_workspace_bytes_up_to(ctypes.byref(layout), M))


def engram_linear(layout: LinearLayout, x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                  residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [..., N] = residual + act(x [..., K] @ w^T + bias), or with the layout's glu
    residual + act(gate) * value from a weight of 2 N rows (engram_linear in include/engram.h).  x,
    residual and out may be slices of wider rows; out may be the residual.  Without a workspace the call
    takes one from torch's allocator where it needs one: calls on other streams, and captured graphs, then
    have their own.  A workspace that is given must hold engram_linear_workspace_bytes of this many rows; one
    kept for steps of different lengths is sized by engram_linear_workspace_bytes_up_to.
    Forward only: with autograd on, a tensor that requires grad is refused."""
    if (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad) or
            (residual is not None and residual.requires_grad) or (out is not None and out.requires_grad)) and torch.is_grad_enabled():
        _refuse_grad("engram_linear", x=x, w=w, bias=bias, residual=residual, out=out)
    K, N, dev, bf16 = layout.in_features, layout.out_features, x.get_device(), torch.bfloat16
    if x.dim() < 1:
        raise ValueError("x has no dimensions")
    lead = tuple(x.shape[:-1])
    M = math.prod(lead)
    x_stride = _rows("x", x, lead, (K,), bf16, dev)
    rows = 2 * N if layout.glu else N
    wp = _tensor("w", w, (rows, K), bf16, dev)
    bp = None if bias is None else _tensor("bias", bias, (rows,), torch.float32, dev)
    stream = torch.float32 if layout.stream_format == STREAM_FP32 else bf16
    rp, r_stride = None, 0
    if residual is not None:
        r_stride = _rows("residual", residual, lead, (N,), stream, dev)
        rp = residual.data_ptr()
    if out is None:
        out, o_stride = x.new_empty((*lead, N), dtype=x.dtype if stream is bf16 else stream), N
    else:
        o_stride = _rows("out", out, lead, (N,), stream, dev)
    ws, ws_bytes = None, 0
    if workspace is not None:
        _contig("workspace", workspace)
        if workspace.get_device() != dev:
            raise ValueError(f"workspace is on {workspace.device}, not with the other tensors")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    args = (layout, x.data_ptr(), x_stride, wp, bp, rp, r_stride, M, out.data_ptr(), o_stride)
    try:
        _launch("engram_linear", dev, _lib.engram_linear, *args, ws, ws_bytes)
    except EngramError as e:
        if e.status != ENGRAM_E_WORKSPACE or workspace is not None:
            raise
        # the shape splits K (a call without a workspace is refused before anything is enqueued)
        with torch.cuda.device(dev):
            need = engram_linear_workspace_bytes(layout, M)
        workspace = x.new_empty(need, dtype=torch.uint8)
        _launch("engram_linear", dev, _lib.engram_linear, *args, workspace.data_ptr(), workspace.numel())
    return out


# ----------------------------------------------------------------------------------------
# The latent cache and the attention that reads it (include/engram.h, "The latent cache").  The plan's
# fields say where the step's tokens are.  Forward only: with autograd on, tensors that require grad are
# refused.
# ----------------------------------------------------------------------------------------

CACHE_BF16, CACHE_MXFP8 = 0, 1  # engram_cache_format


def make_latent_layout(heads: int, latent_dim: int, rope_dim: int, head_dim: int = 128, scale: Optional[float] = None,
                       window: int = 0, cache_format: int = CACHE_BF16) -> LatentLayout:
    """Layout of the latent operators; scale: of the scores, (head_dim + rope_dim) ** -0.5 by default."""
    if scale is None:
        scale = (head_dim + rope_dim) ** -0.5
    return LatentLayout(heads, latent_dim, rope_dim, head_dim, cache_format, window, scale)


def engram_latent_layout_check(layout: LatentLayout) -> int:
    return _lib.engram_latent_layout_check(ctypes.byref(layout))


def engram_latent_row_bytes(layout: LatentLayout) -> int:
    """Bytes of a cache row; 0 for a layout that engram_latent_layout_check refuses."""
    return int(_lib.engram_latent_row_bytes(ctypes.byref(layout)))


def make_latent_cache(layout: LatentLayout, pages: PageLayout, device="cuda") -> torch.Tensor:
    """A cache of zeros: [n_blocks, block_size, latent_dim + rope_dim] bf16, or for MXFP8 the rows' bytes
    [n_blocks, block_size, engram_latent_row_bytes] uint8."""
    return torch.zeros(_cache_shape(layout, pages), dtype=_cache_type(layout), device=device)


def _cache_type(layout: LatentLayout):
    return torch.uint8 if layout.cache_format == CACHE_MXFP8 else torch.bfloat16


def _cache_shape(layout: LatentLayout, pages: PageLayout) -> tuple:
    row = layout.latent_dim + layout.rope_dim
    if layout.cache_format == CACHE_MXFP8:
        row += 16 + layout.rope_dim
    return (pages.n_blocks, pages.block_size, row)


def _no_grad(where: str, **tensors) -> None:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors.values()):
        _refuse_grad(where, **tensors)


def engram_latent_write(layout: LatentLayout, pages: PageLayout, latent: torch.Tensor, rope: torch.Tensor, plan: BatchPlan,
                        cache: torch.Tensor, err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Writes the rows of a plan's tokens into the cache (engram_latent_write in include/engram.h): latent
    [plan.max_tokens, latent_dim] and rope [plan.max_tokens, rope_dim] bf16 may be slices of wider rows.  Returns the
    cache, which is updated in place."""
    _no_grad("engram_latent_write", latent=latent, rope=rope, cache=cache)
    n, dev, bf16 = plan._sizes[1], cache.get_device(), torch.bfloat16
    at = _plan_on(plan, dev)._out
    ls = _rows("latent", latent, (n,), (layout.latent_dim,), bf16, dev)
    rs = _rows("rope", rope, (n,), (layout.rope_dim,), bf16, dev)
    to = _tensor("cache", cache, _cache_shape(layout, pages), _cache_type(layout), dev)
    _launch("engram_latent_write", dev, _lib.engram_latent_write, layout, pages, latent.data_ptr(), ls, rope.data_ptr(), rs, at.slots,
            n, to, _counter(err_count, dev))
    return cache


def engram_latent_read(layout: LatentLayout, pages: PageLayout, cache: torch.Tensor, plan: BatchPlan, block_table: torch.Tensor,
                       max_rows: int, min_tokens: int = 1, latent: Optional[torch.Tensor] = None,
                       rope: Optional[torch.Tensor] = None, row_start: Optional[torch.Tensor] = None,
                       err_count: Optional[torch.Tensor] = None):
    """Reads the rows of a plan's requests with at least min_tokens new tokens back (engram_latent_read in
    include/engram.h): returns (latent [max_rows, latent_dim], rope [max_rows, rope_dim], row_start [R + 1] int32).
    Rows behind the last are left as they were (in tensors that the call makes: not set)."""
    _no_grad("engram_latent_read", cache=cache, latent=latent, rope=rope)
    (R, n), dev, bf16, i32 = plan._sizes, cache.get_device(), torch.bfloat16, torch.int32
    at = _plan_on(plan, dev)._out
    src = _tensor("cache", cache, _cache_shape(layout, pages), _cache_type(layout), dev)
    table = _tensor("block_table", block_table, (R, pages.max_blocks), i32, dev)
    if latent is None:
        latent = cache.new_empty((max_rows, layout.latent_dim), dtype=bf16)
    if rope is None:
        rope = cache.new_empty((max_rows, layout.rope_dim), dtype=bf16)
    if row_start is None:
        row_start = cache.new_empty((R + 1,), dtype=i32)
    _launch("engram_latent_read", dev, _lib.engram_latent_read, layout, pages, src, at.token_start, at.start_pos, R, table, n,
            min_tokens, max_rows, _tensor("row_start", row_start, (R + 1,), i32, dev),
            _tensor("latent", latent, (max_rows, layout.latent_dim), bf16, dev),
            _tensor("rope", rope, (max_rows, layout.rope_dim), bf16, dev), _counter(err_count, dev))
    return latent, rope, row_start


def engram_latent_attention_workspace_bytes(layout: LatentLayout) -> int:
    """For any call of this layout on the current device."""
    return int(_lib.engram_latent_attention_workspace_bytes(ctypes.byref(layout)))


def engram_latent_attention_expanded_workspace_bytes(layout: LatentLayout, R: int, n_tokens: int, n_rows: int) -> int:
    """For n_tokens tokens of R requests over n_rows rows on the current device."""
    return int(_lib.engram_latent_attention_expanded_workspace_bytes(ctypes.byref(layout), R, n_tokens, n_rows))


def engram_latent_attention_expanded_workspace_bytes_up_to(layout: LatentLayout, n_tokens: int, n_rows: int) -> int:
    """Enough for every call with 1 .. n_tokens tokens over 0 .. n_rows rows on the current device."""
    return int(_lib.engram_latent_attention_expanded_workspace_bytes_up_to(ctypes.byref(layout), n_tokens, n_rows))


def _attention_out(q: torch.Tensor, out: Optional[torch.Tensor], n: int, row: tuple, dev: int):
    """(out, its stride)."""
    if out is None:
        return q.new_empty((n, *row)), row[0] * row[1]
    return out, _rows("out", out, (n,), row, torch.bfloat16, dev)


def _given(workspace: torch.Tensor, dev: int):
    _contig("workspace", workspace)
    if workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, not with the other tensors")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def engram_latent_attention(layout: LatentLayout, pages: PageLayout, q: torch.Tensor, cache: torch.Tensor, plan: BatchPlan,
                            block_table: torch.Tensor, max_tokens: int = 0, out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Absorbed attention of a plan's tokens over the cache's pages (engram_latent_attention in include/engram.h):
    out [plan.max_tokens, heads, latent_dim] bf16 of q [plan.max_tokens, heads, latent_dim + rope_dim] bf16, for
    requests with at most max_tokens new tokens (0: all).  q and out may be slices of wider rows.  Rows of other
    tokens are left as they were (in an out that the call makes: not set).  lse [plan.max_tokens, heads] fp32 is
    filled where it is given.  Without a workspace the call takes one from torch's allocator: calls on other streams, and
    captured graphs, then have their own."""
    _no_grad("engram_latent_attention", q=q, cache=cache, out=out, lse=lse)
    (R, n), dev, H, D = plan._sizes, cache.get_device(), layout.heads, layout.latent_dim
    at = _plan_on(plan, dev)._out
    src = _tensor("cache", cache, _cache_shape(layout, pages), _cache_type(layout), dev)
    qs = _rows("q", q, (n,), (H, D + layout.rope_dim), torch.bfloat16, dev)
    table = _tensor("block_table", block_table, (R, pages.max_blocks), torch.int32, dev)
    out, os_ = _attention_out(q, out, n, (H, D), dev)
    lp = None if lse is None else _tensor("lse", lse, (n, H), torch.float32, dev)
    if workspace is None:
        workspace = q.new_empty(_on_device(dev, engram_latent_attention_workspace_bytes, layout), dtype=torch.uint8)
    ws, ws_bytes = _given(workspace, dev)
    _launch("engram_latent_attention", dev, _lib.engram_latent_attention, layout, pages, q.data_ptr(), qs, src, at.token_start,
            at.start_pos, R, table, n, max_tokens, out.data_ptr(), os_, lp, ws, ws_bytes, _counter(err_count, dev))
    return out


def _on_device(dev: int, fn, *args):
    if dev < 0:
        raise ValueError("tensors must be on a GPU, got cpu")
    if dev == _current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def engram_latent_attention_expanded(layout: LatentLayout, q: torch.Tensor, kv: torch.Tensor, rope: torch.Tensor,
                                     row_start: torch.Tensor, plan: BatchPlan, min_tokens: int = 1,
                                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Expanded attention of a plan's tokens (engram_latent_attention_expanded in include/engram.h): out
    [plan.max_tokens, heads, head_dim] bf16 of q [plan.max_tokens, heads, head_dim + rope_dim], kv [n_rows, heads,
    2 * head_dim] (of each head the key part, then the value), rope [n_rows, rope_dim] and row_start [R + 1] as
    engram_latent_read gives it, for requests with at least min_tokens new tokens.  q, kv, rope and out may be slices of
    wider rows; rows of other tokens, lse and workspace as in engram_latent_attention.  A workspace that is kept for steps of
    different lengths is sized by engram_latent_attention_expanded_workspace_bytes_up_to."""
    _no_grad("engram_latent_attention_expanded", q=q, kv=kv, rope=rope, out=out, lse=lse)
    (R, n), dev, H, D, bf16 = plan._sizes, q.get_device(), layout.heads, layout.head_dim, torch.bfloat16
    at = _plan_on(plan, dev)._out
    if kv.dim() != 3:
        raise ValueError(f"kv has shape {tuple(kv.shape)}, expected [n_rows, {H}, {2 * D}]")
    rows = kv.shape[0]
    qs = _rows("q", q, (n,), (H, D + layout.rope_dim), bf16, dev)
    ks = _rows("kv", kv, (rows,), (H, 2 * D), bf16, dev)
    rs = _rows("rope", rope, (rows,), (layout.rope_dim,), bf16, dev)
    first = _tensor("row_start", row_start, (R + 1,), torch.int32, dev)
    out, os_ = _attention_out(q, out, n, (H, D), dev)
    lp = None if lse is None else _tensor("lse", lse, (n, H), torch.float32, dev)
    ws, ws_bytes = None, 0
    if workspace is None:
        need = _on_device(dev, engram_latent_attention_expanded_workspace_bytes, layout, R, n, rows)
        if need > 0:
            workspace = q.new_empty(need, dtype=torch.uint8)
    if workspace is not None:
        ws, ws_bytes = _given(workspace, dev)
    _launch("engram_latent_attention_expanded", dev, _lib.engram_latent_attention_expanded, layout, q.data_ptr(), qs, kv.data_ptr(),
            ks, rope.data_ptr(), rs, first, rows, at.token_start, at.start_pos, R, n, min_tokens, out.data_ptr(), os_, lp, ws,
            ws_bytes)
    return out
