"""Python binding of the C-ABI library ``libgdn_b200.so`` (include/gdn.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the stream.  If the library is
missing this module raises; there is no other implementation to fall back to.

Tensors (all contiguous, on one CUDA device):
  q, k        [T, H_k*d_k]  (or [T, H_k, d_k])   activation dtype
  v, z        [T, H_v*d_v]                       activation dtype
  a, b        [T, H_v]                           activation dtype
  conv_state  [N, 2*H_k*d_k + H_v*d_v, 3]        activation dtype, updated in place
  rec_state   [N, H_v, d_v, d_k] float32         updated in place
  cu_seqlens  [N + 1] int32                      (prefill only)
  weights     dict: conv_w [C, 4], A_log [H_v], dt_bias [H_v], norm_w [d_v], float32
The operators around the mixer (block_norm, quantize_rows, linear_i8, in_proj_i8,
out_proj_i8, beam_select, reorder_states) name their tensors where they are defined;
they take tensors of any one CUDA device, the current one or not.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn_b200.so")

_DT = {torch.bfloat16: 0, torch.float32: 1}
_I8 = 2   # GDN_I8


CUDA_ERROR = 3   # GDN_ERR_CUDA


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = "%s: %s (status %d)" % (what, status_string(status), status)
        if status == CUDA_ERROR:
            msg += " [%s]" % lib().gdn_last_cuda_error().decode()
        super().__init__(msg)
        self.status = status


class _CConfig(ctypes.Structure):
    _fields_ = [("n_k_heads", ctypes.c_int32), ("n_v_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("conv_kernel", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("l2_eps", ctypes.c_float), ("norm_eps", ctypes.c_float),
                ("act_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("prefill_segments", ctypes.c_int32)]


class _CSegment(ctypes.Structure):
    _fields_ = [("dst", ctypes.c_void_p), ("width", ctypes.c_int32)]


class _CNormConfig(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("eps", ctypes.c_float), ("res_scale", ctypes.c_float),
                ("gate", ctypes.c_int32), ("gate_sigmoid", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32)]


class _CStateBuffer(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("bytes", ctypes.c_int64), ("stride", ctypes.c_int64)]


class _CWeights(ctypes.Structure):
    _fields_ = [("conv_weight", ctypes.c_void_p), ("A_log", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p)]


_lib = None
EXPORTS = ("gdn_config_default", "gdn_prefill_workspace_size", "gdn_prefill_segments", "gdn_prefill", "gdn_decode",
           "gdn_decode_multi", "gdn_linear", "gdn_in_proj", "gdn_out_proj", "gdn_cp_workspace_size",
           "gdn_cp_local", "gdn_cp_finish", "gdn_prefill_host_workspace_size", "gdn_prefill_host",
           "gdn_norm_config_default", "gdn_block_norm", "gdn_quantize_rows", "gdn_linear_i8_workspace_size",
           "gdn_linear_i8", "gdn_in_proj_i8", "gdn_out_proj_i8", "gdn_beam_workspace_size", "gdn_beam_select",
           "gdn_reorder_states", "gdn_check_device_error", "gdn_status_string", "gdn_last_cuda_error")
DECODE_MULTI_MAX_TOKENS = 16   # GDN_DECODE_MULTI_MAX_TOKENS
PREFILL_SPLIT = -1             # GDN_PREFILL_SPLIT: Config.prefill_segments value that splits the chain
LINEAR_MAX_SEGMENTS = 8        # GDN_LINEAR_MAX_SEGMENTS
NORM_MAX_DIM = 16384           # GDN_NORM_MAX_DIM
BEAM_MAX_BEAMS, BEAM_MAX_OUT, BEAM_MAX_VOCAB = 32, 64, 1 << 20   # GDN_BEAM_MAX_*
REORDER_MAX_BUFFERS, REORDER_MAX_BEAMS = 128, 32                 # GDN_REORDER_MAX_*


def lib() -> ctypes.CDLL:
    """Load libgdn_b200.so (built in place by ``build.py``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libgdn_b200.so is not built; run `python -m "
                               "hybrid_linear_attention_mixer_b200.build` (needs nvcc)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.gdn_config_default.argtypes = [vp]
        L.gdn_config_default.restype = None
        L.gdn_prefill_workspace_size.argtypes = [vp, i64, i32]
        L.gdn_prefill_workspace_size.restype = sz
        L.gdn_prefill_segments.argtypes = [vp, i64, i32]
        L.gdn_prefill_segments.restype = i32
        L.gdn_prefill.argtypes = [vp, vp] + [vp] * 8 + [vp, i32, i64, vp, vp, sz, vp]
        L.gdn_prefill.restype = ctypes.c_int
        L.gdn_decode.argtypes = [vp, vp] + [vp] * 8 + [i32, vp, vp]
        L.gdn_decode.restype = ctypes.c_int
        L.gdn_decode_multi.argtypes = [vp, vp] + [vp] * 8 + [i32, i32, vp, vp, vp, vp]
        L.gdn_decode_multi.restype = ctypes.c_int
        L.gdn_linear.argtypes = [vp, vp, i64, i32, i32, vp, i32, vp]
        L.gdn_linear.restype = ctypes.c_int
        L.gdn_in_proj.argtypes = [vp, vp, vp, i64, i32] + [vp] * 6 + [vp]
        L.gdn_in_proj.restype = ctypes.c_int
        L.gdn_out_proj.argtypes = [vp, vp, vp, i64, i32, vp, vp]
        L.gdn_out_proj.restype = ctypes.c_int
        L.gdn_cp_workspace_size.argtypes = [vp, i64]
        L.gdn_cp_workspace_size.restype = sz
        L.gdn_cp_local.argtypes = [vp, vp] + [vp] * 5 + [vp, i64, vp, vp, sz, vp]
        L.gdn_cp_local.restype = ctypes.c_int
        L.gdn_cp_finish.argtypes = [vp, vp, vp, vp, i32, i32, vp, i64, vp, vp, vp, sz, vp]
        L.gdn_cp_finish.restype = ctypes.c_int
        L.gdn_prefill_host_workspace_size.argtypes = [vp, i64, i32]
        L.gdn_prefill_host_workspace_size.restype = sz
        L.gdn_prefill_host.argtypes = [vp, vp] + [vp] * 8 + [vp, i32, i64, vp, vp, sz, vp]
        L.gdn_prefill_host.restype = ctypes.c_int
        L.gdn_norm_config_default.argtypes = [vp]
        L.gdn_norm_config_default.restype = None
        L.gdn_block_norm.argtypes = [vp] * 6 + [i64] + [vp] * 4
        L.gdn_block_norm.restype = ctypes.c_int
        L.gdn_quantize_rows.argtypes = [vp, i32, i64, i32, vp, vp, vp]
        L.gdn_quantize_rows.restype = ctypes.c_int
        L.gdn_linear_i8_workspace_size.argtypes = [i64, i32]
        L.gdn_linear_i8_workspace_size.restype = sz
        L.gdn_linear_i8.argtypes = [vp, i32, vp, vp, vp, i64, i32, i32, i32, vp, i32, vp, sz, vp]
        L.gdn_linear_i8.restype = ctypes.c_int
        L.gdn_in_proj_i8.argtypes = [vp, vp, i32, vp, vp, vp, i64, i32] + [vp] * 6 + [vp, sz, vp]
        L.gdn_in_proj_i8.restype = ctypes.c_int
        L.gdn_out_proj_i8.argtypes = [vp, vp, i32, vp, vp, vp, i64, i32, vp, vp, sz, vp]
        L.gdn_out_proj_i8.restype = ctypes.c_int
        L.gdn_beam_workspace_size.argtypes = [i32] * 5
        L.gdn_beam_workspace_size.restype = sz
        L.gdn_beam_select.argtypes = [vp, i32, i64, vp, vp] + [i32] * 5 + [vp] * 4 + [sz, vp]
        L.gdn_beam_select.restype = ctypes.c_int
        L.gdn_reorder_states.argtypes = [vp, i32, i32, vp, i32, vp]
        L.gdn_reorder_states.restype = ctypes.c_int
        L.gdn_check_device_error.argtypes = [vp]
        L.gdn_check_device_error.restype = ctypes.c_int
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_last_cuda_error.argtypes = []
        L.gdn_last_cuda_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().gdn_status_string(int(s)).decode()


class _Fields:
    """A dataclass whose C struct is kept for its next calls while the fields stay as they
    are.  The struct is no part of the object's state: copies and pickles carry the fields."""
    __slots__ = ("_made",)

    def __getstate__(self):
        return self.__dict__.copy()

    def ref(self):
        """A pointer to the C struct, for a call."""
        now = [*self.__dict__.values()]
        try:
            was, made = self._made
            if was == now:
                return made
        except AttributeError:   # the first call
            pass
        made = ctypes.byref(self.c())
        self._made = now, made
        return made


@dataclass
class Config(_Fields):
    """Layer shape; the defaults are the published layer (16 / 48 heads of 128, K = 4)."""
    n_k_heads: int = 16
    n_v_heads: int = 48
    d_k: int = 128
    d_v: int = 128
    conv_kernel: int = 4
    chunk: int = 64
    l2_eps: float = 1e-6
    norm_eps: float = 1e-6
    act_dtype: torch.dtype = torch.bfloat16
    out_dtype: torch.dtype = torch.bfloat16
    state_dtype: torch.dtype = torch.float32   # bf16: the recurrent state stored in bf16
    prefill_segments: int = 0                  # chunk ranges a prefill is pipelined over; 0: automatic;
                                               # PREFILL_SPLIT: one sequence's chain split in two

    @property
    def channels(self) -> int:
        return 2 * self.n_k_heads * self.d_k + self.n_v_heads * self.d_v

    def c(self) -> _CConfig:
        return _CConfig(self.n_k_heads, self.n_v_heads, self.d_k, self.d_v, self.conv_kernel,
                        self.chunk, self.l2_eps, self.norm_eps, _DT[self.act_dtype],
                        _DT[self.out_dtype], _DT[self.state_dtype], self.prefill_segments)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype, device):
    if t.dtype != dtype:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _weights(w: dict, device) -> _CWeights:
    for n in ("conv_w", "A_log", "dt_bias", "norm_w"):
        _check(w[n], n, torch.float32, device)
    return _CWeights(w["conv_w"].data_ptr(), w["A_log"].data_ptr(), w["dt_bias"].data_ptr(),
                     w["norm_w"].data_ptr())


def workspace_size(cfg: Config, T_total: int, n_seqs: int) -> int:
    c = cfg.c()
    return int(lib().gdn_prefill_workspace_size(ctypes.byref(c), int(T_total), int(n_seqs)))


def prefill_segments(cfg: Config, T_total: int, n_seqs: int) -> int:
    """Chunk ranges a prefill of this size is pipelined over (1: one piece); a call
    launches 2 + 4 n kernels (6 for n = 1)."""
    c = cfg.c()
    return int(lib().gdn_prefill_segments(ctypes.byref(c), int(T_total), int(n_seqs)))


def prefill(cfg: Config, w: dict, q, k, v, a, b, z, conv_state, rec_state, cu_seqlens,
            out=None, workspace=None, stream=None):
    """Packed variable-length prefill; returns out [T, H_v*d_v] (out_dtype)."""
    dev = q.device
    T = q.shape[0]
    for n, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("z", z),
                 ("conv_state", conv_state)):
        _check(t, n, cfg.act_dtype, dev)
    _check(rec_state, "rec_state", cfg.state_dtype, dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
    n_seqs = cu_seqlens.shape[0] - 1
    if out is None:
        out = torch.empty((T, cfg.n_v_heads * cfg.d_v), dtype=cfg.out_dtype, device=dev)
    _check(out, "out", cfg.out_dtype, dev)
    need = workspace_size(cfg, T, n_seqs)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    c, cw = cfg.c(), _weights(w, dev)
    s = lib().gdn_prefill(ctypes.byref(c), ctypes.byref(cw), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                          _ptr(b), _ptr(z), _ptr(conv_state), _ptr(rec_state), _ptr(cu_seqlens),
                          n_seqs, T, _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_prefill")
    return out


def decode(cfg: Config, w: dict, q, k, v, a, b, z, conv_state, rec_state, out=None, stream=None):
    """One token per sequence; returns out [N, H_v*d_v] (out_dtype)."""
    dev = q.device
    N = q.shape[0]
    for n, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("z", z),
                 ("conv_state", conv_state)):
        _check(t, n, cfg.act_dtype, dev)
    _check(rec_state, "rec_state", cfg.state_dtype, dev)
    if out is None:
        out = torch.empty((N, cfg.n_v_heads * cfg.d_v), dtype=cfg.out_dtype, device=dev)
    _check(out, "out", cfg.out_dtype, dev)
    c, cw = cfg.c(), _weights(w, dev)
    s = lib().gdn_decode(ctypes.byref(c), ctypes.byref(cw), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                         _ptr(b), _ptr(z), _ptr(conv_state), _ptr(rec_state), N, _ptr(out),
                         _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_decode")
    return out


def decode_multi(cfg: Config, w: dict, q, k, v, a, b, z, conv_state, rec_state, n_tok: int, out=None,
                 state_snapshots=None, conv_snapshots=None, stream=None):
    """n_tok consecutive tokens per sequence (rows token-major within a sequence);
    returns out [N*n_tok, H_v*d_v].  Optional snapshots receive the recurrent state
    [n_tok, N, H_v, d_v, d_k] (state dtype) and the conv state [n_tok, N, C, K-1] after each token."""
    dev = q.device
    rows = q.shape[0]
    if n_tok <= 0 or rows % n_tok:
        raise ValueError("rows (%d) must be a positive multiple of n_tok (%d)" % (rows, n_tok))
    N = rows // n_tok
    for n, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("z", z),
                 ("conv_state", conv_state)):
        _check(t, n, cfg.act_dtype, dev)
    _check(rec_state, "rec_state", cfg.state_dtype, dev)
    if state_snapshots is not None:
        _check(state_snapshots, "state_snapshots", cfg.state_dtype, dev)
    if conv_snapshots is not None:
        _check(conv_snapshots, "conv_snapshots", cfg.act_dtype, dev)
    if out is None:
        out = torch.empty((rows, cfg.n_v_heads * cfg.d_v), dtype=cfg.out_dtype, device=dev)
    _check(out, "out", cfg.out_dtype, dev)
    c, cw = cfg.c(), _weights(w, dev)
    opt = lambda t: None if t is None else _ptr(t)
    s = lib().gdn_decode_multi(ctypes.byref(c), ctypes.byref(cw), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                               _ptr(b), _ptr(z), _ptr(conv_state), _ptr(rec_state), N, int(n_tok),
                               _ptr(out), opt(state_snapshots), opt(conv_snapshots), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_decode_multi")
    return out


def linear(x, w, outs=None, stream=None):
    """y = x . w^T on the tensor cores: x [M, K] and w [N, K] bf16, fp32 accumulation.
    ``outs`` (optional) is a list of bf16 [M, width] tensors that receive consecutive
    column ranges of y (widths adding up to N); default one [M, N] tensor.  Returns
    the list of outputs."""
    dev = x.device
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x [M, K] and w [N, K] expected, got %s and %s" % (tuple(x.shape), tuple(w.shape)))
    M, K = x.shape
    N = w.shape[0]
    _check(x, "x", torch.bfloat16, dev)
    _check(w, "w", torch.bfloat16, dev)
    if outs is None:
        outs = [torch.empty((M, N), dtype=torch.bfloat16, device=dev)]
    if not 1 <= len(outs) <= LINEAR_MAX_SEGMENTS:
        raise ValueError("1..%d output segments" % LINEAR_MAX_SEGMENTS)
    for i, o in enumerate(outs):
        _check(o, "outs[%d]" % i, torch.bfloat16, dev)
        if o.dim() != 2 or o.shape[0] != M:
            raise ValueError("outs[%d] must be [M, width]" % i)
    segs = (_CSegment * len(outs))(*[_CSegment(o.data_ptr(), o.shape[1]) for o in outs])
    s = lib().gdn_linear(_ptr(x), _ptr(w), M, N, K, segs, len(outs), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_linear")
    return outs


def in_proj(cfg: Config, hidden, w_in, out: dict | None = None, stream=None) -> dict:
    """The mixer's input projection: hidden [T, d_model] bf16, w_in [16,480, d_model]
    bf16 at the published shape (channels q | k | v | z | a | b).  Returns q, k
    [T, H_k*d_k], v, z [T, H_v*d_v], a, b [T, H_v], all bf16 (written into ``out``'s
    tensors when given)."""
    dev = hidden.device
    T, D = hidden.shape
    _check(hidden, "hidden", torch.bfloat16, dev)
    _check(w_in, "w_in", torch.bfloat16, dev)
    qk, vz, ab = cfg.n_k_heads * cfg.d_k, cfg.n_v_heads * cfg.d_v, cfg.n_v_heads
    if tuple(w_in.shape) != (2 * qk + 2 * vz + 2 * ab, D):
        raise ValueError("w_in shape %s, expected %s" % (tuple(w_in.shape), (2 * qk + 2 * vz + 2 * ab, D)))
    widths = (("q", qk), ("k", qk), ("v", vz), ("z", vz), ("a", ab), ("b", ab))
    o = out if out is not None else {n: torch.empty((T, wd), dtype=torch.bfloat16, device=dev) for n, wd in widths}
    for n, wd in widths:
        _check(o[n], n, torch.bfloat16, dev)
        if o[n].numel() != T * wd:
            raise ValueError("%s must hold [T, %d]" % (n, wd))
    c = cfg.c()
    s = lib().gdn_in_proj(ctypes.byref(c), _ptr(hidden), _ptr(w_in), T, D, _ptr(o["q"]), _ptr(o["k"]),
                          _ptr(o["v"]), _ptr(o["z"]), _ptr(o["a"]), _ptr(o["b"]), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_in_proj")
    return o


def out_proj(cfg: Config, o, w_out, y=None, stream=None):
    """The mixer's output projection: o [T, H_v*d_v] bf16 (the layer's output),
    w_out [d_model, H_v*d_v] bf16 -> y [T, d_model] bf16."""
    dev = o.device
    o2 = o.flatten(1) if o.dim() > 1 else o.reshape(-1, 1)
    T = o2.shape[0]
    D = w_out.shape[0]
    _check(o2, "o", torch.bfloat16, dev)
    _check(w_out, "w_out", torch.bfloat16, dev)
    if w_out.shape[1] != cfg.n_v_heads * cfg.d_v or o2.shape[1] != w_out.shape[1]:
        raise ValueError("w_out must be [d_model, H_v*d_v] and o [T, H_v*d_v]")
    if y is None:
        y = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    _check(y, "y", torch.bfloat16, dev)
    c = cfg.c()
    s = lib().gdn_out_proj(ctypes.byref(c), _ptr(o2), _ptr(w_out), T, D, _ptr(y), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_out_proj")
    return y


def cp_workspace_size(cfg: Config, T_seg: int) -> int:
    c = cfg.c()
    return int(lib().gdn_cp_workspace_size(ctypes.byref(c), T_seg))


def cp_local(cfg: Config, w: dict, q, k, v, a, b, conv_state, workspace=None, summary=None, stream=None):
    """Context-parallel phase 1 on this rank's segment: returns (summary, workspace).
    conv_state [C, K-1] holds the K-1 input rows before the segment (updated in
    place to the segment's last rows); summary [2, H_v, d_k, d_k] fp32 = (P, S_loc)."""
    dev = q.device
    T = q.shape[0]
    for n, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("conv_state", conv_state)):
        _check(t, n, cfg.act_dtype, dev)
    if workspace is None:
        workspace = torch.empty(cp_workspace_size(cfg, T), dtype=torch.uint8, device=dev)
    if summary is None:
        summary = torch.empty((2, cfg.n_v_heads, cfg.d_k, cfg.d_k), dtype=torch.float32, device=dev)
    _check(summary, "summary", torch.float32, dev)
    c, cw = cfg.c(), _weights(w, dev)
    s = lib().gdn_cp_local(ctypes.byref(c), ctypes.byref(cw), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                           _ptr(conv_state), T, _ptr(summary), _ptr(workspace), workspace.numel(), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_cp_local")
    return summary, workspace


def cp_finish(cfg: Config, w: dict, z, summaries, rank: int, state_in, workspace, out=None, state_out=None,
              stream=None):
    """Context-parallel phase 2: summaries [R, 2, H_v, d_k, d_k] (every rank's, in rank
    order), state_in [H_v, d_v, d_k] the state before the whole sequence.  Returns
    (out [T_seg, H_v*d_v], state_out [H_v, d_v, d_k]: the state after this segment)."""
    dev = z.device
    T = z.shape[0]
    _check(z, "z", cfg.act_dtype, dev)
    _check(summaries, "summaries", torch.float32, dev)
    _check(state_in, "state_in", torch.float32, dev)
    if out is None:
        out = torch.empty((T, cfg.n_v_heads * cfg.d_v), dtype=cfg.out_dtype, device=dev)
    if state_out is None:
        state_out = torch.empty_like(state_in)
    c, cw = cfg.c(), _weights(w, dev)
    s = lib().gdn_cp_finish(ctypes.byref(c), ctypes.byref(cw), _ptr(z), _ptr(summaries), summaries.shape[0],
                            rank, _ptr(state_in), T, _ptr(out), _ptr(state_out), _ptr(workspace),
                            workspace.numel(), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_cp_finish")
    return out, state_out


# ---------------------------------------------------------------------------
# The operators around the mixer in a serving step
# ---------------------------------------------------------------------------
def _index_of(t, name) -> int:
    """The index of the CUDA device that t is on."""
    index = t.get_device()
    if index < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    return index


def _shaped(t, name, dtype, index, shape):
    """A contiguous tensor of this dtype, CUDA device and shape: its address."""
    if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), shape))
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    raise ValueError("%s must be contiguous" % name)


def _too_large(what, *sizes):
    """The error of a size that the library takes as 32 bits (ctypes would cut it off)."""
    return ValueError("%s beyond 32 bits: %s" % (what, ", ".join(str(n) for n in sizes)))


# The current stream's handle by device index: the binding's own lookup where torch has it
# (a Stream object costs several times as much to make as the call's other arguments).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn, what, index, stream, *args):
    """fn(*args, stream) on the tensors' device, which need not be the current one.  The
    stream is the caller's, else that device's current one."""
    if _current_device() != index:
        with torch.cuda.device(index):
            return _call(fn, what, index, stream, *args)
    s = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if s != 0:
        raise GdnError(s, what)


def _empty(shape, dtype, index, stream):
    """Memory for the call to use on ``stream``: taken from that stream's pool, so that
    neither its last user nor its next can still be at work on another stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=index)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=index)


_GATES = {"none": 0, "token": 1, "channel": 2, "full": 3}
_GATE_ACTS = {"linear": 0, "sigmoid": 1}


@dataclass
class NormConfig(_Fields):
    """The norms between two blocks (block_norm)."""
    dim: int = 2560
    eps: float = 1e-6
    res_scale: float = 1.0
    gate: str = "none"              # "token" [T], "channel" [dim] float32, "full" [T, dim]
    gate_act: str = "linear"        # "sigmoid": the factor is sigmoid(gate)
    act_dtype: torch.dtype = torch.bfloat16   # of o, a token or full gate, and y
    res_dtype: torch.dtype = torch.bfloat16   # of x and r

    def c(self) -> _CNormConfig:
        return _CNormConfig(self.dim, self.eps, self.res_scale, _GATES[self.gate], _GATE_ACTS[self.gate_act],
                            _DT[self.act_dtype], _DT[self.res_dtype])


def block_norm(cfg: NormConfig, o, x, gate=None, w_post=None, w_pre=None, r=None, y=None, y_scale=None,
               quantize=False, stream=None):
    """The norm after a block, its gate, the residual sum and the norm before the next
    block, in one pass (gdn_block_norm):

        r = x + res_scale * act(gate) * rmsnorm(o) * w_post,   y = rmsnorm(r) * w_pre

    o [T, dim] (None: no block, y is the norm of x), x [T, dim] the residual stream,
    w_post / w_pre [dim] float32 (None: no norm after / no y).  ``r`` may be x and ``y``
    may be o.  With ``quantize``, or where ``y_scale`` [T] is given, y is int8 rows.
    Returns (r, y, y_scale), None for what there is not."""
    dev = _index_of(x, "x")
    T, D = x.shape[0], cfg.dim
    if D >> 31:
        raise _too_large("dim", D)
    act, res = cfg.act_dtype, cfg.res_dtype
    px = _shaped(x, "x", res, dev, (T, D))
    po = pg = pp = pw = pr = py = ps = None
    if o is not None:
        po = _shaped(o, "o", act, dev, (T, D))
        if r is None:
            r = _empty((T, D), res, dev, stream)
        pr = _shaped(r, "r", res, dev, (T, D))
    elif r is not None:
        raise ValueError("r without a block output o")
    if gate is not None:
        if cfg.gate == "channel":
            pg = _shaped(gate, "gate", torch.float32, dev, (D,))
        elif cfg.gate == "token":
            pg = _shaped(gate, "gate", act, dev, (T,))
        else:
            pg = _shaped(gate, "gate", act, dev, (T, D))
    if w_post is not None:
        pp = _shaped(w_post, "w_post", torch.float32, dev, (D,))
    if w_pre is not None:
        pw = _shaped(w_pre, "w_pre", torch.float32, dev, (D,))
        if y_scale is not None or quantize:
            if y_scale is None:
                y_scale = _empty(T, torch.float32, dev, stream)
            ps = _shaped(y_scale, "y_scale", torch.float32, dev, (T,))
        y_dtype = torch.int8 if ps is not None else act
        if y is None:
            y = _empty((T, D), y_dtype, dev, stream)
        py = _shaped(y, "y", y_dtype, dev, (T, D))
    elif y is not None or y_scale is not None or quantize:
        raise ValueError("y without w_pre")
    _call(lib().gdn_block_norm, "gdn_block_norm", dev, stream, cfg.ref(), po, px, pg, pp, pw, T, pr, py, ps)
    return r, y, y_scale


def quantize_rows(x, q=None, scale=None, stream=None):
    """Rows in 8-bit integers: x [rows, cols] bf16 or float32 -> (q int8 [rows, cols],
    scale float32 [rows]) with x ~ scale * q.  For activations a row is a token; for a
    linear layer's weight it is an output channel."""
    dev = _index_of(x, "x")
    if x.dim() != 2:
        raise ValueError("x [rows, cols] expected, got %s" % (tuple(x.shape),))
    rows, cols = x.shape
    if cols >> 31:
        raise _too_large("cols", cols)
    if x.dtype not in _DT:
        raise TypeError("x: dtype %s, expected bfloat16 or float32" % x.dtype)
    px = _shaped(x, "x", x.dtype, dev, (rows, cols))
    if q is None:
        q = _empty((rows, cols), torch.int8, dev, stream)
    if scale is None:
        scale = _empty(rows, torch.float32, dev, stream)
    _call(lib().gdn_quantize_rows, "gdn_quantize_rows", dev, stream, px, _DT[x.dtype], rows, cols,
          _shaped(q, "q", torch.int8, dev, (rows, cols)), _shaped(scale, "scale", torch.float32, dev, (rows,)))
    return q, scale


def linear_i8_workspace_size(M: int, K: int) -> int:
    if K >> 31 > 0:
        raise _too_large("K", K)
    return int(lib().gdn_linear_i8_workspace_size(int(M), int(K)))


def _i8_operand(x, x_scale, name, dev, M, K, workspace, stream):
    """(x address, dtype code, scale address, workspace address and bytes, workspace) of the
    left operand: int8 rows with their scales, or rows that the call makes int8 itself."""
    if x.dtype == torch.int8:
        if x_scale is None:
            raise ValueError("%s in int8 needs its scales" % name)
        return (_shaped(x, name, torch.int8, dev, (M, K)), _I8,
                _shaped(x_scale, name + "_scale", torch.float32, dev, (M,)), None, 0, None)
    if x_scale is not None:
        raise ValueError("%s_scale is for int8 rows; %s is %s" % (name, name, x.dtype))
    if x.dtype not in _DT:
        raise TypeError("%s: dtype %s, expected bfloat16, float32 or int8" % (name, x.dtype))
    px = _shaped(x, name, x.dtype, dev, (M, K))
    if workspace is None:
        workspace = _empty(linear_i8_workspace_size(M, K), torch.uint8, dev, stream)
    return px, _DT[x.dtype], None, _workspace(workspace, dev), workspace.numel(), workspace


def _workspace(t, dev):
    if t.dtype is not torch.uint8 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be contiguous uint8 on cuda:%d" % dev)
    return t.data_ptr()


def linear_i8(x, w, w_scale, x_scale=None, outs=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """y = (x_scale x) . (w_scale w)^T in 8-bit integers with exact int32 sums: w [N, K] int8
    with w_scale [N] float32; x [M, K] int8 with x_scale [M], or bf16 / float32 rows that the
    call makes int8 first (``workspace``: linear_i8_workspace_size bytes of uint8).  ``outs``
    as in ``linear`` (bf16, or all float32); default one [M, N] tensor of ``out_dtype``.
    Returns the list of outputs."""
    dev = _index_of(x, "x")
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x [M, K] and w [N, K] expected, got %s and %s" % (tuple(x.shape), tuple(w.shape)))
    M, K = x.shape
    N = w.shape[0]
    if (N | K) >> 31:
        raise _too_large("N, K", N, K)
    if outs is None:
        outs = [_empty((M, N), out_dtype, dev, stream)]
    if not 1 <= len(outs) <= LINEAR_MAX_SEGMENTS:
        raise ValueError("1..%d output segments" % LINEAR_MAX_SEGMENTS)
    dt = outs[0].dtype
    if dt not in _DT:
        raise TypeError("outs[0]: dtype %s, expected bfloat16 or float32" % dt)
    segs = (_CSegment * len(outs))()
    for i, o in enumerate(outs):
        if o.dim() != 2:
            raise ValueError("outs[%d] must be [M, width]" % i)
        segs[i].dst = _shaped(o, "outs[%d]" % i, dt, dev, (M, o.shape[1]))
        segs[i].width = o.shape[1]
    px, xdt, pxs, ws, ws_bytes, workspace = _i8_operand(x, x_scale, "x", dev, M, K, workspace, stream)
    _call(lib().gdn_linear_i8, "gdn_linear_i8", dev, stream, px, xdt, pxs, _shaped(w, "w", torch.int8, dev, (N, K)),
          _shaped(w_scale, "w_scale", torch.float32, dev, (N,)), M, N, K, _DT[dt], segs, len(outs), ws, ws_bytes)
    return outs


def in_proj_i8(cfg: Config, hidden, w_in, w_scale, hidden_scale=None, out: dict | None = None, workspace=None,
               stream=None) -> dict:
    """The mixer's input projection in 8-bit integers: ``in_proj`` with w_in int8 and its
    scales [rows of w_in]; hidden as x in ``linear_i8``."""
    dev = _index_of(hidden, "hidden")
    T, D = hidden.shape
    if D >> 31:
        raise _too_large("d_model", D)
    qk, vz, ab = cfg.n_k_heads * cfg.d_k, cfg.n_v_heads * cfg.d_v, cfg.n_v_heads
    N = 2 * qk + 2 * vz + 2 * ab
    widths = (("q", qk), ("k", qk), ("v", vz), ("z", vz), ("a", ab), ("b", ab))
    pw, pws = _shaped(w_in, "w_in", torch.int8, dev, (N, D)), _shaped(w_scale, "w_scale", torch.float32, dev, (N,))
    o = out if out is not None else {n: _empty((T, wd), torch.bfloat16, dev, stream) for n, wd in widths}
    ptrs = []
    for n, wd in widths:   # (flat or by heads, as for in_proj)
        t = o[n]
        if t.dtype is not torch.bfloat16 or t.get_device() != dev or not t.is_contiguous():
            _check(t, n, torch.bfloat16, hidden.device)
        if t.numel() != T * wd:
            raise ValueError("%s must hold [T, %d]" % (n, wd))
        ptrs.append(t.data_ptr())
    px, xdt, pxs, ws, ws_bytes, workspace = _i8_operand(hidden, hidden_scale, "hidden", dev, T, D, workspace, stream)
    _call(lib().gdn_in_proj_i8, "gdn_in_proj_i8", dev, stream, cfg.ref(), px, xdt, pxs, pw, pws, T, D,
          *ptrs, ws, ws_bytes)
    return o


def out_proj_i8(cfg: Config, o, w_out, w_scale, o_scale=None, y=None, workspace=None, stream=None):
    """The mixer's output projection in 8-bit integers: ``out_proj`` with w_out int8 and its
    scales [d_model]; o as x in ``linear_i8``.  y [T, d_model] bf16."""
    dev = _index_of(o, "o")
    o2 = o.flatten(1) if o.dim() > 2 and o.is_contiguous() else o
    T, K, D = o2.shape[0], cfg.n_v_heads * cfg.d_v, w_out.shape[0]
    if D >> 31:
        raise _too_large("d_model", D)
    if y is None:
        y = _empty((T, D), torch.bfloat16, dev, stream)
    px, xdt, pxs, ws, ws_bytes, workspace = _i8_operand(o2, o_scale, "o", dev, T, K, workspace, stream)
    _call(lib().gdn_out_proj_i8, "gdn_out_proj_i8", dev, stream, cfg.ref(), px, xdt, pxs,
          _shaped(w_out, "w_out", torch.int8, dev, (D, K)), _shaped(w_scale, "w_scale", torch.float32, dev, (D,)), T, D,
          _shaped(y, "y", torch.bfloat16, dev, (T, D)), ws, ws_bytes)
    return y


def beam_workspace_size(n_groups: int, n_beams: int, vocab: int, n_out: int, logits_dtype=torch.bfloat16) -> int:
    if (n_groups | n_beams | vocab | n_out) >> 31 > 0:
        raise _too_large("n_groups, n_beams, vocab, n_out", n_groups, n_beams, vocab, n_out)
    return int(lib().gdn_beam_workspace_size(n_groups, n_beams, vocab, n_out, _DT[logits_dtype]))


def beam_select(logits, scores, n_out=None, finished=None, pad_token=0, parents=None, tokens=None, out_scores=None,
                workspace=None, stream=None):
    """Beam search's selection over beams and vocabulary (gdn_beam_select): of all
    scores[g, w] + log_softmax(logits[g, w])[v], the n_out (default: n_beams) best of each
    group g, best first, ties to the lowest w * vocab + v.

    logits [groups, beams, vocab] bf16 or float32 (the last dimension dense, the rows
    evenly spaced), scores [groups, beams] float32, finished [groups, beams] uint8 or bool
    (such a beam goes on with ``pad_token`` and its score).  Returns (parents, tokens,
    scores), each [groups, n_out]; -1, -1, -inf where there are fewer candidates.
    ``out_scores`` may be ``scores`` when n_out is the number of beams."""
    dev = _index_of(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits [groups, beams, vocab] expected, got %s" % (tuple(logits.shape),))
    G, W, V = logits.shape
    if logits.dtype not in _DT:
        raise TypeError("logits: dtype %s, expected bfloat16 or float32" % logits.dtype)
    dt = _DT[logits.dtype]
    if n_out is None:
        n_out = W
    if (G | W | V | n_out | abs(pad_token)) >> 31:
        raise _too_large("groups, beams, vocab, n_out, pad_token", G, W, V, n_out, pad_token)
    ld = V
    if not logits.is_contiguous():
        ld = logits.stride(1) if W > 1 else logits.stride(0) if G > 1 else V
        if (V > 1 and logits.stride(2) != 1) or (G > 1 and W > 1 and logits.stride(0) != W * ld) or ld < V:
            raise ValueError("logits: rows must be dense and evenly spaced, strides %s" % (logits.stride(),))
    pf = None
    if finished is not None:
        pf = _shaped(finished, "finished", torch.bool if finished.dtype == torch.bool else torch.uint8, dev, (G, W))
    if parents is None:
        parents = _empty((G, n_out), torch.int32, dev, stream)
    if tokens is None:
        tokens = _empty((G, n_out), torch.int32, dev, stream)
    if out_scores is None:
        out_scores = _empty((G, n_out), torch.float32, dev, stream)
    if workspace is None:
        workspace = _empty(beam_workspace_size(G, W, V, n_out, logits.dtype), torch.uint8, dev, stream)
    _call(lib().gdn_beam_select, "gdn_beam_select", dev, stream, logits.data_ptr(), dt, ld,
          _shaped(scores, "scores", torch.float32, dev, (G, W)), pf, G, W, V, n_out, pad_token,
          _shaped(parents, "parents", torch.int32, dev, (G, n_out)), _shaped(tokens, "tokens", torch.int32, dev, (G, n_out)),
          _shaped(out_scores, "out_scores", torch.float32, dev, (G, n_out)), _workspace(workspace, dev), workspace.numel())
    return parents, tokens, out_scores


class ReorderPlan:
    """The states that ``reorder_states`` moves, checked and laid out once."""

    def __init__(self, states, n_groups: int, n_beams: int):
        if not 0 < len(states) <= REORDER_MAX_BUFFERS:
            raise ValueError("1..%d states" % REORDER_MAX_BUFFERS)
        # (aliases: the memory behind the addresses stays while the plan does, even where the
        # caller points a tensor at other memory)
        self.states = [t.detach() for t in states]
        self.n_groups, self.n_beams = int(n_groups), int(n_beams)
        if (self.n_groups | self.n_beams) >> 31:
            raise _too_large("n_groups, n_beams", n_groups, n_beams)
        self.device = _index_of(states[0], "states[0]")
        self.buffers = (_CStateBuffer * len(states))()
        for i, t in enumerate(self.states):
            if t.get_device() != self.device:
                raise ValueError("states[%d] is on %s, expected cuda:%d" % (i, t.device, self.device))
            if t.dim() < 2 or t.shape[0] != self.n_groups * self.n_beams:
                raise ValueError("states[%d]: shape %s, expected [%d, ...]"
                                 % (i, tuple(t.shape), self.n_groups * self.n_beams))
            if t.shape[0] and not t[0].is_contiguous():
                raise ValueError("states[%d]: each sequence's state must be contiguous" % i)
            size = t.element_size()
            b = self.buffers[i]
            b.base, b.bytes = t.data_ptr(), t[0].numel() * size if t.shape[0] else 0
            # (a single sequence's stride says nothing)
            b.stride = t.stride(0) * size if t.shape[0] > 1 else b.bytes


def reorder_plan(states, n_groups: int, n_beams: int) -> ReorderPlan:
    """Checks the states (tensors [n_groups * n_beams, ...], each sequence's part
    contiguous) once, for ``reorder_states`` calls that move them again and again.  The
    plan keeps their memory; a tensor that is pointed at other memory needs a new plan."""
    return ReorderPlan(states, n_groups, n_beams)


def reorder_states(parents, states, stream=None) -> None:
    """After a beam selection: in every state, in place, sequence g * beams + w takes what
    sequence g * beams + parents[g, w] held (gdn_reorder_states).  parents [groups, beams]
    int32, -1 to keep; states a list of tensors [groups * beams, ...] or a
    ``reorder_plan`` of them."""
    if not isinstance(states, ReorderPlan):
        if parents.dim() != 2:
            raise ValueError("parents [groups, beams] expected, got %s" % (tuple(parents.shape),))
        states = ReorderPlan(states, *parents.shape)
    dev = states.device
    _call(lib().gdn_reorder_states, "gdn_reorder_states", dev, stream,
          _shaped(parents, "parents", torch.int32, dev, (states.n_groups, states.n_beams)), states.n_groups,
          states.n_beams, states.buffers, len(states.buffers))


def check_device_error(stream=None) -> None:
    """Synchronise the stream and raise GdnError if the device error word holds an
    error: a bounded wait that ran out, a failed device check of a prefill's
    inputs (malformed cu_seqlens, conv output beyond fp16), or a parent outside its
    group in reorder_states.  Every device has its own word: the one read is that of the
    stream's device (without a stream: of the current one)."""
    index = getattr(stream, "device_index", None)
    if index is not None and index != _current_device():
        with torch.cuda.device(index):
            return check_device_error(stream)
    s = lib().gdn_check_device_error(_stream(stream))
    if s != 0:
        raise GdnError(s, "device")


def prefill_host_workspace_size(cfg: Config, T_total: int, n_seqs: int) -> int:
    c = cfg.c()
    return int(lib().gdn_prefill_host_workspace_size(ctypes.byref(c), T_total, n_seqs))


def prefill_host(cfg: Config, w: dict, host: dict, conv_state, rec_state, workspace=None, stream=None):
    """End-to-end prefill from host buffers through gdn_prefill_host: ``host`` holds CPU
    tensors q, k, v, a, b, z (act dtype), cu_seqlens (int32) and out (out dtype), page-
    locked for the copies to overlap the work.  The states stay on the device.  Returns
    host['out'], complete once the stream is synchronised."""
    dev = rec_state.device
    q = host["q"]
    T = q.shape[0]
    cu = host["cu_seqlens"]
    N = cu.shape[0] - 1
    for n in ("q", "k", "v", "a", "b", "z", "cu_seqlens", "out"):
        t = host[n]
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError("host[%r] must be a contiguous CPU tensor" % n)
    for n in ("q", "k", "v", "a", "b", "z"):
        if host[n].dtype != cfg.act_dtype:
            raise TypeError("host[%r]: dtype %s, expected %s" % (n, host[n].dtype, cfg.act_dtype))
    if cu.dtype != torch.int32 or host["out"].dtype != cfg.out_dtype:
        raise TypeError("cu_seqlens must be int32 and out of the out dtype")
    _check(conv_state, "conv_state", cfg.act_dtype, dev)
    _check(rec_state, "rec_state", cfg.state_dtype, dev)
    if workspace is None:
        workspace = torch.empty(prefill_host_workspace_size(cfg, T, N), dtype=torch.uint8, device=dev)
    c, cw = cfg.c(), _weights(w, dev)
    s = lib().gdn_prefill_host(ctypes.byref(c), ctypes.byref(cw), _ptr(q), _ptr(host["k"]), _ptr(host["v"]),
                               _ptr(host["a"]), _ptr(host["b"]), _ptr(host["z"]), _ptr(conv_state),
                               _ptr(rec_state), _ptr(cu), N, T, _ptr(host["out"]), _ptr(workspace),
                               workspace.numel(), _stream(stream))
    if s != 0:
        raise GdnError(s, "gdn_prefill_host")
    return host["out"]
