"""Python binding of ``libmk.so``, the fused MoE decode-step library for B200.

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of ``libmk.so``; PyTorch supplies device memory and streams.  The
ctypes functions carry the names of the C entry points in ``include/mk.h``;
``Decoder`` is a thin convenience wrapper that takes torch tensors.

There is no fallback: if ``libmk.so`` is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, List, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmk.so")

MK_OK = 0
MK_ERR_ARG = -1
MK_ERR_CAPACITY = -2
MK_ERR_CUDA = -3
MK_ERR_LAUNCH = -4
MK_ERR_TIMEOUT = -5
MK_ERR_DEVICE_CHECK = -6
MK_ERR_UNSUPPORTED = -7

MK_MEGAKERNEL = 0
MK_MULTIKERNEL = 1
MK_MULTIKERNEL_GRAPH = 2
MK_TENSORCORE = 3
VARIANTS = {"megakernel": MK_MEGAKERNEL, "multikernel": MK_MULTIKERNEL,
            "multikernel_graph": MK_MULTIKERNEL_GRAPH, "tensorcore": MK_TENSORCORE}

MK_FAULT_NONE = 0
MK_FAULT_UNREACHABLE_WAIT = 1
MK_TRACE_WORDS = 12  # uint64 words per (op, warp) record of mk_set_trace
MK_F32 = 0   # element types of the paged operators
MK_BF16 = 1
MK_E4M3 = 2
MK_SAMPLE_PHASES = 12  # phase stamps of mk_sample_top_p_phases
MK_STATIC_SCRATCH_BYTES = 32 << 20  # the fixed working array of mk_decode_step_static

OP_NAMES = ["EMBED", "QKV", "ATTN", "OPROJ", "SHARED_GU", "ROUTED_GU", "DOWN", "COMBINE", "LMHEAD"]


class mk_model_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_layers", "d_model", "n_q_heads", "n_kv_heads", "head_dim",
        "n_experts", "top_k", "expert_ffn", "shared_ffn", "vocab")] + [
        ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float),
        ("max_rows", ctypes.c_int32), ("max_seqs", ctypes.c_int32),
        ("kv_capacity", ctypes.c_int32), ("variant", ctypes.c_int32)]


class mk_layer_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "attn_norm", "wqkv", "wo", "ffn_norm", "router", "w_gate", "w_up", "w_down",
        "ws_gate", "ws_up", "ws_down")]


class mk_weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p), ("layers", ctypes.POINTER(mk_layer_weights))]


class mk_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class mk_paged_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p)] + [
        (n, ctypes.c_int32) for n in ("n_pages", "page_size", "max_pages", "n_kv_heads", "head_dim", "dtype")]


class mk_strides(ctypes.Structure):
    _fields_ = [("seq", ctypes.c_int64), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class mk_stats(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_uint64), ("expert_union_total", ctypes.c_uint64),
                ("kernel_launches", ctypes.c_uint64), ("graph_launches", ctypes.c_uint64)]


class mk_plan_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_ops", "n_cta", "warps_per_cta", "rows_per_tile", "mmax", "attn_chunk",
        "attn_qsplit", "smem_bytes")] + [("scratch_bytes", ctypes.c_int64)]


class MkError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"mk error {code}: {msg}")
        self.code = code


_lib = None
_I32P = ctypes.POINTER(ctypes.c_int32)


def lib():
    """Load ``libmk.so``; raise if it is missing (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with decode_megakernel_06_b200/build.py")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64
    kvp = ctypes.POINTER(mk_paged_kv)
    sig = {
        "mk_create": (i32, [ctypes.POINTER(mk_model_desc), ctypes.POINTER(mk_weights), ctypes.POINTER(vp)]),
        "mk_decode_step": (i32, [vp, vp, vp, i32, i32, mk_kv_cache, vp, vp, vp]),
        "mk_decode_steps": (i32, [vp, vp, vp, i32, i32, mk_kv_cache, vp, vp, vp]),
        "mk_verify_steps": (i32, [vp, vp, vp, i32, i32, i32, vp, i32, mk_kv_cache, vp, vp, vp, vp]),
        "mk_decode_step_host": (i32, [vp, _I32P, _I32P, i32, i32, mk_kv_cache, vp, _I32P, vp]),
        "mk_decode_step_static": (i32, [vp, vp, vp, i32, i32, mk_kv_cache, vp, vp, vp]),
        "mk_sample_top_p": (i32, [vp, i32, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp]),
        "mk_sample_top_p_phases": (i32, [vp, i32, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp, vp]),
        "mk_decode_step_sample": (i32, [vp, vp, vp, i32, i32, mk_kv_cache, vp, ctypes.c_float,
                                        ctypes.c_float, vp, vp, vp]),
        "mk_decode_steps_sample": (i32, [vp, vp, vp, i32, i32, mk_kv_cache, vp, ctypes.c_float,
                                         ctypes.c_float, vp, vp, vp]),
        "mk_kv_append": (i32, [kvp, vp, mk_strides, vp, mk_strides, i32, vp, vp, i32, i32, vp, i32, vp]),
        "mk_kv_gather": (i32, [kvp, vp, vp, i32, i32, vp, mk_strides, vp, mk_strides, i32, vp]),
        "mk_paged_attention_workspace": (u64, []),
        "mk_paged_attention": (i32, [kvp, vp, mk_strides, i32, i32, vp, vp, i32, i32, ctypes.c_float, vp, i32, vp,
                                     vp, u64, vp]),
        "mk_decode_step_paged": (i32, [vp, vp, vp, i32, i32, kvp, vp, vp, vp]),
        "mk_verify_sample_workspace": (u64, [i32, i32]),
        "mk_verify_sample": (i32, [vp, vp, vp, i32, i32, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp, vp, u64,
                                   vp]),
        "mk_get_device_status": (i32, [vp, vp]),
        "mk_last_device_error_op": (i32, [vp]),
        "mk_last_error": (ctypes.c_char_p, []),
        "mk_destroy": (None, [vp]),
        "mk_set_variant": (i32, [vp, i32]),
        "mk_set_timeout": (i32, [vp, u64]),
        "mk_set_debug": (i32, [vp, vp, vp, vp]),
        "mk_debug_inject": (i32, [vp, i32]),
        "mk_set_trace": (i32, [vp, vp]),
        "mk_get_stats": (i32, [vp, ctypes.POINTER(mk_stats), i32]),
        "mk_hbm_read_probe": (i32, [vp, u64, i32, i32, ctypes.POINTER(ctypes.c_double), vp]),
        "mk_validate_desc": (i32, [ctypes.POINTER(mk_model_desc)]),
        "mk_plan_describe": (i32, [ctypes.POINTER(mk_model_desc), i32, i32, i32,
                                   ctypes.POINTER(mk_plan_info), _I32P, _I32P, _I32P, _I32P, i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def mk_last_error() -> str:
    return lib().mk_last_error().decode()


def _check(rc: int) -> int:
    if rc != MK_OK:
        raise MkError(rc, mk_last_error())
    return rc


# ---- same-named wrappers of the C entry points ---------------------------------

def mk_validate_desc(desc: mk_model_desc) -> int:
    return lib().mk_validate_desc(ctypes.byref(desc))


def mk_plan_describe(desc: mk_model_desc, n_sm: int, B: int, T: int):
    """Returns (rc, mk_plan_info, [(type, layer, dep0, dep1)] per op)."""
    info = mk_plan_info()
    n = 8 * desc.n_layers + 2  # an upper bound on the schedule's length
    arrs = [(ctypes.c_int32 * n)() for _ in range(4)]
    rc = lib().mk_plan_describe(ctypes.byref(desc), n_sm, B, T, ctypes.byref(info),
                                *[ctypes.cast(a, _I32P) for a in arrs], n)
    ops = list(zip(*[list(a)[:info.n_ops] for a in arrs])) if rc == MK_OK else []
    return rc, info, ops


def mk_create(desc: mk_model_desc, weights: mk_weights) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(lib().mk_create(ctypes.byref(desc), ctypes.byref(weights), ctypes.byref(h)))
    return h


def mk_decode_steps(h, tokens: int, positions: int, B: int, n_steps: int, kv: mk_kv_cache,
                    out_logits: int, out_tokens: int, stream: int) -> int:
    """n_steps greedy steps in one launch (see include/mk.h)."""
    return lib().mk_decode_steps(h, tokens, positions, B, n_steps, kv, out_logits, out_tokens, stream)


def mk_verify_steps(h, tokens: int, positions: int, B: int, T: int, n_steps: int, drafts: int,
                    draft_len: int, kv: mk_kv_cache, out_logits: int, out_tokens: int,
                    out_accepted: int, stream: int) -> int:
    """n_steps speculative-verify steps in one launch (see include/mk.h)."""
    return lib().mk_verify_steps(h, tokens, positions, B, T, n_steps, drafts, draft_len, kv, out_logits,
                                 out_tokens, out_accepted, stream)


def mk_decode_step(h, tokens: int, positions: int, B: int, T: int, kv: mk_kv_cache,
                   out_logits: int, out_argmax: int, stream: int) -> int:
    return lib().mk_decode_step(h, tokens, positions, B, T, kv, out_logits, out_argmax, stream)


def mk_decode_step_host(h, tokens_host, positions_host, B: int, T: int, kv: mk_kv_cache,
                        out_logits: int, out_argmax_host, stream: int) -> int:
    return lib().mk_decode_step_host(h, tokens_host, positions_host, B, T, kv, out_logits,
                                     out_argmax_host, stream)


def mk_decode_step_static(h, tokens: int, positions: int, B: int, T: int, kv: mk_kv_cache,
                          out_logits: int, out_argmax: int, stream: int) -> int:
    return lib().mk_decode_step_static(h, tokens, positions, B, T, kv, out_logits, out_argmax,
                                       stream)


def mk_sample_top_p(logits: int, rows: int, vocab: int, temperature: float, top_p: float,
                    uniforms: int, out_tokens: int, stream: int) -> int:
    return lib().mk_sample_top_p(logits, rows, vocab, temperature, top_p, uniforms, out_tokens, stream)


def mk_sample_top_p_phases(logits: int, rows: int, vocab: int, temperature: float, top_p: float,
                           uniforms: int, out_tokens: int, stamps: int, stream: int = 0) -> int:
    return lib().mk_sample_top_p_phases(logits, rows, vocab, temperature, top_p, uniforms, out_tokens, stamps,
                                        stream)


def mk_decode_step_sample(h, tokens: int, positions: int, B: int, T: int, kv: mk_kv_cache,
                          out_logits: int, temperature: float, top_p: float, uniforms: int,
                          out_tokens: int, stream: int) -> int:
    return lib().mk_decode_step_sample(h, tokens, positions, B, T, kv, out_logits, temperature, top_p,
                                       uniforms, out_tokens, stream)


def mk_decode_steps_sample(h, tokens: int, positions: int, B: int, n_steps: int, kv: mk_kv_cache,
                           out_logits: int, temperature: float, top_p: float, uniforms: int,
                           out_tokens: int, stream: int) -> int:
    """n_steps sampled steps as one graph launch (see include/mk.h)."""
    return lib().mk_decode_steps_sample(h, tokens, positions, B, n_steps, kv, out_logits, temperature, top_p,
                                        uniforms, out_tokens, stream)


def mk_kv_append(kv: mk_paged_kv, k: int, ks: mk_strides, v: int, vs: mk_strides, in_dtype: int, positions: int,
                 counts: Optional[int], B: int, T: int, rope: Optional[int], rope_len: int, stream: int) -> int:
    """New rows into the pages of a cache (see include/mk.h)."""
    return lib().mk_kv_append(ctypes.byref(kv), k, ks, v, vs, in_dtype, positions, counts, B, T, rope, rope_len, stream)


def mk_kv_gather(kv: mk_paged_kv, starts: int, counts: Optional[int], B: int, T: int, k: int, ks: mk_strides, v: int,
                 vs: mk_strides, out_dtype: int, stream: int) -> int:
    """Positions of a paged cache read back (see include/mk.h)."""
    return lib().mk_kv_gather(ctypes.byref(kv), starts, counts, B, T, k, ks, v, vs, out_dtype, stream)


def mk_paged_attention_workspace() -> int:
    return lib().mk_paged_attention_workspace()


def mk_paged_attention(kv: mk_paged_kv, q: int, qs: mk_strides, dtype: int, n_q_heads: int, positions: int,
                       counts: Optional[int], B: int, T: int, scale: float, rope: Optional[int], rope_len: int,
                       out: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Attention of the newest rows over the pages (see include/mk.h)."""
    return lib().mk_paged_attention(ctypes.byref(kv), q, qs, dtype, n_q_heads, positions, counts, B, T, scale, rope,
                                    rope_len, out, workspace, workspace_bytes, stream)


def mk_decode_step_paged(h, tokens: int, positions: int, B: int, T: int, layers, out_logits: Optional[int],
                         out_argmax: int, stream: int) -> int:
    """One step over a paged cache; layers: a ctypes array of mk_paged_kv (see include/mk.h)."""
    return lib().mk_decode_step_paged(h, tokens, positions, B, T, layers, out_logits, out_argmax, stream)


def mk_verify_sample_workspace(B: int, T: int) -> int:
    return lib().mk_verify_sample_workspace(B, T)


def mk_verify_sample(logits: int, draft_logits: Optional[int], tokens: int, B: int, T: int, vocab: int,
                     temperature: float, top_p: float, uniforms: Optional[int], out_tokens: int, out_accepted: int,
                     workspace: int, workspace_bytes: int, stream: int) -> int:
    """Acceptance of drafts by the target's probabilities (see include/mk.h)."""
    return lib().mk_verify_sample(logits, draft_logits, tokens, B, T, vocab, temperature, top_p, uniforms, out_tokens,
                                  out_accepted, workspace, workspace_bytes, stream)


def _need(t, dtype, min_numel: int, name: str, device=None, dims: Optional[int] = None):
    """Check a tensor handed to a kernel by its data pointer: dtype, a
    contiguous layout with at least ``min_numel`` elements, optionally the
    number of dimensions, then that it lives on ``device`` (a CUDA device).
    A wrong tensor would otherwise make the kernel read or write past it."""
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name}: {t.dim()}-D, expected {dims}-D")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {min_numel} needed")
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name}: on {t.device}, expected " + (str(device) if device is not None else "a CUDA device"))


def _fits(t, dtype, min_numel: int, index: int) -> bool:
    """Whether _need would accept t, on CUDA device ``index``."""
    return t is not None and t.dtype is dtype and t.get_device() == index and t.numel() >= min_numel and t.is_contiguous()


def sample_top_p(logits, temperature: float, top_p: float, uniforms, out_tokens, stream=None) -> int:
    """Torch-tensor form of mk_sample_top_p: logits fp32 [rows, vocab], uniforms
    fp64 [rows] (or None when temperature <= 0), out_tokens int32 [rows], all
    contiguous on one CUDA device (checked: ValueError otherwise).  Returns the
    launch status code."""
    import torch

    _need(logits, torch.float32, 1, "logits", dims=2)
    rows, vocab = logits.shape
    if uniforms is not None:
        _need(uniforms, torch.float64, rows, "uniforms", logits.device)
    _need(out_tokens, torch.int32, rows, "out_tokens", logits.device)
    s = stream if stream is not None else torch.cuda.current_stream()
    return mk_sample_top_p(logits.data_ptr(), rows, vocab, temperature, top_p, _ptr(uniforms),
                           out_tokens.data_ptr(), s.cuda_stream)


def sample_top_p_phases(logits, temperature: float, top_p: float, uniforms, out_tokens, stamps, stream=None) -> int:
    """sample_top_p, also writing the device clock (ns) at each of the
    MK_SAMPLE_PHASES phase boundaries of row 0 into ``stamps`` (int64 CUDA
    tensor of at least MK_SAMPLE_PHASES elements; see mk_sample_top_p_phases).
    The same checks as sample_top_p; returns the launch status code."""
    import torch

    _need(logits, torch.float32, 1, "logits", dims=2)
    rows, vocab = logits.shape
    if uniforms is not None:
        _need(uniforms, torch.float64, rows, "uniforms", logits.device)
    _need(out_tokens, torch.int32, rows, "out_tokens", logits.device)
    _need(stamps, torch.int64, MK_SAMPLE_PHASES, "stamps", logits.device)
    s = stream if stream is not None else torch.cuda.current_stream()
    return mk_sample_top_p_phases(logits.data_ptr(), rows, vocab, temperature, top_p, _ptr(uniforms),
                                  out_tokens.data_ptr(), stamps.data_ptr(), s.cuda_stream)


def _call_on(index: int, call, *args) -> int:
    """call(*args) with device ``index`` current."""
    import torch

    back = torch.cuda.current_device()
    if back == index:
        return call(*args)
    torch.cuda.set_device(index)
    try:
        return call(*args)
    finally:
        torch.cuda.set_device(back)


def _raw_stream(index: int, stream) -> int:
    """The CUDA stream of a call on device ``index``: the given one, which has to
    be that device's, or its current one."""
    global _current_raw_stream
    if stream is None:
        if _current_raw_stream is None:
            import torch

            _current_raw_stream = torch._C._cuda_getCurrentRawStream
        return _current_raw_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream: on {stream.device}, expected cuda:{index}")
    return stream.cuda_stream


_current_raw_stream = None


@functools.lru_cache(maxsize=1024)
def _strides(seq: int, token: int, head: int) -> mk_strides:
    """The struct of an operand's strides (passed by value)."""
    return mk_strides(seq, token, head)


class PagedKV:
    """One layer's paged cache over torch tensors: ``k`` and ``v`` are bf16 or
    float8_e4m3fn [n_pages, n_kv_heads, page_size, head_dim], ``page_table`` is
    int32 [B, max_pages] for the B sequences of a call, and an 8-bit cache has
    fp32 scales [n_pages, n_kv_heads, page_size].  All contiguous, on one CUDA
    device (ValueError otherwise).  The tensors are kept, not copied; the
    operators are those of include/mk.h and return its status codes."""

    def __init__(self, k, v, page_table, k_scale=None, v_scale=None):
        import torch

        kinds = {torch.bfloat16: MK_BF16, torch.float8_e4m3fn: MK_E4M3}
        if k.dtype not in kinds:
            raise ValueError(f"k: dtype {k.dtype}, expected bfloat16 or float8_e4m3fn")
        _need(k, k.dtype, 1, "k", dims=4)
        self.device = k.device
        _need(v, k.dtype, 1, "v", self.device, dims=4)
        if v.shape != k.shape:
            raise ValueError(f"v: shape {tuple(v.shape)}, expected {tuple(k.shape)}")
        _need(page_table, torch.int32, 1, "page_table", self.device, dims=2)
        n_pages, heads, page, hd = k.shape
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if (t is not None) != (k.dtype == torch.float8_e4m3fn):
                raise ValueError(f"{name}: given for an 8-bit cache, and only for one")
            if t is not None:
                _need(t, torch.float32, 1, name, self.device, dims=3)
                if t.shape != k.shape[:3]:
                    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(k.shape[:3])}")
        self.k, self.v, self.k_scale, self.v_scale, self.page_table = k, v, k_scale, v_scale, page_table
        self.desc = mk_paged_kv(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), page_table.data_ptr(),
                                n_pages, page, page_table.shape[1], heads, hd, kinds[k.dtype])
        self._index, self._batch, self._heads, self._hd = self.device.index, page_table.shape[0], heads, hd
        self._kinds = {torch.float32: MK_F32, torch.bfloat16: MK_BF16}
        self._int, self._byte = torch.int32, torch.uint8
        self._lib, self._ref = lib(), ctypes.byref(self.desc)
        self._current_device = torch.cuda.current_device

    def _rows(self, t, name: str, heads: Optional[int]):
        """Checks a [B, T, heads, head_dim] operand (fp32 or bf16, any strides but a
        contiguous head_dim); returns its shape, strides and type."""
        shape, st, kind = t.shape, t.stride(), self._kinds.get(t.dtype)
        if (kind is None or len(shape) != 4 or shape[3] != self._hd or shape[0] != self._batch or st[3] != 1
                or (heads is not None and shape[2] != heads) or t.get_device() != self._index):
            if kind is None:
                raise ValueError(f"{name}: dtype {t.dtype}, expected float32 or bfloat16")
            if len(shape) == 4 and shape[3] == self._hd and st[3] != 1:
                raise ValueError(f"{name}: the head dimension must be contiguous")
            if t.get_device() != self._index:
                raise ValueError(f"{name}: on {t.device}, expected {self.device}")
            raise ValueError(f"{name}: shape {tuple(shape)}, expected [{self._batch}, T, "
                             f"{'heads' if heads is None else heads}, {self._hd}]")
        return shape, st, kind

    def _call(self, call, *args) -> int:
        """call(cache, *args) with the cache's device current."""
        if self._current_device() == self._index:
            return call(self._ref, *args)
        return _call_on(self._index, call, self._ref, *args)

    def _pair(self, x, y, names: Sequence[str]):
        """Two such operands of one shape and type: (B, T), the type and both strides."""
        shape, st, kind = self._rows(x, names[0], self._heads)
        other, st2, kind2 = self._rows(y, names[1], self._heads)
        if other != shape or kind2 != kind:
            raise ValueError(f"{names[1]}: {tuple(other)} {y.dtype}, expected {tuple(shape)} {x.dtype}")
        return shape[0], shape[1], kind, st, st2

    def _ints(self, t, name: str) -> int:
        """An int32 operand with an entry per sequence; its pointer."""
        if t.dtype != self._int or t.numel() < self._batch or not t.is_contiguous() or t.get_device() != self._index:
            _need(t, self._int, self._batch, name, self.device)
        return t.data_ptr()

    def _rope(self, rope):
        """The rotary table's pointer and number of positions (None, 0 without one)."""
        if rope is None:
            return None, 0
        shape = rope.shape
        if (self._kinds.get(rope.dtype) != MK_F32 or len(shape) != 3 or shape[1] != self._hd // 2 or shape[2] != 2
                or shape[0] < 1 or not rope.is_contiguous() or rope.get_device() != self._index):
            import torch

            _need(rope, torch.float32, 1, "rope", self.device, dims=3)
            raise ValueError(f"rope: shape {tuple(shape)}, expected [positions, {self._hd // 2}, 2]")
        return rope.data_ptr(), shape[0]

    def append(self, k, v, positions, counts=None, rope=None, stream=None) -> int:
        """mk_kv_append: rows k, v [B, T, n_kv_heads, head_dim] at positions[b] + t
        (rows t >= counts[b] are not written); with rope, k is rotated first."""
        B, T, kind, ks, vs = self._pair(k, v, ("k", "v"))
        pos = self._ints(positions, "positions")
        cnt = None if counts is None else self._ints(counts, "counts")
        table, n = self._rope(rope)
        return self._call(self._lib.mk_kv_append, k.data_ptr(), _strides(*ks[:3]), v.data_ptr(), _strides(*vs[:3]), kind,
                          pos, cnt, B, T, table, n, _raw_stream(self._index, stream))

    def gather(self, starts, out_k, out_v, counts=None, stream=None) -> int:
        """mk_kv_gather: positions starts[b] + t into out_k, out_v
        [B, T, n_kv_heads, head_dim] (any strides, e.g. a contiguous cache
        [B, heads, capacity, head_dim] transposed)."""
        B, T, kind, ks, vs = self._pair(out_k, out_v, ("out_k", "out_v"))
        for name, s in (("out_k", ks), ("out_v", vs)):
            if 0 in s and ((s[0] == 0 and B > 1) or (s[1] == 0 and T > 1) or (s[2] == 0 and self._heads > 1)):
                raise ValueError(f"{name}: written rows must not share memory")
        pos = self._ints(starts, "starts")
        cnt = None if counts is None else self._ints(counts, "counts")
        return self._call(self._lib.mk_kv_gather, pos, cnt, B, T, out_k.data_ptr(), _strides(*ks[:3]), out_v.data_ptr(),
                          _strides(*vs[:3]), kind, _raw_stream(self._index, stream))

    def attention(self, q, positions, out, workspace, counts=None, scale: Optional[float] = None, rope=None,
                  stream=None) -> int:
        """mk_paged_attention: rows q [B, T, n_q_heads, head_dim] at positions[b] + t
        over the cache, into out (contiguous, like q); scale defaults to
        1 / sqrt(head_dim).  ``workspace`` is paged_attention_workspace's."""
        shape, st, kind = self._rows(q, "q", None)
        if out.dtype != q.dtype or out.shape != shape or not out.is_contiguous() or out.get_device() != self._index:
            _need(out, q.dtype, 1, "out", self.device, dims=4)
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {tuple(shape)}")
        pos = self._ints(positions, "positions")
        cnt = None if counts is None else self._ints(counts, "counts")
        table, n = self._rope(rope)
        if workspace.dtype != self._byte or not workspace.is_contiguous() or workspace.get_device() != self._index:
            _need(workspace, self._byte, 1, "workspace", self.device)
        if scale is None:
            scale = self._hd ** -0.5
        return self._call(self._lib.mk_paged_attention, q.data_ptr(), _strides(*st[:3]), kind, shape[2], pos, cnt,
                          shape[0], shape[1], scale, table, n, out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                          _raw_stream(self._index, stream))


def paged_attention_workspace(device):
    """A workspace of PagedKV.attention on ``device`` (uint8, zeroed once).  Calls
    that may overlap on the GPU need one each."""
    import torch

    with torch.cuda.device(device):
        n = mk_paged_attention_workspace()
        if n == 0:
            raise MkError(MK_ERR_CUDA, mk_last_error())
        return torch.zeros(n, dtype=torch.uint8, device=device)


def verify_sample_workspace(B: int, T: int, vocab: int, device):
    """A workspace of verify_sample for blocks of that size (uint8)."""
    import torch

    n = mk_verify_sample_workspace(B, T)
    if n == 0 or vocab < 1:
        raise ValueError(f"B, T and vocab must be >= 1 (got {B}, {T}, {vocab})")
    return torch.empty(n, dtype=torch.uint8, device=device)


def verify_sample(logits, tokens, temperature: float, top_p: float, uniforms, out_tokens, out_accepted, workspace,
                  draft_logits=None, stream=None) -> int:
    """Torch-tensor form of mk_verify_sample: logits fp32 [B, T, vocab], tokens int32
    [B, T] (the last accepted token, then the drafts), draft_logits fp32
    [B, T - 1, vocab] or None, uniforms fp64 [B, T] (None when temperature <= 0),
    out_tokens int32 [B, T], out_accepted int32 [B], all contiguous on one CUDA
    device (ValueError otherwise).  Returns the launch status code."""
    import torch

    if logits.dim() != 3 or not _fits(logits, torch.float32, 1, logits.get_device()) or not logits.is_cuda:
        _need(logits, torch.float32, 1, "logits", dims=3)
    index = logits.get_device()
    B, T, vocab = logits.shape
    rows = B * T
    for t, dtype, n, name in ((tokens, torch.int32, rows, "tokens"), (uniforms, torch.float64, rows, "uniforms"),
                              (out_tokens, torch.int32, rows, "out_tokens"),
                              (out_accepted, torch.int32, B, "out_accepted"), (workspace, torch.uint8, 1, "workspace"),
                              (draft_logits, torch.float32, 0, "draft_logits")):
        if not _fits(t, dtype, n, index) and (t is not None or name not in ("uniforms", "draft_logits")):
            _need(t, dtype, n, name, logits.device)
    if draft_logits is not None and draft_logits.shape != (B, T - 1, vocab):
        raise ValueError(f"draft_logits: shape {tuple(draft_logits.shape)}, expected {(B, T - 1, vocab)}")
    args = (logits.data_ptr(), _ptr(draft_logits) if T > 1 else None, tokens.data_ptr(), B, T, vocab, temperature, top_p,
            _ptr(uniforms), out_tokens.data_ptr(), out_accepted.data_ptr(), workspace.data_ptr(), workspace.numel(),
            _raw_stream(index, stream))
    return _call_on(index, lib().mk_verify_sample, *args)


def hbm_read_probe(buf, form: int = 0, reps: int = 5, stream=None) -> float:
    """Read-only HBM bandwidth in GB/s over the CUDA tensor ``buf`` (16-byte
    aligned, >= 64 MiB; see mk_hbm_read_probe).  Raises on failure."""
    import torch

    if buf.device.type != "cuda" or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    s = stream if stream is not None else torch.cuda.current_stream()
    out = ctypes.c_double(0.0)
    _check(lib().mk_hbm_read_probe(buf.data_ptr(), buf.numel() * buf.element_size(), form, reps,
                                   ctypes.byref(out), s.cuda_stream))
    return out.value


def mk_get_device_status(h, stream: int) -> int:
    return lib().mk_get_device_status(h, stream)


def mk_last_device_error_op(h) -> int:
    return lib().mk_last_device_error_op(h)


def mk_destroy(h) -> None:
    lib().mk_destroy(h)


def mk_set_variant(h, variant: int) -> int:
    return lib().mk_set_variant(h, variant)


def mk_set_timeout(h, ns: int) -> int:
    return lib().mk_set_timeout(h, ns)


def mk_set_debug(h, hidden: int, expert_ids: int, expert_w: int) -> int:
    return lib().mk_set_debug(h, hidden, expert_ids, expert_w)


def mk_set_trace(h, trace: int) -> int:
    return lib().mk_set_trace(h, trace)


def mk_debug_inject(h, fault: int) -> int:
    return lib().mk_debug_inject(h, fault)


def mk_get_stats(h, reset: bool = False) -> mk_stats:
    s = mk_stats()
    _check(lib().mk_get_stats(h, ctypes.byref(s), 1 if reset else 0))
    return s


# ---- convenience wrapper over torch tensors -------------------------------------

def make_desc(model, max_rows: int, max_seqs: int, kv_capacity: int,
              variant: int = MK_MEGAKERNEL) -> mk_model_desc:
    """Descriptor from any object with the decoder's dimension attributes."""
    return mk_model_desc(model.n_layers, model.d_model, model.n_q_heads, model.n_kv_heads,
                         model.head_dim, model.n_experts, model.top_k, model.expert_ffn,
                         model.shared_ffn, model.vocab, float(model.rope_theta),
                         float(model.rms_eps), max_rows, max_seqs, kv_capacity, variant)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class Decoder:
    """A handle over torch-resident weights (dict as produced by the synthetic
    generator: embed, final_norm, lm_head, layers[...])."""

    def __init__(self, model, weights: Dict[str, object], max_rows: int, max_seqs: int,
                 kv_capacity: int, variant: str = "megakernel"):
        import torch

        self.model = model
        self.max_rows, self.max_seqs, self.kv_capacity = max_rows, max_seqs, kv_capacity
        self.desc = make_desc(model, max_rows, max_seqs, kv_capacity, VARIANTS[variant])
        layers = (mk_layer_weights * model.n_layers)()
        for l, lw in enumerate(weights["layers"]):
            layers[l] = mk_layer_weights(*[_ptr(lw.get(n)) for n in (
                "attn_norm", "wqkv", "wo", "ffn_norm", "router", "w_gate", "w_up", "w_down",
                "ws_gate", "ws_up", "ws_down")])
        self._layers = layers
        self._weights = weights
        self.w = mk_weights(_ptr(weights["embed"]), _ptr(weights["final_norm"]),
                            _ptr(weights["lm_head"]), layers)
        self.h = mk_create(self.desc, self.w)
        self._torch = torch

    def close(self):
        if self.h:
            mk_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_variant(self, variant: str):
        _check(mk_set_variant(self.h, VARIANTS[variant]))

    def set_timeout(self, ns: int):
        _check(mk_set_timeout(self.h, ns))

    def set_debug(self, hidden=None, expert_ids=None, expert_w=None):
        _check(mk_set_debug(self.h, _ptr(hidden), _ptr(expert_ids), _ptr(expert_w)))

    def set_trace(self, trace=None):
        _check(mk_set_trace(self.h, _ptr(trace)))

    def inject(self, fault: int):
        _check(mk_debug_inject(self.h, fault))

    def _io(self, tokens, positions, B: int, rows: int, k_cache, v_cache, logits=None):
        """The checks every device-tensor call shares (ValueError on a mismatch)."""
        t = self._torch
        _need(tokens, t.int32, rows, "tokens")
        dev = tokens.device
        _need(positions, t.int32, B, "positions", dev)
        kv_numel = (self.model.n_layers * self.max_seqs * self.model.n_kv_heads * self.kv_capacity
                    * self.model.head_dim)
        _need(k_cache, t.bfloat16, kv_numel, "k_cache", dev)
        _need(v_cache, t.bfloat16, kv_numel, "v_cache", dev)
        if logits is not None:
            _need(logits, t.float32, rows * self.model.vocab, "logits", dev)
        return dev

    def step(self, tokens, positions, B: int, T: int, k_cache, v_cache, logits, argmax,
             stream=None) -> int:
        """Enqueue one step (device tensors); returns the launch status code."""
        dev = self._io(tokens, positions, B, B * T, k_cache, v_cache, logits)
        _need(argmax, self._torch.int32, B * T, "argmax", dev)
        s = stream if stream is not None else self._torch.cuda.current_stream()
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        return mk_decode_step(self.h, tokens.data_ptr(), positions.data_ptr(), B, T, kv,
                              _ptr(logits), argmax.data_ptr(), s.cuda_stream)

    def step_sample(self, tokens, positions, B: int, T: int, k_cache, v_cache, logits, temperature: float,
                    top_p: float, uniforms, out_tokens, stream=None) -> int:
        """One step whose next tokens are sampled (temperature / top-p) from its
        logits with the given fp64 uniforms [B*T].  Returns the launch status code."""
        dev = self._io(tokens, positions, B, B * T, k_cache, v_cache, logits)
        if uniforms is not None:
            _need(uniforms, self._torch.float64, B * T, "uniforms", dev)
        _need(out_tokens, self._torch.int32, B * T, "out_tokens", dev)
        s = stream if stream is not None else self._torch.cuda.current_stream()
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        return mk_decode_step_sample(self.h, tokens.data_ptr(), positions.data_ptr(), B, T, kv,
                                     _ptr(logits), temperature, top_p, _ptr(uniforms),
                                     out_tokens.data_ptr(), s.cuda_stream)

    def step_paged(self, tokens, positions, B: int, T: int, layers: "Sequence[PagedKV]", logits, argmax,
                   stream=None) -> int:
        """One step over paged caches, one PagedKV per layer with a page table of
        at least B rows.  Returns the launch status code."""
        t = self._torch
        _need(tokens, t.int32, B * T, "tokens")
        dev = tokens.device
        _need(positions, t.int32, B, "positions", dev)
        if logits is not None:
            _need(logits, t.float32, B * T * self.model.vocab, "logits", dev)
        _need(argmax, t.int32, B * T, "argmax", dev)
        if len(layers) != self.model.n_layers:
            raise ValueError(f"layers: {len(layers)}, the model has {self.model.n_layers}")
        for i, kv in enumerate(layers):
            if kv.device != dev:
                raise ValueError(f"layer {i}: on {kv.device}, expected {dev}")
            if kv.page_table.shape[0] < B:
                raise ValueError(f"layer {i}: a page table of {kv.page_table.shape[0]} sequences, {B} needed")
        descs = (mk_paged_kv * len(layers))(*[kv.desc for kv in layers])
        return _call_on(dev.index, mk_decode_step_paged, self.h, tokens.data_ptr(), positions.data_ptr(), B, T, descs,
                        _ptr(logits), argmax.data_ptr(), _raw_stream(dev.index, stream))

    def steps_sample(self, tokens, positions, B: int, n_steps: int, k_cache, v_cache, logits,
                     temperature: float, top_p: float, uniforms, out_tokens, stream=None) -> int:
        """n_steps sampled steps as one graph launch; uniforms is fp64
        [n_steps, B] (None for greedy), out_tokens int32 [n_steps, B] on the
        device.  Returns the launch status code."""
        dev = self._io(tokens, positions, B, B, k_cache, v_cache, logits)
        if uniforms is not None:
            _need(uniforms, self._torch.float64, n_steps * B, "uniforms", dev)
        _need(out_tokens, self._torch.int32, n_steps * B, "out_tokens", dev)
        s = stream if stream is not None else self._torch.cuda.current_stream()
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        return mk_decode_steps_sample(self.h, tokens.data_ptr(), positions.data_ptr(), B, n_steps, kv,
                                      _ptr(logits), temperature, top_p, _ptr(uniforms),
                                      out_tokens.data_ptr(), s.cuda_stream)

    def steps(self, tokens, positions, B: int, n_steps: int, k_cache, v_cache, logits, out_tokens,
              stream=None) -> int:
        """Enqueue n_steps greedy steps as one launch; out_tokens is int32
        [n_steps, B] on the device.  Returns the launch status code."""
        dev = self._io(tokens, positions, B, B, k_cache, v_cache, logits)
        _need(out_tokens, self._torch.int32, n_steps * B, "out_tokens", dev)
        s = stream if stream is not None else self._torch.cuda.current_stream()
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        return mk_decode_steps(self.h, tokens.data_ptr(), positions.data_ptr(), B, n_steps, kv,
                               _ptr(logits), out_tokens.data_ptr(), s.cuda_stream)

    def verify_steps(self, tokens, positions, B: int, T: int, n_steps: int, drafts, k_cache, v_cache,
                     logits, out_tokens, out_accepted, stream=None) -> int:
        """Enqueue n_steps verify blocks of T rows as one launch; drafts is int32
        [B, draft_len] on the device, out_tokens [n_steps, B*T], out_accepted
        [n_steps, B].  Returns the launch status code."""
        dev = self._io(tokens, positions, B, B * T, k_cache, v_cache, logits)
        _need(drafts, self._torch.int32, B * drafts.shape[-1], "drafts", dev, dims=2)
        _need(out_tokens, self._torch.int32, n_steps * B * T, "out_tokens", dev)
        _need(out_accepted, self._torch.int32, n_steps * B, "out_accepted", dev)
        s = stream if stream is not None else self._torch.cuda.current_stream()
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        return mk_verify_steps(self.h, tokens.data_ptr(), positions.data_ptr(), B, T, n_steps,
                               drafts.data_ptr(), drafts.shape[-1], kv, _ptr(logits),
                               out_tokens.data_ptr(), out_accepted.data_ptr(), s.cuda_stream)

    def step_static(self, tokens, positions, B: int, T: int, k_cache, v_cache, logits, argmax,
                    stream=None) -> int:
        """Like ``step``, but the step's working memory is the library's fixed
        device array (no allocation; overlapping calls on one device race)."""
        dev = self._io(tokens, positions, B, B * T, k_cache, v_cache, logits)
        _need(argmax, self._torch.int32, B * T, "argmax", dev)
        s = stream if stream is not None else self._torch.cuda.current_stream()
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        return mk_decode_step_static(self.h, tokens.data_ptr(), positions.data_ptr(), B, T, kv,
                                     _ptr(logits), argmax.data_ptr(), s.cuda_stream)

    def step_host(self, tokens_host, positions_host, B: int, T: int, k_cache, v_cache,
                  argmax_host, logits=None, stream=None) -> int:
        """Host-buffer step: int32 CPU tensors in/out (pinned is fastest)."""
        s = stream if stream is not None else self._torch.cuda.current_stream()
        kv = mk_kv_cache(k_cache.data_ptr(), v_cache.data_ptr())
        cast = lambda t: ctypes.cast(t.data_ptr(), _I32P)  # noqa: E731
        return mk_decode_step_host(self.h, cast(tokens_host), cast(positions_host), B, T, kv,
                                   _ptr(logits), cast(argmax_host), s.cuda_stream)

    def status(self, stream=None) -> int:
        s = stream if stream is not None else self._torch.cuda.current_stream()
        return mk_get_device_status(self.h, s.cuda_stream)

    def stats(self, reset: bool = False) -> mk_stats:
        return mk_get_stats(self.h, reset)
