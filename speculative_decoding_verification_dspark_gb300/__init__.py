"""Python binding of libdspark.so (ctypes): argument marshalling only.

Every step of the verification path runs in the library's CUDA kernels; this
module converts torch tensors to raw device pointers, passes the current CUDA
stream, and turns non-zero status codes into exceptions.  PyTorch is used for
device memory and streams only.  Importing works without a GPU; calling needs
one (sm_103a) and the built library -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "COMPACT", "STATIC", "CAP_ACCEPT", "F32", "BF16", "DSparkError", "lib", "load",
    "block_rows_hint_for",
    "schedule", "pack", "verify_attn", "accept", "accept_noalloc", "compact", "read_device_error",
    "verify_attn_workspace_size", "accept_workspace_size", "compact_workspace_size",
    "VerifyStep", "StepGraph", "CalibStore", "DEVERR",
    "qk_norm_rope", "KV4_BLOCK_BYTES", "kv4_cache", "kv4_store", "kv4_load",
    "verify_attn_kv4", "verify_attn_kv4_workspace_size",
    "block_rows_hint_for_kv4", "compact_kv4",
    "tree_pack", "verify_attn_tree", "verify_attn_tree_workspace_size", "sample", "accept_tree",
    "TreeStep",
]

COMPACT, STATIC, CAP_ACCEPT = 0, 1, 2
F32, BF16 = 0, 1
DEVERR = {
    0x1: "rows_overflow", 0x2: "no_free_page", 0x4: "page_row_full", 0x8: "wait_timeout",
    0x10: "bad_input", 0x20: "work_overflow",
}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdspark.so")

KV4_BLOCK_BYTES = 2176   # 16 tokens of one KV head in the 4-bit cache

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t
_L = ctypes.c_longlong

_SIGNATURES = {
    "dspark_status_string": (ctypes.c_char_p, [_I]),
    "dspark_read_device_error": (_I, [_P]),
    "dspark_num_sms": (_I, []),
    "dspark_set_wait_limit_ns": (_I, [ctypes.c_ulonglong]),
    "dspark_set_wait_probe": (_I, [_I]),
    "dspark_schedule": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "dspark_calib_collect": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _I, _P]),
    "dspark_calib_ece": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "dspark_sts_fit_workspace_size": (_Z, [_I, _I]),
    "dspark_sts_fit": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _Z, _P]),
    "dspark_block_accept_estimate": (_I, [_P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                          _P, _P, _P]),
    "dspark_markov_draft_workspace_size": (_Z, [_I]),
    "dspark_markov_draft": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _Z, _P]),
    "dspark_pack": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "dspark_verify_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "dspark_verify_attn": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                _F, _I, _I, _P, _P, _P, _Z, _P]),
    "dspark_verify_attn_planned": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                        _I, _I, _F, _I, _I, _P, _P, _P, _Z, _P]),
    "dspark_pack_plan": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                              _I, _I, _I, _I, _I, _I, _I, _P, _Z, _P]),
    "dspark_accept_workspace_size": (_Z, [_I, _I, _I, _I]),
    "dspark_accept": (_I, [_P, _P, _I, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                           _P, _Z, _P]),
    "dspark_accept_noalloc": (_I, [_P, _P, _I, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P,
                                   _P, _P, _P]),
    "dspark_compact_workspace_size": (_Z, [_I]),
    "dspark_step_graph_create": (_I, [_P, _P]),
    "dspark_step_graph_launch": (_I, [_P, _P]),
    "dspark_step_graph_destroy": (_I, [_P]),
    "dspark_step_graph_flags": (_I, [_P]),
    "dspark_compact": (_I, [_P, _P, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                            _P, _P, _P, _P, _Z, _P]),
    "dspark_compact_path": (_I, [_P, _P, _I, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P,
                                 _P, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "dspark_tree_pack": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "dspark_accept_tree": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "dspark_verify_attn_tree_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "dspark_verify_attn_tree": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I,
                                     _I, _F, _I, _I, _P, _P, _P, _Z, _P]),
    "dspark_sample": (_I, [_P, _L, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _P]),
    "dspark_sample_every_row": (_I, [_P, _L, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I,
                                     _P]),
    "dspark_qk_norm_rope": (_I, [_P, _L, _P, _L, _P, _L, _I, _P, _P, _F, _P, _I, _I, _F, _P, _P, _I,
                                 _I, _I, _P, _P, _P, _P]),
    "dspark_kv4_store": (_I, [_P, _L, _P, _L, _I, _P, _P, _I, _I, _I, _I, _P, _I, _I, _F, _F, _P,
                              _P]),
    "dspark_kv4_load": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _I, _I, _F, _F, _I, _P, _P, _P]),
    "dspark_verify_attn_kv4_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "dspark_verify_attn_kv4": (_I, [_P, _P, _P, _P, _F, _F, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                    _F, _I, _I, _P, _P, _P, _Z, _P]),
    "dspark_compact_kv4": (_I, [_P, _P, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                _P, _P, _F, _F, _P, _P, _P, _Z, _P]),
}

_lib = None


class DSparkError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().dspark_status_string(status).decode()
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the in-tree library; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with __graft_entry__.build() "
                              "(speculative_decoding_verification_dspark_gb300/build.py)")
        l = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


lib = load


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


# The current stream's handle without a Stream object in between, 1 us less; private to torch,
# so not counted on.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev=None):
    if stream is None:
        if dev is not None and _raw_stream is not None:
            return _raw_stream(dev)
        stream = torch.cuda.current_stream(dev)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise DSparkError(fn, rc)


def read_device_error(stream=None) -> int:
    rc = lib().dspark_read_device_error(_stream(stream))
    if rc < 0:
        raise DSparkError("dspark_read_device_error", rc)
    return rc


def num_sms() -> int:
    return lib().dspark_num_sms()


def set_wait_limit_ns(ns: int) -> None:
    """Limit of the acceptance pass's bounded waits on the current device (0: 2 s)."""
    _check("dspark_set_wait_limit_ns", lib().dspark_set_wait_limit_ns(int(ns)))


def set_wait_probe(on: bool) -> None:
    """Test hook: the acceptance pass first waits on a barrier nothing arrives at."""
    _check("dspark_set_wait_probe", lib().dspark_set_wait_probe(1 if on else 0))


def schedule(conf, conf_is_logit, sts_temp, cost_table, max_tokens, mode, windows, a_hat, M_out,
             E_out, stream=None, survival=None):
    """``survival``: optional fp32 [B, gamma] output of the uncalibrated prefix survival."""
    B, gamma = conf.shape
    _check("dspark_schedule", lib().dspark_schedule(
        _ptr(conf), int(conf_is_logit), _ptr(sts_temp), _ptr(cost_table), cost_table.numel(), B,
        gamma, int(max_tokens), int(mode), _ptr(windows), _ptr(a_hat), _ptr(survival),
        _ptr(M_out), _ptr(E_out), _stream(stream)))


class CalibStore:
    """Device store of labelled accept outcomes per draft position (dspark_calib_*):
    ``collect`` after a step, ``ece`` and ``sts_fit`` on demand."""

    def __init__(self, gamma, capacity, device="cuda"):
        dev = torch.device(device)
        self.gamma, self.capacity = gamma, capacity
        self.s_a = torch.zeros(gamma, capacity, dtype=torch.float32, device=dev)
        self.s_ahat = torch.zeros(gamma, capacity, dtype=torch.float32, device=dev)
        self.s_y = torch.zeros(gamma, capacity, dtype=torch.int8, device=dev)
        self.count = torch.zeros(gamma, dtype=torch.int32, device=dev)
        self.ws = torch.empty(lib().dspark_sts_fit_workspace_size(gamma, capacity),
                              dtype=torch.uint8, device=dev)

    def collect(self, survival, a_hat, windows, cap_len, mode, stream=None):
        B = windows.numel()
        _check("dspark_calib_collect", lib().dspark_calib_collect(
            _ptr(survival), _ptr(a_hat), _ptr(windows), _ptr(cap_len), int(mode), B, self.gamma,
            _ptr(self.s_a), _ptr(self.s_ahat), _ptr(self.s_y), _ptr(self.count), self.capacity,
            _stream(stream)))

    def ece(self, n_bins, stream=None):
        """(ece fp64 [1], bin counts, bin sums of a_hat, bin sums of y) on the device."""
        dev = self.count.device
        bn = torch.zeros(n_bins, dtype=torch.int32, device=dev)
        bp = torch.zeros(n_bins, dtype=torch.float64, device=dev)
        by = torch.zeros(n_bins, dtype=torch.float64, device=dev)
        e = torch.zeros(1, dtype=torch.float64, device=dev)
        _check("dspark_calib_ece", lib().dspark_calib_ece(
            _ptr(self.s_ahat), _ptr(self.s_y), _ptr(self.count), self.capacity, self.gamma,
            int(n_bins), _ptr(bn), _ptr(bp), _ptr(by), _ptr(e), _stream(stream)))
        return e, bn, bp, by

    def sts_fit(self, iters, temps=None, stream=None):
        """Refitted STS temperatures fp32 [gamma] (device)."""
        if temps is None:
            temps = torch.empty(self.gamma, dtype=torch.float32, device=self.count.device)
        _check("dspark_sts_fit", lib().dspark_sts_fit(
            _ptr(self.s_a), _ptr(self.s_y), _ptr(self.count), self.capacity, self.gamma,
            int(iters), _ptr(temps), _ptr(self.ws), self.ws.numel(), _stream(stream)))
        return temps


class MarkovDraft:
    """Draft-side sampling of one block with a Markov head (dspark_markov_draft).
    Holds the call's workspace, zeroed once at construction; calls on one stream
    share it."""

    def __init__(self, V, device="cuda"):
        n = lib().dspark_markov_draft_workspace_size(int(V))
        if n == 0:
            raise ValueError(f"vocabulary size {V} is not supported (a multiple of 128 is needed)")
        self.V = int(V)
        self.ws = torch.zeros(n, dtype=torch.uint8, device=torch.device(device))

    def __call__(self, U, W1, W2, anchor, exp_noise, draft_tok=None, p_draft=None, stream=None):
        """U, exp_noise fp32 [B, gamma, V]; W1 bf16 [V, 256]; W2 bf16 [256, V]; anchor
        int32 [B].  Returns (draft_tok int32 [B, gamma], p_draft fp32 [B, gamma, V])."""
        B, gamma, V = U.shape
        if draft_tok is None:
            draft_tok = torch.empty(B, gamma, dtype=torch.int32, device=U.device)
        if p_draft is None:
            p_draft = torch.empty(B, gamma, V, dtype=torch.float32, device=U.device)
        _check("dspark_markov_draft", lib().dspark_markov_draft(
            _ptr(U), _ptr(W1), _ptr(W2), int(W2.shape[0]), _ptr(anchor), _ptr(exp_noise), B, gamma,
            V, _ptr(draft_tok), _ptr(p_draft), _ptr(self.ws), self.ws.numel(), _stream(stream)))
        return draft_tok, p_draft


def _host_ptr(t):
    """A pinned host tensor's address (for the mapped tier word), or None."""
    if t is None:
        return None
    if t.is_cuda or not t.is_pinned():
        raise ValueError("expected a pinned host tensor")
    return t.data_ptr()


def pack(windows, ctx_len, anchor, draft_tok, tiers, mode, cu_seqlens, M_out, tier_out, row_req,
         row_pos, row_tok, stream=None, tier_host=None):
    """``tier_host``: optional pinned host int32 tensor that also receives the tier."""
    B, gamma = draft_tok.shape
    _check("dspark_pack", lib().dspark_pack(
        _ptr(windows), _ptr(ctx_len), _ptr(anchor), _ptr(draft_tok), _ptr(tiers), tiers.numel(), B,
        gamma, int(mode), row_req.numel(), _ptr(cu_seqlens), _ptr(M_out), _ptr(tier_out),
        _host_ptr(tier_host), _ptr(row_req), _ptr(row_pos), _ptr(row_tok), _stream(stream)))


def pack_plan(windows, ctx_len, anchor, draft_tok, tiers, mode, cu_seqlens, M_out, tier_out,
              row_req, row_pos, row_tok, Hq, Hkv, d_qk, d_v, attn_max_rows, max_splits,
              attn_workspace, stream=None, max_block_rows=0, tier_host=None):
    """pack, plus the work list of the verify_attn_planned call that follows (same shape
    and workspace)."""
    B, gamma = draft_tok.shape
    _check("dspark_pack_plan", lib().dspark_pack_plan(
        _ptr(windows), _ptr(ctx_len), _ptr(anchor), _ptr(draft_tok), _ptr(tiers), tiers.numel(), B,
        gamma, int(mode), row_req.numel(), _ptr(cu_seqlens), _ptr(M_out), _ptr(tier_out),
        _host_ptr(tier_host), _ptr(row_req), _ptr(row_pos), _ptr(row_tok), int(Hq), int(Hkv),
        int(d_qk), int(d_v),
        int(attn_max_rows), int(max_splits), int(max_block_rows), _ptr(attn_workspace),
        attn_workspace.numel() * attn_workspace.element_size(), _stream(stream)))


def verify_attn_workspace_size(B, max_rows, Hq, Hkv, d_qk, d_v, max_splits,
                               max_block_rows=0) -> int:
    return lib().dspark_verify_attn_workspace_size(B, max_rows, Hq, Hkv, d_qk, d_v, max_splits,
                                                   max_block_rows)


def verify_attn(q, k_new, v_new, k_cache, v_cache, page_table, ctx_len, cu_seqlens, scale,
                max_splits, out, lse, workspace, stream=None, max_block_rows=0):
    """GQA: q [rows, Hq, 128], k/v_new [rows, Hkv, 128], caches [pages, P, Hkv, 128].
    MLA: q [rows, 128, 576], k_new [rows, 576], k_cache [pages, P, 576], v_* None."""
    _verify_attn("dspark_verify_attn", q, k_new, v_new, k_cache, v_cache, page_table, ctx_len,
                 cu_seqlens, scale, max_splits, out, lse, workspace, stream, max_block_rows)


def verify_attn_planned(q, k_new, v_new, k_cache, v_cache, page_table, ctx_len, cu_seqlens,
                        scale, max_splits, out, lse, workspace, stream=None, max_block_rows=0):
    """verify_attn over the work list that pack_plan wrote into ``workspace``."""
    _verify_attn("dspark_verify_attn_planned", q, k_new, v_new, k_cache, v_cache, page_table,
                 ctx_len, cu_seqlens, scale, max_splits, out, lse, workspace, stream,
                 max_block_rows)


def _verify_attn(name, q, k_new, v_new, k_cache, v_cache, page_table, ctx_len, cu_seqlens, scale,
                 max_splits, out, lse, workspace, stream, max_block_rows):
    max_rows, Hq, d_qk = q.shape
    mla = v_cache is None
    Hkv = 1 if mla else k_cache.shape[2]
    d_v = out.shape[2]
    B = ctx_len.numel()
    _check(name, getattr(lib(), name)(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
        _ptr(page_table), page_table.shape[1], _ptr(ctx_len), _ptr(cu_seqlens), B, max_rows, Hq,
        Hkv, d_qk, d_v, k_cache.shape[1], float(scale), int(max_splits), int(max_block_rows),
        _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def accept_workspace_size(B, gamma, max_rows, V) -> int:
    return lib().dspark_accept_workspace_size(B, gamma, max_rows, V)


def accept(p_target, p_draft, draft_tok, uniforms, exp_noise, windows, cu_seqlens, mode,
           accept_len, cap_len, out_tok, cstar, fallback, workspace, stream=None):
    B, gamma, V = p_draft.shape
    pdt = BF16 if p_target.dtype == torch.bfloat16 else F32
    _check("dspark_accept", lib().dspark_accept(
        _ptr(p_target), _ptr(p_draft), pdt, V, _ptr(draft_tok), _ptr(uniforms), _ptr(exp_noise),
        _ptr(windows), _ptr(cu_seqlens), int(mode), B, gamma, p_target.shape[0], _ptr(accept_len),
        _ptr(cap_len), _ptr(out_tok), _ptr(cstar), _ptr(fallback), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def accept_noalloc(p_target, p_draft, draft_tok, uniforms, exp_noise, windows, cu_seqlens, mode,
                   accept_len, cap_len, out_tok, cstar, fallback, stream=None):
    """``accept`` with the library's fixed scratch instead of a workspace argument."""
    B, gamma, V = p_draft.shape
    pdt = BF16 if p_target.dtype == torch.bfloat16 else F32
    _check("dspark_accept_noalloc", lib().dspark_accept_noalloc(
        _ptr(p_target), _ptr(p_draft), pdt, V, _ptr(draft_tok), _ptr(uniforms), _ptr(exp_noise),
        _ptr(windows), _ptr(cu_seqlens), int(mode), B, gamma, p_target.shape[0], _ptr(accept_len),
        _ptr(cap_len), _ptr(out_tok), _ptr(cstar), _ptr(fallback), _stream(stream)))


def block_accept_estimate(p_target, p_draft, draft_tok, uniforms, windows, cu_seqlens, mode,
                          accept_len, cap_len, cap_lo=None, cap_hi=None, stream=None):
    """The uncut cap's interval (cap_lo, cap_hi) int32 [B] from a step's acceptance
    outputs (dspark_block_accept_estimate)."""
    B, gamma, V = p_draft.shape
    pdt = BF16 if p_target.dtype == torch.bfloat16 else F32
    if cap_lo is None:
        cap_lo = torch.empty(B, dtype=torch.int32, device=p_draft.device)
    if cap_hi is None:
        cap_hi = torch.empty(B, dtype=torch.int32, device=p_draft.device)
    _check("dspark_block_accept_estimate", lib().dspark_block_accept_estimate(
        _ptr(p_target), _ptr(p_draft), pdt, V, _ptr(draft_tok), _ptr(uniforms), _ptr(windows),
        _ptr(cu_seqlens), _ptr(accept_len), _ptr(cap_len), int(mode), B, gamma,
        p_target.shape[0], _ptr(cap_lo), _ptr(cap_hi), _stream(stream)))
    return cap_lo, cap_hi


def compact_workspace_size(B) -> int:
    return lib().dspark_compact_workspace_size(B)


def compact(k_new, v_new, cu_seqlens, accept_len, out_tok, draft_tok, page_table, ctx_len, anchor,
            free_pages, free_top, k_cache, v_cache, committed, n_committed, workspace, stream=None,
            path=None):
    """``path`` (int32 [B, gamma + 1], accept_tree's): the rows of a tree that are kept, with
    accept_tree's path_tok as draft_tok (dspark_compact_path)."""
    B, gamma = draft_tok.shape
    row_bytes = k_new.numel() // max(k_new.shape[0], 1) * k_new.element_size()
    name, more = "dspark_compact", ()
    if path is not None:
        name = "dspark_compact_path"
        more = (_arg(path, _current(path), "path", torch.int32, (B, gamma + 1)),)
    _check(name, getattr(lib(), name)(
        _ptr(k_new), _ptr(v_new), row_bytes, k_new.shape[0], _ptr(cu_seqlens), _ptr(accept_len), _ptr(out_tok),
        _ptr(draft_tok), *more, B, gamma, k_cache.shape[1], page_table.shape[1], k_cache.shape[0],
        _ptr(page_table), _ptr(ctx_len), _ptr(anchor), _ptr(free_pages), _ptr(free_top),
        _ptr(k_cache), _ptr(v_cache), _ptr(committed), _ptr(n_committed), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream, _current(k_new))))


# ---- query/key norm with rotation, and the 4-bit cache.  These bindings also check types,
# shapes and that every tensor is on the current device (whose stream the call goes to).

def _current(t):
    """Index of the current CUDA device, asked for once per call; -2, which no tensor has, where
    t is on the host."""
    return torch.cuda.current_device() if t.is_cuda else -2


def _arg(t, dev, name, dtype, shape=None):
    """Address of a dense tensor of this type on the current device `dev`."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.is_contiguous() and (shape is None or t.shape == shape)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise ValueError(f"{name}: expected a {dtype} tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: expected a tensor on the current CUDA device")


def _rows(t, dev, name, rows, heads, dtype):
    """(address, row stride in elements) of [rows, heads, 128] with dense heads."""
    if t.dtype is not dtype or t.shape != (rows, heads, 128):
        raise ValueError(f"{name}: expected {dtype} [{rows}, {heads}, 128], got {t.dtype} "
                         f"{tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if rows == 1:
        s0 = max(s0, heads * 128)   # the stride of one row is never used
        s0 -= s0 % 8
    if s2 != 1 or (heads > 1 and s1 != 128):
        raise ValueError(f"{name}: the heads of a row must be dense")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current CUDA device")
    return t.data_ptr(), s0


def _float_dtype(t, name):
    if t.dtype is torch.bfloat16:
        return BF16
    if t.dtype is torch.float32:
        return F32
    raise ValueError(f"{name}: expected a float32 or bfloat16 tensor")


def qk_norm_rope(q_in, k_in, v_in, q_weight, k_weight, inv_freq, row_pos, q, k_new, v_new,
                 eps=1e-6, interleaved=False, attn_factor=1.0, stream=None, n_rows=None):
    """Projections of packed rows -> q, k_new, v_new of the verify attention
    (dspark_qk_norm_rope): RMS norm per query / key head (weights fp32 [128], None: no
    norm), rotation of the first 2 * len(inv_freq) dims by the row's position, values
    copied.

    q_in [rows, Hq, 128], k_in, v_in [rows, Hkv, 128] fp32 or bf16, possibly views of one
    fused projection; inv_freq fp32 [R / 2] or None; row_pos int32 [rows] (< 0: padding,
    left as it is); n_rows int32 [1] or None: rows from there on are left as they are;
    outputs bf16, dense.  v_in and v_new may be None."""
    rows, Hq, _ = q.shape
    Hkv = k_new.shape[1]
    dev = _current(q)
    dt = _float_dtype(q_in, "q_in")
    qp, qs = _rows(q_in, dev, "q_in", rows, Hq, q_in.dtype)
    kp, ks = _rows(k_in, dev, "k_in", rows, Hkv, q_in.dtype)
    if (v_in is None) != (v_new is None):
        raise ValueError("v_in and v_new go together")
    vp, vs = (None, 0) if v_in is None else _rows(v_in, dev, "v_in", rows, Hkv, q_in.dtype)
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32
    _check("dspark_qk_norm_rope", lib().dspark_qk_norm_rope(
        qp, qs, kp, ks, vp, vs, dt,
        None if q_weight is None else _arg(q_weight, dev, "q_weight", f32, (128,)),
        None if k_weight is None else _arg(k_weight, dev, "k_weight", f32, (128,)), float(eps),
        None if inv_freq is None else _arg(inv_freq, dev, "inv_freq", f32),
        0 if inv_freq is None else 2 * inv_freq.numel(), 1 if interleaved else 0,
        float(attn_factor), _arg(row_pos, dev, "row_pos", i32, (rows,)),
        None if n_rows is None else _arg(n_rows, dev, "n_rows", i32, (1,)), rows, Hq, Hkv,
        _arg(q, dev, "q", bf16, (rows, Hq, 128)), _arg(k_new, dev, "k_new", bf16, (rows, Hkv, 128)),
        None if v_new is None else _arg(v_new, dev, "v_new", bf16, (rows, Hkv, 128)),
        _stream(stream, dev)))


def kv4_cache(n_pages, Hkv, page_size, device="cuda"):
    """A zeroed 4-bit cache: uint8 [n_pages, Hkv, page_size / 16, 2176] (layout: dspark.h)."""
    page_size = int(page_size)
    if page_size < 16 or page_size & (page_size - 1):
        raise ValueError("page_size must be a power of two >= 16")
    return torch.zeros(n_pages, Hkv, page_size // 16, KV4_BLOCK_BYTES, dtype=torch.uint8,
                       device=torch.device(device))


def _kv4(kv_cache, page_table, cu_seqlens):
    """(current device, cache address, n_pages, Hkv, page_size, table address, max_pages, B,
    cu address)."""
    if kv_cache.dim() != 4 or kv_cache.shape[3] != KV4_BLOCK_BYTES:
        raise ValueError("kv_cache: expected uint8 [n_pages, Hkv, page_size / 16, "
                         f"{KV4_BLOCK_BYTES}]")
    n_pages, Hkv, per, _ = kv_cache.shape
    B = cu_seqlens.numel() - 1
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table: expected [{B}, max_pages]")
    i32, dev = torch.int32, _current(kv_cache)
    return (dev, _arg(kv_cache, dev, "kv_cache", torch.uint8), n_pages, Hkv, per * 16,
            _arg(page_table, dev, "page_table", i32), page_table.shape[1], B,
            _arg(cu_seqlens, dev, "cu_seqlens", i32))


def kv4_store(k, v, cu_seqlens, pos0, page_table, kv_cache, k_scale=1.0, v_scale=1.0, stream=None):
    """Quantise packed rows into the 4-bit cache (dspark_kv4_store): row cu_seqlens[r] + i
    of k, v [rows, Hkv, 128] (fp32 or bf16, possibly views of a fused projection) becomes
    position pos0[r] + i of request r."""
    dev, c, n_pages, Hkv, page, tab, max_pages, B, cu = _kv4(kv_cache, page_table, cu_seqlens)
    rows = k.shape[0]
    dt = _float_dtype(k, "k")
    kp, ks = _rows(k, dev, "k", rows, Hkv, k.dtype)
    vp, vs = _rows(v, dev, "v", rows, Hkv, k.dtype)
    _check("dspark_kv4_store", lib().dspark_kv4_store(
        kp, ks, vp, vs, dt, cu, _arg(pos0, dev, "pos0", torch.int32, (B,)), B, rows, Hkv, page, tab,
        max_pages, n_pages, float(k_scale), float(v_scale), c, _stream(stream, dev)))


def kv4_load(kv_cache, cu_seqlens, pos0, page_table, k, v, k_scale=1.0, v_scale=1.0, stream=None):
    """Positions pos0[r] .. of every request back into packed rows k, v [rows, Hkv, 128]
    (fp32 or bf16; dspark_kv4_load)."""
    dev, c, n_pages, Hkv, page, tab, max_pages, B, cu = _kv4(kv_cache, page_table, cu_seqlens)
    rows = k.shape[0]
    dt = _float_dtype(k, "k")
    _check("dspark_kv4_load", lib().dspark_kv4_load(
        c, cu, _arg(pos0, dev, "pos0", torch.int32, (B,)), B, rows, Hkv, page, tab, max_pages,
        n_pages, float(k_scale), float(v_scale), dt, _arg(k, dev, "k", k.dtype, (rows, Hkv, 128)),
        _arg(v, dev, "v", k.dtype, (rows, Hkv, 128)), _stream(stream, dev)))


def verify_attn_kv4_workspace_size(B, max_rows, Hq, Hkv, max_splits, max_block_rows=0) -> int:
    return lib().dspark_verify_attn_kv4_workspace_size(B, max_rows, Hq, Hkv, max_splits,
                                                       max_block_rows)


def verify_attn_kv4(q, k_new, v_new, kv_cache, page_table, ctx_len, cu_seqlens, scale, max_splits,
                    out, lse, workspace, k_scale=1.0, v_scale=1.0, stream=None, max_block_rows=0):
    """verify_attn over the 4-bit cache: q [rows, Hq, 128], k_new / v_new [rows, Hkv, 128]
    bf16, kv_cache as kv4_cache gives it, out bf16 [rows, Hq, 128], lse fp32 [rows, Hq]."""
    dev, c, n_pages, Hkv, page, tab, max_pages, B, cu = _kv4(kv_cache, page_table, cu_seqlens)
    rows, Hq, _ = q.shape
    bf16 = torch.bfloat16
    _check("dspark_verify_attn_kv4", lib().dspark_verify_attn_kv4(
        _arg(q, dev, "q", bf16, (rows, Hq, 128)), _arg(k_new, dev, "k_new", bf16, (rows, Hkv, 128)),
        _arg(v_new, dev, "v_new", bf16, (rows, Hkv, 128)), c, float(k_scale), float(v_scale),
        n_pages, tab, max_pages, _arg(ctx_len, dev, "ctx_len", torch.int32, (B,)), cu, B, rows, Hq,
        Hkv, page, float(scale), int(max_splits), int(max_block_rows),
        _arg(out, dev, "out", bf16, (rows, Hq, 128)), _arg(lse, dev, "lse", torch.float32, (rows, Hq)),
        _arg(workspace, dev, "workspace", torch.uint8), workspace.numel(), _stream(stream, dev)))


def compact_kv4(k_new, v_new, cu_seqlens, accept_len, out_tok, draft_tok, page_table, ctx_len,
                anchor, free_pages, free_top, kv_cache, committed, n_committed, workspace,
                k_scale=1.0, v_scale=1.0, stream=None):
    """compact into the 4-bit cache (dspark_compact_kv4)."""
    dev, c, n_pages, Hkv, page, tab, max_pages, B, cu = _kv4(kv_cache, page_table, cu_seqlens)
    gamma, rows = draft_tok.shape[1], k_new.shape[0]
    bf16, i32 = torch.bfloat16, torch.int32
    _check("dspark_compact_kv4", lib().dspark_compact_kv4(
        _arg(k_new, dev, "k_new", bf16, (rows, Hkv, 128)),
        _arg(v_new, dev, "v_new", bf16, (rows, Hkv, 128)), Hkv, rows, cu,
        _arg(accept_len, dev, "accept_len", i32, (B,)), _arg(out_tok, dev, "out_tok", i32, (B,)),
        _arg(draft_tok, dev, "draft_tok", i32, (B, gamma)), B, gamma, page, max_pages, n_pages, tab,
        _arg(ctx_len, dev, "ctx_len", i32, (B,)), _arg(anchor, dev, "anchor", i32, (B,)),
        _arg(free_pages, dev, "free_pages", i32), _arg(free_top, dev, "free_top", i32), c,
        float(k_scale), float(v_scale), _arg(committed, dev, "committed", i32, (B, gamma + 1)),
        _arg(n_committed, dev, "n_committed", i32, (B,)),
        _arg(workspace, dev, "workspace", torch.uint8), workspace.numel(), _stream(stream, dev)))


# ---- trees of drafted tokens, and sampling from logits

def tree_pack(row_parent, cu_seqlens, ctx_len, row_mask, row_pos, stream=None):
    """Visibility masks and positions of packed trees (dspark_tree_pack): row_parent int32
    [rows] (index in the segment, -1: none), row_mask int64 [rows, words] out, row_pos int32
    [rows] out."""
    i32, dev = torch.int32, _current(row_parent)
    rows, B = row_parent.numel(), ctx_len.numel()
    if row_mask.dim() != 2:
        raise ValueError(f"row_mask: expected int64 [{rows}, words]")
    words = row_mask.shape[1]
    _check("dspark_tree_pack", lib().dspark_tree_pack(
        _arg(row_parent, dev, "row_parent", i32, (rows,)),
        _arg(cu_seqlens, dev, "cu_seqlens", i32, (B + 1,)), _arg(ctx_len, dev, "ctx_len", i32, (B,)),
        B, rows, words, _arg(row_mask, dev, "row_mask", torch.int64, (rows, words)),
        _arg(row_pos, dev, "row_pos", i32, (rows,)), _stream(stream, dev)))


def verify_attn_tree_workspace_size(B, max_rows, Hq, Hkv, max_splits, max_block_rows=0) -> int:
    return lib().dspark_verify_attn_tree_workspace_size(B, max_rows, Hq, Hkv, max_splits,
                                                        max_block_rows)


def verify_attn_tree(q, k_new, v_new, k_cache, v_cache, page_table, ctx_len, cu_seqlens, row_mask,
                     scale, max_splits, out, lse, workspace, stream=None, max_block_rows=0):
    """verify_attn (GQA) of trees: row_mask int64 [rows, words] says which block rows each row
    sees (tree_pack's); out bf16 [rows, Hq, 128], lse fp32 [rows, Hq]."""
    dev = _current(q)
    rows, Hq, _ = q.shape
    if k_cache.dim() != 4 or k_cache.shape[3] != 128:
        raise ValueError("k_cache: expected bf16 [n_pages, page_size, Hkv, 128]")
    n_pages, page, Hkv, _ = k_cache.shape
    B = ctx_len.numel()
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table: expected [{B}, max_pages]")
    if row_mask.dim() != 2:
        raise ValueError(f"row_mask: expected int64 [{rows}, words]")
    words = row_mask.shape[1]
    bf16, i32 = torch.bfloat16, torch.int32
    _check("dspark_verify_attn_tree", lib().dspark_verify_attn_tree(
        _arg(q, dev, "q", bf16, (rows, Hq, 128)), _arg(k_new, dev, "k_new", bf16, (rows, Hkv, 128)),
        _arg(v_new, dev, "v_new", bf16, (rows, Hkv, 128)), _arg(k_cache, dev, "k_cache", bf16),
        _arg(v_cache, dev, "v_cache", bf16, k_cache.shape), n_pages,
        _arg(page_table, dev, "page_table", i32), page_table.shape[1],
        _arg(ctx_len, dev, "ctx_len", i32, (B,)), _arg(cu_seqlens, dev, "cu_seqlens", i32, (B + 1,)),
        _arg(row_mask, dev, "row_mask", torch.int64, (rows, words)), words, B, rows, Hq, Hkv, page,
        float(scale), int(max_splits), int(max_block_rows),
        _arg(out, dev, "out", bf16, (rows, Hq, 128)),
        _arg(lse, dev, "lse", torch.float32, (rows, Hq)),
        _arg(workspace, dev, "workspace", torch.uint8), workspace.numel(), _stream(stream, dev)))


def sample(logits, temperature, top_k, top_p, min_p, exp_noise, tokens=None, probs=None,
           row_req=None, stream=None, n_rows=None, every_row=False):
    """Tokens and distributions from logits (dspark_sample): logits [rows, V] fp32 or bf16, rows
    possibly apart; temperature, top_p, min_p fp32 [B] and top_k int32 [B], each None where it is
    off; exp_noise fp32 [rows, V]; tokens int32 [rows] out or None; probs fp32 or bf16 [rows, V]
    out or None; row_req int32 [rows] (< 0: padding, left as it is) or None: row i has the
    parameters of index i; n_rows int32 [1] or None: rows from there on are left as they are.
    every_row: padding and refused rows before n_rows get token -1 and probs 0
    (dspark_sample_every_row)."""
    dev = _current(logits)
    dt = _float_dtype(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits: expected [rows, V]")
    rows, V = logits.shape
    stride = logits.stride(0) if rows > 1 else V   # the stride of one row is never used
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits: the values of a row must be dense")
    if logits.get_device() != dev:
        raise ValueError("logits: expected a tensor on the current CUDA device")
    f32, i32 = torch.float32, torch.int32
    given = [t for t in (temperature, top_k, top_p, min_p) if t is not None]
    # (without parameters row_req only says which rows are padding)
    B = given[0].numel() if given else rows if row_req is None else 0x7fffffff
    pdt = F32 if probs is None else _float_dtype(probs, "probs")

    def par(t, name, dtype):
        return None if t is None else _arg(t, dev, name, dtype, (B,))

    name = "dspark_sample_every_row" if every_row else "dspark_sample"
    _check(name, getattr(lib(), name)(
        logits.data_ptr(), stride, dt, rows, V,
        None if row_req is None else _arg(row_req, dev, "row_req", i32, (rows,)),
        None if n_rows is None else _arg(n_rows, dev, "n_rows", i32, (1,)), B,
        par(temperature, "temperature", f32), par(top_k, "top_k", i32), par(top_p, "top_p", f32),
        par(min_p, "min_p", f32),
        None if exp_noise is None else _arg(exp_noise, dev, "exp_noise", f32, (rows, V)),
        None if tokens is None else _arg(tokens, dev, "tokens", i32, (rows,)),
        None if probs is None else _arg(probs, dev, "probs", probs.dtype, (rows, V)), pdt,
        _stream(stream, dev)))


def accept_tree(row_tok, row_parent, cu_seqlens, row_sample, path, path_tok, accept_len, out_tok,
                stream=None):
    """The walk down each tree along the sampled tokens (dspark_accept_tree): row_tok,
    row_parent, row_sample int32 [rows]; path int32 [B, gamma + 1], path_tok int32 [B, gamma],
    accept_len, out_tok int32 [B] out."""
    i32, dev = torch.int32, _current(row_tok)
    rows, B = row_tok.numel(), accept_len.numel()
    if path_tok.dim() != 2:
        raise ValueError(f"path_tok: expected int32 [{B}, gamma]")
    gamma = path_tok.shape[1]
    _check("dspark_accept_tree", lib().dspark_accept_tree(
        _arg(row_tok, dev, "row_tok", i32, (rows,)), _arg(row_parent, dev, "row_parent", i32, (rows,)),
        _arg(row_sample, dev, "row_sample", i32, (rows,)),
        _arg(cu_seqlens, dev, "cu_seqlens", i32, (B + 1,)), B, gamma, rows,
        _arg(path, dev, "path", i32, (B, gamma + 1)),
        _arg(path_tok, dev, "path_tok", i32, (B, gamma)),
        _arg(accept_len, dev, "accept_len", i32, (B,)), _arg(out_tok, dev, "out_tok", i32, (B,)),
        _stream(stream, dev)))


class StepDesc(ctypes.Structure):
    """dspark_step_desc (field for field)."""
    _fields_ = (
        [(n, _I) for n in ("B", "gamma", "mode", "Hq", "Hkv", "d_qk", "d_v", "page_size",
                           "max_pages", "n_pages", "V", "pdt", "max_rows", "n_tiers")]
        + [("tiers_host", _P), ("tiers", _P)]
        + [(n, _I) for n in ("conf_is_logit", "cost_len", "max_tokens", "max_splits",
                             "max_block_rows")]
        + [("scale", _F)]
        + [(n, _P) for n in ("conf", "sts_temp", "cost_table", "draft_tok", "q", "k_new", "v_new",
                             "p_target", "p_draft", "uniforms", "exp_noise", "free_pages",
                             "page_table", "ctx_len", "anchor", "free_top", "k_cache", "v_cache",
                             "windows", "a_hat", "survival", "M", "E", "cu_seqlens", "M_pack",
                             "tier",
                             "row_req", "row_pos", "row_tok", "out", "lse", "accept_len",
                             "cap_len", "out_tok", "cstar", "fallback", "committed",
                             "n_committed", "tier_host", "body_log")]
        + [("log_len", _I), ("ws_attn", _P), ("ws_attn_bytes", _Z), ("ws_accept", _P),
           ("ws_accept_bytes", _Z), ("ws_compact", _P), ("ws_compact_bytes", _Z)]
    )


class StepGraph:
    """The whole verification step as one library-built CUDA graph whose captured tier
    is chosen on the device (dspark_step_graph_*): each ``launch`` runs one step from
    the current contents of the buffers it was built on."""

    def __init__(self, desc: StepDesc, keep):
        self._keep = keep            # tensors the descriptor points into
        self._desc = desc
        h = ctypes.c_void_p()
        _check("dspark_step_graph_create",
               lib().dspark_step_graph_create(ctypes.byref(desc), ctypes.byref(h)))
        self._h = h

    def launch(self, stream=None):
        _check("dspark_step_graph_launch", lib().dspark_step_graph_launch(self._h, _stream(stream)))

    @property
    def pdl(self) -> bool:
        """True if the graph's kernels keep their programmatic dependencies."""
        return bool(lib().dspark_step_graph_flags(self._h) & 1)

    def close(self):
        if self._h:
            lib().dspark_step_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def block_rows_hint_for(gamma, Hq, Hkv, mode) -> int:
    """Rows per request the attention's query tile is sized for in ``mode`` (the
    ``max_block_rows`` hint); a request with more rows is split into row tiles (exact;
    its keys are then read once per row tile, mostly from L2).

    Static and cap-accept verify the whole block: gamma + 1.  A compact window is short
    -- a few rows -- and the smallest tile holding four block rows of G = Hq / Hkv heads
    (32 query rows: floor(32 / G) block rows for G <= 8; 64 or 128 for larger groups)
    does far less softmax work per key tile than one sized for the whole block, while
    the rare longer window takes a second row tile.  (Measured with G = 4 and 5; the
    four-row floor keeps wide groups from splitting a typical window into many row
    tiles, each of which reads the request's keys again.)"""
    G = max(1, Hq // Hkv)
    if int(mode) == COMPACT:
        for cols in (32, 64, 128):
            if cols // G >= 4:
                return min(gamma + 1, cols // G)
        return gamma + 1
    return gamma + 1


def block_rows_hint_for_kv4(gamma, Hq, Hkv) -> int:
    """Rows per request the query tile of the 4-bit cache's attention is sized for: the
    block's gamma + 1 rows cut evenly into as few tiles of at most 64 query rows as hold
    them.  The tile is then the next of 8, 16, 32, 48 or 64 rows and takes as many block rows
    as fit: 17 rows of 4 heads give a hint of 9, a tile of 48 and pieces of 12 and 5 rows."""
    G = max(1, Hq // Hkv)
    tiles = -(-(gamma + 1) // max(1, 64 // G))
    return -(-(gamma + 1) // tiles)


class VerifyStep:
    """Device buffers and workspaces for repeated verification steps of one shape.

    ``run`` enqueues the five calls of one step on the current stream:
    schedule -> pack (with the attention work list: pack_plan) -> verify_attn (over that
    work list: verify_attn_planned) -> accept -> compact.  The per-row inputs
    (q, k_new, v_new, p_target) are read from the packed buffers the caller
    fills; state (caches, page table, ctx_len, anchor, free stack) is updated in
    place by compact.

    With ``kv4`` the cache is the 4-bit one: ``inp["kv_cache"]`` (see kv4_cache), with
    ``inp["k_scale"]`` and ``inp["v_scale"]`` (default 1), takes the place of k_cache and
    v_cache, ``out`` is bf16, and ``run`` calls pack and verify_attn_kv4, which builds its
    own work list.

    Where ``inp`` holds ``q_in``, ``k_in`` and ``v_in`` (the packed rows' projections), ``run``
    fills q, k_new and v_new from them after the pack (``norm_rope``).

    Where it holds ``logits`` (the packed rows' target logits, [max_rows, V]), ``run`` fills
    p_target from them before the acceptance (``distributions``).
    """

    def __init__(self, B, gamma, Hq, Hkv, d_qk, d_v, vocab, max_rows, p_dtype=torch.float32,
                 max_splits=8, device="cuda", block_rows_hint=None, kv4=False):
        self.kv4 = bool(kv4)
        if self.kv4 and (d_qk != 128 or d_v != 128):
            raise ValueError("the 4-bit cache holds heads of 128 dims")
        self.B, self.gamma, self.Hq, self.Hkv, self.d_qk, self.d_v = B, gamma, Hq, Hkv, d_qk, d_v
        self.vocab, self.max_rows, self.max_splits = vocab, max_rows, max_splits
        # the attention's query tile per mode (block_rows_hint); ``block_rows_hint``
        # fixes one hint for every mode
        if block_rows_hint is None and self.kv4:
            h = block_rows_hint_for_kv4(gamma, Hq, Hkv)
            self._hints = {COMPACT: h, STATIC: h, CAP_ACCEPT: h}
        elif block_rows_hint is None:
            self._hints = {m: block_rows_hint_for(gamma, Hq, Hkv, m)
                           for m in (COMPACT, STATIC, CAP_ACCEPT)}
        else:
            h = int(block_rows_hint)
            self._hints = {COMPACT: h, STATIC: h, CAP_ACCEPT: h}
        self.block_rows_hint = self._hints[COMPACT]  # of the last pack call
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.windows = torch.zeros(B, **i32)
        self.a_hat = torch.zeros(B, gamma, dtype=torch.float32, device=dev)
        self.survival = torch.zeros(B, gamma, dtype=torch.float32, device=dev)
        self.M = torch.zeros(1, **i32)
        self.E = torch.zeros(1, dtype=torch.float64, device=dev)
        self.cu_seqlens = torch.zeros(B + 1, **i32)
        self.M_pack = torch.zeros(1, **i32)
        self.tier = torch.zeros(1, **i32)
        self.row_req = torch.zeros(max_rows, **i32)
        self.row_pos = torch.zeros(max_rows, **i32)
        self.row_tok = torch.zeros(max_rows, **i32)
        self.out = torch.zeros(max_rows, Hq, d_v, device=dev,
                               dtype=torch.bfloat16 if self.kv4 else torch.float32)
        self.lse = torch.zeros(max_rows, Hq, dtype=torch.float32, device=dev)
        self.accept_len = torch.zeros(B, **i32)
        self.cap_len = torch.zeros(B, **i32)
        self.out_tok = torch.zeros(B, **i32)
        self.fallback = torch.zeros(B, **i32)
        self.cstar = torch.zeros(B, gamma, dtype=torch.float32, device=dev)
        self.committed = torch.zeros(B, gamma + 1, **i32)
        self.n_committed = torch.zeros(B, **i32)
        # sized for the smallest tile (the most work items)
        hint = min(self._hints.values())
        if self.kv4:
            sz = verify_attn_kv4_workspace_size(B, max_rows, Hq, Hkv, max_splits, hint)
        else:
            sz = verify_attn_workspace_size(B, max_rows, Hq, Hkv, d_qk, d_v, max_splits, hint)
        if sz == 0:
            raise ValueError("unsupported attention shape")
        self.ws_attn = torch.empty(sz, dtype=torch.uint8, device=dev)
        self.ws_accept = torch.empty(accept_workspace_size(B, gamma, max_rows, vocab),
                                     dtype=torch.uint8, device=dev)
        self.ws_compact = torch.empty(compact_workspace_size(B), dtype=torch.uint8, device=dev)

    def schedule(self, inp, mode, stream=None):
        schedule(inp["conf"], inp["conf_is_logit"], inp["sts_temp"], inp["cost_table"],
                 inp["max_tokens"], mode, self.windows, self.a_hat, self.M, self.E, stream,
                 survival=self.survival)

    def pack(self, inp, mode, stream=None):
        self.block_rows_hint = self.hint(mode)  # for a following attention()
        pack(self.windows, inp["ctx_len"], inp["anchor"], inp["draft_tok"], inp["tiers"], mode,
             self.cu_seqlens, self.M_pack, self.tier, self.row_req, self.row_pos, self.row_tok,
             stream)

    def norm_rope(self, inp, stream=None):
        """q, k_new, v_new of ``inp`` from q_in, k_in, v_in, at the positions of the last pack
        (q_weight, k_weight, inv_freq, eps, interleaved, attn_factor as in qk_norm_rope)."""
        qk_norm_rope(inp["q_in"], inp["k_in"], inp["v_in"], inp.get("q_weight"),
                     inp.get("k_weight"), inp["inv_freq"], self.row_pos, inp["q"], inp["k_new"],
                     inp["v_new"], inp.get("eps", 1e-6), inp.get("interleaved", False),
                     inp.get("attn_factor", 1.0), stream, n_rows=self.M_pack)

    def distributions(self, inp, stream=None):
        """p_target of ``inp`` from its logits, filtered by its requests' parameters (temperature,
        top_k, top_p, min_p [B], each optional), for the rows of the last pack."""
        sample(inp["logits"], inp.get("temperature"), inp.get("top_k"), inp.get("top_p"),
               inp.get("min_p"), None, None, inp["p_target"], self.row_req, stream, n_rows=self.M_pack,
               every_row=True)   # (none of an earlier step)

    def attention(self, inp, stream=None):
        if self.kv4:
            verify_attn_kv4(inp["q"], inp["k_new"], inp["v_new"], inp["kv_cache"],
                            inp["page_table"], inp["ctx_len"], self.cu_seqlens, inp["scale"],
                            self.max_splits, self.out, self.lse, self.ws_attn,
                            inp.get("k_scale", 1.0), inp.get("v_scale", 1.0), stream,
                            max_block_rows=self.block_rows_hint)
            return
        verify_attn(inp["q"], inp["k_new"], inp.get("v_new"), inp["k_cache"], inp.get("v_cache"),
                    inp["page_table"], inp["ctx_len"], self.cu_seqlens, inp["scale"],
                    self.max_splits, self.out, self.lse, self.ws_attn, stream,
                    max_block_rows=self.block_rows_hint)

    def hint(self, mode) -> int:
        """The block-rows hint (query tile) the step uses in ``mode``."""
        return self._hints[int(mode)]

    def pack_plan(self, inp, mode, stream=None):
        """pack, with the attention work list built in the same kernel (for attention_planned,
        which takes the query tile chosen here)."""
        if self.kv4:
            raise ValueError("the 4-bit cache's attention builds its own work list")
        self.block_rows_hint = self.hint(mode)
        pack_plan(self.windows, inp["ctx_len"], inp["anchor"], inp["draft_tok"], inp["tiers"], mode,
                  self.cu_seqlens, self.M_pack, self.tier, self.row_req, self.row_pos,
                  self.row_tok, self.Hq, self.Hkv, self.d_qk, self.d_v, self.max_rows,
                  self.max_splits, self.ws_attn, stream, max_block_rows=self.block_rows_hint)

    def attention_planned(self, inp, stream=None):
        if self.kv4:
            raise ValueError("the 4-bit cache's attention builds its own work list")
        verify_attn_planned(inp["q"], inp["k_new"], inp.get("v_new"), inp["k_cache"],
                            inp.get("v_cache"), inp["page_table"], inp["ctx_len"],
                            self.cu_seqlens, inp["scale"], self.max_splits, self.out, self.lse,
                            self.ws_attn, stream, max_block_rows=self.block_rows_hint)

    def accept(self, inp, mode, stream=None):
        accept(inp["p_target"], inp["p_draft"], inp["draft_tok"], inp["uniforms"],
               inp["exp_noise"], self.windows, self.cu_seqlens, mode, self.accept_len,
               self.cap_len, self.out_tok, self.cstar, self.fallback, self.ws_accept, stream)

    def compact(self, inp, stream=None):
        if self.kv4:
            compact_kv4(inp["k_new"], inp["v_new"], self.cu_seqlens, self.accept_len, self.out_tok,
                        inp["draft_tok"], inp["page_table"], inp["ctx_len"], inp["anchor"],
                        inp["free_pages"], inp["free_top"], inp["kv_cache"], self.committed,
                        self.n_committed, self.ws_compact, inp.get("k_scale", 1.0),
                        inp.get("v_scale", 1.0), stream)
            return
        compact(inp["k_new"], inp.get("v_new"), self.cu_seqlens, self.accept_len, self.out_tok,
                inp["draft_tok"], inp["page_table"], inp["ctx_len"], inp["anchor"],
                inp["free_pages"], inp["free_top"], inp["k_cache"], inp.get("v_cache"),
                self.committed, self.n_committed, self.ws_compact, stream)

    def graph(self, inp, mode, tier_host=None, body_log=None) -> StepGraph:
        """The step on these buffers and ``inp``'s tensors as a StepGraph (tier chosen
        on the device).  ``tier_host``: optional pinned host int32 word receiving each
        step's tier; ``body_log``: optional device int32 [1 + n] recording the body
        index each launch ran (element 0 counts launches; the caller zeroes it).
        The graph takes the bf16 cache only, and q, k_new and v_new as they are: it has
        no norm_rope, so an ``inp`` with projections (``q_in``) is refused."""
        if self.kv4:
            raise ValueError("the step graph does not take the 4-bit cache")
        if "q_in" in inp:
            raise ValueError("the step graph does not run norm_rope: pass inputs without q_in")
        if "logits" in inp:
            raise ValueError("the step graph does not sample: pass inputs without logits")
        pdt = inp["p_target"].dtype
        tiers = inp["tiers"]
        tiers_dev = tiers.to(self.windows.device, torch.int32)
        tiers_host = tiers.cpu().to(torch.int32).contiguous()
        d = StepDesc()
        d.B, d.gamma, d.mode = self.B, self.gamma, int(mode)
        d.Hq, d.Hkv, d.d_qk, d.d_v = self.Hq, self.Hkv, self.d_qk, self.d_v
        d.page_size, d.max_pages = inp["k_cache"].shape[1], inp["page_table"].shape[1]
        d.n_pages, d.V = inp["k_cache"].shape[0], self.vocab
        d.pdt = BF16 if pdt == torch.bfloat16 else F32
        d.max_rows, d.n_tiers = self.max_rows, tiers_host.numel()
        d.tiers_host, d.tiers = tiers_host.data_ptr(), _ptr(tiers_dev)
        d.conf_is_logit, d.cost_len = int(inp["conf_is_logit"]), inp["cost_table"].numel()
        d.max_tokens, d.max_splits, d.max_block_rows = (int(inp["max_tokens"]), self.max_splits,
                                                      self.hint(mode))
        d.scale = float(inp["scale"])
        for k in ("conf", "sts_temp", "cost_table", "draft_tok", "q", "k_new", "p_target", "p_draft",
                  "uniforms", "exp_noise", "free_pages", "page_table", "ctx_len", "anchor",
                  "free_top", "k_cache"):
            setattr(d, k, _ptr(inp[k]))
        d.v_new, d.v_cache = _ptr(inp.get("v_new")), _ptr(inp.get("v_cache"))
        for k in ("windows", "a_hat", "survival", "M", "E", "cu_seqlens", "M_pack", "tier",
                  "row_req",
                  "row_pos", "row_tok", "out", "lse", "accept_len", "cap_len", "out_tok", "cstar",
                  "fallback", "committed", "n_committed"):
            setattr(d, k, _ptr(getattr(self, k)))
        d.tier_host = _host_ptr(tier_host)
        d.body_log = _ptr(body_log)
        d.log_len = 0 if body_log is None else body_log.numel() - 1
        d.ws_attn, d.ws_attn_bytes = _ptr(self.ws_attn), self.ws_attn.numel()
        d.ws_accept, d.ws_accept_bytes = _ptr(self.ws_accept), self.ws_accept.numel()
        d.ws_compact, d.ws_compact_bytes = _ptr(self.ws_compact), self.ws_compact.numel()
        return StepGraph(d, (tiers_dev, tiers_host, inp, tier_host, body_log))

    def run(self, inp, mode, stream=None):
        self.schedule(inp, mode, stream)
        (self.pack if self.kv4 else self.pack_plan)(inp, mode, stream)
        if "q_in" in inp:
            self.norm_rope(inp, stream)
        (self.attention if self.kv4 else self.attention_planned)(inp, stream)
        if "logits" in inp:
            self.distributions(inp, stream)
        self.accept(inp, mode, stream)
        self.compact(inp, stream)


class TreeStep:
    """Device buffers and workspaces for repeated verification steps on trees of drafted tokens,
    of one shape.

    ``run`` enqueues one step on the current stream: tree_pack -> (qk_norm_rope, where ``inp``
    holds q_in, k_in and v_in) -> verify_attn_tree -> sample -> accept_tree -> compact along the
    path.  ``inp`` holds cu_seqlens, row_tok, row_parent (the packed trees, row 0 of a segment the
    anchor), row_req int32 [max_rows] (each row's request), q, k_new, v_new,
    logits, exp_noise [max_rows, V], scale, the caches, the state that VerifyStep has too, and
    optionally temperature, top_k, top_p, min_p [B].
    """

    def __init__(self, B, gamma, Hq, Hkv, max_rows, max_nodes, max_splits=32, device="cuda"):
        if not 1 <= max_nodes <= 512:
            raise ValueError("a tree has 1 to 512 rows")
        self.B, self.gamma, self.max_rows = B, gamma, max_rows
        self.max_nodes, self.max_splits = max_nodes, max_splits
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.row_mask = torch.zeros(max_rows, -(-max_nodes // 64), dtype=torch.int64, device=dev)
        self.row_pos = torch.zeros(max_rows, **i32)
        self.out = torch.zeros(max_rows, Hq, 128, dtype=torch.bfloat16, device=dev)
        self.lse = torch.zeros(max_rows, Hq, dtype=torch.float32, device=dev)
        self.row_sample = torch.zeros(max_rows, **i32)
        self.path = torch.zeros(B, gamma + 1, **i32)
        self.path_tok = torch.zeros(B, gamma, **i32)
        self.accept_len = torch.zeros(B, **i32)
        self.out_tok = torch.zeros(B, **i32)
        self.committed = torch.zeros(B, gamma + 1, **i32)
        self.n_committed = torch.zeros(B, **i32)
        sz = verify_attn_tree_workspace_size(B, max_rows, Hq, Hkv, max_splits, max_nodes)
        if sz == 0:
            raise ValueError("unsupported attention shape")
        self.ws_attn = torch.empty(sz, dtype=torch.uint8, device=dev)
        self.ws_compact = torch.empty(compact_workspace_size(B), dtype=torch.uint8, device=dev)

    def pack(self, inp, stream=None):
        tree_pack(inp["row_parent"], inp["cu_seqlens"], inp["ctx_len"], self.row_mask, self.row_pos,
                  stream)

    def norm_rope(self, inp, stream=None):
        """q, k_new, v_new of ``inp`` from q_in, k_in, v_in, at the positions of the last pack."""
        qk_norm_rope(inp["q_in"], inp["k_in"], inp["v_in"], inp.get("q_weight"),
                     inp.get("k_weight"), inp["inv_freq"], self.row_pos, inp["q"], inp["k_new"],
                     inp["v_new"], inp.get("eps", 1e-6), inp.get("interleaved", False),
                     inp.get("attn_factor", 1.0), stream, n_rows=inp["cu_seqlens"][-1:])

    def attention(self, inp, stream=None):
        verify_attn_tree(inp["q"], inp["k_new"], inp["v_new"], inp["k_cache"], inp["v_cache"],
                         inp["page_table"], inp["ctx_len"], inp["cu_seqlens"], self.row_mask,
                         inp["scale"], self.max_splits, self.out, self.lse, self.ws_attn, stream,
                         max_block_rows=self.max_nodes)

    def sample(self, inp, stream=None):
        sample(inp["logits"], inp.get("temperature"), inp.get("top_k"), inp.get("top_p"),
               inp.get("min_p"), inp["exp_noise"], self.row_sample, None, inp["row_req"], stream,
               n_rows=inp["cu_seqlens"][-1:], every_row=True)   # (none of an earlier step)

    def accept(self, inp, stream=None):
        accept_tree(inp["row_tok"], inp["row_parent"], inp["cu_seqlens"], self.row_sample, self.path,
                    self.path_tok, self.accept_len, self.out_tok, stream)

    def compact(self, inp, stream=None):
        compact(inp["k_new"], inp["v_new"], inp["cu_seqlens"], self.accept_len, self.out_tok,
                self.path_tok, inp["page_table"], inp["ctx_len"], inp["anchor"], inp["free_pages"],
                inp["free_top"], inp["k_cache"], inp["v_cache"], self.committed, self.n_committed,
                self.ws_compact, stream, path=self.path)

    def run(self, inp, stream=None):
        self.pack(inp, stream)
        if "q_in" in inp:
            self.norm_rope(inp, stream)
        self.attention(inp, stream)
        self.sample(inp, stream)
        self.accept(inp, stream)
        self.compact(inp, stream)
