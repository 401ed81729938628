"""Python binding of ``libsvd.so`` -- argument marshalling only.

Every entry point has the name of its C function in ``include/svd.h``, ``svd_vocab.h`` or
``svd_tree.h`` and calls it through
ctypes with device pointers taken from torch tensors and the current CUDA stream.  PyTorch is
used for device memory and streams only; all arithmetic runs in the CUDA kernels.  There is no
fallback: if the library is missing or no GPU is present the call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsvd.so")

SVD_OK = 0
STATUS_NAMES = {0: "SVD_OK", 1: "SVD_ERR_INVALID_ARG", 2: "SVD_ERR_ALIGNMENT",
                3: "SVD_ERR_WORKSPACE", 4: "SVD_ERR_CUDA", 5: "SVD_ERR_TIMEOUT",
                6: "SVD_ERR_UNSUPPORTED", 7: "SVD_ERR_TOKEN_RANGE", 8: "SVD_ERR_PAGE_RANGE",
                9: "SVD_ERR_TREE"}
GREEDY, STOCHASTIC = 0, 1
BK_CEIL, BK_FLOOR = 0, 1

# field order of svd_row_info (8 x 4 bytes)
ROW_INFO_FIELDS = ("draft_token", "target_argmax", "accepted", "sample_token", "ratio",
                   "lse_draft", "lse_target", "loss")

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_U64 = ctypes.c_uint64
_SZ = ctypes.c_size_t


class SvdError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__("%s: %s" % (where, STATUS_NAMES.get(code, "status %d" % code)))
        self.code = code


class VerifyDistillArgs(ctypes.Structure):
    """Mirror of ``svd_verify_distill_args``."""
    _fields_ = [
        ("h", _P), ("W1", _P), ("b1", _P), ("w2", _P), ("b2", _F), ("H", _I), ("M", _I),
        ("gamma", _F), ("rnd", _I), ("bk_in", _P),
        ("D", _P), ("T", _P), ("draft_tok", _P), ("B", _I), ("k", _I), ("kt", _I), ("V", _I),
        ("mode", _I), ("temperature", _F), ("seed", _U64), ("step", _U64),
        ("lambda_", _F), ("clip_c", _F), ("grad_scale", _F), ("dlogits_fp32", _I),
        ("bhat", _P), ("bk", _P), ("accept_len", _P), ("emitted", _P), ("n_emitted", _P),
        ("loss_rows", _P), ("loss_total", _P), ("dlogits", _P), ("row_info", _P),
        ("full_k", _I), ("label_proxy", _P), ("label_full", _P), ("head_preact", _P),
    ]


class HeadUpdateArgs(ctypes.Structure):
    """Mirror of ``svd_head_update_args``."""
    _fields_ = [
        ("h", _P), ("label", _P), ("B", _I), ("H", _I), ("M", _I),
        ("W1m", _P), ("b1", _P), ("w2m", _P), ("b2", _P), ("W1", _P), ("w2", _P),
        ("mW1", _P), ("vW1", _P), ("mb1", _P), ("vb1", _P), ("mw2", _P), ("vw2", _P),
        ("mb2", _P), ("vb2", _P), ("step", _I),
        ("lr", _F), ("beta1", _F), ("beta2", _F), ("eps", _F), ("weight_decay", _F),
        ("loss", _P), ("bhat", _P), ("preact", _P),
    ]


class VsArgs(ctypes.Structure):
    """Mirror of ``svd_vs_args`` (include/svd_vocab.h)."""
    _fields_ = [
        ("D", _P), ("T", _P), ("draft_tok", _P), ("bk", _P), ("B", _I), ("k", _I), ("kt", _I),
        ("V", _I), ("v0", _I), ("Vl", _I), ("P", _I), ("rank", _I), ("mode", _I),
        ("temperature", _F), ("seed", _U64), ("step", _U64), ("distill", _I),
        ("lambda_", _F), ("clip_c", _F), ("grad_scale", _F), ("dlogits", _P), ("dlogits_fp32", _I),
        ("loss_rows", _P), ("loss_total", _P), ("accept_len", _P), ("emitted", _P),
        ("n_emitted", _P), ("row_info", _P),
    ]


_I64 = ctypes.c_int64


class TreeAttentionArgs(ctypes.Structure):
    """Mirror of ``svd_tree_attention_args`` (include/svd_tree.h)."""
    _fields_ = [
        ("q", _P), ("k_new", _P), ("v_new", _P), ("cache_k", _P), ("cache_v", _P),
        ("page_stride_k", _I64), ("page_stride_v", _I64), ("page_table", _P), ("cache_len", _P),
        ("parent", _P), ("n_nodes", _P), ("B", _I), ("n", _I), ("Hq", _I), ("Hkv", _I), ("D", _I),
        ("n_pages", _I), ("page_size", _I), ("max_pages", _I), ("dtype", _I), ("scale", _F),
        ("out", _P), ("lse", _P),
    ]


class LogitsProcessArgs(ctypes.Structure):
    """Mirror of ``svd_logits_process_args``."""
    _fields_ = [
        ("logits", _P), ("B", _I), ("n", _I), ("V", _I), ("history", _P), ("hist_stride", _I),
        ("prompt_len", _P), ("hist_len", _P), ("node_tok", _P), ("parent", _P),
        ("repetition", _P), ("frequency", _P), ("presence", _P), ("bias_tok", _P), ("bias_val", _P),
        ("n_bias", _I), ("mask", _P), ("mask_rows", _I), ("mask_value", _F), ("out", _P),
        ("argmax", _P), ("dz", _P), ("dlogits", _P), ("grad_fp32", _I),
    ]


class TreeVerifyArgs(ctypes.Structure):
    """Mirror of ``svd_tree_verify_args``."""
    _fields_ = [
        ("T", _P), ("target_tok", _P), ("node_tok", _P), ("parent", _P), ("n_nodes", _P),
        ("B", _I), ("n", _I), ("V", _I), ("target_argmax", _P), ("path", _P), ("n_path", _P),
        ("accept_len", _P), ("emitted", _P), ("n_emitted", _P),
    ]


class CacheAppendArgs(ctypes.Structure):
    """Mirror of ``svd_cache_append_args``."""
    _fields_ = [
        ("k_new", _P), ("v_new", _P), ("cache_k", _P), ("cache_v", _P), ("page_stride_k", _I64),
        ("page_stride_v", _I64), ("page_table", _P), ("cache_len", _P), ("count", _P), ("path", _P),
        ("B", _I), ("n", _I), ("Hkv", _I), ("D", _I), ("n_pages", _I), ("page_size", _I),
        ("max_pages", _I), ("new_len", _P),
    ]


_lib = None


def lib():
    """The loaded ``libsvd.so`` with argument types declared (raises if absent)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libsvd.so is not built (%s); run "
                           "`python -m speculative_decoding_verify_distill_b200.build`" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    L.svd_workspace_bytes.argtypes = [_I, _I, _I, _I]
    L.svd_workspace_bytes.restype = _SZ
    L.svd_workspace_reset.argtypes = [_P, _SZ, _P]
    L.svd_length_head.argtypes = [_P, _P, _P, _P, _F, _I, _I, _I, _I, _F, _I, _P, _P, _P, _SZ, _P]
    L.svd_verify.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _U64, _U64, _P, _P, _P, _P,
                             _P, _SZ, _P]
    L.svd_distill_loss_grad.argtypes = [_P, _P, _P, _I, _I, _I, _I, _F, _F, _F, _F, _P, _P, _P, _I,
                                        _P, _SZ, _P]
    L.svd_verify_distill.argtypes = [ctypes.POINTER(VerifyDistillArgs), _P, _SZ, _P]
    L.svd_get_device_error.argtypes = [_P, _P]
    L.svd_status_string.argtypes = [_I]
    L.svd_status_string.restype = ctypes.c_char_p
    L.svd_selftest_wait_timeout.argtypes = [_P, _SZ, _U64, _P]
    L.svd_verify_distill_noalloc.argtypes = [ctypes.POINTER(VerifyDistillArgs), _P, _P]
    L.svd_speedup_report.argtypes = [_P, _P, _P, _I, _I, ctypes.c_double, _P, _P]
    L.svd_length_head_update.argtypes = [ctypes.POINTER(HeadUpdateArgs), _P, _SZ, _P]
    L.svd_vs_exchange_bytes.argtypes = [_I, _I, _I]
    L.svd_vs_exchange_bytes.restype = _SZ
    L.svd_vs_workspace_bytes.argtypes = [_I, _I, _I]
    L.svd_vs_workspace_bytes.restype = _SZ
    L.svd_vs_stats.argtypes = [ctypes.POINTER(VsArgs), _P, _P, _SZ, _P]
    L.svd_vs_resolve.argtypes = [ctypes.POINTER(VsArgs), _P, _P, _P, _SZ, _P]
    L.svd_vs_finish.argtypes = [ctypes.POINTER(VsArgs), _P, _P, _SZ, _P]
    L.svd_tree_attention_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
    L.svd_logits_process_workspace_bytes.argtypes = [_I, _I]
    L.svd_tree_verify_workspace_bytes.argtypes = [_I, _I]
    L.svd_cache_append_workspace_bytes.argtypes = [_I]
    for fn in ("svd_tree_attention", "svd_logits_process", "svd_tree_verify", "svd_cache_append"):
        getattr(L, fn + "_workspace_bytes").restype = _SZ
    for fn, args in (("svd_tree_attention", TreeAttentionArgs), ("svd_logits_process", LogitsProcessArgs),
                     ("svd_logits_process_grad", LogitsProcessArgs), ("svd_tree_verify", TreeVerifyArgs),
                     ("svd_cache_append", CacheAppendArgs)):
        getattr(L, fn).argtypes = [ctypes.POINTER(args), _P, _SZ, _P]
        getattr(L, fn).restype = _I
    for fn in ("svd_workspace_reset", "svd_length_head", "svd_verify", "svd_distill_loss_grad",
               "svd_verify_distill", "svd_get_device_error", "svd_selftest_wait_timeout",
               "svd_verify_distill_noalloc", "svd_speedup_report", "svd_length_head_update",
               "svd_vs_stats", "svd_vs_resolve", "svd_vs_finish"):
        getattr(L, fn).restype = _I
    _lib = L
    return L


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(code: int, where: str):
    if code != SVD_OK:
        raise SvdError(code, where)


def _bits(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.bfloat16:
        raise TypeError("expected bf16 logits / weights, got %s" % t.dtype)
    return t


class Workspace:
    """Caller-owned scratch for the kernels: zeroed once, reused across calls on one stream."""

    def __init__(self, B: int, k: int, kt: Optional[int] = None, M: int = 0, device=None):
        kt = k if kt is None else kt
        n = int(lib().svd_workspace_bytes(B, k, kt, M))
        self.nbytes = max(n, 256)
        # torch's caching allocator returns 512-byte aligned blocks
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        assert self.buf.data_ptr() % 256 == 0
        self.shape = (B, k, kt, M)

    def fits(self, B, k, kt, M=0) -> bool:
        return int(lib().svd_workspace_bytes(B, k, kt, M)) <= self.nbytes

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())


def _ws(ws, B, k, kt, M, device):
    if ws is None or not ws.fits(B, k, kt, M):
        ws = Workspace(B, k, kt, M, device=device)
    return ws


def svd_workspace_bytes(B: int, k: int, kt: int, M: int = 0) -> int:
    return int(lib().svd_workspace_bytes(B, k, kt, M))


def svd_get_device_error(ws: Workspace, stream=None) -> int:
    return int(lib().svd_get_device_error(ws.ptr, _stream(stream)))


def svd_status_string(code: int) -> str:
    return lib().svd_status_string(int(code)).decode()


def svd_length_head(h, W1, b1, w2, b2: float, k: int, gamma: float = 1.0, rnd: int = BK_CEIL,
                    ws: Optional[Workspace] = None, stream=None):
    """a1: returns (bhat [B] fp32, b_k [B] int32) on h's device."""
    B, H = h.shape
    M = W1.shape[0]
    dev = h.device
    ws = _ws(ws, B, k, k, M, dev)
    bhat = torch.empty(B, dtype=torch.float32, device=dev)
    bk = torch.empty(B, dtype=torch.int32, device=dev)
    _check(lib().svd_length_head(_ptr(_bits(h)), _ptr(_bits(W1)), _ptr(b1), _ptr(_bits(w2)),
                                 float(b2), B, H, M, k, float(gamma), int(rnd), _ptr(bhat),
                                 _ptr(bk), ws.ptr, ws.nbytes, _stream(stream)), "svd_length_head")
    return bhat, bk


def _row_info_tensor(B, kt, dev):
    return torch.empty((B, kt, 8), dtype=torch.int32, device=dev)


def row_info_dict(ri: torch.Tensor) -> dict:
    """Split a [B, kt, 8] int32 row-info buffer into named fields (ints / floats)."""
    out = {}
    for j, name in enumerate(ROW_INFO_FIELDS):
        col = ri[..., j]
        out[name] = col if j < 4 else col.view(torch.float32)
    return out


def svd_verify(D, T, draft_tok, bk, mode: int = GREEDY, temperature: float = 1.0, seed: int = 0,
               step: int = 0, row_info: bool = False, ws: Optional[Workspace] = None, stream=None):
    """a2-a4: truncated verification.  Returns dict(accept_len, emitted, n_emitted[, row_info])."""
    B, k, V = D.shape
    kt = T.shape[1]
    dev = D.device
    ws = _ws(ws, B, k, kt, 0, dev)
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    emitted = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    ne = torch.empty(B, dtype=torch.int32, device=dev)
    ri = _row_info_tensor(B, kt, dev) if row_info else None
    _check(lib().svd_verify(_ptr(_bits(D)), _ptr(_bits(T)), _ptr(draft_tok), _ptr(bk), B, k, kt, V,
                            int(mode), float(temperature), int(seed), int(step), _ptr(acc),
                            _ptr(emitted), _ptr(ne), _ptr(ri), ws.ptr, ws.nbytes, _stream(stream)),
           "svd_verify")
    out = dict(accept_len=acc, emitted=emitted, n_emitted=ne)
    if ri is not None:
        out["row_info"] = ri
    return out


def svd_distill_loss_grad(D, T, bk, lam: float, clip_c: float, temperature: float = 1.0,
                          grad_scale: float = 1.0, dlogits_fp32: bool = False,
                          ws: Optional[Workspace] = None, stream=None, dlogits=None):
    """a5: returns dict(loss_rows [B,k], loss_total [1], dlogits [B,k,V])."""
    B, k, V = D.shape
    kt = T.shape[1]
    dev = D.device
    ws = _ws(ws, B, k, kt, 0, dev)
    loss_rows = torch.empty((B, k), dtype=torch.float32, device=dev)
    loss_total = torch.empty(1, dtype=torch.float32, device=dev)
    if dlogits is None:
        dlogits = torch.empty((B, k, V), dtype=torch.float32 if dlogits_fp32 else torch.bfloat16,
                              device=dev)
    _check(lib().svd_distill_loss_grad(_ptr(_bits(D)), _ptr(_bits(T)), _ptr(bk), B, k, kt, V,
                                       float(lam), float(clip_c), float(temperature),
                                       float(grad_scale), _ptr(loss_rows), _ptr(loss_total),
                                       _ptr(dlogits), int(bool(dlogits_fp32)), ws.ptr, ws.nbytes,
                                       _stream(stream)), "svd_distill_loss_grad")
    return dict(loss_rows=loss_rows, loss_total=loss_total, dlogits=dlogits)


class VerifyDistill:
    """Preallocated outputs + argument block for repeated fused calls (the benchmark path)."""

    def __init__(self, D, T, *, head=None, bk_in=None, draft_tok=None, mode=GREEDY,
                 temperature=1.0, seed=0, step=0, lam=0.5, clip_c=1.0, grad_scale=1.0,
                 gamma=1.0, rnd=BK_CEIL, dlogits_fp32=False, row_info=False, ws=None,
                 full_k=False, labels=False, head_preact=False):
        B, k, V = D.shape
        kt = T.shape[1]
        dev = D.device
        self.D, self.T, self.head, self.draft_tok, self.bk_in = D, T, head, draft_tok, bk_in
        M = head[1].shape[0] if head is not None else 0
        self.ws = _ws(ws, B, k, kt, M, dev)
        self.bhat = torch.empty(B, dtype=torch.float32, device=dev)
        self.bk = torch.empty(B, dtype=torch.int32, device=dev)
        self.accept_len = torch.empty(B, dtype=torch.int32, device=dev)
        self.emitted = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
        self.n_emitted = torch.empty(B, dtype=torch.int32, device=dev)
        self.loss_rows = torch.empty((B, k), dtype=torch.float32, device=dev)
        self.loss_total = torch.empty(1, dtype=torch.float32, device=dev)
        self.dlogits = torch.empty((B, k, V), dtype=torch.float32 if dlogits_fp32 else torch.bfloat16,
                                   device=dev)
        self.row_info = _row_info_tensor(B, kt, dev) if row_info else None
        # length-head labels: a / b_k as truncated verification sees it, and a / k (full-k mode)
        self.label_proxy = torch.empty(B, dtype=torch.float32, device=dev) if labels else None
        self.label_full = torch.empty(B, dtype=torch.float32, device=dev) if labels else None
        # the head's pre-activations, for an online update that reuses this forward
        self.head_preact = (torch.empty((B, M), dtype=torch.float32, device=dev)
                            if head_preact and head is not None else None)
        a = VerifyDistillArgs()
        if head is not None:
            h, W1, b1, w2, b2 = head
            a.h, a.W1, a.b1, a.w2 = _ptr(_bits(h)), _ptr(_bits(W1)), _ptr(b1), _ptr(_bits(w2))
            a.b2, a.H, a.M = float(b2), h.shape[1], W1.shape[0]
        else:
            if bk_in is None:
                raise ValueError("either head or bk_in is required")
            a.bk_in = _ptr(bk_in)
        a.gamma, a.rnd = float(gamma), int(rnd)
        a.D, a.T, a.draft_tok = _ptr(_bits(D)), _ptr(_bits(T)), _ptr(draft_tok)
        a.B, a.k, a.kt, a.V = B, k, kt, V
        a.mode, a.temperature, a.seed, a.step = int(mode), float(temperature), int(seed), int(step)
        a.lambda_, a.clip_c, a.grad_scale = float(lam), float(clip_c), float(grad_scale)
        a.dlogits_fp32 = int(bool(dlogits_fp32))
        a.bhat, a.bk = _ptr(self.bhat), _ptr(self.bk)
        a.accept_len, a.emitted, a.n_emitted = _ptr(self.accept_len), _ptr(self.emitted), _ptr(self.n_emitted)
        a.loss_rows, a.loss_total, a.dlogits = _ptr(self.loss_rows), _ptr(self.loss_total), _ptr(self.dlogits)
        a.row_info = _ptr(self.row_info)
        a.full_k = int(bool(full_k))
        a.label_proxy, a.label_full = _ptr(self.label_proxy), _ptr(self.label_full)
        a.head_preact = _ptr(self.head_preact)
        self.args = a

    def set_step(self, step: int):
        self.args.step = int(step)

    def __call__(self, stream=None):
        _check(lib().svd_verify_distill(ctypes.byref(self.args), self.ws.ptr, self.ws.nbytes,
                                        _stream(stream)), "svd_verify_distill")
        return self

    def outputs(self) -> dict:
        out = dict(bhat=self.bhat, bk=self.bk, accept_len=self.accept_len, emitted=self.emitted,
                   n_emitted=self.n_emitted, loss_rows=self.loss_rows, loss_total=self.loss_total,
                   dlogits=self.dlogits)
        if self.row_info is not None:
            out["row_info"] = self.row_info
        if self.label_proxy is not None:
            out["label_proxy"] = self.label_proxy
            out["label_full"] = self.label_full
        if self.head_preact is not None:
            out["head_preact"] = self.head_preact
        return out


def svd_verify_distill(D, T, **kw) -> dict:
    """a1-a5 in one call; keyword arguments as in :class:`VerifyDistill`."""
    return VerifyDistill(D, T, **kw)().outputs()


class LengthHeadTrainer:
    """Online AdamW training of the length head through ``svd_length_head_update``.

    Holds fp32 master weights, AdamW moments and the bf16 copies the forward serves
    (``W1``, ``w2``; pass ``head()`` to :class:`VerifyDistill`).  Defaults: learning rate 2e-4
    (the pages' value), betas (0.9, 0.999), eps 1e-8, weight decay 0.01.
    """

    def __init__(self, W1, b1, w2, b2: float, B: int, lr=2e-4, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.01):
        dev = W1.device
        M, H = W1.shape
        self.B, self.H, self.M = B, H, M
        self.W1m = W1.float().contiguous().clone()
        self.b1 = (torch.zeros(M, device=dev) if b1 is None else b1.float().clone()).contiguous()
        self.w2m = w2.float().contiguous().clone()
        self.b2 = torch.full((1,), float(b2), dtype=torch.float32, device=dev)
        self.W1 = self.W1m.to(torch.bfloat16).contiguous()
        self.w2 = self.w2m.to(torch.bfloat16).contiguous()
        self.moments = [torch.zeros_like(t) for t in (self.W1m, self.W1m, self.b1, self.b1,
                                                      self.w2m, self.w2m, self.b2, self.b2)]
        self.loss = torch.zeros(1, dtype=torch.float32, device=dev)
        self.bhat = torch.zeros(B, dtype=torch.float32, device=dev)
        self.ws = Workspace(B, 1, 1, M, device=dev)
        self.step_count = 0
        self.hyper = (float(lr), float(betas[0]), float(betas[1]), float(eps), float(weight_decay))

    def head(self, h):
        """The (h, W1, b1, w2, b2) tuple for :class:`VerifyDistill` (b2 read back from device)."""
        return (h, self.W1, self.b1, self.w2, float(self.b2.item()))

    def step(self, h, label, stream=None, preact=None, bhat=None):
        """One AdamW step on l = mean_b (bhat_b - label_b)^2; returns (loss, bhat) tensors.

        With ``preact`` and ``bhat`` (the ``head_preact`` and ``bhat`` of a
        :class:`VerifyDistill` step on the same h with this trainer's current weights), the
        step reuses that forward instead of running its own."""
        if h.shape != (self.B, self.H):
            raise ValueError("h must be [B, H] = [%d, %d]" % (self.B, self.H))
        if (preact is None) != (bhat is None):
            raise ValueError("preact and bhat go together")
        self.step_count += 1
        a = HeadUpdateArgs()
        bhat_buf = self.bhat
        if preact is not None:
            if preact.shape != (self.B, self.M) or preact.dtype != torch.float32:
                raise ValueError("preact must be fp32 [B, M]")
            if bhat.shape != (self.B,) or bhat.dtype != torch.float32 or not bhat.is_contiguous():
                raise ValueError("bhat must be a contiguous fp32 [B] tensor")
            bhat_buf = bhat            # read by the update, not written
            a.preact = _ptr(preact.contiguous())
        lab = label.float().contiguous()
        self._label = lab   # alive until the launch is enqueued
        a.h, a.label = _ptr(_bits(h)), _ptr(lab)
        a.B, a.H, a.M = self.B, self.H, self.M
        a.W1m, a.b1, a.w2m, a.b2 = _ptr(self.W1m), _ptr(self.b1), _ptr(self.w2m), _ptr(self.b2)
        a.W1, a.w2 = _ptr(self.W1), _ptr(self.w2)
        (a.mW1, a.vW1, a.mb1, a.vb1, a.mw2, a.vw2, a.mb2, a.vb2) = [_ptr(t) for t in self.moments]
        a.step = self.step_count
        a.lr, a.beta1, a.beta2, a.eps, a.weight_decay = self.hyper
        a.loss, a.bhat = _ptr(self.loss), _ptr(bhat_buf)
        _check(lib().svd_length_head_update(ctypes.byref(a), self.ws.ptr, self.ws.nbytes,
                                            _stream(stream)), "svd_length_head_update")
        return self.loss, bhat_buf


REPORT_FIELDS = ("tau_measured", "acc", "tau_model", "eta_model", "eta_measured", "mean_bk",
                 "mean_accept", "B")


def svd_speedup_report(accept_len, bk, n_emitted, k: int, rho: float = 0.0, stream=None):
    """E[tau] (measured and modelled), Acc, eta and per-position acceptance as a fp64 CUDA
    tensor [8 + k]; see :func:`report_dict` for the field names."""
    out = torch.empty(8 + int(k), dtype=torch.float64, device=accept_len.device)
    _check(lib().svd_speedup_report(_ptr(accept_len), _ptr(bk), _ptr(n_emitted),
                                    int(accept_len.numel()), int(k), float(rho), _ptr(out),
                                    _stream(stream)), "svd_speedup_report")
    return out


def report_dict(out) -> dict:
    v = out.double().cpu().tolist()
    d = dict(zip(REPORT_FIELDS, v[:8]))
    d["alpha"] = v[8:]
    return d


NOALLOC_SCRATCH_BYTES = 4 << 20


def svd_verify_distill_noalloc(vd: VerifyDistill, status_out=None, stream=None) -> None:
    """The fused call on the library's static per-device scratch instead of ``vd.ws``.

    For callers that cannot allocate device memory on their path (a runtime that has claimed
    nearly all HBM for its own pools, or a host program without a device allocator): the C
    entry point allocates nothing.  ``status_out`` is an optional one-element int32/uint32 CUDA
    tensor that receives the device status word.  Overlapping calls on one device race on the
    shared scratch; the first call per device must come before any stream capture.
    """
    _check(lib().svd_verify_distill_noalloc(ctypes.byref(vd.args), _ptr(status_out),
                                            _stream(stream)), "svd_verify_distill_noalloc")


def svd_selftest_wait_timeout(ws: Workspace, limit_ns: int, stream=None) -> None:
    _check(lib().svd_selftest_wait_timeout(ws.ptr, ws.nbytes, int(limit_ns), _stream(stream)),
           "svd_selftest_wait_timeout")


INF = math.inf


# ------------------------------------------------------------------------------------------
# vocab-sharded pass (include/svd_vocab.h)
# ------------------------------------------------------------------------------------------
def svd_vs_exchange_bytes(B: int, kt: int, which: int) -> int:
    return int(lib().svd_vs_exchange_bytes(B, kt, which))


def svd_vs_workspace_bytes(B: int, k: int, kt: int) -> int:
    return int(lib().svd_vs_workspace_bytes(B, k, kt))


class VocabShard:
    """One rank's part of the vocab-sharded verify-and-distill pass.

    ``D`` [B, k, Vl] and ``T`` [B, kt, Vl] are this rank's slices (ids ``v0 .. v0+Vl-1``) of
    the logit rows.  The three calls ``svd_vs_stats``, ``svd_vs_resolve`` and ``svd_vs_finish``
    read and write the exchange buffers ``send1``/``recv1`` and ``send2``/``recv2`` (uint8,
    rank r's records at block r of ``recv*``); moving ``send*`` of every rank into ``recv*``
    is the caller's all-gather (``vocab_parallel``)."""

    def __init__(self, D, T, bk, *, V: int, v0: int, P: int, rank: int, draft_tok=None,
                 mode: int = GREEDY, temperature: float = 1.0, seed: int = 0, step: int = 0,
                 distill: bool = True, lam: float = 0.5, clip_c: float = 1.0,
                 grad_scale: float = 1.0, dlogits_fp32: bool = False, row_info: bool = False):
        B, k, Vl = D.shape
        kt = T.shape[1]
        dev = D.device
        self.shape = (B, k, kt, V, v0, Vl, P, rank)
        self.mode = int(mode)
        self.distill = bool(distill)
        self._keep = [_bits(D), _bits(T), bk, draft_tok]
        i32 = dict(dtype=torch.int32, device=dev)
        self.accept_len = torch.empty(B, **i32)
        self.emitted = torch.empty((B, k + 1), **i32)
        self.n_emitted = torch.empty(B, **i32)
        self.loss_rows = torch.empty((B, k), dtype=torch.float32, device=dev) if distill else None
        self.loss_total = torch.empty(1, dtype=torch.float32, device=dev) if distill else None
        self.dlogits = (torch.empty((B, k, Vl), dtype=torch.float32 if dlogits_fp32 else torch.bfloat16,
                                    device=dev) if distill else None)
        self.row_info = _row_info_tensor(B, kt, dev) if row_info else None
        u8 = dict(dtype=torch.uint8, device=dev)
        n1, n2 = svd_vs_exchange_bytes(B, kt, 1), svd_vs_exchange_bytes(B, kt, 2)
        self.send1 = torch.empty(max(n1, 16), **u8)
        self.recv1 = torch.empty(max(P * n1, 16), **u8)
        self.send2 = torch.empty(max(n2, 16), **u8)
        self.recv2 = torch.empty(max(P * n2, 16), **u8)
        nw = max(svd_vs_workspace_bytes(B, k, kt), 256)
        self.ws = torch.zeros(nw, **u8)
        assert self.ws.data_ptr() % 256 == 0
        a = VsArgs()
        a.D, a.T = _ptr(D), _ptr(T)
        a.draft_tok, a.bk = _ptr(draft_tok), _ptr(bk)
        a.B, a.k, a.kt, a.V, a.v0, a.Vl, a.P, a.rank = B, k, kt, V, v0, Vl, P, rank
        a.mode, a.temperature, a.seed, a.step = int(mode), float(temperature), int(seed), int(step)
        a.distill = 1 if distill else 0
        a.lambda_, a.clip_c, a.grad_scale = float(lam), float(clip_c), float(grad_scale)
        a.dlogits, a.dlogits_fp32 = _ptr(self.dlogits), 1 if dlogits_fp32 else 0
        a.loss_rows, a.loss_total = _ptr(self.loss_rows), _ptr(self.loss_total)
        a.accept_len, a.emitted, a.n_emitted = _ptr(self.accept_len), _ptr(self.emitted), _ptr(self.n_emitted)
        a.row_info = _ptr(self.row_info)
        self.args = a

    @property
    def stochastic(self) -> bool:
        return self.mode == STOCHASTIC

    def set_step(self, step: int):
        self.args.step = int(step)

    def _ws(self):
        return ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel()

    def stats(self, stream=None):
        w, n = self._ws()
        _check(lib().svd_vs_stats(ctypes.byref(self.args), _ptr(self.send1), w, n, _stream(stream)),
               "svd_vs_stats")

    def resolve(self, stream=None):
        w, n = self._ws()
        _check(lib().svd_vs_resolve(ctypes.byref(self.args), _ptr(self.recv1), _ptr(self.send2), w, n,
                                    _stream(stream)), "svd_vs_resolve")

    def finish(self, stream=None):
        w, n = self._ws()
        _check(lib().svd_vs_finish(ctypes.byref(self.args), _ptr(self.recv2), w, n, _stream(stream)),
               "svd_vs_finish")

    def device_error(self, stream=None) -> int:
        return int(lib().svd_get_device_error(ctypes.c_void_p(self.ws.data_ptr()), _stream(stream)))

    def outputs(self) -> dict:
        out = dict(accept_len=self.accept_len, emitted=self.emitted, n_emitted=self.n_emitted)
        if self.distill:
            out.update(loss_rows=self.loss_rows, loss_total=self.loss_total, dlogits=self.dlogits)
        if self.row_info is not None:
            out["row_info"] = self.row_info
        return out


# ------------------------------------------------------------------------------------------
# operators on a tree of drafts (include/svd_tree.h)
# ------------------------------------------------------------------------------------------
TREE_MAX_NODES = 64
MASK_VALUE = -32768.0   # finite: svd_verify and svd_verify_distill want finite logits


def _tensor(t, name: str, dtype, shape, dev):
    """Pointer of a contiguous CUDA tensor with this dtype (or one of them) and shape; None passes."""
    if t is None:
        return None
    p = _ptr(t)
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s: unexpected dtype %s" % (name, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    return p


def _pages(t, name: str, dtype, like, dev):
    """Pointer and page stride of a cache [n_pages, page_size, Hkv, D]; pages may lie apart (a slice
    of a buffer that holds K and V pages), their inside is contiguous."""
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if t.dtype != dtype or t.device != dev:
        raise TypeError("%s must be %s on %s, got %s on %s" % (name, dtype, dev, t.dtype, t.device))
    if t.dim() != 4 or tuple(t.shape[2:]) != tuple(like):
        raise ValueError("%s must be [n_pages, page_size, %d, %d], got %s" % ((name,) + tuple(like) + (tuple(t.shape),)))
    if t.shape[0] and not t[0].is_contiguous():
        raise ValueError("%s: the inside of a page must be contiguous" % name)
    stride = t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2] * t.shape[3]
    return ctypes.c_void_p(t.data_ptr()), stride


def _raw_stream(index: int) -> int:
    """cudaStream_t of the current stream of a device."""
    return torch._C._cuda_getCurrentRawStream(index)


class _TreeOp:
    """Preallocated outputs, argument block and workspace of one operator, for repeated calls.

    The calls of one object share its workspace and outputs: a call on another stream than the
    last one first waits for that stream (not while it is being captured: order captured calls
    yourself, give graphs that may run at the same time an object each, and keep the object as
    long as the graph)."""

    _fn = ""

    def _set_up(self, args, nbytes: int, dev, keep):
        self.args, self.device, self._keep = args, dev, keep
        with torch.cuda.device(dev):
            self.ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=dev)
            self._last = torch.cuda.current_stream(dev)
        self._raw = self._last.cuda_stream
        assert self.ws.data_ptr() % 256 == 0
        self._call = getattr(lib(), self._fn)
        self._ws, self._nws = ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel()
        self._ref = ctypes.byref(args)

    def _order(self, s):
        if s.device != self.device:
            raise ValueError("the stream is on %s, the tensors on %s" % (s.device, self.device))
        with torch.cuda.stream(s):
            capturing = torch.cuda.is_current_stream_capturing()
        if not capturing:
            s.wait_stream(self._last)
            self._record(s)
            self._last, self._raw = s, s.cuda_stream

    def _record(self, s):
        """The memory of this object's tensors is not handed out again before the work on s has ended."""
        for t in [self.ws, *self._keep, *self.outputs().values()]:
            if t is not None:
                t.record_stream(s)

    def __call__(self, stream=None):
        # the raw handle is enough while the stream stays the same (a Stream object costs 2 us)
        raw = _raw_stream(self.device.index) if stream is None else stream.cuda_stream
        if raw != self._raw or stream is not None and stream.device != self.device:
            self._order(torch.cuda.current_stream(self.device) if stream is None else stream)
        if torch.cuda.current_device() == self.device.index:
            code = self._call(self._ref, self._ws, self._nws, raw)
        else:
            with torch.cuda.device(self.device):
                code = self._call(self._ref, self._ws, self._nws, raw)
        if code:
            raise SvdError(code, self._fn)
        return self

    def device_error(self, stream=None) -> int:
        """The status word of the calls so far; synchronizes the stream of the last call (give the one
        that a graph was replayed on)."""
        with torch.cuda.device(self.device):
            s = self._last if stream is None else stream
            return int(lib().svd_get_device_error(self._ws, s.cuda_stream))

    def reset(self):
        """Zeroes the workspace, the status word with it, on the stream of the last call
        (``svd_workspace_reset``): for use after a device error."""
        with torch.cuda.device(self.device):
            _check(lib().svd_workspace_reset(self._ws, self._nws, self._last.cuda_stream), "svd_workspace_reset")
        return self


def _once(op, args, kw, stream):
    """One call of a fresh object, with its buffers allocated on the stream that it runs on.  The caller orders a
    ``stream`` behind the work that made the inputs, but may let go of them as soon as the call returns."""
    if stream is None:
        return op(*args, **kw)().outputs()
    with torch.cuda.stream(stream):
        once = op(*args, **kw)(stream)
        if not torch.cuda.is_current_stream_capturing():
            once._record(stream)
        return once.outputs()


class TreeAttention(_TreeOp):
    """Attention of the drafted nodes over the paged cache and over their ancestors.

    ``q`` [B, n, Hq, D], ``k_new`` and ``v_new`` [B, n, Hkv, D], ``cache_k`` and ``cache_v``
    [n_pages, page_size, Hkv, D], all bf16 or all fp16; ``page_table`` [B, max_pages] and
    ``cache_len`` [B] int32.  ``parent`` [B, n] int32 gives the tree (default: a chain), ``n_nodes``
    [B] int32 the nodes in use.  ``n = 1`` is a decode step; more than 64 new tokens at once, as within
    a prompt, are not offered.  Softmax weights are rounded to q's type for the product with V, all
    else is fp32.  Outputs: ``out`` [B, n, Hq, D] and, with ``lse=True``, ``lse`` [B, n, Hq] fp32."""

    _fn = "svd_tree_attention"

    def __init__(self, q, k_new, v_new, cache_k, cache_v, page_table, cache_len, *, parent=None,
                 n_nodes=None, scale: Optional[float] = None, lse: bool = False):
        if q.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("expected bf16 or fp16 queries, got %s" % q.dtype)
        if q.dim() != 4 or k_new.dim() != 4:
            raise ValueError("q is [B, n, Hq, D], k_new and v_new are [B, n, Hkv, D]")
        B, n, Hq, D = q.shape
        Hkv, dev, i32 = k_new.shape[2], q.device, torch.int32
        a = TreeAttentionArgs()
        a.q = _tensor(q, "q", q.dtype, q.shape, dev)
        a.k_new = _tensor(k_new, "k_new", q.dtype, (B, n, Hkv, D), dev)
        a.v_new = _tensor(v_new, "v_new", q.dtype, (B, n, Hkv, D), dev)
        a.cache_k, a.page_stride_k = _pages(cache_k, "cache_k", q.dtype, (Hkv, D), dev)
        a.cache_v, a.page_stride_v = _pages(cache_v, "cache_v", q.dtype, (Hkv, D), dev)
        if cache_k.shape != cache_v.shape:
            raise ValueError("cache_k and cache_v differ in shape")
        a.n_pages, a.page_size, a.max_pages = cache_k.shape[0], cache_k.shape[1], page_table.shape[-1]
        a.page_table = _tensor(page_table, "page_table", i32, (B, a.max_pages), dev)
        a.cache_len = _tensor(cache_len, "cache_len", i32, (B,), dev)
        a.parent = _tensor(parent, "parent", i32, (B, n), dev)
        a.n_nodes = _tensor(n_nodes, "n_nodes", i32, (B,), dev)
        a.B, a.n, a.Hq, a.Hkv, a.D = B, n, Hq, Hkv, D
        a.dtype = 0 if q.dtype == torch.bfloat16 else 1
        a.scale = float(1.0 / math.sqrt(max(D, 1)) if scale is None else scale)
        self.out = torch.empty_like(q)
        self.lse = torch.empty((B, n, Hq), dtype=torch.float32, device=dev) if lse else None
        a.out, a.lse = _ptr(self.out), _ptr(self.lse)
        self._set_up(a, lib().svd_tree_attention_workspace_bytes(B, n, Hq, Hkv, D), dev,
                     [q, k_new, v_new, cache_k, cache_v, page_table, cache_len, parent, n_nodes])

    def outputs(self) -> dict:
        return dict(out=self.out) if self.lse is None else dict(out=self.out, lse=self.lse)


def svd_tree_attention(*args, stream=None, **kw) -> dict:
    """One call; arguments as in :class:`TreeAttention`."""
    return _once(TreeAttention, args, kw, stream)


def _lists(a, logits, history, prompt_len, hist_len, node_tok, parent, repetition, mask):
    """The arguments that the processing and its gradient share."""
    if logits.dim() != 3:
        raise ValueError("logits are [B, n, V]")
    B, n, V = logits.shape
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    a.logits = _ptr(_bits(logits))
    a.B, a.n, a.V = B, n, V
    if history is None and (prompt_len is not None or hist_len is not None):
        raise ValueError("prompt_len and hist_len go with history")
    if history is not None:
        a.hist_stride = history.shape[-1]
        a.history = _tensor(history, "history", i32, (B, a.hist_stride), dev)
    a.prompt_len = _tensor(prompt_len, "prompt_len", i32, (B,), dev)
    a.hist_len = _tensor(hist_len, "hist_len", i32, (B,), dev)
    a.node_tok = _tensor(node_tok, "node_tok", i32, (B, n), dev)
    a.parent = _tensor(parent, "parent", i32, (B, n), dev)
    a.repetition = _tensor(repetition, "repetition", f32, (B,), dev)
    if mask is not None:
        if mask.dim() != 3 or mask.shape[1] not in (1, n):
            raise ValueError("mask is [B, 1 or n, ceil(V / 32)]")
        a.mask_rows = mask.shape[1]
        a.mask = _tensor(mask, "mask", (i32, torch.uint32), (B, a.mask_rows, (V + 31) // 32), dev)


class LogitsProcess(_TreeOp):
    """Penalties, biases and grammar masks on the logits [B, n, V] of every row of a tree.

    ``history`` [B, S] int32 holds a sequence's tokens: ``prompt_len`` [B] of the prompt, then the
    generated ones up to ``hist_len`` [B]; ``node_tok`` [B, n] and ``parent`` [B, n] the drafted
    ones, of which a row sees its ancestors' and its own.  ``repetition``, ``frequency`` and
    ``presence`` [B] fp32; ``bias_tok`` [B, nb] int32 with ``bias_val`` [B, nb] fp32; ``mask``
    [B, 1 or n, ceil(V / 32)] int32, a set bit allows the id, the others get ``mask_value``.
    -1 in a list of ids is padding.  ``out`` may be ``logits`` (in place).  Outputs: ``out`` bf16
    (unless ``values=False``) and, with ``argmax=True``, ``argmax`` [B, n] int32 of the result."""

    _fn = "svd_logits_process"

    def __init__(self, logits, *, history=None, prompt_len=None, hist_len=None, node_tok=None,
                 parent=None, repetition=None, frequency=None, presence=None, bias_tok=None,
                 bias_val=None, mask=None, mask_value: float = MASK_VALUE, out=None,
                 values: bool = True, argmax: bool = False):
        a = LogitsProcessArgs()
        _lists(a, logits, history, prompt_len, hist_len, node_tok, parent, repetition, mask)
        B, n, V = logits.shape
        dev, i32, f32 = logits.device, torch.int32, torch.float32
        a.frequency = _tensor(frequency, "frequency", f32, (B,), dev)
        a.presence = _tensor(presence, "presence", f32, (B,), dev)
        if (bias_tok is None) != (bias_val is None):
            raise ValueError("bias_tok and bias_val go together")
        if bias_tok is not None:
            a.n_bias = bias_tok.shape[-1]
            a.bias_tok = _tensor(bias_tok, "bias_tok", i32, (B, a.n_bias), dev)
            a.bias_val = _tensor(bias_val, "bias_val", f32, (B, a.n_bias), dev)
        a.mask_value = float(mask_value)
        if not values and (out is not None or not argmax):
            raise ValueError("values=False leaves argmax=True alone, without out")
        self.out = (torch.empty_like(logits) if out is None else out) if values else None
        self.argmax = torch.empty((B, n), dtype=i32, device=dev) if argmax else None
        a.out = _tensor(self.out, "out", torch.bfloat16, (B, n, V), dev)
        a.argmax = _ptr(self.argmax)
        self._set_up(a, lib().svd_logits_process_workspace_bytes(B, n), dev,
                     [logits, history, prompt_len, hist_len, node_tok, parent, repetition, frequency,
                      presence, bias_tok, bias_val, mask])

    def outputs(self) -> dict:
        return {k: t for k, t in (("out", self.out), ("argmax", self.argmax)) if t is not None}


def svd_logits_process(logits, stream=None, **kw) -> dict:
    """One call; arguments as in :class:`LogitsProcess`."""
    return _once(LogitsProcess, (logits,), kw, stream)


class LogitsProcessGrad(_TreeOp):
    """Gradient of :class:`LogitsProcess` with respect to the raw ``logits``, from the gradient ``dz``
    [B, n, V] (bf16 or fp32) with respect to its output, e.g. ``dlogits`` of :class:`VerifyDistill`
    on processed logits.  ``out`` may be ``dz`` (in place).  Frequency, presence and bias shift a
    logit and do not appear.  Output: ``dlogits`` of dz's type."""

    _fn = "svd_logits_process_grad"

    def __init__(self, dz, logits, *, history=None, prompt_len=None, hist_len=None, node_tok=None,
                 parent=None, repetition=None, frequency=None, presence=None, bias_tok=None,
                 bias_val=None, mask=None, out=None):
        a = LogitsProcessArgs()
        _lists(a, logits, history, prompt_len, hist_len, node_tok, parent, repetition, mask)
        B, n, V = logits.shape
        dev = logits.device
        a.dz = _tensor(dz, "dz", (torch.bfloat16, torch.float32), (B, n, V), dev)
        self.dlogits = torch.empty_like(dz) if out is None else out
        a.dlogits = _tensor(self.dlogits, "out", dz.dtype, (B, n, V), dev)
        a.grad_fp32 = int(dz.dtype == torch.float32)
        self._set_up(a, lib().svd_logits_process_workspace_bytes(B, n), dev,
                     [dz, logits, history, prompt_len, hist_len, node_tok, parent, repetition, mask])

    def outputs(self) -> dict:
        return dict(dlogits=self.dlogits)


def svd_logits_process_grad(dz, logits, stream=None, **kw) -> dict:
    """One call; arguments as in :class:`LogitsProcessGrad`."""
    return _once(LogitsProcessGrad, (dz, logits), kw, stream)


class TreeVerify(_TreeOp):
    """Greedy acceptance over a tree of drafts: ``node_tok`` [B, n] int32 with ``parent`` [B, n]
    (default: a chain) and ``n_nodes`` [B], against the target's ``logits`` [B, n, V] bf16 or its
    choice ``target_tok`` [B, n] int32 after every node.  Outputs: ``path`` [B, n] (nodes, -1
    padded), ``n_path``, ``accept_len``, ``emitted`` [B, n], ``n_emitted`` and ``target_argmax``."""

    _fn = "svd_tree_verify"

    def __init__(self, node_tok, *, logits=None, target_tok=None, parent=None, n_nodes=None):
        if (logits is None) == (target_tok is None):
            raise ValueError("either logits or target_tok is required")
        if node_tok.dim() != 2:
            raise ValueError("node_tok is [B, n]")
        B, n = node_tok.shape
        dev, i32 = node_tok.device, torch.int32
        a = TreeVerifyArgs()
        if logits is not None:
            if logits.dim() != 3:
                raise ValueError("logits are [B, n, V]")
            a.V = logits.shape[2]
            a.T = _tensor(logits, "logits", torch.bfloat16, (B, n, a.V), dev)
        a.target_tok = _tensor(target_tok, "target_tok", i32, (B, n), dev)
        a.node_tok = _tensor(node_tok, "node_tok", i32, (B, n), dev)
        a.parent = _tensor(parent, "parent", i32, (B, n), dev)
        a.n_nodes = _tensor(n_nodes, "n_nodes", i32, (B,), dev)
        a.B, a.n = B, n
        new = lambda *shape: torch.empty(shape, dtype=i32, device=dev)  # noqa: E731
        self.target_argmax, self.path, self.emitted = new(B, n), new(B, n), new(B, n)
        self.n_path, self.accept_len, self.n_emitted = new(B), new(B), new(B)
        for name in ("target_argmax", "path", "emitted", "n_path", "accept_len", "n_emitted"):
            setattr(a, name, _ptr(getattr(self, name)))
        self._set_up(a, lib().svd_tree_verify_workspace_bytes(B, n), dev,
                     [logits, target_tok, node_tok, parent, n_nodes])

    def outputs(self) -> dict:
        return dict(target_argmax=self.target_argmax, path=self.path, n_path=self.n_path,
                    accept_len=self.accept_len, emitted=self.emitted, n_emitted=self.n_emitted)


def svd_tree_verify(node_tok, stream=None, **kw) -> dict:
    """One call; arguments as in :class:`TreeVerify`."""
    return _once(TreeVerify, (node_tok,), kw, stream)


class CacheAppend(_TreeOp):
    """Append of ``count`` [B] int32 entries of ``k_new``, ``v_new`` [B, n, Hkv, D] to the paged cache
    behind ``cache_len`` [B]: the nodes ``path`` [B, n] names (``path`` and ``n_path`` of
    :class:`TreeVerify`), or the first ones.  ``new_len`` may be ``cache_len`` (updated in place).
    The cache is written in place.  Outputs: ``cache_k``, ``cache_v``, ``new_len`` [B]."""

    _fn = "svd_cache_append"

    def __init__(self, k_new, v_new, cache_k, cache_v, page_table, cache_len, count, *, path=None,
                 new_len=None):
        if k_new.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("expected bf16 or fp16 keys, got %s" % k_new.dtype)
        if k_new.dim() != 4:
            raise ValueError("k_new and v_new are [B, n, Hkv, D]")
        B, n, Hkv, D = k_new.shape
        dev, i32 = k_new.device, torch.int32
        a = CacheAppendArgs()
        a.k_new = _tensor(k_new, "k_new", k_new.dtype, (B, n, Hkv, D), dev)
        a.v_new = _tensor(v_new, "v_new", k_new.dtype, (B, n, Hkv, D), dev)
        a.cache_k, a.page_stride_k = _pages(cache_k, "cache_k", k_new.dtype, (Hkv, D), dev)
        a.cache_v, a.page_stride_v = _pages(cache_v, "cache_v", k_new.dtype, (Hkv, D), dev)
        if cache_k.shape != cache_v.shape:
            raise ValueError("cache_k and cache_v differ in shape")
        a.n_pages, a.page_size, a.max_pages = cache_k.shape[0], cache_k.shape[1], page_table.shape[-1]
        a.page_table = _tensor(page_table, "page_table", i32, (B, a.max_pages), dev)
        a.cache_len = _tensor(cache_len, "cache_len", i32, (B,), dev)
        a.count = _tensor(count, "count", i32, (B,), dev)
        a.path = _tensor(path, "path", i32, (B, n), dev)
        a.B, a.n, a.Hkv, a.D = B, n, Hkv, D
        self.cache_k, self.cache_v = cache_k, cache_v
        self.new_len = torch.empty(B, dtype=i32, device=dev) if new_len is None else new_len
        a.new_len = _tensor(self.new_len, "new_len", i32, (B,), dev)
        self._set_up(a, lib().svd_cache_append_workspace_bytes(B), dev,
                     [k_new, v_new, page_table, cache_len, count, path])

    def outputs(self) -> dict:
        return dict(cache_k=self.cache_k, cache_v=self.cache_v, new_len=self.new_len)


def svd_cache_append(*args, stream=None, **kw) -> dict:
    """One call; arguments as in :class:`CacheAppend`."""
    return _once(CacheAppend, args, kw, stream)
