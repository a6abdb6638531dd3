"""GB300 (sm_103a) speculative-decoding verify/accept library -- Python binding.

A thin ctypes layer over ``libspecverify.so`` (C ABI: the headers in ``include/``).
Each function carries the name of the C entry point it calls and only marshals
arguments: torch tensors become device pointers, the current torch stream
becomes the launch stream, outputs are allocated with torch when not given.
Every step of the verify path runs in the library's CUDA kernels; there is no
fallback -- a missing library raises.

Build the library with ``python -m speculative_decoding_verification_53_gb300.build``
(or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_UNSUPPORTED, SV_ERR_CUDA, SV_ERR_TIMEOUT, SV_ERR_BAD_INPUT = range(6)
SV_F32, SV_BF16 = 0, 1
SV_DRAFT_PROBS, SV_DRAFT_LOGITS = 0, 1
SV_SIBLINGS_WITHOUT_REPLACEMENT, SV_SIBLINGS_IID = 0, 1
SV_CACHE_BF16, SV_CACHE_E4M3 = 0, 1

EXPORTS = ("spec_verify_workspace_size", "spec_verify_chain", "spec_greedy_accept", "spec_verify_tree",
           "spec_verify_status_string", "spec_verify_last_cuda_error", "spec_verify_chain_noalloc",
           "spec_tree_mask", "spec_kv_compact", "spec_verify_tree_rule", "spec_sample_and_verify",
           "spec_verify_count_invalid", "spec_verify_rows_status", "spec_verify_chain_host",
           "spec_verify_host_sizes", "spec_kv_append", "spec_kv_read", "spec_kv_compact_paged",
           "spec_paged_attention", "spec_paged_attention_workspace_size", "spec_adjust_logits")

# out_count value of a batch row whose kernel gave up a bounded device-side wait
COUNT_TIMEOUT = -1

_lib = None


class PagedCache(ctypes.Structure):
    """sv_paged_cache of include/spec_paged_kv.h."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("num_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class SpecVerifyError(RuntimeError):
    """A non-zero sv_status returned by the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        detail = f" ({lib().spec_verify_last_cuda_error().decode()})" if status == SV_ERR_CUDA else ""
        super().__init__(f"{where}: {spec_verify_status_string(status)}{detail}")


def lib() -> ctypes.CDLL:
    """The loaded library with argument types set (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m speculative_decoding_verification_53_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, ci, u64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
    L.spec_verify_workspace_size.argtypes = [ci, ci, ci]
    L.spec_verify_workspace_size.restype = sz
    L.spec_verify_chain.argtypes = [vp, ci, vp, ci, ci, vp, vp, ci, ci, ci, u64, u64, vp, vp, vp, vp, sz, vp]
    L.spec_verify_chain.restype = ci
    L.spec_verify_chain_noalloc.argtypes = [vp, ci, vp, ci, ci, vp, vp, ci, ci, ci, u64, u64, vp, vp, vp, vp]
    L.spec_verify_chain_noalloc.restype = ci
    L.spec_greedy_accept.argtypes = [vp, ci, vp, ci, ci, ci, vp, vp, vp]
    L.spec_greedy_accept.restype = ci
    L.spec_verify_tree.argtypes = [vp, ci, vp, ci, ci, vp, vp, vp, ci, ci, ci, ci, u64, u64, vp, vp, vp, vp]
    L.spec_verify_tree.restype = ci
    L.spec_verify_tree_rule.argtypes = [vp, ci, vp, ci, ci, vp, vp, vp, ci, ci, ci, ci, ci, u64, u64, vp, vp, vp,
                                        vp]
    L.spec_verify_tree_rule.restype = ci
    L.spec_sample_and_verify.argtypes = [vp, ci, vp, ci, vp, ci, ci, ci, u64, u64, vp, vp, vp, vp, vp, sz, vp]
    L.spec_sample_and_verify.restype = ci
    L.spec_tree_mask.argtypes = [vp, ci, ci, vp, vp, vp, vp]
    L.spec_tree_mask.restype = ci
    i64 = ctypes.c_int64
    L.spec_kv_compact.argtypes = [ctypes.POINTER(vp), ci, i64, i64, ci, i64, i64, ci, vp, vp, vp, ci, ci, vp]
    L.spec_kv_compact.restype = ci
    L.spec_verify_status_string.argtypes = [ci]
    L.spec_verify_status_string.restype = ctypes.c_char_p
    L.spec_verify_last_cuda_error.argtypes = []
    L.spec_verify_last_cuda_error.restype = ctypes.c_char_p
    L.spec_verify_count_invalid.argtypes = [vp, ci, vp, vp]
    L.spec_verify_count_invalid.restype = ci
    L.spec_verify_rows_status.argtypes = [vp, ci, vp, vp]
    L.spec_verify_rows_status.restype = ci
    L.spec_verify_chain_host.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, u64, u64, vp, sz, vp]
    L.spec_verify_chain_host.restype = ci
    L.spec_verify_host_sizes.argtypes = [ci, ci, ci, ci, ci, ci, vp, vp, vp]
    L.spec_verify_host_sizes.restype = ci
    pc = ctypes.POINTER(PagedCache)
    L.spec_kv_append.argtypes = [vp, vp, ci, vp, pc, vp, vp, ci, ci, vp]
    L.spec_kv_append.restype = ci
    L.spec_kv_read.argtypes = [pc, vp, vp, ci, ci, vp, vp, ci, vp]
    L.spec_kv_read.restype = ci
    L.spec_kv_compact_paged.argtypes = [vp, ci, i64, i64, ci, i64, i64, vp, ci, ci, ci, vp, vp, vp, ci, ci, vp]
    L.spec_kv_compact_paged.restype = ci
    L.spec_paged_attention.argtypes = [vp, vp, ci, pc, vp, vp, vp, ctypes.c_float, ci, ci, ci, vp, vp, vp, sz, vp]
    L.spec_paged_attention.restype = ci
    L.spec_paged_attention_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci, ci]
    L.spec_paged_attention_workspace_size.restype = sz
    L.spec_adjust_logits.argtypes = [vp, ci, vp, vp, vp, ci, vp, vp, vp, vp, vp, vp, vp, ci, vp, ci, ci, ci, vp, vp]
    L.spec_adjust_logits.restype = ci
    _lib = L
    return L


def spec_verify_status_string(status: int) -> str:
    return lib().spec_verify_status_string(int(status)).decode()


def spec_verify_workspace_size(B: int, K: int, V: int) -> int:
    return int(lib().spec_verify_workspace_size(int(B), int(K), int(V)))


# ---------------------------------------------------------------- helpers

def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _dev(t, name, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _dtype_code_of(dtype) -> int:
    """The sv_dtype of a torch dtype (float32 or bfloat16)."""
    torch = _torch()
    if dtype == torch.float32:
        return SV_F32
    if dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_workspaces = {}


def _auto_workspace(B, K, V, stream):
    """A zero-initialised workspace cached per (device, stream) and grown on demand; the
    library leaves it zeroed after every call, so it is reused as is.  Calls on one stream
    never overlap, which is what the library requires of a shared workspace."""
    torch = _torch()
    need = spec_verify_workspace_size(B, K, V)
    if need == 0:
        return None
    s = torch.cuda.current_stream() if stream is None else stream
    key = (s.device.index, s.cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=s.device)
        _workspaces[key] = ws
    return ws


def _kind(draft_kind) -> int:
    if draft_kind in ("probs", SV_DRAFT_PROBS):
        return SV_DRAFT_PROBS
    if draft_kind in ("logits", SV_DRAFT_LOGITS):
        return SV_DRAFT_LOGITS
    raise ValueError("draft_kind must be 'probs' or 'logits'")


# ------------------------------------------------------------ entry points

def spec_verify_chain(target_logits, draft, draft_tokens, temperature, seed: int, offset: int, *,
                      draft_kind, out_tokens=None, out_count=None, out_accept_prob=None,
                      want_accept_prob: bool = False, workspace="auto", stream=None):
    """Chain verify.  target_logits [B][K+1][V] (fp32/bf16), draft [B][K][V] (probs fp32 or
    logits), draft_tokens int32 [B][K], temperature fp32 [B] (T <= 0: greedy row).
    workspace: "auto" (a cached zeroed buffer per stream), None (none: the kernels that need
    no scratch), or a caller-owned zero-initialised uint8 CUDA tensor.
    Returns (out_tokens int32 [B][K+1], out_count int32 [B], out_accept_prob fp32 [B][K] or None)."""
    torch = _torch()
    _dev(target_logits, "target_logits")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dk = _kind(draft_kind)
    _dev(draft, "draft")
    _dev(draft_tokens, "draft_tokens", torch.int32)
    _dev(temperature, "temperature", torch.float32)
    ddt = SV_F32 if draft is None else _dtype_code(draft)
    if draft is not None and tuple(draft.shape) != (B, K, V):
        raise ValueError(f"draft shape {tuple(draft.shape)} != {(B, K, V)}")
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_accept_prob is None and want_accept_prob:
        out_accept_prob = torch.empty((B, K), dtype=torch.float32, device=dev)
    if isinstance(workspace, str):
        workspace = _auto_workspace(B, K, V, stream) if B > 0 else None
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
    st = lib().spec_verify_chain(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft), ddt, dk,
                                 _ptr(draft_tokens), _ptr(temperature), B, K, V, int(seed), int(offset),
                                 _ptr(out_tokens), _ptr(out_count), _ptr(out_accept_prob), ws_ptr, ws_bytes,
                                 _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_chain")
    return out_tokens, out_count, out_accept_prob


def spec_verify_chain_noalloc(target_logits, draft, draft_tokens, temperature, seed: int, offset: int, *,
                              draft_kind, out_tokens=None, out_count=None, out_accept_prob=None,
                              want_accept_prob: bool = False, stream=None):
    """spec_verify_chain for callers that cannot provide a workspace: the library uses a
    fixed 256 KiB scratch array of its own (first call on a device sets it up, so make it
    before any graph capture; overlapping calls race).  Same arguments and results."""
    torch = _torch()
    _dev(target_logits, "target_logits")
    B, K1, V = target_logits.shape
    K = K1 - 1
    dk = _kind(draft_kind)
    _dev(draft, "draft")
    _dev(draft_tokens, "draft_tokens", torch.int32)
    _dev(temperature, "temperature", torch.float32)
    ddt = SV_F32 if draft is None else _dtype_code(draft)
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_accept_prob is None and want_accept_prob:
        out_accept_prob = torch.empty((B, K), dtype=torch.float32, device=dev)
    st = lib().spec_verify_chain_noalloc(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft), ddt, dk,
                                         _ptr(draft_tokens), _ptr(temperature), B, K, V, int(seed), int(offset),
                                         _ptr(out_tokens), _ptr(out_count), _ptr(out_accept_prob), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_chain_noalloc")
    return out_tokens, out_count, out_accept_prob


def spec_sample_and_verify(target_logits, draft_logits, temperature, seed: int, offset: int, *,
                           out_draft_tokens=None, out_tokens=None, out_count=None, out_accept_prob=None,
                           want_accept_prob: bool = False, workspace="auto", stream=None):
    """Draft sampling and verify in one call: x_k ~ softmax(draft_logits_k / T) (argmax for
    greedy rows), then the chain verify of those tokens.  target_logits [B][K+1][V],
    draft_logits [B][K][V], temperature fp32 [B].  Returns (out_draft_tokens [B][K],
    out_tokens [B][K+1], out_count [B], out_accept_prob [B][K] or None)."""
    torch = _torch()
    _dev(target_logits, "target_logits")
    _dev(draft_logits, "draft_logits")
    _dev(temperature, "temperature", torch.float32)
    B, K1, V = target_logits.shape
    K = K1 - 1
    if tuple(draft_logits.shape) != (B, K, V):
        raise ValueError(f"draft_logits shape {tuple(draft_logits.shape)} != {(B, K, V)}")
    dev = target_logits.device
    if out_draft_tokens is None:
        out_draft_tokens = torch.empty((B, K), dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_accept_prob is None and want_accept_prob:
        out_accept_prob = torch.empty((B, K), dtype=torch.float32, device=dev)
    if isinstance(workspace, str):
        workspace = _auto_workspace(B, K, V, stream) if B > 0 else None
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
    st = lib().spec_sample_and_verify(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft_logits),
                                      _dtype_code(draft_logits), _ptr(temperature), B, K, V, int(seed), int(offset),
                                      _ptr(out_draft_tokens), _ptr(out_tokens), _ptr(out_count),
                                      _ptr(out_accept_prob), ws_ptr, ws_bytes, _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_sample_and_verify")
    return out_draft_tokens, out_tokens, out_count, out_accept_prob


def spec_greedy_accept(target_logits, draft_tokens, *, out_tokens=None, out_count=None, stream=None):
    """Greedy acceptance for every row.  Returns (out_tokens [B][K+1], out_count [B])."""
    torch = _torch()
    _dev(target_logits, "target_logits")
    B, K1, V = target_logits.shape
    K = K1 - 1
    _dev(draft_tokens, "draft_tokens", torch.int32)
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty((B,), dtype=torch.int32, device=dev)
    st = lib().spec_greedy_accept(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft_tokens), B, K, V,
                                  _ptr(out_tokens), _ptr(out_count), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_greedy_accept")
    return out_tokens, out_count


def spec_verify_tree(target_logits, draft, node_tokens, parent, temperature, max_depth: int, seed: int,
                     offset: int, *, draft_kind, out_tokens=None, out_count=None, out_path=None,
                     sibling_rule="without_replacement", stream=None):
    """Tree verify.  target_logits/draft [B][N+1][V], node_tokens/parent int32 [B][N],
    temperature fp32 [B].  sibling_rule: "without_replacement" (children drawn without
    replacement from q) or "iid" (drawn independently; a token may repeat).
    Returns (out_tokens [B][D+1], out_count [B], out_path [B][D])."""
    torch = _torch()
    _dev(target_logits, "target_logits")
    B, N1, V = target_logits.shape
    N = N1 - 1
    dk = _kind(draft_kind)
    _dev(draft, "draft")
    _dev(node_tokens, "node_tokens", torch.int32)
    _dev(parent, "parent", torch.int32)
    _dev(temperature, "temperature", torch.float32)
    if tuple(draft.shape) != (B, N + 1, V):
        raise ValueError(f"draft shape {tuple(draft.shape)} != {(B, N + 1, V)}")
    D = int(max_depth)
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_path is None:
        out_path = torch.empty((B, D), dtype=torch.int32, device=dev)
    rules = {"without_replacement": SV_SIBLINGS_WITHOUT_REPLACEMENT, "iid": SV_SIBLINGS_IID}
    if sibling_rule not in rules:
        raise ValueError("sibling_rule must be 'without_replacement' or 'iid'")
    st = lib().spec_verify_tree_rule(_ptr(target_logits), _dtype_code(target_logits), _ptr(draft),
                                     _dtype_code(draft), dk, _ptr(node_tokens), _ptr(parent), _ptr(temperature), B,
                                     N, V, D, rules[sibling_rule], int(seed), int(offset), _ptr(out_tokens),
                                     _ptr(out_count), _ptr(out_path), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_tree")
    return out_tokens, out_count, out_path


def spec_verify_count_invalid(out_count, *, out_invalid=None, stream=None):
    """Number of invalid batch rows (out_count == 0) of a finished verify call, counted
    on the device in stream order; returns an int32 device tensor of one element."""
    torch = _torch()
    _dev(out_count, "out_count", torch.int32)
    if out_invalid is None:
        out_invalid = torch.empty((1,), dtype=torch.int32, device=out_count.device)
    st = lib().spec_verify_count_invalid(_ptr(out_count), out_count.numel(), _ptr(out_invalid), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_count_invalid")
    return out_invalid


def spec_verify_host_sizes(B: int, K: int, V: int, *, target_dtype, draft_dtype, draft_kind):
    """(offsets of target, draft, tokens, temperature in the packed input, input bytes,
    output bytes) of spec_verify_chain_host's buffers; dtypes are torch dtypes."""
    off = (ctypes.c_size_t * 4)()
    nin, nout = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = lib().spec_verify_host_sizes(B, K, V, _dtype_code_of(target_dtype), _dtype_code_of(draft_dtype),
                                      _kind(draft_kind), ctypes.cast(off, ctypes.c_void_p), ctypes.byref(nin),
                                      ctypes.byref(nout))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_host_sizes")
    return tuple(off), nin.value, nout.value


def spec_verify_chain_host(h_in, d_in, h_out, d_out, B: int, K: int, V: int, seed: int, offset: int, *,
                           target_dtype, draft_dtype, draft_kind, workspace=None, stream=None):
    """One round from host memory: h_in (pinned uint8, the packed inputs of
    spec_verify_host_sizes) copied into d_in (uint8 CUDA), the chain verify, and the
    tokens [B][K+1] then counts [B] (int32) copied from d_out into h_out (pinned), all
    enqueued on the stream.  h_out holds them once the stream has passed this call."""
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
    st = lib().spec_verify_chain_host(h_in.data_ptr(), _ptr(d_in), h_out.data_ptr(), _ptr(d_out),
                                      _dtype_code_of(target_dtype), _dtype_code_of(draft_dtype), _kind(draft_kind),
                                      B, K, V, int(seed), int(offset), ws_ptr, ws_bytes, _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_chain_host")


def spec_verify_rows_status(out_count, *, out_status=None, stream=None):
    """Row-status summary of a finished verify call, computed on the device in stream
    order: an int32 device tensor [3] = (the call's sv_status -- SV_ERR_TIMEOUT if a row
    has count -1, else SV_ERR_BAD_INPUT if a row has count 0, else SV_OK --, the rows
    with count 0, the rows with count -1)."""
    torch = _torch()
    _dev(out_count, "out_count", torch.int32)
    if out_status is None:
        out_status = torch.empty((3,), dtype=torch.int32, device=out_count.device)
    st = lib().spec_verify_rows_status(_ptr(out_count), out_count.numel(), _ptr(out_status), _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_verify_rows_status")
    return out_status


def rows_status(out_count, *, stream=None) -> int:
    """The sv_status of a finished verify call's rows: SV_ERR_TIMEOUT if a bounded
    device-side wait gave up on some row (count -1), SV_ERR_BAD_INPUT if some row held
    invalid data (count 0), else SV_OK.  Reads three int32 back, so it waits for the
    stream."""
    s = spec_verify_rows_status(out_count, stream=stream)
    (_torch().cuda.current_stream() if stream is None else stream).synchronize()
    return int(s[0].cpu().item())


def spec_tree_mask(parent, *, out_mask=None, out_depth=None, out_valid=None, stream=None):
    """Ancestor-or-self attention mask of each draft tree.  parent int32 [B][N].
    Returns (out_mask int32 [B][N][ceil(N/32)] holding the uint32 bit words, out_depth
    int32 [B][N], out_valid int32 [B])."""
    torch = _torch()
    _dev(parent, "parent", torch.int32)
    B, N = parent.shape
    W = (N + 31) // 32
    dev = parent.device
    if out_mask is None:
        out_mask = torch.empty((B, N, W), dtype=torch.int32, device=dev)
    if out_depth is None:
        out_depth = torch.empty((B, N), dtype=torch.int32, device=dev)
    if out_valid is None:
        out_valid = torch.empty((B,), dtype=torch.int32, device=dev)
    st = lib().spec_tree_mask(_ptr(parent), B, N, _ptr(out_mask), _ptr(out_depth), _ptr(out_valid),
                              _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_tree_mask")
    return out_mask, out_depth, out_valid


def spec_kv_compact(kv_buffers, path, count, base=None, *, stream=None):
    """Move each batch row's accepted tree nodes' cache rows to the front, in place.
    kv_buffers: CUDA tensors of one dtype and identical shape [B][planes][rows][width]
    and strides (any strided view whose last dimension is contiguous, e.g. a
    [B][rows][heads][dim] cache permuted to [B][heads][rows][dim]).  path int32
    [B][D] and count int32 [B] as spec_verify_tree returns them; base int32 [B] (the
    cache row of tree node 0) or None for 0."""
    torch = _torch()
    bufs = list(kv_buffers)
    if not bufs:
        raise ValueError("kv_buffers is empty")
    t0 = bufs[0]
    for t in bufs:
        if not t.is_cuda or t.dim() != 4 or t.shape != t0.shape or t.stride() != t0.stride() or t.dtype != t0.dtype:
            raise ValueError("kv_buffers must be CUDA tensors [B][planes][rows][width] of one shape, stride and dtype")
        if t.stride(3) != 1:
            raise ValueError("the last dimension of every kv buffer must be contiguous")
    _dev(path, "path", torch.int32)
    _dev(count, "count", torch.int32)
    _dev(base, "base", torch.int32)
    B, H, R, Wd = t0.shape
    es = t0.element_size()
    arr = (ctypes.c_void_p * len(bufs))(*[t.data_ptr() for t in bufs])
    st = lib().spec_kv_compact(arr, len(bufs), t0.stride(0) * es, t0.stride(1) * es, H, t0.stride(2) * es,
                               Wd * es, R, _ptr(path), _ptr(count), _ptr(base), B, path.shape[1],
                               _stream(stream))
    if st != SV_OK:
        raise SpecVerifyError(st, "spec_kv_compact")


# --------------------------------------------- a verification round on a paged cache

def _one_device(first, stream, **tensors):
    """Checks that every given tensor is on the device of `first` (the first of them); returns
    that device's index, the handle of the stream to launch on (that device's current one
    unless given), and the stream itself where it is not the current one."""
    torch = _torch()
    at = first.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != at:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            raise ValueError(f"{name} is on {t.device}, other arguments on {first.device}")
    if at < 0:
        raise ValueError(f"{next(iter(tensors))} must be a CUDA tensor")
    current = torch._C._cuda_getCurrentRawStream(at)
    if stream is None:
        return at, current, None
    if stream.device_index != at:
        raise ValueError(f"the stream is on device {stream.device_index}, the arguments on {first.device}")
    handle = stream.cuda_stream
    return at, handle, None if handle == current else stream


def _shaped(name, t, shape, dtype):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _adr(t):
    return None if t is None else t.data_ptr()


def _launch(where, at, call, *args):
    """call(*args) with device `at` current; raises on a non-zero status."""
    torch = _torch()
    if at == torch._C._cuda_getDevice():
        st = call(*args)
    else:
        with torch.cuda.device(at):
            st = call(*args)
    if st != SV_OK:
        raise SpecVerifyError(st, where)


def _new(make, shape, dtype, at, side):
    """A new tensor (make: torch.empty or torch.zeros) that belongs to the launch's stream."""
    if side is None:
        return make(shape, dtype=dtype, device=at)
    with _torch().cuda.stream(side):
        return make(shape, dtype=dtype, device=at)


def _paged_cache(k_pages, v_pages, page_table, k_scale, v_scale, B):
    """The sv_paged_cache of tensors [pages][heads][page_size][head_dim] (checked)."""
    torch = _torch()
    shape, stride, dtype = k_pages.shape, k_pages.stride(), k_pages.dtype
    if len(shape) != 4:
        raise ValueError("k_pages and v_pages must be [pages][heads][page_size][head_dim]")
    if v_pages.shape != shape or v_pages.dtype != dtype or v_pages.stride() != stride:
        raise ValueError("k_pages and v_pages must have one shape, stride and dtype")
    P, H, ps, D = shape
    sp, sh, sr, sd = stride
    if sd != 1 and D > 1:
        raise ValueError("the last dimension of k_pages and v_pages must be contiguous")
    if dtype == torch.bfloat16:
        code, es = SV_CACHE_BF16, 2
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale belong to float8_e4m3fn pages")
    elif dtype == torch.float8_e4m3fn:
        code, es = SV_CACHE_E4M3, 1
        if k_scale is None or v_scale is None:
            raise ValueError("float8_e4m3fn pages need k_scale and v_scale")
        _shaped("k_scale", k_scale, (P, H, ps), torch.float32)
        _shaped("v_scale", v_scale, (P, H, ps), torch.float32)
    else:
        raise TypeError(f"pages must be bfloat16 or float8_e4m3fn, got {dtype}")
    table = page_table.shape
    if len(table) != 2 or table[0] != B:
        raise ValueError(f"page_table must be [{B}][max_pages], got {tuple(table)}")
    _shaped("page_table", page_table, table, torch.int32)
    return PagedCache(k_pages.data_ptr(), v_pages.data_ptr(), _adr(k_scale), _adr(v_scale), page_table.data_ptr(),
                      sp * es, sh * es, max(sr, D) * es if ps == 1 else sr * es, code, P, ps, table[1], H, D)


def _strides3(t, name):
    """Element strides of the first three dimensions of [B][N][heads][head_dim]."""
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


def _src_code(dtype, name) -> int:
    torch = _torch()
    if dtype == torch.bfloat16:
        return SV_BF16
    if dtype == torch.float32:
        return SV_F32
    raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")


def spec_kv_append(key, value, k_pages, v_pages, page_table, base, *, new_len=None, k_scale=None, v_scale=None,
                   stream=None):
    """Write new tokens' keys and values into a paged cache, in place.  key, value
    [B][N][heads][head_dim] (fp32/bf16, any strides with contiguous elements, one shape,
    stride and dtype); k_pages, v_pages [pages][heads][page_size][head_dim] bf16, or
    float8_e4m3fn with k_scale, v_scale fp32 [pages][heads][page_size] (any strides with
    contiguous elements: a [pages][page_size][heads][head_dim] cache is passed permuted);
    page_table int32 [B][max_pages]; base int32 [B] (positions before token 0); new_len
    int32 [B] or None (all N tokens are real)."""
    torch = _torch()
    at, handle, side = _one_device(key, stream, key=key, value=value, k_pages=k_pages, v_pages=v_pages,
                              page_table=page_table, base=base, new_len=new_len, k_scale=k_scale, v_scale=v_scale)
    if key.dim() != 4 or key.shape != value.shape or key.dtype != value.dtype or key.stride() != value.stride():
        raise ValueError("key and value must be [B][N][heads][head_dim] of one shape, stride and dtype")
    B, N, H, D = key.shape
    cache = _paged_cache(k_pages, v_pages, page_table, k_scale, v_scale, B)
    if (cache.num_heads, cache.head_dim) != (H, D):
        raise ValueError(f"key has {H} heads of {D}, the cache {cache.num_heads} of {cache.head_dim}")
    _shaped("base", base, (B,), torch.int32)
    _shaped("new_len", new_len, (B,), torch.int32)
    _launch("spec_kv_append", at, lib().spec_kv_append, _adr(key), _adr(value), _src_code(key.dtype, "key"),
            _strides3(key, "key"), cache, _adr(base), _adr(new_len), B, N, handle)


def spec_kv_read(k_pages, v_pages, page_table, base, num_tokens: int, *, new_len=None, k_scale=None, v_scale=None,
                 out_key=None, out_value=None, dtype=None, stream=None):
    """Read positions base[b] .. base[b] + new_len[b] - 1 (new_len None: num_tokens for every
    row) of a paged cache into dense arrays [B][num_tokens][heads][head_dim] of dtype
    (bf16 unless given; that of out_key where that is given).  Arguments as
    spec_kv_append.  Rows of new outputs at and behind new_len are zero; rows of given
    outputs there keep what they hold.  Returns (out_key, out_value)."""
    torch = _torch()
    at, handle, side = _one_device(k_pages, stream, k_pages=k_pages, v_pages=v_pages, page_table=page_table, base=base,
                              new_len=new_len, k_scale=k_scale, v_scale=v_scale, out_key=out_key,
                              out_value=out_value)
    B, N = page_table.shape[0], int(num_tokens)
    cache = _paged_cache(k_pages, v_pages, page_table, k_scale, v_scale, B)
    shape = (B, N, cache.num_heads, cache.head_dim)
    given = out_key if out_key is not None else out_value
    if dtype is None:
        dtype = given.dtype if given is not None else torch.bfloat16
    code = _src_code(dtype, "dtype")
    if N < 0:
        raise ValueError("num_tokens must not be negative")
    _shaped("base", base, (B,), torch.int32)
    _shaped("new_len", new_len, (B,), torch.int32)
    _shaped("out_key", out_key, shape, dtype)
    _shaped("out_value", out_value, shape, dtype)
    if out_key is None or out_value is None:
        out_key = _new(torch.zeros, shape, dtype, at, side) if out_key is None else out_key
        out_value = _new(torch.zeros, shape, dtype, at, side) if out_value is None else out_value
    _launch("spec_kv_read", at, lib().spec_kv_read, cache, _adr(base), _adr(new_len), B, N, _adr(out_key),
            _adr(out_value), code, handle)
    return out_key, out_value


def spec_kv_compact_paged(kv_buffers, page_table, path, count, base=None, *, stream=None):
    """spec_kv_compact on a paged cache, in place: every batch row's accepted tree nodes'
    cache rows move to base[b], base[b] + 1, ... through the page table.  kv_buffers: CUDA
    tensors [pages][planes][page_size][width] of one dtype, shape and stride with a
    contiguous last dimension (each layer's K and V pages; their e4m3 scales in a call of
    their own, as [pages][planes][page_size][1] views), or one tensor
    [buffers][pages][planes][page_size][width].  page_table int32 [B][max_pages]; path,
    count, base as spec_kv_compact."""
    torch = _torch()
    if isinstance(kv_buffers, torch.Tensor):
        if kv_buffers.dim() != 5 or not kv_buffers.shape[0]:
            raise ValueError("a single kv_buffers tensor must be [buffers][pages][planes][page_size][width]")
        n, shape, strides, t0 = kv_buffers.shape[0], kv_buffers.shape[1:], kv_buffers.stride()[1:], kv_buffers
        es = t0.element_size()
        origin, step = t0.data_ptr(), kv_buffers.stride(0) * es
        ptrs = range(origin, origin + n * step, step) if step else [origin] * n
    else:
        bufs = list(kv_buffers)
        if not bufs:
            raise ValueError("kv_buffers is empty")
        t0 = bufs[0]
        n, shape, strides, dtype, where = len(bufs), t0.shape, t0.stride(), t0.dtype, t0.get_device()
        if len(shape) != 4:
            raise ValueError("kv_buffers must be tensors [pages][planes][page_size][width]")
        for t in bufs:
            if t.shape != shape or t.stride() != strides or t.dtype != dtype or t.get_device() != where:
                raise ValueError("kv_buffers must be tensors [pages][planes][page_size][width] of one shape, stride, "
                                 "dtype and device")
        es = t0.element_size()
        ptrs = [t.data_ptr() for t in bufs]
    if len(set(ptrs)) != n:
        raise ValueError("kv_buffers names a buffer twice: its rows would move twice")
    at, handle, side = _one_device(t0, stream, kv_buffers=t0, page_table=page_table, path=path, count=count, base=base)
    P, H, ps, W = shape
    if strides[3] != 1 and W > 1:
        raise ValueError("the last dimension of every kv buffer must be contiguous")
    if path.dim() != 2 or page_table.dim() != 2 or page_table.shape[0] != path.shape[0]:
        raise ValueError("path must be [B][max_depth] and page_table [B][max_pages]")
    B = path.shape[0]
    _shaped("page_table", page_table, page_table.shape, torch.int32)
    _shaped("path", path, path.shape, torch.int32)
    _shaped("count", count, (B,), torch.int32)
    _shaped("base", base, (B,), torch.int32)
    row = max(strides[2], W) if ps == 1 else strides[2]
    _launch("spec_kv_compact_paged", at, lib().spec_kv_compact_paged, (ctypes.c_void_p * n)(*ptrs), n,
            strides[0] * es, strides[1] * es, H, row * es, W * es, _adr(page_table), P, ps, page_table.shape[1],
            _adr(path), _adr(count), _adr(base), B, path.shape[1], handle)


def spec_paged_attention_workspace_size(B: int, Q: int, num_q_heads: int, num_heads: int, head_dim: int, cache_dtype,
                                        max_len: int) -> int:
    """Bytes of scratch spec_paged_attention uses for such a call on the current device;
    cache_dtype is the pages' torch dtype."""
    torch = _torch()
    if cache_dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError(f"pages must be bfloat16 or float8_e4m3fn, got {cache_dtype}")
    code = SV_CACHE_BF16 if cache_dtype == torch.bfloat16 else SV_CACHE_E4M3
    return int(lib().spec_paged_attention_workspace_size(B, Q, num_q_heads, num_heads, head_dim, code, max_len))


_attention_needs = {}


def _attention_need(at, *sizes):
    """spec_paged_attention_workspace_size(*sizes) on a device, remembered by the sizes."""
    key = (at, *sizes)
    need = _attention_needs.get(key)
    if need is None:
        with _torch().cuda.device(at):
            need = int(lib().spec_paged_attention_workspace_size(*sizes))
        if len(_attention_needs) >= 4096:  # context lengths vary: keep the table small
            _attention_needs.clear()
        _attention_needs[key] = need
    return need


def spec_paged_attention(q, k_pages, v_pages, page_table, base, *, max_len=None, new_len=None, tree_mask=None,
                         scale=None, k_scale=None, v_scale=None, out=None, out_lse=None, want_lse: bool = False,
                         workspace="auto", stream=None):
    """Attention of a chunk of new tokens over a paged cache that already holds their keys
    and values (spec_kv_append).  q bf16 [B][Q][q_heads][head_dim] (any strides with
    contiguous elements, multiples of 8); pages, scales, page_table, base and new_len as
    spec_kv_append.  Query i sees the base[b] positions before the chunk and, of the chunk,
    tokens 0..i; with tree_mask (int32 [B][Q-1][ceil((Q-1)/32)] from spec_tree_mask: token 0
    is the root, token i + 1 node i) the root, itself and its ancestors.  max_len: a bound
    on base + new_len that the caller knows (the page table's capacity unless given);
    scale: 1 / sqrt(head_dim) unless given.  workspace: "auto" (allocated for the call), a
    uint8 CUDA tensor, or None (long contexts are not split).
    Returns (out bf16 [B][Q][q_heads][head_dim], lse fp32 [B][Q][q_heads] or None)."""
    torch = _torch()
    auto = isinstance(workspace, str)
    at, handle, side = _one_device(q, stream, q=q, k_pages=k_pages, v_pages=v_pages, page_table=page_table, base=base,
                              new_len=new_len, tree_mask=tree_mask, k_scale=k_scale, v_scale=v_scale, out=out,
                              out_lse=out_lse, workspace=None if auto else workspace)
    if q.dim() != 4 or q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16 [B][Q][q_heads][head_dim]")
    B, Q, Hq, D = q.shape
    cache = _paged_cache(k_pages, v_pages, page_table, k_scale, v_scale, B)
    if cache.head_dim != D or Hq % cache.num_heads:
        raise ValueError(f"q has {Hq} heads of {D}, the cache {cache.num_heads} of {cache.head_dim}")
    if Q < 1:
        raise ValueError("q holds no query")
    _shaped("base", base, (B,), torch.int32)
    _shaped("new_len", new_len, (B,), torch.int32)
    _shaped("tree_mask", tree_mask, (B, Q - 1, (Q + 30) // 32), torch.int32)
    _shaped("out", out, (B, Q, Hq, D), torch.bfloat16)
    _shaped("out_lse", out_lse, (B, Q, Hq), torch.float32)
    if max_len is None:
        max_len = cache.max_pages * cache.page_size
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = _new(torch.empty, (B, Q, Hq, D), torch.bfloat16, at, side)
    if out_lse is None and want_lse:
        out_lse = _new(torch.empty, (B, Q, Hq), torch.float32, at, side)
    if auto:
        need = _attention_need(at, B, Q, Hq, cache.num_heads, D, cache.dtype, max_len) if B else 0
        workspace = _new(torch.empty, (need,), torch.uint8, at, side) if need else None
    elif workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch("spec_paged_attention", at, lib().spec_paged_attention, _adr(q), _strides3(q, "q"), Hq, cache,
            _adr(base), _adr(new_len), _adr(tree_mask), scale, B, Q, max_len, _adr(out), _adr(out_lse),
            _adr(workspace), ws_bytes, handle)
    return out, out_lse


def spec_adjust_logits(logits, *, history=None, history_len=None, prompt_len=None, draft_tokens=None, tree_mask=None,
                       repetition=None, presence=None, frequency=None, bias_tokens=None, bias_values=None,
                       allowed=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on the logits [B][R][V]
    (fp32/bf16) of a verify call, R = K + 1 rows of a chain or N + 1 of a tree.  history
    int32 [B][H] (history_len int32 [B], all H unless given; tokens before prompt_len int32
    [B] are the prompt); draft_tokens int32 [B][R-1], which row r has as output so far where
    they precede it in the chain, or with tree_mask (int32 [B][R-1][ceil((R-1)/32)] from
    spec_tree_mask) where they are node r-1 or its ancestors; repetition, presence,
    frequency fp32 [B]; bias_tokens int32 and bias_values fp32 [B][M]; allowed int32
    [B][R][ceil(V/32)], bit v % 32 of word v / 32 set where token v is allowed.  Any of them
    may be None.  Returns out (a new tensor unless given; logits itself works in place)."""
    torch = _torch()
    at, handle, side = _one_device(logits, stream, logits=logits, history=history, history_len=history_len,
                              prompt_len=prompt_len, draft_tokens=draft_tokens, tree_mask=tree_mask,
                              repetition=repetition, presence=presence, frequency=frequency, bias_tokens=bias_tokens,
                              bias_values=bias_values, allowed=allowed, out=out)
    if logits.dim() != 3 or not logits.is_contiguous():
        raise ValueError("logits must be contiguous [B][R][V]")
    code = _dtype_code(logits)
    B, R, V = logits.shape
    i32, f32 = torch.int32, torch.float32
    H = M = 0
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history must be [B][H]")
        H = history.shape[1]
        _shaped("history", history, (B, H), i32)
        if history_len is None:
            history_len = _new(lambda size, **kw: torch.full(size, H, **kw), (B,), i32, at, side)
    elif history_len is not None or prompt_len is not None:
        raise ValueError("history_len and prompt_len belong to a history")
    _shaped("history_len", history_len, (B,), i32)
    _shaped("prompt_len", prompt_len, (B,), i32)
    _shaped("draft_tokens", draft_tokens, (B, R - 1), i32)
    if tree_mask is not None and draft_tokens is None:
        raise ValueError("tree_mask belongs to draft_tokens")
    _shaped("tree_mask", tree_mask, (B, R - 1, (R + 30) // 32), i32)
    _shaped("repetition", repetition, (B,), f32)
    _shaped("presence", presence, (B,), f32)
    _shaped("frequency", frequency, (B,), f32)
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values belong together")
    if bias_tokens is not None:
        if bias_tokens.dim() != 2:
            raise ValueError("bias_tokens must be [B][M]")
        M = bias_tokens.shape[1]
        _shaped("bias_tokens", bias_tokens, (B, M), i32)
        _shaped("bias_values", bias_values, (B, M), f32)
    _shaped("allowed", allowed, (B, R, (V + 31) // 32), i32)
    _shaped("out", out, (B, R, V), logits.dtype)
    if out is None:
        out = _new(torch.empty, (B, R, V), logits.dtype, at, side)
    _launch("spec_adjust_logits", at, lib().spec_adjust_logits, _adr(logits), code, _adr(history),
            _adr(history_len), _adr(prompt_len), H, _adr(draft_tokens), _adr(tree_mask), _adr(repetition),
            _adr(presence), _adr(frequency), _adr(bias_tokens), _adr(bias_values), M, _adr(allowed), B, R, V,
            _adr(out), handle)
    return out
