"""Thin ctypes binding of libdn.so (include/dn.h) for torch tensors.

Argument marshalling only: shapes, dtypes and devices are checked, raw device
pointers and the current CUDA stream are passed to the C ABI, and a non-OK
status raises ``DnError``. Every step of the computation runs in the library's
CUDA kernels; there is no other implementation to fall back to, so a missing
library raises at load time.
"""

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdn.so")

DN_OK, DN_ERR_INVALID_ARG, DN_ERR_UNSUPPORTED, DN_ERR_CUDA = 0, 1, 2, 3
DN_F16, DN_F32, DN_BF16, DN_E4M3 = 0, 1, 2, 3
MAX_BLOCK = 16
PREFILL_CHUNK = 64

_DT = {torch.float16: DN_F16, torch.float32: DN_F32}
# types of the paged cache and of the tensors that go with it
_KV_DT = {torch.float16: DN_F16, torch.float32: DN_F32, torch.bfloat16: DN_BF16, torch.float8_e4m3fn: DN_E4M3}

# Every exported symbol of include/dn.h with its ctypes signature.
_P, _I, _S, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
SIGNATURES = {
    "dn_verify_block": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "dn_accept_workspace_bytes": (_S, [_I, _I, _I]),
    "dn_accept_greedy": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P]),
    "dn_commit": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "dn_prefill_checkpoint": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                   _P, _P, _P]),
    "dn_prefill_checkpoint_tc": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                      _P, _P, _P]),
    "dn_status_string": (ctypes.c_char_p, [_I]),
    "dn_accept_greedy_noalloc": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "dn_prefill_wait_timeouts": (ctypes.c_uint, []),
    "dn_wait_selftest": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "dn_verify_block_deltas": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "dn_commit_deltas": (_I, [_I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "dn_prefix_cache_create": (_P, [_I, _I]),
    "dn_prefix_cache_destroy": (None, [_P]),
    "dn_prefix_cache_insert": (_I, [_P, _P, _I, ctypes.c_int32, _P]),
    "dn_prefix_cache_lookup": (_I, [_P, _P, _I, _P, _P]),
    "dn_prefix_cache_size": (_I, [_P]),
    "dn_kv_append": (_I, [_I] * 9 + [_P, _P, _L, _L] + [_P] * 8),
    "dn_kv_gather": (_I, [_I] * 9 + [_P] * 10),
    "dn_attn_workspace_bytes": (_S, [_I] * 5),
    "dn_attn_paged": (_I, [_I] * 10 + [_P, _L] + [_P] * 7 + [ctypes.c_float, _I, _P, _P, _P, _S, _P]),
    "dn_attn_wait_timeouts": (ctypes.c_uint, []),
    "dn_sample_workspace_bytes": (_S, [_I] * 3),
    "dn_accept_sampled": (_I, [_I] * 4 + [_P] * 11 + [_S, _P]),
    "dn_rope_append": (_I, [_I] * 12 + [_P, _L] * 3 + [_P, _P, ctypes.c_float, _P, _P, ctypes.c_float] + [_P] * 9),
    "dn_head_norm": (_I, [_I] * 6 + [_P, _L, _P, _L, _P, ctypes.c_float, _P, _P]),
    "dn_residual_norm": (_I, [_I] * 5 + [_P, _L, _P, _L, _P, ctypes.c_float, _P, _P, _P, ctypes.c_float, _P, _P]),
    "dn_context_drafts": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
}


class DnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = load_library().dn_status_string(status).decode()
        super().__init__("%s failed: %s" % (fn, msg))


_lib = None


def load_library(path=None):
    """Load libdn.so (once) and declare the C signatures. Raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            "libdn.so is not built (%s); build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'`" % p)
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _stream(stream):
    if stream is None:
        # the handle that torch.cuda.current_stream().cuda_stream gives, without the Stream object (3 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _other(stream):
    """The torch stream of `stream` if it is not the current one, else None."""
    if stream is None or _stream(stream) == _stream(None):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _new(other, make, kept=True):
    """A tensor that a call makes for itself, from make(). The allocator hands memory out again in the order of the
    stream it was made on, so that has to be the launch's stream; `kept` ones go to the caller, whose work on
    the current stream the allocator then waits for too.
    """
    if other is None:
        return make()
    with torch.cuda.stream(other):
        t = make()
    if kept and t.is_cuda:
        t.record_stream(torch.cuda.current_stream())
    return t


def _check(name, status):
    if status != DN_OK:
        raise DnError(name, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(cond, what):
    """Argument check that survives python -O: the C ABI receives raw pointers and cannot
    see a tensor's size, so a wrong shape must stop here."""
    if not cond:
        raise ValueError(what)


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("all tensors must be CUDA tensors")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")


def dn_verify_block(q, k, v, beta, g, state_in, out=None, ckpt=None, stream=None):
    """q, k [N,T,H,dk]; v [N,T,H,dv]; beta, g [N,T,H] fp32; state_in [N,H,dv,dk].

    Returns (out [N,T,H,dv], ckpt [N,T,H,dv,dk]); allocates them with torch if not given.
    """
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    other = _other(stream)
    if out is None:
        out = _new(other, lambda: torch.empty((N, T, H, dv), dtype=q.dtype, device=q.device))
    if ckpt is None:
        ckpt = _new(other, lambda: torch.empty((N, T, H, dv, dk), dtype=state_in.dtype, device=q.device))
    _dev(q, k, v, beta, g, state_in, out, ckpt)
    _require(k.shape == q.shape and v.shape == (N, T, H, dv), "k like q, v [N,T,H,dv]")
    _require(beta.shape == (N, T, H) and g.shape == (N, T, H), "beta, g [N,T,H]")
    _require(beta.dtype == torch.float32 and g.dtype == torch.float32, "beta, g fp32")
    _require(state_in.shape == (N, H, dv, dk) and ckpt.shape == (N, T, H, dv, dk),
             "state_in [N,H,dv,dk], ckpt [N,T,H,dv,dk]")
    _require(out.shape == (N, T, H, dv) and out.dtype == q.dtype and ckpt.dtype == state_in.dtype,
             "out [N,T,H,dv] in q's dtype, ckpt in the state's")
    st = load_library().dn_verify_block(
        N, H, T, dk, dv, _DT[q.dtype], _DT[state_in.dtype], _ptr(q), _ptr(k), _ptr(v),
        _ptr(beta), _ptr(g), _ptr(state_in), _ptr(out), _ptr(ckpt), _stream(stream))
    _check("dn_verify_block", st)
    return out, ckpt


def dn_verify_block_deltas(q, k, v, beta, g, state_in, out=None, delta=None, stream=None):
    """As dn_verify_block, but writes delta [N,T,H,dv] fp32 instead of checkpoints."""
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    other = _other(stream)
    if out is None:
        out = _new(other, lambda: torch.empty((N, T, H, dv), dtype=q.dtype, device=q.device))
    if delta is None:
        delta = _new(other, lambda: torch.empty((N, T, H, dv), dtype=torch.float32, device=q.device))
    _dev(q, k, v, beta, g, state_in, out, delta)
    _require(k.shape == q.shape and v.shape == (N, T, H, dv) and state_in.shape == (N, H, dv, dk),
             "k like q, v [N,T,H,dv], state_in [N,H,dv,dk]")
    _require(delta.shape == (N, T, H, dv) and delta.dtype == torch.float32, "delta [N,T,H,dv] fp32")
    st = load_library().dn_verify_block_deltas(
        N, H, T, dk, dv, _DT[q.dtype], _DT[state_in.dtype], _ptr(q), _ptr(k), _ptr(v),
        _ptr(beta), _ptr(g), _ptr(state_in), _ptr(out), _ptr(delta), _stream(stream))
    _check("dn_verify_block_deltas", st)
    return out, delta


def dn_commit_deltas(k, g, delta, accepted_len, state, stream=None):
    """Rebuild the accepted state in place from delta [N,T,H,dv], k [N,T,H,dk], g [N,T,H]."""
    N, H, dv, dk = state.shape
    T = k.shape[1]
    B = accepted_len.shape[0]
    _dev(k, g, delta, accepted_len, state)
    _require(k.shape == (N, T, H, dk) and g.shape == (N, T, H) and delta.shape == (N, T, H, dv),
             "k [N,T,H,dk], g [N,T,H], delta [N,T,H,dv]")
    st = load_library().dn_commit_deltas(N, B, H, T, dk, dv, _DT[state.dtype], _ptr(k), _ptr(g),
                                         _ptr(delta), _ptr(accepted_len), _ptr(state),
                                         _stream(stream))
    _check("dn_commit_deltas", st)
    return state


def dn_accept_workspace_bytes(B, T, V):
    return int(load_library().dn_accept_workspace_bytes(B, T, V))


def accept_workspace(B, T, V, device):
    """A zeroed workspace of dn_accept_workspace_bytes(B, T, V) bytes."""
    n = dn_accept_workspace_bytes(B, T, V)
    return torch.zeros((max(n, 16),), dtype=torch.uint8, device=device)


def dn_accept_greedy(logits, draft_ids, target_ids=None, accepted_len=None, workspace=None,
                     stream=None):
    """logits [B,T,V] fp16/fp32, draft_ids [B,T] int32 -> (target_ids [B,T], accepted_len [B])."""
    B, T, V = logits.shape
    dev = logits.device
    other = _other(stream)
    if target_ids is None:
        target_ids = _new(other, lambda: torch.empty((B, T), dtype=torch.int32, device=dev))
    if accepted_len is None:
        accepted_len = _new(other, lambda: torch.empty((B,), dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = _new(other, lambda: accept_workspace(B, T, V, dev), kept=False)
    _dev(logits, draft_ids, target_ids, accepted_len, workspace)
    _require(draft_ids.shape == (B, T) and draft_ids.dtype == torch.int32, "draft_ids [B,T] int32")
    _require(target_ids.shape == (B, T) and accepted_len.shape == (B,), "target_ids [B,T], accepted_len [B]")
    st = load_library().dn_accept_greedy(
        B, T, V, _DT[logits.dtype], _ptr(logits), _ptr(draft_ids), _ptr(target_ids),
        _ptr(accepted_len), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check("dn_accept_greedy", st)
    return target_ids, accepted_len


def dn_accept_greedy_noalloc(logits, draft_ids, target_ids, accepted_len, stream=None):
    """dn_accept_greedy with its scratch in the library's fixed device array (no workspace).

    For callers that cannot allocate device memory where they verify; the outputs must
    be passed in. Calls that overlap on one GPU race on the shared array.
    """
    B, T, V = logits.shape
    _dev(logits, draft_ids, target_ids, accepted_len)
    _require(draft_ids.shape == (B, T) and draft_ids.dtype == torch.int32, "draft_ids [B,T] int32")
    _require(target_ids.shape == (B, T) and target_ids.dtype == torch.int32, "target_ids [B,T] int32")
    _require(accepted_len.shape == (B,) and accepted_len.dtype == torch.int32, "accepted_len [B] int32")
    st = load_library().dn_accept_greedy_noalloc(
        B, T, V, _DT[logits.dtype], _ptr(logits), _ptr(draft_ids), _ptr(target_ids),
        _ptr(accepted_len), _stream(stream))
    _check("dn_accept_greedy_noalloc", st)
    return target_ids, accepted_len


def dn_commit(ckpt, accepted_len, state, stream=None):
    """ckpt [N,T,H,dv,dk], accepted_len [B] int32 (device), state [N,H,dv,dk] updated in place."""
    N, H, dv, dk = state.shape
    T = ckpt.shape[1]
    B = accepted_len.shape[0]
    _dev(ckpt, accepted_len, state)
    _require(ckpt.shape == (N, T, H, dv, dk) and ckpt.dtype == state.dtype, "ckpt [N,T,H,dv,dk] in the state's dtype")
    _require(accepted_len.dtype == torch.int32, "accepted_len int32")
    st = load_library().dn_commit(N, B, H, T, dk, dv, _DT[state.dtype], _ptr(ckpt),
                                  _ptr(accepted_len), _ptr(state), _stream(stream))
    _check("dn_commit", st)
    return state


def dn_prefill_checkpoint(q, k, v, beta, g, state_in=None, out=None, ckpt=None, state_out=None,
                          chunk=PREFILL_CHUNK, state_dtype=None, stream=None, engine="mma"):
    """q, k [N,P,H,dk]; v [N,P,H,dv]; beta, g [N,P,H]; state_in [N,H,dv,dk] or None.

    Returns (out [N,P,H,dv], ckpt [N,P//chunk,H,dv,dk], state_out [N,H,dv,dk]).
    engine "mma" calls dn_prefill_checkpoint, "tc" dn_prefill_checkpoint_tc (fp16, 128 x 128).
    """
    N, P, H, dk = q.shape
    dv = v.shape[-1]
    sdt = state_in.dtype if state_in is not None else (state_dtype or q.dtype)
    dev = q.device
    other = _other(stream)
    if out is None:
        out = _new(other, lambda: torch.empty((N, P, H, dv), dtype=q.dtype, device=dev))
    if ckpt is None:
        ckpt = _new(other, lambda: torch.empty((N, P // chunk, H, dv, dk), dtype=sdt, device=dev))
    if state_out is None:
        state_out = _new(other, lambda: torch.empty((N, H, dv, dk), dtype=sdt, device=dev))
    _dev(q, k, v, beta, g, state_in, out, ckpt, state_out)
    _require(k.shape == q.shape and v.shape == (N, P, H, dv) and beta.shape == (N, P, H),
             "k like q, v [N,P,H,dv], beta [N,P,H]")
    _require(g.shape == (N, P, H) and out.shape == (N, P, H, dv), "g [N,P,H], out [N,P,H,dv]")
    _require(beta.dtype == torch.float32 and g.dtype == torch.float32, "beta and g are fp32")
    _require(ckpt.shape == (N, P // chunk, H, dv, dk) and state_out.shape == (N, H, dv, dk),
             "ckpt [N,P/chunk,H,dv,dk], state_out [N,H,dv,dk]")
    name = {"mma": "dn_prefill_checkpoint", "tc": "dn_prefill_checkpoint_tc"}[engine]
    st = getattr(load_library(), name)(
        N, H, P, chunk, dk, dv, _DT[q.dtype], _DT[sdt], _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
        _ptr(g), _ptr(state_in), _ptr(out), _ptr(ckpt) if ckpt.numel() else None,
        _ptr(state_out), _stream(stream))
    _check(name, st)
    return out, ckpt, state_out


def dn_prefill_wait_timeouts():
    return int(load_library().dn_prefill_wait_timeouts())


def dn_wait_selftest(budget_us, device=None, stream=None):
    """Runs the bounded-wait self-test; returns (gave_up, returned, drained, failures_counted)."""
    result = torch.tensor([11, 22, 33, 44], dtype=torch.int32, device=device or "cuda")
    _check("dn_wait_selftest", load_library().dn_wait_selftest(int(budget_us), result.data_ptr(), _stream(stream)))
    torch.cuda.synchronize(result.device)
    return tuple(int(x) for x in result.cpu())


def dn_context_drafts(context, lengths, n_max=4, n_min=1, K=8, drafts=None, count=None,
                      match_len=None, stream=None):
    """Drafts copied from each request's context: context [N, stride] int32, lengths [N] int32.

    Returns (drafts [N, K] int32 padded with -1, count [N] int32, match_len [N] int32).
    """
    N, stride = context.shape
    dev = context.device
    other = _other(stream)
    if drafts is None:
        drafts = _new(other, lambda: torch.empty((N, K), dtype=torch.int32, device=dev))
    if count is None:
        count = _new(other, lambda: torch.empty((N,), dtype=torch.int32, device=dev))
    if match_len is None:
        match_len = _new(other, lambda: torch.empty((N,), dtype=torch.int32, device=dev))
    _dev(context, lengths, drafts, count, match_len)
    _require(context.dtype == lengths.dtype == drafts.dtype == count.dtype == torch.int32,
             "context, lengths, drafts, count int32")
    _require(lengths.shape == (N,) and drafts.shape == (N, K) and count.shape == (N,),
             "lengths [N], drafts [N,K], count [N]")
    st = load_library().dn_context_drafts(N, stride, n_max, n_min, K, _ptr(context), _ptr(lengths),
                                          _ptr(drafts), _ptr(count), _ptr(match_len),
                                          _stream(stream))
    _check("dn_context_drafts", st)
    return drafts, count, match_len


_I32, _U8, _F32, _E4M3 = torch.int32, torch.uint8, torch.float32, torch.float8_e4m3fn


def _kv_pool(start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp):
    """Checks the paged cache's tensors; returns (B, heads, D, page, max_pages, pages, cache dtype).

    One expression for the good case (these checks are a good part of a small call's time); what is
    wrong is looked for only if something is.
    """
    shape, dt = k_cache.shape, k_cache.dtype
    table = page_table.shape
    if (len(shape) == 4 and len(table) == 2 and v_cache.shape == shape and v_cache.dtype is dt
            and start.shape == (table[0] + 1,) and kv_len.shape == (table[0],)
            and start.dtype is _I32 and kv_len.dtype is _I32 and page_table.dtype is _I32
            and start.is_cuda and kv_len.is_cuda and page_table.is_cuda and k_cache.is_cuda and v_cache.is_cuda
            and start.is_contiguous() and kv_len.is_contiguous() and page_table.is_contiguous()
            and k_cache.is_contiguous() and v_cache.is_contiguous()
            and (k_exp is None and v_exp is None and dt in _KV_DT if dt is not _E4M3 else
                 k_exp is not None and v_exp is not None and k_exp.dtype is _U8 and v_exp.dtype is _U8
                 and k_exp.shape == shape[:3] and v_exp.shape == shape[:3] and k_exp.is_cuda and v_exp.is_cuda
                 and k_exp.is_contiguous() and v_exp.is_contiguous())):
        return table[0], shape[1], shape[3], shape[2], table[1], shape[0], _KV_DT[dt]
    _require(len(shape) == 4 and v_cache.shape == shape and v_cache.dtype == dt,
             "k_cache, v_cache [pages,heads,page,D] of one dtype")
    _dev(start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp)
    _require(start.dtype == kv_len.dtype == page_table.dtype == torch.int32, "start, kv_len, page_table int32")
    _require(dt in _KV_DT, "k_cache, v_cache fp16, bf16 or float8_e4m3fn")
    _require(dt == _E4M3 or (k_exp is None and v_exp is None), "k_exp, v_exp go with an e4m3 cache")
    _require(dt != _E4M3 or (k_exp is not None and v_exp is not None and k_exp.dtype == v_exp.dtype == torch.uint8
                             and k_exp.shape == v_exp.shape == shape[:3]),
             "an e4m3 cache has k_exp, v_exp [pages,heads,page] uint8")
    raise ValueError("start [B+1], kv_len [B], page_table [B,max_pages]")


def _rows(t, heads, D, name):
    """Checks packed rows [total, heads, D], dense inside a row; returns (total, row stride in elements, dtype)."""
    shape, dt = t.shape, t.dtype
    if len(shape) == 3 and shape[1] == heads and shape[2] == D and t.is_cuda and dt in _KV_DT:
        if t.is_contiguous():
            return shape[0], heads * D, _KV_DT[dt]
        if t.stride(2) == 1 and (heads == 1 or t.stride(1) == D):
            return shape[0], t.stride(0) if shape[0] > 1 else heads * D, _KV_DT[dt]
    _require(t.is_cuda, "all tensors must be CUDA tensors")
    _require(len(shape) == 3 and shape[1] == heads and shape[2] == D, "%s [total,heads,D]" % name)
    _require(dt in _KV_DT, "%s fp16 or bf16" % name)
    raise ValueError("%s dense inside a row" % name)


def dn_kv_append(k, v, start, kv_len, page_table, k_cache, v_cache, k_exp=None, v_exp=None, stream=None):
    """Write packed rows k, v [total,heads,D] (the newest tokens) to their places in the paged cache.

    start [B+1], kv_len [B] (the newest included), page_table [B,max_pages] int32; k_cache, v_cache
    [pages,heads,page,D] in k's dtype, or float8_e4m3fn with k_exp, v_exp [pages,heads,page] uint8.
    k and v may be slices of a wider projection (rows dense inside). Returns (k_cache, v_cache).
    """
    B, heads, D, page, max_pages, pages, cdt = _kv_pool(start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp)
    total, ks, dt = _rows(k, heads, D, "k")
    total_v, vs, dt_v = _rows(v, heads, D, "v")
    if total_v != total or dt_v != dt:
        raise ValueError("v like k")
    st = (_lib or load_library()).dn_kv_append(
        B, total, heads, D, page, max_pages, pages, dt, cdt, k.data_ptr(), v.data_ptr(), ks, vs,
        start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_exp),
        _ptr(v_exp), _stream(stream))
    if st:
        _check("dn_kv_append", st)
    return k_cache, v_cache


def dn_kv_gather(start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp, k, v, stream=None):
    """Read the newest tokens' keys and values back into packed rows k, v [total,heads,D] (dense).

    The cache's tensors as for dn_kv_append (k_exp, v_exp None unless it is e4m3). Returns (k, v).
    """
    B, heads, D, page, max_pages, pages, cdt = _kv_pool(start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp)
    total, _, dt = _rows(k, heads, D, "k")
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("v like k")
    _dev(k, v)
    st = (_lib or load_library()).dn_kv_gather(
        B, total, heads, D, page, max_pages, pages, dt, cdt, start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_exp), _ptr(v_exp), k.data_ptr(), v.data_ptr(), _stream(stream))
    if st:
        _check("dn_kv_gather", st)
    return k, v


def dn_attn_workspace_bytes(B, total, heads_kv, group, D):
    return int(load_library().dn_attn_workspace_bytes(B, total, heads_kv, group, D))


def attn_workspace(q, k_cache, page_table):
    """A workspace for dn_attn_paged on tensors of these shapes (any contents)."""
    heads = max(k_cache.shape[1], 1)
    n = dn_attn_workspace_bytes(page_table.shape[0], q.shape[0], heads, q.shape[1] // heads, q.shape[2])
    return torch.empty((max(n, 16),), dtype=torch.uint8, device=q.device)


def dn_attn_paged(q, start, kv_len, page_table, k_cache, v_cache, k_exp=None, v_exp=None, scale=None, window=0,
                  out=None, lse=None, workspace=None, stream=None):
    """Attention of the newest tokens q [total,heads,D] over their requests' cached keys and values.

    The cache's tensors as for dn_kv_append; heads is a multiple of the cache's. scale defaults to
    D ** -0.5; window is how many tokens a row looks back, itself included (0, or 2^30 and more: all). q may be a slice of
    a wider projection. Returns (out [total,heads,D] in q's dtype, lse [total,heads] fp32).
    """
    B, heads_kv, D, page, max_pages, pages, cdt = _kv_pool(start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp)
    shape = q.shape
    if len(shape) != 3 or heads_kv < 1 or shape[1] % heads_kv or shape[1] < 1:
        raise ValueError("q's heads a multiple of the cache's")
    heads = shape[1]
    total, qs, dt = _rows(q, heads, D, "q")
    other = _other(stream)
    if out is None:
        out = _new(other, lambda: torch.empty((total, heads, D), dtype=q.dtype, device=q.device))
    if lse is None:
        lse = _new(other, lambda: torch.empty((total, heads), dtype=torch.float32, device=q.device))
    if workspace is None:
        workspace = _new(other, lambda: attn_workspace(q, k_cache, page_table), kept=False)
    if not (out.is_cuda and out.is_contiguous() and lse.is_cuda and lse.is_contiguous() and workspace.is_cuda
            and workspace.is_contiguous()):
        raise ValueError("out, lse and workspace are contiguous CUDA tensors")
    if out.shape != shape or out.dtype is not q.dtype:
        raise ValueError("out [total,heads,D] in q's dtype")
    if lse.shape != shape[:2] or lse.dtype is not torch.float32:
        raise ValueError("lse [total,heads] fp32")
    st = (_lib or load_library()).dn_attn_paged(
        B, total, heads_kv, heads // heads_kv, D, page, max_pages, pages, dt, cdt, q.data_ptr(), qs, start.data_ptr(),
        kv_len.data_ptr(), page_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_exp), _ptr(v_exp),
        D ** -0.5 if scale is None else scale, max(-1, min(window, 1 << 30)), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, _stream(stream))
    if st:
        _check("dn_attn_paged", st)
    return out, lse


def dn_attn_wait_timeouts():
    return int(load_library().dn_attn_wait_timeouts())


def dn_sample_workspace_bytes(B, T, V):
    return int(load_library().dn_sample_workspace_bytes(B, T, V))


def sample_workspace(B, T, V, device):
    """A zeroed workspace of dn_sample_workspace_bytes(B, T, V) bytes."""
    return torch.zeros((max(dn_sample_workspace_bytes(B, T, V), 16),), dtype=torch.uint8, device=device)


def dn_accept_sampled(logits, draft_ids, uniform, temperature, top_k=None, top_p=None, min_p=None, target_ids=None,
                      accepted_len=None, logprob=None, workspace=None, stream=None):
    """dn_accept_greedy with sampled targets: (target_ids [B,T], accepted_len [B], logprob [B,T] fp32).

    logits [B,T,V] fp16/bf16/fp32, draft_ids [B,T] int32, uniform [B,T] fp32 in [0, 1); a request's temperature [B] fp32 (0:
    greedy), top_k [B] int32, top_p [B] and min_p [B] fp32 are device tensors, None for no filter.
    """
    B, T, V = logits.shape
    bt, b = (B, T), (B,)
    # one expression for the good case, as for the paged cache
    if not (logits.is_cuda and logits.is_contiguous() and logits.dtype in _KV_DT
            and draft_ids.shape == bt and draft_ids.dtype is _I32 and draft_ids.is_cuda and draft_ids.is_contiguous()
            and uniform.shape == bt and uniform.dtype is _F32 and uniform.is_cuda and uniform.is_contiguous()
            and temperature.shape == b and temperature.dtype is _F32 and temperature.is_cuda and temperature.is_contiguous()
            and (top_k is None or top_k.shape == b and top_k.dtype is _I32 and top_k.is_cuda and top_k.is_contiguous())
            and (top_p is None or top_p.shape == b and top_p.dtype is _F32 and top_p.is_cuda and top_p.is_contiguous())
            and (min_p is None or min_p.shape == b and min_p.dtype is _F32 and min_p.is_cuda and min_p.is_contiguous())):
        _dev(logits, draft_ids, uniform, temperature, top_k, top_p, min_p)
        _require(logits.dtype in _KV_DT, "logits fp16, bf16 or fp32")
        _require(draft_ids.dtype is _I32 and uniform.dtype is _F32, "draft_ids int32, uniform fp32")
        raise ValueError("draft_ids, uniform [B,T]; temperature, top_p, min_p [B] fp32, top_k [B] int32")
    other = _other(stream)
    if other is None and target_ids is None and accepted_len is None and logprob is None:
        target_ids, logprob = torch.empty_like(draft_ids), torch.empty_like(uniform)
        accepted_len = torch.empty(b, dtype=_I32, device=logits.device) if top_k is None else torch.empty_like(top_k)
    else:
        if target_ids is None:
            target_ids = _new(other, lambda: torch.empty_like(draft_ids))
        if logprob is None:
            logprob = _new(other, lambda: torch.empty_like(uniform))
        if accepted_len is None:
            accepted_len = _new(other, lambda: torch.empty(b, dtype=_I32, device=logits.device))
        if not (target_ids.shape == bt and target_ids.dtype is _I32 and target_ids.is_cuda and target_ids.is_contiguous()
                and accepted_len.shape == b and accepted_len.dtype is _I32 and accepted_len.is_cuda and accepted_len.is_contiguous()
                and logprob.shape == bt and logprob.dtype is _F32 and logprob.is_cuda and logprob.is_contiguous()):
            raise ValueError("target_ids [B,T] and accepted_len [B] int32, logprob [B,T] fp32: contiguous CUDA tensors")
    if workspace is None:
        workspace = _new(other, lambda: sample_workspace(B, T, V, logits.device), kept=False)
    elif not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace is a contiguous CUDA tensor")
    st = (_lib or load_library()).dn_accept_sampled(
        B, T, V, _KV_DT[logits.dtype], logits.data_ptr(), draft_ids.data_ptr(), uniform.data_ptr(), temperature.data_ptr(), _ptr(top_k),
        _ptr(top_p), _ptr(min_p), target_ids.data_ptr(), accepted_len.data_ptr(), logprob.data_ptr(), workspace.data_ptr(),
        workspace.nbytes, _stream(stream))
    if st:
        _check("dn_accept_sampled", st)
    return target_ids, accepted_len, logprob


def rope_freqs(rot, base=10000.0, scaling=None, factor=1.0, context=4096, device="cuda"):
    """The frequencies of dn_rope_append: (freqs [rot/2] int64 in 2^-64 of a turn a token, amplitude).

    Pair j turns base ** (-2j / rot) radians a token. `scaling` stretches that for contexts `factor` times longer
    than the `context` tokens a model was trained on: "linear" divides every frequency by factor; "base" raises the base so that
    the slowest pair is slowed by factor and the fastest stays; "ramp" keeps pairs that turn 32 times or more in
    `context` tokens, divides those that turn once or less, goes linearly between, and grows the amplitude by 0.1 ln(factor).
    The line is one in a pair's turns, f * (w + (1 - w) / factor) with w = (turns - 1) / 31. A model that was trained with other borders, or with a line in
    the pair's number j, needs frequencies of its own: round(turns a token * 2^64) as int64.
    """
    _require(rot >= 2 and rot % 2 == 0 and base > 1.0 and factor >= 1.0 and context > 0, "rot even, base > 1, factor >= 1, context > 0")
    _require(scaling in (None, "linear", "base", "ramp"), 'scaling None, "linear", "base" or "ramp"')
    amplitude = 1.0
    if scaling == "base" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    turns = [base ** (-2.0 * j / rot) / (2 * math.pi) for j in range(rot // 2)]
    if scaling == "linear":
        turns = [f / factor for f in turns]
    elif scaling == "ramp":
        keep = [min(1.0, max(0.0, (context * f - 1.0) / 31.0)) for f in turns]
        turns = [f * (w + (1 - w) / factor) for f, w in zip(turns, keep)]
        amplitude += 0.1 * math.log(factor)
    return torch.tensor([round(f * 2.0 ** 64) for f in turns], dtype=torch.int64, device=device), amplitude


def dn_rope_append(q, k, v, freqs, start, kv_len, page_table, k_cache, v_cache, k_exp=None, v_exp=None, positions=None,
                   q_weight=None, k_weight=None, eps=1e-6, amplitude=1.0, interleaved=False, q_out=None, stream=None):
    """dn_kv_append of k and v [total,heads,D] with q [total,heads_q,D] and k turned by their tokens' positions; returns q_out.

    freqs [rot/2] int64 and amplitude from rope_freqs: the first rot elements of a head turn, pairs rot/2 apart or side by
    side (interleaved). positions [total] int32 replaces the tokens' places in their requests. q_weight, k_weight [D]: each
    head row is normed first. The cache's tensors as for dn_kv_append; q, k and v may be slices of one projection.
    """
    B, heads, D, page, max_pages, pages, cdt = _kv_pool(start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp)
    shape = q.shape
    if len(shape) != 3 or heads < 1 or shape[1] % heads or shape[1] < 1:
        raise ValueError("q's heads a multiple of the cache's")
    total = shape[0]
    (qs, q1, q2), (ks, k1, k2), (vs, v1, v2) = q.stride(), k.stride(), v.stride()
    kv = (total, heads, D)
    if (k.shape == kv and v.shape == kv and shape[2] == D and q.dtype is k.dtype is v.dtype and q.dtype in _KV_DT
            and q1 == k1 == v1 == D and q2 == k2 == v2 == 1 and q.is_cuda and k.is_cuda and v.is_cuda
            and (total > 1 or qs >= shape[1] * D and ks >= heads * D <= vs and not (qs | ks | vs) % 8)):
        dt = _KV_DT[q.dtype]
    else:
        total, qs, dt = _rows(q, shape[1], D, "q")
        total_k, ks, dt_k = _rows(k, heads, D, "k")
        total_v, vs, dt_v = _rows(v, heads, D, "v")
        if not (total_k == total_v == total and dt_k == dt_v == dt):
            raise ValueError("q, k and v with rows of the same tokens in one dtype")
    if not (freqs.dtype is torch.int64 and freqs.dim() == 1 and freqs.is_cuda and freqs.is_contiguous()):
        raise ValueError("freqs [rot/2] int64, a contiguous CUDA tensor")
    if positions is not None and not (positions.dtype is _I32 and positions.shape == (total,) and positions.is_cuda
                                      and positions.is_contiguous()):
        raise ValueError("positions [total] int32, a contiguous CUDA tensor")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight both or none")
    for w in (q_weight, k_weight):
        if w is not None and not (w.shape == (D,) and w.dtype is q.dtype and w.is_cuda and w.is_contiguous()):
            raise ValueError("q_weight, k_weight [D] in q's dtype, contiguous CUDA tensors")
    if q_out is None:
        q_out = _new(_other(stream), lambda: torch.empty(shape, dtype=q.dtype, device=q.device))
    elif not (q_out.shape == shape and q_out.dtype is q.dtype and q_out.is_cuda and q_out.is_contiguous()):
        raise ValueError("q_out like q, a contiguous CUDA tensor")
    st = (_lib or load_library()).dn_rope_append(
        B, total, heads, shape[1] // heads, D, 2 * freqs.shape[0], page, max_pages, pages, dt, cdt, 1 if interleaved else 0, q.data_ptr(), qs,
        k.data_ptr(), ks, v.data_ptr(), vs, _ptr(positions), freqs.data_ptr(), amplitude, _ptr(q_weight), _ptr(k_weight), eps,
        start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _ptr(k_exp),
        _ptr(v_exp), q_out.data_ptr(), _stream(stream))
    if st:
        _check("dn_rope_append", st)
    return q_out


_ACT = {None: 0, "sigmoid": 1, "silu": 2}
_ORDER = {"norm_gate": 0, "gate_norm": 1, "gate": 2}


def dn_head_norm(x, gate=None, weight=None, eps=1e-6, act="silu", order="norm_gate", out=None, stream=None):
    """Norm and gate of each head's output x [rows,heads,D]; returns out (like x, dense).

    order "norm_gate": N(x) * weight * act(gate); "gate_norm": N(x * act(gate)) * weight; "gate": x * act(gate).
    act "silu", "sigmoid" or None (the gate itself). gate and weight [D] may be None where the order allows it; x
    and gate may be slices of wider tensors, and out may be x if that is dense.
    """
    shape = x.shape
    if len(shape) != 3 or shape[1] < 1 or act not in _ACT or order not in _ORDER:
        raise ValueError('x [rows,heads,D], act "silu", "sigmoid" or None, order "norm_gate", "gate_norm" or "gate"')
    rows, heads, D = shape
    _, xs, dt = _rows(x, heads, D, "x")
    gs = 0
    if gate is not None:
        rows_g, gs, dt_g = _rows(gate, heads, D, "gate")
        if rows_g != rows or dt_g != dt:
            raise ValueError("gate like x")
    if weight is not None and not (weight.shape == (D,) and weight.dtype is x.dtype and weight.is_cuda and weight.is_contiguous()):
        raise ValueError("weight [D] in x's dtype, a contiguous CUDA tensor")
    if out is None:
        out = _new(_other(stream), lambda: torch.empty(shape, dtype=x.dtype, device=x.device))
    elif not (out.shape == shape and out.dtype is x.dtype and out.is_cuda and out.is_contiguous()):
        raise ValueError("out like x, a contiguous CUDA tensor")
    st = (_lib or load_library()).dn_head_norm(rows, heads, D, dt, _ORDER[order], _ACT[act], x.data_ptr(), xs, _ptr(gate), gs, _ptr(weight),
                                               eps, out.data_ptr(), _stream(stream))
    if st:
        _check("dn_head_norm", st)
    return out


def _wide_rows(t, shape, dtype, name):
    """Checks rows [rows, C], dense inside a row; returns the row stride in elements."""
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError("%s [rows,C] in y's dtype, a CUDA tensor dense inside a row" % name)
    return t.stride(0) if shape[0] > 1 else shape[1]


def dn_residual_norm(y, residual, weight=None, after_weight=None, gate=None, act="sigmoid", scale=1.0, eps=1e-6, residual_out=None,
                     out=None, stream=None):
    """residual + scale * z of a block's output y [rows,C], and its norm for the next block; returns (out, residual_out).

    z is y, normed with after_weight [C] if that is given, times act(gate [rows,C]) if that is given. out is
    N(residual + scale * z) * weight in y's dtype. residual [rows,C] in y's dtype or fp32; residual_out None updates it in place.
    y None: out = N(residual) * weight alone, in the weight's dtype (or the residual's).
    """
    shape = residual.shape
    if len(shape) != 2 or act not in _ACT or not residual.is_cuda or not residual.is_contiguous():
        raise ValueError('residual [rows,C], a contiguous CUDA tensor; act "sigmoid", "silu" or None')
    dtype = y.dtype if y is not None else weight.dtype if weight is not None else out.dtype if out is not None else residual.dtype
    if dtype not in _KV_DT or residual.dtype not in _KV_DT:
        raise ValueError("y and residual fp16, bf16 or fp32")
    ys = 0 if y is None else _wide_rows(y, shape, dtype, "y")
    gs = 0 if gate is None else _wide_rows(gate, shape, dtype, "gate")
    for w in (weight, after_weight):
        if w is not None and not (w.shape == shape[1:] and w.dtype is dtype and w.is_cuda and w.is_contiguous()):
            raise ValueError("weight, after_weight [C] in y's dtype, contiguous CUDA tensors")
    if residual_out is None:
        residual_out = residual
    elif not (residual_out.shape == shape and residual_out.dtype is residual.dtype and residual_out.is_cuda and residual_out.is_contiguous()):
        raise ValueError("residual_out like residual, a contiguous CUDA tensor")
    if out is None:
        out = _new(_other(stream), lambda: torch.empty(shape, dtype=dtype, device=residual.device))
    elif not (out.shape == shape and out.dtype is dtype and out.is_cuda and out.is_contiguous()):
        raise ValueError("out [rows,C] in y's dtype, a contiguous CUDA tensor")
    st = (_lib or load_library()).dn_residual_norm(
        shape[0], shape[1], _KV_DT[dtype], _KV_DT[residual.dtype], _ACT[act], _ptr(y), ys, _ptr(gate), gs, _ptr(after_weight), scale,
        residual.data_ptr(), residual_out.data_ptr(), _ptr(weight), eps, out.data_ptr(), _stream(stream))
    if st:
        _check("dn_residual_norm", st)
    return out, residual_out


class PrefixCache:
    """Host-side prefix index of state checkpoints (dn_prefix_cache_* in include/dn.h)."""

    def __init__(self, capacity, chunk=PREFILL_CHUNK):
        self._lib = load_library()
        self._h = self._lib.dn_prefix_cache_create(chunk, capacity)
        if not self._h:
            raise ValueError("dn_prefix_cache_create failed")
        self.chunk = chunk

    @staticmethod
    def _tokens(tokens):
        import numpy as np
        a = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        return a, a.ctypes.data_as(ctypes.c_void_p)

    def insert(self, tokens, position, slot):
        """Record that the state after tokens[:position] is in `slot`; returns an evicted slot or -1."""
        a, p = self._tokens(tokens)
        if position > a.shape[0]:
            raise ValueError("position beyond the tokens")
        ev = ctypes.c_int32(-1)
        _check("dn_prefix_cache_insert",
               self._lib.dn_prefix_cache_insert(self._h, p, int(position), int(slot), ctypes.byref(ev)))
        return ev.value

    def lookup(self, tokens):
        """(position, slot) of the longest cached prefix of `tokens`, (0, -1) if none."""
        a, p = self._tokens(tokens)
        pos, slot = ctypes.c_int(0), ctypes.c_int32(-1)
        _check("dn_prefix_cache_lookup",
               self._lib.dn_prefix_cache_lookup(self._h, p, int(a.shape[0]), ctypes.byref(pos),
                                                ctypes.byref(slot)))
        return pos.value, slot.value

    def __len__(self):
        return int(self._lib.dn_prefix_cache_size(self._h))

    def close(self):
        if self._h:
            self._lib.dn_prefix_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dn_status_string(status):
    return load_library().dn_status_string(int(status)).decode()
