"""Operators over a paged KV cache, and the selection of a beam search, on torch tensors.

PyTorch is used for device memory and streams only; the work runs in libmk.so, through the
C ABI of include/mk.h (mk_rope_append, mk_paged_attention, mk_update_pages, mk_compact_pages,
mk_beam_select), whose comments define each operator.  Layout: a layer's keys and values are
[n_pages, n_kv_heads, page_size, head_dim]; position t of table row r lies in page
table[r, t // page_size] at row t % page_size.

Every call enqueues on the current stream of the tensors' device, waits for nothing and can
be captured into a CUDA graph.  Wrong arguments raise before anything is enqueued (ValueError
for tensors, MkError with the C status otherwise); what only the device can see goes to the
`status` tensor (int32 [4], zeroed by the caller), which `check_status` reads.  A call's
workspace is allocated per call by torch, so calls on different streams or in different
captured graphs do not share one.
"""
import ctypes
import math

import torch

from . import (MK_BF16, MK_F16, MK_F32, check, mk_append_args, mk_attend_args, mk_beam_select, mk_beam_select_workspace,
               mk_compact_pages, mk_page_pool, mk_page_view, mk_paged_attention, mk_paged_attention_workspace,
               mk_paged_status, mk_rope_append, mk_rope_desc, mk_rope_freqs, mk_select_args, mk_update_args,
               mk_update_pages, mk_update_pages_workspace)

_DTYPE = {torch.float16: MK_F16, torch.bfloat16: MK_BF16, torch.float32: MK_F32}
ROPE_KINDS = {"none": 0, "linear": 1, "base": 2, "blended": 3, "wavelength": 4}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _int32(t, shape, dev, name):
    _need(isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.device == dev and t.shape == shape
          and t.is_contiguous(), f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {dev}")


def _status(t, dev):
    if t is not None:
        _int32(t, (4,), dev, "status")
    return _ptr(t)


class _On:
    """The tensors' device as the current one for the call (nothing to do when it is)."""
    __slots__ = ("guard",)

    def __init__(self, dev):
        self.guard = None if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *a):
        if self.guard is not None:
            self.guard.__exit__(*a)


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _cuda(t, name):
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name} must be a CUDA tensor")
    return t.device


def _table(table, dev):
    _need(isinstance(table, torch.Tensor) and table.dtype == torch.int32 and table.device == dev and table.dim() == 2
          and (table.stride(1) == 1 or table.shape[1] == 1), "table must be an int32 [rows, pages] tensor on the pages' device")
    n, w = table.shape
    return n, w, table.stride(0) if n > 1 else max(table.stride(0), w)


def _same_pages(k, v, dims, what):
    dev = _cuda(k, what)
    _need(isinstance(v, torch.Tensor) and k.dim() == dims and k.shape == v.shape and k.dtype == v.dtype
          and k.stride() == v.stride() and v.device == dev, f"{what}: keys and values must have {dims} dims, and one "
          "shape, type, layout and device")
    h, s, d = k.shape[-3:]
    _need(k.stride()[-3:] == (s * d, d, 1), f"{what}: a page's heads, positions and dims must be contiguous")
    _need(k.dtype in (torch.float16, torch.bfloat16), f"{what} must be float16 or bfloat16")
    return dev, h, s, d


def _page_view(k, v, table):
    dev, h, s, d = _same_pages(k, v, 4, "pages")
    n = k.shape[0]
    rows, width, stride = _table(table, dev)
    return dev, mk_page_view(k.data_ptr(), v.data_ptr(), k.stride(0) if n > 1 else h * s * d, n, h, s, d,
                             _DTYPE[k.dtype], table.data_ptr(), rows, width, stride)


def _heads(t, n, heads, dim, dtype, dev, name):
    _need(isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == dev and t.shape == (n, heads, dim)
          and t.stride(2) == 1, f"{name} must be [{n}, {heads}, {dim}] {dtype} on {dev}, its last dim contiguous")


def rope_freqs(theta, n_rot, kind="none", factor=1.0, original=0.0, beta_fast=0.0, beta_slow=0.0, device=None):
    """The rotary frequencies (float64 [n_rot / 2], on `device`) and the factor of cos and sin, of the
    kinds that mk_rope_desc defines: none, linear, base, blended, wavelength."""
    _need(kind in ROPE_KINDS, f"kind must be one of {sorted(ROPE_KINDS)}")
    f, m = (ctypes.c_double * 64)(), ctypes.c_float()
    desc = mk_rope_desc(theta, int(n_rot), ROPE_KINDS[kind], factor, original, beta_fast, beta_slow)
    check(mk_rope_freqs(ctypes.byref(desc), f, ctypes.byref(m)), "mk_rope_freqs")
    return torch.tensor(list(f)[: int(n_rot) // 2], dtype=torch.float64, device=device), m.value


def rope_append(q, k, v, k_pages, v_pages, table, positions, rows=None, freqs=None, interleaved=False, mscale=1.0,
                q_out=None, status=None):
    """Rotates q and k ([tokens, heads, head_dim], any strides with contiguous dims) at `positions`
    and writes k and v into the pages of table rows `rows` (default: token t is row t).  Returns the
    rotated queries (`q_out`, which may be q; None without q).  freqs None: nothing is rotated."""
    dev, view = _page_view(k_pages, v_pages, table)
    _need(isinstance(k, torch.Tensor) and k.dim() == 3 and k.dtype in _DTYPE, "k must be [tokens, kv heads, head_dim]")
    n, hd = k.shape[0], view.head_dim
    _heads(k, n, view.n_kv_heads, hd, k.dtype, dev, "k")
    _heads(v, n, view.n_kv_heads, hd, k.dtype, dev, "v")
    _int32(positions, (n,), dev, "positions")
    if rows is not None:
        _int32(rows, (n,), dev, "rows")
    hq = 0
    if q is not None:
        _need(isinstance(q, torch.Tensor) and q.dim() == 3, "q must be [tokens, heads, head_dim]")
        hq = q.shape[1]
        _heads(q, n, hq, hd, k.dtype, dev, "q")
        if q_out is None:
            q_out = torch.empty((n, hq, hd), dtype=q.dtype, device=dev)
        else:
            _heads(q_out, n, hq, hd, k.dtype, dev, "q_out")
    else:
        _need(q_out is None, "q_out without q")
    n_freqs = 0
    if freqs is not None:
        _need(isinstance(freqs, torch.Tensor) and freqs.dtype == torch.float64 and freqs.dim() == 1 and freqs.device == dev
              and freqs.is_contiguous(), f"freqs must be a contiguous float64 vector on {dev}")
        n_freqs = freqs.numel()
    st = _status(status, dev)
    if n == 0:
        return q_out
    a = mk_append_args(_ptr(q), k.data_ptr(), v.data_ptr(), _ptr(q_out), _DTYPE[k.dtype], n, hq,
                       *(q.stride()[:2] if hq else (0, 0)), *k.stride()[:2], *v.stride()[:2],
                       *(q_out.stride()[:2] if hq else (0, 0)), positions.data_ptr(), _ptr(rows), _ptr(freqs), n_freqs,
                       int(bool(interleaved)), mscale)
    with _On(dev):
        check(mk_rope_append(ctypes.byref(a), ctypes.byref(view), st, _stream(dev)), "mk_rope_append")
    return q_out


def paged_attention(q, k_pages, v_pages, table, lens, rows=None, scale=None, softcap=0.0, window=0, len_add=0, out=None,
                    return_lse=False, status=None):
    """Attention of q ([rows, heads, head_dim], one new token per row) over the first lens + len_add
    positions of table rows `rows` (default: query r is row r).  scale defaults to
    1 / sqrt(head_dim).  Returns the output, with return_lse also the float32 log-sum-exp."""
    dev, view = _page_view(k_pages, v_pages, table)
    _need(isinstance(q, torch.Tensor) and q.dim() == 3 and q.dtype in _DTYPE, "q must be [rows, heads, head_dim]")
    n, hq, hd = q.shape[0], q.shape[1], view.head_dim
    _heads(q, n, hq, hd, q.dtype, dev, "q")
    if out is None:
        out = torch.empty((n, hq, hd), dtype=q.dtype, device=dev)
    else:
        _heads(out, n, hq, hd, q.dtype, dev, "out")
    _int32(lens, (n,), dev, "lens")
    if rows is not None:
        _int32(rows, (n,), dev, "rows")
    lse = torch.empty((n, hq), dtype=torch.float32, device=dev) if return_lse else None
    st = _status(status, dev)
    if n:
        with _On(dev):
            need = ctypes.c_size_t()
            check(mk_paged_attention_workspace(hq, view.n_kv_heads, hd, ctypes.byref(need)), "mk_paged_attention_workspace")
            ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
            a = mk_attend_args(q.data_ptr(), out.data_ptr(), _ptr(lse), _DTYPE[q.dtype], n, hq, *q.stride()[:2],
                               *out.stride()[:2], lens.data_ptr(), len_add, _ptr(rows),
                               1.0 / math.sqrt(hd) if scale is None else scale, softcap, window, ws.data_ptr(), need.value)
            check(mk_paged_attention(ctypes.byref(a), ctypes.byref(view), st, _stream(dev)), "mk_paged_attention")
    return (out, lse) if return_lse else out


def _pool(k, v, table, refs):
    dev, h, s, d = _same_pages(k, v, 5, "the pool")
    n_layers, n = k.shape[:2]
    rows, width, stride = _table(table, dev)
    _int32(refs, (n,), dev, "refs")
    e = k.element_size()
    page = h * s * d * e
    return dev, mk_page_pool(k.data_ptr(), v.data_ptr(), n_layers, n, s, page, k.stride(1) * e if n > 1 else page,
                             k.stride(0) * e if n_layers > 1 else page, table.data_ptr(), rows, width, stride,
                             refs.data_ptr())


def _pool_workspace(pool, dev):
    need = ctypes.c_size_t()
    check(mk_update_pages_workspace(pool.n_rows, pool.table_width, pool.n_pages, ctypes.byref(need)),
          "mk_update_pages_workspace")
    return torch.empty(need.value, dtype=torch.uint8, device=dev), need.value


def update_pages(k, v, table, lens, refs, parents=None, reserve=None, status=None):
    """Fork, free and reserve (mk_update_pages), in place: table, lens, refs and the copied pages of
    k and v ([layers, n_pages, n_kv_heads, page_size, head_dim])."""
    dev, pool = _pool(k, v, table, refs)
    n = pool.n_rows
    _int32(lens, (n,), dev, "lens")
    for t, name in ((parents, "parents"), (reserve, "reserve")):
        if t is not None:
            _int32(t, (n,), dev, name)
    st = _status(status, dev)
    with _On(dev):
        ws, size = _pool_workspace(pool, dev)
        a = mk_update_args(lens.data_ptr(), _ptr(parents), _ptr(reserve), ws.data_ptr(), size)
        check(mk_update_pages(ctypes.byref(a), ctypes.byref(pool), st, _stream(dev)), "mk_update_pages")


def compact_pages(k, v, table, refs, status=None):
    """Moves the held pages to the lowest places (mk_compact_pages), in place: table, refs, k and v."""
    dev, pool = _pool(k, v, table, refs)
    st = _status(status, dev)
    with _On(dev):
        ws, size = _pool_workspace(pool, dev)
        check(mk_compact_pages(ctypes.byref(pool), ws.data_ptr(), size, st, _stream(dev)), "mk_compact_pages")


def beam_select(logits, scores, ended, eos=-1, status=None):
    """One step of a beam search (mk_beam_select).  logits [groups * beams, vocab], its rows at any
    stride; scores float32 and ended int32 [groups, beams].  Returns tokens, parents (rows of logits),
    scores and ended, each [groups, beams], best first."""
    dev = _cuda(logits, "logits")
    _need(logits.dim() == 2 and logits.dtype in _DTYPE and (logits.stride(1) == 1 or logits.shape[1] == 1),
          "logits must be [rows, vocab] with contiguous rows, float16, bfloat16 or float32")
    _need(isinstance(scores, torch.Tensor) and scores.dim() == 2 and scores.dtype == torch.float32 and scores.device == dev
          and scores.is_contiguous(), f"scores must be a contiguous float32 [groups, beams] tensor on {dev}")
    groups, beams = scores.shape
    _need(logits.shape[0] == groups * beams, "logits must have groups * beams rows")
    _int32(ended, (groups, beams), dev, "ended")
    vocab = logits.shape[1]
    st = _status(status, dev)
    with _On(dev):
        need = ctypes.c_size_t()
        check(mk_beam_select_workspace(groups, beams, vocab, ctypes.byref(need)), "mk_beam_select_workspace")
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        tokens, parents, done = torch.empty((3, groups, beams), dtype=torch.int32, device=dev).unbind()
        best = torch.empty((groups, beams), dtype=torch.float32, device=dev)
        a = mk_select_args(logits.data_ptr(), _DTYPE[logits.dtype],
                           logits.stride(0) if logits.shape[0] > 1 else vocab, groups, beams, vocab,
                           eos, scores.data_ptr(), ended.data_ptr(), tokens.data_ptr(), parents.data_ptr(),
                           best.data_ptr(), done.data_ptr(), ws.data_ptr(), need.value)
        check(mk_beam_select(ctypes.byref(a), st, _stream(dev)), "mk_beam_select")
    return tokens, parents, best, done


def check_status(status):
    """Waits for the current stream and raises MkError if a call reported something; clears it."""
    dev = _cuda(status, "status")
    _int32(status, (4,), dev, "status")
    with _On(dev):
        check(mk_paged_status(status.data_ptr(), _stream(dev)), "paged status")
