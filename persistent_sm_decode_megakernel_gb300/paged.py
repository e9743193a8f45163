"""Operators over a paged KV cache, trees of drafted tokens and the selection of a beam search, on torch tensors.

PyTorch is used for device memory and streams only; the work runs in libmk.so, through the
C ABI of include/mk.h (mk_rope_append, mk_paged_attention, mk_update_pages, mk_compact_pages,
mk_beam_select, mk_tree_attention, mk_accept_drafts, mk_update_bounds, mk_page_scores,
mk_sparse_attention), whose comments define each operator.  Layout: a layer's keys and values are
[n_pages, n_kv_heads, page_size, head_dim]; position t of table row r lies in page
table[r, t // page_size] at row t % page_size.

Every call enqueues on the current stream of the tensors' device, waits for nothing and can
be captured into a CUDA graph.  Wrong arguments raise before anything is enqueued (ValueError
for tensors, MkError with the C status otherwise); what only the device can see goes to the
`status` tensor (int32 [4], zeroed by the caller), which `check_status` reads.  A call's
workspace is allocated per call by torch, so calls on different streams or in different
captured graphs do not share one.  What a call writes in place counts as changed, as after torch's
own operators.  These are operators of generation: they have no backward pass and no
forward-mode derivative, and refuse tensors that require a gradient or have a tangent (ValueError)
unless gradients or that mode are switched off.
"""
import ctypes

import torch

from . import MkError, check, mk_rope_desc, mk_rope_freqs
try:
    from . import _mk_torch
except ImportError as e:
    raise ImportError("the torch extension of the paged operators is not built or does not fit this torch: run "
                      "__graft_entry__.build() with g++ and a torch with CUDA") from e

_mk_torch.set_error(MkError)
ROPE_KINDS = {"none": 0, "linear": 1, "base": 2, "blended": 3, "wavelength": 4}


def rope_freqs(theta, n_rot, kind="none", factor=1.0, original=0.0, beta_fast=0.0, beta_slow=0.0, device=None):
    """The rotary frequencies (float64 [n_rot / 2], on `device`) and the factor of cos and sin, of the
    kinds that mk_rope_desc defines: none, linear, base, blended, wavelength."""
    if kind not in ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(ROPE_KINDS)}")
    f, m = (ctypes.c_double * 64)(), ctypes.c_float()
    desc = mk_rope_desc(theta, int(n_rot), ROPE_KINDS[kind], factor, original, beta_fast, beta_slow)
    check(mk_rope_freqs(ctypes.byref(desc), f, ctypes.byref(m)), "mk_rope_freqs")
    return torch.tensor(list(f)[: int(n_rot) // 2], dtype=torch.float64, device=device), m.value


def rope_append(q, k, v, k_pages, v_pages, table, positions, rows=None, freqs=None, interleaved=False, mscale=1.0,
                q_out=None, status=None, slots=None):
    """Rotates q and k ([tokens, heads, head_dim], any strides with contiguous dims) at `positions`
    and writes k and v into the pages of table rows `rows` (default: token t is row t).  Returns the
    rotated queries (`q_out`, which may be q; None without q).  freqs None: nothing is rotated.  slots
    (int32 [tokens]): where in its row a token's key and value go, if not to its position."""
    return _mk_torch.rope_append(q, k, v, k_pages, v_pages, table, positions, rows, freqs, interleaved, mscale, q_out,
                                 status, slots)


def paged_attention(q, k_pages, v_pages, table, lens, rows=None, scale=None, softcap=0.0, window=0, len_add=0, out=None,
                    return_lse=False, status=None):
    """Attention of q ([rows, heads, head_dim], one new token per row) over the first lens + len_add
    positions of table rows `rows` (default: query r is row r).  scale defaults to
    1 / sqrt(head_dim).  Returns the output, with return_lse also the float32 log-sum-exp."""
    return _mk_torch.paged_attention(q, k_pages, v_pages, table, lens, rows, scale, softcap, window, len_add, out,
                                     return_lse, status)


def tree_attention(q, k_pages, v_pages, table, lens, parents, rows=None, scale=None, softcap=0.0, window=0, out=None,
                   return_lse=False, status=None):
    """Attention of trees of drafted tokens (mk_tree_attention): q [rows, nodes, heads, head_dim], parents int32
    [rows, nodes] (a lower node, -1 for a root, else the node is absent).  Node i, whose key and value lie in
    slot lens[r] + i of table row `rows` (default: r), sees slots 0..lens[r] - 1, its ancestors and itself.
    Returns the output, with return_lse also the float32 log-sum-exp [rows, nodes, heads]."""
    return _mk_torch.tree_attention(q, k_pages, v_pages, table, lens, parents, rows, scale, softcap, window, out,
                                    return_lse, status)


def accept_drafts(k, v, table, lens, tokens, parents, choices, status=None):
    """Takes over the drafted tokens that the model chose (mk_accept_drafts): tokens, parents and choices (the model's
    token after each node) int32 [rows of the table, nodes], node 0 being the token that stands.  In place: the
    accepted nodes' keys and values of every layer (k and v as in update_pages) and lens.  Returns the choices of the
    accepted nodes, the nodes (both [rows, nodes], -1 behind the last) and their number [rows]."""
    return _mk_torch.accept_drafts(k, v, table, lens, tokens, parents, choices, status)


def update_bounds(k_pages, bounds, table, lens, rows=None, new=1, status=None):
    """The least and greatest elements of the keys of every page that holds one of the last `new` positions of table
    rows `rows` (mk_update_bounds), into bounds [n_pages, n_kv_heads, 2, head_dim]."""
    _mk_torch.update_bounds(k_pages, bounds, table, lens, rows, new, status)


def page_scores(q, bounds, table, lens, page_size, rows=None, status=None):
    """What the product of q ([rows, heads, head_dim]) with a key within a page's bounds can be at most, the greatest of
    the heads of a kv head: float32 [rows, kv heads, table width], -inf where a row has no page."""
    return _mk_torch.page_scores(q, bounds, table, lens, page_size, rows, status)


def sparse_attention(q, k_pages, v_pages, table, lens, scores, n_blocks, rows=None, first=1, last=1, scale=None,
                     softcap=0.0, out=None, return_lse=False, return_pages=False, status=None):
    """paged_attention over n_blocks pages of each row and kv head (mk_sparse_attention): the first `first`, the last
    `last` and of the others those with the greatest scores ([rows, kv heads, table width]), ties to the lower page.
    Returns the output, with return_lse also the log-sum-exp, with return_pages also the pages' numbers in the row
    (int32 [rows, kv heads, n_blocks], rising, -1 behind them)."""
    return _mk_torch.sparse_attention(q, k_pages, v_pages, table, lens, scores, n_blocks, rows, first, last, scale, softcap,
                                      out, return_lse, return_pages, status)


def update_pages(k, v, table, lens, refs, parents=None, reserve=None, status=None):
    """Fork, free and reserve (mk_update_pages), in place: table, lens, refs and the copied pages of
    k and v ([layers, n_pages, n_kv_heads, page_size, head_dim])."""
    _mk_torch.update_pages(k, v, table, lens, refs, parents, reserve, status)


def compact_pages(k, v, table, refs, status=None):
    """Moves the held pages to the lowest places (mk_compact_pages), in place: table, refs, k and v."""
    _mk_torch.compact_pages(k, v, table, refs, status)


def beam_select(logits, scores, ended, eos=-1, status=None):
    """One step of a beam search (mk_beam_select).  logits [groups * beams, vocab], its rows at any
    stride; scores float32 and ended int32 [groups, beams].  Returns tokens, parents (rows of logits),
    scores and ended, each [groups, beams], best first."""
    return _mk_torch.beam_select(logits, scores, ended, eos, status)


def check_status(status):
    """Waits for the current stream and raises MkError if a call reported something; clears it."""
    _mk_torch.check_status(status)
