"""The checks of arguments of the operators on drafted trees and chosen pages (they run before any CUDA call), and the
plain forms the GPU tests compare with, on the CPU."""
import ctypes
import math

import numpy as np
import pytest

from drafts_plain import accept, choose, lineage, page_score, tree_seen
from test_paged_cpu import BAD_VIEWS, P, _attend, _pool, _view, mk  # noqa: F401  (mk: the library's fixture)


def _tree(mk, view, **kw):
    # q [2][3][4][64]
    a = mk.mk_tree_args(P, P, None, mk.MK_BF16, 2, 3, 4, 768, 256, 64, 768, 256, 64, P, P, None, 0.125, 0.0, 0, P, 1 << 40)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_tree_attention(ctypes.byref(a), ctypes.byref(view), None, None)


def _accept(mk, pool, **kw):
    a = mk.mk_accept_args(P, 2, 4, P, P, P, P, P, P)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_accept_drafts(ctypes.byref(a), ctypes.byref(pool), None, None)


def _bounds(mk, view, **kw):
    a = mk.mk_bounds_args(P, P, None, 2, 1)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_update_bounds(ctypes.byref(a), ctypes.byref(view), None, None)


def _scores(mk, view, **kw):
    a = mk.mk_scores_args(P, mk.MK_BF16, 2, 4, 256, 64, P, P, None, P)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_page_scores(ctypes.byref(a), ctypes.byref(view), None, None)


def _sparse(mk, view, attend=(), **kw):
    a = mk.mk_attend_args(P, P, None, mk.MK_BF16, 2, 4, 256, 64, 256, 64, P, 0, None, 0.125, 0.0, 0, P, 1 << 40)
    for k, x in dict(attend).items():
        setattr(a, k, x)
    s = mk.mk_sparse_args(P, 4, 2, 2, 1, 1, None)
    for k, x in kw.items():
        setattr(s, k, x)
    return mk.mk_sparse_attention(ctypes.byref(a), ctypes.byref(s), ctypes.byref(view), None, None)


@pytest.mark.parametrize("bad", BAD_VIEWS, ids=str)
def test_bad_page_views_are_refused(mk, bad):  # noqa: F811
    for call in (_tree, _bounds, _scores, _sparse):
        assert call(mk, _view(mk, **bad)) == mk.MK_ERR_INVALID, call


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(lens=None), dict(parents=None), dict(dtype=3), dict(dtype=-1),
                                 dict(n_rows=-1), dict(n_nodes=0), dict(n_nodes=129), dict(n_heads=0), dict(n_heads=3), dict(n_heads=34),
                                 dict(n_rows=1 << 24), dict(window=-1), dict(scale=math.nan), dict(scale=math.inf), dict(softcap=-1.0),
                                 dict(softcap=math.inf), dict(softcap=math.nan), dict(softcap=1e-39), dict(q=P + 1), dict(out=P + 1),
                                 dict(o_row=256), dict(o_node=64), dict(o_head=32), dict(o_node=0), dict(o_row=0), dict(workspace=None),
                                 dict(workspace=P + 8)], ids=str)
def test_bad_tree_arguments_are_refused(mk, bad):  # noqa: F811
    assert _tree(mk, _view(mk), **bad) == mk.MK_ERR_INVALID
    assert mk.mk_last_error()


def test_tree_of_no_rows_and_null_structures(mk):  # noqa: F811
    assert _tree(mk, _view(mk), n_rows=0) == mk.MK_OK
    v = _view(mk)
    for f in (mk.mk_tree_attention, mk.mk_update_bounds, mk.mk_page_scores):
        assert f(None, ctypes.byref(v), None, None) == mk.MK_ERR_INVALID
    assert mk.mk_sparse_attention(None, None, ctypes.byref(v), None, None) == mk.MK_ERR_INVALID
    p = _pool(mk, refs=None)
    assert mk.mk_accept_drafts(None, ctypes.byref(p), None, None) == mk.MK_ERR_INVALID
    # a line of work that 32 bits do not count
    assert _tree(mk, _view(mk, table_width=1 << 26, table_stride=1 << 26), n_rows=200) == mk.MK_ERR_INVALID


def test_append_at_checks_as_append_does(mk):  # noqa: F811
    a = mk.mk_append_args(P, P, P, P, mk.MK_BF16, 2, 4, 256, 64, 128, 64, 128, 64, 256, 64, None, None, P, 32, 0, 1.0)
    v = _view(mk)
    assert mk.mk_rope_append_at(ctypes.byref(a), P, ctypes.byref(v), None, None) == mk.MK_ERR_INVALID
    a.positions, a.n_tokens = P, 0
    assert mk.mk_rope_append_at(ctypes.byref(a), P, ctypes.byref(v), None, None) == mk.MK_OK


@pytest.mark.parametrize("bad", [dict(lens=None), dict(tokens=None), dict(parents=None), dict(choices=None), dict(out_tokens=None),
                                 dict(out_path=None), dict(out_count=None), dict(n_nodes=0), dict(n_nodes=129), dict(n_kv_heads=0),
                                 dict(n_kv_heads=3)], ids=str)
def test_bad_accept_arguments_are_refused(mk, bad):  # noqa: F811
    assert _accept(mk, _pool(mk, refs=None), **bad) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(table=None), dict(k=P + 8), dict(n_layers=0), dict(n_pages=0), dict(n_rows=0),
                                 dict(table_width=0), dict(table_stride=1), dict(page_size=8), dict(page_size=2048), dict(page_bytes=4104),
                                 dict(page_bytes=16384, page_stride=16384, layer_stride=1 << 20), dict(page_stride=4000), dict(page_stride=2048),
                                 dict(layer_stride=24), dict(layer_stride=16), dict(n_layers=1 << 24)], ids=str)
def test_bad_accept_pools_are_refused(mk, bad):  # noqa: F811
    assert _accept(mk, _pool(mk, refs=None, **bad)) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(bounds=None), dict(bounds=P + 8), dict(lens=None), dict(n_rows=-1), dict(n_new=0), dict(n_new=-5),
                                 dict(n_rows=1 << 30, n_new=1 << 20)], ids=str)
def test_bad_bounds_arguments_are_refused(mk, bad):  # noqa: F811
    assert _bounds(mk, _view(mk), **bad) == mk.MK_ERR_INVALID
    assert _bounds(mk, _view(mk), n_rows=0) == mk.MK_OK


@pytest.mark.parametrize("bad", [dict(q=None), dict(bounds=None), dict(bounds=P + 4), dict(lens=None), dict(scores=None), dict(scores=P + 2),
                                 dict(dtype=3), dict(q=P + 1), dict(n_rows=-1), dict(n_rows=65536), dict(n_heads=0), dict(n_heads=5),
                                 dict(n_heads=66)], ids=str)
def test_bad_score_arguments_are_refused(mk, bad):  # noqa: F811
    assert _scores(mk, _view(mk), **bad) == mk.MK_ERR_INVALID
    assert _scores(mk, _view(mk), n_rows=0) == mk.MK_OK


@pytest.mark.parametrize("bad", [dict(scores=None), dict(scores=P + 2), dict(n_blocks=0), dict(n_blocks=1), dict(n_blocks=65537), dict(first=-1),
                                 dict(last=0), dict(last=2), dict(first=2 ** 31 - 1, last=2 ** 31 - 1)], ids=str)
def test_bad_sparse_arguments_are_refused(mk, bad):  # noqa: F811
    assert _sparse(mk, _view(mk), **bad) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(lens=None), dict(window=3), dict(n_rows=-1), dict(n_heads=3), dict(n_heads=0),
                                 dict(workspace=None), dict(workspace=P + 8), dict(workspace_bytes=64), dict(scale=math.nan), dict(o_row=0)], ids=str)
def test_bad_attention_arguments_of_chosen_pages_are_refused(mk, bad):  # noqa: F811
    assert _sparse(mk, _view(mk), attend=bad) in (mk.MK_ERR_INVALID, mk.MK_ERR_CUDA)   # (the workspace's size asks the device)


def test_workspace_queries_check_their_arguments(mk):  # noqa: F811
    n = ctypes.c_size_t()
    for args in ((0, 4, 2, 64), (129, 4, 2, 64), (4, 3, 2, 64), (4, 4, 0, 64), (4, 34, 2, 64), (4, 4, 2, 96)):
        assert mk.mk_tree_attention_workspace(*args, ctypes.byref(n)) == mk.MK_ERR_INVALID, args
    assert mk.mk_tree_attention_workspace(4, 4, 2, 64, None) == mk.MK_ERR_INVALID
    for args in ((-1, 4, 2, 64, 4), (2, 4, 2, 64, 0), (2, 4, 2, 64, 65537), (2, 3, 2, 64, 4)):
        assert mk.mk_sparse_attention_workspace(*args, ctypes.byref(n)) == mk.MK_ERR_INVALID, args
    assert mk.mk_sparse_attention_workspace(2, 4, 2, 64, 4, None) == mk.MK_ERR_INVALID


# ------------------------------------------------------------------------------- the plain forms
def test_plain_trees():
    assert lineage([-1, 0, 1, 0, -1, 4]) == [[0], [1, 0], [2, 1, 0], [3, 0], [4], [5, 4]]
    assert lineage([-1, 1, 0, 5, -2, 4]) == [[0], None, [2, 0], None, None, None]
    seen = tree_seen(3, [-1, 0, 0, 2], window=0)
    assert [s.astype(int).tolist() for s in seen] == [[1, 1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 1, 0, 0], [1, 1, 1, 1, 0, 1, 0], [1, 1, 1, 1, 0, 1, 1]]
    # a window of 2: a node sees its own position and the one before
    assert [np.nonzero(s)[0].tolist() for s in tree_seen(3, [-1, 0, 0, 2], window=2)] == [[2, 3], [3, 4], [3, 5], [5, 6]]


def test_plain_acceptance():
    #        0
    #   1(7) 2(7) 3(9)     4 under 2, 5 under 1
    parents, tokens = [-1, 0, 0, 0, 2, 1], [1, 7, 7, 9, 8, 8]
    assert accept(tokens, parents, [7, 8, 8, 0, 0, 3]) == [0, 1, 5]      # the lower of two equal drafts
    assert accept(tokens, parents, [9, 8, 8, 0, 0, 3]) == [0, 3]
    assert accept(tokens, parents, [5, 8, 8, 0, 0, 3]) == [0]
    assert accept(tokens, [-2] + parents[1:], [7] * 6) == []


def test_plain_scores_and_choice():
    assert page_score([[1.0, -2.0]], [-3.0, -1.0], [2.0, 4.0]) == 2.0 + 2.0
    s = [1.0, 5.0, 3.0, 5.0, math.nan, -math.inf, 2.0]
    assert choose(s, 7, 4, 1, 1) == [0, 1, 4, 6] and choose(s, 7, 5, 1, 1) == [0, 1, 3, 4, 6]
    assert choose(s, 4, 4, 1, 1) == [0, 1, 2, 3] and choose(s, 7, 2, 0, 2) == [5, 6] and choose(s, 0, 3, 1, 1) == []
