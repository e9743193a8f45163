"""The paged-cache operators' checks of arguments (they run before any CUDA call), the rotary
frequencies, and the plain page bookkeeping the GPU tests compare with, on the CPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from paged_plain import Pages

P = 0x10000  # a 16-byte aligned address that is never followed


@pytest.fixture(scope="module")
def mk():
    import __graft_entry__
    __graft_entry__.build()
    import persistent_sm_decode_megakernel_gb300 as m
    return m


def _view(mk, **kw):
    v = mk.mk_page_view(P, P, 2 * 16 * 64, 4, 2, 16, 64, mk.MK_BF16, P, 3, 2, 2)
    for k, x in kw.items():
        setattr(v, k, x)
    return v


def _append(mk, view, **kw):
    a = mk.mk_append_args(P, P, P, P, mk.MK_BF16, 2, 4, 256, 64, 128, 64, 128, 64, 256, 64, P, None, P, 32, 0, 1.0)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_rope_append(ctypes.byref(a), ctypes.byref(view), None, None)


def _attend(mk, view, **kw):
    a = mk.mk_attend_args(P, P, None, mk.MK_BF16, 2, 4, 256, 64, 256, 64, P, 0, None, 0.125, 0.0, 0, P, 1 << 30)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_paged_attention(ctypes.byref(a), ctypes.byref(view), None, None)


def _pool(mk, **kw):
    p = mk.mk_page_pool(P, P, 2, 8, 16, 4096, 4096, 32768, P, 3, 2, 2, P)
    for k, x in kw.items():
        setattr(p, k, x)
    return p


def _update(mk, pool, **kw):
    a = mk.mk_update_args(P, None, None, P, 1 << 20)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_update_pages(ctypes.byref(a), ctypes.byref(pool), None, None)


def _select(mk, **kw):
    a = mk.mk_select_args(P, mk.MK_F32, 100, 2, 4, 100, 2, P, P, P, P, 2 * P, 2 * P, P, 1 << 20)
    for k, x in kw.items():
        setattr(a, k, x)
    return mk.mk_beam_select(ctypes.byref(a), None, None)


BAD_VIEWS = [dict(k=None), dict(table=None), dict(k=P + 8), dict(v=P + 2), dict(head_dim=96), dict(page_size=8),
             dict(page_size=24), dict(page_size=2048), dict(n_pages=0), dict(n_kv_heads=0), dict(n_rows=0),
             dict(table_width=0), dict(table_stride=1), dict(page_stride=16 * 64), dict(page_stride=2 * 16 * 64 + 4),
             dict(dtype=2), dict(dtype=-1), dict(table_width=1 << 28, table_stride=1 << 28)]


@pytest.mark.parametrize("bad", BAD_VIEWS, ids=str)
def test_bad_page_views_are_refused(mk, bad):
    assert _append(mk, _view(mk, **bad)) == mk.MK_ERR_INVALID
    assert _attend(mk, _view(mk, **bad)) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(k=None), dict(positions=None), dict(q=None), dict(q_out=None), dict(dtype=3),
                                 dict(n_tokens=-1), dict(n_heads=0), dict(n_freqs=33), dict(n_freqs=-1), dict(freqs=None),
                                 dict(interleaved=2), dict(v=P + 1), dict(o_token=512), dict(o_head=128)], ids=str)
def test_bad_append_arguments_are_refused(mk, bad):
    assert _append(mk, _view(mk), **bad) == mk.MK_ERR_INVALID
    assert mk.mk_last_error()


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(lens=None), dict(dtype=3), dict(n_heads=3),
                                 dict(n_heads=0), dict(n_heads=34), dict(n_rows=-1), dict(window=-1), dict(softcap=-1.0),
                                 dict(softcap=math.nan), dict(softcap=math.inf), dict(scale=math.nan), dict(scale=math.inf), dict(q=P + 1), dict(workspace=None),
                                 dict(workspace=P + 4)], ids=str)
def test_bad_attention_arguments_are_refused(mk, bad):
    assert _attend(mk, _view(mk), **bad) == mk.MK_ERR_INVALID
    assert mk.mk_last_error()


def test_attention_over_more_tiles_than_it_counts_is_refused(mk):
    view = _view(mk, table_width=1 << 26, table_stride=1 << 26)
    assert _attend(mk, view, n_rows=16) == mk.MK_ERR_INVALID
    assert b"2^31" in mk.mk_last_error()


def test_calls_without_tokens_or_rows_do_nothing(mk):
    assert _append(mk, _view(mk), n_tokens=0) == mk.MK_OK
    assert _attend(mk, _view(mk), n_rows=0) == mk.MK_OK


BAD_POOLS = [dict(k=None), dict(refs=None), dict(table=None), dict(k=P + 8), dict(n_layers=0), dict(n_pages=0),
             dict(n_rows=0), dict(n_rows=4097), dict(table_width=0), dict(page_size=20), dict(page_bytes=0),
             dict(page_bytes=24), dict(page_stride=2048), dict(page_stride=4104), dict(layer_stride=8),
             dict(table_stride=1), dict(n_pages=1 << 30)]


@pytest.mark.parametrize("bad", BAD_POOLS, ids=str)
def test_bad_page_pools_are_refused(mk, bad):
    pool = _pool(mk, **bad)
    assert _update(mk, pool) == mk.MK_ERR_INVALID
    assert mk.mk_compact_pages(ctypes.byref(pool), P, 1 << 20, None, None) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(lens=None), dict(workspace=None), dict(workspace=P + 4), dict(workspace_bytes=64)], ids=str)
def test_bad_update_arguments_are_refused(mk, bad):
    assert _update(mk, _pool(mk), **bad) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(logits=None), dict(scores=None), dict(ended=None), dict(out_tokens=None),
                                 dict(out_scores=P), dict(out_ended=P), dict(dtype=3), dict(row_stride=99), dict(groups=0),
                                 dict(beams=0), dict(beams=33), dict(vocab=3), dict(eos=-2), dict(eos=100),
                                 dict(logits=P + 2), dict(workspace=None)], ids=str)
def test_bad_selection_arguments_are_refused(mk, bad):
    assert _select(mk, **bad) == mk.MK_ERR_INVALID


def test_workspace_queries_refuse_what_the_calls_refuse(mk):
    n = ctypes.c_size_t()
    for args in ((3, 2, 64), (34, 2, 64), (4, 0, 64), (4, 2, 80)):
        assert mk.mk_paged_attention_workspace(*args, ctypes.byref(n)) == mk.MK_ERR_INVALID
    for args in ((0, 1, 1), (4097, 1, 1), (1, 0, 1), (1, 1, 0)):
        assert mk.mk_update_pages_workspace(*args, ctypes.byref(n)) == mk.MK_ERR_INVALID
    for args in ((1, 33, 100), (0, 1, 100), (1, 4, 3)):
        assert mk.mk_beam_select_workspace(*args, ctypes.byref(n)) == mk.MK_ERR_INVALID
    assert mk.mk_update_pages_workspace(3, 5, 7, ctypes.byref(n)) == mk.MK_OK and n.value % 16 == 0


def test_tensors_that_are_not_on_a_gpu_are_refused(mk):
    from persistent_sm_decode_megakernel_gb300 import paged
    pages, table = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        paged.rope_append(q, q[:, :2], q[:, :2], pages, pages, table, one)
    with pytest.raises(ValueError):
        paged.paged_attention(q, pages, pages, table, one)
    with pytest.raises(ValueError):
        paged.update_pages(pages[None], pages[None], table, one, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        paged.beam_select(torch.zeros(2, 8), torch.zeros(1, 2), torch.zeros(1, 2, dtype=torch.int32))


# ------------------------------------------------------------------------------ frequencies
def _freqs(**kw):
    from persistent_sm_decode_megakernel_gb300 import paged
    f, m = paged.rope_freqs(**kw)
    return f.numpy(), m


@pytest.mark.parametrize("theta,n", [(10000.0, 128), (10000.0, 64), (500000.0, 2), (1e6, 24)])
def test_plain_linear_and_base_frequencies(mk, theta, n):
    i = np.arange(n // 2)
    base = theta ** (-2.0 * i / n)
    f, m = _freqs(theta=theta, n_rot=n)
    np.testing.assert_allclose(f, base, rtol=1e-14)
    assert m == 1.0
    f, _ = _freqs(theta=theta, n_rot=n, kind="linear", factor=4.0)
    np.testing.assert_allclose(f, base / 4, rtol=1e-14)
    if n > 2:
        f, _ = _freqs(theta=theta, n_rot=n, kind="base", factor=4.0)
        # the first pair keeps its frequency, the last one is divided by the factor
        np.testing.assert_allclose([f[0], f[-1]], [base[0], base[-1] / 4], rtol=1e-13)


def test_blended_and_wavelength_frequencies(mk):
    theta, n, s, L = 10000.0, 128, 8.0, 4096.0
    i = np.arange(n // 2)
    base = theta ** (-2.0 * i / n)
    turns = L * base / (2 * math.pi)
    f, m = _freqs(theta=theta, n_rot=n, kind="blended", factor=s, original=L)
    assert m == pytest.approx(0.1 * math.log(s) + 1, rel=1e-7)
    # the ramp's ends are whole indices outside [beta_slow, beta_fast]
    keep, div = i <= np.floor(n * math.log(L / (32 * 2 * math.pi)) / (2 * math.log(theta))), turns < 0.8
    np.testing.assert_allclose(f[keep], base[keep], rtol=1e-13)
    np.testing.assert_allclose(f[div], base[div] / s, rtol=1e-13)
    assert keep.any() and div.any() and np.all(np.diff(f) < 0)
    f, m = _freqs(theta=theta, n_rot=n, kind="wavelength", factor=s, original=L)
    share = np.clip((turns - 1) / 3, 0, 1)
    np.testing.assert_allclose(f, base * share + base / s * (1 - share), rtol=1e-12)
    assert m == 1.0 and (share == 0).any() and (share == 1).any() and ((share > 0) & (share < 1)).any()


@pytest.mark.parametrize("bad", [dict(theta=0.0), dict(theta=math.inf), dict(n_rot=3), dict(n_rot=0), dict(n_rot=130),
                                 dict(kind="linear", factor=0.5), dict(kind="base", n_rot=2, factor=2.0),
                                 dict(kind="blended", factor=2.0, original=0.0),
                                 dict(kind="wavelength", factor=2.0, original=4096.0, beta_fast=1.0, beta_slow=2.0),
                                 dict(kind="blended", factor=2.0, original=4096.0, theta=1.0)], ids=str)
def test_bad_frequencies_are_refused(mk, bad):
    from persistent_sm_decode_megakernel_gb300 import MkError, paged
    with pytest.raises(MkError):
        paged.rope_freqs(**{"theta": 10000.0, "n_rot": 64, **bad})


# -------------------------------------------------------------------------- the plain pages
def test_plain_pages_keep_their_invariants():
    """Random forks, frees and reservations: refs are the table's holders, the page a row writes
    next belongs to it alone, a refused step changes nothing."""
    rng = np.random.default_rng(3)
    p, ps = Pages(6, 5, 17, 16), 16
    refused = 0
    for _ in range(400):
        before = (p.table.copy(), p.lens.copy(), p.refs.copy())
        parents = rng.integers(-1, 6, 6)
        reserve = rng.integers(0, 20, 6)
        copies = p.update(parents, reserve)
        if copies is None:
            refused += 1
            for a, b in zip(before, (p.table, p.lens, p.refs)):
                np.testing.assert_array_equal(a, b)
            continue
        np.testing.assert_array_equal(p.refs, np.bincount(p.table[p.table >= 0], minlength=17))
        for r in range(6):
            if parents[r] >= 0 and reserve[r] > 0:
                for t in range(p.lens[r], p.lens[r] + reserve[r]):
                    assert p.refs[p.table[r, t // ps]] == 1
                p.lens[r] += rng.integers(0, reserve[r] + 1)
    assert 20 < refused < 380


@pytest.mark.parametrize("bad", [dict(k=None), dict(table=None), dict(page_size=24), dict(n_pages=0), dict(layer_stride=64),
                                 dict(page_stride=64), dict(table_width=0)], ids=str)
def test_bad_paged_contexts_are_refused(mk, bad):
    """mk_create_paged checks the descriptor, pages and rotary frequencies before any CUDA call."""
    import synth
    c = synth.CONFIGS["tiny"]
    page = c.n_kv_heads * 16 * c.head_dim

    def create(pages, rope=None, interleaved=0, exec_mode=0, **desc):
        d = mk.mk_model_desc(c.n_layers, c.d_model, c.n_heads, c.n_kv_heads, c.head_dim, c.ffn_dim, c.vocab, mk.MK_BF16,
                             c.rms_eps, c.rope_theta, 4, 1)
        for k, x in desc.items():
            setattr(d, k, x)
        o, h = mk.mk_options(exec_mode=exec_mode), ctypes.c_void_p()
        return mk.mk_create_paged(ctypes.byref(d), None, ctypes.byref(pages) if pages else None,
                                  ctypes.byref(rope) if rope else None, interleaved, ctypes.byref(o), None, ctypes.byref(h))

    good = dict(k=P, v=P, layer_stride=8 * page, page_stride=page, n_pages=8, page_size=16, table=P, n_rows=2, table_width=4,
                table_stride=4)
    assert create(mk.mk_paged_kv(**{**good, **bad})) == mk.MK_ERR_INVALID
    ok = mk.mk_paged_kv(**good)
    assert create(None) == mk.MK_ERR_INVALID
    assert create(ok, vocab=0) == mk.MK_ERR_INVALID
    assert create(ok, interleaved=2) == mk.MK_ERR_INVALID
    assert create(ok, exec_mode=2) == mk.MK_ERR_INVALID
    assert create(ok, rope=mk.mk_rope_desc(10000.0, 128, 0, 1.0, 0, 0, 0)) == mk.MK_ERR_INVALID
    assert create(ok, rope=mk.mk_rope_desc(10000.0, 64, 1, 0.5, 0, 0, 0)) == mk.MK_ERR_INVALID


def test_tensors_that_require_a_gradient_are_refused():
    import torch
    from persistent_sm_decode_megakernel_gb300 import paged
    pages, ids = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="gradient"):
        paged.paged_attention(q, pages.clone().requires_grad_(), pages, ids, ids[:, 0])
    with pytest.raises(ValueError, match="gradient"):
        paged.beam_select(torch.zeros(2, 8, requires_grad=True), torch.zeros(1, 2), ids)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        paged.beam_select(torch.zeros(2, 8, requires_grad=True), torch.zeros(1, 2), ids)


def test_tensors_with_a_forward_tangent_are_refused():
    """A tangent of forward-mode differentiation would be dropped: refused, unless that mode is off."""
    import torch.autograd.forward_ad as fwd
    from persistent_sm_decode_megakernel_gb300 import paged
    ids, q = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with fwd.dual_level():
        x = fwd.make_dual(torch.zeros(2, 8), torch.ones(2, 8))
        with pytest.raises(ValueError, match="tangent"):
            paged.beam_select(x, torch.zeros(1, 2), ids)
        p = fwd.make_dual(pages, torch.ones_like(pages))
        with pytest.raises(ValueError, match="tangent"):
            paged.paged_attention(q, p, pages, ids, ids[:, 0])
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
            paged.beam_select(x, torch.zeros(1, 2), ids)
        with fwd._set_fwd_grad_enabled(False), pytest.raises(ValueError, match="CUDA"):
            paged.beam_select(x, torch.zeros(1, 2), ids)
    with pytest.raises(ValueError, match="CUDA"):
        paged.beam_select(torch.zeros(2, 8), torch.zeros(1, 2), ids)


@pytest.mark.parametrize("bad", [dict(o_token=0), dict(o_head=0), dict(o_head=32, o_token=512), dict(o_head=-32),
                                 dict(o_token=63), dict(q=2 * P, q_out=2 * P, q_token=0, o_token=0)], ids=str)
def test_rotated_queries_that_share_memory_are_refused(mk, bad):
    """An output whose heads or tokens lie over one another (an expanded tensor) would hold whichever came last."""
    assert _append(mk, _view(mk), **{**dict(q_out=3 * P), **bad}) == mk.MK_ERR_INVALID
    assert b"overlap" in mk.mk_last_error()


@pytest.mark.parametrize("bad", [dict(o_row=0), dict(o_head=0), dict(o_head=63), dict(o_row=-32)], ids=str)
def test_attention_outputs_that_share_memory_are_refused(mk, bad):
    assert _attend(mk, _view(mk), **bad) == mk.MK_ERR_INVALID
    assert b"overlap" in mk.mk_last_error()


def test_strides_of_a_single_token_or_head_do_not_count(mk):
    """(n_tokens and n_rows 0: the checks are passed, and nothing is enqueued)"""
    assert _append(mk, _view(mk), n_tokens=0, o_token=0, q_out=3 * P) == mk.MK_OK
    assert _attend(mk, _view(mk), n_rows=0, o_row=0) == mk.MK_OK
    assert _append(mk, _view(mk, n_kv_heads=1, page_stride=16 * 64), n_tokens=0, n_heads=1, o_head=0, q_out=3 * P) == mk.MK_OK


@pytest.mark.parametrize("bad", [dict(scale=3e38), dict(scale=-3e38), dict(softcap=1e-38, scale=100.0), dict(softcap=1e-45),
                                 dict(softcap=3e38)], ids=str)
def test_attention_factors_beyond_the_floats_are_refused(mk, bad):
    """scale log2 e, scale / softcap and softcap log2 e are factors of the kernel: infinite ones give NaN at a score of 0."""
    assert _attend(mk, _view(mk), **bad) == mk.MK_ERR_INVALID
    assert b"scale" in mk.mk_last_error()


def test_negated_views_are_refused():
    """A tensor whose values are the negatives of what lies in its memory (imaginary part of a conjugate)."""
    from persistent_sm_decode_megakernel_gb300 import paged
    scores = torch.complex(torch.zeros(1, 1), torch.ones(1, 1)).conj().imag
    assert scores.is_neg() and scores.is_contiguous()
    with pytest.raises(ValueError, match="negated"):
        paged.beam_select(scores, scores, torch.zeros(1, 1, dtype=torch.int32))
