"""The paged-cache operators on the GPU against plain 64-bit implementations.

Tolerances: a result rounded to a type is off by at most half a step, eps / 2 relative (plus
the smallest subnormal's half for fp16), and by what its 32-bit arithmetic adds, which each
test bounds from its own inputs."""
import math

import numpy as np
import pytest
import torch

from paged_plain import Pages, attend, rope, select

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def paged():
    import __graft_entry__
    __graft_entry__.build()
    from persistent_sm_decode_megakernel_gb300 import paged
    return paged


def half_step(dtype, x):
    """The largest rounding error of |x| to dtype (fp16: or half its smallest subnormal step)."""
    return torch.finfo(dtype).eps / 2 * np.abs(x) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(4, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------------- append
def _append_case(paged, T, hq, hkv, hd, ps, vec, cache, rot, inter, far, layout, scaled=False):
    g = torch.Generator(device=DEV).manual_seed(1)
    dt, ct = TYPES[vec], TYPES[cache]
    rows, width = 3, far // ps + T // ps + 3
    n_pages = rows * (T // ps + 3) + 2
    pages = torch.randn(2, n_pages, hkv, ps, hd, generator=g, device=DEV).to(ct)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    table[:, far // ps:] = torch.randperm(n_pages, generator=g, device=DEV)[: rows * (width - far // ps)].view(rows, -1).int()
    if layout == "fused":          # one row of q, k and v heads per token
        qkv = torch.randn(T, hq + 2 * hkv, hd, generator=g, device=DEV).to(dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    elif layout == "heads":        # heads before tokens
        q, k, v = (torch.randn(h, T, hd, generator=g, device=DEV).to(dt).transpose(0, 1) for h in (hq, hkv, hkv))
    else:                          # rows that start off any 16-byte boundary
        q, k, v = (torch.randn(T, h, hd + 1, generator=g, device=DEV).to(dt)[..., 1:] for h in (hq, hkv, hkv))
    r = np.arange(T) % rows
    pos = far + np.arange(T) // rows
    pos[T // 2] = -1 if T > 2 else pos[T // 2]
    freqs, m = paged.rope_freqs(10000.0, rot, *(("linear", 8.0) if scaled else ()), device=DEV) if rot else (None, 1.0)
    if scaled:
        m = 1.25
    st = status()
    out = torch.full((T, hq, hd), 7.0, dtype=dt, device=DEV)
    before = [f64(p) for p in pages]
    got = paged.rope_append(q, k, v, pages[0], pages[1], table, ints(pos), rows=ints(r), freqs=freqs, interleaved=inter,
                            mscale=m, q_out=out, status=st)
    assert got is out
    paged.check_status(st)
    fr = [] if freqs is None else freqs.cpu().tolist()
    want_k, want_v, size_k = before[0].copy(), before[1].copy(), np.zeros_like(before[0])
    touched = np.zeros(before[0].shape, dtype=bool)
    qd, kd, vd, od, tb = f64(q), f64(k), f64(v), f64(out), table.cpu().numpy()
    for t in range(T):
        if pos[t] < 0:
            assert np.all(od[t] == 7.0)
            continue
        # the rotation in 32 bits: two products and a sum of terms good to 2^-24 each, cos and
        # sin off by a few 2^-24
        w = rope(qd[t], pos[t], fr, inter, m)
        big = np.abs(qd[t]).max(-1, keepdims=True) * abs(m) * (16 * 2.0 ** -24)
        assert np.all(np.abs(od[t] - w) <= half_step(dt, w) + (big if rot else 0.0)), t
        at = (tb[r[t], pos[t] // ps], slice(None), pos[t] % ps)
        want_k[at], want_v[at], touched[at] = rope(kd[t], pos[t], fr, inter, m), vd[t], True
        size_k[at] = np.abs(kd[t]).max(-1, keepdims=True) * abs(m) * (16 * 2.0 ** -24) if rot else 0.0
    for got, want, tol in ((f64(pages[0]), want_k, half_step(ct, want_k) + size_k), (f64(pages[1]), want_v, half_step(ct, want_v))):
        assert np.all(got[~touched] == want[~touched])
        assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("vec,cache", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f16"), ("f32", "bf16"), ("bf16", "f16"),
                                       ("f16", "bf16")])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("layout", ["fused", "heads", "unaligned"])
def test_append_types_and_layouts(paged, vec, cache, inter, layout):
    _append_case(paged, 37, 4, 2, 64, 16, vec, cache, 64, inter, 0, layout)


@pytest.mark.parametrize("hd,rot", [(64, 0), (64, 2), (64, 16), (64, 32), (64, 24), (128, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
def test_append_parts_of_the_head(paged, hd, rot, inter):
    _append_case(paged, 19, 8, 8, hd, 48, "f32", "bf16", rot, inter, 0, "fused")


@pytest.mark.parametrize("T,ps,far", [(1, 16, 0), (1, 64, 511), (2, 128, 4194240), (300, 1024, 1000000), (700, 16, 131072)])
def test_append_lengths_and_far_positions(paged, T, ps, far):
    _append_case(paged, T, 4, 2, 128, ps, "f32", "f16", 128, False, far // ps * ps, "fused", scaled=True)


def test_append_in_place_and_without_queries(paged):
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(5, 4, 64, generator=g, device=DEV)
    k = torch.randn(5, 2, 64, generator=g, device=DEV)
    table, pos = ints([[0], [1], [2], [3], [4]]), ints([3, 0, 15, 7, 1])
    freqs, _ = paged.rope_freqs(10000.0, 64, device=DEV)
    pages = [torch.zeros(2, 5, 2, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = paged.rope_append(q, k, k, pages[0][0], pages[0][1], table, pos, freqs=freqs)
    assert paged.rope_append(None, k, k, pages[1][0], pages[1][1], table, pos, freqs=freqs) is None
    assert torch.equal(pages[0], pages[1]) and pages[0].abs().sum() > 0
    q2 = q.clone()
    assert paged.rope_append(q2, k, k, pages[1][0], pages[1][1], table, pos, freqs=freqs, q_out=q2) is q2
    assert torch.equal(q2, out) and not torch.equal(q2, q)


@pytest.mark.parametrize("what,row,pos,page", [("row", 9, 0, 0), ("row", -1, 0, 0), ("position", 0, 32, 0),
                                               ("page", 0, 0, 77), ("page", 0, 0, -1), ("page", 0, 0, -5)])
def test_append_reports_a_place_that_is_none(paged, what, row, pos, page):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    k = torch.ones(2, 2, 64, device=DEV)
    pages = torch.zeros(2, 3, 2, 16, 64, dtype=torch.float16, device=DEV)
    table = ints([[page, 1], [2, 2]])
    st = status()
    q = paged.rope_append(k, k, k, pages[0], pages[1], table, ints([pos, 1]), rows=ints([row, 1]), status=st)
    assert torch.equal(q, k)       # the queries do not need a place
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_PAGES and "append" in str(e.value)
    paged.check_status(st)         # cleared
    want = torch.zeros_like(pages)
    want[:, 2, :, 1] = 1           # the other token is where it belongs
    assert torch.equal(pages, want)


def test_append_of_more_shares_of_tokens_than_31_bits_count(paged):
    """Many tokens of very many heads (expanded: they take no memory), nearly all of them skipped: each token's heads are
    dealt to 4096 warps, 2.2e9 in all.  The last token and one in the middle are where they belong."""
    heads, tokens = 65535, 530000
    pages = torch.zeros(2, 2, heads, 16, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.randn(1, heads, 128, device=DEV).bfloat16()
    pos = torch.full((tokens,), -1, dtype=torch.int32, device=DEV)
    row = torch.zeros(tokens, dtype=torch.int32, device=DEV)
    pos[tokens // 2], pos[-1], row[-1] = 3, 7, 1
    st = status()
    paged.rope_append(None, k.expand(tokens, heads, 128), k.expand(tokens, heads, 128), pages[0], pages[1], ints([[0], [1]]), pos,
                      rows=row, status=st)
    paged.check_status(st)
    for p in pages:
        assert torch.equal(p[0, :, 3], k[0]) and torch.equal(p[1, :, 7], k[0])
        p[0, :, 3] = 0
        p[1, :, 7] = 0
        assert not p.any()


# ------------------------------------------------------------------------------- attention
def _make_cache(g, lens, hkv, hd, ps, cache, extra=3, poison=True):
    """Pages with random order whose places behind a sequence's end hold NaN, infinities and large values."""
    need = [-(-n // ps) for n in lens]
    n_pages = sum(need) + extra
    ids = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    width = max(max(need), 1) + 1
    table = -np.ones((len(lens), width), dtype=np.int32)
    pages = torch.randn(2, n_pages, hkv, ps, hd, generator=g, device=DEV).to(TYPES[cache])
    if poison:
        used = torch.zeros(n_pages, ps, dtype=torch.bool, device=DEV)
    at = 0
    for r, n in enumerate(lens):
        table[r, : need[r]] = ids[at: at + need[r]]
        at += need[r]
        for i in range(need[r] if poison else 0):
            used[table[r, i], : min(ps, n - i * ps)] = True
    if poison:
        junk = torch.tensor([math.nan, math.inf, -math.inf, 6e4], device=DEV)
        bad = junk[torch.randint(0, 4, pages.shape, generator=g, device=DEV)].to(pages.dtype)
        pages = torch.where(used[None, :, None, :, None], pages, bad)
    return pages[0], pages[1], table


def _check_attend(q, kp, vp, table, lens, out, lse, scale, window=0, cap=0.0, rows=None, n_pages=None):
    """Each row and head against the plain form.  With A = scale sum |q||k| at its largest: a score's
    32-bit products and sums are off by at most (hd + 16) 2^-23 A, its query parts by 2^-17 A (bf16 cache,
    fp16 queries), 2^-22 A (fp16) or nothing; the conversion to units of log 2, exp2 and the maximum add
    2^-21 (1 + |score| / 4); a probability's parts are good to 2^-17; sums over the tiles and pieces add
    2^-23 each.  A relative error d of every probability moves the output by at most 2 d sum p |v|."""
    R, hq, hd = q.shape
    hkv, ps = kp.shape[1], kp.shape[2]
    qd, od, ld = f64(q), f64(out), f64(lse)
    kd, vd = kp.double().cpu().numpy(), vp.double().cpu().numpy()
    n_pages = kp.shape[0] if n_pages is None else n_pages
    qbits = 0.0 if q.dtype == kp.dtype else 2.0 ** -17 if kp.dtype == torch.bfloat16 and q.dtype == torch.float16 else 2.0 ** -22
    pbits = 2.0 ** -17 if kp.dtype == torch.bfloat16 and q.dtype != torch.float32 else 2.0 ** -22
    for r in range(R):
        tr, n = (r if rows is None else rows[r]), lens[r]
        if not 0 <= tr < len(table):
            n = 0
        lo, hi = (max(0, n - window) if window else 0), min(max(n, 0), table.shape[1] * ps)
        t = np.arange(hi)
        page = table[tr, t // ps] if hi else np.zeros(0, dtype=int)
        seen = (t >= lo) & (page >= 0) & (page < n_pages)
        page = np.where(seen, page, 0)
        for h in range(hq):
            j = h // (hq // hkv)
            with np.errstate(invalid="ignore"):
                w, l, mass, size = attend(qd[r, h], kd[page, j, t % ps], vd[page, j, t % ps], seen, scale, cap)
            if not seen.any():
                assert np.all(od[r, h] == 0) and ld[r, h] == -math.inf, (r, h)
                continue
            d = size * ((hd + 16) * 2.0 ** -23 + qbits) + 2.0 ** -21 * (1 + (size if not cap else min(size, cap)) / 4)
            sums = (hi / 16 + 64) * 2.0 ** -23
            assert np.all(np.abs(od[r, h] - w) <= half_step(q.dtype, w) + (2 * d + 2 * pbits + sums) * mass), (r, h, n)
            assert abs(ld[r, h] - l) <= d + sums + 2.0 ** -22 * abs(l), (r, h, n)


def _attend_case(paged, lens, hq, hkv, hd, ps, cache, vec, window=0, cap=0.0, strided=False, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kp, vp, table = _make_cache(g, lens, hkv, hd, ps, cache)
    q = torch.randn(len(lens), hq, hd, generator=g, device=DEV).mul_(1.5).to(TYPES[vec])
    out = None
    if strided:
        q = torch.cat((q, q), -1).transpose(0, 1).contiguous().transpose(0, 1)[..., hd:]
        out = torch.full((len(lens), hq, hd + 4), 9.0, dtype=q.dtype, device=DEV)
    st = status()
    got, lse = paged.paged_attention(q, kp, vp, ints(table), ints(lens), window=window, softcap=cap, return_lse=True,
                                     out=out[..., :hd] if strided else None, status=st)
    paged.check_status(st)
    if strided:
        assert got.data_ptr() == out.data_ptr() and torch.all(out[..., hd:] == 9.0)
    _check_attend(q, kp, vp, table, lens, got, lse, 1 / math.sqrt(hd), window, cap)


EDGES = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 129, 300, -1]


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (6, 2), (8, 2), (8, 1), (18, 2), (16, 1)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_groups_and_edges(paged, hq, hkv, hd):
    _attend_case(paged, EDGES, hq, hkv, hd, 16, "bf16", "bf16")


@pytest.mark.parametrize("cache,vec", [("f16", "f16"), ("f16", "f32"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("bf16", "f16")])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (10, 1)], ids=["up to 8", "over 8"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_types(paged, cache, vec, hq, hkv, hd):
    _attend_case(paged, [700, 3, 0, 1025, 128], hq, hkv, hd, 32, cache, vec, strided=True)


@pytest.mark.parametrize("vec", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-100, -40, -24, -16, 8, 20, 60])
@pytest.mark.parametrize("hq,hkv,hd", [(8, 2, 64), (4, 2, 128), (16, 1, 128), (12, 1, 64)])
def test_attention_small_and_large_queries_over_fp16_pages(paged, vec, power, hq, hkv, hd):
    """Queries far from 1 in size, with a scale that makes up for it: the same results as at size 1, bit for bit, as
    a power of two is no rounding."""
    g = torch.Generator(device=DEV).manual_seed(13)
    lens = [300, 17, 0, 1]
    kp, vp, table = _make_cache(g, lens, hkv, hd, 16, "f16")
    q = torch.randn(4, hq, hd, generator=g, device=DEV).mul_(1.5).to(TYPES[vec])
    want = paged.paged_attention(q, kp, vp, ints(table), ints(lens), scale=0.125, return_lse=True)
    got = paged.paged_attention((q.float() * 2.0 ** power).to(q.dtype), kp, vp, ints(table), ints(lens),
                                scale=0.125 * 2.0 ** -power, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _check_attend(q, kp, vp, table, lens, *want, 0.125)


@pytest.mark.parametrize("vec", ["f32", "bf16"])
def test_attention_queries_of_unlike_heads_over_fp16_pages(paged, vec):
    """Heads, and elements of a head, of sizes from 1e-9 to 1e5 in one query, zeros and empty heads among them."""
    g = torch.Generator(device=DEV).manual_seed(14)
    lens = [200, 64, 33]
    kp, vp, table = _make_cache(g, lens, 2, 128, 16, "f16")
    q = torch.randn(3, 16, 128, generator=g, device=DEV)
    q[0] *= 10.0 ** -torch.arange(16, device=DEV)[:, None] / 2
    q[1, :, ::3] *= 1e-5
    q[1, :, 1::3] = 0.0
    q[2, 3:6] = 0.0
    q = q.to(TYPES[vec])
    out, lse = paged.paged_attention(q, kp, vp, ints(table), ints(lens), scale=0.2, return_lse=True)
    _check_attend(q, kp, vp, table, lens, out, lse, 0.2)
    q *= 2.0 ** 17
    out, lse = paged.paged_attention(q, kp, vp, ints(table), ints(lens), scale=0.2 * 2.0 ** -17, return_lse=True)
    _check_attend(q, kp, vp, table, lens, out, lse, 0.2 * 2.0 ** -17)


@pytest.mark.parametrize("window,cap", [(1, 0.0), (16, 0.0), (100, 5.0), (1000000, 0.0), (0, 2.0), (33, 30.0)])
@pytest.mark.parametrize("ps", [16, 48, 1024])
def test_attention_windows_caps_and_pages(paged, window, cap, ps):
    _attend_case(paged, EDGES + [1500], 8, 2, 64, ps, "f16", "f32", window, cap)


@pytest.mark.parametrize("lens", [[5000], [20000, 7], [1] * 700, list(range(1, 200)), [0] * 5, [3000] + [2] * 90],
                         ids=["one", "long", "many of one", "rising", "empty", "one among many"])
def test_attention_shapes_of_batches(paged, lens):
    """One long row over every CTA, more rows than a CTA's threads, empty batches, uneven ones."""
    _attend_case(paged, lens, 4, 2, 64, 64, "bf16", "f32")


def test_attention_large_scores_and_minus_infinity(paged):
    """Scores of +-hundreds (the maximum moves far between tiles), rows whose keys hold -inf so that a score
    is -inf, and a row whose scores all are."""
    g = torch.Generator(device=DEV).manual_seed(4)
    kp, vp, table = _make_cache(g, [200, 200, 40], 1, 64, 16, "f16", poison=False)
    kp.mul_(20)
    q = torch.randn(3, 2, 64, generator=g, device=DEV).half()
    q[1:, :, 0] = 1.0
    at = ints(table).long()
    kp[at[1, 3], 0, :, 0] = -math.inf           # positions 48..63 of row 1 score -inf
    kp[at[2, :3], 0, :, 0] = -math.inf          # every position of row 2
    out, lse = paged.paged_attention(q, kp, vp, ints(table), ints([200, 200, 40]), return_lse=True)
    assert torch.all(out[2] == 0) and torch.all(lse[2] == -math.inf)
    kd = kp.clone()
    kd[at[1, 3]] = 0                            # the plain form leaves those positions out
    masked = table.copy()
    masked[1, 3] = -1
    _check_attend(q[:2], kd, vp, masked[:2], [200, 200], out[:2], lse[:2], 0.125)


def test_attention_rows_share_tables(paged):
    """Several queries of one table row at different lengths (a prompt's last positions), with len_add."""
    g = torch.Generator(device=DEV).manual_seed(5)
    kp, vp, table = _make_cache(g, [90, 300], 2, 128, 32, "bf16")
    rows, lens = [1, 1, 0, 1, 1, 0], [299, 298, 89, 0, 17, -1]
    q = torch.randn(6, 4, 128, generator=g, device=DEV).bfloat16()
    out, lse = paged.paged_attention(q, kp, vp, ints(table), ints(lens), rows=ints(rows), len_add=1, return_lse=True)
    _check_attend(q, kp, vp, table, [n + 1 for n in lens], out, lse, 1 / math.sqrt(128), rows=rows)


@pytest.mark.parametrize("hd", [64, 128])
def test_attention_many_tiles_of_a_warp(paged, hd):
    """Queries long enough together that a warp's part passes 32 and 64 tiles, of one table row."""
    g = torch.Generator(device=DEV).manual_seed(6)
    kp, vp, table = _make_cache(g, [20011], 8, hd, 16, "f16")
    lens = [20011 - 13 * i for i in range(16)]
    q = torch.randn(16, 8, hd, generator=g, device=DEV).half()
    out, lse = paged.paged_attention(q, kp, vp, ints(table), ints(lens), rows=ints([0] * 16), return_lse=True)
    _check_attend(q, kp, vp, table, lens, out, lse, 1 / math.sqrt(hd), rows=[0] * 16)


@pytest.mark.parametrize("cache,hd", [("bf16", 64), ("f16", 64), ("bf16", 128), ("f16", 128)])
def test_attention_of_long_batches_does_not_shrink(paged, cache, hd):
    """Many rows over one long sequence, some 900 tiles a warp, 32-bit outputs.  The tensor cores truncate: each of at most
    two products per tile takes up to 2^-23 of the sum so far, half of which 32 tiles have on average before it is
    put away rounded to nearest, 32 * 2^-23 in all, and the rest of the arithmetic is not biased."""
    g = torch.Generator(device=DEV).manual_seed(16)
    R, n = 128, 32768
    kp, vp, table = _make_cache(g, [n], 8, hd, 64, cache, poison=False)
    vp.abs_()                                  # outputs that do not cancel
    q = torch.randn(R, 16, hd, generator=g, device=DEV)
    out, lse = paged.paged_attention(q, kp, vp, ints(table), ints([n] * R), rows=ints([0] * R), return_lse=True)
    at = ints(table)[0, : n // 64].long()
    k, v = (p[at].double().permute(1, 0, 2, 3).reshape(8, n, hd) for p in (kp, vp))
    for r in range(0, R, 32):
        s = torch.einsum("jgd,jtd->jgt", q[r].double().view(8, 2, hd), k) / math.sqrt(hd)
        want = torch.einsum("jgt,jtd->jgd", torch.softmax(s, -1), v).reshape(16, hd)
        shrink = ((out[r].double() * want).sum() / (want * want).sum()).item() - 1
        assert abs(shrink) <= 32 * 2.0 ** -23, (r, shrink)
        assert (lse[r].double() - torch.logsumexp(s, -1).reshape(-1)).abs().max().item() <= 2.0 ** -18


@pytest.mark.parametrize("longest", [150, 400, 900])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_of_as_many_segments_as_ctas(paged, longest, hd):
    """About a CTA per (row, kv head), rows without positions among them: each whole, or in equal shares."""
    lens = [0 if i % 9 == 4 else longest - (17 * i) % (longest // 3) for i in range(52)]
    _attend_case(paged, lens, 8, 8, hd, 32, "bf16", "bf16")


@pytest.mark.parametrize("what", ["page", "negative page", "row", "length"])
def test_attention_reports_and_masks_what_is_not_there(paged, what):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    g = torch.Generator(device=DEV).manual_seed(6)
    lens, rows = [200, 80, 64], [0, 1, 2]
    kp, vp, table = _make_cache(g, lens, 2, 64, 16, "f16")
    if what == "page":
        table[0, 3] = len(kp) + 5
    if what == "negative page":
        table[0, 3] = -7
    if what == "row":
        rows[1] = 3
    if what == "length":
        table = table[:, :6].copy()      # row 0 has 200 positions, the table holds 96
    st = status()
    q = torch.randn(3, 4, 64, generator=g, device=DEV).half()
    out, lse = paged.paged_attention(q, kp, vp, ints(table), ints(lens), rows=ints(rows), return_lse=True, status=st)
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_PAGES and "attention" in str(e.value)
    _check_attend(q, kp, vp, table, lens, out, lse, 0.125, rows=rows)
    paged.paged_attention(q, kp, vp, ints(table), ints(lens), rows=ints(rows))   # no status: not reported, no fault


def test_attention_offsets_past_32_bits(paged):
    """A pool of more than 2^31 elements per plane, strided over a larger allocation; the sequence's pages lie
    at both of its ends.  The append finds the same places."""
    hkv, ps, hd = 2, 64, 128
    n_pages = 2 ** 31 // (hkv * ps * hd) + 40
    pool = torch.empty(2, n_pages, hkv, ps, hd, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(7)
    ids = [n_pages - 1, 0, n_pages // 2, n_pages - 2]
    small = torch.randn(2, 4, hkv, ps, hd, generator=g, device=DEV).bfloat16()
    k = torch.randn(1, hkv, hd, generator=g, device=DEV).bfloat16()
    pool[:, ids] = small
    table, few = ints([ids]), ints([[0, 1, 2, 3]])
    for pages, t in ((pool, table), (small, few)):
        paged.rope_append(None, k, k, pages[0], pages[1], t, ints([199]))
        paged.rope_append(None, k, k, pages[0], pages[1], t, ints([5]))
    assert torch.equal(pool[:, ids], small)
    q = torch.randn(1, 4, hd, generator=g, device=DEV).bfloat16()
    a = paged.paged_attention(q, pool[0], pool[1], table, ints([200]), return_lse=True)
    b = paged.paged_attention(q, small[0], small[1], few, ints([200]), return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attention_repeats_bit_for_bit_and_replays(paged):
    """The same call twice, captured and replayed with new lengths and queries, and two captured graphs
    replayed at the same time on two streams."""
    g = torch.Generator(device=DEV).manual_seed(8)
    lens = [3000, 1, 700, 0, 2222]
    kp, vp, table = _make_cache(g, lens, 8, 128, 64, "bf16")
    tb = ints(table)
    qs = [torch.randn(5, 16, 128, generator=g, device=DEV).bfloat16() for _ in range(2)]
    ls = [ints(lens), ints([17, 0, 699, 0, 2000])]
    want = [paged.paged_attention(q, kp, vp, tb, n, return_lse=True) for q, n in zip(qs, ls)]
    again = paged.paged_attention(qs[0], kp, vp, tb, ls[0], return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(want[0], again))
    q, n = qs[0].clone(), ls[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = paged.paged_attention(q, kp, vp, tb, n, return_lse=True)
    for i in (0, 1, 0):
        q.copy_(qs[i])
        n.copy_(ls[i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want[i], got))
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(paged.paged_attention(qs[i], kp, vp, tb, ls[i], return_lse=True))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(50):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(want[i], outs[i]))


# ---------------------------------------------------------------------------- page updates
class _Gpu:
    """A GPU state beside a plain one; a page's cells hold a value that its copies carry along."""

    def __init__(self, rows, width, n_pages, ps, layers=2, hkv=2, hd=64, dtype=torch.bfloat16, stride=0):
        self.plain = Pages(rows, width, n_pages, ps)
        cells = torch.zeros(2, layers, n_pages + stride, hkv, ps, hd, dtype=dtype, device=DEV)
        self.k, self.v = cells[0][:, :n_pages], cells[1][:, :n_pages]
        self.k.copy_(torch.arange(n_pages, device=DEV).view(1, -1, 1, 1, 1) % 200)
        self.v.copy_(-1 - self.k)
        for l in range(layers):
            self.k[l] += 0.25 * l
        wide = torch.full((rows, width + stride), -1, dtype=torch.int32, device=DEV)
        self.table = wide[:, :width]
        self.lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        self.status = status()
        self.want_k, self.want_v = self.k.clone(), self.v.clone()

    def put(self):
        self.table.copy_(torch.as_tensor(self.plain.table))
        self.lens.copy_(torch.as_tensor(self.plain.lens))
        self.refs.copy_(torch.as_tensor(self.plain.refs))

    def update(self, paged, parents, reserve):
        copies = self.plain.update(parents, reserve)
        paged.update_pages(self.k, self.v, self.table, self.lens, self.refs, parents=ints(parents), reserve=ints(reserve),
                           status=self.status)
        if copies:
            src, dst = (torch.tensor(x, device=DEV) for x in zip(*copies))
            for t in (self.want_k, self.want_v):
                t[:, dst] = t[:, src]
        return copies

    def same(self):
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.plain.table)
        np.testing.assert_array_equal(self.lens.cpu().numpy(), self.plain.lens)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.plain.refs)
        assert torch.equal(self.k, self.want_k) and torch.equal(self.v, self.want_v)


@pytest.mark.parametrize("rows,width,n_pages,ps", [(1, 3, 4, 16), (6, 5, 17, 16), (40, 9, 200, 48), (130, 300, 9000, 16)])
def test_update_follows_the_plain_bookkeeping(paged, rows, width, n_pages, ps):
    """Random forks, frees and reservations, among them ones that do not fit and are refused whole."""
    from persistent_sm_decode_megakernel_gb300 import MkError
    rng = np.random.default_rng(rows)
    s = _Gpu(rows, width, n_pages, ps, stride=3)
    refused = 0
    for step in range(40):
        parents = rng.integers(-1, rows, rows) if step % 3 else np.arange(rows)
        reserve = rng.integers(0, 2 * ps if rows < 100 else 60 * ps, rows) * (rng.random(rows) < 0.7)
        if s.update(paged, parents, reserve) is None:
            refused += 1
            with pytest.raises(MkError):
                paged.check_status(s.status)
        else:
            for r in range(rows):
                if parents[r] >= 0:
                    s.plain.lens[r] += rng.integers(0, reserve[r] + 1)
            s.lens.copy_(torch.as_tensor(s.plain.lens))
            paged.check_status(s.status)
        s.same()
    assert refused < 40


@pytest.mark.parametrize("parents", [[0, 5], [0, -2], [2, 0]])
def test_update_refuses_parents_that_are_none(paged, parents):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    s = _Gpu(2, 4, 12, 16)
    s.update(paged, [0, 1], [20, 30])
    s.plain.lens[:] = [20, 30]
    s.put()
    assert s.update(paged, parents, [1, 1]) is None
    with pytest.raises(MkError) as e:
        paged.check_status(s.status)
    assert e.value.status == MK_ERR_PAGES
    s.same()


def test_update_refuses_lengths_past_the_table_and_bad_lengths(paged):
    from persistent_sm_decode_megakernel_gb300 import MkError
    s = _Gpu(2, 2, 12, 16)
    assert s.update(paged, [0, 1], [32, 33]) is None       # 33 positions, a table of 32
    with pytest.raises(MkError):
        paged.check_status(s.status)
    s.same()
    assert s.update(paged, [0, 1], [2 ** 31 - 1, 1]) is None
    with pytest.raises(MkError):
        paged.check_status(s.status)
    s.same()
    for bad in (-1, 33):
        s.lens[1] = bad
        paged.update_pages(s.k, s.v, s.table, s.lens, s.refs, reserve=ints([1, 1]), status=s.status)
        with pytest.raises(MkError):
            paged.check_status(s.status)
        assert s.lens.tolist() == [0, bad] and int(s.refs.sum()) == 0
        s.lens[1] = 0
    s.same()


def test_update_with_holders_outside_the_table_and_bad_entries(paged):
    """A page that something else holds as well is copied by every row that will write into it; an entry that
    names no page is reported and dropped."""
    from persistent_sm_decode_megakernel_gb300 import MkError
    s = _Gpu(3, 3, 20, 16)
    s.update(paged, [0, 1, 2], [20, 0, 0])
    s.plain.lens[0] = 20
    s.plain.refs[1] += 1          # held from outside: the partly filled page
    s.put()
    copies = s.update(paged, [0, 0, 0], [1, 1, 0])
    assert len(copies) == 2
    paged.check_status(s.status)
    s.same()
    s.table[2, 0] = 99
    s.plain.table[2, 0] = -1
    s.plain.refs[0] -= 1
    s.refs[0] -= 1
    s.update(paged, [0, 1, 2], [0, 0, 0])
    with pytest.raises(MkError):
        paged.check_status(s.status)
    s.same()


def test_update_without_parents_or_reservations(paged):
    s = _Gpu(2, 4, 12, 16)
    s.update(paged, [0, 1], [20, 30])
    s.plain.lens[:] = [20, 17]
    s.put()
    s.plain.update([0, 1], [0, 0])
    paged.update_pages(s.k, s.v, s.table, s.lens, s.refs)
    s.same()


def test_update_of_the_largest_table_of_rows(paged):
    """4096 rows: groups of eight that fork from one of them each, with the copies of their last pages."""
    s = _Gpu(4096, 3, 20000, 16, layers=1, hkv=1)
    s.update(paged, list(range(4096)), [20] * 4096)
    s.plain.lens[:] = 20
    s.put()
    s.same()
    parents = [r // 8 * 8 + (r * 5 + r // 8) % 8 // 3 for r in range(4096)]
    copies = s.update(paged, parents, [1] * 4096)
    assert len(copies) > 1000
    s.same()
    paged.check_status(s.status)


@pytest.mark.parametrize("n_pages,held", [(1, 1), (7, 0), (40, 13), (9000, 4000)])
def test_compact_moves_the_held_pages_down(paged, n_pages, held):
    rng = np.random.default_rng(n_pages)
    ids = rng.permutation(n_pages)[:held]
    s = _Gpu(3, max(1, -(-held // 2)), n_pages, 16, stride=2)
    flat = -np.ones(3 * s.table.shape[1], dtype=np.int32)
    flat[:held] = ids
    if held > 3:
        flat[-2:] = ids[:2]                       # pages shared by two rows
    table = flat.reshape(3, -1)
    refs = np.bincount(flat[flat >= 0], minlength=n_pages)
    s.table.copy_(torch.as_tensor(table))
    s.refs.copy_(torch.as_tensor(refs))
    used = int((refs > 0).sum())
    src = [i for i in range(used, n_pages) if refs[i]]
    dst = [i for i in range(used) if not refs[i]]
    to = {a: b for a, b in zip(src, dst)}
    before_k, before_v = s.k.clone(), s.v.clone()
    paged.compact_pages(s.k, s.v, s.table, s.refs, status=s.status)
    paged.check_status(s.status)
    want = np.array([to.get(i, i) for i in table.reshape(-1)]).reshape(table.shape)
    np.testing.assert_array_equal(s.table.cpu().numpy(), want)
    np.testing.assert_array_equal(s.refs.cpu().numpy(), np.bincount(want[want >= 0], minlength=n_pages))
    for now, old in ((s.k, before_k), (s.v, before_v)):
        for l in range(now.shape[0]):
            live = want >= 0
            assert torch.equal(now[l][ints(want[live]).long()], old[l][ints(table[live]).long()])


def test_compact_reports_an_entry_that_names_no_page(paged):
    from persistent_sm_decode_megakernel_gb300 import MkError
    s = _Gpu(1, 3, 8, 16)
    s.table.copy_(ints([[6, 50, -1]]))
    s.refs[6] = 1
    paged.compact_pages(s.k, s.v, s.table, s.refs, status=s.status)
    with pytest.raises(MkError):
        paged.check_status(s.status)
    assert s.table.tolist() == [[0, 50, -1]] and s.refs.tolist() == [1] + [0] * 7


# ------------------------------------------------------------------------------- selection
def _check_select(got, logits, scores, ended, eos):
    """Tokens, beams and flags as the plain form's; a score is the 64-bit sum rounded to 32, whose lse is off
    by no more than 2^-19: each exponential by 2^-22 and its argument's rounding, x 2^-24, of its share."""
    groups, beams = scores.shape
    lg, sc, en = f64(logits).reshape(groups, beams, -1), f64(scores), ended.cpu().numpy()
    token, parent, best, done = (t.cpu().numpy() for t in got)
    for g in range(groups):
        want = select(lg[g], sc[g], en[g], eos)
        assert token[g].tolist() == [w[0] for w in want], g
        assert parent[g].tolist() == [g * beams + w[1] for w in want], g
        assert done[g].tolist() == [int(w[3]) for w in want], g
        for s, w in zip(best[g], want):
            assert s == w[2] or abs(s - w[2]) <= 2.0 ** -24 * abs(w[2]) + 2.0 ** -19, (g, s, w)


def _select_inputs(groups, beams, vocab, dtype, done=0.0, seed=1, scale=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = torch.randn(groups * beams, vocab, generator=g, device=DEV).mul_(scale).to(TYPES[dtype])
    scores = -20 * torch.rand(groups, beams, generator=g, device=DEV)
    ended = (torch.rand(groups, beams, generator=g, device=DEV) < done).int()
    return logits, scores, ended


@pytest.mark.parametrize("beams,vocab", [(1, 1), (1, 50), (3, 3), (4, 1000), (5, 2049), (8, 8193), (16, 30001), (32, 32), (32, 40000)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_select_sizes_and_types(paged, beams, vocab, dtype):
    """Odd vocabularies; 16-bit logits tie often, and ties go to the lowest token."""
    x = _select_inputs(3, beams, vocab, dtype, 0.2)
    _check_select(paged.beam_select(*x, eos=0), *x, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_many_rows_and_strided_logits(paged, dtype):
    """Enough rows for the large chunks; rows at an odd stride, off any 16-byte boundary."""
    x = list(_select_inputs(40, 4, 9001, dtype, 0.1))
    _check_select(paged.beam_select(*x, eos=7), *x, 7)
    wide = torch.full((160, 9003), 99.0, dtype=x[0].dtype, device=DEV)
    wide[:, 1:9002] = x[0]
    got = paged.beam_select(wide[:, 1:9002], x[1], x[2], eos=7)
    _check_select(got, *x, 7)


@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "signed zeros", "few values", "stripes"])
@pytest.mark.parametrize("beams,groups", [(8, 1), (32, 1), (32, 8)])
def test_select_ties_and_layouts_of_the_large_logits(paged, kind, beams, groups):
    """All equal, sorted both ways, +-0, three values, and all large logits in a few lanes of each warp (more
    candidates above the threshold than the list holds)."""
    vocab = 20000
    i = torch.arange(vocab, device=DEV)
    row = {"equal": torch.zeros(vocab, device=DEV), "rising": i / 1000.0, "falling": -i / 1000.0,
           "signed zeros": torch.where(i % 2 == 0, -0.0, 0.0), "few values": (i * 7919 % 3).float(),
           "stripes": torch.where(i // 4 % 32 < beams - 1, (i * 37 % 1009) / 100.0, -5.0 - (i % 7))}[kind]
    logits = row.repeat(groups * beams, 1)
    scores = torch.zeros(groups, beams, device=DEV) - torch.arange(beams, device=DEV) * (0.0 if kind == "equal" else 0.01)
    ended = torch.zeros(groups, beams, dtype=torch.int32, device=DEV)
    _check_select(paged.beam_select(logits, scores, ended), logits, scores, ended, -1)


@pytest.mark.parametrize("kind", ["few allowed", "half masked", "others lowest", "thin mask", "rising", "best first, then rising"])
@pytest.mark.parametrize("groups,beams,vocab", [(16, 8, 70000), (2, 32, 32000), (1, 4, 9001)])
def test_select_masked_and_rising_parts_of_several_steps(paged, kind, groups, beams, vocab):
    """Masks that leave few tokens, none of the first half, one of a thousand, the type's lowest in the place of
    -inf; logits of which ever more enter the list, with and without its first entries staying the best."""
    logits, scores, ended = _select_inputs(groups, beams, vocab, "f32", seed=9)
    i = torch.arange(vocab, device=DEV)
    if kind == "few allowed":
        logits[:, (i < 100) | (i >= 105)] = -math.inf
    elif kind == "half masked":
        logits[:, : vocab // 2] = -math.inf
    elif kind == "others lowest":
        logits[:, 5 + beams:] = torch.finfo(torch.float32).min
    elif kind == "thin mask":
        logits[:, i % 1000 != 7] = -math.inf
    else:
        logits[:] = -5.0 + i / 16384.0 + (logits - logits.min()) * 1e-7
        if kind != "rising":
            logits[:, : beams - 1] = 60.0 - i[: beams - 1] / 8.0
    _check_select(paged.beam_select(logits, scores, ended), logits, scores, ended, -1)


def test_select_minus_infinity(paged):
    """Masked tokens, a row with fewer finite logits than beams, a row without any, beams that are not alive yet
    (score -inf, as at the first step), and ended beams among them."""
    logits, scores, ended = _select_inputs(4, 4, 500, "f32")
    logits[:, 100:] = -math.inf
    logits[4:8, 2:] = -math.inf
    logits[8] = -math.inf
    logits[12:, :] = -math.inf
    scores[0, 1:] = -math.inf
    scores[2, 3] = -math.inf
    ended[1, 2] = 1
    ended[3, 1] = 1
    _check_select(paged.beam_select(logits, scores, ended, eos=3), logits, scores, ended, 3)
    ended[:] = 1
    _check_select(paged.beam_select(logits, scores, ended, eos=3), logits, scores, ended, 3)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_select_reports_nan_and_plus_infinity(paged, bad):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_NAN, MkError
    logits, scores, ended = _select_inputs(2, 3, 5000, "f32")
    logits[4, 4321] = bad
    st = status()
    got = paged.beam_select(logits, scores, ended, status=st)
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_NAN and "row 4" in str(e.value)
    logits[4, 4321] = -math.inf
    _check_select(got, logits, scores, ended, -1)
    scores[0, 1] = math.nan
    got = paged.beam_select(logits, scores, ended, status=st)
    with pytest.raises(MkError):
        paged.check_status(st)
    scores[0, 1] = -math.inf
    _check_select(got, logits, scores, ended, -1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_wide_ranges(paged, dtype):
    """Logits of thousands (all but one of the exponentials vanish), all far below zero, and one above 2^126,
    which is reported."""
    from persistent_sm_decode_megakernel_gb300 import MkError
    logits, scores, ended = _select_inputs(3, 3, 3000, dtype)
    logits[:3] *= 2000
    logits[3:6] -= 20000
    _check_select(paged.beam_select(logits, scores, ended), logits, scores, ended, -1)
    logits[7, 5] = 2e38
    st = status()
    got = paged.beam_select(logits, scores, ended, status=st)
    with pytest.raises(MkError):
        paged.check_status(st)
    logits[7, 5] = -math.inf
    _check_select(got, logits, scores, ended, -1)
    logits[6:9] = -3e38                       # a row below -2^126: like one at -inf
    got = paged.beam_select(logits, scores, ended, status=st)
    paged.check_status(st)
    logits[6:9] = -math.inf
    _check_select(got, logits, scores, ended, -1)


# --------------------------------------------------------------- selection over finite masks
def _select_exact(logits, scores, ended, eos):
    """The selection in 64 bits on the GPU, with log softmax as (x - max) - log sum e^(x - max): the maximum of a
    row of large logits takes nothing from the sum."""
    groups, beams = scores.shape
    x = logits.double()
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    lsum = torch.exp(x - top).sum(-1, keepdim=True).log()
    best, token = torch.sort(x, dim=-1, descending=True, stable=True)
    best, token = best[:, :beams], token[:, :beams]
    s, done = scores.double().view(-1, 1), ended.view(-1, 1) != 0
    key = torch.where(best == -math.inf, -math.inf, s + ((best - top) - lsum))
    first = torch.arange(beams, device=DEV)[None] == 0
    key = torch.where(done, torch.where(first, s, -math.inf), key).view(groups, -1)
    token = torch.where(done, eos, token).view(groups, -1)
    key, at = torch.sort(key, dim=-1, descending=True, stable=True)
    key, at = key[:, :beams], at[:, :beams]
    return token.gather(1, at), torch.arange(groups, device=DEV)[:, None] * beams + at // beams, key


def _check_select_exact(got, logits, scores, ended, eos=-1):
    """As _check_select, against _select_exact."""
    token, parent, key = _select_exact(logits, scores, ended, eos)
    assert torch.equal(got[0].long(), token)
    assert torch.equal(got[1].long(), parent)
    off, same = (got[2].double() - key).abs(), got[2].double() == key
    assert torch.all(same | (off <= 2.0 ** -24 * key.abs() + 2.0 ** -19)), off[~same].max()


MASKS = [-1e4, -1e9, -1e10, -1e12, -1e18, -1e20, -1e30]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("kind", ["allowed first", "allowed last", "half", "three quarters", "thin"])
@pytest.mark.parametrize("groups,beams,vocab,dtype", [(16, 8, 70000, "f32"), (16, 8, 70001, "bf16"), (2, 32, 32000, "f32"),
                                                      (1, 4, 9001, "f32"), (1, 4, 9001, "bf16")])
def test_select_finite_masks(paged, mask, kind, groups, beams, vocab, dtype):
    """A mask that is a large negative number, in parts of one step and of several, with the allowed tokens in
    the first or in the last step, behind masked steps, or in between: a masked logit's exponential is 0."""
    logits, scores, ended = _select_inputs(groups, beams, vocab, dtype, seed=3)
    i = torch.arange(vocab, device=DEV)
    allowed = {"allowed first": (i >= 3) & (i < 43), "allowed last": i >= vocab - 41, "half": i >= vocab // 2,
               "three quarters": i >= vocab * 3 // 4, "thin": i % 500 == 7}[kind]
    if kind == "thin" and vocab < 500 * beams:
        allowed = i % 50 == 7
    logits[:, ~allowed] = mask
    _check_select_exact(paged.beam_select(logits, scores, ended), logits, scores, ended)


@pytest.mark.parametrize("value", MASKS + [1e9, 1e10, 1e18, 8e37, -8e37])
@pytest.mark.parametrize("groups,beams,vocab,dtype", [(16, 8, 70000, "f32"), (16, 8, 70000, "bf16"), (1, 4, 9001, "f32"),
                                                      (2, 3, 50, "bf16")])
def test_select_rows_of_one_large_value(paged, value, groups, beams, vocab, dtype):
    """Rows whose every logit is one value offer each token at -ln(vocab), whatever the value; live rows among them."""
    logits, scores, ended = _select_inputs(groups, beams, vocab, dtype, seed=4)
    logits[::2] = value
    _check_select_exact(paged.beam_select(logits, scores, ended), logits, scores, ended)


@pytest.mark.parametrize("value", [1e9, 1e10, 1e18, 1e30])
@pytest.mark.parametrize("at", [0, 5000, 69999])
def test_select_one_large_logit(paged, value, at):
    """One logit far above the others takes the whole sum, in a part of its own or not."""
    logits, scores, ended = _select_inputs(16, 8, 70000, "f32", seed=5)
    logits[:, at] = value
    _check_select_exact(paged.beam_select(logits, scores, ended), logits, scores, ended)


@pytest.mark.parametrize("power", [12, 18, 20, 21, 22])
@pytest.mark.parametrize("sign", [1, -1])
def test_select_rows_around_a_power_of_two(paged, power, sign):
    """Rows that lie within a few hundred of +-2^power: their largest logits are a step of 32 bits apart there, and
    count for the sum on both sides of it.  (Ties are frequent; they go to the lowest token and beam.)"""
    g = torch.Generator(device=DEV).manual_seed(power)
    x = (torch.rand(24, 40000, generator=g, device=DEV, dtype=torch.float64) - 0.5) * 600 + sign * 2.0 ** power
    x[:, ::1000] = sign * 2.0 ** power + 300 + torch.arange(40, device=DEV)
    x[1::3, :30000] -= 2000
    scores = -20 * torch.rand(6, 4, generator=g, device=DEV)
    ended = torch.zeros(6, 4, dtype=torch.int32, device=DEV)
    logits = x.float()
    _check_select_exact(paged.beam_select(logits, scores, ended), logits, scores, ended)


def test_select_large_steps_that_rise(paged):
    """A row whose steps' largest logits go from -1e30 over -1e9, 0 and 1e9 to 1e30, a few equal ones in each."""
    logits, scores, ended = _select_inputs(8, 4, 90000, "f32", seed=6)
    for k, v in enumerate([-1e30, -1e9, None, 1e9, 1e30]):
        if v is not None:
            logits[:, 18000 * k: 18000 * (k + 1)] = v
    for top in (5, 4, 3, 2, 1):
        _check_select_exact(paged.beam_select(logits[:, : 18000 * top], scores, ended), logits[:, : 18000 * top], scores, ended)


@pytest.mark.parametrize("place", [0.0, 0.3, 0.9])
@pytest.mark.parametrize("groups,beams,vocab,dtype", [(1, 8, 1000, "f32"), (1, 8, 20000, "f32"), (16, 8, 70000, "f32"),
                                                      (16, 8, 70000, "bf16"), (2, 3, 300, "bf16"), (2, 3, 20000, "bf16")])
def test_select_of_fewer_tokens_than_beams_over_the_lowest_mask(paged, place, groups, beams, vocab, dtype):
    """One live beam, two allowed tokens, the type's lowest in the place of -inf: what is below -2^126 counts as
    -inf wherever it lies, and of equal logits the lowest tokens are chosen."""
    logits, scores, ended = _select_inputs(groups, beams, vocab, dtype, seed=7)
    i, at = torch.arange(vocab, device=DEV), int(place * vocab)
    logits[:, (i < at) | (i >= at + 2)] = torch.finfo(logits.dtype).min
    logits[:, (i % 2 == 1) & (i != at) & (i != at + 1)] = -math.inf
    scores[:, 1:] = -math.inf
    got = paged.beam_select(logits, scores, ended)
    logits[logits < -2.0 ** 126] = -math.inf
    _check_select_exact(got, logits, scores, ended)
    logits[:, at: at + 2] = -math.inf
    lowest = torch.full_like(logits, torch.finfo(logits.dtype).min)
    _check_select_exact(paged.beam_select(lowest, scores, ended), logits, scores, ended)


@pytest.mark.parametrize("vocab", [500, 20000])
def test_select_sums_beyond_the_range_of_32_bits(paged, vocab):
    """Scores and logits whose sum lies below the lowest float: such a candidate's score is -inf, and not NaN."""
    logits, scores, ended = _select_inputs(2, 4, vocab, "f32", seed=8)
    scores[:] = -3.3e38 + torch.arange(4, device=DEV) * 1e37
    logits[:, 3:] = -8e37
    logits[4:, 1:] = -8e37
    got = paged.beam_select(logits, scores, ended)
    token, parent, key = _select_exact(logits, scores, ended, -1)
    assert torch.equal(got[0].long(), token) and torch.equal(got[1].long(), parent)
    assert torch.equal(got[2], key.float())
    scores[:, 1:] = -math.inf
    got = paged.beam_select(logits, scores, ended)
    token, parent, key = _select_exact(logits, scores, ended, -1)
    assert torch.equal(got[0].long(), token) and torch.equal(got[1].long(), parent)
    assert torch.equal(got[2], key.float()) and key.float().isneginf().any()


def test_select_orders_beams_up_to_the_accuracy_of_their_sums(paged):
    """Beams of identical rows and equal scores tie: the lower beam's tokens come first.  Rows that are permutations of
    one another have the same exact log-sum-exp, which each of them sees to 2^-19 (as _check_select says): their
    beams come in order once the scores are further apart than twice that, and below in an order of their own, with
    scores that are right all the same."""
    logits, _, _ = _select_inputs(1, 1, 30000, "f32", seed=10)
    ended = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    rows = logits.expand(12, -1).contiguous()
    scores = torch.full((3, 4), -3.25, device=DEV)
    token, parent, best, _ = paged.beam_select(rows, scores, ended)
    top = int(logits.argmax())
    assert token.tolist() == [[top] * 4] * 3 and parent.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11]]
    assert torch.all(best == best[0, 0])
    g = torch.Generator(device=DEV).manual_seed(11)
    perms = [torch.randperm(30000, generator=g, device=DEV) for _ in range(12)]
    rows = torch.stack([logits[0][p] for p in perms])
    want = (logits.double().amax() - torch.logsumexp(logits.double(), -1)).item() - 3.25
    for gap in (0.0, 2.0 ** -24, 2.0 ** -16):
        scores = torch.full((3, 4), -3.25, device=DEV) + gap * torch.arange(4, device=DEV)
        token, parent, best, _ = paged.beam_select(rows, scores, ended)
        assert torch.all((best.double() - want - (scores.double() + 3.25).gather(1, parent.long() % 4)).abs() <= 2.0 ** -24 * 16 + 2.0 ** -19)
        assert sorted(parent.flatten().tolist()) == list(range(12))
        assert all(int(perms[p][t]) == top for p, t in zip(parent.flatten().tolist(), token.flatten().tolist()))
        if gap > 2.0 ** -18:
            assert parent.tolist() == [[3, 2, 1, 0], [7, 6, 5, 4], [11, 10, 9, 8]]


# ------------------------------------------------------------------------------ refusals
def test_tensors_that_do_not_fit_are_refused(paged):
    """Shapes, types, layouts and devices, each refused before anything is enqueued."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_INVALID, MkError
    pages = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    k, v = pages
    table, lens, pos = ints([[0, 1], [2, 3]]), ints([5, 6]), ints([1, 2])
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    f = torch.zeros(32, dtype=torch.float64, device=DEV)
    append = lambda **a: paged.rope_append(**{**dict(q=q, k=kv, v=kv, k_pages=k, v_pages=v, table=table, positions=pos), **a})
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[..., :32]), dict(k=kv[:, :1]), dict(v=kv.half()),
                dict(k=kv.transpose(1, 2)), dict(positions=pos.long()), dict(positions=pos[:1]), dict(positions=pos.cpu()),
                dict(rows=pos.float()), dict(freqs=f.float()), dict(freqs=f.cpu()), dict(freqs=f[None]), dict(table=table.long()),
                dict(table=table[0]), dict(table=table.t()), dict(v_pages=v[:2]), dict(k_pages=k.float(), v_pages=v.float()),
                dict(k_pages=k.transpose(1, 2), v_pages=v.transpose(1, 2)), dict(q_out=q.float()), dict(q=None, q_out=q),
                dict(status=torch.zeros(3, dtype=torch.int32, device=DEV)), dict(k=kv.cpu()), dict(k=3), dict(q=[1])):
        with pytest.raises(ValueError):
            append(**bad)
    with pytest.raises(MkError) as e:
        append(freqs=torch.zeros(33, dtype=torch.float64, device=DEV))
    assert e.value.status == MK_ERR_INVALID
    attend_ = lambda **a: paged.paged_attention(**{**dict(q=q, k_pages=k, v_pages=v, table=table, lens=lens), **a})
    for bad in (dict(q=q[0]), dict(q=q.double()), dict(lens=lens[:1]), dict(lens=lens.long()), dict(out=q.float()),
                dict(out=q[:1]), dict(rows=lens[:1]), dict(window=2 ** 40), dict(q=q.to_sparse())):
        with pytest.raises(ValueError):
            attend_(**bad)
    for bad in (dict(window=-1), dict(softcap=-2.0), dict(scale=math.nan), dict(q=q[:, :3])):
        with pytest.raises(MkError):
            attend_(**bad)
    refs = ints([1] * 4)
    update = lambda **a: paged.update_pages(**{**dict(k=k[None], v=v[None], table=table, lens=lens, refs=refs), **a})
    for bad in (dict(k=k), dict(refs=refs[:3]), dict(lens=lens[:1]), dict(parents=lens.long()), dict(reserve=lens[:1]),
                dict(v=v[None].half())):
        with pytest.raises(ValueError):
            update(**bad)
    x = torch.zeros(6, 10, device=DEV)
    s, n = torch.zeros(2, 3, device=DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for bad in ((x[:5], s, n), (x.t(), s, n), (x, s.double(), n), (x, s, n.long()), (x, s[:, :2], n), (x.long(), s, n), (x, s.t(), n)):
        with pytest.raises(ValueError):
            paged.beam_select(*bad)
    with pytest.raises(MkError):
        paged.beam_select(x[:, :2], s, n)
    with pytest.raises(MkError):
        paged.beam_select(x, s, n, eos=10)
    assert paged.paged_attention(q[:0], k, v, table, lens[:0]).shape == (0, 4, 64)
    assert paged.rope_append(q[:0], kv[:0], kv[:0], k, v, table, pos[:0]).shape == (0, 4, 64)
    torch.cuda.synchronize()
    assert pages.abs().sum() == 0


def test_what_is_written_in_place_counts_as_changed(paged):
    """The version of every tensor a call writes goes up, and of no other, so that torch refuses a backward pass over
    what a call has changed since; tensors of inference mode have none and are taken as they are."""
    g = torch.Generator(device=DEV).manual_seed(15)
    pages = torch.randn(2, 1, 6, 2, 16, 64, generator=g, device=DEV).bfloat16()
    k, v = pages[0].clone(), pages[1].clone()
    table, lens, refs, st = ints([[0, 1], [2, 3]]), ints([5, 20]), ints([1, 1, 1, 1, 0, 0]), status()
    q, kv = torch.randn(2, 4, 64, generator=g, device=DEV).bfloat16(), torch.randn(2, 2, 64, generator=g, device=DEV).bfloat16()
    out, pos, rows = torch.zeros_like(q), ints([1, 2]), ints([0, 1])
    logits, scores, ended = torch.randn(2, 50, generator=g, device=DEV), torch.zeros(1, 2, device=DEV), ints([[0, 0]])
    named = dict(k=k, v=v, table=table, lens=lens, refs=refs, st=st, q=q, kv=kv, out=out, pos=pos, rows=rows,
                 logits=logits, scores=scores, ended=ended)

    def written(call):
        before = {n: t._version for n, t in named.items()}
        call()
        return {n for n, t in named.items() if t._version > before[n]}

    assert written(lambda: paged.rope_append(q, kv, kv, k[0], v[0], table, pos, rows=rows)) == {"k", "v"}
    assert written(lambda: paged.rope_append(q, kv, kv, k[0], v[0], table, pos, q_out=out, status=st)) == {"k", "v", "out", "st"}
    assert written(lambda: paged.rope_append(q[:0], kv[:0], kv[:0], k[0], v[0], table, pos[:0], q_out=out[:0], status=st)) == set()
    assert written(lambda: paged.paged_attention(q, k[0], v[0], table, lens)) == set()
    assert written(lambda: paged.paged_attention(q, k[0], v[0], table, lens, out=out, status=st)) == {"out", "st"}
    assert written(lambda: paged.update_pages(k, v, table, lens, refs)) == {"k", "v", "table", "lens", "refs"}
    assert written(lambda: paged.compact_pages(k, v, table, refs, status=st)) == {"k", "v", "table", "refs", "st"}
    assert written(lambda: paged.beam_select(logits, scores, ended)) == set()
    assert written(lambda: paged.check_status(st)) == set()
    w = torch.ones(64, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    y = (w * k).sum()                          # its backward pass wants k as it is now
    paged.rope_append(None, kv, kv, k[0], v[0], table, pos)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        k2, v2 = pages[0].clone(), pages[1].clone()
    paged.rope_append(None, kv, kv, k2[0], v2[0], table, pos)
    assert torch.equal(k2[0, 0, :, 1], kv[0])


def test_outputs_that_share_memory_are_refused(paged):
    """An expanded q_out or out, whose rows are one and the same memory."""
    from persistent_sm_decode_megakernel_gb300 import MkError
    pages = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    q, kv = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV), torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    table, pos = ints([[0], [1], [2]]), ints([1, 2, 3])
    for out in (q[:1].clone().expand(3, 4, 64), q[:, :1].clone().expand(3, 4, 64)):
        with pytest.raises(MkError):
            paged.rope_append(q, kv, kv, *pages, table, pos, q_out=out)
        with pytest.raises(MkError):
            paged.paged_attention(q, *pages, table, pos, out=out)
    torch.cuda.synchronize()
    assert not pages.any()
    assert torch.equal(paged.rope_append(q[:1], kv[:1], kv[:1], *pages, table, pos[:1]), q[:1])


# ------------------------------------------------------------------------------ all of them
def test_a_beam_search_of_the_four_operators_captured(paged):
    """Steps as a beam search makes them -- reserve and fork, append, attend, select -- eagerly and as one
    replayed graph, with the same tokens, tables, counts and pages; the eager ones against a search that keeps
    every beam's keys and values in a list of its own."""
    G, K, hq, hkv, hd, ps, vocab, steps = 2, 3, 4, 2, 64, 16, 97, 20
    R = G * K
    g = torch.Generator(device=DEV).manual_seed(11)
    emb = torch.randn(vocab, (hq + 2 * hkv) * hd, generator=g, device=DEV).mul_(0.7)
    head = torch.randn(hq * hd, vocab, generator=g, device=DEV).mul_(0.6)
    freqs, _ = paged.rope_freqs(10000.0, hd, device=DEV)
    first = ints([5, 9]).repeat_interleave(K)

    class Search:
        def __init__(self):
            self.pages = torch.zeros(2, 1, 64, hkv, ps, hd, dtype=torch.bfloat16, device=DEV)
            self.table = torch.full((R, 4), -1, dtype=torch.int32, device=DEV)
            self.lens, self.refs = torch.zeros(R, dtype=torch.int32, device=DEV), torch.zeros(64, dtype=torch.int32, device=DEV)
            self.parents, self.one = ints(range(R)), ints([1] * R)
            self.tokens = first.clone()
            self.scores = torch.full((G, K), -math.inf, device=DEV)
            self.scores[:, 0] = 0.0
            self.ended, self.status = torch.zeros(G, K, dtype=torch.int32, device=DEV), status()

        def step(self):
            k, v = self.pages
            paged.update_pages(k, v, self.table, self.lens, self.refs, self.parents, self.one, status=self.status)
            x = emb[self.tokens.long()].view(R, hq + 2 * hkv, hd)
            q = paged.rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], k[0], v[0], self.table, self.lens,
                                  freqs=freqs, status=self.status)
            o = paged.paged_attention(q, k[0], v[0], self.table, self.lens, len_add=1, status=self.status)
            logits = (o.view(R, -1) @ head) * 3
            tok, par, sc, en = paged.beam_select(logits, self.scores, self.ended, eos=1, status=self.status)
            self.lens += 1
            self.tokens.copy_(tok.view(-1))
            self.parents.copy_(par.view(-1))
            self.scores.copy_(sc)
            self.ended.copy_(en)
            return logits

        def state(self):
            return [t.clone() for t in (self.pages, self.table, self.lens, self.refs, self.tokens, self.parents, self.scores, self.ended)]

    s = Search()
    seqs = [[] for _ in range(R)]                       # the tokens each row has consumed
    states = []
    e64, h64 = emb.double(), head.double()
    for t in range(steps):
        seqs = [seqs[p] + [int(c)] for p, c in zip(s.parents.tolist(), s.tokens.tolist())]
        logits = s.step()
        states.append(s.state())
        for r in range(R):                              # this row's logits from its own history
            x = e64[torch.tensor(seqs[r], device=DEV)].view(-1, hq + 2 * hkv, hd).cpu().numpy()
            rot = np.stack([rope(x[i], i, freqs.tolist(), False, 1.0) for i in range(len(x))])
            kk = torch.tensor(rot[:, hq:hq + hkv]).bfloat16().double().numpy()
            vv = torch.tensor(x[:, hq + hkv:]).bfloat16().double().numpy()
            o = [attend(rot[-1, h], kk[:, h // 2], vv[:, h // 2], np.ones(len(x), bool), 0.125, 0.0)[0] for h in range(hq)]
            want = 3 * np.concatenate(o) @ h64.cpu().numpy()
            # a key on the other side of a rounding border moves a score by 2^-8 |q_i k_i| / 8; the head's product
            # runs in 32 bits
            assert np.abs(f64(logits[r]) - want).max() <= 0.02 * max(1.0, np.abs(want).max()), (t, r)
    paged.check_status(s.status)
    held = s.table[s.table >= 0].long()
    assert torch.equal(torch.bincount(held, minlength=64).int(), s.refs)

    s = Search()
    s.step()                                            # warm, and the first state
    graph = torch.cuda.CUDAGraph()
    fresh = [t.clone() for t in (s.pages, s.table, s.lens, s.refs, s.tokens, s.parents, s.scores, s.ended)]
    with torch.cuda.graph(graph):
        s.step()
    for a, b in zip((s.pages, s.table, s.lens, s.refs, s.tokens, s.parents, s.scores, s.ended), fresh):
        a.copy_(b)
    for t in range(1, steps):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(s.state(), states[t])), t
    paged.check_status(s.status)


def test_operators_on_another_stream(paged):
    """The work runs on the current stream: behind a long kernel there, the results are that stream's."""
    g = torch.Generator(device=DEV).manual_seed(12)
    kp, vp, table = _make_cache(g, [500, 100], 2, 64, 16, "bf16", poison=False)
    q = torch.randn(2, 4, 64, generator=g, device=DEV).bfloat16()
    want = paged.paged_attention(q, kp, vp, ints(table), ints([500, 100]))
    late, tb, n = torch.zeros_like(q), ints(table), ints([500, 100])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):
            x = x @ x * 1e-3
        late.copy_(q)
        got = paged.paged_attention(late, kp, vp, tb, n)
    s.synchronize()
    assert torch.equal(got, want)
