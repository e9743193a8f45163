"""The operators on trees of drafted tokens, and attention over chosen pages, on the GPU against plain
64-bit implementations.

Tolerances: a result rounded to a type is off by at most half a step, eps / 2 relative (plus the
smallest subnormal's half for fp16), and by what its 32-bit arithmetic adds, which each test bounds
from its own inputs."""
import math

import numpy as np
import pytest
import torch

from drafts_plain import accept, choose, page_score, tree_seen
from paged_plain import attend

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
    return np.abs(x) * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def f64(t):
    return t.double().cpu().numpy()


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(4, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_cache(g, lens, hkv, hd, ps, cache, extra=3, skip=()):
    """Pages in random order for sequences of those lengths; places behind a sequence's end, and the slots
    `skip` [(row, slot)], hold NaN, infinities and large values."""
    need = [-(-max(n, 0) // ps) for n in lens]
    n_pages = sum(need) + extra
    ids = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    width = max(max(need), 1) + 1
    table = -np.ones((len(lens), width), dtype=np.int32)
    pages = torch.randn(2, n_pages, hkv, ps, hd, generator=g, device=DEV).to(TYPES[cache])
    used = torch.zeros(n_pages, ps, dtype=torch.bool, device=DEV)
    at = 0
    for r, n in enumerate(lens):
        table[r, : need[r]] = ids[at: at + need[r]]
        at += need[r]
        for i in range(need[r]):
            used[table[r, i], : min(ps, n - i * ps)] = True
    for r, t in skip:
        used[table[r, t // ps], t % ps] = False
    junk = torch.tensor([math.nan, math.inf, -math.inf, 6e4], device=DEV)
    bad = junk[torch.randint(0, 4, pages.shape, generator=g, device=DEV)].to(pages.dtype)
    pages = torch.where(used[None, :, None, :, None], pages, bad)
    return pages[0], pages[1], table


def trees(rng, rows, nodes, shape, absent=True):
    """parents [rows][nodes]; some rows with absent nodes, several roots, subtrees under absent nodes."""
    out = []
    for r in range(rows):
        p = [-1]
        for i in range(1, nodes):
            if shape == "chain":
                p.append(i - 1)
            elif shape == "wide":
                p.append((i - 1) // 4)
            else:
                p.append(int(rng.integers(-1, i)) if rng.random() < 0.9 or not absent else int(rng.choice([-2, i, i + 3, 2 ** 31 - 1])))
        if absent and r % 3 == 2:
            for i in range(nodes // 2 + 1, nodes):
                p[i] = -2
        out.append(p)
    return out


# --------------------------------------------------------------------------- tree attention
def check_tree(q, kp, vp, table, lens, parents, out, lse, scale, window=0, cap=0.0, rows=None):
    """Each row, node and head against the plain form.  With A = scale sum |q||k| at its largest: a score's 32-bit
    products and sums are off by at most (hd + 16) 2^-23 A, its query parts by 2^-17 A (bf16 cache, fp16
    queries), 2^-22 A (fp16 cache, other queries) or nothing; the conversion to units of log 2, exp2 and the maximum
    add 2^-21 (1 + |score| / 4); a probability is rounded to the cache's type (half a step: 2^-8, 2^-11) where the
    outputs have 16 bits, and has parts good to 2^-22 where they have 32; sums over the tiles and pieces add 2^-23
    each.  A relative error d of every probability moves the output by at most 2 d sum p |v|."""
    R, T, hq, hd = q.shape
    hkv, ps = kp.shape[1], kp.shape[2]
    qd, od, ld = f64(q), f64(out), f64(lse)
    kd, vd = f64(kp), f64(vp)
    same = q.dtype == kp.dtype
    qbits = 0.0 if same else 2.0 ** -17 if kp.dtype == torch.bfloat16 and q.dtype == torch.float16 else 2.0 ** -22
    pbits = 2.0 ** -22 if q.dtype == torch.float32 else torch.finfo(kp.dtype).eps / 2
    for r in range(R):
        tr, n = (r if rows is None else rows[r]), lens[r]
        there = n >= 0 and 0 <= tr < len(table)
        rows_seen = tree_seen(n, parents[r], window) if there else [None] * T
        for i in range(T):
            if rows_seen[i] is None:
                assert np.all(od[r, i] == 0) and np.all(ld[r, i] == -math.inf), (r, i)
                continue
            t = np.arange(min(n + T, table.shape[1] * ps))
            page = table[tr, t // ps]
            seen = rows_seen[i][: len(t)] & (page >= 0) & (page < kp.shape[0])
            page = np.where(seen, page, 0)
            for h in range(hq):
                j = h // (hq // hkv)
                with np.errstate(invalid="ignore"):
                    w, l, mass, size = attend(qd[r, i, h], kd[page, j, t % ps], vd[page, j, t % ps], seen, scale, cap)
                if not seen.any():
                    assert np.all(od[r, i, h] == 0) and ld[r, i, h] == -math.inf, (r, i, h)
                    continue
                d = size * ((hd + 16) * 2.0 ** -23 + qbits) + 2.0 ** -21 * (1 + (size if not cap else min(size, cap)) / 4)
                sums = (len(t) / 16 + 64) * 2.0 ** -23
                assert np.all(np.abs(od[r, i, h] - w) <= half_step(q.dtype, w) + (2 * d + 2 * pbits + sums) * mass), (r, i, h)
                assert abs(ld[r, i, h] - l) <= d + sums + 2.0 ** -22 * abs(l), (r, i, h)


def tree_case(paged, lens, nodes, hq, hkv, hd, ps, cache, vec, window=0, cap=0.0, shape="random", strided=False, seed=1):
    g = gen(seed)
    parents = trees(np.random.default_rng(seed), len(lens), nodes, shape)
    ends = [n + nodes if n >= 0 else 0 for n in lens]
    gone = [(r, lens[r] + i) for r in range(len(lens)) if lens[r] >= 0
            for i, s in enumerate(tree_seen(lens[r], parents[r])) if s is None]
    kp, vp, table = make_cache(g, ends, hkv, hd, ps, cache, skip=gone)
    q = torch.randn(len(lens), nodes, hq, hd, generator=g, device=DEV).mul_(1.5).to(TYPES[vec])
    out = None
    if strided:
        q = torch.cat((q, q), -1).permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)[..., hd:]
        out = torch.full((nodes, len(lens), hq, hd + 2), 9.0, dtype=q.dtype, device=DEV).transpose(0, 1)
    st = status()
    got, lse = paged.tree_attention(q, kp, vp, ints(table), ints(lens), ints(parents), window=window, softcap=cap,
                                    return_lse=True, out=out[..., :hd] if strided else None, status=st)
    paged.check_status(st)
    if strided:
        assert got.data_ptr() == out.data_ptr() and torch.all(out[..., hd:] == 9.0)
    check_tree(q, kp, vp, table, lens, parents, got, lse, 1 / math.sqrt(hd), window, cap)


EDGES = [0, 1, 15, 16, 17, 63, 64, 121, 127, 128, 129, 300, -1]


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (6, 2), (8, 1), (9, 1), (16, 1)])
@pytest.mark.parametrize("hd", [64, 128])
def test_tree_groups_and_edges(paged, hq, hkv, hd):
    tree_case(paged, EDGES, 7, hq, hkv, hd, 16, "bf16", "bf16")


@pytest.mark.parametrize("nodes", [1, 2, 8, 31, 32, 33, 64, 65, 127, 128])
@pytest.mark.parametrize("shape", ["random", "chain", "wide"])
def test_tree_sizes_and_shapes(paged, nodes, shape):
    tree_case(paged, [0, 5, 130], nodes, 6, 2, 64, 32, "f16", "f16", shape=shape)


@pytest.mark.parametrize("cache,vec", [("f16", "f16"), ("f16", "f32"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("bf16", "f16")])
@pytest.mark.parametrize("hd", [64, 128])
def test_tree_types_and_strides(paged, cache, vec, hd):
    tree_case(paged, [700, 3, 0, 1025, 128], 9, 8, 2, hd, 32, cache, vec, strided=True)


@pytest.mark.parametrize("window", [1, 3, 16, 100, 400, 5000])
@pytest.mark.parametrize("cap,ps", [(0.0, 16), (20.0, 48)])
def test_tree_windows_caps_and_pages(paged, window, cap, ps):
    tree_case(paged, [0, 2, 17, 127, 128, 390, 401, 1000], 13, 4, 2, 64, ps, "bf16", "bf16", window=window, cap=cap)


@pytest.mark.parametrize("ps", [16, 80, 128, 256, 1008, 1024])
def test_tree_page_sizes(paged, ps):
    tree_case(paged, [1100, 7, 0, 240], 5, 4, 2, 128, ps, "f16", "f32")


def test_tree_of_many_rows(paged):
    tree_case(paged, [(37 * i) % 211 - (i % 10 == 7) * 300 for i in range(400)], 3, 4, 2, 64, 16, "bf16", "bf16")


@pytest.mark.parametrize("cache,vec,hd,hq,hkv", [("bf16", "bf16", 128, 8, 2), ("f16", "f32", 128, 16, 8), ("f16", "f16", 64, 8, 8)])
def test_tree_long_contexts_as_rows_of_paged_attention(paged, cache, vec, hd, hq, hkv):
    """A chain of nodes is a batch of rows of rising length; each result within what both operators may be off."""
    g = gen(3)
    lens, nodes = [9000, 33001, 4095], 6
    kp, vp, table = make_cache(g, [n + nodes for n in lens], hkv, hd, 64, cache)
    q = torch.randn(3, nodes, hq, hd, generator=g, device=DEV).to(TYPES[vec])
    out, lse = paged.tree_attention(q, kp, vp, ints(table), ints(lens), ints([[i - 1 for i in range(nodes)]] * 3), return_lse=True)
    rows = [r for r in range(3) for _ in range(nodes)]
    want, wl = paged.paged_attention(q.view(-1, hq, hd), kp, vp, ints(table), ints([lens[r] + i + 1 for r in range(3) for i in range(nodes)]),
                                     rows=ints(rows), return_lse=True)
    # sum p |v| is about 0.8 of normal values; a probability of one part adds eps / 2 of it at most
    bound = (torch.finfo(TYPES[cache]).eps * 0.9 if vec != "f32" else 2.0 ** -16) + 2 * half_step(TYPES[vec], f64(want)).max()
    assert np.abs(f64(out) - f64(want).reshape(f64(out).shape)).max() <= bound
    assert np.abs(f64(lse).reshape(-1) - f64(wl).reshape(-1)).max() <= 2.0 ** -17


def test_tree_values_reach_only_who_sees_them(paged):
    """NaN and infinities in the keys or values of a node, and of positions that only some windows hold."""
    g = gen(4)
    for hd, hq, hkv, dtype in ((64, 4, 2, "bf16"), (128, 2, 1, "f16"), (128, 16, 1, "bf16")):
        n, nodes, window = 200, 6, 40
        parents = [-1, 0, 0, 1, 3, 2]
        kp, vp, table = make_cache(g, [n + nodes], hkv, hd, 16, dtype)
        q = torch.randn(1, nodes, hq, hd, generator=g, device=DEV).to(TYPES[dtype])
        args = (ints(table), ints([n]), ints([parents]))
        clean, cl = paged.tree_attention(q, kp, vp, *args, window=window, return_lse=True)
        assert torch.isfinite(clean).all()
        for slot in (n + 1, n + 2, n + 5, n - window + 1, n - window + 2, n - window + 3, n - window, n - 1, 100, n):
            sees = [bool(s[slot]) for s in tree_seen(n, parents, window)]
            for bad in (math.nan, math.inf, -math.inf):
                for plane in (kp, vp):
                    at = plane[int(table[0, slot // 16]), :, slot % 16]
                    keep = at.clone()
                    at[:, 5] = bad
                    got, gl = paged.tree_attention(q, kp, vp, *args, window=window, return_lse=True)
                    for i in range(nodes):
                        if not sees[i]:
                            assert torch.equal(got[0, i], clean[0, i]) and torch.equal(gl[0, i], cl[0, i]), (slot, bad, i)
                        elif plane is vp:
                            assert torch.equal(gl[0, i], cl[0, i])
                            assert not torch.isfinite(got[0, i, :, 5]).any(), (slot, bad, i)
                            rest = torch.arange(hd, device=DEV) != 5
                            assert torch.equal(got[0, i][:, rest], clean[0, i][:, rest]), (slot, bad, i)
                        elif math.isnan(bad):
                            assert not torch.isfinite(got[0, i]).any()
                    at.copy_(keep)


def test_tree_scores_of_minus_infinity_and_far_apart(paged):
    """A node all of whose scores are -inf gets zeros; very large scores of either sign do not overflow."""
    g = gen(5)
    n, nodes, hd = 150, 3, 64
    kp, vp, table = make_cache(g, [n + nodes], 1, hd, 16, "bf16")
    q = torch.randn(1, nodes, 2, hd, generator=g, device=DEV).bfloat16()
    kp[..., 0] = -math.inf
    q[..., 0] = 1.0
    q[0, 1, :, 0] = 0.5
    out, lse = paged.tree_attention(q, kp, vp, ints(table), ints([n]), ints([[-1, 0, 1]]), return_lse=True)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    kp, vp, table = make_cache(g, [n + nodes], 1, hd, 16, "bf16")
    q = (torch.randn(1, nodes, 2, hd, generator=g, device=DEV) * 2e4).bfloat16()
    out, lse = paged.tree_attention(q, kp, vp, ints(table), ints([n]), ints([[-1, 0, 1]]), return_lse=True)
    check_tree(q, kp, vp, table, [n], [[-1, 0, 1]], out, lse, 0.125)


@pytest.mark.parametrize("what", ["page", "negative page", "row", "length", "tree's page"])
def test_tree_reports_and_masks_what_is_not_there(paged, what):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    g = gen(6)
    lens, rows, nodes = [200, 80, 64], [0, 1, 2], 5
    kp, vp, table = make_cache(g, [n + nodes for n in lens], 2, 64, 16, "f16")
    if what == "page":
        table[0, 3] = len(kp) + 5
    if what == "negative page":
        table[0, 3] = -7
    if what == "tree's page":
        table[1, 5] = -1                # slots 80..84
    if what == "row":
        rows[1] = 3
    if what == "length":
        table = table[:, :6].copy()      # row 0 has 200 positions, the table holds 96
    parents = [[-1, 0, 1, 0, 3]] * 3
    st = status()
    q = torch.randn(3, nodes, 4, 64, generator=g, device=DEV).half()
    args = (q, kp, vp, ints(table), ints(lens), ints(parents))
    out, lse = paged.tree_attention(*args, rows=ints(rows), return_lse=True, status=st)
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_PAGES and "tree" in str(e.value)
    check_tree(q, kp, vp, table, lens, parents, out, lse, 0.125, rows=rows)
    paged.tree_attention(*args, rows=ints(rows))   # no status: not reported, no fault


def test_tree_slots_of_absent_nodes_need_no_page(paged):
    """Padded trees whose pages end with their last node: nothing is reported, and what the table holds behind is not used."""
    g = gen(18)
    lens, nodes = [30, 15, 48, 9], 40
    parents = [[-1] + [i - 1 if i < m else -2 for i in range(1, nodes)] for m in (2, 1, 16, 7)]
    ends = [n + m for n, m in zip(lens, (2, 1, 16, 7))]
    kp, vp, table = make_cache(g, ends, 2, 64, 16, "bf16")
    table = table[:, :4].copy()                       # 64 slots: the padding of row 2 ends past the table
    for fill in (-1, 10 ** 6):
        table[table < 0] = fill
        table[table >= len(kp)] = fill
        q = torch.randn(4, nodes, 4, 64, generator=g, device=DEV).bfloat16()
        st = status()
        out, lse = paged.tree_attention(q, kp, vp, ints(table), ints(lens), ints(parents), return_lse=True, status=st)
        paged.check_status(st)
        check_tree(q, kp, vp, table, lens, parents, out, lse, 0.125)


@pytest.mark.parametrize("vec", ["bf16", "f32"])
def test_tree_caps_of_nan_infinite_and_small_scores(paged, vec):
    """A cap: NaN keys make who sees them NaN, infinite ones count as the cap (queries of the cache's type); scores far below the cap are kept to their
    own size's accuracy, which check_tree bounds by the scores and not by the cap."""
    g = gen(19)
    n, nodes, parents = 90, 3, [[-1, 0, 0]]
    kp, vp, table = make_cache(g, [n + nodes], 1, 64, 16, "bf16")
    q = torch.randn(1, nodes, 2, 64, generator=g, device=DEV).to(TYPES[vec])
    q[..., 0] = 1.0
    args = (ints(table), ints([n]), ints(parents))
    for size, cap in ((1.0, 50.0), (0.01, 5.0), (30.0, 2.0)):
        out, lse = paged.tree_attention(q * size, kp, vp, *args, softcap=cap, return_lse=True)
        check_tree(q * size, kp, vp, table, [n], parents, out, lse, 0.125, cap=cap)
    at = kp[int(table[0, (n + 1) // 16]), :, (n + 1) % 16]
    at[:, 0] = math.nan
    out, lse = paged.tree_attention(q, kp, vp, *args, softcap=5.0, return_lse=True)
    assert torch.isnan(lse[0, 1]).all() and torch.isnan(out[0, 1]).all()
    assert torch.isfinite(out[0, 0]).all() and torch.isfinite(out[0, 2]).all() and torch.isfinite(lse[0, [0, 2]]).all()
    if vec == "f32":       # (a query in several parts meets an infinite key with a part of 0)
        return
    at[:, 0] = math.inf
    out, lse = paged.tree_attention(q, kp, vp, *args, softcap=5.0, return_lse=True)
    assert torch.isfinite(out).all()
    at[:, 0] = 1e30
    want, wl = paged.tree_attention(q, kp, vp, *args, softcap=5.0, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_tree_extreme_lengths(paged):
    """Lengths near 2^31 (past any table) are cut to the table's positions and reported."""
    from persistent_sm_decode_megakernel_gb300 import MkError
    g = gen(16)
    kp, vp, table = make_cache(g, [90, 90], 2, 64, 16, "f16")
    table = table[:, :5].copy()
    q = torch.randn(2, 3, 4, 64, generator=g, device=DEV).half()
    lens = [2 ** 31 - 1, -2 ** 31]
    for window in (0, 2 ** 31 - 1):
        st = status()
        out, lse = paged.tree_attention(q, kp, vp, ints(table), ints(lens), ints([[-1, 0, 1]] * 2), window=window, return_lse=True, status=st)
        with pytest.raises(MkError):
            paged.check_status(st)
        assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)
        if not window:
            want, wl = paged.paged_attention(q[0], kp, vp, ints(table), ints([80] * 3), rows=ints([0] * 3), return_lse=True)
            assert (out[0].float() - want.float()).abs().max() <= 2.0 ** -9 and (lse[0] - wl).abs().max() <= 2.0 ** -17


def test_tree_offsets_past_32_bits(paged):
    hkv, ps, hd = 2, 64, 128
    n_pages = 2 ** 31 // (hkv * ps * hd) + 40
    pool = torch.empty(2, n_pages, hkv, ps, hd, dtype=torch.bfloat16, device=DEV)
    g = gen(7)
    ids = [n_pages - 1, 0, n_pages // 2, n_pages - 2]
    small = torch.randn(2, 4, hkv, ps, hd, generator=g, device=DEV).bfloat16()
    pool[:, ids] = small
    q = torch.randn(1, 3, 4, hd, generator=g, device=DEV).bfloat16()
    tree = ints([[-1, 0, 0]])
    a = paged.tree_attention(q, pool[0], pool[1], ints([ids]), ints([200]), tree, return_lse=True)
    b = paged.tree_attention(q, small[0], small[1], ints([[0, 1, 2, 3]]), ints([200]), tree, return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # and the other operators over the same pages
    bound = [torch.zeros(n, hkv, 2, hd, dtype=torch.bfloat16, device=DEV) for n in (n_pages, 4)]
    for k, t, c in ((pool[0], ids, bound[0]), (small[0], [0, 1, 2, 3], bound[1])):
        paged.update_bounds(k, c, ints([t]), ints([200]), new=200)
    assert torch.equal(bound[0][ids], bound[1])
    s = [paged.page_scores(q[:, 0], c, ints([t]), ints([200]), ps) for c, t in zip(bound, (ids, [0, 1, 2, 3]))]
    assert torch.equal(s[0], s[1])
    a = paged.sparse_attention(q[:, 0], pool[0], pool[1], ints([ids]), ints([200]), s[0], 3, return_lse=True, return_pages=True)
    b = paged.sparse_attention(q[:, 0], small[0], small[1], ints([[0, 1, 2, 3]]), ints([200]), s[1], 3, return_lse=True, return_pages=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    one = ints([[5, 7, 8]])
    for k, t in ((pool, ids), (small, [0, 1, 2, 3])):
        n = ints([190])
        paged.accept_drafts(k[0][None], k[1][None], ints([t]), n, one, ints([[-1, 0, 0]]), ints([[8, 1, 2]]))
        assert n.item() == 192
    assert torch.equal(pool[:, ids], small)


@pytest.mark.parametrize("lens,nodes,hq,hkv,vec", [
    ([20000], 16, 8, 2, "f32"),              # one block of rows, tiles by turns
    ([9000, 3, 70, 0, 5000], 5, 8, 4, "bf16"),
    ([6000, 100], 64, 32, 4, "bf16"),        # two blocks
    ([700] * 40, 7, 16, 8, "bf16"),          # a share to a warpgroup
])
def test_tree_answers_stay_the_same_beside_other_traffic(paged, lens, nodes, hq, hkv, vec):
    """Many calls while another stream moves memory, which lets the copies of a call land in other orders: the same bits."""
    g = gen(20)
    kp, vp, table = make_cache(g, [n + nodes for n in lens], hkv, 128, 64, "bf16")
    q = torch.randn(len(lens), nodes, hq, 128, generator=g, device=DEV).to(TYPES[vec])
    tree = ints(trees(np.random.default_rng(20), len(lens), nodes, "random"))
    tb, ls, st = ints(table), ints(lens), status()
    want = paged.tree_attention(q, kp, vp, tb, ls, tree, return_lse=True, status=st)
    a, b = (torch.zeros(64 << 20, dtype=torch.uint8, device=DEV) for _ in range(2))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(300):
        with torch.cuda.stream(other):
            a.copy_(b)
        got = paged.tree_attention(q, kp, vp, tb, ls, tree, return_lse=True, status=st)
        differ += sum((x != y).sum() for x, y in zip(got, want))
    torch.cuda.current_stream().wait_stream(other)
    paged.check_status(st)
    assert differ.item() == 0


def test_tree_repeats_bit_for_bit_and_replays(paged):
    """The same call twice, captured and replayed with new lengths, trees and queries, two captured graphs at the
    same time on two streams, and a call on another stream."""
    g = gen(8)
    lens, nodes = [3000, 1, 700, 0, 2222], 11
    kp, vp, table = make_cache(g, [n + nodes for n in lens], 8, 128, 64, "bf16")
    tb = ints(table)
    rng = np.random.default_rng(8)
    qs = [torch.randn(5, nodes, 16, 128, generator=g, device=DEV).bfloat16() for _ in range(2)]
    ls = [ints(lens), ints([17, 0, 699, 0, 2000])]
    ps = [ints(trees(rng, 5, nodes, "random")) for _ in range(2)]
    call = lambda q, n, p: paged.tree_attention(q, kp, vp, tb, n, p, return_lse=True)  # noqa: E731
    want = [call(*x) for x in zip(qs, ls, ps)]
    assert all(torch.equal(a, b) for a, b in zip(want[0], call(qs[0], ls[0], ps[0])))
    q, n, p = qs[0].clone(), ls[0].clone(), ps[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(q, n, p)
    for i in (0, 1, 0):
        q.copy_(qs[i])
        n.copy_(ls[i])
        p.copy_(ps[i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want[i], got))
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(call(qs[i], ls[i], ps[i]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(50):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(want[i], outs[i]))
    with torch.cuda.stream(streams[0]):
        other = call(qs[1], ls[1], ps[1])
    streams[0].synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[1], other))


# ------------------------------------------------------------------------------- acceptance
def accept_case(paged, rows, nodes, layers, hkv, hd, ps, dtype, lens, tokens, parents, choices, strided=False, seed=1, table=None,
                refused=()):
    g = gen(seed)
    width = (max(max(lens), 0) + nodes) // ps + 2
    n_pages = rows * width + 2
    pages = torch.randn(2, layers, n_pages + strided, hkv, ps, hd, generator=g, device=DEV).to(TYPES[dtype])
    k, v = pages[0][:, :n_pages], pages[1][:, :n_pages]
    if table is None:
        table = torch.randperm(n_pages, generator=g, device=DEV)[: rows * width].view(rows, width).cpu().numpy().astype(np.int32)
    want_k, want_v, n = k.clone(), v.clone(), ints(lens)
    st = status()
    got = paged.accept_drafts(k, v, ints(table), n, ints(tokens), ints(parents), ints(choices), status=st)
    tok, path, count = (x.cpu().numpy() for x in got)
    for r in range(rows):
        p = accept(tokens[r], parents[r], choices[r]) if lens[r] >= 0 and r not in refused else []
        assert count[r] == len(p) and path[r].tolist() == p + [-1] * (nodes - len(p)), r
        assert tok[r].tolist() == [choices[r][i] for i in p] + [-1] * (nodes - len(p)), r
        assert n[r].item() == lens[r] + len(p)
        place = lambda t: (int(table[r, t // ps]), t % ps)  # noqa: E731
        src = [place(lens[r] + i) for i in p]
        for x in (want_k, want_v):
            vectors = [x[:, a, :, b].clone() for a, b in src]
            for j, vec in enumerate(vectors):
                a, b = place(lens[r] + j)
                x[:, a, :, b] = vec
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    if strided:
        assert torch.equal(pages[:, :, n_pages:], pages[:, :, n_pages:])
    return st


@pytest.mark.parametrize("nodes", [1, 2, 7, 32, 33, 64, 128])
@pytest.mark.parametrize("few", [2, 5, 1000])
def test_accept_random_trees(paged, nodes, few):
    """Tokens of few kinds, so that siblings are alike and walks go deep; some rows without a tree or sequence."""
    rng = np.random.default_rng(nodes * 7 + few)
    rows = 9
    lens = [0, 1, 15, 16, 40, 100, -1, 31, 5]
    parents = trees(rng, rows, nodes, "random")
    parents[8][0] = -2
    tokens, choices = (rng.integers(0, few, (rows, nodes)).tolist() for _ in range(2))
    st = accept_case(paged, rows, nodes, 2, 2, 64, 16, "bf16", lens, tokens, parents, choices, strided=True)
    paged.check_status(st)


@pytest.mark.parametrize("hd,ps,dtype", [(64, 48, "f16"), (128, 16, "bf16"), (128, 1024, "f16")])
def test_accept_chains_of_every_length(paged, hd, ps, dtype):
    rows, nodes = 18, 17
    tokens = [[100 * r + i for i in range(nodes)] for r in range(rows)]
    # chains laid on every second node, of r accepted ones
    parents = [[-1] + [max(0, (i - 1) // 2 * 2 - (i % 2 == 0) * 0) if i % 2 else i - 2 for i in range(1, nodes)] for _ in range(rows)]
    choices = [[tokens[r][i + 2] if i + 2 < nodes and i < 2 * r else -5 for i in range(nodes)] for r in range(rows)]
    st = accept_case(paged, rows, nodes, 3, 2, hd, ps, dtype, [(7 * r) % 50 for r in range(rows)], tokens, parents, choices)
    paged.check_status(st)


@pytest.mark.parametrize("what", ["page", "negative page", "length", "far"])
def test_accept_reports_what_is_not_there_and_leaves_the_row(paged, what):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    rows, nodes, ps = 3, 4, 16
    lens = [14, 30, 12]
    table = np.arange(rows * 3, dtype=np.int32).reshape(rows, 3)
    if what == "page":
        table[1, 2] = 10 ** 6
    if what == "negative page":
        table[1, 2] = -1
    if what == "length":
        table = table[:, :2].copy()
    if what == "far":
        lens[1] = 2 ** 31 - 2
    chain = [[-1, 0, 1, 2]] * rows
    k, v = (torch.randn(2, 9, 2, ps, 64, generator=gen(2), device=DEV).half() for _ in range(2))
    keep, n, st = k.clone(), ints(lens), status()
    tokens = [[1, 2, 3, 4], [1, 2, 3, 4], [1, 2, 9, 4]]
    tok, path, count = paged.accept_drafts(k, v, ints(table), n, ints(tokens), ints(chain), ints([[2, 3, 4, 5]] * rows), status=st)
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_PAGES and "acceptance" in str(e.value)
    assert count.tolist() == [4, 0, 2] and n.tolist() == [18, lens[1], 14]
    assert path.tolist() == [[0, 1, 2, 3], [-1] * 4, [0, 1, -1, -1]] and tok.tolist() == [[2, 3, 4, 5], [-1] * 4, [2, 3, -1, -1]]
    assert torch.equal(k, keep)            # a chain lies in its places already


def test_accept_captured_and_replayed(paged):
    g = gen(9)
    rng = np.random.default_rng(9)
    rows, nodes = 4, 8
    table = ints(np.arange(rows * 6).reshape(rows, 6))
    base = torch.randn(2, 2, 24, 2, 16, 64, generator=g, device=DEV).bfloat16()
    sets = [[ints(x) for x in (rng.integers(0, 3, (rows, nodes)), trees(rng, rows, nodes, "random"), rng.integers(0, 3, (rows, nodes)))]
            for _ in range(2)]
    wants = []
    for s in sets:
        k, n = base.clone(), ints([20, 0, 31, 60])
        wants.append([*paged.accept_drafts(k[0], k[1], table, n, *s), k, n])
    k, n, held = base.clone(), ints([20, 0, 31, 60]), [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = paged.accept_drafts(k[0], k[1], table, n, *held)
    for i in (0, 1, 0):
        k.copy_(base)
        n.copy_(ints([20, 0, 31, 60]))
        for x, y in zip(held, sets[i]):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(wants[i], [*got, k, n]))


# ---------------------------------------------------------------------------- chosen pages
def plain_bounds(kp, bounds, table, lens, new, rows=None):
    want, ps = bounds.double().cpu().numpy(), kp.shape[2]
    kd = f64(kp)
    for r, n in enumerate(lens):
        tr = r if rows is None else rows[r]
        if not 0 <= tr < len(table):
            continue
        n = min(n, table.shape[1] * ps)
        for j in range(max(0, n - new) // ps, -(-n // ps)):
            p = table[tr, j]
            if 0 <= p < kp.shape[0]:
                x = kd[p, :, : n - j * ps]
                want[p, :, 0], want[p, :, 1] = x.min(1), x.max(1)
    return want


@pytest.mark.parametrize("hd,ps,dtype,hkv", [(64, 16, "bf16", 3), (128, 48, "f16", 2), (128, 1024, "bf16", 1), (64, 80, "f16", 8)])
@pytest.mark.parametrize("new", [1, 2, 17, 100, 5000])
def test_bounds(paged, hd, ps, dtype, hkv, new):
    g = gen(10)
    lens = [0, 1, 15, 16, 17, 100, 1025, 2047, -3]
    kp, _, table = make_cache(g, lens, hkv, hd, ps, dtype)
    bounds = torch.full((kp.shape[0], hkv, 2, hd), 3.0, dtype=kp.dtype, device=DEV)
    want = plain_bounds(kp, bounds, table, lens, new)
    st = status()
    paged.update_bounds(kp, bounds, ints(table), ints(lens), new=new, status=st)
    paged.check_status(st)
    assert np.array_equal(f64(bounds), want)
    # some of the rows, the other way round
    rows = [6, 2, 5]
    some = torch.full_like(bounds, 3.0)
    paged.update_bounds(kp, some, ints(table), ints([lens[r] for r in rows]), rows=ints(rows), new=new)
    assert np.array_equal(f64(some), plain_bounds(kp, torch.full_like(bounds, 3.0), table, [lens[r] for r in rows], new, rows))


def test_bounds_of_nan_and_infinite_keys(paged):
    kp = torch.randn(2, 2, 16, 64, generator=gen(11), device=DEV).bfloat16()
    kp[0, 0, 3, 7], kp[0, 1, 0, 1], kp[0, 1, 1, 2], kp[1, 0, 5, 0] = math.nan, math.inf, -math.inf, math.nan
    bounds = torch.zeros(2, 2, 2, 64, dtype=torch.bfloat16, device=DEV)
    paged.update_bounds(kp, bounds, ints([[0, 1]]), ints([20]), new=20)
    want = torch.stack((kp[0].amin(1), kp[0].amax(1)), 1)
    assert torch.equal(bounds[0].nan_to_num(9e9), want.nan_to_num(9e9)) and bounds[0, 0, :, 7].isnan().all()
    assert torch.isfinite(bounds[1]).all()         # its NaN lies behind the row's end


@pytest.mark.parametrize("what", ["page", "row", "length"])
def test_bounds_and_scores_report_what_is_not_there(paged, what):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    g = gen(12)
    lens, rows = [60, 33], [0, 1]
    kp, _, table = make_cache(g, lens, 2, 64, 16, "f16")
    if what == "page":
        table[0, 1] = 500
    if what == "row":
        rows[0] = -1
    if what == "length":
        table = table[:, :3].copy()
    bounds = torch.full((kp.shape[0], 2, 2, 64), 3.0, dtype=kp.dtype, device=DEV)
    want = plain_bounds(kp, bounds, table, lens, 60, rows)
    st = status()
    paged.update_bounds(kp, bounds, ints(table), ints(lens), rows=ints(rows), new=60, status=st)
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_PAGES and "bounds" in str(e.value)
    assert np.array_equal(f64(bounds), want)
    q = torch.randn(2, 4, 64, generator=g, device=DEV).half()
    scores = paged.page_scores(q, bounds, ints(table), ints(lens), 16, rows=ints(rows), status=st)
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_PAGES and "scores" in str(e.value)
    there = torch.isfinite(scores[:, 0]).cpu().numpy()
    assert there.tolist() == [[(0 <= rows[r] < 2 and j * 16 < lens[r] and 0 <= table[r, j] < len(kp)) for j in range(table.shape[1])]
                              for r in range(2)]


@pytest.mark.parametrize("cache,vec", [("f16", "f16"), ("f16", "f32"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("bf16", "f16")])
@pytest.mark.parametrize("hd,hq,hkv", [(64, 6, 2), (128, 4, 4), (128, 16, 1), (64, 10, 1), (128, 8, 2)])
def test_scores(paged, cache, vec, hd, hq, hkv):
    """Sums of 2 hd products in 32 bits: off by at most (hd + 16) 2^-23 of the sum of the absolute products, query parts
    by 2^-22 (fp16 cache), 2^-17 (bf16 cache, fp16 queries) of it or nothing."""
    g = gen(13)
    lens, ps = [0, 1, 16, 17, 300, 1000, -4], 16
    _, _, table = make_cache(g, lens, 1, 64, ps, cache)
    n_pages = table.max() + 2
    b = torch.randn(n_pages, hkv, 2, hd, generator=g, device=DEV)
    bounds = torch.stack((b.amin(2), b.amax(2)), 2).to(TYPES[cache])
    q = torch.cat([torch.randn(len(lens), hq, hd, generator=g, device=DEV).to(TYPES[vec])] * 2, -1)[..., hd:]
    st = status()
    got = f64(paged.page_scores(q, bounds, ints(table), ints(lens), ps, status=st))
    paged.check_status(st)
    bd, qd = f64(bounds), f64(q)
    qbits = 0.0 if q.dtype == bounds.dtype else 2.0 ** -17 if cache == "bf16" and vec == "f16" else 2.0 ** -22
    for r, n in enumerate(lens):
        for j in range(table.shape[1]):
            for h in range(hkv):
                if j * ps >= n:
                    assert got[r, h, j] == -math.inf
                    continue
                low, high = bd[table[r, j], h]
                heads = qd[r, h * (hq // hkv): (h + 1) * (hq // hkv)]
                size = (np.abs(heads) @ np.maximum(np.abs(low), np.abs(high))).max()
                assert abs(got[r, h, j] - page_score(heads, low, high)) <= size * ((hd + 16) * 2.0 ** -23 + qbits), (r, h, j)


def test_scores_of_nan_and_infinite_bounds(paged):
    bounds = torch.stack((-torch.ones(4, 1, 64), torch.ones(4, 1, 64)), 2).to(DEV).bfloat16()
    bounds[0, 0, 1, 3], bounds[1, 0, 0, 3], bounds[2, 0, 0, 5] = math.inf, -math.inf, math.nan
    q = torch.ones(1, 2, 64, device=DEV).bfloat16()
    q[0, 1] = -1
    got = paged.page_scores(q, bounds, ints([[0, 1, 2, 3]]), ints([64]), 16)[0, 0].tolist()
    assert got[0] == math.inf and got[1] == math.inf and math.isnan(got[2]) and got[3] == 64


def check_sparse(paged, q, kp, vp, table, lens, scores, n_blocks, first, last, cap=0.0, rows=None, **kw):
    """The pages one by one, and the attention over them as paged_attention gives it over a table of those pages, bit for
    bit, and against the plain form."""
    hkv, ps, hd = kp.shape[1], kp.shape[2], kp.shape[3]
    st = status()
    out, lse, pages = paged.sparse_attention(q, kp, vp, ints(table), ints(lens), scores, n_blocks, first=first, last=last,
                                             softcap=cap, rows=None if rows is None else ints(rows), return_lse=True, return_pages=True,
                                             status=st, **kw)
    paged.check_status(st)
    got, sd = pages.cpu().numpy(), f64(scores)
    qd, od, ld, kd, vd = f64(q), f64(out), f64(lse), f64(kp), f64(vp)
    group = q.shape[1] // hkv
    pbits = 2.0 ** -17 if kp.dtype == torch.bfloat16 and q.dtype != torch.float32 else 2.0 ** -22
    qbits = 0.0 if q.dtype == kp.dtype else 2.0 ** -17 if kp.dtype == torch.bfloat16 and q.dtype == torch.float16 else 2.0 ** -22
    for r, n in enumerate(lens):
        tr, n = (r if rows is None else rows[r]), max(n, 0)
        for h in range(hkv):
            want = choose(sd[r, h].tolist(), -(-n // ps), n_blocks, first, last)
            assert got[r, h].tolist() == want + [-1] * (n_blocks - len(want)), (r, h)
            t = np.concatenate([np.arange(j * ps, min(n, (j + 1) * ps)) for j in want] + [np.zeros(0, dtype=int)]).astype(int)
            page = table[tr, t // ps]
            for x in range(h * group, (h + 1) * group):
                w, l, mass, size = attend(qd[r, x], kd[page, h, t % ps], vd[page, h, t % ps], np.ones(len(t), dtype=bool),
                                          1 / math.sqrt(hd), cap)
                if not len(t):
                    assert np.all(od[r, x] == 0) and ld[r, x] == -math.inf
                    continue
                d = size * ((hd + 16) * 2.0 ** -23 + qbits) + 2.0 ** -21 * (1 + (size if not cap else min(size, cap)) / 4)
                sums = (len(t) / 16 + 64) * 2.0 ** -23
                assert np.all(np.abs(od[r, x] - w) <= half_step(q.dtype, w) + (2 * d + 2 * pbits + sums) * mass), (r, x)
                assert abs(ld[r, x] - l) <= d + sums + 2.0 ** -22 * abs(l), (r, x)


def sparse_inputs(lens, hq, hkv, hd, ps, cache, vec, seed=1):
    g = gen(seed)
    kp, vp, table = make_cache(g, lens, hkv, hd, ps, cache)
    q = torch.randn(len(lens), hq, hd, generator=g, device=DEV).mul_(1.5).to(TYPES[vec])
    scores = torch.randn(len(lens), hkv, table.shape[1], generator=g, device=DEV)
    return q, kp, vp, table, scores


@pytest.mark.parametrize("n_blocks,first,last", [(1, 0, 1), (2, 1, 1), (3, 1, 1), (7, 2, 3), (8, 0, 8), (40, 1, 1), (300, 1, 2)])
@pytest.mark.parametrize("hd,hq,hkv", [(64, 6, 2), (128, 4, 4), (128, 12, 1)])
def test_sparse(paged, n_blocks, first, last, hd, hq, hkv):
    lens = [0, 1, 15, 16, 17, 112, 113, 700, 2000, -2]
    q, kp, vp, table, scores = sparse_inputs(lens, hq, hkv, hd, 16, "bf16", "bf16")
    check_sparse(paged, q, kp, vp, table, lens, scores, n_blocks, first, last)


@pytest.mark.parametrize("cache,vec", [("f16", "f16"), ("f16", "f32"), ("bf16", "f32"), ("bf16", "f16")])
def test_sparse_types_rows_and_caps(paged, cache, vec):
    lens = [900, 30, 1300]
    q, kp, vp, table, scores = sparse_inputs(lens, 8, 2, 128, 48, cache, vec)
    check_sparse(paged, q, kp, vp, table, lens, scores, 6, 1, 1, cap=15.0)
    rows = [2, 0]
    check_sparse(paged, q[:2], kp, vp, table, [1300, 900], scores.permute(1, 0, 2).contiguous().permute(1, 0, 2)[:2], 6, 1, 2, rows=rows)


def test_sparse_ties_nan_and_infinite_scores(paged):
    lens = [16 * 1000 - 3, 16 * 700, 16 * 50]
    q, kp, vp, table, scores = sparse_inputs(lens, 2, 2, 64, 16, "bf16", "bf16")
    scores = (scores * 2).round() / 2                    # a few values, zeros of either sign among them
    scores[0, 0, 40:60], scores[0, 1, ::7], scores[1, 0, 3] = math.nan, math.inf, math.nan
    scores[1, 1] = -math.inf
    scores[2, 0] = 0.0
    scores[2, 0, 1::2] = -0.0
    scores[2, 1] = math.nan
    for n_blocks in (2, 5, 23, 64, 257):
        check_sparse(paged, q, kp, vp, table, lens, scores, n_blocks, 1, 1)


@pytest.mark.parametrize("pages,n_blocks", [(2049, 7), (3000, 130), (4100, 4099), (2100, 2200)])
def test_sparse_of_more_pages_than_registers_hold(paged, pages, n_blocks):
    lens = [16 * pages - 5, 16 * (pages // 2)]
    q, kp, vp, table, scores = sparse_inputs(lens, 2, 1, 64, 16, "bf16", "bf16", seed=pages)
    scores[1] = (scores[1] * 4).round()
    check_sparse(paged, q, kp, vp, table, lens, scores, n_blocks, 1, 2)


def test_sparse_of_all_pages_is_paged_attention(paged):
    lens = [500, 3, 4000, 0]
    q, kp, vp, table, scores = sparse_inputs(lens, 8, 2, 128, 64, "f16", "f32")
    want = paged.paged_attention(q, kp, vp, ints(table), ints(lens), return_lse=True)
    got = paged.sparse_attention(q, kp, vp, ints(table), ints(lens), scores, table.shape[1], return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("what", ["page", "row", "length"])
def test_sparse_reports_what_is_not_there(paged, what):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    lens, rows = [200, 300], [0, 1]
    q, kp, vp, table, scores = sparse_inputs(lens, 4, 2, 64, 16, "f16", "f16")
    if what == "page":
        table[1, 0] = -9
    if what == "row":
        rows[1] = 7
    if what == "length":
        table, scores = table[:, :14].copy(), scores[..., :14].contiguous()
    st = status()
    out, lse, pages = paged.sparse_attention(q, kp, vp, ints(table), ints(lens), scores, 4, rows=ints(rows), return_lse=True,
                                             return_pages=True, status=st)
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_PAGES
    assert torch.isfinite(out).all()
    n = [200, {"page": 300, "row": 0, "length": 224}[what]]
    for r in range(2):
        for h in range(2):
            want = choose(f64(scores)[r, h].tolist(), -(-n[r] // 16), 4, 1, 1)
            assert pages[r, h].tolist() == want + [-1] * (4 - len(want))
    if what == "row":
        assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)


# --------------------------------------------------------------------------------- together
def test_long_decoding_over_chosen_pages_captured(paged):
    """Append, bounds, scores, attention over the chosen pages, step after step from one captured graph: with as many
    blocks as pages the full attention, bit for bit, and with few of them what the calls give one by one."""
    g = gen(14)
    hq, hkv, hd, ps, start, steps = 8, 2, 64, 16, [70, 95], 20
    kp, vp, table = make_cache(g, [n + steps for n in start], hkv, hd, ps, "bf16")
    tb = ints(table)
    freqs, m = paged.rope_freqs(10000.0, hd, device=DEV)
    data = torch.randn(steps, 2, hq + 2 * hkv, hd, generator=g, device=DEV).bfloat16()

    class Run:
        def __init__(self):
            self.k, self.v = kp.clone(), vp.clone()
            self.b = torch.zeros(kp.shape[0], hkv, 2, hd, dtype=kp.dtype, device=DEV)
            self.n = ints(start)
            self.x = torch.zeros_like(data[0])
            self.st = status()
            paged.update_bounds(self.k, self.b, tb, self.n, new=max(start), status=self.st)

        def step(self):
            q = paged.rope_append(self.x[:, :hq], self.x[:, hq:hq + hkv], self.x[:, hq + hkv:], self.k, self.v, tb, self.n,
                                  freqs=freqs, mscale=m, status=self.st)
            self.n += 1
            paged.update_bounds(self.k, self.b, tb, self.n, status=self.st)
            s = paged.page_scores(q, self.b, tb, self.n, ps, status=self.st)
            full = paged.paged_attention(q, self.k, self.v, tb, self.n, status=self.st)
            every = paged.sparse_attention(q, self.k, self.v, tb, self.n, s, 8, status=self.st)
            few = paged.sparse_attention(q, self.k, self.v, tb, self.n, s, 3, return_pages=True, status=self.st)
            return full, every, *few, s

    one, two = Run(), Run()
    graph = torch.cuda.CUDAGraph()
    state = [x.clone() for x in (two.k, two.v, two.b, two.n)]
    with torch.cuda.graph(graph):
        got = two.step()
    for x, y in zip((two.k, two.v, two.b, two.n), state):
        x.copy_(y)
    for i in range(steps):
        one.x.copy_(data[i])
        two.x.copy_(data[i])
        want = one.step()
        graph.replay()
        assert torch.equal(want[0], want[1])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        for r in range(2):           # a page's score is no less than any of its keys' products
            n = start[r] + i + 1
            t = np.arange(n)
            k = f64(one.k)[table[r, t // ps], :, t % ps]
            assert np.isfinite(k).all()
    paged.check_status(one.st)
    paged.check_status(two.st)


def test_drafted_decoding_of_the_three_operators(paged):
    """Append into slots, tree attention and acceptance, step after step, as one captured graph: what the accepted path
    attends to and leaves in the cache is what appending its tokens one by one gives."""
    g = gen(15)
    hq, hkv, hd, ps, nodes, steps, L = 8, 2, 64, 16, 7, 12, 1
    start = [33, 0, 100]
    R = len(start)
    width = 20
    table = ints(torch.randperm(R * width, generator=g, device=DEV).view(R, width).cpu())
    base = torch.randn(2, L, R * width, hkv, ps, hd, generator=g, device=DEV).half()
    freqs, m = paged.rope_freqs(10000.0, hd, device=DEV)
    rng = np.random.default_rng(15)
    plans = []
    for s in range(steps):
        parents = trees(rng, R, nodes, "random")
        tokens = rng.integers(0, 3, (R, nodes)).tolist()
        choices = rng.integers(0, 3, (R, nodes)).tolist()
        plans.append((parents, tokens, choices, torch.randn(R, nodes, hq + 2 * hkv, hd, generator=g, device=DEV).half()))

    class Run:
        def __init__(self):
            self.k, self.v, self.n, self.st = base[0].clone(), base[1].clone(), ints(start), status()
            self.parents, self.tokens, self.choices, self.depth = (torch.zeros(R, nodes, dtype=torch.int32, device=DEV) for _ in range(4))
            self.x = torch.zeros_like(plans[0][3])
            self.rows = ints([r for r in range(R) for _ in range(nodes)])
            self.node = ints([list(range(nodes))] * R)

        def load(self, plan):
            parents, tokens, choices, x = plan
            self.parents.copy_(ints(parents))
            self.tokens.copy_(ints(tokens))
            self.choices.copy_(ints(choices))
            self.depth.copy_(ints([[-10 ** 6 if s is None else int(s[9:].sum()) - 1 for s in tree_seen(9, p)] for p in parents]))
            self.x.copy_(x)

        def step(self):
            slots, pos = self.n[:, None] + self.node, self.n[:, None] + self.depth
            x = self.x.view(-1, hq + 2 * hkv, hd)
            q = paged.rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], self.k[0], self.v[0], table, pos.view(-1).contiguous(),
                                  rows=self.rows, freqs=freqs, mscale=m, slots=slots.view(-1).contiguous(), status=self.st)
            out, lse = paged.tree_attention(q.view(R, nodes, hq, hd), self.k[0], self.v[0], table, self.n, self.parents, return_lse=True,
                                            status=self.st)
            return (out, lse, *paged.accept_drafts(self.k, self.v, table, self.n, self.tokens, self.parents, self.choices, status=self.st))

    one, two = Run(), Run()
    for r in (one, two):
        r.load(plans[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = two.step()
    for x, y in ((two.k, base[0]), (two.v, base[1]), (two.n, ints(start))):
        x.copy_(y)
    # the accepted tokens appended one by one, for comparison
    k, v, n = base[0].clone(), base[1].clone(), list(start)
    for plan in plans:
        one.load(plan)
        two.load(plan)
        want = one.step()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        parents, tokens, choices, x = plan
        for r in range(R):
            path = accept(tokens[r], parents[r], choices[r])
            assert want[3][r, : len(path)].tolist() == path
            for i in path:
                y = x[r, i][None]
                q = paged.rope_append(y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], k[0], v[0], table, ints([n[r]]), rows=ints([r]),
                                      freqs=freqs, mscale=m)
                n[r] += 1
                ref, rl = paged.paged_attention(q, k[0], v[0], table, ints([n[r]]), rows=ints([r]), return_lse=True)
                # both are off by their rounding, 2^-12 of values up to 4, and by that of probabilities, 2^-11 of sum p |v| < 4
                assert (want[0][r, i].float() - ref[0].float()).abs().max().item() <= 2.0 ** -8
                assert (want[1][r, i] - rl[0]).abs().max().item() <= 2.0 ** -17
            t = np.arange(n[r])
            at = table[r].cpu().numpy()[t // ps]
            assert torch.equal(one.k[0][at, :, t % ps], k[0][at, :, t % ps]) and torch.equal(one.v[0][at, :, t % ps], v[0][at, :, t % ps])
        assert one.n.tolist() == n
    paged.check_status(one.st)
    paged.check_status(two.st)


# ------------------------------------------------------------------------------ refusals
def _small():
    pages = torch.zeros(2, 4, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=DEV)
    bounds = torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16, device=DEV)
    return pages, q, bounds, ints([[0, 1], [2, 3]]), ints([5, 6]), ints([[-1, 0, 1]] * 2), torch.zeros(2, 2, 2, device=DEV)


def test_tensors_that_do_not_fit_are_refused(paged):
    from persistent_sm_decode_megakernel_gb300 import MkError
    pages, q, bounds, table, lens, tree, scores = _small()
    k, v = pages
    call = lambda f, base: lambda **a: f(**{**base, **a})  # noqa: E731
    attend_ = call(paged.tree_attention, dict(q=q, k_pages=k, v_pages=v, table=table, lens=lens, parents=tree))
    accept_ = call(paged.accept_drafts, dict(k=k[None], v=v[None], table=table, lens=lens, tokens=tree, parents=tree, choices=tree))
    bounds_ = call(paged.update_bounds, dict(k_pages=k, bounds=bounds, table=table, lens=lens))
    scores_ = call(paged.page_scores, dict(q=q[:, 0], bounds=bounds, table=table, lens=lens, page_size=16))
    sparse_ = call(paged.sparse_attention, dict(q=q[:, 0], k_pages=k, v_pages=v, table=table, lens=lens, scores=scores, n_blocks=2))
    append_ = call(paged.rope_append, dict(q=q[:, 0], k=k[:2, :, 0], v=k[:2, :, 0], k_pages=k, v_pages=v, table=table, positions=lens))
    grown = q.float().requires_grad_()
    st3 = torch.zeros(3, dtype=torch.int32, device=DEV)
    for f, bads in ((attend_, (dict(q=q[0]), dict(q=q.double()), dict(q=q[..., :32]), dict(q=grown), dict(q=q.cpu()), dict(q=q.transpose(2, 3)),
                               dict(lens=lens[:1]), dict(lens=lens.long()), dict(parents=tree[:1]), dict(parents=tree.long()),
                               dict(parents=tree.t()), dict(parents=tree[:, :2]), dict(out=q.float()), dict(out=q[:1]), dict(rows=lens[:1]),
                               dict(window=2 ** 40), dict(status=st3), dict(v_pages=v.half()), dict(q=3), dict(lens=None))),
                    (accept_, (dict(k=k), dict(v=v[None].half()), dict(lens=lens[:1]), dict(tokens=tree[:1]), dict(tokens=tree[0]),
                               dict(parents=tree[:, :2]), dict(choices=tree.long()), dict(choices=tree.t()), dict(table=table.long()),
                               dict(status=st3), dict(tokens=tree.cpu()))),
                    (bounds_, (dict(bounds=bounds[:3]), dict(bounds=bounds.half()), dict(bounds=bounds[:, :, :1]), dict(bounds=bounds.transpose(1, 2)),
                               dict(bounds=bounds[:1].expand(4, 2, 2, 64)), dict(lens=lens.long()), dict(lens=table), dict(rows=lens[:1]),
                               dict(new=2 ** 40), dict(k_pages=k.float()), dict(bounds=bounds.float().requires_grad_()))),
                    (scores_, (dict(q=q), dict(q=q[:, 0].double()), dict(q=q[:1, 0]), dict(q=q[:, 0, :, :32]), dict(bounds=bounds.float()),
                               dict(bounds=bounds[0]), dict(bounds=bounds.transpose(0, 1)), dict(table=table[0]), dict(lens=lens[:1]),
                               dict(bounds=bounds.cpu()), dict(q=grown[:, 0]))),
                    (sparse_, (dict(q=q), dict(scores=scores[:1]), dict(scores=scores[..., :1]), dict(scores=scores.half()), dict(scores=scores.cpu()),
                               dict(scores=scores.permute(0, 2, 1).contiguous().permute(0, 2, 1)), dict(scores=None), dict(out=q[:, 1].float()),
                               dict(lens=lens.long()), dict(n_blocks=2 ** 40))),
                    (append_, (dict(slots=lens.long()), dict(slots=lens[:1]), dict(slots=lens.cpu())))):
        for bad in bads:
            with pytest.raises(ValueError):
                f(**bad)
    for f, bads in ((attend_, (dict(window=-1), dict(softcap=-2.0), dict(scale=math.nan), dict(q=q[:, :, :3]), dict(q=q[:, :0], parents=tree[:, :0]),
                               dict(out=q[:1].clone().expand(2, 3, 4, 64)), dict(out=q[:, :1].clone().expand(2, 3, 4, 64)),
                               dict(out=q[:, :, :1].clone().expand(2, 3, 4, 64)),
                               dict(q=q[:, :1].expand(2, 129, 4, 64), parents=tree[:, :1].expand(2, 129).contiguous()))),
                    (accept_, (dict(tokens=tree[:, :0].contiguous(), parents=tree[:, :0].contiguous(), choices=tree[:, :0].contiguous()),)),
                    (bounds_, (dict(new=0), dict(new=-1))),
                    (scores_, (dict(page_size=8), dict(page_size=2048), dict(q=q[:, 0, :3]))),
                    (sparse_, (dict(n_blocks=1), dict(n_blocks=0), dict(first=-1), dict(last=0), dict(first=2), dict(scale=math.inf)))):
        for bad in bads:
            with pytest.raises(MkError):
                f(**bad)
    assert attend_(q=q[:0], lens=lens[:0], parents=tree[:0]).shape == (0, 3, 4, 64)
    assert scores_(q=q[:0, 0], lens=lens[:0]).shape == (0, 2, 2)
    assert sparse_(q=q[:0, 0], lens=lens[:0], scores=scores[:0], return_pages=True)[1].shape == (0, 2, 2)
    bounds_(lens=lens[:0])
    with torch.no_grad():
        attend_(q=grown)
    torch.cuda.synchronize()
    assert not pages.any() and not bounds.any() and lens.tolist() == [5, 6]


def test_what_is_written_in_place_counts_as_changed(paged):
    pages, q, bounds, table, lens, tree, scores = _small()
    k, v, st, out = pages[0].clone(), pages[1].clone(), status(), torch.zeros_like(q)
    named = dict(k=k, v=v, q=q, bounds=bounds, table=table, lens=lens, tree=tree, scores=scores, st=st, out=out)

    def written(call):
        before = {n: t._version for n, t in named.items()}
        call()
        return {n for n, t in named.items() if t._version > before[n]}

    assert written(lambda: paged.tree_attention(q, k, v, table, lens, tree)) == set()
    assert written(lambda: paged.tree_attention(q, k, v, table, lens, tree, out=out, status=st)) == {"out", "st"}
    assert written(lambda: paged.update_bounds(k, bounds, table, lens)) == {"bounds"}
    assert written(lambda: paged.page_scores(q[:, 0], bounds, table, lens, 16, status=st)) == {"st"}
    assert written(lambda: paged.sparse_attention(q[:, 0], k, v, table, lens, scores, 2, out=out[:, 0])) == {"out"}
    assert written(lambda: paged.accept_drafts(k[None], v[None], table, lens, tree, tree, tree)) == {"k", "v", "lens"}


def test_one_slot_for_two_tokens_and_slots_that_are_none(paged):
    """Tokens of one position in slots of their own; slots below 0 or past the table are reported and cache nothing."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    pages = torch.zeros(2, 4, 2, 16, 64, dtype=torch.float16, device=DEV)
    k = torch.randn(3, 2, 64, generator=gen(17), device=DEV).half()
    freqs, m = paged.rope_freqs(10000.0, 64, device=DEV)
    st = status()
    for strided in (k, torch.cat((k, k), -1)[..., 3:67].copy_(k)):      # whole vectors, and element pairs
        pages.zero_()
        paged.rope_append(None, strided, strided, pages[0], pages[1], ints([[2, 0]]), ints([9, 9, 9]), rows=ints([0, 0, 0]), freqs=freqs,
                          slots=ints([20, 9, 31]), status=st)
        paged.check_status(st)
        want = torch.zeros_like(pages[0])
        paged.rope_append(None, k, k, want, torch.zeros_like(want), ints([[0, 1], [1, 2], [2, 3]]), ints([9, 9, 9]), freqs=freqs)
        for t, (page, at) in enumerate(((0, 4), (2, 9), (0, 15))):
            assert torch.equal(pages[0][page, :, at], want[t, :, 9]) and torch.equal(pages[1][page, :, at], k[t])
        for bad in (-1, 32, -2 ** 31, 2 ** 31 - 1):
            keep = pages.clone()
            paged.rope_append(None, strided[:1], strided[:1], pages[0], pages[1], ints([[2, 0]]), ints([9]), freqs=freqs, slots=ints([bad]),
                              status=st)
            with pytest.raises(MkError) as e:
                paged.check_status(st)
            assert e.value.status == MK_ERR_PAGES and torch.equal(pages, keep)


# --------------------------------------------------------------------- what the tests above do not look at
def test_accept_leaves_what_lies_between_the_layers(paged):
    """Layers that hold a page more than the pool: trees that are taken over to the end change nothing of it."""
    rows, nodes, ps, n_pages = 3, 6, 16, 8
    pages = torch.randn(2, 3, n_pages + 1, 2, ps, 64, generator=gen(23), device=DEV).half()
    keep = pages.clone()
    table = ints([[7, 0], [1, 6], [5, 2]])
    # every second node is the chosen one's child: all of the others' vectors move
    parents, tokens = [[-1, 0, 0, 2, 2, 4]] * rows, [[1, 9, 2, 9, 3, 4]] * rows
    n = ints([14, 0, 26])
    count = paged.accept_drafts(pages[0][:, :n_pages], pages[1][:, :n_pages], table, n, ints(tokens), ints(parents),
                                ints([[2, 0, 3, 0, 4, 5]] * rows))[2]
    assert count.tolist() == [4, 4, 4] and n.tolist() == [18, 4, 30]
    assert torch.equal(pages[:, :, n_pages], keep[:, :, n_pages]) and not torch.equal(pages, keep)
    assert torch.equal(pages[:, :, [3, 4]], keep[:, :, [3, 4]])          # pages of no row


@pytest.mark.parametrize("vec", ["bf16", "f32"])
@pytest.mark.parametrize("hq", [2, 12])
def test_scores_of_nan_bounds_under_any_query(paged, vec, hq):
    """A NaN bound makes the score NaN whatever the query holds there, zeros of either sign included; an infinite one
    under a zero adds nothing."""
    for zero in (0.0, -0.0, 2.0, -2.0):
        bounds = torch.stack((-torch.ones(6, 1, 64), torch.ones(6, 1, 64)), 2).to(DEV).bfloat16()
        bounds[0, 0, :, 5], bounds[1, 0, 0, 5], bounds[2, 0, 1, 5] = math.nan, math.nan, math.nan
        bounds[3, 0, 0, 5], bounds[3, 0, 1, 5] = -math.inf, math.inf
        bounds[4, 0, 0, 7], bounds[4, 0, 1, 9] = math.nan, math.inf
        q = torch.ones(1, hq, 64, device=DEV).to(TYPES[vec])
        q[..., 5] = zero
        got = paged.page_scores(q, bounds, ints([[0, 1, 2, 3, 4, 5]]), ints([96]), 16)[0, 0].tolist()
        assert all(math.isnan(got[i]) for i in (0, 1, 2, 4)), got
        assert got[3] == (63 if zero == 0 else math.inf) and got[5] == 63 + abs(zero), got
    q[..., 5] = 0.0
    q[0, 1, 3] = math.nan
    got = paged.page_scores(q, bounds, ints([[0, 1, 2, 3, 4, 5]]), ints([96]), 16)[0, 0].tolist()
    assert all(math.isnan(x) for x in got), got


@pytest.mark.parametrize("cache,vec", [("f16", "f32"), ("bf16", "f32"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("hd,hq,hkv", [(128, 16, 1), (64, 8, 2)])
def test_scores_are_held_in_32_bits(paged, cache, vec, hd, hq, hkv):
    """Bounds of 1 at one dim and of 0 at all others, so that a score is one element of a head, beside a large one at a dim of
    its own.  Queries that enter whole give it exactly; of 32-bit ones over fp16 bounds, whose two parts hold 11 bits each of
    what is left, at most 2^-12 of at most 2^-11 of it is lost."""
    g = gen(24)
    ps, pages = 16, 64
    at = torch.arange(pages, device=DEV) % (hd - 1) + 1                  # the dim that page j looks at
    bounds = torch.zeros(pages, hkv, 2, hd, device=DEV)
    bounds.scatter_(3, at[:, None, None, None].expand(pages, hkv, 2, 1), 1.0)
    q = torch.randn(1, hq, hd, generator=g, device=DEV).abs().add_(0.5).to(TYPES[vec])
    q[..., 0] = 30.0
    got = paged.page_scores(q, bounds.to(TYPES[cache]), ints([list(range(pages))]), ints([ps * pages]), ps)[0]
    want = q[0].view(hkv, hq // hkv, hd).amax(1).float()[:, at]
    if (cache, vec) == ("f16", "f32"):
        assert ((got - want).abs() <= want * 2.0 ** -23).all()
    else:
        assert torch.equal(got, want)


@pytest.mark.parametrize("cache,vec,hq,hkv", [("bf16", "bf16", 8, 2), ("f16", "f32", 16, 1), ("f16", "f16", 3, 3)])
def test_no_key_of_a_page_exceeds_its_score(paged, cache, vec, hq, hkv):
    """Append, bounds and scores together, step after step: a page's score is no less than the product of any of the heads with
    any key in it, but for the rounding of sums of 2 hd products of which each element is at most the bounds' greater one (as in
    test_scores)."""
    g = gen(25)
    hd, ps, start, steps = 64, 16, [30, 61, 0], 20
    kp, vp, table = make_cache(g, [n + steps for n in start], hkv, hd, ps, cache)
    tb, n = ints(table), ints(start)
    freqs, m = paged.rope_freqs(10000.0, hd, device=DEV)
    bounds = torch.full((kp.shape[0], hkv, 2, hd), math.nan, dtype=kp.dtype, device=DEV)
    paged.update_bounds(kp, bounds, tb, n, new=max(start))
    for i in range(steps):
        x = torch.randn(3, hq + 2 * hkv, hd, generator=g, device=DEV).to(TYPES[vec])
        q = paged.rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kp, vp, tb, n, freqs=freqs, mscale=m)
        n += 1
        paged.update_bounds(kp, bounds, tb, n)
        got, qd, kd = f64(paged.page_scores(q, bounds, tb, n, ps)), f64(q), f64(kp)
        for r in range(3):
            for j in range(-(-(start[r] + i + 1) // ps)):
                keys = kd[table[r, j], :, : start[r] + i + 1 - j * ps]
                for h in range(hkv):
                    heads = qd[r, h * (hq // hkv): (h + 1) * (hq // hkv)]
                    size = (np.abs(heads) @ np.abs(keys[h]).max(0)).max()
                    assert got[r, h, j] >= (heads @ keys[h].T).max() - size * ((hd + 16) * 2.0 ** -23 + 2.0 ** -22), (i, r, h, j)
