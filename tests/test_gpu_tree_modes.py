"""Tree attention on the GPU in each of the ways its kernel deals the rows, against a plain 64-bit computation (torch,
from the definitions in include/mk.h): shares of the line to each warpgroup (many short trees), pairs of blocks (more than
128 rows per kv head, queries of the cache's type), single blocks of several parts (queries of another type).  And the sums of
long contexts, whose accuracy must not go with the length.

Tolerances: a result rounded to a type is off by at most half a step, eps / 2 relative (plus the smallest subnormal's half
for fp16); what the 32-bit arithmetic adds is said at the check."""
import math

import numpy as np
import pytest
import torch

from drafts_plain import tree_seen
from test_gpu_drafts import DEV, EDGES, TYPES, gen, ints, make_cache, paged, status, trees  # noqa: F401 (paged: the fixture)

pytestmark = pytest.mark.gpu


def plain_tree(q, kp, vp, table, n, row, parents, scale, window=0, cap=0.0):
    """One row's trees in 64 bits: outputs, log-sum-exps, sum p |v|, the largest scale sum |q||k|; absent nodes zeros and -inf."""
    T, hq, hd = q.shape
    hkv, ps = kp.shape[1], kp.shape[2]
    lines = tree_seen(n, parents, window) if n >= 0 else [None] * T
    there = torch.tensor([s is not None for s in lines], device=DEV)
    out, lse = torch.zeros(T, hq, hd, dtype=torch.float64, device=DEV), torch.full((T, hq), -math.inf, dtype=torch.float64, device=DEV)
    mass, size = torch.zeros_like(out), torch.zeros_like(lse)
    if not there.any():
        return out, lse, mass, size
    seen = torch.as_tensor(np.stack([s if s is not None else np.zeros(n + T, dtype=bool) for s in lines]), device=DEV)
    some = seen.any(0).nonzero()[:, 0]                      # the slots that any node sees
    page = torch.as_tensor(table, device=DEV)[row, some // ps].long()
    for j in range(hkv):
        k, v = (x[page, j, some % ps].double() for x in (kp, vp))
        h = slice(j * (hq // hkv), (j + 1) * (hq // hkv))
        x = q[:, h].double()
        s = torch.einsum("thd,ld->thl", x, k) * scale
        big = torch.einsum("thd,ld->thl", x.abs(), k.abs()) * abs(scale)
        if cap:
            s = cap * torch.tanh(s / cap)
        mask = seen[:, None, some]
        s = torch.where(mask, s, torch.tensor(-math.inf, dtype=torch.float64, device=DEV))
        m = s.amax(2, keepdim=True).clamp_min(-1e300)
        p = torch.exp(s - m)
        z = p.sum(2, keepdim=True)
        p = torch.where(z > 0, p / z, torch.zeros_like(p))
        out[:, h], mass[:, h] = torch.einsum("thl,ld->thd", p, v), torch.einsum("thl,ld->thd", p, v.abs())
        lse[:, h] = (m + torch.log(z))[..., 0]
        size[:, h] = torch.where(mask, big, torch.zeros_like(big)).amax(2)
    return out, lse, mass, size


def check(q, kp, vp, table, lens, parents, out, lse, window=0, cap=0.0):
    """With A = scale sum |q||k| at its largest: a score's 32-bit products and sums are off by at most (hd + 16) 2^-23 A, its
    query parts by 2^-17 A (bf16 cache, fp16 queries), 2^-22 A (fp16 cache, other queries) or nothing; the conversion to units
    of log 2, exp2 and the maximum add 2^-21 (1 + |score| / 4).  A probability has parts good to 2^-17 (bf16, two parts) or 2^-22.
    A sum of n products of up to 16 probabilities, each cut off, is off by at most n 2^-23; the maxima's slack, the pieces, the sum
    of the probabilities and their least parts, below 2^-34 each, stay below 64 2^-23 at these lengths.  A relative error d of
    every probability moves the output by at most 2 d sum p |v|."""
    hd, scale = q.shape[-1], 1 / math.sqrt(q.shape[-1])
    eps, least = torch.finfo(q.dtype).eps / 2, 2.0 ** -25 if q.dtype == torch.float16 else 0.0
    qbits = 0.0 if q.dtype == kp.dtype else 2.0 ** -17 if (kp.dtype, q.dtype) == (torch.bfloat16, torch.float16) else 2.0 ** -22
    pbits = 2.0 ** -17 if kp.dtype == torch.bfloat16 and q.dtype != torch.float32 else 2.0 ** -22
    for r, n in enumerate(lens):
        w, l, mass, size = plain_tree(q[r], kp, vp, table, n, r, parents[r], scale, window, cap)
        d = size * ((hd + 16) * 2.0 ** -23 + qbits) + 2.0 ** -21 * (1 + (size.clamp_max(cap) if cap else size) / 4)
        sums = (3 * max(n, 0) / 16 + 64) * 2.0 ** -23
        off = (out[r].double() - w).abs()
        assert torch.all(off <= w.abs() * eps + least + (2 * d[..., None] + 2 * pbits + sums) * mass), (r, (off / mass).max())
        none = torch.isinf(l)
        assert torch.equal(none, torch.isinf(lse[r])) and torch.all(lse[r][none] == -math.inf), r
        assert torch.all((lse[r].double() - l).abs()[~none] <= (d + sums + 2.0 ** -22 * l.abs())[~none]), r


def run(paged, lens, nodes, hq, hkv, hd, ps, cache, vec, window=0, cap=0.0, shape="random", seed=1, size=1.5):  # noqa: F811
    g = gen(seed)
    parents = trees(np.random.default_rng(seed), len(lens), nodes, shape)
    gone = [(r, n + i) for r, n in enumerate(lens) if n >= 0 for i, s in enumerate(tree_seen(n, parents[r])) if s is None]
    kp, vp, table = make_cache(g, [n + nodes if n >= 0 else 0 for n in lens], hkv, hd, ps, cache, skip=gone)
    q = torch.randn(len(lens), nodes, hq, hd, generator=g, device=DEV).mul_(size).to(TYPES[vec])
    st = status()
    out, lse = paged.tree_attention(q, kp, vp, ints(table), ints(lens), ints(parents), window=window, softcap=cap, return_lse=True,
                                    status=st)
    paged.check_status(st)
    check(q, kp, vp, table, lens, parents, out, lse, window, cap)


PAIRS = [("f16", "f16"), ("f16", "f32"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("bf16", "f16")]
MANY = EDGES * 3 + [511, 700, 1025, 64, 191, 5]          # 45 rows: with two kv heads a share for every warpgroup


@pytest.mark.parametrize("cache,vec", PAIRS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window,cap", [(0, 0.0), (70, 20.0)])
def test_many_rows(paged, cache, vec, hd, window, cap):  # noqa: F811
    run(paged, MANY, 7, 8, 2, hd, 16, cache, vec, window, cap)


@pytest.mark.parametrize("cache,vec", PAIRS)
@pytest.mark.parametrize("nodes,hq,hkv", [(13, 8, 2), (1, 4, 4), (8, 32, 2), (20, 16, 4)])
def test_many_rows_of_other_sizes(paged, cache, vec, nodes, hq, hkv):  # noqa: F811
    run(paged, MANY, nodes, hq, hkv, 128, 64, cache, vec, 3, shape="chain")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nodes,hq,hkv", [(33, 8, 2), (65, 8, 2), (128, 8, 2), (50, 6, 1), (17, 16, 1)])
@pytest.mark.parametrize("window,cap", [(0, 0.0), (70, 20.0)])
def test_pairs_of_blocks(paged, dtype, hd, nodes, hq, hkv, window, cap):  # noqa: F811
    """Two, three and four blocks of rows, the last of three without a partner."""
    run(paged, [0, 5, 130, 700, -1, 1025], nodes, hq, hkv, hd, 32, dtype, dtype, window, cap)


@pytest.mark.parametrize("cache,vec", [p for p in PAIRS if p[0] != p[1]])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nodes,rows", [(33, 6), (65, 6), (128, 2), (40, 45)])
@pytest.mark.parametrize("window,cap", [(0, 0.0), (70, 20.0)])
def test_blocks_of_other_types(paged, cache, vec, hd, nodes, rows, window, cap):  # noqa: F811
    """More than 128 rows per kv head whose queries are in parts: a block to a CTA."""
    run(paged, ([0, 5, 130, 700, -1, 1025] + MANY)[:rows], nodes, 8, 2, hd, 32, cache, vec, window, cap)


@pytest.mark.parametrize("cache,vec", PAIRS)
@pytest.mark.parametrize("cap", [0.5, 50.0, 64.0, 65.0, 1e3, 1e5, 1e8, 1e15, 1e30, 1e37])
def test_caps_of_any_size(paged, cache, vec, cap):  # noqa: F811
    """A capped score is as exact as an uncapped one, whatever the cap."""
    run(paged, [0, 90, 300], 3, 4, 2, 64, 16, cache, vec, cap=cap, size=3.0)


@pytest.mark.parametrize("cache,vec", PAIRS)
def test_caps_beyond_all_scores_are_none(paged, cache, vec):  # noqa: F811
    """From 2^64 on, bit for bit, here and in the attention of single tokens and of chosen pages."""
    g = gen(26)
    kp, vp, table = make_cache(g, [203], 2, 64, 16, cache)
    q = torch.randn(1, 3, 4, 64, generator=g, device=DEV).to(TYPES[vec])
    tb, n = ints(table), ints([200])
    scores = torch.randn(1, 2, table.shape[1], generator=g, device=DEV)
    calls = (lambda c: paged.tree_attention(q, kp, vp, tb, n, ints([[-1, 0, 1]]), softcap=c, return_lse=True),
             lambda c: paged.paged_attention(q[:, 0], kp, vp, tb, n, softcap=c, return_lse=True),
             lambda c: paged.sparse_attention(q[:, 0], kp, vp, tb, n, scores, 5, softcap=c, return_lse=True))
    for call in calls:
        want = call(0.0)
        for cap in (2.0 ** 64, 1e37):
            assert all(torch.equal(x, y) for x, y in zip(call(cap), want)), cap
        w, l = call(1e19)
        assert (w.float() - want[0].float()).abs().max() <= 2.0 ** -6 and (l - want[1]).abs().max() <= 2.0 ** -17


def long_sums(paged, cache, vec, n, rows, nodes, hq, hkv, hd):  # noqa: F811
    """Relative errors [some rows, nodes, heads, dims] of rows that all read one sequence of n positions, each of about the same
    weight, the values of every dim about a mean of its own in [1, 2]."""
    g = gen(21)
    ps, pages = 64, -(-(n + nodes) // 64)
    kp, vp = (torch.randn(pages, hkv, ps, hd, generator=g, device=DEV) for _ in range(2))
    vp = vp * 0.25 + 1 + torch.rand(hkv, 1, hd, generator=g, device=DEV)
    kp, vp = kp.to(TYPES[cache]), vp.to(TYPES[cache])
    table = torch.randperm(pages, generator=g, device=DEV)[None].cpu().numpy().astype(np.int32)
    q = torch.randn(rows, nodes, hq, hd, generator=g, device=DEV).mul_(0.2).to(TYPES[vec])
    parents = [[-1] + [0] * (nodes - 1)] * rows
    st = status()
    out, lse = paged.tree_attention(q, kp, vp, ints(table), ints([n] * rows), ints(parents), rows=ints([0] * rows), return_lse=True,
                                    status=st)
    paged.check_status(st)
    off = []
    for r in range(0, rows, max(1, rows // 4)):
        w, l, _, _ = plain_tree(q[r], kp, vp, table, n, 0, parents[r], 1 / math.sqrt(hd))
        off.append((out[r].double() - w) / w)
        # scores of 32-bit sums, exp2 and the maximum (scores below 2), the parts' rounding and sums that are rounded
        assert (lse[r].double() - l).abs().max() <= 2.0 ** -16
    return torch.stack(off)


@pytest.mark.parametrize("cache,nodes,rows,hq,hkv,hd", [
    ("f16", 4, 64, 8, 4, 64),        # a share to each warpgroup
    ("bf16", 4, 64, 8, 4, 64),
    ("bf16", 4, 64, 8, 4, 128),
    ("f16", 40, 52, 16, 4, 128),     # two blocks of parts
    ("bf16", 64, 16, 4, 2, 64),      # one block, tiles by turns
    ("f16", 16, 2, 16, 8, 128),
])
def test_long_sums_of_32_bits(paged, cache, nodes, rows, hq, hkv, hd):  # noqa: F811
    """The products of the values are cut off, not rounded: at most 128 of them are added before what they gave is put away,
    which is off by 128 2^-23 at most.  The rest, all of it roundings that know no direction, stays below 2^-19."""
    off = long_sums(paged, cache, "f32", 32768, rows, nodes, hq, hkv, hd)
    assert off.abs().max() <= 128 * 2.0 ** -23 + 2.0 ** -19


@pytest.mark.parametrize("nodes,rows", [(33, 80), (4, 160)])
def test_long_sums_of_16_bits(paged, nodes, rows):  # noqa: F811
    """The same with 512 products at a time, as the mean over many values, whose own roundings of up to 2^-12 cancel: 512 2^-23
    and three deviations, 2^-12 / sqrt(3 * 256) each, of the mean over 256 dims."""
    off = long_sums(paged, "f16", "f16", 131072, rows, nodes, 8, 2, 128)
    assert off.mean().abs() <= 512 * 2.0 ** -23 + 3 * 2.0 ** -12 / math.sqrt(3 * 256)


@pytest.mark.parametrize("nodes,rows", [(33, 80), (2, 160)])
def test_long_sums_of_bf16(paged, nodes, rows):  # noqa: F811
    """Of each 64 values 33 are 1 + 2^-7 and 31 are 1, whose mean lies 2^-13 above the middle of these neighbours; weights of about
    the same size (a deviation of 0.2, and of the mean 2^-7 * 0.2 / 2 / sqrt(n), 2e-6) hardly move it.  Sums that lose 2^-14
    of themselves at most leave it above, and it is rounded up."""
    g = gen(27)
    n, hkv, hd = 131072, 2, 64
    kp = torch.randn(n // 64 + 1, hkv, 64, hd, generator=g, device=DEV).bfloat16()
    vp = torch.ones_like(kp)
    vp[:, :, torch.randperm(64, generator=g, device=DEV)[:33]] = 1 + 2.0 ** -7
    q = torch.randn(rows, nodes, 4 * hkv, hd, generator=g, device=DEV).mul_(0.2).bfloat16()
    out = paged.tree_attention(q, kp, vp, ints([list(range(len(kp)))]), ints([n] * rows), ints([[-1] + [0] * (nodes - 1)] * rows),
                               rows=ints([0] * rows))
    assert torch.all(out == 1 + 2.0 ** -7)


@pytest.mark.parametrize("cache,vec,nodes,rows", [("f16", "f32", 4, 45), ("bf16", "f32", 4, 45), ("f16", "f16", 40, 45), ("bf16", "f32", 40, 25)])
@pytest.mark.parametrize("falling", [False, True])
def test_long_sums_under_growing_maxima(paged, cache, vec, nodes, rows, falling):  # noqa: F811
    """Scores that rise along the sequence by far more than a maximum may be passed by, so that what was put away is worth ever
    less, or fall, so that what comes is."""
    g = gen(29)
    n, hkv, hd = 24000, 4, 64
    kp, vp, table = make_cache(g, [n + nodes], hkv, hd, 64, cache)
    place = torch.empty(kp.shape[0], device=DEV)
    place[ints(table[0, :-1]).long()] = torch.linspace(0, 4, table.shape[1] - 1, device=DEV)
    kp = (kp.float() * (4 - place if falling else place)[:, None, None, None]).to(kp.dtype)
    q = torch.randn(rows, nodes, 2 * hkv, hd, generator=g, device=DEV).mul_(2).to(TYPES[vec])
    lens, parents = [n] * rows, [[-1] + [0] * (nodes - 1)] * rows
    out, lse = paged.tree_attention(q, kp, vp, ints(table), ints(lens), ints(parents), rows=ints([0] * rows), return_lse=True)
    for r in (0, rows - 1):
        check(q[r:r + 1], kp, vp, table, lens[:1], parents[:1], out[r:r + 1], lse[r:r + 1])


@pytest.mark.parametrize("cache,vec,nodes,rows", [("f16", "f32", 4, 40), ("bf16", "bf16", 40, 20), ("bf16", "f32", 40, 20)])
def test_long_sums_repeat_bit_for_bit(paged, cache, vec, nodes, rows):  # noqa: F811
    """Sums that are put away: the same call again, and two captured graphs at the same time on two streams."""
    g = gen(28)
    n, hkv, hd = 30000, 4, 64
    kp, vp, table = make_cache(g, [n + nodes], hkv, hd, 64, cache)
    tb, ls = ints(table), ints([n - 100 * r for r in range(rows)])
    tree, at = ints(trees(np.random.default_rng(28), rows, nodes, "random")), ints([0] * rows)
    qs = [torch.randn(rows, nodes, 4 * hkv, hd, generator=g, device=DEV).mul_(2).to(TYPES[vec]) for _ in range(2)]
    call = lambda q: paged.tree_attention(q, kp, vp, tb, ls, tree, rows=at, return_lse=True)  # noqa: E731
    want = [call(q) for q in qs]
    assert all(torch.isfinite(w[0]).all() for w in want)
    assert all(torch.equal(x, y) for x, y in zip(want[0], call(qs[0])))
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(q))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, y) for x, y in zip(w, o))


def test_a_window_of_one_past_a_full_table_is_reported(paged):  # noqa: F811
    """A sequence that fills its table: every node's own slot is past it.  Nothing is seen, and it is told, unless no node is there."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    g = gen(22)
    kp, vp, table = make_cache(g, [64, 64], 2, 64, 16, "f16")
    table = table[:, :4].copy()
    q = torch.randn(2, 3, 4, 64, generator=g, device=DEV).half()
    for window in (1, 2, 0):
        for parents, told in (([[-2, 0, 1], [-2, 0, 1]], False), ([[-2, 0, 1], [-2, -1, 1]], True), ([[-1, 0, 1]] * 2, True)):
            for lens in ([64, 64], [64, 100]):
                st = status()
                out, lse = paged.tree_attention(q, kp, vp, ints(table), ints(lens), ints(parents), window=window, return_lse=True, status=st)
                if told:
                    with pytest.raises(MkError) as e:
                        paged.check_status(st)
                    assert e.value.status == MK_ERR_PAGES and "tree" in str(e.value)
                else:
                    paged.check_status(st)
                if window == 1 or not told:
                    assert torch.all(out == 0) and torch.all(lse == -math.inf)


def test_a_wait_that_ran_out_is_told_as_one(paged):  # noqa: F811
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_TIMEOUT, MkError
    st = ints([MK_ERR_TIMEOUT, 6, -1, 17])
    with pytest.raises(MkError) as e:
        paged.check_status(st)
    assert e.value.status == MK_ERR_TIMEOUT and "wait" in str(e.value) and "bad page" not in str(e.value)
    paged.check_status(st)
