"""More operators over a paged key-value cache, as cases that can be timed: a tree of drafted tokens and
attention over chosen pages.

Five operators.  Two serve drafts: the attention of a tree of drafted tokens over a sequence's cache,
and the acceptance, which follows the tree along the tokens that the model chose and moves the accepted
tokens' keys and values to their places.  Three serve long contexts: the bounds of every page's keys,
a cheap score of every page for a query by those bounds, and the attention over the best pages.  `run`
computes each either in its plain form (elementary torch operations) or, with `own`, through the
package's entry points.  `exact` computes the same from the definitions in 64 bits.

Layout: a layer's pages are [n_pages, n_kv_heads, page_size, head_dim]; slot t of the sequence in table
row r lies in page table[r, t // page_size] at row t % page_size.  Slots 0..lens[r] - 1 hold the
sequence; node i of a tree lies in slot lens[r] + i.
"""
import math

import torch

own = False  # set from outside: the package's entry points instead of the plain form

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

# (query heads, kv heads, head_dim) of the package's model shapes, and wider groups
HEADS = ((4, 2, 64), (16, 8, 64), (16, 8, 128), (32, 8, 128), (8, 2, 64), (8, 8, 64), (32, 4, 128), (32, 2, 128))
DOUBLINGS = 7  # a tree has at most 2^7 nodes


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one sequence of the benchmark's length, a small tree: the latency of a drafted step
        dict(name="tree 8 x 512", kind="tree", rows=1, nodes=8, longest=512, spread=0.0, hq=16, hkv=8, hd=128, page=64,
             dtype="f16", qtype="f16", window=0, cap=0.0, shape="random", absent=0.0),
        # one long sequence; 32-bit queries and outputs, as the decode step keeps them
        dict(name="tree 16 x 32768", kind="tree", rows=1, nodes=16, longest=32768, spread=0.0, hq=16, hkv=8, hd=128,
             page=64, dtype="f16", qtype="f32", window=0, cap=0.0, shape="wide", absent=0.0),
        # a ragged batch of small trees (some smaller than the others), small heads and pages, a window, capped scores
        dict(name="tree 33 rows x 7 x 900", kind="tree", rows=33, nodes=7, longest=900, spread=0.97, hq=16, hkv=8, hd=64,
             page=16, dtype="bf16", qtype="bf16", window=400, cap=30.0, shape="random", absent=0.3),
        # a full batch of large trees at long contexts: the largest call
        dict(name="tree 16 rows x 64 x 32768", kind="tree", rows=16, nodes=64, longest=32768, spread=0.5, hq=32, hkv=8,
             hd=128, page=64, dtype="bf16", qtype="bf16", window=0, cap=0.0, shape="random", absent=0.0),
        # one sequence takes over four drafted tokens in every layer
        dict(name="accept 1 row", kind="accept", rows=1, nodes=8, deep=4, longest=600, layers=24, hkv=8, hd=64, page=16,
             dtype="bf16"),
        # a batch of large trees, up to twelve drafted tokens each
        dict(name="accept 64 rows", kind="accept", rows=64, nodes=61, deep=12, longest=150, layers=24, hkv=8, hd=128,
             page=64, dtype="f16"),
        # the bounds after one step of a batch: the page that grew
        dict(name="bounds 16 rows + 1", kind="bounds", rows=16, longest=8192, spread=0.5, new=1, hkv=8, hd=128, page=64,
             dtype="bf16"),
        # the bounds of whole prompts
        dict(name="bounds 16 x 8192", kind="bounds", rows=16, longest=8192, spread=0.5, new=8192, hkv=8, hd=128, page=32,
             dtype="f16"),
        # the pages' scores for one query of a long sequence; 32-bit queries
        dict(name="score 1 x 32768", kind="score", rows=1, longest=32768, spread=0.0, hq=16, hkv=8, hd=128, page=64,
             dtype="f16", qtype="f32"),
        # and for a ragged batch, small pages
        dict(name="score 16 x 32768 ragged", kind="score", rows=16, longest=32768, spread=0.5, hq=32, hkv=8, hd=128,
             page=16, dtype="bf16", qtype="bf16"),
        # one long sequence, a sixteenth of its pages
        dict(name="sparse 1 x 32768", kind="sparse", rows=1, longest=32768, spread=0.0, blocks=32, hq=16, hkv=8, hd=128,
             page=64, dtype="f16", qtype="f32", cap=0.0),
        # a ragged batch, 4096 positions of each sequence
        dict(name="sparse 16 x 32768 ragged", kind="sparse", rows=16, longest=32768, spread=0.5, blocks=128, hq=32, hkv=8,
             hd=128, page=32, dtype="bf16", qtype="bf16", cap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(("tree", "tree", "accept", "bounds", "score", "sparse"))
    hq, hkv, hd = rng.choice(HEADS)
    page = rng.choice((16, 32, 48, 64, 128))
    dtype = rng.choice(("f16", "bf16"))
    qtype = rng.choice((dtype, dtype, "f32"))
    spread = rng.choice((0.0, 0.5, 0.97))
    if kind == "tree":
        rows, nodes = _log(rng, 1, 64), _log(rng, 1, 128)
        most = min(32768, 16 * 32768 * 8 * 128 // (rows * hkv * hd), 16 * 32768 * 32 * 64 * 128 // (rows * hq * nodes * hd))
        return dict(kind=kind, rows=rows, nodes=nodes, longest=_log(rng, 1, most), spread=spread, hq=hq, hkv=hkv, hd=hd,
                    page=page, dtype=dtype, qtype=qtype, window=rng.choice((0, 0, _log(rng, 1, 4096))),
                    cap=rng.choice((0.0, 0.0, 30.0)), shape=rng.choice(("chain", "random", "wide")),
                    absent=rng.choice((0.0, 0.5)))
    if kind == "accept":
        nodes = _log(rng, 1, 64)
        return dict(kind=kind, rows=_log(rng, 1, 64), nodes=nodes, deep=rng.randint(0, min(12, nodes - 1)),
                    longest=_log(rng, 1, 150), layers=rng.randint(1, 24), hkv=hkv, hd=hd, page=rng.choice((16, 32, 48, 64)),
                    dtype=dtype)
    rows = _log(rng, 1, 32)
    if kind == "bounds":
        longest = _log(rng, 1, min(8192, 16 * 8192 * 8 * 128 // (rows * hkv * hd)))
        return dict(kind=kind, rows=rows, longest=longest, spread=spread, new=rng.choice((1, _log(rng, 1, longest), longest)),
                    hkv=hkv, hd=hd, page=page, dtype=dtype)
    longest = _log(rng, 1, min(32768, 16 * 32768 * 8 * 128 // (rows * hkv * hd)))
    if kind == "score":
        return dict(kind=kind, rows=rows, longest=longest, spread=spread, hq=hq, hkv=hkv, hd=hd, page=page, dtype=dtype,
                    qtype=qtype)
    return dict(kind=kind, rows=rows, longest=longest, spread=spread, blocks=_log(rng, 2, max(2, 4096 // page)), hq=hq,
                hkv=hkv, hd=hd, page=page, dtype=dtype, qtype=qtype, cap=rng.choice((0.0, 0.0, 30.0)))


# ------------------------------------------------------------------------- sizes of a case
def _lens(c):
    """The rows' lengths: the same ones for every seed, in an order of the seed's."""
    n = c["rows"]
    return [max(1, int(round(c["longest"] * (1 - c.get("spread", 0.7) * ((i * 0.6180339887498949) % 1.0))))) for i in range(n)]


def _accepted(c):
    """Drafted tokens that each row accepts."""
    return [int(round(c["deep"] * (1 - 0.8 * ((i * 0.6180339887498949) % 1.0)))) for i in range(c["rows"])]


def _pages(c, n):
    return -(-n // c["page"])


def work(c):
    s = SIZE[c["dtype"]]
    vec = c["hkv"] * c["hd"] * s                                    # a position's keys, or its values
    if c["kind"] == "accept":
        # the accepted tokens' keys and values of every layer read and written once, the tree read, the tokens written
        return {"bytes": 2 * sum(_accepted(c)) * c["layers"] * 2 * vec + 20 * c["rows"] * c["nodes"], "flops": 0}
    if c["kind"] == "bounds":
        # the pages that hold new positions, up to their last one; a lower and an upper bound of each
        spans = [(max(0, n - c["new"]) // c["page"], n) for n in _lens(c)]
        held = sum(n - first * c["page"] for first, n in spans)
        pages = sum(_pages(c, n) - first for first, n in spans)
        return {"bytes": (held + 2 * pages) * vec, "flops": 2 * held * c["hkv"] * c["hd"]}
    heads = c["hq"] * c["hd"]
    if c["kind"] == "tree":
        # the visible keys and values once, queries and outputs
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c)) + c["rows"] * c["nodes"]
        return {"bytes": 2 * seen * vec + 2 * c["rows"] * c["nodes"] * heads * SIZE[c["qtype"]],
                "flops": 4 * seen * c["nodes"] * heads}
    pages = sum(_pages(c, n) for n in _lens(c))
    if c["kind"] == "score":
        return {"bytes": 2 * pages * vec + c["rows"] * heads * SIZE[c["qtype"]] + 4 * pages * c["hkv"],
                "flops": 4 * pages * heads}
    # the chosen pages' keys and values once, the scores, queries and outputs
    seen = sum(min(n, c["blocks"] * c["page"]) for n in _lens(c))
    return {"bytes": 2 * seen * vec + 2 * c["rows"] * heads * SIZE[c["qtype"]] + 4 * pages * c["hkv"], "flops": 4 * seen * heads}


# --------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(*shape, generator=g, device=DEV, dtype=dtype)
    return x.mul_(scale) if scale != 1.0 else x


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _perm(g, n):
    return torch.randperm(n, generator=g, device=DEV)


def _int(x):
    return x.to(device=DEV, dtype=torch.int32)


def _status():
    return torch.zeros(4, device=DEV, dtype=torch.int32)


def prepare(c, seed):
    g = _gen(seed)
    if c["kind"] == "accept":
        return _prepare_accept(c, g)
    return {"tree": _prepare_tree, "bounds": _prepare_bounds, "score": _prepare_score, "sparse": _prepare_sparse}[c["kind"]](
        c, g, *_prepare_table(c, g, c.get("nodes", 0)))


def _prepare_table(c, g, more):
    """Rows of _lens(c) positions and `more` slots behind them, their pages scattered over a pool."""
    ps = c["page"]
    lens = torch.tensor(_lens(c), device=DEV)[_perm(g, c["rows"])]
    need = (lens + more + ps - 1) // ps
    total = sum(_pages(c, n + more) for n in _lens(c))
    at = torch.cumsum(need, 0) - need
    i = torch.arange(_pages(c, c["longest"] + more) + 1, device=DEV)
    ids = _perm(g, total + 3)
    table = torch.where(i[None] < need[:, None], ids[(at[:, None] + i[None]).clamp_max(total - 1)], -1)
    return _int(lens), _int(table), total + 3


def _query(c, g, *lead):
    """Queries as views of the fused q/k/v rows that a model's projection gives."""
    qkv = _randn(g, *lead, c["hq"] + 2 * c["hkv"], c["hd"], scale=1.5).to(TYPES[c["qtype"]])
    return qkv[..., : c["hq"], :]


def _tree(c, g):
    """Parents before their children; node 0 is the one root.  Rows may have fewer nodes than the widest tree."""
    r, n = c["rows"], c["nodes"]
    i = torch.arange(n, device=DEV)[None].expand(r, n)
    if c["shape"] == "chain":
        parent = i - 1
    elif c["shape"] == "wide":
        parent = torch.div(i - 1, 4, rounding_mode="floor")
    else:
        parent = torch.where(i > 0, (_rand(g, r, n) * i).long().clamp_max(n - 1).minimum((i - 1).clamp_min(0)), -1)
    held = n - (_rand(g, r, 1) * c["absent"] * n).long()
    return _int(torch.where(i < held.clamp_min(1), parent, -2))


def _prepare_tree(c, g, lens, table, n_pages):
    """A tree's queries; its keys and values lie behind the sequence's, as the append has left them there."""
    shape = (n_pages, c["hkv"], c["page"], c["hd"])
    k, v = (_randn(g, *shape, dtype=TYPES[c["dtype"]], scale=0.9) for _ in range(2))
    return dict(kind="tree", q=_query(c, g, c["rows"], c["nodes"]), k_pages=k, v_pages=v, table=table, lens=lens,
                parents=_tree(c, g), window=c["window"], cap=c["cap"], scale=1.0 / math.sqrt(c["hd"]), status=_status())


def _prepare_accept(c, g):
    """Trees whose model choices follow one branch of _accepted(c) drafted tokens; the other nodes' choices lead nowhere."""
    r, n, ps = c["rows"], c["nodes"], c["page"]
    order = _perm(g, r)
    deep = torch.tensor(_accepted(c), device=DEV)[order]
    lens = torch.tensor(_lens(c), device=DEV)[order]
    i = torch.arange(n, device=DEV)[None].expand(r, n)
    # the branch: node 0 and `deep` others, by chance
    key = torch.where(i > 0, _rand(g, r, n), -1.0)
    on = key.argsort(1).argsort(1) <= deep[:, None]
    before = torch.cummax(torch.where(on, i, -1), 1).values.roll(1, 1)           # the last branch node before each
    before[:, 0] = -1
    other = (_rand(g, r, n) * i).long().minimum((i - 1).clamp_min(0))
    parent = torch.where(on, before, other)
    tokens = torch.rand(r, 32000, generator=g, device=DEV).argsort(1)[:, : 2 * n]   # all of them different
    choices = tokens[:, n:].clone()
    child = torch.where(on & (i > 0), i, 0)
    choices.scatter_(1, torch.where(on & (i > 0), before, n - 1).clamp_min(0),
                     torch.where(on & (i > 0), tokens.gather(1, child), choices[:, n - 1:]))
    last = torch.where(on, i, -1).amax(1, keepdim=True)
    choices.scatter_(1, last, 32000 + _int(_rand(g, r, 1) * 1000).long())
    width = _pages(c, c["longest"] + n) + 1
    need = (lens + n + ps - 1) // ps
    at = torch.cumsum(need, 0) - need
    total = sum(_pages(c, m + n) for m in _lens(c))
    ids = _perm(g, total + 2)
    j = torch.arange(width, device=DEV)
    table = torch.where(j[None] < need[:, None], ids[(at[:, None] + j[None]).clamp_max(total - 1)], -1)
    pages = _randn(g, 2, c["layers"], total + 2, c["hkv"], ps, c["hd"], dtype=TYPES[c["dtype"]])
    return dict(kind="accept", k=pages[0], v=pages[1], table=_int(table), lens0=_int(lens), lens=_int(lens),
                tokens=_int(tokens[:, :n]), parents=_int(parent), choices=_int(choices), status=_status())


def _prepare_bounds(c, g, lens, table, n_pages):
    """Pages whose new positions have just been appended, and the bounds that earlier calls left."""
    k = _randn(g, n_pages, c["hkv"], c["page"], c["hd"], dtype=TYPES[c["dtype"]], scale=0.9)
    bounds = _randn(g, n_pages, c["hkv"], 2, c["hd"], dtype=TYPES[c["dtype"]])
    return dict(kind="bounds", k_pages=k, bounds=bounds, table=table, lens=lens, new=c["new"], status=_status())


def _prepare_score(c, g, lens, table, n_pages):
    """Bounds as pages of normally distributed keys have them."""
    mid = _randn(g, n_pages, c["hkv"], 1, c["hd"], scale=0.4)
    half = 1.8 + 0.4 * _rand(g, n_pages, c["hkv"], 1, c["hd"])
    bounds = torch.cat((mid - half, mid + half), 2).to(TYPES[c["dtype"]])
    return dict(kind="score", q=_query(c, g, c["rows"]), bounds=bounds, table=table, lens=lens, page=c["page"],
                status=_status())


def _prepare_sparse(c, g, lens, table, n_pages):
    """One new query per sequence and the scores of its pages; -inf where there is no page."""
    shape = (n_pages, c["hkv"], c["page"], c["hd"])
    k, v = (_randn(g, *shape, dtype=TYPES[c["dtype"]], scale=0.9) for _ in range(2))
    scores = _randn(g, c["rows"], c["hkv"], table.shape[1], scale=6.0) + 80.0
    there = torch.arange(table.shape[1], device=DEV)[None, None] * c["page"] < lens[:, None, None]
    return dict(kind="sparse", q=_query(c, g, c["rows"]), k_pages=k, v_pages=v, table=table, lens=lens,
                scores=torch.where(there, scores, -math.inf), blocks=c["blocks"], cap=c["cap"],
                scale=1.0 / math.sqrt(c["hd"]), status=_status())


# -------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        from persistent_sm_decode_megakernel_gb300 import paged
        if s["kind"] == "tree":
            return paged.tree_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["parents"],
                                        scale=s["scale"], softcap=s["cap"], window=s["window"], return_lse=True,
                                        status=s["status"])
        if s["kind"] == "accept":
            s["lens"].copy_(s["lens0"])
            accepted = paged.accept_drafts(s["k"], s["v"], s["table"], s["lens"], s["tokens"], s["parents"], s["choices"],
                                           status=s["status"])
            return (*accepted, s["lens"], s["k"], s["v"])
        if s["kind"] == "bounds":
            paged.update_bounds(s["k_pages"], s["bounds"], s["table"], s["lens"], new=s["new"], status=s["status"])
            return s["bounds"]
        if s["kind"] == "score":
            return paged.page_scores(s["q"], s["bounds"], s["table"], s["lens"], s["page"], status=s["status"])
        return paged.sparse_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["scores"], s["blocks"],
                                      scale=s["scale"], softcap=s["cap"], return_lse=True, return_pages=True,
                                      status=s["status"])
    return {"tree": _run_tree, "accept": _run_accept, "bounds": _run_bounds, "score": _run_score, "sparse": _run_sparse}[
        s["kind"]](s)


def _ancestors(parents):
    """[rows, i, j] 1 where j is i or an ancestor of i: the sum of the powers of the parent matrix, by squaring."""
    n = parents.shape[1]
    j = torch.arange(n, device=parents.device)
    power = ((parents[:, :, None] == j) & (j[None, None] < j[None, :, None])).float()
    total = torch.eye(n, device=parents.device) + power
    for _ in range(DOUBLINGS - 1):
        power = torch.matmul(power, power)
        total = total + torch.matmul(total, power)
    return total


def _softmax_values(score, seen, v):
    """Softmax over the last dim where `seen`, the weighted values [.., positions, dims], and the log-sum-exp."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    z = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(z == 0, 1.0, z), (top + torch.log(z))[..., 0]


def _run_tree(s):
    q, ps, lens = s["q"].float(), s["k_pages"].shape[2], s["lens"].long()
    r, n, hq, hd = q.shape
    hkv = s["k_pages"].shape[1]
    at = s["table"].long().clamp_min(0)
    k = s["k_pages"][at].float().transpose(1, 2).reshape(r, hkv, -1, hd)      # [rows, kv heads, slots, head_dim]
    v = s["v_pages"][at].float().transpose(1, 2).reshape(r, hkv, -1, hd)
    above = _ancestors(s["parents"])
    depth = above.sum(2) - 1                                                  # [rows, nodes]
    there = torch.matmul(above, (s["parents"] == -1).float()[..., None])[..., 0] > 0
    t = torch.arange(k.shape[2], device=q.device)
    node = (t[None] - lens[:, None]).clamp(0, n - 1)                          # of each slot
    tree = (above.gather(2, node[:, None].expand(r, n, -1)) > 0) & (t[None] >= lens[:, None])[:, None]
    tree = tree & (t[None] < lens[:, None] + n)[:, None]
    place = torch.where(t[None] < lens[:, None], t[None], lens[:, None] + depth.gather(1, node).long())   # position of a slot
    seen = tree | (t[None] < lens[:, None])[:, None]
    if s["window"]:
        seen = seen & (place[:, None] > (lens[:, None] + depth.long() - s["window"])[..., None])
    seen = seen & there[..., None]
    held = (t[None] < lens[:, None] + n)[:, None, :, None]
    score = torch.matmul(q.view(r, n, hkv, hq // hkv, hd).transpose(1, 2).reshape(r, hkv, -1, hd), k.transpose(2, 3)) * s["scale"]
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    seen = seen.repeat_interleave(hq // hkv, 1)[:, None]
    out, lse = _softmax_values(score, seen, torch.where(held, v, 0.0))
    out = out.view(r, hkv, n, hq // hkv, hd).transpose(1, 2).reshape(r, n, hq, hd)
    return out.to(s["q"].dtype), lse.view(r, hkv, n, hq // hkv).transpose(1, 2).reshape(r, n, hq)


def _run_accept(s):
    """A node is accepted if every node of its way from node 0 is the first child whose token its parent's choice is."""
    s["lens"].copy_(s["lens0"])
    parents, tokens, choices, lens, table, ps = s["parents"].long(), s["tokens"], s["choices"], s["lens"], s["table"], s["k"].shape[3]
    r, n = parents.shape
    i = torch.arange(n, device=parents.device)
    wanted = (choices.gather(1, parents.clamp_min(0)) == tokens) & (parents >= 0)
    twin = wanted[:, None] & wanted[:, :, None] & (parents[:, None] == parents[:, :, None]) & (i[None] < i[:, None])[None]
    good = (wanted & ~twin.any(2)) | (i == 0)
    above = _ancestors(s["parents"])
    on = (torch.matmul(above, good.float()[..., None])[..., 0] == above.sum(2)) & (above[:, :, 0] > 0)
    count = on.sum(1)
    path = torch.sort(torch.where(on, i, n), 1).values
    held = i[None] < count[:, None]
    path = torch.where(held, path, -1)
    token = torch.where(held, choices.gather(1, path.clamp_min(0)), -1)
    # the accepted nodes' keys and values, from slot lens + path[j] to slot lens + j
    row, j = torch.nonzero(held & (path != i[None]), as_tuple=True)
    src, dst = lens[row].long() + path[row, j], lens[row].long() + j
    sp, dp = table[row, src // ps].long(), table[row, dst // ps].long()
    s["k"][:, dp, :, dst % ps] = s["k"][:, sp, :, src % ps]
    s["v"][:, dp, :, dst % ps] = s["v"][:, sp, :, src % ps]
    lens += count.int()
    return token.int(), path.int(), count.int(), lens, s["k"], s["v"]


def _run_bounds(s):
    k, table, lens, ps = s["k_pages"], s["table"], s["lens"].long(), s["k_pages"].shape[2]
    j = torch.arange(table.shape[1], device=k.device)[None]
    row, page = torch.nonzero((j * ps < lens[:, None]) & ((j + 1) * ps > lens[:, None] - s["new"]), as_tuple=True)
    at = table[row, page].long()
    held = (page[:, None] * ps + torch.arange(ps, device=k.device)[None] < lens[row][:, None])[:, None, :, None]
    keys = k[at].float()
    low = torch.where(held, keys, math.inf).amin(2)
    high = torch.where(held, keys, -math.inf).amax(2)
    s["bounds"][at] = torch.stack((low, high), 2).to(k.dtype)
    return s["bounds"]


def _run_score(s):
    """Of each head the largest product that keys within the bounds can have; the largest of the heads of a group."""
    q, hkv = s["q"].float(), s["bounds"].shape[1]
    r, hq, hd = q.shape
    b = s["bounds"][s["table"].long().clamp_min(0)].float()                   # [rows, pages, kv heads, 2, head_dim]
    q = q.view(r, hkv, hq // hkv, hd)
    score = torch.matmul(q.clamp_max(0), b[:, :, :, 0].permute(0, 2, 3, 1)) + torch.matmul(q.clamp_min(0), b[:, :, :, 1].permute(0, 2, 3, 1))
    there = torch.arange(b.shape[1], device=q.device)[None] * s["page"] < s["lens"][:, None]
    return torch.where(there[:, None], score.amax(2), -math.inf)


def _run_sparse(s):
    """The first and the last page and the best others, ties to the lowest; then attention over their positions."""
    q, ps, lens, n = s["q"].float(), s["k_pages"].shape[2], s["lens"].long(), s["blocks"]
    r, hq, hd = q.shape
    hkv = s["k_pages"].shape[1]
    width = s["scores"].shape[2]
    j = torch.arange(width, device=q.device)
    pages = ((lens + ps - 1) // ps)[:, None, None]
    forced = (j == 0) | (j == pages - 1)
    key = torch.where(forced, math.inf, torch.nan_to_num(s["scores"], nan=3e38, posinf=3e38, neginf=-3e38))
    order = torch.sort(torch.where(j < pages, key, -math.inf), dim=-1, descending=True, stable=True).indices[..., :n]
    chosen = torch.sort(torch.where(order < pages, order, width), -1).values   # [rows, kv heads, blocks], none behind
    none = chosen == width
    at = s["table"].long()[:, None].expand(r, hkv, -1).gather(2, chosen.clamp_max(width - 1)).clamp_min(0)
    head = torch.arange(hkv, device=q.device)[None, :, None]
    k, v = (x[at, head].float().view(r, hkv, -1, hd) for x in (s["k_pages"], s["v_pages"]))
    t = (chosen[..., None] * ps + torch.arange(ps, device=q.device)).view(r, hkv, 1, -1)
    seen = (t < lens[:, None, None, None]) & ~none.repeat_interleave(ps, 2)[:, :, None]
    score = torch.matmul(q.view(r, hkv, hq // hkv, hd), k.transpose(2, 3)) * s["scale"]
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    out, lse = _softmax_values(score, seen, torch.where(seen.transpose(2, 3), v, 0.0))
    chosen = torch.where(none, -1, chosen)
    if chosen.shape[2] < n:  # a table narrower than the pages asked for
        chosen = torch.cat((chosen, chosen.new_full((r, hkv, n - chosen.shape[2]), -1)), 2)
    return out.view(r, hq, hd).to(s["q"].dtype), lse.view(r, hq), chosen.int()


# ---------------------------------------------------------------------------- in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "accept":
        return None  # keys and values are moved, nothing is computed
    lens, ps = s["lens"].tolist(), c["page"]
    if c["kind"] == "bounds":
        b = s["bounds"].double()
        for r, n in enumerate(lens):
            for j in range(max(0, n - c["new"]) // ps, -(-n // ps)):
                keys = s["k_pages"][s["table"][r, j].long(), :, : n - j * ps].double()
                b[s["table"][r, j].long()] = torch.stack((keys.min(1).values, keys.max(1).values), 1)
        return b
    group = c["hq"] // c["hkv"]
    if c["kind"] == "score":
        got = torch.full((c["rows"], c["hkv"], s["table"].shape[1]), -math.inf, device=DEV, dtype=torch.float64)
        for r, n in enumerate(lens):
            b = s["bounds"][s["table"][r, : -(-n // ps)].long()].double()     # [pages, kv heads, 2, head_dim]
            for h in range(c["hkv"]):
                q = s["q"][r, h * group: (h + 1) * group].double()
                got[r, h, : b.shape[0]] = torch.maximum(q[:, None] * b[None, :, h, 0], q[:, None] * b[None, :, h, 1]).sum(-1).amax(0)
        return got
    out, lse = [], []

    def attend(q, k, v, seen):
        z = torch.einsum("gd,td->gt", q, k) * s["scale"]
        if c["cap"]:
            z = c["cap"] * torch.tanh(z / c["cap"])
        z = z.masked_fill(~seen, -math.inf)
        return torch.softmax(z, -1) @ v, torch.logsumexp(z, -1)

    if c["kind"] == "sparse":
        for r, n in enumerate(lens):
            pages = -(-n // ps)
            for h in range(c["hkv"]):
                z = s["scores"][r, h, :pages].tolist()
                best = sorted(range(pages), key=lambda j: (j not in (0, pages - 1), -z[j], j))[: c["blocks"]]
                ids = s["table"][r].long()[torch.tensor(sorted(best), device=DEV)]
                k, v = (x[ids, h].double().reshape(-1, c["hd"])[: n - (pages - len(best)) * ps] for x in (s["k_pages"], s["v_pages"]))
                o, z = attend(s["q"][r, h * group: (h + 1) * group].double(), k, v, torch.ones((), device=DEV, dtype=torch.bool))
                out.append(o)
                lse.append(z)
        return torch.stack(out).view(c["rows"], c["hq"], c["hd"]), torch.stack(lse).view(c["rows"], c["hq"]), None
    for r, (n, parents) in enumerate(zip(lens, s["parents"].tolist())):
        ids = s["table"][r, : -(-(n + c["nodes"]) // ps)].long()
        k, v = (x[ids].permute(1, 0, 2, 3).reshape(c["hkv"], -1, c["hd"])[:, : n + c["nodes"]].double() for x in (s["k_pages"], s["v_pages"]))
        depth, sees, there = [], [], []
        for i, p in enumerate(parents):
            up = 0 <= p < i
            depth.append(depth[p] + 1 if up else 0)
            sees.append((sees[p] if up else []) + [i])
            there.append(there[p] if up else p == -1)
        seen = torch.zeros(c["nodes"], n + c["nodes"], dtype=torch.bool)
        for i in range(c["nodes"]):
            if there[i]:
                lo = n + depth[i] + 1 - c["window"] if c["window"] else 0
                seen[i, max(0, lo): n] = True
                seen[i, [n + j for j in sees[i] if n + depth[j] >= lo]] = True
        seen = seen.to(DEV).repeat_interleave(group, 0)
        q = s["q"][r].double().view(c["nodes"], c["hkv"], group, c["hd"])
        o, z = zip(*(attend(q[:, h].reshape(-1, c["hd"]), k[h], v[h], seen) for h in range(c["hkv"])))
        gone = ~torch.tensor(there, device=DEV)
        o = torch.stack(o, 1).view(c["nodes"], group, c["hkv"], c["hd"]).transpose(1, 2).reshape(c["nodes"], c["hq"], c["hd"])
        z = torch.stack(z, 1).view(c["nodes"], group, c["hkv"]).transpose(1, 2).reshape(c["nodes"], c["hq"])
        out.append(o.masked_fill(gone[:, None, None], 0.0))
        lse.append(z.masked_fill(gone[:, None], -math.inf))
    return torch.stack(out), torch.stack(lse)
