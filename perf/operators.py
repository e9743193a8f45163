"""The operators of decoding over a paged key-value cache, as cases that can be timed.

Four operators, used together by a beam search or a serving loop: rotary positions with the
append into the pages, attention of one new token over the pages, the page table's update
(fork, free, reserve, compact) and the selection over beams and vocabulary.  `run` computes
each either in its plain form (elementary torch operations) or, with `own`, through the
package's entry points.  `exact` computes the same from the definitions in 64 bits.

Layout: a layer's pages are [n_pages, n_kv_heads, page_size, head_dim]; position t of the
sequence in table row r lies in page table[r, t // page_size] at row t % page_size.
"""
import math

import torch

own = False  # set from outside: the package's entry points instead of the plain form

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

# (query heads, kv heads, head_dim) of the package's model shapes, and two wider groups
HEADS = ((4, 2, 64), (16, 8, 64), (16, 8, 128), (32, 8, 128), (8, 2, 64), (8, 8, 64), (32, 4, 128), (32, 2, 128))


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of one sequence, the fused q/k/v row of a 16-head model
        dict(name="append 1 token", kind="append", tokens=1, seqs=1, hq=16, hkv=8, hd=128, page=64, dtype="f16",
             rot=128, inter=False, far=512),
        # one decode step of a ragged batch, far positions, the interleaved layout on half of the head
        dict(name="append 48 tokens", kind="append", tokens=48, seqs=48, hq=32, hkv=8, hd=128, page=16, dtype="bf16",
             rot=64, inter=True, far=1000000),
        # a long prompt written in one call
        dict(name="append 8192 tokens", kind="append", tokens=8192, seqs=1, hq=32, hkv=8, hd=128, page=64,
             dtype="bf16", rot=128, inter=False, far=0),
        # the benchmark's context: one sequence at 512 positions
        dict(name="attend 1 x 512", kind="attend", rows=1, longest=512, spread=0.0, hq=16, hkv=8, hd=128, page=64,
             dtype="f16", qtype="f16", window=0, cap=0.0),
        # one long sequence: the work has to be split over its length; 32-bit queries and outputs, as
        # the decode step keeps them
        dict(name="attend 1 x 32768", kind="attend", rows=1, longest=32768, spread=0.0, hq=16, hkv=8, hd=128,
             page=64, dtype="f16", qtype="f32", window=0, cap=0.0),
        # many short sequences of ragged lengths, small heads, small pages, a window and capped scores
        dict(name="attend 61 x 700 ragged", kind="attend", rows=61, longest=700, spread=0.97, hq=16, hkv=8, hd=64,
             page=16, dtype="bf16", qtype="bf16", window=400, cap=30.0),
        # a full batch at long contexts: the largest call
        dict(name="attend 16 x 32768 ragged", kind="attend", rows=16, longest=32768, spread=0.5, hq=32, hkv=8,
             hd=128, page=32, dtype="bf16", qtype="bf16", window=0, cap=0.0),
        # one group of four beams: the rows follow their parents, partial pages become private
        dict(name="fork 4 rows", kind="fork", groups=1, beams=4, kept=2, longest=600, layers=24, hkv=8, hd=64,
             page=16, dtype="bf16", reserve=1),
        # sixteen groups of eight beams over every layer's pages
        dict(name="fork 128 rows", kind="fork", groups=16, beams=8, kept=3, longest=900, layers=24, hkv=8, hd=128,
             page=32, dtype="f16", reserve=40),
        # a fragmented cache pushed together
        dict(name="compact 1500 pages", kind="compact", pages=1500, used=0.6, layers=24, hkv=8, hd=64, page=16,
             dtype="bf16"),
        # one group of four beams over a small vocabulary
        dict(name="select 4 of 32000", kind="select", groups=1, beams=4, vocab=32000, dtype="f32", done=0.0),
        # sixteen groups of eight beams over the large vocabulary, some of them finished
        dict(name="select 16 x 8 of 128256", kind="select", groups=16, beams=8, vocab=128256, dtype="f32", done=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("append", "attend", "attend", "fork", "compact", "select"))
    hq, hkv, hd = rng.choice(HEADS)
    page = rng.choice((16, 32, 48, 64, 128))
    dtype = rng.choice(("f16", "bf16"))
    if kind == "append":
        tokens = _log(rng, 1, 8192)
        return dict(kind=kind, tokens=tokens, seqs=rng.randint(1, min(tokens, 64)), hq=hq, hkv=hkv, hd=hd, page=page,
                    dtype=dtype, rot=rng.choice((hd, hd // 2, hd // 4)), inter=rng.random() < 0.5,
                    far=rng.choice((0, _log(rng, 1, 4000000))))
    if kind == "attend":
        rows = _log(rng, 1, 64)
        most = min(32768, 16 * 32768 * 8 * 128 // (rows * hkv * hd))
        return dict(kind=kind, rows=rows, longest=_log(rng, 1, most), spread=rng.choice((0.0, 0.5, 0.97)), hq=hq,
                    hkv=hkv, hd=hd, page=page, dtype=dtype, qtype=rng.choice((dtype, dtype, "f32")),
                    window=rng.choice((0, 0, _log(rng, 1, 4096))), cap=rng.choice((0.0, 0.0, 30.0)))
    if kind == "fork":
        beams = rng.randint(1, 8)
        return dict(kind=kind, groups=_log(rng, 1, 16), beams=beams, kept=rng.randint(1, beams),
                    longest=_log(rng, 2, 900), layers=rng.randint(1, 24), hkv=hkv, hd=hd, page=rng.choice((16, 32, 48)),
                    dtype=dtype, reserve=rng.choice((1, _log(rng, 1, 200))))
    if kind == "compact":
        return dict(kind=kind, pages=_log(rng, 8, 1500), used=rng.uniform(0.2, 0.9), layers=rng.randint(1, 24),
                    hkv=min(hkv, 8), hd=64, page=16, dtype=dtype)
    beams = rng.randint(1, 16)
    return dict(kind=kind, groups=_log(rng, 1, 128 // beams), beams=beams, vocab=_log(rng, 50, 128256),
                dtype=rng.choice(("f32", "f16", "bf16")), done=rng.choice((0.0, 0.2)))


# ------------------------------------------------------------------------- sizes of a case
def _lens(c):
    """The rows' lengths: the same ones for every seed, in an order of the seed's."""
    n = c["rows"]
    return [max(1, int(round(c["longest"] * (1 - c["spread"] * ((i * 0.6180339887498949) % 1.0))))) for i in range(n)]


def _group_lens(c):
    """A length per group of beams, never on a page's border, so that every copy is of one page."""
    got = []
    for g in range(c["groups"]):
        n = max(1, int(round(c["longest"] * (1 - 0.7 * ((g * 0.6180339887498949) % 1.0)))))
        got.append(n + 1 if n % c["page"] == 0 else n)
    return got


def _moved(c):
    """Of `used` pages spread over the pool, those that lie behind the first `used` places."""
    used = max(1, int(c["pages"] * c["used"]))
    return used, min(used, c["pages"] - used) * 3 // 4


def work(c):
    s = SIZE[c["dtype"]]
    if c["kind"] == "append":
        # every vector read and written once; the rotation's products and sums
        elems = c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["hd"]
        return {"bytes": 2 * elems * s + 8 * c["tokens"], "flops": c["tokens"] * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    if c["kind"] == "attend":
        # the visible keys and values once, queries and outputs
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c))
        qo = c["rows"] * c["hq"] * c["hd"] * SIZE[c["qtype"]]
        return {"bytes": 2 * seen * c["hkv"] * c["hd"] * s + 2 * qo, "flops": 4 * seen * c["hq"] * c["hd"]}
    if c["kind"] == "select":
        n = c["groups"] * c["beams"] * c["vocab"]
        return {"bytes": n * s, "flops": 4 * n}
    page = c["hkv"] * c["page"] * c["hd"] * s * 2 * c["layers"]
    if c["kind"] == "fork":
        # one private page per beam that shares its parent, read and written in every layer; the table
        copies = c["groups"] * (c["beams"] - c["kept"])
        return {"bytes": 2 * copies * page + 8 * sum(-(-n // c["page"]) for n in _group_lens(c)) * c["beams"], "flops": 0}
    used, moved = _moved(c)
    return {"bytes": 2 * moved * page + 8 * c["pages"], "flops": 0}


# --------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(*shape, generator=g, device=DEV, dtype=dtype)
    return x.mul_(scale) if scale != 1.0 else x


def _perm(g, n):
    return torch.randperm(n, generator=g, device=DEV)


def _int(x):
    return x.to(device=DEV, dtype=torch.int32)


def prepare(c, seed):
    g = _gen(seed)
    return {"append": _prepare_append, "attend": _prepare_attend, "fork": _prepare_fork, "compact": _prepare_compact,
            "select": _prepare_select}[c["kind"]](c, g)


def _prepare_append(c, g):
    """The fused q/k/v rows of a step (k and v are strided views of them) and the pages they go to."""
    t, hq, hkv, hd, ps, dt = c["tokens"], c["hq"], c["hkv"], c["hd"], c["page"], TYPES[c["dtype"]]
    qkv = _randn(g, t, hq + 2 * hkv, hd, dtype=dt)
    # tokens dealt to the sequences in runs; a sequence's run starts at an offset into its own pages
    seqs = c["seqs"]
    row = torch.arange(t, device=DEV) * seqs // t
    first = torch.searchsorted(row, torch.arange(seqs, device=DEV))
    start = torch.randint(0, ps, (seqs,), generator=g, device=DEV)
    local = torch.arange(t, device=DEV) - first[row] + start[row]
    each = -(-(-(-t // seqs) + ps) // ps) + 1                       # pages a sequence writes at most
    skip = c["far"] // ps                                           # pages before them, none of them written
    n_pages = seqs * each + max(2, seqs * each // 8)
    table = torch.full((seqs, skip + each), -1, device=DEV, dtype=torch.int32)
    table[:, skip:] = _int(_perm(g, n_pages)[: seqs * each].view(seqs, each))
    inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
    if c["far"]:
        inv = inv / 8.0                                             # positions scaled for a long context
    pages = _randn(g, 2, n_pages, hkv, ps, hd, dtype=dt)
    return dict(kind="append", q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], k_pages=pages[0],
                v_pages=pages[1], table=table, rows=_int(row), positions=_int(local + skip * ps), freqs=inv,
                inter=c["inter"], mscale=1.1 if c["far"] else 1.0, status=torch.zeros(4, device=DEV, dtype=torch.int32))


def _prepare_attend(c, g):
    """One new query per sequence, its pages scattered over the pool; what lies behind a sequence's end is left over."""
    ps, dt = c["page"], TYPES[c["dtype"]]
    lens = torch.tensor(_lens(c), device=DEV)[_perm(g, c["rows"])]
    width = -(-c["longest"] // ps) + 1
    need = (lens + ps - 1) // ps
    total = sum(-(-n // ps) for n in _lens(c))
    at = torch.cumsum(need, 0) - need
    i = torch.arange(width, device=DEV)
    ids = _perm(g, total + 3)
    table = torch.where(i[None] < need[:, None], ids[(at[:, None] + i[None]).clamp_max(total - 1)], -1)
    k = _randn(g, total + 3, c["hkv"], ps, c["hd"], dtype=dt, scale=0.9)
    v = _randn(g, total + 3, c["hkv"], ps, c["hd"], dtype=dt, scale=0.9)
    q = _randn(g, c["rows"], c["hq"], c["hd"], scale=1.5).to(TYPES[c["qtype"]])
    return dict(kind="attend", q=q, k_pages=k, v_pages=v, table=_int(table), lens=_int(lens), window=c["window"],
                cap=c["cap"], scale=1.0 / math.sqrt(c["hd"]), status=torch.zeros(4, device=DEV, dtype=torch.int32))


def _prepare_fork(c, g):
    """Groups of beams that share their prompt's pages and have a last page of their own each."""
    n, k, ps = c["groups"], c["beams"], c["page"]
    lens = torch.tensor(_group_lens(c), device=DEV)[_perm(g, n)]
    full = lens // ps
    width = max(-(-(m + c["reserve"]) // ps) for m in _group_lens(c)) + 1
    shared = sum(m // ps for m in _group_lens(c))
    grown = -(-c["reserve"] // ps) + 1
    n_pages = shared + n * k * (2 + grown) + 5
    ids = _perm(g, n_pages)
    at = torch.cumsum(full, 0) - full
    i = torch.arange(width, device=DEV)
    r = torch.arange(n * k, device=DEV)
    gr = r // k
    table = torch.where(i[None] < full[gr][:, None], ids[(at[gr][:, None] + i[None]).clamp_max(n_pages - 1)], -1)
    table[r, full[gr]] = ids[shared + r]
    refs = torch.zeros(n_pages, device=DEV, dtype=torch.int64)
    refs.index_add_(0, table[table >= 0], torch.ones_like(table[table >= 0]))
    # every group keeps `kept` of its beams; the other rows repeat one of those
    order = torch.rand(n, k, generator=g, device=DEV).argsort(1)
    pick = torch.arange(k, device=DEV)[None].expand(n, k)
    extra = torch.randint(0, c["kept"], (n, k), generator=g, device=DEV)
    parent = order.gather(1, torch.where(pick < c["kept"], pick, extra)) + torch.arange(n, device=DEV)[:, None] * k
    pages = _randn(g, 2, c["layers"], n_pages, c["hkv"], ps, c["hd"], dtype=TYPES[c["dtype"]])
    return dict(kind="fork", k=pages[0], v=pages[1], table=_int(table), lens=_int(lens[gr]), refs=_int(refs),
                parents=_int(parent.reshape(-1)), reserve=torch.full((n * k,), c["reserve"], device=DEV, dtype=torch.int32),
                status=torch.zeros(4, device=DEV, dtype=torch.int32))


def _prepare_compact(c, g):
    """A pool whose used pages lie scattered after sequences were freed; a table of eight rows holds them."""
    used, moved = _moved(c)
    low, high = _perm(g, used)[: used - moved], used + _perm(g, c["pages"] - used)[:moved]
    ids = torch.cat((low, high))[_perm(g, used)]
    width = -(-used // 8)
    table = torch.full((8 * width,), -1, device=DEV, dtype=torch.int64)
    table[:used] = ids
    refs = torch.zeros(c["pages"], device=DEV, dtype=torch.int32)
    refs[ids] = 1
    pages = _randn(g, 2, c["layers"], c["pages"], c["hkv"], c["page"], c["hd"], dtype=TYPES[c["dtype"]])
    table = _int(table.view(8, width))
    return dict(kind="compact", k=pages[0], v=pages[1], table0=table, refs0=refs, table=table.clone(), refs=refs.clone(),
                status=torch.zeros(4, device=DEV, dtype=torch.int32))


def _prepare_select(c, g):
    """The logits of every beam, the beams' sums of log probabilities so far and which of them have ended."""
    rows = c["groups"] * c["beams"]
    logits = _randn(g, rows, c["vocab"], scale=2.0)
    logits += 6.0 * (torch.rand(rows, c["vocab"], generator=g, device=DEV) > 0.999)   # a few likely tokens
    scores = -20.0 * torch.rand(c["groups"], c["beams"], generator=g, device=DEV)
    done = _int(torch.rand(c["groups"], c["beams"], generator=g, device=DEV) < c["done"])
    return dict(kind="select", logits=logits.to(TYPES[c["dtype"]]), scores=scores, done=done, eos=2,
                status=torch.zeros(4, device=DEV, dtype=torch.int32))


# -------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        from persistent_sm_decode_megakernel_gb300 import paged
        if s["kind"] == "append":
            q = paged.rope_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["positions"],
                                  rows=s["rows"], freqs=s["freqs"], interleaved=s["inter"], mscale=s["mscale"],
                                  status=s["status"])
            return q, s["k_pages"], s["v_pages"]
        if s["kind"] == "attend":
            return paged.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], scale=s["scale"],
                                         window=s["window"], softcap=s["cap"], return_lse=True, status=s["status"])
        if s["kind"] == "fork":
            paged.update_pages(s["k"], s["v"], s["table"], s["lens"], s["refs"], parents=s["parents"],
                               reserve=s["reserve"], status=s["status"])
            return s["table"], s["lens"], s["refs"], s["k"], s["v"]
        if s["kind"] == "compact":
            s["table"].copy_(s["table0"])
            s["refs"].copy_(s["refs0"])
            paged.compact_pages(s["k"], s["v"], s["table"], s["refs"], status=s["status"])
            return s["table"], s["refs"], s["k"], s["v"]
        return paged.beam_select(s["logits"], s["scores"], s["done"], eos=s["eos"], status=s["status"])
    return {"append": _append, "attend": _attend, "fork": _fork, "compact": _compact, "select": _select}[s["kind"]](s)


def _append(s):
    """Angles in 64 bits (far positions), the rotation in 32, one rounding at the end."""
    pos, ps = s["positions"].long(), s["k_pages"].shape[2]
    angle = pos.double()[:, None] * s["freqs"]
    cos, sin = (s["mscale"] * angle.cos()).float()[:, None], (s["mscale"] * angle.sin()).float()[:, None]
    half = s["freqs"].numel()

    def turned(x):
        y = x.float()
        part = y[..., : 2 * half]
        a, b = (part[..., 0::2], part[..., 1::2]) if s["inter"] else (part[..., :half], part[..., half:])
        a, b = a * cos - b * sin, b * cos + a * sin
        part = torch.stack((a, b), -1).flatten(-2) if s["inter"] else torch.cat((a, b), -1)
        return torch.cat((part, y[..., 2 * half:]), -1).to(x.dtype)

    page = s["table"][s["rows"].long(), pos // ps].long()
    s["k_pages"][page, :, pos % ps] = turned(s["k"])
    s["v_pages"][page, :, pos % ps] = s["v"]
    return turned(s["q"]), s["k_pages"], s["v_pages"]


def _attend(s):
    q, ps = s["q"].float(), s["k_pages"].shape[2]
    r, hq, hd = q.shape
    hkv = s["k_pages"].shape[1]
    at = s["table"].long().clamp_min(0)
    k = s["k_pages"][at].float().transpose(1, 2).reshape(r, hkv, -1, hd)      # [rows, kv heads, positions, head_dim]
    v = s["v_pages"][at].float().transpose(1, 2).reshape(r, hkv, -1, hd)
    score = torch.matmul(q.view(r, hkv, hq // hkv, hd), k.transpose(2, 3)) * s["scale"]
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    t, n = torch.arange(k.shape[2], device=q.device), s["lens"].long()[:, None]
    seen = t < n
    if s["window"]:
        seen = seen & (t >= n - s["window"])
    seen = seen[:, None, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, torch.where(seen.transpose(2, 3), v, 0.0)) / torch.where(z == 0, 1.0, z)
    return out.view(r, hq, hd).to(s["q"].dtype), (top + torch.log(z)).view(r, hq)


def _count(ids, n):
    ids = ids[ids >= 0].long()
    return torch.zeros(n, device=ids.device, dtype=torch.int32).index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))


def _fork(s):
    """Every row takes its parent's pages; one that will be written becomes private; new pages are the lowest free ones."""
    table, lens, refs, ps = s["table"], s["lens"], s["refs"], s["k"].shape[3]
    n, i = refs.numel(), torch.arange(table.shape[1], device=table.device)[None]
    live = s["parents"] >= 0
    par = s["parents"].long().clamp_min(0)
    length = torch.where(live, lens[par], 0)
    room = torch.where(live, s["reserve"], 0)
    held = (length + ps - 1) // ps
    new = torch.where(i < held[:, None], table[par], -1)
    refs += _count(new, n) - _count(table, n)
    # of the rows that will write into one page, each but the page's last holder copies it
    last = new.gather(1, (held - 1).clamp_min(0).long()[:, None])[:, 0]
    writes = (length % ps > 0) & (room > 0)
    row = torch.arange(last.numel(), device=table.device)
    before = ((last[None] == last[:, None]) & writes[None] & (row[None] < row[:, None])).sum(1)
    copies = writes & (before < refs[last.clamp_min(0).long()] - 1)
    ends = torch.where(room > 0, (length + room + ps - 1) // ps, held)
    need = copies + ends - held
    at = torch.cumsum(need, 0) - need
    free = torch.nonzero(refs == 0)[:, 0]
    src, dst = last[copies].long(), free[at[copies]]
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    new = torch.where((i >= held[:, None]) & (i < ends[:, None]),
                      free[(at + copies - held)[:, None].add(i).clamp(0, free.numel() - 1)].int(), new)
    refs -= _count(src, n)
    new[row[copies], held[copies].long() - 1] = dst.int()
    refs[free[: int(need.sum())]] = 1
    table.copy_(new)
    lens.copy_(length)
    return table, lens, refs, s["k"], s["v"]


def _compact(s):
    """The used pages behind the first `used` places move, in order, to the lowest free places."""
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    table, refs = s["table"], s["refs"]
    held = refs > 0
    used = int(held.sum())
    src = used + torch.nonzero(held[used:])[:, 0]
    dst = torch.nonzero(~held[:used])[:, 0]
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    to = torch.arange(refs.numel(), device=refs.device, dtype=torch.int32)
    to[src] = dst.int()
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()], table))
    refs[dst] = refs[src]
    refs[src] = 0
    return table, refs, s["k"], s["v"]


def _select(s):
    """A beam's candidates by logit, ties to the lowest token; across beams by the 64-bit sums, ties to the lower beam."""
    groups, beams = s["scores"].shape
    top, token = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    top, token = top[:, :beams].double(), token[:, :beams]
    x = s["logits"].double()
    peak = x.amax(-1, keepdim=True)
    lse = peak + torch.exp(x - peak).sum(-1, keepdim=True).log()
    score, done = s["scores"].double().view(-1, 1), s["done"].view(-1, 1) != 0
    first = torch.arange(beams, device=top.device)[None] == 0
    key = torch.where(done, torch.where(first, score, -math.inf), (score + (top - lse)).clamp_min(-1.7e308))
    token = torch.where(done, s["eos"], token)
    best, at = torch.sort(key.view(groups, -1), dim=-1, descending=True, stable=True)
    best, at = best[:, :beams], at[:, :beams]
    row = torch.arange(groups, device=at.device)[:, None] * beams + at // beams
    token = token.view(groups, -1).gather(1, at)
    ended = (s["done"].view(-1)[row] != 0) | (token == s["eos"])
    return token.int(), row.int(), best.float(), ended.int()


# ---------------------------------------------------------------------------- in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "append":
        turn = torch.polar(torch.full((1,), s["mscale"], device=DEV, dtype=torch.float64),
                           s["positions"].double()[:, None] * s["freqs"])[:, None]
        n = s["freqs"].numel()

        def rotate(x):
            y = x.double().clone()
            a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if c["inter"] else (slice(0, n), slice(n, 2 * n))
            z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
            y[..., a], y[..., b] = z.real, z.imag
            return y

        k, v, ps = s["k_pages"].double(), s["v_pages"].double(), c["page"]
        slot = s["table"].long()[s["rows"].long(), torch.div(s["positions"].long(), ps, rounding_mode="floor")]
        k[slot, :, s["positions"].long() % ps] = rotate(s["k"])
        v[slot, :, s["positions"].long() % ps] = s["v"].double()
        return rotate(s["q"]), k, v
    if c["kind"] == "attend":
        out, lse, group = [], [], c["hq"] // c["hkv"]
        for r, n in enumerate(s["lens"].tolist()):
            lo = max(0, n - c["window"]) if c["window"] else 0
            ids = s["table"][r, : -(-n // c["page"])].long()
            k = s["k_pages"][ids].double().permute(1, 0, 2, 3).reshape(c["hkv"], -1, c["hd"])[:, lo:n]
            v = s["v_pages"][ids].double().permute(1, 0, 2, 3).reshape(c["hkv"], -1, c["hd"])[:, lo:n]
            z = torch.einsum("jgd,jtd->jgt", s["q"][r].double().view(c["hkv"], group, c["hd"]), k) * s["scale"]
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            lse.append(torch.logsumexp(z, -1).reshape(-1))
            out.append(torch.einsum("jgt,jtd->jgd", torch.softmax(z, -1), v).reshape(c["hq"], c["hd"]))
        return torch.stack(out), torch.stack(lse)
    if c["kind"] == "select":
        got = []
        logp = torch.log_softmax(s["logits"].double(), -1).view(c["groups"], c["beams"], -1)
        for g in range(c["groups"]):
            fresh = s["done"][g] == 0
            every = torch.cat(((s["scores"][g].double()[fresh][:, None] + logp[g][fresh]).reshape(-1),
                               s["scores"][g].double()[~fresh]))
            got.append(torch.topk(every, c["beams"]).values)
        return None, None, torch.stack(got), None
    return None  # pages are moved, nothing is computed
