"""The paged decoder's steps over trees of drafted tokens (mk_decode_step_tree, PagedDecoder.step_tree, verify and
generate) against the fp64 oracle and the same decoder's single steps."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from helpers import assert_parity, oracle_run
from test_gpu_paged_decoder import _paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from persistent_sm_decode_megakernel_gb300 import model
    return model


@pytest.mark.parametrize("name,B,nodes,max_batch", [("tiny", 1, 1, 1), ("tiny", 1, 9, 9), ("tiny", 2, 5, 16), ("tiny-g4", 1, 16, 16),
                                                    ("tiny-g4", 3, 4, 16)])
def test_a_chain_of_drafts_matches_the_oracle(lib, name, B, nodes, max_batch):
    """The forced tokens of several steps as one chain per row: every node's logits are the oracle's of its step."""
    cfg = synth.CONFIGS[name]
    w = synth.gen_weights(cfg)
    P = 37
    prompt = synth.gen_prompts(cfg, B, P)
    toks, zref = oracle_run(cfg, w, prompt, nodes + 1)
    dec = _paged(lib, cfg, w, max_batch, B + 1, P + nodes + 1)
    rows = [(b + 1) % (B + 1) for b in range(B)]
    z0 = {r: torch.zeros(cfg.vocab, device=dec.dm.device) for r in rows}
    first = dec.prefill({r: prompt[b] for b, r in enumerate(rows)}, z0)
    dec.update(reserve=[nodes if r in rows else 0 for r in range(B + 1)])
    z = torch.zeros((B, nodes, cfg.vocab), device=dec.dm.device)
    at = dec._int32(rows)
    out = dec.step_tree(dec._int32(toks[:, P:P + nodes]), dec._int32([[i - 1 for i in range(nodes)]] * B), dec.lens[at.long()], at, z)
    dec.synchronize()
    got = torch.cat((torch.stack([z0[r] for r in rows])[:, None], z), 1).cpu().numpy()
    tokens = torch.cat((torch.stack([first[r] for r in rows]), out), 1).cpu().numpy()
    dec.close()
    assert assert_parity(got, tokens, zref, toks, P) < 5e-3


def test_branches_see_their_own_ancestors_only(lib):
    """A tree of two branches gives each what a chain of its own gives, and the accepted branch's cache what single steps
    leave: the next steps' logits agree."""
    cfg = synth.CONFIGS["tiny-g4"]
    w = synth.gen_weights(cfg)
    P = 50
    prompt = synth.gen_prompts(cfg, 1, P)[0]
    V = cfg.vocab
    a, b = _paged(lib, cfg, w, 16, 1, P + 20), _paged(lib, cfg, w, 16, 1, P + 20)
    first = int(a.prefill({0: prompt})[0])
    b.prefill({0: prompt})
    dev = a.dm.device

    def single(tokens):
        zs = []
        for t in tokens:
            b.update(reserve=[1])
            z = torch.zeros((1, V), device=dev)
            nxt = b.step(b._int32([t]), b.lens, None, z)
            b.lens += 1
            zs.append(z[0])
        return zs, int(nxt)

    want, second = single([first])
    x, y = (second + 1) % V, (second + 2) % V            # drafts the model does not choose
    third_want, third = single([second])
    fourth_want, fourth = single([third])
    # node 0 the pending token; a wrong branch 1 -> 2; the right branch 3 -> 4 laid between wrong ones
    tokens = [first, x, y, second, y, third, x]
    parents = [-1, 0, 1, 0, 3, 3, 5]
    n = len(tokens)
    z = torch.zeros((1, n, V), device=dev)
    got, path, count = a.verify([tokens], [parents], [0], z)
    a.synchronize()
    assert path[0, : int(count)].tolist() == [0, 3, 5] and got[0, :3].tolist() == [second, third, fourth]
    assert a.lens.tolist() == [P + 3] and b.lens.tolist() == [P + 3]
    scale = want[0].abs().max().item()
    for node, ref in ((0, want[0]), (3, third_want[0]), (5, fourth_want[0])):
        assert (z[0, node] - ref).abs().max().item() <= 1e-3 * scale, node
    # the wrong branch is what a chain of its own would be
    c = _paged(lib, cfg, w, 16, 1, P + 20)
    c.prefill({0: prompt})
    zc = torch.zeros((1, 3, V), device=dev)
    c.update(reserve=[3])
    c.step_tree(c._int32([[first, x, y]]), c._int32([[-1, 0, 1]]), c.lens, None, zc)
    c.synchronize()
    assert (zc[0, 1] - z[0, 1]).abs().max().item() <= 1e-3 * scale and (zc[0, 2] - z[0, 2]).abs().max().item() <= 1e-3 * scale
    # the cache that the acceptance left
    a.update(reserve=[1])
    za = torch.zeros((1, V), device=dev)
    a.step(a._int32([fourth]), a.lens, None, za)
    a.lens += 1
    a.synchronize()
    zb = single([fourth])[0][0]
    assert (za[0] - zb).abs().max().item() <= 1e-3 * scale
    for d in (a, b, c):
        d.close()


@pytest.mark.parametrize("guess", ["none", "right", "wrong", "mixed", "too many"])
def test_generate_gives_what_single_steps_give(lib, guess):
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    P, n_new = 20, 24
    prompt = synth.gen_prompts(cfg, 1, P)
    toks, _ = oracle_run(cfg, w, prompt, n_new)
    dec = _paged(lib, cfg, w, 8, 2, P + n_new)
    plain, steps = dec.generate(prompt[0], n_new, lambda t: ([], []))
    assert steps == n_new - 1 and len(plain) == n_new
    rng = np.random.default_rng(5)
    every = list(prompt[0]) + plain

    def draft(t):
        ahead = [int(x) for x in every[len(t): len(t) + 3]]
        wrong = [int(x) for x in rng.integers(0, cfg.vocab, 3)]
        if guess == "none":
            return [], []
        if guess == "right":
            return ahead, list(range(-1, len(ahead) - 1))
        if guess == "wrong":
            return wrong, [-1, 0, 0]
        if guess == "too many":
            return (ahead + wrong * 9)[:30], ([i - 1 for i in range(len(ahead))] + [-1] * 30)[: min(30, len(ahead) + 27)]
        return wrong[:2] + ahead, [-1, 0] + [-1] + [i + 2 for i in range(len(ahead) - 1)] if ahead else [-1, 0]

    got, fewer = dec.generate(prompt[0], n_new, draft)
    # (a tree's scores are summed in another order than a single token's: a near tie of two logits may fall either way,
    # which the tiny model's margins do not have)
    assert got == plain
    assert fewer <= (steps if guess in ("none", "wrong") else -(-(n_new - 1) // 4) + 1)
    assert dec.refs.sum().item() == 0 and dec.lens.tolist() == [0, 0]
    stop = plain[10]
    ended, _ = dec.generate(prompt[0], n_new, draft, eos=stop)
    assert ended == plain[: plain.index(stop) + 1]
    dec.close()


def test_tree_steps_refuse_what_does_not_fit(lib):
    from persistent_sm_decode_megakernel_gb300 import (MK_ERR_INVALID, MK_ERR_PAGES, MK_ERR_STATE, MkError, mk_decode_step_tree)
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    dec = _paged(lib, cfg, w, 4, 2, 48)
    one = dec._int32([[0, 1]])
    lens = dec._int32([0])
    for bad in (dict(tokens=one.long()), dict(tokens=one[:, :1]), dict(parents=one[0]), dict(lens=lens.long()), dict(lens=dec._int32([0, 0])),
                dict(rows=one), dict(logits=torch.zeros(1, 2, cfg.vocab - 1, device=dec.dm.device)), dict(tokens=one.cpu())):
        with pytest.raises(ValueError):
            dec.step_tree(**{**dict(tokens=one, parents=one, lens=lens), **bad})
    five = dec._int32([[0] * 5])
    with pytest.raises(MkError) as e:
        dec.step_tree(five, five, lens)
    assert e.value.status == MK_ERR_INVALID
    p = ctypes.c_void_p(one.data_ptr())
    for args in ((None, p, p, None, 1, 1), (p, None, p, None, 1, 1), (p, p, None, None, 1, 1), (p, p, p, None, 0, 1), (p, p, p, None, 1, 0),
                 (p, p, p, None, 2 ** 16, 2 ** 16)):
        assert mk_decode_step_tree(dec.h, *args, None, None) == MK_ERR_INVALID
    assert mk_decode_step_tree(None, p, p, p, None, 1, 1, None, None) == MK_ERR_INVALID
    for rows in ([0, 0], [2], [-1]):
        with pytest.raises(ValueError):
            dec.verify([[0, 1]] * len(rows), [[-1, 0]] * len(rows), rows)
    for t in ([[0] * 5], [[0], [0]], [0]):
        with pytest.raises(ValueError):
            dec.verify(t, t, [0])
    graph = torch.cuda.CUDAGraph()
    dec.synchronize()
    torch.cuda.synchronize()
    side = _paged(lib, cfg, w, 4, 1, 40, stream=torch.cuda.Stream())
    with torch.cuda.graph(graph, stream=side.stream):
        keep = torch.zeros(1, device=dec.dm.device)
        with pytest.raises(MkError) as e:
            side.step_tree(one, one, lens)
        assert e.value.status == MK_ERR_STATE
    assert keep.numel() == 1
    # drafts past the row's pages: nothing is taken over, the error is reported, the decoder goes on
    prompt = list(range(46))             # three pages of 16 hold 48 positions
    dec.prefill({0: prompt})
    with pytest.raises(MkError) as e:
        dec.verify([[1, 2, 3, 4]], [[-1, 0, 1, 2]], [0])
        dec.synchronize()
    assert e.value.status == MK_ERR_PAGES
    dec.reset()
    for bad in (dict(n_new=0), dict(n_new=48), dict(prompt=[cfg.vocab]), dict(prompt=[])):
        with pytest.raises(ValueError):
            dec.generate(**{**dict(prompt=[1, 2], n_new=3, draft=lambda t: ([], [])), **bad})
    for bad in (([1], []), ([1, 2], [-1, 1]), ([1], [-2]), ([cfg.vocab], [-1])):
        with pytest.raises(ValueError):
            dec.generate([1, 2], 3, lambda t, bad=bad: bad)
    tokens, _ = dec.generate([1, 2], 3, lambda t: ([], []))
    assert len(tokens) == 3
    dec.close()
    side.close()


def test_verify_leaves_other_rows_what_they_reserved(lib):
    """A row that reserved ahead steps on after another row's verify, and its pages stay counted."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    dec = _paged(lib, cfg, w, 8, 3, 96)
    a, b = (synth.gen_prompts(cfg, 1, 14)[0], synth.gen_prompts(cfg, 1, 10)[0])
    first = dec.prefill({0: a, 1: b})
    dec.update(reserve=[0, 40, 0])
    held = (dec.table[1] >= 0).sum().item()
    assert held == 4
    dec.verify([[int(first[0]), 5, 6]], [[-1, 0, 0]], [0])
    dec.synchronize()
    assert (dec.table[1] >= 0).sum().item() == held and (dec.table[2] >= 0).sum().item() == 0
    assert dec.refs.sum().item() == (dec.table >= 0).sum().item()
    tok = first[1]
    for i in range(30):
        tok = dec.step(tok.contiguous(), dec.lens[1:2].contiguous(), dec._int32([1]))
        dec.lens[1] += 1
    dec.synchronize()
    dec.close()


def test_verify_without_pages_takes_nothing_over(lib):
    """A row whose last page is shared, and no free page for its copy: the shared page, both rows and what is returned say so."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    dec = _paged(lib, cfg, w, 8, 2, 16, n_pages=1)
    first = dec.prefill({0: synth.gen_prompts(cfg, 1, 9)[0]})
    dec.update(parents=[0, 0])
    dec.synchronize()
    keep = [x.clone() for x in (dec.k, dec.v, dec.table, dec.lens, dec.refs)]
    got, path, count = dec.verify([[int(first[0]), 3]], [[-1, 0]], [1])
    with pytest.raises(MkError) as e:
        dec.synchronize()
    assert e.value.status == MK_ERR_PAGES
    assert count.tolist() == [0] and got.tolist() == [[-1, -1]] and path.tolist() == [[-1, -1]]
    assert all(torch.equal(x, y) for x, y in zip(keep, (dec.k, dec.v, dec.table, dec.lens, dec.refs)))
    # an error that nobody has read yet (a refused update, which changes nothing): nothing either, then all is as ever
    dec.update(parents=[0, -1])
    dec.update(reserve=[16, 0])
    got, path, count = dec.verify([[int(first[0]), 3]], [[-1, 0]], [0])
    assert count.tolist() == [0] and dec.lens.tolist() == [9, 0]
    with pytest.raises(MkError):
        dec.synchronize()
    got, path, count = dec.verify([[int(first[0]), 3]], [[-1, 0]], [0])
    dec.synchronize()
    assert count.item() >= 1 and dec.lens.tolist() == [9 + count.item(), 0]
    dec.close()


def test_verify_of_tokens_that_are_none_takes_nothing_over(lib):
    from persistent_sm_decode_megakernel_gb300 import MkError
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    dec = _paged(lib, cfg, w, 8, 2, 64)
    first = int(dec.prefill({0: synth.gen_prompts(cfg, 1, 9)[0]})[0])
    for bad in (-1, cfg.vocab, -2 ** 31):
        with pytest.raises(ValueError):
            dec.verify([[first, bad]], [[-1, 0]], [0])
        keep = [x.clone() for x in (dec.lens, dec.k[:, :, :, :9], dec.v[:, :, :, :9])]
        got, path, count = dec.verify(dec._int32([[first, bad]]), dec._int32([[-1, 0]]), [0])
        with pytest.raises(MkError):
            dec.synchronize()
        dec.reset()
        dec.synchronize()
        assert count.tolist() == [0] and path.tolist() == [[-1, -1]]
        assert all(torch.equal(x, y) for x, y in zip(keep, (dec.lens, dec.k[:, :, :, :9], dec.v[:, :, :, :9])))
    with pytest.raises(ValueError):
        dec.verify(torch.tensor([[first, cfg.vocab]]), [[-1, 0]], [0])
    _, _, count = dec.verify([[first, 1]], [[-1, 0]], [0])
    dec.synchronize()
    assert count.item() >= 1
    dec.close()


def test_drafts_of_two_lengths_are_refused_however_long(lib):
    cfg = synth.CONFIGS["tiny"]
    dec = _paged(lib, cfg, synth.gen_weights(cfg), 4, 1, 48)
    for bad in (([1] * 9, [-1] * 8), ([1] * 8, [-1] * 7 + [8]), ([1] * 7 + [cfg.vocab], [-1] * 8)):
        with pytest.raises(ValueError):
            dec.generate([1, 2], 3, lambda t, bad=bad: bad)
    dec.close()
