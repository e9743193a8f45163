"""The decoder over a paged cache (PagedDecoder: mk_create_paged, mk_decode_step_paged) against the
fp64 oracle and the contiguous decoder, its forks, and its beam search."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import LOGIT_RTOL, assert_parity, oracle_run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from persistent_sm_decode_megakernel_gb300 import model
    return model


def _paged(lib, cfg, w, max_batch, n_rows, positions, page_size=16, n_pages=None, **kw):
    dm = lib.DeviceModel(cfg, w, max_batch=max_batch, max_ctx=1)
    n_pages = n_pages or n_rows * (-(-positions // page_size)) + 2
    return lib.PagedDecoder(dm, n_rows=n_rows, n_pages=n_pages, max_positions=positions, page_size=page_size, **kw)


def _forced(dec, prompt, toks, n_new, rows):
    """Prefill, then steps fed the given tokens: logits [B, n_new, V] and tokens [B, n_new]."""
    B, P = prompt.shape
    V = dec.dm.cfg.vocab
    z0 = {r: torch.zeros(V, device=dec.dm.device) for r in rows}
    first = dec.prefill({r: prompt[b] for b, r in enumerate(rows)}, z0)
    out, z = [torch.cat([first[r] for r in rows])], [torch.stack([z0[r] for r in rows])]
    row = dec._int32(rows)
    for t in range(P, P + n_new - 1):
        reserve = [0] * len(dec.lens)
        for r in rows:
            reserve[r] = 1
        dec.update(reserve=reserve)
        lg = torch.zeros((B, V), device=dec.dm.device)
        out.append(dec.step(dec._int32(toks[:, t]), dec.lens[row.long()], row, lg))
        dec.lens[row.long()] += 1
        z.append(lg)
    dec.synchronize()
    return torch.stack(z, 1).cpu().numpy(), torch.stack(out, 1).cpu().numpy()


@pytest.mark.parametrize("name,B,max_batch", [("tiny", 1, 1), ("tiny", 2, 2), ("tiny", 3, 4), ("tiny", 11, 16), ("tiny-g4", 2, 2),
                                              ("tiny-g4", 5, 8)])
def test_paged_decoder_matches_the_oracle(lib, name, B, max_batch):
    """Prompts in chunks of up to max_batch rows, then forced steps, rows in an order of their own."""
    cfg = synth.CONFIGS[name]
    w = synth.gen_weights(cfg)
    P, n_new = 37, 9
    prompt = synth.gen_prompts(cfg, B, P)
    toks, zref = oracle_run(cfg, w, prompt, n_new)
    dec = _paged(lib, cfg, w, max_batch, B + 1, P + n_new)
    z, tg = _forced(dec, prompt, toks, n_new, [(b + 1) % (B + 1) for b in range(B)])
    dec.close()
    assert assert_parity(z, tg, zref, toks, P) < 5e-3


def test_paged_decoder_next_to_the_contiguous_one(lib):
    """The same prompt and tokens through both: logits apart by the key's second rounding only."""
    cfg = synth.CONFIGS["tiny-g4"]
    w = synth.gen_weights(cfg)
    P = 300
    prompt = synth.gen_prompts(cfg, 1, P)
    a = lib.DeviceModel(cfg, w, max_batch=4, max_ctx=P + 1)
    dec = lib.Decoder(a)
    za = torch.zeros((1, cfg.vocab), device=a.device)
    ta = dec.prefill(prompt, logits=za)
    b = _paged(lib, cfg, w, 4, 1, P + 1, page_size=48)
    zb = {0: torch.zeros(cfg.vocab, device=a.device)}
    tb = b.prefill({0: prompt[0]}, zb)
    b.synchronize()
    scale = za.abs().max().item()
    assert (za[0] - zb[0]).abs().max().item() <= 5e-3 * scale
    top = za[0].topk(2).values
    if (top[0] - top[1]).item() > 1e-2 * scale:
        assert int(ta[0]) == int(tb[0])
    dec.close()
    b.close()


@pytest.mark.parametrize("name,max_batch", [("tiny", 1), ("tiny-g4", 2), ("tiny-g4", 16)])
def test_keys_are_rounded_once(lib, name, max_batch):
    """The first layer's keys in the pages are the contiguous decoder's: both come from the same products, rotated in
    32 bits and rounded once, so that only a key within 2^-20 of a rounding border (2^-8 of them over 16-bit
    types of up to 11 bits, doubled for products summed in another order) may differ, and then by one step.  Of
    keys rounded before their rotation as well, a third differs."""
    cfg = synth.CONFIGS[name]
    w = synth.gen_weights(cfg)
    P = 200
    prompt = synth.gen_prompts(cfg, 1, P)
    a = lib.DeviceModel(cfg, w, max_batch=max_batch, max_ctx=P)
    plain = lib.Decoder(a)
    plain.prefill(prompt)
    dec = _paged(lib, cfg, w, max_batch, 1, P)
    dec.prefill({0: prompt[0]})
    dec.synchronize()
    at = dec.table[0].long()
    for got, want, share in ((dec.k, a.k_cache, 2.0 ** -6), (dec.v, a.v_cache, 2.0 ** -6)):
        got = got[0][at].transpose(0, 1).reshape(cfg.n_kv_heads, -1, cfg.head_dim)[:, :P].float()
        want = want[0][0].view(dec.k.dtype).float()
        step = torch.finfo(dec.k.dtype).eps * want.abs()
        assert torch.all((got - want).abs() <= step + 2.0 ** -14)
        assert (got != want).float().mean().item() <= share
    dec.close()
    plain.close()


@pytest.mark.parametrize("factor", [2.0, 8.0])
def test_paged_decoder_scaled_rotary_base(lib, factor):
    """Rotary positions with the scaled base are those of a model whose theta is the scaled one."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    other = synth.with_overrides(cfg, rope_theta=cfg.rope_theta * factor ** (cfg.head_dim / (cfg.head_dim - 2)))
    prompt = synth.gen_prompts(cfg, 1, 60)
    toks, zref = oracle_run(other, w, prompt, 3)
    dec = _paged(lib, cfg, w, 4, 1, 64, rope=dict(kind="base", factor=factor))
    z, tg = _forced(dec, prompt, toks, 3, [0])
    dec.close()
    assert_parity(z, tg, zref, toks, 60)


def test_forked_rows_go_their_own_ways(lib):
    """A row forked in the middle of a page: parent and child get different tokens and match the oracle's two
    sequences, while the pages of their common prompt stay shared."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    P, n = 40, 12
    prompt = synth.gen_prompts(cfg, 1, P)
    tails = synth.gen_prompts(cfg, 2, n)
    m = oracle.Model(cfg, w)
    cache = oracle.KVCache(cfg, 2, P + n)
    oracle.prefill(m, np.repeat(prompt, 2, 0), cache)
    want = [oracle.decode_step(m, cache, tails[:, t], [P + t] * 2) for t in range(n)]
    dec = _paged(lib, cfg, w, 4, 3, P + n)
    dec.prefill({1: prompt[0]})
    dec.update(parents=[1, 1, -1], reserve=[n, n, 0])
    assert torch.equal(dec.table[0, :2], dec.table[1, :2]) and dec.table[0, 2] != dec.table[1, 2]
    assert int((dec.refs == 2).sum()) == 2
    for t in range(n):
        lg = torch.zeros((2, cfg.vocab), device=dec.dm.device)
        dec.step(dec._int32(tails[:, t]), dec.lens[:2].contiguous(), None, lg)
        dec.lens[:2] += 1
        z = lg.cpu().numpy()
        for b in range(2):
            assert np.abs(z[b] - want[t][b]).max() <= LOGIT_RTOL * np.abs(want[t][b]).max(), (t, b)
    dec.synchronize()
    dec.update(parents=[-1, -1, -1])
    assert int(dec.refs.sum()) == 0
    dec.close()


def test_beam_search_of_one_beam_is_greedy(lib):
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 21)
    dec = _paged(lib, cfg, w, 4, 4, 64)
    seqs, scores = dec.beam_search(prompt[0], 1, 10)
    tok = dec.prefill({2: prompt[0]})[2]
    greedy = [int(tok)]
    for _ in range(9):
        dec.update(reserve=[0, 0, 1, 0])
        tok = dec.step(tok, dec.lens[2:3].contiguous(), dec._int32([2]))
        dec.lens[2] += 1
        greedy.append(int(tok))
    dec.synchronize()
    dec.close()
    assert seqs[0].tolist() == greedy and scores[0] < 0


@pytest.mark.parametrize("beams,eos", [(4, -1), (16, -1), (5, 7)])
def test_beam_search_scores_are_the_sequences_log_probabilities(lib, beams, eos):
    """Each returned sequence's score is what the oracle gives that sequence, they come best first, and no
    continuation that the oracle ranks clearly higher under the same pruning is missing: its own search, in
    64 bits, has the same scores."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    P, n = 30, 6
    prompt = synth.gen_prompts(cfg, 1, P)
    dec = _paged(lib, cfg, w, 16, 16, P + n)
    seqs, scores = dec.beam_search(prompt[0], beams, n, eos=eos)
    again = dec.beam_search(prompt[0], beams, n, eos=eos)
    assert int(dec.refs.sum()) == 0
    dec.close()
    assert np.array_equal(seqs, again[0]) and np.array_equal(scores, again[1])   # and rows are reusable
    assert np.all(np.diff(scores) <= 0) and len({tuple(s) for s in seqs}) == beams

    def logp(z):
        z = z - z.max(-1, keepdims=True)
        return z - np.log(np.exp(z).sum(-1, keepdims=True))

    m = oracle.Model(cfg, w)
    cache = oracle.KVCache(cfg, beams, P + n)
    z0 = oracle.prefill(m, np.repeat(prompt, beams, 0), cache)[:, -1]
    # a logit is off by at most LOGIT_RTOL of the largest, its log probability by twice that, per step
    tol = 2 * LOGIT_RTOL * np.abs(z0).max() * n
    got, z, done = np.zeros(beams), logp(z0), np.zeros(beams, bool)
    for i in range(n):
        t = seqs[:, i]
        got += np.where(done, 0.0, z[np.arange(beams), t])
        done |= t == eos
        if i + 1 < n:
            z = logp(oracle.decode_step(m, cache, t, [P + i] * beams))
    assert np.abs(got - scores).max() <= tol
    # the oracle's own beam search: its scores, place by place
    hist = [((), 0.0)]
    for i in range(n):
        grown = []
        cache = oracle.KVCache(cfg, len(hist), P + n)
        z = oracle.prefill(m, np.array([list(prompt[0]) + list(h) for h, _ in hist]), cache)[:, -1]
        for (h, s), lp in zip(hist, logp(z)):
            if eos in h:
                grown.append((s, h + (eos,)))
            else:
                grown += [(s + lp[t], h + (int(t),)) for t in np.argsort(-lp, kind="stable")[:beams]]
        grown.sort(key=lambda g: -g[0])
        hist = [(h, s) for s, h in grown[:beams]]
    assert np.abs(np.array([s for _, s in hist]) - scores).max() <= tol


def test_paged_steps_report_what_is_not_there(lib):
    """A step whose position has no page, and one whose row is none, end in MK_ERR_PAGES; the context goes on."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 16)
    dec = _paged(lib, cfg, w, 4, 2, 64)
    want = int(dec.prefill({0: prompt[0]})[0])
    one = dec._int32([want])
    for pos, row in ((16, 0), (0, 9), (64, 0)):
        dec.step(one, dec._int32([pos]), dec._int32([row]))
        with pytest.raises(MkError) as e:
            dec.synchronize()
        assert e.value.status == MK_ERR_PAGES
    dec.update(parents=[-1, -1])
    assert int(dec.prefill({1: prompt[0]})[1]) == want
    dec.update(reserve=[0, 100])                       # past the table
    with pytest.raises(MkError):
        dec.synchronize()
    dec.synchronize()
    dec.close()


def test_prompts_that_do_not_fit_leave_the_rows_as_they_were(lib):
    """Too long a prompt, an empty one, no such row, too few pages: refused before any step, and the rows go on."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 33)[0]
    dec = _paged(lib, cfg, w, 4, 3, 48, n_pages=4)
    want = int(dec.prefill({0: prompt})[0])            # three of four pages
    before = dec.lens.tolist(), dec.table.tolist(), dec.refs.tolist()
    for bad in ({1: [1] * 49}, {0: [1] * 16}, {1: []}, {3: [1]}, {-1: [1]}):
        with pytest.raises(ValueError):
            dec.prefill(bad)
    with pytest.raises(MkError) as e:
        dec.prefill({1: prompt})
    assert e.value.status == MK_ERR_PAGES
    assert before == (dec.lens.tolist(), dec.table.tolist(), dec.refs.tolist())
    dec.update(parents=[-1, -1, -1])
    assert int(dec.prefill({1: prompt})[1]) == want
    dec.close()


def test_a_refused_search_leaves_no_error_behind(lib):
    """A beam search that runs out of pages raises once: what its steps reported besides (positions without a page)
    does not come up in the next call."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_PAGES, MkError
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 30)[0]
    dec = _paged(lib, cfg, w, 4, 4, 64, n_pages=6)
    want = int(dec.prefill({0: prompt})[0])
    with pytest.raises(MkError) as e:
        dec.beam_search(prompt, 4, 20)             # four beams of 49 positions over six pages
    assert e.value.status == MK_ERR_PAGES
    assert int(dec.refs.sum()) == 0 and not dec.lens.any()
    assert int(dec.prefill({1: prompt})[1]) == want
    dec.synchronize()
    dec.update(reserve=[0, 1000, 0, 0])            # refused, and a step of a row that has no page: both, one error
    one = dec._int32([1])
    dec.step(one, dec._int32([40]), dec._int32([3]))
    with pytest.raises(MkError) as e:
        dec.synchronize()
    assert e.value.status == MK_ERR_PAGES
    dec.synchronize()
    dec.close()


def _busy(stream):
    """Some tens of milliseconds of work on a stream."""
    with torch.cuda.stream(stream):
        x = torch.randn(4096, 4096, device="cuda:0")
        for _ in range(60):
            x = x @ x * 1e-3


def test_tensors_of_another_stream_live_until_they_were_read(lib):
    """Tokens, positions, rows, logits, parents and reservations that the caller drops as soon as step and update
    return, the decoder's stream being busy with something else: what the caller allocates next is other memory."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 20)[0]
    got = []
    for drop in (False, True):
        dec = _paged(lib, cfg, w, 4, 4, 64, stream=torch.cuda.Stream())
        dec.prefill({0: prompt, 2: prompt[:7]})
        dec.synchronize()
        torch.cuda.synchronize()
        held, over = [], []

        def ints(x):
            t = dec._int32(x)
            torch.cuda.current_stream().synchronize()  # ready before the other stream looks at it
            if not drop:
                held.append(t)
            return t

        def others(n):
            for _ in range(8):                         # the next taker of what was dropped
                over.append(torch.full((n,), 1, dtype=torch.int32, device=dec.dm.device))

        _busy(dec.stream)
        dec.update(ints([0, 0, 2, 2]), ints([3, 2, 1, 1]))
        others(4)
        z = torch.zeros(3, cfg.vocab, device=dec.dm.device)
        torch.cuda.current_stream().synchronize()
        out = dec.step(ints([5, 6, 7]), ints([20, 20, 7]), ints([0, 1, 2]), z)
        others(3)
        torch.cuda.synchronize()
        dec.synchronize()
        got.append((dec.table.clone(), dec.refs.clone(), out.clone(), z.clone()))
        dec.close()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    # logits that are dropped do not become the caller's next tensor before they are written
    dec = _paged(lib, cfg, w, 4, 1, 64, stream=torch.cuda.Stream())
    dec.prefill({0: prompt})
    dec.update(reserve=[3])
    dec.synchronize()
    one, pos = dec._int32([5]), dec._int32([20])
    torch.cuda.synchronize()
    _busy(dec.stream)
    dec.step(one, pos, None, torch.empty(1, cfg.vocab, device=dec.dm.device))
    mine = [torch.zeros(1, cfg.vocab, device=dec.dm.device) for _ in range(4)]
    dec.synchronize()
    assert not any(t.any() for t in mine)
    dec.update(parents=[-1])
    dec.prefill({0: prompt}, {0: torch.empty(cfg.vocab, device=dec.dm.device)})
    dec.synchronize()
    dec.close()


def test_contexts_are_made_and_freed_on_their_models_device(lib, monkeypatch):
    """Whatever device is current: the calls that allocate and free run with the model's."""
    import persistent_sm_decode_megakernel_gb300 as pkg
    inside, seen = [], []

    class Device(torch.cuda.device):
        def __enter__(self):
            inside.append(torch.device("cuda", self.idx))
            return super().__enter__()

        def __exit__(self, *a):
            inside.pop()
            return super().__exit__(*a)

    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    create, destroy = pkg.mk_create_paged, lib.mk_destroy
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(pkg, "mk_create_paged", lambda *a: (seen.append(list(inside)), create(*a))[1])
    monkeypatch.setattr(lib, "mk_destroy", lambda *a: (seen.append(list(inside)), destroy(*a))[1])
    dec = _paged(lib, cfg, w, 1, 1, 16)
    dec.close()
    assert len(seen) == 2 and all(s and s[-1] == dec.dm.device for s in seen)


def test_a_prompt_with_a_token_that_is_none_is_refused(lib):
    """A token outside the vocabulary, in any of the prompts, raises before anything is changed."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 20)[0]
    dec = _paged(lib, cfg, w, 4, 2, 48)
    want = int(dec.prefill({0: prompt})[0])
    before = dec.lens.tolist(), dec.table.tolist(), dec.refs.tolist()
    for bad in (-1, cfg.vocab):
        with pytest.raises(ValueError):
            dec.prefill({1: [1, 2, bad]})
        with pytest.raises(ValueError):
            dec.prefill({0: [3], 1: [bad]})
    assert before == (dec.lens.tolist(), dec.table.tolist(), dec.refs.tolist())
    assert int(dec.prefill({1: prompt})[1]) == want
    dec.synchronize()
    dec.close()


def test_a_context_in_error_goes_on_after_reset(lib):
    """A device token outside the vocabulary stops the context until reset(), as it does a contiguous one's; rows and
    pages are the caller's and stay."""
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_STATE, MkError
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 20)[0]
    dec = _paged(lib, cfg, w, 4, 2, 48)
    tok = dec.prefill({0: prompt})[0]
    dec.update(parents=[0, 0], reserve=[2, 2])
    z = torch.zeros(2, cfg.vocab, device=dec.dm.device)
    dec.step(torch.cat((tok, tok)), dec.lens.clone(), None, z)
    dec.synchronize()
    for bad in (-1, cfg.vocab):
        dec.step(dec._int32([bad]), dec._int32([21]))
        with pytest.raises(MkError) as e:
            dec.synchronize()
        assert e.value.status == MK_ERR_STATE
        with pytest.raises(MkError):
            dec.step(tok, dec._int32([20]))
        dec.reset()
        dec.synchronize()
        z2 = torch.zeros_like(z)
        dec.step(torch.cat((tok, tok)), dec.lens.clone(), None, z2)
        dec.synchronize()
        assert torch.equal(z, z2)
    dec.close()


def test_a_beam_search_that_cannot_be_leaves_the_rows(lib):
    """An eos or a token that is none, more beams than tokens: refused before the rows are freed."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 20)[0]
    dec = _paged(lib, cfg, w, 4, 4, 48)
    dec.prefill({0: prompt, 3: prompt[:5]})
    before = dec.lens.tolist(), dec.table.tolist(), dec.refs.tolist()
    for kw in (dict(eos=cfg.vocab), dict(eos=-2)):
        with pytest.raises(ValueError):
            dec.beam_search(prompt, 2, 4, **kw)
    for bad in (-1, cfg.vocab):
        with pytest.raises(ValueError):
            dec.beam_search([1, bad], 2, 4)
    assert before == (dec.lens.tolist(), dec.table.tolist(), dec.refs.tolist())
    dec.synchronize()
    dec.close()


def test_rope_arguments_that_are_none_are_refused(lib):
    """A misspelt word or kind of the rotary positions is not left out in silence."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    for bad in (dict(factr=8.0), dict(kind="base", factor=2.0, orignal=4096.0), dict(kind="bases")):
        with pytest.raises(ValueError):
            _paged(lib, cfg, w, 1, 1, 16, rope=bad)


def test_ended_beams_take_no_more_pages(lib):
    """Beams that ended need no positions: a search whose beams all end at once fits the prompt's own pages, and one
    that ends in between has the scores it has with room to spare."""
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    prompt = synth.gen_prompts(cfg, 1, 16)[0]
    dec = _paged(lib, cfg, w, 4, 4, 64, n_pages=2)
    eos = int(dec.beam_search(prompt, 1, 1)[0][0, 0])
    want = dec.beam_search(prompt, 1, 1, eos=eos)
    seqs, scores = dec.beam_search(prompt, 1, 40, eos=eos)
    assert seqs.tolist() == [[eos] * 40] and scores[0] == want[1][0]
    dec.close()
    few, many = (_paged(lib, cfg, w, 4, 4, 64, n_pages=n) for n in (10, 16))
    first = many.beam_search(prompt, 4, 3)[0]
    for eos in sorted({int(t) for t in first.reshape(-1)})[:4]:
        a, b = many.beam_search(prompt, 4, 20, eos=eos), few.beam_search(prompt, 4, 20, eos=eos)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    few.close()
    many.close()


def test_steps_refuse_tensors_that_do_not_fit_and_capture(lib):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_STATE, mk_decode_step_paged
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    dec = _paged(lib, cfg, w, 2, 2, 32, stream=torch.cuda.Stream())
    want = int(dec.prefill({0: [5, 6, 7]})[0])
    one, two = dec._int32([want]), dec._int32([3, 4])
    wide = torch.zeros(4, dtype=torch.int32, device=one.device)
    z = torch.zeros(2, cfg.vocab + 1, device=one.device)
    for args in ((one.long(), one), (one, one.long()), (one, two), (one, one, two), (one, one, one.cpu()), (wide[::2], two),
                 (two, two, None, z), (two, two, None, z[:, 1:]), (two, two, None, z[:, 1:].half().contiguous())):
        with pytest.raises(ValueError):
            dec.step(*args)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=dec.stream):
        junk = one + 1                                 # a graph of something
        status = mk_decode_step_paged(dec.h, one.data_ptr(), one.data_ptr(), None, 1, None, None)
    assert status == MK_ERR_STATE
    dec.update(reserve=[1, 0])
    torch.cuda.synchronize()
    assert int(dec.step(one, dec._int32([3]))[0]) >= 0
    dec.synchronize()
    dec.close()


def test_entry_points_keep_to_their_context(lib):
    from persistent_sm_decode_megakernel_gb300 import MK_ERR_INVALID, mk_decode_step_paged
    cfg = synth.CONFIGS["tiny"]
    w = synth.gen_weights(cfg)
    dec = _paged(lib, cfg, w, 2, 1, 16)
    plain = lib.Decoder(lib.DeviceModel(cfg, w, max_batch=1, max_ctx=8))
    one = torch.zeros(1, dtype=torch.int32, device=dec.dm.device)
    assert lib.Decoder.decode_step_status(dec, [1], [0])[0] == MK_ERR_INVALID
    t, tp = lib._i32([1])
    out, op = lib._i32([0])
    assert lib.mk_prefill(dec.h, tp, 1, 1, op, None) == MK_ERR_INVALID
    assert lib.mk_decode_steps(dec.h, tp, tp, 1, 1, None) == MK_ERR_INVALID
    assert mk_decode_step_paged(plain.h, one.data_ptr(), one.data_ptr(), None, 1, None, None) == MK_ERR_INVALID
    for B in (0, 3):
        assert mk_decode_step_paged(dec.h, one.data_ptr(), one.data_ptr(), None, B, None, None) == MK_ERR_INVALID
    assert mk_decode_step_paged(dec.h, None, one.data_ptr(), None, 1, None, None) == MK_ERR_INVALID
    with pytest.raises(ValueError):
        dec.beam_search([1, 2], 2, 4)
    with pytest.raises(ValueError):
        dec.beam_search([1, 2], 1, 16)
    dec.close()
    plain.close()
