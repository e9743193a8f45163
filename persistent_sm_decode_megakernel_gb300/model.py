"""Device-side model holder and a decoder handle over the C ABI.

PyTorch is used for device memory and streams only: weights and KV caches are torch
tensors on the GPU whose raw addresses go into mk_weights / mk_kv; all arithmetic of
the decode step runs in libmk.so.
"""
import ctypes

import numpy as np
import torch

from . import (MK_BF16, MK_F16, MK_OK, MK_ERR_NAN, check, mk_create, mk_decode_step, mk_decode_steps,
               mk_destroy, mk_get_trace, mk_info, mk_info_t, mk_kv, mk_model_desc, mk_options, mk_prefill,
               mk_read_activation, mk_reset, mk_synchronize, mk_trace_rec, mk_weights, P_i32)

_LAYER_TENSORS = ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "w_gate", "w_up", "w_down")


def _to_device(bits: np.ndarray, device) -> torch.Tensor:
    """uint16 storage bits -> int16 device tensor holding the same bytes."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device, non_blocking=False)


class DeviceModel:
    """Weights (storage bits) resident in HBM plus a KV cache of max_ctx positions."""

    def __init__(self, cfg, weights, max_batch, max_ctx, device="cuda:0"):
        self.cfg = cfg
        self.device = torch.device(device)
        self.max_batch = max_batch
        self.max_ctx = max_ctx
        self.embed = _to_device(weights["embed"], self.device)
        self.final_norm = _to_device(weights["final_norm"], self.device)
        self.lm_head = _to_device(weights["lm_head"], self.device)
        self.layers = [{n: _to_device(weights["layers"][l][n], self.device) for n in _LAYER_TENSORS}
                       for l in range(cfg.n_layers)]
        shape = (max_batch, cfg.n_kv_heads, max_ctx, cfg.head_dim)
        self.k_cache = [torch.zeros(shape, dtype=torch.int16, device=self.device) for _ in range(cfg.n_layers)]
        self.v_cache = [torch.zeros(shape, dtype=torch.int16, device=self.device) for _ in range(cfg.n_layers)]

    def desc(self):
        c = self.cfg
        return mk_model_desc(c.n_layers, c.d_model, c.n_heads, c.n_kv_heads, c.head_dim, c.ffn_dim, c.vocab,
                             MK_F16 if c.dtype == "f16" else MK_BF16, c.rms_eps, c.rope_theta,
                             self.max_batch, self.max_ctx)

    def abi_structs(self):
        L = self.cfg.n_layers
        arr = ctypes.c_void_p * L
        tabs = {n: arr(*[self.layers[l][n].data_ptr() for l in range(L)]) for n in _LAYER_TENSORS}
        w = mk_weights(self.embed.data_ptr(), self.final_norm.data_ptr(), self.lm_head.data_ptr(),
                       *[ctypes.cast(tabs[n], ctypes.POINTER(ctypes.c_void_p)) for n in _LAYER_TENSORS])
        kt = arr(*[t.data_ptr() for t in self.k_cache])
        vt = arr(*[t.data_ptr() for t in self.v_cache])
        kv = mk_kv(ctypes.cast(kt, ctypes.POINTER(ctypes.c_void_p)), ctypes.cast(vt, ctypes.POINTER(ctypes.c_void_p)))
        return w, kv, (tabs, kt, vt)   # keep the host tables alive while mk_create reads them

    def set_kv(self, layer, b, k_bits, v_bits):
        """Fill positions 0..T-1 of sequence b's cache in one layer from storage bits
        [n_kv_heads, T, head_dim] (uint16)."""
        T = k_bits.shape[1]
        self.k_cache[layer][b, :, :T] = _to_device(k_bits, self.device)
        self.v_cache[layer][b, :, :T] = _to_device(v_bits, self.device)

    def weight_bytes(self):
        n = self.lm_head.numel() + self.final_norm.numel()
        for lt in self.layers:
            n += sum(t.numel() for t in lt.values())
        return 2 * n


def _i32(a):
    a = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return a, a.ctypes.data_as(P_i32)


class Decoder:
    """A context over a DeviceModel (mk_create ... mk_destroy)."""

    def __init__(self, dm: DeviceModel, sync_mode=0, exec_mode=0, trace=0, timeout_s=2.0, page_bytes=0,
                 n_pages=0, kv_splits=0, max_ctas=0, fault_drop_signal=0, backoff_max_ns=0,
                 split_min_positions=0, attn_merge=0, inflight_pages=0, attn_pool=0, attn_tensor_cores=0,
                 stream=None):
        self.dm = dm
        self.stream = stream if stream is not None else torch.cuda.current_stream(dm.device)
        self.opts = mk_options(sync_mode, exec_mode, page_bytes, n_pages, kv_splits, trace, timeout_s,
                               backoff_max_ns, max_ctas, fault_drop_signal, split_min_positions,
                               attn_merge, inflight_pages, attn_pool, attn_tensor_cores)
        d = dm.desc()
        w, kv, _keep = dm.abi_structs()
        h = ctypes.c_void_p()
        check(mk_create(ctypes.byref(d), ctypes.byref(w), ctypes.byref(kv), ctypes.byref(self.opts),
                        ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(h)), "mk_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            mk_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def info(self):
        i = mk_info_t()
        check(mk_info(self.h, ctypes.byref(i)), "mk_info")
        return {k: getattr(i, k) for k, _ in mk_info_t._fields_}

    def prefill(self, tokens, logits=None, allow_nan=False):
        tokens = np.asarray(tokens, dtype=np.int32)
        B, P = tokens.shape
        t, tp = _i32(tokens)
        out, op = _i32(np.zeros(B))
        st = mk_prefill(self.h, tp, B, P, op, ctypes.c_void_p(logits.data_ptr() if logits is not None else 0))
        if not (allow_nan and st == MK_ERR_NAN):
            check(st, "mk_prefill")
        return out.copy()

    def decode_step(self, in_tok, pos, logits=None):
        B = len(in_tok)
        t, tp = _i32(in_tok)
        p, pp = _i32(pos)
        out, op = _i32(np.zeros(B))
        st = mk_decode_step(self.h, tp, pp, B, op, ctypes.c_void_p(logits.data_ptr() if logits is not None else 0))
        check(st, "mk_decode_step")
        return out.copy()

    def decode_step_status(self, in_tok, pos, logits=None):
        B = len(in_tok)
        t, tp = _i32(in_tok)
        p, pp = _i32(pos)
        out, op = _i32(np.zeros(B))
        st = mk_decode_step(self.h, tp, pp, B, op, ctypes.c_void_p(logits.data_ptr() if logits is not None else 0))
        return st, out.copy()

    def decode_steps(self, in_tok, pos0, n_steps, out_dev=None):
        """in_tok None continues from the token the previous step chose on the device."""
        B = len(pos0)
        if in_tok is None:
            tp = None
        else:
            t, tp = _i32(in_tok)
        p, pp = _i32(pos0)
        ptr = ctypes.c_void_p(out_dev.data_ptr() if out_dev is not None else 0)
        check(mk_decode_steps(self.h, tp, pp, B, n_steps, ptr), "mk_decode_steps")

    def synchronize(self):
        check(mk_synchronize(self.h), "mk_synchronize")

    def reset(self):
        check(mk_reset(self.h), "mk_reset")

    def read_activation(self, which, layer):
        c = self.dm.cfg
        width = {0: c.d_model, 1: c.d_model, 2: c.q_dim, 3: c.q_dim, 4: c.ffn_dim}[which]
        out = np.zeros((self.dm.max_batch, width), dtype=np.float32)
        check(mk_read_activation(self.h, which, layer, out.ctypes.data_as(ctypes.POINTER(ctypes.c_float)),
                                 out.nbytes), "mk_read_activation")
        return out

    def trace(self, max_records=1 << 20):
        buf = (mk_trace_rec * max_records)()
        n = ctypes.c_int()
        check(mk_get_trace(self.h, buf, max_records, ctypes.byref(n)), "mk_get_trace")
        return [(r.cta, r.pc, r.op, r.layer, r.t_fetch, r.t_ready, r.t_end, *list(r.t_mark))
                for r in buf[: n.value]]


class PagedDecoder:
    """A decoder whose KV cache lies in pages (mk_create_paged), for several sequences that share,
    fork and free them, and a beam search over it.

    n_rows sequences (rows of the page table) of up to max_positions each, n_pages pages of
    page_size positions; a step takes up to dm.max_batch rows.  dm's own contiguous cache is not
    used (max_ctx=1 keeps it small).  rope: keyword arguments of paged.rope_freqs (theta, n_rot,
    kind, factor, ..) where the model's rotary positions are not plain."""

    def __init__(self, dm: DeviceModel, n_rows, n_pages, max_positions, page_size=64, rope=None, interleaved=False,
                 stream=None):
        from . import MK_BF16, mk_create_paged, mk_paged_kv, mk_rope_desc, paged
        c = dm.cfg
        self.dm, self.paged, self.page_size, self.max_positions = dm, paged, page_size, max_positions
        self.stream = stream if stream is not None else torch.cuda.current_stream(dm.device)
        dtype = torch.bfloat16 if dm.desc().dtype == MK_BF16 else torch.float16
        with torch.cuda.stream(self.stream):
            pages = torch.zeros((2, c.n_layers, n_pages, c.n_kv_heads, page_size, c.head_dim), dtype=dtype, device=dm.device)
            self.k, self.v = pages[0], pages[1]
            self.table = torch.full((n_rows, -(-max_positions // page_size)), -1, dtype=torch.int32, device=dm.device)
            self.lens = torch.zeros(n_rows, dtype=torch.int32, device=dm.device)
            self.refs = torch.zeros(n_pages, dtype=torch.int32, device=dm.device)
            self.status = torch.zeros(4, dtype=torch.int32, device=dm.device)
        d = dm.desc()
        w, _, _keep = dm.abi_structs()
        pk = mk_paged_kv(self.k.data_ptr(), self.v.data_ptr(), self.k.stride(0), self.k.stride(1), n_pages, page_size,
                         self.table.data_ptr(), n_rows, self.table.shape[1], self.table.stride(0))
        r = None
        if rope is not None:
            kw = {"theta": c.rope_theta, "n_rot": c.head_dim, "kind": "none", "factor": 1.0, "original": 0.0,
                  "beta_fast": 0.0, "beta_slow": 0.0}
            if not set(rope) <= set(kw):
                raise ValueError(f"rope's arguments are {sorted(kw)}")
            kw.update(rope)
            if kw["kind"] not in paged.ROPE_KINDS:
                raise ValueError(f"kind must be one of {sorted(paged.ROPE_KINDS)}")
            r = ctypes.byref(mk_rope_desc(kw["theta"], kw["n_rot"], paged.ROPE_KINDS[kw["kind"]], kw["factor"],
                                          kw["original"], kw["beta_fast"], kw["beta_slow"]))
        h = ctypes.c_void_p()
        with torch.cuda.device(dm.device):
            check(mk_create_paged(ctypes.byref(d), ctypes.byref(w), ctypes.byref(pk), r, int(interleaved), None,
                                  ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(h)), "mk_create_paged")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            with torch.cuda.device(self.dm.device):
                mk_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _int32(self, x):
        return torch.as_tensor(x, dtype=torch.int32, device=self.dm.device)

    def _used(self, t):
        """A caller's tensor that self.stream reads or writes: its memory is not given to anyone else before that."""
        if t is not None and t.is_cuda:
            t.record_stream(self.stream)
        return t

    def synchronize(self):
        """Waits for the stream and raises MkError for what a page update or a step reported: the update's where
        both did, and neither report is left for a later call."""
        from . import MkError
        first = None
        with torch.cuda.stream(self.stream):
            for read in (lambda: self.paged.check_status(self.status), lambda: check(mk_synchronize(self.h), "mk_synchronize")):
                try:
                    read()
                except MkError as e:
                    first = first or e
        if first is not None:
            raise first

    def reset(self):
        """Makes the context usable again after an error of a step (a token that is none, a NaN logit, a timeout).
        Rows, pages and their counts stay as they are."""
        with torch.cuda.device(self.dm.device):
            check(mk_reset(self.h), "mk_reset")

    def update(self, parents=None, reserve=None):
        """Every row continues row parents[r] (-1: it is freed) and reserves pages for reserve[r] more
        positions (mk_update_pages).  It runs on self.stream, where tensors given have to be ready."""
        with torch.cuda.stream(self.stream):
            parents, reserve = (None if x is None else self._used(self._int32(x)) for x in (parents, reserve))
            self.paged.update_pages(self.k, self.v, self.table, self.lens, self.refs, parents, reserve, self.status)

    def step(self, tokens, positions, rows=None, logits=None):
        """One step of device int32 tensors: token i at positions[i] of table row rows[i] (default i).  The
        argmax tokens; positions need their pages (update).  lens is the caller's to advance.  It runs on
        self.stream, where its tensors have to be ready; they may be dropped as soon as it returns."""
        from . import mk_decode_step_paged
        n = len(tokens)
        for name, t, shape, dtype in (("tokens", tokens, (n,), torch.int32), ("positions", positions, (n,), torch.int32),
                                      ("rows", rows, (n,), torch.int32),
                                      ("logits", logits, (n, self.dm.cfg.vocab), torch.float32)):
            if t is None and name in ("rows", "logits"):
                continue
            if tuple(t.shape) != shape or t.dtype != dtype or t.device != self.k.device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of {shape} on {self.k.device}")
        with torch.cuda.stream(self.stream):
            for t in (tokens, positions, rows, logits):
                self._used(t)
            out = torch.empty(n, dtype=torch.int32, device=self.k.device)
            check(mk_decode_step_paged(self.h, tokens.data_ptr(), positions.data_ptr(),
                                       rows.data_ptr() if rows is not None else None, n, out.data_ptr(),
                                       logits.data_ptr() if logits is not None else None), "mk_decode_step_paged")
        return out

    def _tokens(self, prompt):
        tokens = [int(t) for t in prompt]
        if any(not 0 <= t < self.dm.cfg.vocab for t in tokens):
            raise ValueError("a prompt's tokens must be in [0, vocab)")
        return tokens

    def prefill(self, prompts, logits=None):
        """Appends prompts {row: tokens} to their rows, up to dm.max_batch positions per step.  Returns
        {row: next token} (device int32 [1] each); logits {row: float32 [vocab]} receives the last ones.  Raises
        ValueError for a prompt that does not fit or a token that is none, and MkError when the pages run out,
        before any of it."""
        with torch.cuda.stream(self.stream):
            n_rows, V = self.table.shape[0], self.dm.cfg.vocab
            start = self.lens.tolist()
            reserve = [0] * n_rows
            prompts = {r: self._tokens(p) for r, p in prompts.items()}
            for r, p in prompts.items():
                if not 0 <= r < n_rows or len(p) < 1 or start[r] + len(p) > self.max_positions:
                    raise ValueError("a prompt must be of a row of the table, not empty and fit max_positions")
                reserve[r] = len(p)
            self.update(reserve=reserve)
            self.synchronize()
            jobs = [(t, start[r] + i, r, i == len(p) - 1) for r, p in prompts.items() for i, t in enumerate(p)]
            last = {}
            for at in range(0, len(jobs), self.dm.max_batch):
                part = jobs[at: at + self.dm.max_batch]
                tok, pos, row = (self._int32([j[x] for j in part]) for x in range(3))
                z = torch.empty((len(part), V), dtype=torch.float32, device=self.dm.device) if logits is not None else None
                out = self.step(tok, pos, row, z)
                for i, j in enumerate(part):
                    if j[3]:
                        last[j[2]] = out[i: i + 1]
                        if logits is not None:
                            self._used(logits[j[2]]).copy_(z[i])
            self.lens += self._int32(reserve)
        return last

    def beam_search(self, prompt, beams, n_new, eos=-1):
        """The `beams` best continuations of up to n_new tokens of one prompt by their summed log probability,
        best first: (tokens [beams, n_new] int32, scores [beams]) on the host; a beam that ended repeats eos.
        Uses table rows 0..beams-1, which are freed before and after."""
        dev, c = self.dm.device, self.dm.cfg
        n_rows = self.table.shape[0]
        if not 1 <= beams <= min(32, self.dm.max_batch, n_rows):
            raise ValueError("beams must be in [1, 32] and at most max_batch and n_rows")
        if n_new < 1 or len(prompt) < 1 or len(prompt) + n_new - 1 > self.max_positions:
            raise ValueError("the prompt and the new tokens must be positive and fit max_positions")
        if beams > c.vocab or not -1 <= eos < c.vocab:
            raise ValueError("beams must be at most vocab, eos a token or -1")
        prompt = self._tokens(prompt)
        keep = list(range(n_rows))
        with torch.cuda.stream(self.stream):
            self.update(parents=[-1] * beams + keep[beams:])
            first = {0: torch.empty(c.vocab, dtype=torch.float32, device=dev)}
            self.prefill({0: prompt}, first)
            logits = first[0].expand(beams, c.vocab).contiguous()
            scores = torch.full((1, beams), -float("inf"), device=dev)
            scores[0, 0] = 0.0                        # one beam until the first choice tells them apart
            ended = torch.zeros((1, beams), dtype=torch.int32, device=dev)
            parents, reserve = self._int32(keep), torch.zeros(n_rows, dtype=torch.int32, device=dev)
            history = []
            for i in range(n_new):
                tokens, par, scores, ended = self.paged.beam_select(logits, scores, ended, eos, self.status)
                history.append((tokens[0], par[0]))
                if i + 1 == n_new:
                    break
                # beam 0 holds the prompt for all of them at first
                parents[:beams] = par[0] if i else 0
                live = 1 - ended[0]                   # an ended beam has no further positions
                reserve[:beams] = live
                self.update(parents, reserve)
                self.step(tokens[0].contiguous(), torch.where(live != 0, self.lens[:beams], -1), None, logits)
                self.lens[:beams] += live
            self.update(parents=[-1] * beams + keep[beams:])
            self.synchronize()
            seqs = np.zeros((beams, n_new), dtype=np.int32)
            at = np.arange(beams)
            for i in reversed(range(n_new)):          # back along the parents
                tokens, par = (x.cpu().numpy() for x in history[i])
                seqs[:, i] = tokens[at]
                at = par[at]
            return seqs, scores[0].cpu().numpy()
