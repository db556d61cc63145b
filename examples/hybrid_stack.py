"""A small hybrid stack served with the library's operators: a Mamba2 layer (short convolution,
SSD scan), a channel-wise (Mamba) layer (short convolution, selective scan) and an attention layer
with grouped heads over a paged 8-bit key / value cache.

Packed prompts go through ``Stack.prompt`` (fresh, or continuing what their slots and pages hold),
verify steps of a few tokens through ``Stack.verify``, and ``Stack.commit`` rolls every layer back to
the accepted counts. Everything with a state is the library's; projections and norms are plain
torch, or (``four_bit``) the library's too: the residual's addition and the norm into 8 bits, products
with 4-bit weights, the gated norm behind the scan. ``speculate`` answers with it: drafts from a
head on the embeddings alone, token probabilities, the verification of the drafts and the commit
of what was accepted. Random weights: run as a program, it checks that a prompt in two parts followed
by verify steps with rejected drafts gives what one pass over the same tokens gives, and prints
times.

    python examples/hybrid_stack.py [--hidden 1024 --tokens 2048 --seqs 4]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import state_space_model_varlen_amd as ssd  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class Stack:
    HEADDIM, D_STATE, CHUNK, WIDTH = 64, 128, 128, 4      # Mamba2
    STATES = 16                                           # channel-wise scan
    PAGE, KV_DIM = 64, 64                                 # cache

    def __init__(self, hidden: int, max_seqs: int, max_tokens: int, device="cuda", seed=0,
                 four_bit=False, vocab=0):
        self.dev, self.h, self.slots = torch.device(device), hidden, max_seqs
        self.inner = 2 * hidden
        self.heads = self.inner // self.HEADDIM           # SSD heads
        self.q_heads = hidden // self.KV_DIM
        self.kv_heads = max(1, self.q_heads // 4)
        self.pages_per_seq = -(-max_tokens // self.PAGE)
        g = torch.Generator(device).manual_seed(seed)
        w = lambda o, i: (torch.randn(i, o, generator=g, device=self.dev) * i ** -0.5).to(BF)  # noqa: E731
        p = lambda *s: torch.randn(*s, generator=g, device=self.dev)                         # noqa: E731
        step = lambda n: torch.log(torch.expm1(torch.exp(                                    # noqa: E731
            torch.rand(n, generator=g, device=self.dev) * 4.6 - 6.9)))
        N, d = self.D_STATE, self.inner
        # Mamba2: rows [z | x B C | dt]
        self.conv2_c = d + 2 * N
        self.in2, self.out2 = w(d + self.conv2_c + self.heads, hidden), w(hidden, d)
        self.conv2_w, self.conv2_b = p(self.conv2_c, self.WIDTH) * 0.5, p(self.conv2_c) * 0.1
        self.A2, self.D2 = -torch.exp(p(self.heads)), p(self.heads)
        self.tf2 = ssd.make_dt_transform(step(self.heads), 0.0, 1e30)
        # channel-wise: rows [x | z], then [dt low rank | B | C] of the convolved x
        self.rank = max(16, hidden // 16)
        self.in1, self.out1 = w(2 * d, hidden), w(hidden, d)
        self.conv1_w, self.conv1_b = p(d, self.WIDTH) * 0.5, p(d) * 0.1
        self.x1, self.dt1 = w(self.rank + 2 * self.STATES, d), w(d, self.rank)
        self.A1 = -torch.arange(1, self.STATES + 1, device=self.dev).float().repeat(d, 1)
        self.D1, self.tf1 = p(d), ssd.make_dt_transform(step(d), 0.0, 1e30)
        # attention: rows [q | k | v]
        self.qkv = w((self.q_heads + 2 * self.kv_heads) * self.KV_DIM, hidden)
        self.out_a = w(hidden, self.q_heads * self.KV_DIM)
        # what the slots hold
        z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device=self.dev)               # noqa: E731
        self.conv2_s, self.conv1_s = (z(max_seqs, self.WIDTH - 1, c) for c in (self.conv2_c, d))
        self.ssd_s = z(max_seqs, self.heads, self.HEADDIM, N, dtype=F32)
        self.scan_s = z(max_seqs, d, self.STATES, dtype=F32)
        self.kv = ssd.make_kv_cache_problem(max_seqs * self.pages_per_seq, self.PAGE,
                                            self.kv_heads, self.KV_DIM, BF, torch.float8_e4m3fn)
        self.cache = ssd.alloc_kv_cache(self.kv, self.dev)
        self.pages = torch.arange(max_seqs * self.pages_per_seq, device=self.dev,
                                  dtype=torch.int32).view(max_seqs, -1).flip(1).contiguous()
        self.lens = torch.zeros(max_seqs, dtype=torch.int64)
        self.four_bit, self.vocab = four_bit, vocab
        if vocab:
            self.head, self.emb = w(vocab, hidden), torch.randn(vocab, hidden, generator=g,
                                                                device=self.dev).to(BF)
        if four_bit:
            self.gate_w = p(d) * 0.1 + 1
            for name in ("in2", "out2", "in1", "out1", "qkv", "out_a") + (("head",) if vocab else ()):
                setattr(self, name, self._encoded(getattr(self, name)))

    def _encoded(self, m):
        """m [in,out] as 4-bit weights."""
        k, n = m.shape
        lp = ssd.make_linear_problem(1, k, n, BF, BF)
        held = ssd.alloc_linear_weights(lp, self.dev)
        ssd.linear_w4_encode(lp, m.t().contiguous(), **held)
        return held

    def _product(self, x, w, scale=None):
        """x [T,K], bfloat16 or 8-bit rows with their scales, times 4-bit weights."""
        out = torch.empty(x.shape[0], w["weight"].shape[0], dtype=BF, device=self.dev)
        lp = ssd.make_linear_problem(x.shape[0], x.shape[1], out.shape[1], x.dtype, BF)
        ssd.linear_w4(lp, x, w["weight"], w["weight_scale"], out, x_scale=scale,
                      workspace=ssd.alloc_linear_workspace(lp, self.dev))
        return out

    def _into(self, x, add, w):
        """The residual stream with a layer's output added, and its norm times w."""
        if not self.four_bit:
            x = x if add is None else x + add
            return x, self._norm(x) @ w
        T, h = x.shape
        rows = torch.empty(T, h, dtype=torch.float8_e4m3fn, device=self.dev)
        scale = torch.empty(T, h // 32, dtype=torch.uint8, device=self.dev)
        np_ = ssd.make_norm_problem(T, h, BF, torch.float8_e4m3fn)
        if add is None:
            ssd.rms_norm(np_, x, None, rows, out_scale=scale)
        else:
            total = torch.empty_like(x)
            ssd.rms_norm(np_, add, None, rows, residual=x, residual_out=total, out_scale=scale)
            x = total
        return x, self._product(rows, w, scale)

    def _out(self, y, w):
        return self._product(y, w) if self.four_bit else y @ w

    def _gated(self, y, z):
        """The scan's result under its gate (and, in 4 bits, normed)."""
        if not self.four_bit:
            return y * torch.nn.functional.silu(z)
        out = torch.empty_like(y)
        ssd.rms_norm(ssd.make_norm_problem(*y.shape, BF, BF), y, self.gate_w, out, gate=z)
        return out

    def _norm(self, x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).to(BF)

    def _check_room(self, slots, counts):
        """Before any state changes: every slot's pages hold the new tokens too."""
        room = self.pages_per_seq * self.PAGE
        for s, n in zip(slots, counts):
            if int(self.lens[s]) + n > room:
                raise ValueError(f"slot {s} holds {int(self.lens[s])} tokens and has room for {room} "
                                 f"(got {n} more)")

    def _positions(self, slots, counts):
        """Cache position of every new row: page * page size + place."""
        pos = torch.cat([torch.arange(int(self.lens[s]), int(self.lens[s]) + n)
                         for s, n in zip(slots, counts)]).to(self.dev)
        row = torch.repeat_interleave(torch.tensor(slots), torch.tensor(counts)).to(self.dev)
        return self.pages[row, pos // self.PAGE].long() * self.PAGE + pos % self.PAGE

    def _split_qkv(self, x, add):
        q, k = self.q_heads * self.KV_DIM, self.kv_heads * self.KV_DIM
        x, r = self._into(x, add, self.qkv)
        return (x, r[:, :q].unflatten(1, (-1, self.KV_DIM)), r[:, q:q + k].unflatten(1, (-1, self.KV_DIM)),
                r[:, q + k:].unflatten(1, (-1, self.KV_DIM)))

    def prompt(self, x, slots, counts):
        """x [T,hidden]: counts[i] new tokens for slot slots[i], behind what it holds."""
        self._check_room(slots, counts)
        T, S, d, N, dev = x.shape[0], len(slots), self.inner, self.D_STATE, self.dev
        cu = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(dev)
        idx = torch.tensor(slots, dtype=torch.int32, device=dev)
        has = torch.tensor([int(self.lens[s] > 0) for s in slots], dtype=torch.uint8, device=dev)
        new = lambda *s: torch.empty(*s, dtype=BF, device=dev)                               # noqa: E731
        # Mamba2
        x, r = self._into(x, None, self.in2)
        xs, B, C = new(T, d), new(T, N), new(T, N)
        p = ssd.make_conv_problem(T, S, self.conv2_c, self.WIDTH, self.slots, BF, BF)
        ssd.causal_conv1d_varlen(p, r[:, d:d + self.conv2_c], self.conv2_w, self.conv2_b, cu,
                                 self.conv2_s, idx, has, (xs, B, C))
        sp = ssd.make_problem(T, S, self.heads, self.HEADDIM, N, 1, self.CHUNK, self.slots, BF, F32)
        y = new(T, self.heads, self.HEADDIM)
        ssd.ssd_combined_varlen_dt(sp, self.tf2, xs.view_as(y), r[:, -self.heads:].contiguous(), self.A2,
                                   B.view(T, 1, N), C.view(T, 1, N), self.D2, cu, self.ssd_s, idx, has,
                                   y, None, ssd.alloc_workspace(sp, dev))
        add = self._out(self._gated(y.view(T, d), r[:, :d]), self.out2)
        # channel-wise scan
        x, r = self._into(x, add, self.in1)
        p = ssd.make_conv_problem(T, S, d, self.WIDTH, self.slots, BF, BF)
        xs = new(T, d)
        ssd.causal_conv1d_varlen(p, r[:, :d], self.conv1_w, self.conv1_b, cu, self.conv1_s, idx, has, xs)
        dt, B, C = self._dt_b_c(xs)
        p = ssd.make_scan_problem(T, S, d, self.STATES, 1, self.slots, BF, F32)
        y = new(T, d)
        ssd.selective_scan_varlen(p, xs, dt, self.A1, B, C, self.D1, r[:, d:], self.tf1, cu, self.scan_s,
                                  idx, has, y, ssd.alloc_scan_workspace(p, dev))
        add = self._out(y, self.out1)
        # attention: the new rows join the cache, a continued prompt reads its own back
        x, q, k, v = self._split_qkv(x, add)
        ssd.kv_cache_store(self.kv, k, v, self._positions(slots, counts), **self.cache)
        full = [int(self.lens[s]) + n for s, n in zip(slots, counts)]
        cuk = torch.tensor([0] + full).cumsum(0).to(torch.int32).to(dev)
        kk, vv = (new(sum(full), self.kv_heads, self.KV_DIM) for _ in range(2))
        ssd.kv_cache_load(self.kv, cuk, self.pages[idx.long()], self.cache["k_cache"],
                          self.cache["v_cache"], self.cache["k_scale"], self.cache["v_scale"], kk, vv)
        p = ssd.make_attn_problem(T, sum(full), S, self.q_heads, self.kv_heads, self.KV_DIM, BF)
        o = new(T, self.q_heads, self.KV_DIM)
        ssd.attention_varlen(p, q, kk, vv, cu, cuk, o)
        for s, n in zip(slots, counts):
            self.lens[s] += n
        return x + self._out(o.view(T, -1), self.out_a)

    def _dt_b_c(self, xs):
        r = xs @ self.x1
        n = self.STATES
        return (r[:, :self.rank] @ self.dt1, r[:, self.rank:self.rank + n].unflatten(1, (1, n)),
                r[:, self.rank + n:].unflatten(1, (1, n)))

    def verify(self, x, slots, tokens):
        """x [R T,hidden]: `tokens` tokens for every slot of `slots`; states stay where they were
        until commit() says how many of them count."""
        self._check_room(slots, [tokens] * len(slots))
        R, T, d, N, dev = len(slots), tokens, self.inner, self.D_STATE, self.dev
        idx = torch.tensor(slots, dtype=torch.int32, device=dev)
        new = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device=dev)                  # noqa: E731
        x, r = self._into(x, None, self.in2)
        xs, B, C = new(R * T, d), new(R * T, N), new(R * T, N)
        p2 = ssd.make_conv_problem(R * T, R, self.conv2_c, self.WIDTH, self.slots, BF, BF)
        raw2 = r[:, d:d + self.conv2_c]
        ssd.causal_conv1d_update(p2, raw2, self.conv2_w, self.conv2_b, self.conv2_s, idx, (xs, B, C),
                                 update_cache=False)
        up = ssd.make_ssu_problem(R, T, self.heads, self.HEADDIM, N, 1, self.slots, BF, F32)
        y = new(R, T, self.heads, self.HEADDIM)
        st2 = new(R, T, self.heads, self.HEADDIM, N, dtype=F32)
        ssd.selective_state_update_ex(up, ssd.make_options(dt_transform=self.tf2), self.ssd_s, idx,
                                      xs.view_as(y),
                                      r[:, -self.heads:].contiguous().view(R, T, -1),
                                      self.A2, B.view(R, T, 1, N), C.view(R, T, 1, N), self.D2, y, st2)
        add = self._out(self._gated(y.view(R * T, d), r[:, :d]), self.out2)
        x, r = self._into(x, add, self.in1)
        p1 = ssd.make_conv_problem(R * T, R, d, self.WIDTH, self.slots, BF, BF)
        xs, y, raw1 = new(R * T, d), new(R * T, d), r[:, :d]
        ssd.causal_conv1d_update(p1, raw1, self.conv1_w, self.conv1_b, self.conv1_s, idx, xs,
                                 update_cache=False)
        dt, B, C = self._dt_b_c(xs)
        ps = ssd.make_scan_problem(R * T, R, d, self.STATES, 1, self.slots, BF, F32)
        st1 = new(R * T, d, self.STATES, dtype=F32)
        ssd.selective_scan_update(ps, xs, dt, self.A1, B, C, self.D1, r[:, d:], self.tf1, self.scan_s,
                                  idx, y, st1)
        add = self._out(y, self.out1)
        x, q, k, v = self._split_qkv(x, add)
        ssd.kv_cache_store(self.kv, k, v, self._positions(slots, [T] * R), **self.cache)
        pd = ssd.make_attn_decode_problem(self.kv, R, T, self.q_heads, self.pages.shape[1])
        o = new(R, T, self.q_heads, self.KV_DIM)
        lens = torch.tensor([int(self.lens[s]) + T for s in slots], dtype=torch.int32, device=dev)
        ssd.attention_decode(pd, q.reshape(o.shape), self.cache["k_cache"], self.cache["v_cache"],
                             self.cache["k_scale"], self.cache["v_scale"],
                             self.pages[idx.long()].contiguous(), lens, o,
                             workspace=ssd.alloc_attn_decode_workspace(pd, dev))
        self._pending = (slots, T, p2, raw2, up, st2, p1, raw1, st1, idx)
        return x + self._out(o.view(R * T, -1), self.out_a)

    def commit(self, accepted):
        """accepted[r] drafts of the last verify step count (its first token always does)."""
        slots, T, p2, raw2, up, st2, p1, raw1, st1, idx = self._pending
        acc = torch.tensor(accepted, dtype=torch.int32, device=self.dev)
        ssd.causal_conv1d_commit(p2, raw2, self.conv2_s, idx, acc)
        ssd.ssd_state_commit(up, self.ssd_s, idx, st2, acc)
        ssd.causal_conv1d_commit(p1, raw1, self.conv1_s, idx, acc)
        # the scan's states as rows [C / 64, 64, 16] of the same commit
        R, d, n = len(slots), self.inner, self.STATES
        us = ssd.make_ssu_problem(R, T, d // 64, 64, n, 1, self.slots, BF, F32)
        ssd.ssd_state_commit(us, self.scan_s.view(-1, d // 64, 64, n), idx,
                             st1.view(R, T, d // 64, 64, n), acc)
        for s, a in zip(slots, accepted):     # a rejected token's rows are overwritten by the next
            self.lens[s] += 1 + a


    # -- answers: vocab > 0 --

    def logits(self, x):
        return self._into(x, None, self.head)[1]

    def probs(self, logits, temperature):
        """[R,T,V] of logits [R T,V] at a temperature a request."""
        R, V = temperature.shape[0], self.vocab
        p = ssd.make_probs_problem(R, logits.shape[0] // R, V, BF)
        out = torch.empty(R, p.tokens_per_req, V, device=self.dev)
        ssd.token_probs(p, logits.view(out.shape), temperature, out,
                        ssd.alloc_probs_workspace(p, self.dev))
        return out

    def judged(self, target, draft, drafts, uniform):
        """Accepted counts and tokens of target [R,T,V], draft [R,T-1,V], drafts [R,T-1]."""
        R, T, V = target.shape
        p = ssd.make_verify_problem(R, T, V)
        acc = torch.empty(R, dtype=torch.int32, device=self.dev)
        tokens = torch.empty(R, T, dtype=torch.int32, device=self.dev)
        ssd.verify_drafts(p, target, draft, drafts, None, uniform, acc, tokens,
                          ssd.alloc_verify_workspace(p, self.dev))
        return acc, tokens

    def speculate(self, last, slots, drafts, temperature, gen):
        """One step behind each slot's last token: `drafts` tokens from the head on the embeddings
        alone, verified together. Returns the tokens that count, per slot, and what the step saw."""
        R, u = len(slots), lambda t: torch.rand(R, t, generator=gen, device=self.dev)        # noqa: E731
        rows, qs, at = [last], [], last
        for _ in range(drafts):
            q = self.probs(self.logits(self.emb[at.long()]), temperature)
            at = self.judged(q, None, None, u(1))[1][:, 0]          # plain sampling
            rows.append(at)
            qs.append(q)
        T = drafts + 1
        x = self.emb[torch.stack(rows, 1).flatten().long()]
        target = self.probs(self.logits(self.verify(x, slots, T)), temperature)
        draft = torch.cat(qs, 1) if drafts else None
        tokens = torch.stack(rows[1:], 1).to(torch.int32) if drafts else None
        uniform = u(T)
        acc, out = self.judged(target, draft, tokens, uniform)
        self.commit(acc.tolist())
        return ([r[:a + 1].tolist() for r, a in zip(out.cpu(), acc.tolist())],
                (target, draft, tokens, uniform, acc, out))


def check(hidden=256, lens=(70, 1, 133), steps=3, tokens=3, seed=0, four_bit=False):
    """A prompt in two parts and verify steps with rejected drafts, against one pass over all the
    tokens that counted: the largest difference relative to the result's norm, per sequence."""
    dev, S = "cuda", len(lens)
    g = torch.Generator(dev).manual_seed(seed + 1)
    accepted = [[(i + k) % tokens for i in range(S)] for k in range(steps)]
    total = [n + sum(1 + accepted[k][i] for k in range(steps)) for i, n in enumerate(lens)]
    xs = [torch.randn(n, hidden, generator=g, device=dev).to(BF) for n in total]
    whole = Stack(hidden, S, max(total) + tokens, dev, seed, four_bit)
    want = whole.prompt(torch.cat(xs), list(range(S)), total).split(total)
    st = Stack(hidden, S, max(total) + tokens, dev, seed, four_bit)
    order = list(range(S))[::-1]              # slots other than the order of the batch
    cut = [n // 2 for n in lens]
    parts = [i for i in order if cut[i] > 0]
    got = [[] for _ in lens]

    def keep(rows, who, counts):
        for i, r in zip(who, rows.split(counts)):
            got[i].append(r)

    keep(st.prompt(torch.cat([xs[i][:cut[i]] for i in parts]), parts, [cut[i] for i in parts]), parts,
         [cut[i] for i in parts])
    keep(st.prompt(torch.cat([xs[i][cut[i]:lens[i]] for i in order]), order,
                   [lens[i] - cut[i] for i in order]), order, [lens[i] - cut[i] for i in order])
    at = list(lens)
    for k in range(steps):
        rows = []
        for i in order:                       # tokens that count, then drafts that will not
            keepn = 1 + accepted[k][i]
            rows += [xs[i][at[i]:at[i] + keepn],
                     torch.randn(tokens - keepn, hidden, generator=g, device=dev).to(BF)]
        y = st.verify(torch.cat(rows), order, tokens).split(tokens)
        st.commit([accepted[k][i] for i in order])
        for i, r in zip(order, y):
            got[i].append(r[:1 + accepted[k][i]])
            at[i] += 1 + accepted[k][i]
    return [float((torch.cat(a).double() - w.double()).norm() / w.double().norm())
            for a, w in zip(got, want)]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--seqs", type=int, default=4)
    a = ap.parse_args()
    print("prompt in two parts + verify steps against one pass, relative difference a sequence:",
          ["%.1e" % e for e in check()], "4-bit weights, 8-bit rows:",
          ["%.1e" % e for e in check(four_bit=True)])
    for four_bit in (False, True):
        times(a, four_bit)


def times(a, four_bit):
    st = Stack(a.hidden, a.seqs, a.tokens + 64, four_bit=four_bit, vocab=32000)
    per = [a.tokens // a.seqs] * a.seqs
    x = torch.randn(sum(per), a.hidden, device="cuda").to(BF)
    y = torch.randn(3 * a.seqs, a.hidden, device="cuda").to(BF)

    def timed(f, n=10):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e3

    def fresh():
        st.lens.zero_()
        st.prompt(x, list(range(a.seqs)), per)

    print("4-bit weights" if four_bit else "bfloat16 weights")
    print("  prompt, %d sequences, %d tokens: %.2f ms" % (a.seqs, sum(per), timed(fresh)))
    print("  verify step, 3 tokens each: %.2f ms" % timed(lambda: st.verify(y, list(range(a.seqs)), 3)))
    gen, temp = torch.Generator("cuda").manual_seed(0), torch.full((a.seqs,), 0.8, device="cuda")
    last = torch.zeros(a.seqs, dtype=torch.int32, device="cuda")
    print("  draft, verify and commit 3 tokens each: %.2f ms" % timed(
        lambda: st.speculate(last, list(range(a.seqs)), 2, temp, gen), 5))


if __name__ == "__main__":
    main()
