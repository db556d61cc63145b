"""A small hybrid stack served with the library's operators: a Mamba2 layer (short convolution,
SSD scan), a channel-wise (Mamba) layer (short convolution, selective scan) and an attention layer
with grouped heads over a paged 8-bit key / value cache.

Packed prompts go through ``Stack.prompt`` (fresh, or continuing what their slots and pages hold),
verify steps of a few tokens through ``Stack.verify``, and ``Stack.commit`` rolls every layer back to
the accepted counts. Projections and norms are plain torch; everything with a state is the
library's. Random weights: run as a program, it checks that a prompt in two parts followed by
verify steps with rejected drafts gives what one pass over the same tokens gives, and prints times.

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

    def __init__(self, hidden: int, max_seqs: int, max_tokens: int, device="cuda", seed=0):
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

    def _split_qkv(self, x):
        q, k = self.q_heads * self.KV_DIM, self.kv_heads * self.KV_DIM
        r = self._norm(x) @ self.qkv
        return (r[:, :q].unflatten(1, (-1, self.KV_DIM)), r[:, q:q + k].unflatten(1, (-1, self.KV_DIM)),
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
        r = self._norm(x) @ self.in2
        xs, B, C = new(T, d), new(T, N), new(T, N)
        p = ssd.make_conv_problem(T, S, self.conv2_c, self.WIDTH, self.slots, BF, BF)
        ssd.causal_conv1d_varlen(p, r[:, d:d + self.conv2_c], self.conv2_w, self.conv2_b, cu,
                                 self.conv2_s, idx, has, (xs, B, C))
        sp = ssd.make_problem(T, S, self.heads, self.HEADDIM, N, 1, self.CHUNK, self.slots, BF, F32)
        y = new(T, self.heads, self.HEADDIM)
        ssd.ssd_combined_varlen_dt(sp, self.tf2, xs.view_as(y), r[:, -self.heads:].contiguous(), self.A2,
                                   B.view(T, 1, N), C.view(T, 1, N), self.D2, cu, self.ssd_s, idx, has,
                                   y, None, ssd.alloc_workspace(sp, dev))
        x = x + (y.view(T, d) * torch.nn.functional.silu(r[:, :d])) @ self.out2
        # channel-wise scan
        r = self._norm(x) @ self.in1
        p = ssd.make_conv_problem(T, S, d, self.WIDTH, self.slots, BF, BF)
        xs = new(T, d)
        ssd.causal_conv1d_varlen(p, r[:, :d], self.conv1_w, self.conv1_b, cu, self.conv1_s, idx, has, xs)
        dt, B, C = self._dt_b_c(xs)
        p = ssd.make_scan_problem(T, S, d, self.STATES, 1, self.slots, BF, F32)
        y = new(T, d)
        ssd.selective_scan_varlen(p, xs, dt, self.A1, B, C, self.D1, r[:, d:], self.tf1, cu, self.scan_s,
                                  idx, has, y, ssd.alloc_scan_workspace(p, dev))
        x = x + y @ self.out1
        # attention: the new rows join the cache, a continued prompt reads its own back
        q, k, v = self._split_qkv(x)
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
        return x + o.view(T, -1) @ self.out_a

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
        r = self._norm(x) @ self.in2
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
        x = x + (y.view(R * T, d) * torch.nn.functional.silu(r[:, :d])) @ self.out2
        r = self._norm(x) @ self.in1
        p1 = ssd.make_conv_problem(R * T, R, d, self.WIDTH, self.slots, BF, BF)
        xs, y, raw1 = new(R * T, d), new(R * T, d), r[:, :d]
        ssd.causal_conv1d_update(p1, raw1, self.conv1_w, self.conv1_b, self.conv1_s, idx, xs,
                                 update_cache=False)
        dt, B, C = self._dt_b_c(xs)
        ps = ssd.make_scan_problem(R * T, R, d, self.STATES, 1, self.slots, BF, F32)
        st1 = new(R * T, d, self.STATES, dtype=F32)
        ssd.selective_scan_update(ps, xs, dt, self.A1, B, C, self.D1, r[:, d:], self.tf1, self.scan_s,
                                  idx, y, st1)
        x = x + y @ self.out1
        q, k, v = self._split_qkv(x)
        ssd.kv_cache_store(self.kv, k, v, self._positions(slots, [T] * R), **self.cache)
        pd = ssd.make_attn_decode_problem(self.kv, R, T, self.q_heads, self.pages.shape[1])
        o = new(R, T, self.q_heads, self.KV_DIM)
        lens = torch.tensor([int(self.lens[s]) + T for s in slots], dtype=torch.int32, device=dev)
        ssd.attention_decode(pd, q.reshape(o.shape), self.cache["k_cache"], self.cache["v_cache"],
                             self.cache["k_scale"], self.cache["v_scale"],
                             self.pages[idx.long()].contiguous(), lens, o,
                             workspace=ssd.alloc_attn_decode_workspace(pd, dev))
        self._pending = (slots, T, p2, raw2, up, st2, p1, raw1, st1, idx)
        return x + o.view(R * T, -1) @ self.out_a

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


def check(hidden=256, lens=(70, 1, 133), steps=3, tokens=3, seed=0):
    """A prompt in two parts and verify steps with rejected drafts, against one pass over all the
    tokens that counted: the largest difference relative to the result's norm, per sequence."""
    dev, S = "cuda", len(lens)
    g = torch.Generator(dev).manual_seed(seed + 1)
    accepted = [[(i + k) % tokens for i in range(S)] for k in range(steps)]
    total = [n + sum(1 + accepted[k][i] for k in range(steps)) for i, n in enumerate(lens)]
    xs = [torch.randn(n, hidden, generator=g, device=dev).to(BF) for n in total]
    whole = Stack(hidden, S, max(total) + tokens, dev, seed)
    want = whole.prompt(torch.cat(xs), list(range(S)), total).split(total)
    st = Stack(hidden, S, max(total) + tokens, dev, seed)
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
          ["%.1e" % e for e in check()])
    st = Stack(a.hidden, a.seqs, a.tokens + 64)
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

    print("prompt, %d sequences, %d tokens: %.2f ms" % (a.seqs, sum(per), timed(fresh)))
    print("verify step, 3 tokens each: %.2f ms" % timed(lambda: st.verify(y, list(range(a.seqs)), 3)))


if __name__ == "__main__":
    main()
