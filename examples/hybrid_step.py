#!/usr/bin/env python3
"""A hybrid model's token mixing through prompt, speculative verify and decode.

Three gated delta-rule layers (ReplayStore) and one softmax-attention layer
(KVCache) with random weights, as a serving loop runs them: prompts of different
lengths, windows of draft tokens of which some are rejected, a request forked in
two, and single tokens in one CUDA graph. Run it to see the same tokens give the
same hidden states whichever way they come:

    python examples/hybrid_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_state_rssm_gb300.store import KVCache, ReplayStore, RotaryTable  # noqa: E402

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


class HybridStack:
    """`layers` delta-rule layers, then one attention layer; pre-norm, residual."""

    def __init__(self, width=256, layers=3, n_slots=4, dtype="f32", tokens=512, seed=0,
                 HK=2, HV=4, dk=64, HQ=4, HKV=2, D=64, max_T=4):
        gen = torch.Generator("cuda").manual_seed(seed)
        t = DTYPE[dtype]

        def weight(n, m):
            return (torch.randn(n, m, device="cuda", generator=gen) * n ** -0.5).to(t)

        self.width, self.layers, self.t = width, layers, t
        self.HK, self.HV, self.dk, self.HQ, self.HKV, self.D = HK, HV, dk, HQ, HKV, D
        self.gdn_in = [weight(width, (2 * HK + HV) * dk + 2 * HV) for _ in range(layers)]
        self.gdn_out = [weight(HV * dk, width) for _ in range(layers)]
        self.attn_in, self.attn_out = weight(width, (HQ + 2 * HKV) * D), weight(HQ * D, width)
        self.state = ReplayStore("gdn", layers, n_slots, HK, HV, dk, dk, L=8, max_T=max_T,
                                 in_dtype=dtype, state_dtype="f32")
        page = 16
        self.cache = KVCache(1, n_slots, HQ, HKV, D, n_pages=n_slots * tokens // page,
                             page_size=page, max_pages=tokens // page, dtype=dtype)
        self.rope = RotaryTable.from_base(tokens, D // 2, 1e4)

    def _norm(self, x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(self.t)

    def _gdn(self, i, x, call):
        N, HK, HV, dk = x.shape[0], self.HK, self.HV, self.dk
        y = self._norm(x) @ self.gdn_in[i]
        q, k, v, b, g = y.split((HK * dk, HK * dk, HV * dk, HV, HV), -1)

        def unit(z):
            return torch.nn.functional.normalize(z.float().view(N, HK, dk), dim=-1).to(self.t)

        o = torch.empty(N, HV, dk, dtype=self.t, device="cuda")
        call(i, unit(q), unit(k), v.reshape(N, HV, dk).contiguous(), torch.sigmoid(b.float()),
             -torch.nn.functional.softplus(g.float()), o)
        return x + o.view(N, -1) @ self.gdn_out[i]

    def _attention(self, x, append, attend):
        N = x.shape[0]
        y = (self._norm(x) @ self.attn_in).view(N, self.HQ + 2 * self.HKV, self.D)
        q, k, v = y.split((self.HQ, self.HKV, self.HKV), 1)  # views: tokens are strided
        turned = torch.empty(N, self.HQ, self.D, dtype=self.t, device="cuda")
        append(q, k, v, turned)
        o = torch.empty_like(turned)
        attend(turned, k, v, o)
        return x + o.view(N, -1) @ self.attn_out

    def prompt(self, x, slot, cu):
        """Prompts of empty slots, packed: rows [cu[r], cu[r + 1]) of x belong to slot[r]."""
        S, C = self.state, self.cache
        C.rssm_kv_reserve(slot, cu_seqlens=cu)
        for i in range(self.layers):
            x = self._gdn(i, x, lambda l, q, k, v, b, g, o: S.rssm_prefill(
                l, q, k, v, b, g, cu, slot, o, reset_cursor=l == self.layers - 1))
        keys = torch.empty(x.shape[0], self.HKV, self.D, dtype=self.t, device="cuda")

        def append(q, k, v, turned):  # the prompt's own attention reads the keys in a row
            C.rssm_kv_append(0, q, k, v, slot, q_out=turned, rope=self.rope, cu_seqlens=cu,
                             k_out=keys)

        x = self._attention(x, append, lambda q, k, v, o: C.rssm_attn_prefill(
            q, keys, v, cu, slot, o))
        C.rssm_kv_commit(slot, cu_seqlens=cu)
        return x

    def window(self, x, slot, T):
        """T tokens of each row (T = 1: decode); commit says how many stand."""
        S, C = self.state, self.cache
        C.rssm_kv_reserve(slot, T)
        for i in range(self.layers):
            x = self._gdn(i, x, (lambda l, q, k, v, b, g, o: S.rssm_decode(
                l, q, k, v, b, g, slot, o, advance_cursor=l == self.layers - 1)) if T == 1
                else (lambda l, q, k, v, b, g, o: S.rssm_verify(l, q, k, v, b, g, slot, T, o)))
        return self._attention(
            x, lambda q, k, v, turned: C.rssm_kv_append(0, q, k, v, slot, T, turned, rope=self.rope),
            lambda q, k, v, o: C.rssm_attn_decode(0, q, slot, T, o))

    def commit(self, slot, T, accept=None):
        if T > 1:
            self.state.rssm_commit(slot, accept, T)
        self.cache.rssm_kv_commit(slot, T, accept_len=accept)

    def fork(self, src, dst):
        """Slots dst continue slots src: pages are shared, the recurrent state is copied."""
        self.state.rssm_fold(src)  # the whole state stands in the checkpoint
        self.state.state[:, dst.long()] = self.state.state[:, src.long()]
        self.state.rssm_reset_slots(dst)
        self.cache.rssm_kv_fork(src, dst)


def run(dtype="f32", verbose=False):
    """Largest relative difference between tokens that came as one prompt and the same
    tokens that came as prompt, draft windows, forked requests and single tokens."""
    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    model = HybridStack(dtype=dtype)
    gen = torch.Generator("cuda").manual_seed(1)
    lens, total = (37, 90), 24
    tokens = [torch.randn(n + total, model.width, device="cuda", generator=gen).to(model.t)
              for n in lens]
    whole = model.prompt(torch.cat(tokens), ints(0, 1), ints(0, lens[0] + total,
                                                             lens[0] + lens[1] + 2 * total))
    want = list(whole.split([n + total for n in lens]))
    model.state.state.zero_()
    model.state.rssm_reset_slots(ints(0, 1))
    model.cache.rssm_kv_release(ints(0, 1))

    got = [[], []]
    slot = ints(0, 1)
    out = model.prompt(torch.cat([x[:n] for x, n in zip(tokens, lens)]), slot,
                       ints(0, lens[0], sum(lens)))
    for r, o in enumerate(out.split(lens)):
        got[r].append(o)
    at = list(lens)
    for accept in ((4, 2), (0, 3), (3, 4), (1, 1)):       # verify windows of four drafts
        drafts = []
        for r in range(2):
            x = tokens[r][at[r]:at[r] + 4].clone()
            x[accept[r]:] = torch.nan                      # what is rejected must not matter
            drafts.append(x)
        out = model.window(torch.cat(drafts), slot, 4)
        model.commit(slot, 4, ints(*accept))
        for r in range(2):
            got[r].append(out[4 * r:4 * r + accept[r]])
            at[r] += accept[r]
    model.fork(ints(1), ints(2))                           # request 1 goes on in two slots
    slot = ints(0, 1, 2)
    x = torch.zeros(3, model.width, dtype=model.t, device="cuda")
    y = torch.empty_like(x)

    def step():
        y.copy_(model.window(x, slot, 1))
        model.commit(slot, 1)

    def load(i):
        for r, s in enumerate((0, 1, 1)):
            x[r] = tokens[s][at[s] + i]

    side = torch.cuda.Stream()                             # one step outside: libraries warm up
    load(0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = [first]
    for i in range(1, 8):
        load(i)
        graph.replay()
        outs.append(y.clone())
    worst = 0.0
    for r in range(2):
        have = torch.cat(got[r] + [o[r:r + 1] for o in outs]).float()
        ref = want[r][:len(have)].float()
        worst = max(worst, float((have - ref).abs().max() / ref.abs().max()))
    ref = want[1][at[1]:at[1] + 8].float()
    have = torch.cat([o[2:3] for o in outs]).float()       # the fork's own steps
    worst = max(worst, float((have - ref).abs().max() / ref.abs().max()))
    assert model.cache.rssm_kv_get_device_error() == 0
    assert model.state.rssm_get_device_error() == 0
    if verbose:
        print(f"{dtype}: prompt of {lens} tokens, drafts, a fork and {len(outs)} steps against one "
              f"prompt: largest difference {worst:.1e} of the largest value; pages in use "
              f"{int((model.cache.refs > 0).sum())}")
    return worst


if __name__ == "__main__":
    for d in ("f32", "bf16"):
        run(d, verbose=True)
