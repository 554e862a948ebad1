"""Beam search through one attention layer whose keys and values lie in 4 bits,
from the library's calls.

    python examples/beam_search.py

P virtual ranks split the heads and the vocabulary's columns.  The weights are
random; what is shown is how the calls fit together:

  prompts  kv_plan -> tp_qk_norm_rope -> tp_attention, tp_kv4_write -> logits of
           the last tokens -> beam_select (one beam becomes W) -> kv_fork
  step     kv_copy_pages -> kv_plan -> tp_qk_norm_rope -> tp_kv4_write ->
           tp_attention_decode_kv4 -> logits -> beam_select -> kv_fork
  now and  kv_compact -> kv_copy_pages: the pages in use at the front of the
  then     cache
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ring_collectives_amd import attention as A                   # noqa: E402
from ring_collectives_amd import collectives as rc                # noqa: E402
from ring_collectives_amd import search as S                      # noqa: E402

BF = torch.bfloat16


def i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


class BeamSearch:
    """A layer's weights over P ranks, its 4-bit cache and the state of a search."""

    def __init__(self, P=2, model=256, vocab=1000, Hq=4, Hkv=2, D=64, pages=128, page=16, positions=1024, end=7, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")     # noqa: E731
        self.P, self.model, self.vocab, self.Hq, self.Hkv, self.D = P, model, vocab, Hq, Hkv, D
        self.pages, self.page, self.end = pages, page, end
        self.width = -(-vocab // (128 * P)) * 128                        # a rank's columns, padded
        self.embed = rnd(vocab, model).to(BF)
        self.wqkv = [(rnd(model, (Hq + 2 * Hkv) * D) * model ** -0.5).to(BF) for _ in range(P)]
        self.wo = [(rnd(Hq * D, model) * (P * Hq * D) ** -0.5).to(BF) for _ in range(P)]
        self.wvocab = [(rnd(model, self.width) * 2 * model ** -0.5).to(BF) for _ in range(P)]
        f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
        self.cache = [S.kv4_cache(pages, Hkv, D, page) for _ in range(P)]
        self.free = torch.randperm(pages, generator=g, device="cuda").int()
        self.used = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = {}                                                     # a workspace for each call

    def plan(self, new_tokens, capacity):
        """Pages and cache slots of the tokens that each row adds."""
        B = self.lengths.numel()
        after, cu, pos, used = i32(B), i32(B + 1), i32(capacity), i32(1)
        slots = torch.empty(capacity, dtype=torch.int64, device="cuda")
        A.kv_plan(self.lengths, new_tokens, self.free, self.used, self.table, after, cu, pos, slots, used, page_size=self.page)
        self.lengths, self.used = after, used
        return cu, pos, slots

    def project(self, x, pos):
        """Rotated queries and keys, and values, of token rows x (T, model)."""
        T = x.shape[0]
        e = lambda H: [torch.empty(T, H, self.D, dtype=BF, device="cuda") for _ in range(self.P)]     # noqa: E731
        q, k, v = e(self.Hq), e(self.Hkv), e(self.Hkv)
        A.tp_qk_norm_rope([(x @ w).float() for w in self.wqkv], None, None, self.cos_sin, pos, q, k, v)
        return q, k, v

    def logits(self, x, o):
        """Each rank's columns of the logits, from the residual stream after the layer."""
        part = [o[r].reshape(x.shape[0], -1).float() @ self.wo[r].float() for r in range(self.P)]
        out = [torch.empty_like(t) for t in part]
        rc.all_reduce(part, out)
        return [(x.float() + out[r]) @ self.wvocab[r].float() for r in range(self.P)]

    def choose(self, logits, beams):
        """The next beams of every group, and the table, pages and lengths that go with them."""
        N = self.scores.shape[0]
        K = beams
        parents, tokens, scores = i32(N, K), i32(N, K), torch.empty(N, K, device="cuda")
        done = torch.empty(N, K, dtype=torch.bool, device="cuda")
        self.ws["select", self.scores.shape[1]] = S.beam_select(
            logits, self.scores, parents, tokens, scores, vocab=self.vocab, done=self.done, done_after=done, end_token=self.end,
            ws=self.ws.get(("select", self.scores.shape[1])))
        rows, width = N * K, self.table.shape[1]
        table, lengths, copies, n, used = i32(rows, width), i32(rows), i32(rows, 2), i32(1), i32(1)
        self.shared = i32(N)
        self.ws["fork"] = S.kv_fork(self.table, self.lengths, parents, self.free, self.used, table, lengths, copies, n, used,
                                    page_size=self.page, pages=self.pages, shared=self.shared, group=K, ws=self.ws.get("fork"))
        S.kv_copy_pages(self.cache, copies, n, pages=self.pages)
        self.table, self.lengths, self.used, self.scores, self.done = table, lengths, used, scores, done
        self.history.append((parents, tokens))
        return tokens.view(-1)

    def prompts(self, tokens, lens, beams, room):
        """Runs prompts (packed tokens, their lengths) and makes `beams` of each; room: pages of a row."""
        B, T = len(lens), sum(lens)
        self.table = torch.full((B, room), -1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.scores, self.done = torch.zeros(B, 1, device="cuda"), torch.zeros(B, 1, dtype=torch.bool, device="cuda")
        self.beams, self.history = beams, []
        cu, pos, slots = self.plan(torch.tensor(lens, dtype=torch.int32, device="cuda"), T)
        x = self.embed[tokens]
        q, k, v = self.project(x, pos)
        o = [torch.empty_like(t) for t in q]
        A.tp_attention(q, k, v, o, cu, cu)
        S.tp_kv4_write(k, v, self.cache, slots, page_size=self.page)
        last = cu[1:].long() - 1
        return self.choose(self.logits(x[last], [t[last] for t in o]), beams)

    def step(self, tokens, share=True):
        """One more token on every beam; share: read what a group's beams have in common once."""
        B = tokens.numel()
        _, pos, slots = self.plan(torch.ones(B, dtype=torch.int32, device="cuda"), B)
        x = self.embed[tokens.long()]
        q, k, v = self.project(x, pos)
        S.tp_kv4_write(k, v, self.cache, slots, page_size=self.page)
        o = [torch.empty_like(t) for t in q]
        self.ws["decode"] = S.tp_attention_decode_kv4(q, self.cache, o, self.table, self.lengths, page_size=self.page,
                                                      shared=self.shared if share else None, group=self.beams, ws=self.ws.get("decode"))
        return self.choose(self.logits(x, o), self.beams)

    def compact(self):
        """The pages in use at the front of the cache; returns how many there are (on the GPU)."""
        table, copies, n, used = torch.empty_like(self.table), i32(self.pages // 2, 2), i32(1), i32(1)
        self.ws["compact"] = S.kv_compact(self.table, self.lengths, table, self.free, copies, n, used, page_size=self.page,
                                          ws=self.ws.get("compact"))
        S.kv_copy_pages(self.cache, copies, n, pages=self.pages)
        self.table, self.used = table, used
        return used

    def results(self):
        """Every beam's tokens since its prompt, best first: [groups][beams] lists, and their scores."""
        N, K = self.scores.shape
        out = []
        for row in range(N * K):
            seq, at = [], row
            for parents, tokens in reversed(self.history):
                seq.append(int(tokens.view(-1)[at]))
                at = int(parents.view(-1)[at])
            out.append(seq[::-1])
        return [out[n * K:(n + 1) * K] for n in range(N)], self.scores.tolist()


def search(lens=(40, 17, 90), beams=4, steps=12, compact_every=0, share=True, seed=0):
    s = BeamSearch(seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    prompt = torch.randint(0, s.vocab, (sum(lens),), generator=g, device="cuda")
    tokens = s.prompts(prompt, list(lens), beams, room=-(-(max(lens) + steps + 1) // s.page))
    for i in range(steps):
        if compact_every and i % compact_every == 0:
            s.compact()
        tokens = s.step(tokens, share)
    return s


def main():
    torch.cuda.set_device(0)
    s = search(compact_every=4)
    n = s.compact()
    beams, scores = s.results()
    for seqs, sc in zip(beams, scores):
        print("prompt's beams:")
        for seq, x in zip(seqs, sc):
            print("  %8.3f  %s" % (x, seq))
    print("%d of %d pages in use, shared tokens %s of %s" % (n.item(), s.pages, s.shared.tolist(), s.lengths.view(-1, 4)[:, 0].tolist()))


if __name__ == "__main__":
    main()
