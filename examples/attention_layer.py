"""The attention half of a tensor-parallel layer, from the library's calls:
a prompt batch, decode steps behind it, and a training step.

    python examples/attention_layer.py

P virtual ranks split the heads; the tokens of a batch lie packed, sharded by
rows over the ranks, as in tp_mlp_layer.

  prompts  all_gather_gemm (x Wqkv) -> kv_plan -> tp_qk_norm_rope (to q, k, v
           and the paged cache) -> tp_attention -> gemm_reduce_scatter (o Wo)
  step     one token per request: kv_plan -> tp_qk_norm_rope (to q and the
           cache) -> tp_attention_decode -> ring all-reduce of the ranks' o Wo
  train    tp_attention and tp_attention_grad, tp_qk_norm_rope_grad, and the
           ring all-reduce of the gains' gradients
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ring_collectives_amd import attention as A                   # noqa: E402
from ring_collectives_amd import collectives as rc                # noqa: E402

BF = torch.bfloat16


class AttentionLayer:
    """Weights of one layer over P ranks, its cos/sin table and its cache."""

    def __init__(self, P=4, model=1024, Hq=2, Hkv=1, D=128, pages=256, page=16, positions=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")     # noqa: E731
        self.P, self.model, self.Hq, self.Hkv, self.D, self.page = P, model, Hq, Hkv, D, page
        self.wqkv = [(rnd(model, (Hq + 2 * Hkv) * D) * model ** -0.5).to(BF) for _ in range(P)]
        self.wo = [(rnd(Hq * D, model) * (P * Hq * D) ** -0.5).to(BF) for _ in range(P)]
        gq, gk = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)          # the same on every rank
        self.gain_q, self.gain_k = [gq.clone() for _ in range(P)], [gk.clone() for _ in range(P)]
        f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
        self.k_cache, self.v_cache = ([torch.zeros(pages * page, Hkv, D, dtype=BF, device="cuda") for _ in range(P)]
                                      for _ in range(2))
        self.free = torch.randperm(pages, generator=g, device="cuda").int()
        self.used = torch.zeros(1, dtype=torch.int32, device="cuda")

    def requests(self, B, longest):
        """Empty block table and lengths of B requests of up to `longest` tokens."""
        self.table = torch.full((B, -(-longest // self.page)), -1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(B, dtype=torch.int32, device="cuda")

    def plan(self, new_tokens, capacity):
        """kv_plan for the tokens each request adds; (cu, positions, slots)."""
        B = self.lengths.numel()
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")     # noqa: E731
        after, cu, pos, used = i32(B), i32(B + 1), i32(capacity), i32(1)
        slots = torch.empty(capacity, dtype=torch.int64, device="cuda")
        A.kv_plan(self.lengths, new_tokens, self.free, self.used, self.table, after, cu, pos, slots, used, page_size=self.page)
        self.lengths, self.used = after, used
        return cu, pos, slots

    def heads(self, T, kv=True):
        e = lambda H: [torch.empty(T, H, self.D, dtype=BF, device="cuda") for _ in range(self.P)]     # noqa: E731
        return e(self.Hq), e(self.Hkv) if kv else None, e(self.Hkv) if kv else None

    def prompts(self, x_shard, new_tokens):
        """The layer's output shards (fp32) of a packed prompt batch: M rows in
        all, a multiple of 256 P; new_tokens: each prompt's tokens, M in all."""
        P, M = self.P, x_shard[0].shape[0] * self.P
        width = (self.Hq + 2 * self.Hkv) * self.D
        full = [torch.empty(M, self.model, dtype=BF, device="cuda") for _ in range(P)]
        qkv = [torch.empty(M, width, device="cuda") for _ in range(P)]
        rc.all_gather_gemm(x_shard, self.wqkv, full, qkv)
        cu, pos, slots = self.plan(new_tokens, M)
        q, k, v = self.heads(M)
        A.tp_qk_norm_rope(qkv, self.gain_q, self.gain_k, self.cos_sin, pos, q, k, v, self.k_cache, self.v_cache, slots)
        o = self.heads(M, kv=False)[0]
        A.tp_attention(q, k, v, o, cu, cu)
        out = [torch.empty(M // P, self.model, device="cuda") for _ in range(P)]
        rc.gemm_reduce_scatter([t.view(M, -1) for t in o], self.wo, out)
        return out

    def step(self, x):
        """One token per request, x (B, model) on every rank: the output on
        every rank (fp32).  The projections of so few tokens are torch's; the
        fused products take multiples of 256."""
        B = x.shape[0]
        qkv = [(x @ w).float() for w in self.wqkv]
        _, pos, slots = self.plan(torch.ones(B, dtype=torch.int32, device="cuda"), B)
        q, _, _ = self.heads(B, kv=False)
        A.tp_qk_norm_rope(qkv, self.gain_q, self.gain_k, self.cos_sin, pos, q, None, None, self.k_cache, self.v_cache, slots)
        o = self.heads(B, kv=False)[0]
        A.tp_attention_decode(q, self.k_cache, self.v_cache, o, self.table, self.lengths, page_size=self.page)
        part = [o[r].view(B, -1).float() @ self.wo[r].float() for r in range(self.P)]
        out = [torch.empty_like(t) for t in part]
        rc.all_reduce(part, out)
        return out

    def train(self, qkv, pos, cu, do):
        """Gradients of sum(o do) to the projected rows and the gains, which
        are one set of weights kept by every rank: their gradients are summed
        over the ranks.  Returns (o, dqkv, dgain_q, dgain_k)."""
        P, T, D = self.P, qkv[0].shape[0], self.D
        q, k, v = self.heads(T)
        A.tp_qk_norm_rope(qkv, self.gain_q, self.gain_k, self.cos_sin, pos, q, k, v)
        o, dk, dv = self.heads(T)
        dq = self.heads(T, kv=False)[0]
        lse = [torch.empty(self.Hq, T, device="cuda") for _ in range(P)]
        A.tp_attention(q, k, v, o, cu, cu, lse=lse)
        A.tp_attention_grad(do, q, k, v, o, lse, dq, dk, dv, cu, cu)
        dqkv = [torch.empty_like(t) for t in qkv]
        dg = [torch.empty(2 * D, device="cuda") for _ in range(P)]           # both gains' gradients in one buffer per rank
        A.tp_qk_norm_rope_grad(dq, dk, dv, qkv, self.gain_q, self.gain_k, self.cos_sin, pos, dqkv,
                               [t[:D] for t in dg], [t[D:] for t in dg])
        total = [torch.empty_like(t) for t in dg]
        rc.all_reduce(dg, total)
        return o, dqkv, total[0][:D], total[0][D:]


def main():
    torch.cuda.set_device(0)
    layer = AttentionLayer()
    lens = [300, 17, 511, 196]                               # 1024 tokens, packed
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(lens), layer.model, generator=g, device="cuda").to(BF)
    layer.requests(len(lens), max(lens) + 8)
    out = layer.prompts(list(x.chunk(layer.P)), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    print("prompts of %s: output %s, mean square %.3f" % (lens, tuple(torch.cat(out).shape), torch.cat(out).square().mean()))
    for i in range(3):
        y = layer.step(torch.randn(len(lens), layer.model, generator=g, device="cuda").to(BF))
        print("step %d: lengths %s, mean square %.3f" % (i, layer.lengths.tolist(), y[0].square().mean()))
    T = 777
    qkv = [torch.randn(T, 4 * layer.D, generator=g, device="cuda") for _ in range(layer.P)]
    do = [torch.randn(T, layer.Hq, layer.D, generator=g, device="cuda").to(BF) for _ in range(layer.P)]
    cu = torch.tensor([0, 500, T], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(500), torch.arange(T - 500)]).int().cuda()
    _, d, gq, gk = layer.train(qkv, pos, cu, do)
    print("train on %d tokens: |dqkv| %.3f, |dgain_q| %.3f, |dgain_k| %.3f" % (
        T, torch.stack(d).norm(), gq.norm(), gk.norm()))


if __name__ == "__main__":
    main()
