"""Drafted tokens verified by one MoE block: the calls around the layer together.

A block of the "tiny" layer configuration (hidden size 512: 8 query heads of 64 on 2 key heads) serves a few sequences
behind one shared prompt.  Every step drafts K tokens a sequence, runs the K + 1 positions through

    projections -> KvCache.append (head norms, rotation, paged append) -> KvCache.attend (shared prefix + own suffix)
    -> projection -> the bit-plane MoE layer (moe_forward_fused) -> token probabilities -> verify_draft

and keeps the verified tokens; the cache rolls back by lengths alone.  Weights are random: the run shows the calls, not a
language.

    python examples/speculative_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import any_precision_expert_gb300 as pw  # noqa: E402
from synth import bits_plan, get_config, make_expert, make_router  # noqa: E402

HQ, HKV, D, PAGE, VOCAB, MAX_POS = 8, 2, 64, 16, 1000, 512
BATCH, DRAFTS, PROMPT = 4, 3, 100
MOST_STEPS = (MAX_POS - PROMPT) // (DRAFTS + 1)  # that the rotation table and the pages hold, every draft kept


class Block:
    """Attention over a paged cache, then the MoE layer."""

    def __init__(self, batch: int, drafts: int, seed: int = 0):
        self.cfg, self.seed, self.B, self.K = get_config("tiny"), seed, batch, drafts
        d = self.cfg.d
        self.bits = bits_plan(self.cfg, seed)
        self.pool = pw.Pool(256 << 20)
        self.layer = pw.Layer(self.pool, d, self.cfg.f, self.cfg.E, self.cfg.K, self.cfg.renormalize)
        self.experts = [make_expert(self.cfg, e, seed, with_w16=True) for e in range(self.cfg.E)]
        for e, ex in enumerate(self.experts):
            self.layer.load_expert(e, 16, ex["code6"], ex["lut"], ex["w16"])
            self.layer.set_expert_bitwidth(e, int(self.bits[e]))
        self.router_w, self.router_b = make_router(self.cfg, seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).half()
        self.gen = gen
        self.embed = rand(VOCAB, d, scale=1.0)
        self.w_qkv = rand(d, (HQ + 2 * HKV) * D, scale=d ** -0.5)
        self.w_o = rand(HQ * D, d, scale=(HQ * D) ** -0.5)
        self.w_head = rand(d, d, scale=d ** -0.5)
        self.wr = torch.from_numpy(self.router_w).cuda()
        self.bias = None if self.router_b is None else torch.from_numpy(self.router_b).cuda()
        inv = 10000.0 ** (-torch.arange(D // 2, device="cuda") * 2 / D)
        ang = torch.arange(MAX_POS, device="cuda")[:, None] * inv
        self.rotary = pw.Rotary(torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(),
                                q_weight=1 + rand(D, scale=0.1), k_weight=1 + rand(D, scale=0.1))
        # pages: the shared prompt's, then a fixed run for every sequence
        own = MAX_POS // PAGE
        pages = own * (batch + 1)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        self.prefix_table, self.table = order[:own][None].contiguous(), order[own:].view(batch, own).contiguous()
        k = torch.zeros(pages, HKV, PAGE, D, dtype=torch.float16, device="cuda")
        self.kv = pw.KvCache(k, torch.zeros_like(k), n_heads=HQ)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.prefix_lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.buf = pw.Buffers(self.layer, batch * (drafts + 1))
        self.ws = torch.empty(self.kv.attend_workspace_size(batch, drafts + 1, 1), dtype=torch.uint8, device="cuda")

    def _heads(self, x):
        qkv = x @ self.w_qkv
        T = x.shape[0]
        return (qkv[:, :HQ * D].view(T, HQ, D), qkv[:, HQ * D:(HQ + HKV) * D].view(T, HKV, D),
                qkv[:, (HQ + HKV) * D:].view(T, HKV, D))

    def prompt(self, tokens):
        """Put the shared prompt's keys and values (of this one block) into the prefix pages."""
        t = torch.arange(len(tokens), device="cuda")
        _, k, v = self._heads(self.embed[tokens])
        slots = self.prefix_table[0, t // PAGE] * PAGE + t % PAGE
        self.kv.append(k, v, slots.to(torch.int32), rotary=self.rotary, positions=t.to(torch.int32))
        self.prefix_lens.fill_(len(tokens))

    def draft(self, last):
        """K tokens after `last` [B] from the output head alone, without the block: tokens [B, K], distributions [B, K, V]."""
        toks, probs = [], []
        for _ in range(self.K):
            p = torch.softmax((self.embed[last.long()] @ self.w_head @ self.embed.T).float() / 16, -1)
            e = torch.empty_like(p).exponential_(generator=self.gen)
            last = (p / e).argmax(-1)
            toks.append(last)
            probs.append(p)
        return torch.stack(toks, 1).to(torch.int32), torch.stack(probs, 1).contiguous()

    def step(self, last):
        """One decode step after the tokens `last` [B]; every intermediate, for checks."""
        B, K = self.B, self.K
        drafted, q_p = self.draft(last)
        tokens = torch.cat([last[:, None].to(torch.int32), drafted], 1)      # [B, K + 1]
        x = self.embed[tokens.view(-1).long()]
        q, k, v = self._heads(x)
        at = self.lens[:, None].long() + torch.arange(K + 1, device="cuda")  # places in the suffixes
        positions = (at + self.prefix_lens.long()).view(-1).to(torch.int32)
        slots = (self.table.gather(1, at // PAGE) * PAGE + at % PAGE).view(-1).to(torch.int32)
        q_rot = torch.empty(B * (K + 1), HQ, D, dtype=torch.float16, device="cuda")
        self.kv.append(k, v, slots, rotary=self.rotary, positions=positions, q=q, q_out=q_rot)
        lens = self.lens + (K + 1)
        att = torch.empty_like(q_rot)
        self.kv.attend(q_rot, self.table, lens, att, self.ws, q_len=K + 1, prefix_table=self.prefix_table,
                       prefix_lens=self.prefix_lens)
        x1 = x + att.view(-1, HQ * D) @ self.w_o
        y = pw.moe_forward_fused(self.layer, x1, self.wr, self.bias, self.buf)
        x2 = x1 + y
        p = torch.softmax((x2 @ self.w_head @ self.embed.T).float() / 16, -1).view(B, K + 1, VOCAB).contiguous()
        u = torch.rand(B, K, generator=self.gen, device="cuda")
        noise = torch.empty(B, VOCAB, device="cuda").exponential_(generator=self.gen)
        out = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
        accepted = torch.empty(B, dtype=torch.int32, device="cuda")
        n_draft = torch.full((B,), K, dtype=torch.int32, device="cuda")
        pw.verify_draft(p, q_p, drafted, n_draft, u, noise, out, accepted)
        before, self.lens = self.lens, self.lens + accepted + 1              # the refused drafts' slots are free again
        return dict(tokens=tokens, q=q, k=k, v=v, q_rot=q_rot, positions=positions, slots=slots, att=att, lens=lens,
                    before=before, x1=x1, y=y, p=p, q_p=q_p, drafted=drafted, n_draft=n_draft, u=u, noise=noise, out=out,
                    accepted=accepted, next=out.gather(1, accepted[:, None].long())[:, 0])

    def close(self):
        self.kv.close()
        self.layer.destroy()
        self.pool.close()


def main(steps: int = 8):
    if not 0 <= steps <= MOST_STEPS:
        raise SystemExit(f"0 to {MOST_STEPS} steps: {MAX_POS} positions hold the prompt's {PROMPT} and {DRAFTS + 1} a step")
    block = Block(batch=BATCH, drafts=DRAFTS)
    try:
        block.prompt(torch.randint(0, VOCAB, (PROMPT,), generator=block.gen, device="cuda"))
        last = torch.randint(0, VOCAB, (BATCH,), generator=block.gen, device="cuda")
        for i in range(steps):
            r = block.step(last)
            last = r["next"]
            print(f"step {i}: accepted {r['accepted'].tolist()} of {block.K}, lengths {block.lens.tolist()}, "
                  f"next {last.tolist()}")
        assert block.kv.check_device() == 0 and block.layer.check_device() == 0
    finally:
        block.close()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
