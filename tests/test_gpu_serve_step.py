"""The calls around the layer and the layer itself in one decode step with drafts (examples/speculative_step.py), each
stage held to the fp64 oracle on the stage's own inputs."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import pw_oracle as O
from oracle import pw_serve as S

from gpu_layers import assert_close

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples", "speculative_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def host(t):
    return t.double().cpu().numpy()


def test_decode_steps_match_the_oracle_stage_by_stage():
    ex = _example()
    b = ex.Block(batch=3, drafts=3, seed=1)
    try:
        b.prompt(torch.arange(70, device="cuda") * 13 % ex.VOCAB)
        last = torch.tensor([3, 500, 999], device="cuda")
        total = 0
        for _ in range(4):
            k0 = host(b.kv.k)
            r = b.step(last)
            torch.cuda.synchronize()
            cs, qw, kw = (host(t) for t in b.rotary._keep)
            pos, slots = r["positions"].cpu().numpy(), r["slots"].cpu().numpy()
            # fp16 roundings of values up to about 5: half a unit is 2^-9; fp32 arithmetic in front of it
            q_ref = S.norm_rope(host(r["q"]), qw, 1e-6, cs, pos, False)
            assert np.abs(host(r["q_rot"]) - q_ref).max() <= 2.0 ** -11 * np.abs(q_ref).max() + 1e-4
            k_ref = S.append(k0, S.norm_rope(host(r["k"]), kw, 1e-6, cs, pos, False), slots)
            assert np.abs(host(b.kv.k) - k_ref).max() <= 2.0 ** -11 * np.abs(k_ref).max() + 1e-4
            att = S.attend(host(r["q_rot"]), host(b.kv.k), host(b.kv.v), b.table.cpu().numpy(), r["lens"].cpu().numpy(),
                           b.K + 1, ex.D ** -0.5, b.prefix_table.cpu().numpy(), b.prefix_lens.cpu().numpy())[0]
            assert_close(host(r["att"]), att, what="attention")
            x1 = r["x1"].cpu().numpy()
            ref = O.moe_layer(x1, b.router_w, b.router_b, b.experts, b.bits, b.cfg.K, b.cfg.renormalize,
                              idx_override=b.buf.idx[:x1.shape[0]].cpu().numpy())
            assert_close(r["y"].float().cpu().numpy(), ref["y"], what="MoE layer")
            out, acc = S.verify(*(r[n].cpu().numpy() for n in ("p", "q_p", "drafted", "n_draft", "u", "noise")))
            assert np.array_equal(r["out"].cpu().numpy(), out) and np.array_equal(r["accepted"].cpu().numpy(), acc)
            assert torch.equal(b.lens, r["before"] + r["accepted"] + 1)
            total += int(acc.sum())
            last = r["next"]
        assert b.kv.check_device() == 0 and b.layer.check_device() == 0
        assert 0 < total < 4 * 3 * 3  # some drafts kept, some refused
    finally:
        b.close()
