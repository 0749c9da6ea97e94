"""Refusals and flags of the calls around the layer that need a GPU to be seen."""
import pytest
import torch

import any_precision_expert_gb300 as pw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream,error", [("no stream", AttributeError), (1 << 70, OverflowError),
                                          (type("S", (), {"cuda_stream": "x"})(), TypeError)])
def test_an_argument_that_is_no_stream_enqueues_nothing(stream, error):
    q = torch.ones(3, 4, 64, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 7.0)
    with pytest.raises(error):
        pw.qk_norm_rope(pw.Rotary(None), q, None, None, out, None, stream=stream)
    torch.cuda.synchronize()
    assert (out == 7.0).all()


def verify(B, K, V, n_draft, tokens, refused):
    """Flat distributions; the drafts at places in `refused` are refused by their uniform numbers."""
    p, q = (torch.full((B, k, V), 1.0 / V, device="cuda") for k in (K + 1, K))
    u = torch.zeros(B, K, device="cuda")
    for b, i in refused:
        u[b, i] = 2.0
    out, acc = torch.empty(B, K + 1, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pw.verify_draft(p, q, tokens.cuda(), torch.tensor(n_draft, dtype=torch.int32, device="cuda"), u,
                    torch.ones(B, V, device="cuda"), out, acc, err=err)
    return out.tolist(), acc.tolist(), err.item()


@pytest.mark.parametrize("K,at,bad", [(3, 1, 50), (3, 2, -1), (40, 35, 50), (64, 63, -7), (64, 1, 2 ** 31 - 1)])
def test_verify_flags_a_bad_token_behind_a_refusal(K, at, bad):
    tokens = torch.full((2, K), 5, dtype=torch.int32)
    out, acc, err = verify(2, K, 50, [K, K], tokens, [(0, 0), (1, 0)])
    assert acc == [0, 0] and err == 0
    tokens[1, at] = bad
    again, acc, err = verify(2, K, 50, [K, K], tokens, [(0, 0), (1, 0)])
    assert again == out and acc == [0, 0] and err != 0
    # past the sequence's count it is padding
    again, acc, err = verify(2, K, 50, [K, at], tokens, [(0, 0), (1, 0)])
    assert again == out and acc == [0, 0] and err == 0


@pytest.mark.parametrize("K", [1, 33, 64])
def test_verify_keeps_up_to_the_first_refusal_in_any_block_of_drafts(K):
    tokens = torch.arange(K, dtype=torch.int32)[None].expand(3, K).contiguous()
    last = K - 1
    out, acc, err = verify(3, K, 100, [K, K, last], tokens, [(0, last)])
    assert acc == [last, K, last] and err == 0
    want = tokens[0].tolist()
    assert [r[:a] for r, a in zip(out, acc)] == [want[:a] for a in acc]
    assert all(r[a + 1:] == [-1] * (K - a) for r, a in zip(out, acc))
    # two refusals: the first one ends them
    assert verify(1, K, 100, [K], tokens[:1], [(0, last), (0, last // 2)])[1] == [last // 2]


def test_verify_ties_an_empty_distribution_and_infinite_quotients_each_by_itself():
    V, K = 5000, 2
    p, q = torch.full((3, K + 1, V), 1.0 / V, device="cuda"), torch.full((3, K, V), 1.0 / V, device="cuda")
    u, e = torch.full((3, K), 2.0, device="cuda"), torch.ones(3, V, device="cuda")
    p[0] = 0
    for i in (4999, 1234, 77):
        p[0, :, i] = 0.25               # equal quotients: the lowest index
    q[0] = 0.5                          # more than the target anywhere: no residual, so from the target itself
    p[1] = 0                            # nothing at all: index 0
    e[2, 3:6] = 0.0                     # infinite quotients: the first of them
    tokens = torch.full((3, K), 9, dtype=torch.int32, device="cuda")
    n = torch.tensor([K, K, 0], dtype=torch.int32, device="cuda")
    out, acc = torch.empty(3, K + 1, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    pw.verify_draft(p, q, tokens, n, u, e, out, acc)
    assert acc.tolist() == [0, 0, 0]
    assert out[0].tolist() == [77, -1, -1]
    assert out[1].tolist() == [0, -1, -1]
    assert out[2].tolist() == [3, -1, -1]
