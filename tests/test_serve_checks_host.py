"""What the Python calls around the layer refuse before anything is enqueued: whole calls of another type than the cache's,
arguments that only make sense together, memory that a kernel cannot use.  Runs without a GPU (host-simulated device, where
an accepted call answers PW_ERR_UNSUPPORTED)."""
import pytest
import torch

import any_precision_expert_gb300 as pw
from any_precision_expert_gb300._lib import lib

UNSUPPORTED = 2
F16, BF16 = torch.float16, torch.bfloat16
HQ, HK, D = 4, 2, 64


@pytest.fixture(autouse=True)
def sim():
    lib.pw_testing_host_sim(1)
    yield
    lib.pw_testing_host_sim(0)


def cache(dtype=F16):
    k = torch.zeros(4, HK, 16, D, dtype=dtype)
    return pw.KvCache(k, k.clone(), n_heads=HQ)


def ints(*shape, device="cpu"):
    return torch.zeros(*shape, dtype=torch.int32, device=device)


def workspace(c):
    ws = torch.empty(c.attend_workspace_size(3, 1, 1) + 256, dtype=torch.uint8)
    return ws[-ws.data_ptr() % 256:]


def append(c, dtype=F16, device="cpu", **kw):
    k, q = (torch.zeros(3, h, D, dtype=dtype, device=device) for h in (HK, HQ))
    a = {**dict(k=k, v=k.clone(), slots=ints(3, device=device), q=q, q_out=torch.empty_like(q)), **kw}
    c.append(**a)


def attend(c, dtype=F16, device="cpu", **kw):
    q = torch.zeros(3, HQ, D, dtype=dtype, device=device)
    a = {**dict(q=q, table=ints(3, 2, device=device), lens=ints(3, device=device), out=torch.empty_like(q), ws=workspace(c),
                prefix_table=ints(1, 2, device=device), prefix_lens=ints(1, device=device)), **kw}
    c.attend(**a)


def accepted(f, *a, **kw):
    with pytest.raises(pw.PwError) as e:
        f(*a, **kw)
    assert e.value.status == UNSUPPORTED


@pytest.mark.parametrize("of", [F16, BF16])
@pytest.mark.parametrize("call", [append, attend])
def test_calls_hold_the_caches_type(call, of):
    c = cache(of)
    accepted(call, c, of)
    for other in (F16, BF16, torch.float32, torch.uint8, torch.int16, torch.int64, torch.float64):
        if other != of:
            with pytest.raises(ValueError):
                call(c, other)


@pytest.mark.parametrize("name,heads", [("k", HK), ("v", HK), ("q", HQ), ("q_out", HQ)])
def test_append_one_argument_of_another_type(name, heads):
    with pytest.raises(ValueError):
        append(cache(), **{name: torch.zeros(3, heads, D, dtype=BF16)})


@pytest.mark.parametrize("name", ["q", "out"])
def test_attend_one_argument_of_another_type(name):
    with pytest.raises(ValueError):
        attend(cache(), **{name: torch.zeros(3, HQ, D, dtype=BF16)})


def test_append_norm_weights_have_the_caches_type():
    pos = ints(3)
    for dtype in (F16, BF16):
        r = pw.Rotary(torch.zeros(8, D), k_weight=torch.zeros(D, dtype=dtype))
        if dtype == F16:
            accepted(append, cache(F16), rotary=r, positions=pos)
        else:
            with pytest.raises(ValueError):
                append(cache(F16), rotary=r, positions=pos)


@pytest.mark.parametrize("call", [append, attend])
def test_calls_hold_the_caches_device(call):
    with pytest.raises(ValueError):
        call(cache(), device="meta")


@pytest.mark.parametrize("kw", [
    dict(prefix_lens=None), dict(prefix_table=None), dict(prefix_lens=None, group_offsets=ints(2)),
    dict(prefix_table=None, prefix_lens=None, group_offsets=ints(2))])
def test_attend_takes_a_prefix_whole_or_not_at_all(kw):
    with pytest.raises(ValueError):
        attend(cache(), **kw)


def test_attend_with_and_without_a_prefix():
    accepted(attend, cache(), group_offsets=ints(2))
    accepted(attend, cache(), prefix_table=None, prefix_lens=None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(q_out=None)])
def test_append_takes_queries_and_their_place_together(kw):
    with pytest.raises(ValueError):
        append(cache(), **kw)
    accepted(append, cache(), q=None, q_out=None)


def test_attend_workspace_is_memory_of_the_caches_device():
    c = cache()
    n = c.attend_workspace_size(3, 1, 1)
    for ws in (torch.empty(n + 256, dtype=torch.uint8, device="meta"), workspace(c)[:1].expand(1 << 30),
               torch.empty(2 * n + 512, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            attend(c, ws=ws)


def test_rotary_is_on_the_device_of_the_call():
    w, pos = torch.zeros(D, dtype=F16), ints(3)
    for kw in (dict(q_weight=w.to("meta")), dict(k_weight=w.to("meta")), dict(q_weight=w, k_weight=w.to("meta"))):
        with pytest.raises(ValueError):
            pw.Rotary(torch.zeros(8, D), **kw)
    q = torch.zeros(3, HQ, D, dtype=F16)
    for r in (pw.Rotary(torch.zeros(8, D, device="meta")), pw.Rotary(None, k_weight=w.to("meta"))):
        with pytest.raises(ValueError):
            append(cache(), rotary=r, positions=pos)
        with pytest.raises(ValueError):
            pw.qk_norm_rope(r, q, None, pos, torch.empty_like(q), None)
    accepted(pw.qk_norm_rope, pw.Rotary(None, q_weight=w), q, None, None, torch.empty_like(q), None)
    accepted(pw.qk_norm_rope, pw.Rotary(None), q, None, None, torch.empty_like(q), None)


def test_tensors_are_on_a_gpu():
    c, q = cache(), torch.zeros(3, HQ, D, dtype=F16)
    lib.pw_testing_host_sim(0)      # the refusals below come before any launch
    with pytest.raises(ValueError):
        cache()
    with pytest.raises(ValueError):
        pw.qk_norm_rope(pw.Rotary(None), q, None, None, torch.empty_like(q), None)
    with pytest.raises(ValueError):
        pw.qk_norm_rope(pw.Rotary(None), None, q, None, None, torch.empty_like(q))
    with pytest.raises(ValueError):
        append(c)
    with pytest.raises(ValueError):
        attend(c)
    with pytest.raises(ValueError):
        pw.verify_draft(torch.zeros(1, 1, 8), None, None, None, None, torch.zeros(1, 8), ints(1, 1), ints(1))


def test_sizes_past_32_bits_are_refused():
    c, n, one = cache(), (1 << 32) + 1, torch.zeros(1, HQ, D, dtype=F16)
    with pytest.raises(ValueError):
        pw.qk_norm_rope(pw.Rotary(None), one.expand(n, HQ, D), None, None, one.expand(n, HQ, D), None)
    with pytest.raises(ValueError):
        pw.qk_norm_rope(pw.Rotary(None), one[:, :1].expand(1, n, D), None, None, one[:, :1].expand(1, n, D), None)
    empty = torch.zeros(1, 0, dtype=torch.int32)     # tables without pages
    q = torch.zeros(3, HQ, D, dtype=F16)
    with pytest.raises(ValueError):
        attend(c, prefix_table=empty.expand(n, 0), prefix_lens=ints(1))
    with pytest.raises(ValueError):
        attend(c, q=q[:1], out=q[:1].clone(), table=torch.empty(n, 0, dtype=torch.int32), lens=ints(1))
    with pytest.raises(ValueError):
        attend(c, q=q[:0], out=q[:0], lens=ints(0), table=torch.empty(0, n, dtype=torch.int32))
