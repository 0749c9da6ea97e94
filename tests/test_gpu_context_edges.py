"""Ends of the types and sizes of the calls of test_gpu_context: the same oracle, bounds and equalities."""
import numpy as np
import pytest
import torch

import any_precision_expert_gb300 as pw
from test_gpu_context import DEVICE_CHECK, TYPES, Cached, Case4, check_logprobs, check_prompt, held, ints, prompt_case, run_prompt

pytestmark = pytest.mark.gpu


def append_and_load(x):
    """What rows x [T, H, D] give back, as keys and as values of a 4-bit cache."""
    T, H, D = x.shape
    kv = pw.KvCache4.empty(-(-T // 16), H, H, 16, D, x.dtype)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kv.append(x, x, slots)
    k, v = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    kv.load(slots, k, v)
    assert kv.check_device() == 0
    return k.cpu(), v.cpu()


def same_as_definition(x):
    """x: rows on the CPU."""
    ref = held(x)[2]
    for got in append_and_load(x.cuda()):
        bad = torch.nan_to_num(got, nan=77.0) != torch.nan_to_num(ref, nan=77.0)
        assert not bad.any(), f"{int(bad.sum())} values, first at {bad.nonzero()[0].tolist()}"
    return ref


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,unit,most", [("f16", 2.0 ** -24, 500), ("bf16", 2.0 ** -133, 120)])
def test_four_bit_steps_of_few_bits(dt, unit, most, D):
    # groups of whole multiples of a type's least number: their steps are rounded up or down by up to a half, quotients pass
    # 15 (15.5 among them, where a step has lost a thirty-first) and many lie on halves; ranges below 8 have a step of 0
    rng = np.random.default_rng(D)
    rows = []
    for n in range(241):
        x = rng.integers(0, n + 1, (2, D // 32, 32))
        x[..., rng.integers(32)] = 0
        x[..., rng.integers(32)] = n  # may be the same place: a smaller range
        rows.append(x + rng.integers(-most, most - n + 1, (2, D // 32, 1)))
    x = np.concatenate(rows).reshape(-1, 1, D)
    x[0, 0, :8], x[0, 0, 8:32] = [0, 31, 5, 3, 10, 12, 7, 1], 0
    x = torch.from_numpy((x * unit).astype(np.float32)).to(TYPES[dt])
    ref = same_as_definition(x)
    assert torch.isfinite(ref).all() and (ref != 0).any()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_four_bit_quotients_on_halves(dt):
    # least + (j + 1/2) step for every j, at steps of all sizes, and the numbers next to them
    T = TYPES[dt]
    rows = []
    for e in (range(-24, 11) if dt == "f16" else range(-133, 120, 7)):
        for least in (0.0, -8.0, -15.0):
            g = np.concatenate([[least, least + 15], least + np.arange(15) + 0.5, np.arange(15) + least])
            x = torch.from_numpy((g * 2.0 ** e).astype(np.float32)).to(T)
            rows += [x, x.clone()]
            near = x[2:17].view(torch.int16)
            rows[-1][2:17] = (near + torch.from_numpy(np.random.default_rng(e + 200).integers(-1, 2, 15).astype(np.int16))).view(T)
    x = torch.stack(rows)
    x = torch.cat([x, x[torch.randperm(len(x), generator=torch.Generator().manual_seed(1))]], dim=1)[:, None]  # heads of 64
    same_as_definition(torch.where(torch.isfinite(x), x, torch.zeros_like(x)))


def least_with_a_longer_step(dtype):
    """The least value of a group up to the largest number whose step is rounded up so far that 15 of them pass it."""
    return 0.0 if dtype == torch.float16 else 8 * 2.0 ** 120


def ends_of_a_type(rng, dtype, n):
    """n groups of 32 finite values that reach to a type's largest numbers or near them."""
    most = torch.finfo(dtype).max
    ends = [0.0, 1.0, -1.0, most, -most, most / 2, -most / 2, most * 0.999, -most * 0.99, most / 15]
    rows = []
    for i in range(n):
        a, b = rng.choice(ends, 2)
        g = np.clip(a + (b - a) * rng.random(32), -most, most)
        g[rng.permutation(32)[:2]] = a, b
        x = torch.from_numpy(g).to(dtype)
        rows.append(torch.where(torch.isfinite(x), x, torch.full_like(x, most)))
    rows[0][:], rows[0][3] = 0, most
    rows[1][:], rows[1][4] = least_with_a_longer_step(dtype), most
    return torch.stack(rows)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_four_bit_groups_at_the_ends_of_a_type_stay_numbers(dt):
    # a top code would stand for an infinity where rounding has lengthened the step: the next lower step is taken
    dtype = TYPES[dt]
    x = ends_of_a_type(np.random.default_rng(7), dtype, 400).view(200, 1, 64)
    ref = same_as_definition(x)
    g, r = x.double().view(-1, 32), ref.double().view(-1, 32)
    wide = g.max(-1).values - g.min(-1).values > torch.finfo(torch.float32).max  # bf16: no step in fp32, so no numbers
    assert torch.isnan(r[wide]).all() and torch.isfinite(r[~wide]).all() and (dt == "bf16" or not wide.any())
    step = (g.max(-1).values - g.min(-1).values)[~wide] / 15
    u = torch.finfo(dtype).eps
    # half a step, 15 times what the step has moved (2 half bits), and the rounding of what is loaded
    bound = step * (0.5 + 15 * u) + u / 2 * torch.finfo(dtype).max
    assert ((g - r).abs().amax(-1)[~wide] <= bound).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D,page", [(64, 8), (128, 16)])
def test_four_bit_values_at_the_ends_of_a_type_reach_only_their_queries(D, page, dt):
    rng = np.random.default_rng(D)
    lens, ql = [3, 40, 130, 35], 3
    c = Case4(rng, lens, 8, 2, D, page, TYPES[dt], ql, qscale=0.5)
    clean, _ = c.run()
    for b, n in enumerate(lens):
        t = n - 1  # only a sequence's last query sees it
        g = torch.full((2, D // 32, 32), least_with_a_longer_step(TYPES[dt]))
        g[..., 5] = torch.finfo(TYPES[dt]).max
        c.v[int(c.table[b][t // page]) * page + t % page] = g.view(2, D).to(TYPES[dt]).cuda()
    c.kv.append(c.k, c.v, torch.arange(len(c.k), dtype=torch.int32, device="cuda"))
    out, lse = c.run()
    for b in range(len(lens)):
        assert torch.equal(out[b * ql:b * ql + ql - 1], clean[b * ql:b * ql + ql - 1])
    if dt == "f16":  # bf16's largest times weights of up to 2^14 leaves fp32
        c.check(out, lse)


@pytest.mark.parametrize("qe,ke,ve", [(-100, 80, 80), (60, -61, -100), (-100, 100, -20), (0, 0, 80)])
@pytest.mark.parametrize("D,ql", [(64, 3), (128, 1)])
def test_four_bit_attention_of_large_and_small_numbers(D, ql, qe, ke, ve):
    # bf16 has the exponents of fp32: powers of two that cancel in the scores change nothing
    c = Case4(np.random.default_rng(5), [200, 3, 33], 8, 2, D, 16, torch.bfloat16, ql)
    c.scale *= 2.0 ** -(qe + ke)
    c.k *= 2.0 ** ke
    c.v *= 2.0 ** ve
    c.q *= 2.0 ** qe
    c.kv.append(c.k, c.v, torch.arange(len(c.k), dtype=torch.int32, device="cuda"))
    c.check(*c.run())


def test_evict_the_most_tokens_that_a_table_may_have():
    # 2^31 - 4096 masses, and a table that names four pages over and over; the heavy ones lie at the ends of the range
    n, page, budget, recent = 0x7ffff000, 1024, 40, 3
    rng = np.random.default_rng(3)
    k, v = (torch.from_numpy(rng.standard_normal((5, 1, page, 64)).astype(np.float16)).cuda() for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    kv = pw.KvCache(k, v, n_heads=1)
    table = (torch.arange(n // page, dtype=torch.int32, device="cuda") % 4)[None].contiguous()
    mass = torch.zeros(1, n, device="cuda")
    heavy = np.unique(np.concatenate([rng.integers(0, n, 20), [0, n - 4, n - 5, n - 8192, n - 8193, n - 12289, 2 ** 30]]))
    heavy = heavy[heavy < n - recent]
    mass[0, torch.from_numpy(heavy).cuda()] = torch.from_numpy(rng.permutation(len(heavy)).astype(np.float32) + 1).cuda()
    ends = mass[0, -recent:] = torch.tensor([0.25, 0.0, 0.5], device="cuda")
    few = [int(x) for x in range(1, budget) if x not in heavy][:budget - recent - len(heavy)]  # of equal masses the first
    who = sorted(heavy.tolist() + few) + list(range(n - recent, n))
    was = mass[0, torch.tensor(who, device="cuda")].clone()
    lens, new, kept = ints([n]), ints([[4]]), ints(np.zeros((1, budget)))
    ws = torch.empty(kv.evict_workspace_size(1, budget), dtype=torch.uint8, device="cuda")
    kv.evict(table, lens, mass, budget, ws, recent=recent, new_table=new, kept=kept)
    assert kv.check_device() == 0 and lens.tolist() == [budget]
    assert kept[0].tolist() == who and torch.equal(mass[0, :budget], was) and torch.equal(was[-recent:], ends)
    assert not mass[0, budget:].any()
    at = torch.tensor(who, device="cuda")
    for now, then in ((k, k0), (v, v0)):
        assert torch.equal(now[4, 0, :budget], then[at // page % 4, 0, at % page]) and torch.equal(now[:4], then[:4])


def test_four_bit_append_and_load_of_more_rows_than_32_bits_count():
    # 2^20 tokens of 2049 key heads: one token's row of each head, again and again, of which the slots take three
    T, hk, D = 1 << 20, 2049, 64
    rng = np.random.default_rng(1)
    one = torch.from_numpy(rng.standard_normal((1, hk, D)).astype(np.float16)).cuda()
    kv = pw.KvCache4.empty(1, hk, hk, 8, D)
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    for slot, t in enumerate((0, T // 2, T - 1)):
        slots[t] = slot
    k = one.expand(T, hk, D)
    kv.append(k, -one.expand(T, hk, D), slots)
    back, vback = torch.full((4, hk, D), 9.0, dtype=torch.float16, device="cuda"), torch.full((4, hk, D), 9.0, dtype=torch.float16, device="cuda")
    kv.load(ints([0, 1, 2, 3]), back, vback)
    for got, x in ((back, one), (vback, -one)):
        assert torch.equal(got[:3].cpu(), held(x)[2].expand(3, hk, D)) and not got[3].any()
    # a load of the same many tokens, all into one row of places, of which one is asked for
    slots[:] = -1
    slots[T - 2] = 1
    ko, vo = torch.full_like(one, 9.0), torch.full_like(one, 9.0)
    kv.load(slots, ko.expand(T, hk, D), vo.expand(T, hk, D))
    assert torch.equal(ko[0], back[1]) and torch.equal(vo[0], vback[1])
    assert kv.check_device() == 0


# ---- prompts ------------------------------------------------------------------

def test_prompt_calls_without_an_error_word_share_one():
    q, k, v = prompt_case(np.random.default_rng(11), 50, 2, 1, 64, torch.float16)
    ref, _, _ = run_prompt(q, k, v, [0, 20, 50])
    out = torch.empty_like(ref)
    pw.prompt_check_device()
    pw.prompt_attend(q, k, v, ints([0, 20, 51]), out)
    assert torch.equal(out, ref)
    assert pw.prompt_check_device() == DEVICE_CHECK and pw.prompt_check_device(q.device) == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pw.prompt_attend(q, k, v, ints([-1, 20, 50]), out, stream=s)
    assert pw.prompt_check_device(stream=s) == DEVICE_CHECK
    pw.prompt_attend(q, k, v, ints([0, 20, 50]), out)
    _, _, err = run_prompt(q, k, v, [0, 20, 51])  # a call's own word is its own
    assert err != 0 and pw.prompt_check_device() == 0


def test_prompt_offsets_that_ask_for_rows_over_and_over():
    q, k, v = prompt_case(np.random.default_rng(12), 50, 2, 1, 64, torch.float16)
    ref, _, _ = run_prompt(q, k, v, [0, 50])
    for off in ([0, 50, 0, 50], [0, 30, 10, 50], [0, 50, 49, 50], [0, 50] * 2048):
        out, lse, err = run_prompt(q, k, v, off)
        assert err != 0 and (out == 7).all() and (lse == 7).all()
    out, _, err = run_prompt(q, k, v, [0, 20, 5, 35])  # rows 5 .. 19 twice, but 50 in all: the others as they are asked for
    own, _, _ = run_prompt(q[5:35], k[5:35], v[5:35], [0, 30])
    assert err != 0 and torch.equal(out[:5], ref[:5]) and torch.equal(out[20:35], own[15:]) and (out[35:] == 7).all()
    # 2^30 pairs of row tiles of up to 8192 key tiles each, of one buffer's overlapping rows
    T, B, hq = 1 << 20, 4096, 128
    buf = torch.zeros((T + hq) * 64, dtype=torch.float16, device="cuda")
    rows = lambda h: buf.as_strided((T, h, 64), (64, 64, 1))  # noqa: E731
    out = torch.full_like(buf, 7.0).as_strided((T, hq, 64), (64, 64, 1))
    err = ints([0])
    pw.prompt_attend(rows(hq), rows(1), rows(1), ints([0, T] * (B // 2) + [0]), out, err=err)
    torch.cuda.synchronize()
    assert err.item() != 0 and (out[:, 0] == 7).all()


@pytest.mark.parametrize("hq,hk,T,D", [(64, 1, 2300, 64), (128, 1, 2600, 128), (256, 2, 1500, 64)])
def test_prompt_places_in_buckets_of_several_tiles(hq, hk, T, D):
    # 2 tokens and 1 a row tile: more than 512 pairs of row tiles fit the call's tokens, so that its places are sorted 2 and
    # 4 to a bucket; alone, a sequence is sorted by itself
    rng = np.random.default_rng(T)
    lens = [T // 2 + 3, 0, 1] + rng.integers(1, 60, 12).tolist() + [5, 2, T // 6]
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    assert off[-1] <= T
    q, k, v = prompt_case(rng, T, hq, hk, D, torch.float16)
    out, lse, err = run_prompt(q, k, v, off)
    assert err == 0 and (out[off[-1]:] == 7).all()
    for a, z in zip(off[:-1], off[1:]):
        if z > a:
            one, l1, _ = run_prompt(q[a:z], k[a:z], v[a:z], [0, z - a])
            assert torch.equal(one, out[a:z]) and torch.equal(l1, lse[a:z])
    a, z = off[5], off[9]
    some = [x - a for x in off[5:10]]
    check_prompt(q[a:z, :2], k[a:z, :1], v[a:z, :1], some, out[a:z, :2], lse[a:z, :2])


# ---- layouts and streams ----------------------------------------------------------

@pytest.mark.parametrize("layout", ["projection", "heads first"])
@pytest.mark.parametrize("D,ql", [(64, 3), (128, 1)])
def test_queries_and_outputs_of_other_layouts(D, ql, layout):
    rng = np.random.default_rng(D)
    lens, hq, hk, page = [70, 5, 200], 12, 3, 16
    c = Case4(rng, lens, hq, hk, D, page, torch.bfloat16, ql)
    f = Cached(rng, lens, hq, hk, D, page, torch.bfloat16)
    B = len(lens)
    T = B * ql

    def other(x):  # [T, hq, D] with the same values
        if layout == "heads first":
            return x.transpose(0, 1).contiguous().transpose(0, 1)
        wide = torch.full((T, (hq + 2 * hk) * D + 8), 7.0, dtype=x.dtype, device="cuda")
        y = wide[:, 8:8 + hq * D].view(T, hq, D)
        y.copy_(x)
        return y

    ref, lse = c.run()
    q, out = other(c.q), other(torch.zeros_like(c.q))
    ws = torch.full((c.kv.attend_workspace_size(B, ql),), 255, dtype=torch.uint8, device="cuda")
    c.kv.attend(q, ints(c.table), ints(lens), out, ws, q_len=ql)
    assert torch.equal(out, ref) and q.stride() == out.stride() != ref.stride()
    m0, m1 = (torch.zeros(B, f.table.shape[1] * page, device="cuda") for _ in range(2))
    f.kv.weigh(c.q, ints(f.table), ints(lens), lse, m0, q_len=ql)
    f.kv.weigh(q, ints(f.table), ints(lens), lse, m1, q_len=ql)
    assert torch.equal(m0, m1) and m0[2, :200].sum() > 0
    if layout == "projection":
        assert (out.as_strided((T, 8), (out.stride(0), 1), 0) == 7).all()  # in front of the heads


def test_every_call_on_a_side_stream_and_in_a_graph_of_its_own():
    rng = np.random.default_rng(2)
    lens, hq, hk, D, page = [90, 33], 8, 2, 64, 16
    c = Case4(rng, lens, hq, hk, D, page, torch.float16)
    f = Cached(rng, lens, hq, hk, D, page, torch.float16)
    x = torch.from_numpy(rng.standard_normal((3, 40000)).astype(np.float32)).cuda()
    tokens = ints([5, 39999, -1])
    table4, table, dl = ints(c.table), ints(f.table), ints(lens)
    kept_k, kept_v = f.k.clone(), f.v.clone()

    def buffers():
        return dict(out=torch.full_like(c.q, 7.0), lse=torch.full((2, hq), 7.0, device="cuda"),
                    mass=torch.zeros(2, f.table.shape[1] * page, device="cuda"), lens=ints([0, 0]), kept=ints(np.zeros((2, 20))),
                    lp=torch.full((3,), 7.0, device="cuda"), ent=torch.full((3,), 7.0, device="cuda"),
                    ids=ints(np.zeros((3, 9))), tops=torch.full((3, 9), 7.0, device="cuda"),
                    ko=torch.full_like(c.k, 9.0), vo=torch.full_like(c.v, 9.0),
                    ws4=torch.empty(c.kv.attend_workspace_size(2), dtype=torch.uint8, device="cuda"),
                    wse=torch.empty(f.kv.evict_workspace_size(2, 20), dtype=torch.uint8, device="cuda"))

    slots = torch.arange(len(c.k), dtype=torch.int32, device="cuda")

    def step(b, stream=None):
        c.kv.append(c.k, c.v, slots, stream=stream)
        c.kv.load(slots, b["ko"], b["vo"], stream=stream)
        c.kv.attend(c.q, table4, dl, b["out"], b["ws4"], lse=b["lse"], stream=stream)
        f.kv.weigh(c.q, table, dl, b["lse"], b["mass"], decay=0.0, stream=stream)
        f.kv.evict(table, dl, b["mass"], 20, b["wse"], recent=3, new_lens=b["lens"], kept=b["kept"], stream=stream)
        pw.token_logprobs(x, tokens, b["lp"], entropy=b["ent"], top_ids=b["ids"], top_logprobs=b["tops"], stream=stream)

    def restore():
        f.k.copy_(kept_k), f.v.copy_(kept_v)
        torch.cuda.synchronize()

    ref = buffers()
    step(ref)
    torch.cuda.synchronize()
    keys = f.k.clone()
    names = [k for k in ref if not k.startswith("ws")]
    b = buffers()
    restore()
    s = torch.cuda.Stream()
    step(b, s)
    s.synchronize()
    assert all(torch.equal(b[k], ref[k]) for k in names) and torch.equal(f.k, keys)
    b = buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    for _ in range(2):
        restore()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b[k], ref[k]) for k in names) and torch.equal(f.k, keys)
    check_logprobs(x, [5, 39999, -1], 9)


# ---- a row's bits are its own -----------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(11, 1), (44, 4), (3, 1), (100, 1)])
def test_prompt_repeats_itself_whatever_ran_before(hq, hk, D):
    # groups that leave rows of a tile to nobody: what shared memory holds there comes from earlier kernels
    rng = np.random.default_rng(hq)
    off = [0, 700, 701, 950]
    q, k, v = prompt_case(rng, off[-1], hq, hk, D, torch.float16)
    ref, rl, _ = run_prompt(q, k, v, off)
    for scale in (1e-3, 30.0, 3000.0):
        for d in (64, 128):
            other = [torch.from_numpy(rng.standard_normal((600, h, d)) * scale).half().cuda() for h in (16, 2, 2)]
            run_prompt(*other, [0, 600])
        out, lse, _ = run_prompt(q, k, v, off)
        assert torch.equal(out, ref) and torch.equal(lse, rl)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D", [(4, 1, 64), (2, 2, 128), (11, 1, 128), (1, 1, 64)])
def test_prompt_rows_do_not_change_with_what_they_do_not_see(hq, hk, D, dt):
    # large queries and keys of later tokens, and of the next sequence, against the same rows with small ones
    rng = np.random.default_rng(D + hq)
    off = [0, 610, 850]
    q, k, v = prompt_case(rng, off[-1], hq, hk, D, TYPES[dt])
    ref, rl, _ = run_prompt(q, k, v, off)
    for t in (1, 129, 300, 301, 520, 609):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        q2[t:] *= 20
        k2[t:] *= 20
        out, lse, _ = run_prompt(q2, k2, v2, off)
        assert torch.equal(out[:t], ref[:t]) and torch.equal(lse[:t], rl[:t]), t
        out, lse, _ = run_prompt(q2[:t], k2[:t], v2[:t], [0, t])
        assert torch.equal(out, ref[:t]) and torch.equal(lse, rl[:t]), t
    q2, k2 = q.clone(), k.clone()
    q2[610:] *= 50
    k2[610:] *= 50
    out, lse, _ = run_prompt(q2, k2, v, off)
    assert torch.equal(out[:610], ref[:610]) and torch.equal(lse[:610], rl[:610])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,D,ql", [(4, 2, 64, 3), (8, 1, 128, 5), (2, 1, 128, 2), (16, 4, 64, 4)])
def test_four_bit_queries_do_not_change_with_what_they_do_not_see(hq, hk, D, ql, dt):
    # the last token's keys and queries large, against the earlier queries' bits with small ones
    page = 16
    lens = [ql + 3, 40, 130, 257, 700]
    c = Case4(np.random.default_rng(hq), lens, hq, hk, D, page, TYPES[dt], ql, qscale=1.0)
    ref, lse = c.run()
    n4 = torch.arange(len(c.k), dtype=torch.int32, device="cuda")
    for size in (20.0, 200.0):
        k, q = c.k.clone(), c.q.clone()
        for b, n in enumerate(lens):
            k[int(c.table[b][(n - 1) // page]) * page + (n - 1) % page] *= size
            c.q[(b + 1) * ql - 1] *= size
        c.kv.append(k, c.v, n4)
        out, l2 = c.run()
        c.q.copy_(q)
        for b in range(len(lens)):
            a, z = b * ql, (b + 1) * ql - 1
            assert torch.equal(out[a:z], ref[a:z]) and torch.equal(l2[a:z], lse[a:z]), b


def test_four_bit_attention_repeats_itself_whatever_ran_before():
    rng = np.random.default_rng(1)
    for hq, hk, D, ql in ((11, 1, 64, 1), (44, 4, 64, 3), (5, 1, 128, 1), (32, 8, 128, 2), (16, 1, 128, 5)):
        c = Case4(rng, [int(x) for x in rng.integers(0, 900, 20)], hq, hk, D, 16, torch.float16, ql)
        ref, lse = c.run()
        for scale in (1e-3, 3000.0):
            x = [torch.from_numpy(rng.standard_normal((600, h, D)) * scale).half().cuda() for h in (16, 2, 2)]
            run_prompt(*x, [0, 600])
            o = Case4(rng, [300, 70], 8, 2, D, 32, torch.float16, 2, qscale=scale)
            o.run()
            out, l2 = c.run()
            assert torch.equal(out, ref) and torch.equal(l2, lse)
