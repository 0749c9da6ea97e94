"""Whole prompts, token log probabilities, the 4-bit cache and eviction on the GPU against the fp64 oracle.

Error bounds.  u is the heads' type's unit roundoff (2^-11 fp16, 2^-8 bf16), e = 2^-24 fp32's.
* prompt attention: as attention over the cache (test_gpu_serve): a score is off by (D + 16) e of scale sum |q||k|, the
  weights are rounded to the type (fp16 ones below its normal numbers by 2^-25 of the row's largest), sums of n add 2e n.
* 4-bit cache: codes, least values and steps are single fp32 operations, so they and what is loaded are equal, bit for bit.
  Attention takes keys as they are held: a score is a sum of products q c step and q least, of sizes |q| (|least| + c step),
  in (2 D + 32) steps of 2e; queries are cut at 2^-29 of a row's largest.  Values are rounded to the type once: one u more.
* weights by key: e^(s - lse) is off by 2^-22 (the exponential) and by the error of its argument, (D + 16) 2e of scale
  |q||k| and 4e of |lse|; sums of R rows add (R + 16) e.
* log probabilities: with d = x - m every e^d is off by 2^-22 + 4e |d|, where e^d |d| < 1/2, a thread adds up to V / 256 + 64
  of them and 13 joins follow: l and t are off by L = 2^-21 + (V / 256 + 64 + 16 + 13 * 8) e of their size (t's terms of
  one sign), ln p by that and 4e of |x - m| + ln l, H by L (1 + |t| / l) and 4e of its terms.
"""
import numpy as np
import pytest
import torch

import any_precision_expert_gb300 as pw
from oracle import pw_context as X
from oracle import pw_serve as S

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DEVICE_CHECK = 7
NAN, INF = float("nan"), float("inf")


def host(t):
    return t.double().cpu().numpy()


def rand(rng, *shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype).cuda()


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def close(got, ref, bound, what=""):
    got = host(got)
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), f"{what}: {(err / np.maximum(bound, 1e-30)).max():.3g} of the bound"


# ---- prompts ------------------------------------------------------------------

def prompt_case(rng, T, hq, hk, D, dtype, qscale=2.0):
    qkv = rand(rng, T, (hq + 2 * hk) * D, dtype=dtype)
    qkv[:, :hq * D] *= qscale
    return (x.view(T, -1, D) for x in qkv.split([hq * D, hk * D, hk * D], dim=1))


def run_prompt(q, k, v, offsets, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pw.prompt_attend(q, k, v, ints(offsets), out, lse=lse, err=err, **kw)
    torch.cuda.synchronize()
    return out, lse, err.item()


def check_prompt(q, k, v, offsets, out, lse, scale=None):
    D = q.shape[2]
    ref, rl, A, ds, n = X.prompt(host(q), host(k), host(v), offsets, D ** -0.5 if scale is None else scale)
    own = ~np.isnan(rl[:, 0])
    u = UNIT[q.dtype]
    off = (D + 16) * E32 * ds + (n + 16) * 2 * E32
    bound = u * np.abs(ref) + TINY[q.dtype] + (u + 2 * off + n * 2.0 ** -24)[..., None] * A
    close(out[torch.from_numpy(own)], ref[own], bound[own], "out")
    assert (np.abs(host(lse)[own] - rl[own]) <= (off + 4 * E32 * np.abs(rl))[own]).all()
    assert (host(out)[~own] == 7).all() and (host(lse)[~own] == 7).all()  # rows of no sequence stay as they were


PROMPTS = [
    # offsets, T, hq, hk, D
    ([0, 1], 1, 1, 1, 128), ([0, 1], 1, 32, 8, 128), ([0, 2], 2, 4, 2, 64), ([0, 127], 127, 2, 2, 64),
    ([0, 128], 128, 2, 1, 128), ([0, 129], 129, 1, 1, 64), ([0, 255], 255, 1, 1, 128), ([0, 257], 257, 2, 2, 128),
    ([0, 385], 385, 1, 1, 64), ([0, 64], 64, 4, 1, 128), ([0, 65], 65, 8, 2, 64), ([0, 300], 300, 11, 1, 64),
    ([0, 90], 90, 22, 2, 64), ([0, 5, 5, 5, 12, 150, 151], 151, 4, 4, 128), ([3, 40, 41, 200], 230, 6, 2, 64),
    ([0, 0, 0], 9, 2, 1, 64), ([0, 33], 33, 128, 1, 64), ([0, 3, 10], 10, 96, 1, 128),
    ([0] + list(range(1, 81)), 80, 4, 2, 64), ([0, 600], 600, 2, 1, 64), ([10, 530, 531, 800], 801, 3, 1, 128)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(PROMPTS)))
def test_prompt_matches_oracle(i, dt):
    off, T, hq, hk, D = PROMPTS[i]
    q, k, v = prompt_case(np.random.default_rng(i), T, hq, hk, D, TYPES[dt])
    out, lse, err = run_prompt(q, k, v, off)
    check_prompt(q, k, v, off, out, lse)
    assert err == 0
    again = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    pw.prompt_attend(q, k, v, ints(off), again)  # without lse and error word: the same bits
    assert torch.equal(out, again)


def test_prompt_many_tiles_a_cta():
    # more row tiles than CTAs, of many lengths, so that every CTA takes several at different places
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 90, 40)] + [400, 1, 300]
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v = prompt_case(rng, off[-1], 16, 16, 64, torch.float16)
    out, lse, err = run_prompt(q, k, v, off)
    check_prompt(q[:, :2], k[:, :2], v[:, :2], off, out[:, :2], lse[:, :2])
    # each head for itself gives the same bits
    for h in (3, 15):
        one, l1, _ = run_prompt(q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], off)
        assert torch.equal(one, out[:, h:h + 1]) and torch.equal(l1, lse[:, h:h + 1])
    # and each sequence
    for b in (40, 42):
        a, z = off[b], off[b + 1]
        one, l1, _ = run_prompt(q[a:z], k[a:z], v[a:z], [0, z - a])
        assert torch.equal(one, out[a:z]) and torch.equal(l1, lse[a:z])


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_second_row_tiles_that_come_and_go(D):
    # many pieces a CTA, most of whose second row tile is empty: the warpgroups go through the pieces at different paces
    for seed, (B, hq, hk) in enumerate([(106, 16, 16), (160, 16, 16), (60, 64, 16)]):
        rng = np.random.default_rng(40 + seed)
        tokens = 128 // (hq // hk)
        lens = np.where(rng.random(B) < (0.5, 0.15, 0.3)[seed], rng.integers(tokens + 1, 2 * tokens, B), rng.integers(1, tokens + 1, B))
        off = np.concatenate([[0], np.cumsum(lens)]).tolist()
        q, k, v = prompt_case(rng, off[-1], hq, hk, D, torch.float16)
        out, lse, err = run_prompt(q, k, v, off)
        assert err == 0
        for b in (0, B // 2, B - 1):
            a, z = off[b], off[b + 1]
            one, l1, _ = run_prompt(q[a:z], k[a:z], v[a:z], [0, z - a])
            assert torch.equal(one, out[a:z]) and torch.equal(l1, lse[a:z])
        a, z = off[1], off[2]
        check_prompt(q[a:z, :1], k[a:z, :1], v[a:z, :1], [0, z - a], out[a:z, :1], lse[a:z, :1])


def test_prompt_long_rows_against_32_bit_products():
    # 5000 tokens: rows sampled at tile borders, scores in 64 bits
    rng = np.random.default_rng(6)
    T, hq, hk, D = 5000, 4, 2, 128
    q, k, v = prompt_case(rng, T, hq, hk, D, torch.float16)
    out, lse, _ = run_prompt(q, k, v, [0, T])
    for i in (0, 127, 128, 2047, 2048, 4095, 4096, 4999):
        for h in range(hq):
            kk, vv = host(k[:i + 1, h // 2]), host(v[:i + 1, h // 2])
            s = (kk @ host(q[i, h])) * D ** -0.5
            w = np.exp(s - s.max())
            ref, A = (w @ vv) / w.sum(), (w @ np.abs(vv)) / w.sum()
            off = (D + 16) * E32 * D ** -0.5 * (np.abs(kk) @ np.abs(host(q[i, h]))).max() + (i + 17) * 2 * E32
            close(out[i, h], ref, 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -11 + 2 * off + i * E32) * A, f"row {i}")
            assert abs(host(lse[i, h]) - s.max() - np.log(w.sum())) <= off + 4 * E32 * 20


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_prompt_scales(scale):
    q, k, v = prompt_case(np.random.default_rng(7), 150, 4, 2, 64, torch.float16, qscale=1.0)
    out, lse, _ = run_prompt(q, k, v, [0, 150], scale=scale)
    check_prompt(q, k, v, [0, 150], out, lse, scale=scale)


def test_prompt_scores_that_keep_growing():
    q, k, v = prompt_case(np.random.default_rng(8), 500, 2, 1, 64, torch.float16)
    q[:] = 0
    q[..., 0] = 8
    k[..., 0] = torch.arange(500, device="cuda")[:, None] * 0.25
    out, lse, _ = run_prompt(q, k, v, [0, 500])
    check_prompt(q, k, v, [0, 500], out, lse)


def test_prompt_strides():
    rng = np.random.default_rng(9)
    off = [0, 70, 131]
    big = rand(rng, 16, 131, 64, dtype=torch.bfloat16)  # heads first
    q, k, v = (x.transpose(0, 1) for x in (big[:8], big[8:12], big[12:]))
    ref, rl, _ = run_prompt(q.contiguous(), k.contiguous(), v.contiguous(), off)
    out = torch.full((8, 131, 64), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    pw.prompt_attend(q, k, v, ints(off), out)
    assert torch.equal(out, ref)
    check_prompt(q, k, v, off, out, rl)
    # rows that begin inside a sector
    wide = torch.full((131, 8, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    pw.prompt_attend(q, k, v, ints(off), wide[..., 8:])
    assert torch.equal(wide[..., 8:], ref) and (wide[..., :8] == 7).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("off,hq,hk,D", [([0, 300], 4, 1, 64), ([0, 130, 135, 400], 2, 2, 128), ([2, 700], 1, 1, 64), ([0, 520], 8, 1, 128)])
def test_prompt_numbers_that_are_none_reach_only_rows_that_see_them(off, hq, hk, D, dt):
    rng = np.random.default_rng(10)
    T = off[-1] + 60
    q, k, v = prompt_case(rng, T, hq, hk, D, TYPES[dt], qscale=0.5)
    clean, lse, _ = run_prompt(q, k, v, off)
    want, wl = clean.clone(), lse.clone()
    v2, k2 = v.clone(), k.clone()
    G = hq // hk
    for a, z in zip(off[:-1], off[1:]):
        n = z - a
        for t, x in ((n - 1, NAN), (n // 2, INF), (n - n // 4 - 1, -INF)):
            v2[a + t, :, 5] = x
            want[a + t:z, :, 5] += x
        k2[z - 1, 0, 3] = NAN
        want[z - 1, :G], wl[z - 1, :G] = NAN, NAN
    for pad in (slice(0, off[0]), slice(off[-1], T)):  # rows of no sequence
        v2[pad], k2[pad] = NAN, INF
    out, lse, _ = run_prompt(q, k2, v2, off)
    assert torch.equal(torch.nan_to_num(out, nan=99.0), torch.nan_to_num(want, nan=99.0))
    assert torch.equal(torch.nan_to_num(lse, nan=99.0), torch.nan_to_num(wl, nan=99.0))


def test_prompt_offsets_out_of_range_are_clamped_and_flagged():
    q, k, v = prompt_case(np.random.default_rng(11), 50, 2, 1, 64, torch.float16)
    ref, rl, err = run_prompt(q, k, v, [0, 20, 50])
    assert err == 0
    for off in ([-4, 20, 90], [0, 20, 51]):
        out, lse, err = run_prompt(q, k, v, off)
        assert err != 0 and torch.equal(out, ref) and torch.equal(lse, rl)
    out, _, err = run_prompt(q, k, v, [20, 10, 10])  # a descending bound ends its sequence at once
    assert err != 0 and (out == 7).all()


def test_prompt_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(12)
    q, k, v = prompt_case(rng, 200, 4, 2, 64, torch.float16)
    off, out = ints([0, 90, 200]), torch.empty(200, 4, 64, dtype=torch.float16, device="cuda")
    ref, _, _ = run_prompt(q, k, v, [0, 90, 200])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pw.prompt_attend(q, k, v, off, out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pw.prompt_attend(q, k, v, off, out)
    off.copy_(ints([0, 30, 199]))  # other lengths in the same buffer
    out.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:199], run_prompt(q, k, v, [0, 30, 199])[0][:199]) and (out[199] == 7).all()


# ---- log probabilities ----------------------------------------------------------

def run_logprobs(x, tokens, n):
    T = x.shape[0]
    lp, ent, err = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda"), ints([0])
    ids = torch.full((T, n), 77, dtype=torch.int32, device="cuda") if n else None
    tops = torch.full((T, n), 7.0, device="cuda") if n else None
    pw.token_logprobs(x, ints(tokens), lp, entropy=ent, top_ids=ids, top_logprobs=tops, err=err)
    torch.cuda.synchronize()
    return lp, ent, ids, tops, err.item()


def same(got, ref, bound):
    got = host(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
    ok = np.isfinite(ref)
    assert (np.abs(got - ref)[ok] <= np.broadcast_to(bound, ref.shape)[ok]).all(), np.abs(got - ref)[ok].max()


def check_logprobs(x, tokens, n):
    lp, ent, ids, tops, err = run_logprobs(x, tokens, n)
    xs, V = host(x), x.shape[1]
    rl, re, ri, rt = X.logprobs(xs, tokens, n)
    L = 2.0 ** -21 + (V / 256 + 64 + 16 + 13 * 8) * E32
    with np.errstate(all="ignore"):
        m = np.where(np.isfinite(xs), xs, -np.inf).max(1)
        lnl = np.log(np.exp(xs - m[:, None]).sum(1))
        lnl = np.where(np.isfinite(lnl), lnl, 0)
        b = L + 4 * E32 * (np.abs(rl) + 2 * lnl)
        same(lp, rl, np.where(np.isfinite(b), b, 0))
        tl = np.where(np.isfinite(re), np.abs(re - lnl), 0)
        same(ent, re, 2 * L * (1 + tl) + 4 * E32 * (lnl + tl))
        if n:
            assert np.array_equal(ids.cpu().numpy(), ri)
            same(tops, rt, L + 4 * E32 * (np.where(np.isfinite(rt), np.abs(rt), 0) + 2 * lnl[:, None]))
    assert (err != 0) == any(t >= V for t in tokens)
    return lp, ent, ids, tops


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,n", [(1, 1, 1), (1, 2, 0), (3, 7, 7), (2, 33, 20), (5, 1000, 5), (1, 32000, 20), (2, 50257, 32),
                                   (40, 333, 1), (700, 64, 3), (1, 131072, 8), (2, 300001, 4), (3, 4096, 32)])
def test_logprobs_match_oracle(T, V, n, dt):
    rng = np.random.default_rng(T + V)
    x = rand(rng, T, V, dtype=TYPES[dt], scale=3.0)
    check_logprobs(x, rng.integers(0, V, T), n)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_logprobs_rows_of_every_alignment_and_stride(dt):
    rng = np.random.default_rng(1)
    base = rand(rng, 9, 1100, dtype=TYPES[dt], scale=2.0)
    tokens = rng.integers(0, 990, 9)
    for at in range(9):
        x = base[:, at:at + 990 + at]
        check_logprobs(x, tokens, 5)
    x = base[:1].expand(4, 1100)  # one row for all
    a = check_logprobs(x, [3, 4, 5, 6], 2)
    assert torch.equal(a[1], a[1][:1].expand(4))


def test_logprobs_masked_and_extreme_rows():
    rng = np.random.default_rng(2)
    lowest = torch.finfo(torch.float32).min
    x = rand(rng, 12, 5000, dtype=torch.float32, scale=2.0)
    x[0, 7:] = -INF                 # fewer left than alternatives
    x[1, :4990] = -INF
    x[2] = -INF                     # nothing left
    x[3, 100:] = lowest
    x[4] = lowest
    x[5] = 0                        # equal
    x[6, 17] = NAN
    x[7, 4999] = INF
    x[8] *= 1e37
    x[9] = torch.arange(5000)       # each the largest so far
    x[10, 50:4000] = x[10, 49]      # many equal ones
    x[11] = -torch.arange(5000).float() * 1e-3 + 80
    check_logprobs(x, [3, 4, 0, 50, 9, 4999, 1, 2, int(x[8].argmax()), 4998, -1, 5000], 10)
    check_logprobs(x.to(torch.bfloat16), [8, 4992, 0, 50, 9, 4999, 1, 2, int(x[8].argmax()), 4998, -7, 70000], 10)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_logprobs_maxima_at_the_ends_of_a_type(dt):
    lo, hi = torch.finfo(TYPES[dt]).min, torch.finfo(TYPES[dt]).max
    x = torch.full((8, 700), -INF)
    x[0, 5:600:7] = lo
    x[1, 3:500] = lo * 0.9375
    x[2] = hi
    x[3, 9] = hi
    x[4, ::3], x[4, 1::3] = hi * 0.875, lo
    x[5, :300], x[5, 300:] = lo, lo * 0.5
    x[6] = torch.linspace(0.1, 0.2, 700) * lo
    x[7] = torch.linspace(-1, 1, 700) * hi * 2.0 ** -100
    check_logprobs(x.to(TYPES[dt]).cuda(), [5, 4, 0, 9, 3, 299, 0, 699], 6)


def test_logprobs_bounds_over_rounds():
    # rows of several rounds whose best lie in the last, in ascending and in equal runs
    V = 150001
    x = torch.zeros(3, V, device="cuda")
    x[0] = torch.arange(V, device="cuda") / 1000.0
    x[1, 140000:] = 1.0
    x[2, V - 1] = 5.0
    check_logprobs(x, [0, 1, V - 1], 32)


# ---- the cache in 4 bits -----------------------------------------------------------

def to_type(dtype):
    return lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype).float().numpy()


def held(x):
    """(values fp64, |least| + c step, what load gives) of rows x in 4 bits."""
    c, least, step = X.quantise(x.float().cpu().numpy(), to_type(x.dtype))
    v = X.values(c, least, step)
    f = np.float32
    with np.errstate(all="ignore"):
        one = (X.values(c, least * 0, step).astype(f) + np.repeat(least, 32, axis=-1).astype(f)).astype(f)
    size = np.abs(np.repeat(least, 32, axis=-1)) + c * np.repeat(step, 32, axis=-1)
    return v, size, torch.from_numpy(one).to(x.dtype)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,hk,D,page", [(1, 1, 64, 8), (3, 8, 128, 16), (65, 2, 128, 8), (130, 5, 64, 128), (1000, 4, 128, 64)])
def test_four_bit_append_and_load(T, hk, D, page, dt):
    rng = np.random.default_rng(T)
    dtype = TYPES[dt]
    kv = pw.KvCache4.empty(T // page + 3, 2 * hk, hk, page, D, dtype)
    qkv = rand(rng, T, 3 * hk * D, dtype=dtype, scale=3.0)
    k, v = (x.view(T, hk, D) for x in qkv.split(hk * D, dim=1)[1:])
    k[0, 0, :32] = 2.5                                  # a flat group: step 0
    v[0, 0, :32] = torch.linspace(0, 15.5, 32).to(dtype)  # halves of a step
    if T > 2:
        k[2, 0, 3], v[2, 0, D - 1], v[1, 0, 0] = NAN, INF, -INF
        v[2, 0, 0], v[2, 0, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min
    slots = rng.permutation((T // page + 3) * page)[:T]
    kv.append(k, v, ints(slots))
    ko, vo = torch.full((T, hk, D), 9.0, dtype=dtype, device="cuda"), torch.full((T, hk, D), 9.0, dtype=dtype, device="cuda")
    kv.load(ints(slots), ko, vo)
    for x, y in ((k, ko), (v, vo)):
        ref = held(x)[2]
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=77.0), torch.nan_to_num(ref, nan=77.0))
    assert kv.check_device() == 0
    # a slot past the cache or none: nothing is written or read
    state = [x.clone() for x in (kv.k, kv.v, kv.k_steps.view(torch.int16), kv.v_steps.view(torch.int16))]
    kv.append(k[:1], v[:1], ints([-1]))
    assert kv.check_device() == 0
    kv.append(k[:1], v[:1], ints([(T // page + 3) * page]))
    assert kv.check_device() == DEVICE_CHECK
    ko.fill_(9)
    kv.load(ints([-3] * T), ko, vo)
    assert (ko == 9).all() and kv.check_device() == 0
    for x, y in zip(state, (kv.k, kv.v, kv.k_steps.view(torch.int16), kv.v_steps.view(torch.int16))):
        assert torch.equal(x, y)


def test_calls_of_the_4_bit_cache_and_eviction_in_a_graph():
    """Append, attend, weigh and evict captured once and replayed on other contents of the same buffers."""
    rng = np.random.default_rng(30)
    B, hq, hk, D, page = 3, 8, 2, 64, 16
    c = Case4(rng, [40, 20, 31], hq, hk, D, page, torch.float16)
    f = Cached(rng, [40, 20, 31], hq, hk, D, page, torch.float16)
    t4, t16, lens, lens0 = ints(c.table), ints(f.table), ints([40, 20, 31]), ints([40, 20, 31])
    out, lse = torch.empty_like(c.q), torch.empty(B, hq, device="cuda")
    o16, l16 = torch.empty_like(c.q), torch.empty(B, hq, device="cuda")
    w4 = torch.empty(c.kv.attend_workspace_size(B), dtype=torch.uint8, device="cuda")
    w16 = torch.empty(f.kv.attend_workspace_size(B), dtype=torch.uint8, device="cuda")
    we = torch.empty(f.kv.evict_workspace_size(B, 16), dtype=torch.uint8, device="cuda")
    mass, kept = torch.zeros(B, f.table.shape[1] * page, device="cuda"), ints(np.zeros((B, 16)))
    slots = torch.arange(len(c.k), dtype=torch.int32, device="cuda")

    def step():
        c.kv.append(c.k, c.v, slots)
        c.kv.attend(c.q, t4, lens0, out, w4, lse=lse)
        lens.copy_(lens0)
        f.kv.attend(c.q, t16, lens, o16, w16, lse=l16)
        f.kv.weigh(c.q, t16, lens, l16, mass, decay=0.0)
        f.kv.evict(t16, lens, mass, 16, we, recent=4, kept=kept)

    step()  # sets up what a first call sets up
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        r = np.random.default_rng(seed)
        for x in (c.k, c.v, c.q, f.k, f.v):
            x.copy_(rand(r, *x.shape, dtype=torch.float16))
        k0, v0 = host(f.k), host(f.v)
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
        _, rl, _, _, _ = S.attend(host(c.q), k0, v0, f.table, [40, 20, 31], 1, D ** -0.5)
        w, _ = X.weigh(host(c.q), k0, f.table, [40, 20, 31], host(l16), np.zeros(mass.shape), 1, D ** -0.5, 1.0)
        assert lens.tolist() == [16, 16, 16]
        for b in range(B):
            who = kept[b].tolist()
            n = [40, 20, 31][b]
            assert who == sorted(who) and who[-4:] == list(range(n - 4, n))
            gone = [i for i in range(n) if i not in who]
            assert w[b][who[:-4]].min() >= w[b][gone].max() * (1 - 1e-5)


class Case4:
    def __init__(self, rng, lens, hq, hk, D, page, dtype, q_len=1, qscale=2.0, width=None):
        B = len(lens)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + 2
        order = rng.permutation(self.pages - 1) + 1
        self.table = np.zeros((B, width or max(1, max(need))), dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.kv = pw.KvCache4.empty(self.pages, hq, hk, page, D, dtype)
        n = self.pages * page
        self.k, self.v = rand(rng, n, hk, D, dtype=dtype), rand(rng, n, hk, D, dtype=dtype)
        self.q = rand(rng, B * q_len, hq, D, dtype=dtype, scale=qscale)
        self.lens, self.q_len, self.page, self.scale = lens, q_len, page, D ** -0.5
        self.kv.append(self.k, self.v, torch.arange(n, dtype=torch.int32, device="cuda"))

    def run(self, lse=True):
        B = len(self.lens)
        out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda")
        ls = torch.full(self.q.shape[:2], 7.0, device="cuda") if lse else None
        ws = torch.full((self.kv.attend_workspace_size(B, self.q_len),), 255, dtype=torch.uint8, device="cuda")
        self.kv.attend(self.q, ints(self.table), ints(self.lens), out, ws, q_len=self.q_len, scale=self.scale, lse=ls)
        torch.cuda.synchronize()
        return out, ls

    def check(self, out, lse):
        D, dtype = self.q.shape[2], self.q.dtype
        hk = self.k.shape[1]
        paged = lambda a: a.reshape(self.pages, self.page, hk, D).transpose(0, 2, 1, 3)  # noqa: E731
        kv, ksize, _ = held(self.k)
        vv, _, _ = held(self.v)
        q = host(self.q)
        ref, rl, A, _, n = S.attend(q, paged(kv), paged(vv), self.table, self.lens, self.q_len, self.scale)
        ds = S.attend(np.abs(q), paged(ksize), paged(vv), self.table, self.lens, self.q_len, abs(self.scale))[3]
        cut = D * 2.0 ** -28 * np.abs(q).max(-1) * ksize.max() * abs(self.scale)
        u = UNIT[dtype]
        off = (2 * D + 32) * 2 * E32 * ds + cut + (n + 16) * 2 * E32
        close(out, ref, u * np.abs(ref) + 2 * TINY[dtype] + (2 * u + 2 * off + n * 2.0 ** -24)[..., None] * A, "out")
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(host(lse)), none)
        assert (np.abs(host(lse)[~none] - rl[~none]) <= (off + 4 * E32 * np.abs(rl))[~none]).all()
        assert not host(out)[none].any()


ATTEND4 = [
    # lens, hq, hk, D, page, q_len
    ([1], 1, 1, 128, 16, 1), ([0], 4, 2, 64, 8, 1), ([5, 0, 1, 64, 65], 8, 2, 128, 16, 1), ([129, 127, 128], 4, 4, 64, 8, 1),
    ([300, 31, 33], 11, 1, 64, 16, 1), ([40, 700], 32, 2, 128, 128, 1), ([1000], 16, 16, 128, 64, 1), ([5, 9, 200], 8, 2, 128, 8, 5),
    ([5, 1, 0, 33], 4, 4, 64, 32, 4), ([2, 0], 2, 1, 128, 16, 5), ([70, 64], 4, 2, 64, 16, 64), ([90, 12], 128, 1, 64, 16, 1),
    ([30, 4, 260], 48, 2, 128, 1024, 2), ([2500, 1], 4, 1, 64, 256, 1), ([i % 90 for i in range(400)], 4, 2, 64, 16, 1),
    ([3000] * 3, 8, 4, 128, 32, 3)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(ATTEND4)))
def test_four_bit_attention_matches_oracle(i, dt):
    lens, hq, hk, D, page, ql = ATTEND4[i]
    c = Case4(np.random.default_rng(i), lens, hq, hk, D, page, TYPES[dt], ql)
    out, lse = c.run()
    c.check(out, lse)
    assert c.kv.check_device() == 0
    assert torch.equal(out, c.run(lse=False)[0])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_four_bit_attention_small_and_large_queries(dt):
    for scale in (0.0, 1e-6, 300.0):
        c = Case4(np.random.default_rng(3), [150, 9], 4, 2, 64, 16, TYPES[dt], qscale=scale)
        c.scale = 64 ** -0.5 / max(scale, 1e-3)
        c.q[0, 0, 1:] *= 2.0 ** -12
        c.check(*c.run())
        c.scale = -c.scale
        c.check(*c.run())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D,page,ql", [(128, 16, 1), (64, 8, 1), (128, 64, 5), (64, 16, 3)])
def test_four_bit_groups_that_are_no_numbers_reach_only_their_queries(D, page, ql, dt):
    lens = [40, 130, 3, 300]
    c = Case4(np.random.default_rng(4), lens, 8, 2, D, page, TYPES[dt], ql, qscale=0.5)
    clean, lse = c.run()
    want = clean.clone()

    def slot(b, t):
        return int(c.table[b][t // page]) * page + t % page

    for b, n in enumerate(lens):
        for t in {n - 1, max(n - ql + 1, 0), n - 1 - ql // 2}:
            c.v[slot(b, t), :, 40] = NAN
            for j in range(ql):
                if n - ql + j >= t:
                    want[b * ql + j, :, 32:64] = NAN
        for t in range(n, c.table.shape[1] * page):  # behind the length, where the table has a page of the sequence
            if t // page < -(-n // page):
                c.k[slot(b, t)], c.v[slot(b, t)] = INF, NAN
    c.k[:page], c.v[:page] = NAN, NAN  # a page of nobody
    c.kv.append(c.k, c.v, torch.arange(len(c.k), dtype=torch.int32, device="cuda"))
    out, l2 = c.run()
    assert torch.equal(torch.nan_to_num(out, nan=99.0), torch.nan_to_num(want, nan=99.0))
    assert torch.equal(l2, lse)


def test_four_bit_attention_flags_lengths_and_pages():
    c = Case4(np.random.default_rng(5), [40, 20], 4, 2, 64, 16, torch.float16)
    ref, _ = c.run()
    c.lens = [40, 999]  # cut to what the table holds; a page of zeros past its own
    out, _ = c.run()
    assert c.kv.check_device() == DEVICE_CHECK and torch.equal(out[0], ref[0])
    c.lens, was = [40, 20], c.table[1, 1]
    for bad in (-1, c.pages, 2 ** 31 - 1):
        c.table[1, 1] = bad
        out, lse = c.run()
        assert c.kv.check_device() == DEVICE_CHECK and torch.equal(out[0], ref[0])
        v, _, _ = held(c.v)
        k, _, _ = held(c.k)
        paged = lambda a: a.reshape(c.pages, 16, 2, 64).transpose(0, 2, 1, 3)  # noqa: E731
        want = S.attend(host(c.q), paged(k), paged(v), c.table, c.lens, 1, c.scale)[0]  # zeros there
        assert np.abs(host(out) - want).max() < 0.02
    c.table[1, 1] = was
    assert torch.equal(c.run()[0], ref) and c.kv.check_device() == 0


# ---- eviction -------------------------------------------------------------------------

class Cached:
    def __init__(self, rng, lens, hq, hk, D, page, dtype, spare=0, layout="head"):
        B = len(lens)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + B * spare + 1
        order = rng.permutation(self.pages - 1) + 1
        self.table = np.zeros((B, max(1, max(need))), dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.spare = order[at:at + B * spare].reshape(B, spare)
        shape = (self.pages, hk, page, D) if layout == "head" else (self.pages, page, hk, D)
        self.k, self.v = rand(rng, *shape, dtype=dtype), rand(rng, *shape, dtype=dtype)
        if layout != "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.kv, self.lens, self.page, self.rng, self.hq = pw.KvCache(self.k, self.v, n_heads=hq), lens, page, rng, hq


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,hq,hk,D,page,ql,layout", [
    ([1], 1, 1, 128, 16, 1, "head"), ([0, 5], 4, 2, 64, 8, 1, "head"), ([64, 65, 63], 8, 2, 128, 16, 1, "token"),
    ([200, 9, 130], 44, 4, 64, 32, 3, "head"), ([30, 2, 0, 77], 16, 16, 64, 16, 4, "token"), ([100], 64, 1, 128, 8, 2, "head"),
    ([70], 24, 24, 64, 1024, 1, "head")])
def test_weigh_matches_oracle(lens, hq, hk, D, page, ql, layout, dt):
    rng = np.random.default_rng(len(lens) + hq)
    c = Cached(rng, lens, hq, hk, D, page, TYPES[dt], layout=layout)
    B, cap = len(lens), c.table.shape[1] * page
    q = rand(rng, B * ql, hq, D, dtype=TYPES[dt], scale=2.0)
    _, lse, _, _, _ = S.attend(host(q), host(c.k), host(c.v), c.table, lens, ql, D ** -0.5)
    ls = torch.from_numpy(lse.astype(np.float32)).cuda()
    for M in {cap, cap + 5}:
        mass = torch.from_numpy(rng.random((B, M)).astype(np.float32)).cuda()
        out = torch.full((B, M), 7.0, device="cuda")
        c.kv.weigh(q, ints(c.table), ints(lens), ls, mass, out=out, q_len=ql, decay=0.5)
        ref, size = X.weigh(host(q), host(c.k), c.table, lens, host(ls), host(mass), ql, D ** -0.5, 0.5)
        bound = size * (2.0 ** -22 + (2 * D + 32) * E32 * 2 + (ql * hq + 16) * E32) + 2 * E32 * np.abs(ref)
        for b, n in enumerate(lens):
            close(out[b, :n], ref[b, :n], bound[b, :n])
            assert (out[b, n:] == 7).all()
        c.kv.weigh(q, ints(c.table), ints(lens), ls, mass, q_len=ql, decay=0.5)  # in place: the same bits
        for b, n in enumerate(lens):
            assert torch.equal(mass[b, :n], out[b, :n])
    assert c.kv.check_device() == 0
    # room for less than the lengths is flagged, and the rest of the keys weighed
    if max(lens) > 3:
        mass = torch.zeros(B, 3, device="cuda")
        c.kv.weigh(q, ints(c.table), ints([min(n, 3) for n in lens]), ls, mass, q_len=ql)
        assert c.kv.check_device() == 0
        c.kv.weigh(q, ints(c.table), ints([max(n, 4) for n in lens]), ls, mass, q_len=ql)
        assert c.kv.check_device() == DEVICE_CHECK


def test_weigh_ignores_what_is_behind_a_length_and_rows_that_saw_nothing():
    rng = np.random.default_rng(3)
    c = Cached(rng, [20, 9], 4, 2, 64, 16, torch.float16)
    q = rand(rng, 2, 4, 64, dtype=torch.float16)
    ls = torch.full((2, 4), 3.0, device="cuda")
    a, b = torch.zeros(2, 32, device="cuda"), torch.zeros(2, 32, device="cuda")
    c.kv.weigh(q, ints(c.table), ints(c.lens), ls, a)
    c.k[int(c.table[0, 1]), :, 4:] = NAN
    c.k[int(c.table[1, 0]), :, 9:] = INF
    c.kv.weigh(q, ints(c.table), ints(c.lens), ls, b)
    assert torch.equal(a, b) and (a[0, :20] > 0).all() and (a[1, 9:] == 0).all()
    ls[1] = -INF
    b.fill_(NAN)  # a decay of 0 starts anew
    c.kv.weigh(q, ints(c.table), ints(c.lens), ls, b, decay=0.0)
    assert (b[1, :9] == 0).all() and torch.equal(b[0, :20], a[0, :20])


def test_weigh_many_sequences():
    # more tiles than the shape for few CTAs takes; every head's weights still sum to 1
    rng = np.random.default_rng(9)
    for D, page in ((64, 16), (128, 64)):
        lens = rng.integers(1, 700, 300)
        lens[:2] = 700, 129
        c = Cached(rng, lens.tolist(), 8, 2, D, page, torch.float16)
        q = rand(rng, 300, 8, D, dtype=torch.float16, scale=2.0)
        out, lse = torch.empty_like(q), torch.empty(300, 8, device="cuda")
        ws = torch.empty(c.kv.attend_workspace_size(300), dtype=torch.uint8, device="cuda")
        c.kv.attend(q, ints(c.table), ints(lens), out, ws, lse=lse)
        mass = torch.zeros(300, c.table.shape[1] * page, device="cuda")
        c.kv.weigh(q, ints(c.table), ints(lens), lse, mass)
        assert np.allclose(host(mass).sum(1), 8, rtol=1e-4)
        for b in (0, 1, 299):
            ref, size = X.weigh(host(q[b:b + 1]), host(c.k), c.table[b:b + 1], lens[b:b + 1], host(lse[b:b + 1]),
                                np.zeros((1, mass.shape[1])), 1, D ** -0.5, 1.0)
            close(mass[b:b + 1], ref, size * (2.0 ** -22 + (2 * D + 32) * E32 * 2 + 24 * E32))


def run_evict(c, lens, mass, budget, recent, table=None, in_place=True):
    B = len(lens)
    kept = torch.full((B, budget), 77, dtype=torch.int32, device="cuda")
    ws = torch.full((c.kv.evict_workspace_size(B, budget),), 255, dtype=torch.uint8, device="cuda")
    dl, dm, dt = ints(lens), mass.clone(), ints(c.table)
    if in_place:
        c.kv.evict(dt, dl, dm, budget, ws, recent=recent, kept=kept, **({} if table is None else dict(new_table=ints(table))))
        return dl, dm, kept
    nl, nm = torch.full((B,), -5, dtype=torch.int32, device="cuda"), torch.full_like(mass, 7.0)
    c.kv.evict(dt, dl, dm, budget, ws, recent=recent, new_table=ints(table), new_lens=nl, new_mass=nm, kept=kept)
    assert torch.equal(dm, mass) and dl.tolist() == list(lens)
    return nl, nm, kept


EVICT = [
    # lens, hk, D, page, budget, recent
    ([1], 1, 64, 8, 1, 0), ([0, 7], 2, 128, 16, 3, 1), ([40, 100, 3], 2, 64, 16, 32, 8), ([65, 64, 0, 63], 1, 128, 8, 64, 64),
    ([500, 501], 4, 64, 32, 499, 0), ([1000, 37], 8, 128, 64, 100, 100), ([2100, 1500, 2099], 3, 128, 16, 1025, 16),
    ([300] * 200, 2, 64, 16, 200, 10), ([90, 20], 2, 128, 16, 50, 500)]


@pytest.mark.parametrize("where", ["in place", "a copy of the table", "other pages"])
@pytest.mark.parametrize("i", range(len(EVICT)))
def test_evict_matches_oracle(i, where):
    lens, hk, D, page, budget, recent = EVICT[i]
    rng = np.random.default_rng(i)
    spare = -(-min(budget, max(lens)) // page)
    c = Cached(rng, lens, hk, hk, D, page, torch.bfloat16 if i % 2 else torch.float16, spare=spare, layout="token" if i % 3 == 1 else "head")
    cap = c.table.shape[1] * page + (3 if i % 2 else 0)
    m = rng.choice([0.0, 0.25, 1.0], (len(lens), cap)) if i % 2 else rng.standard_normal((len(lens), cap))
    mass = torch.from_numpy(m.astype(np.float32)).cuda()
    new = c.spare if where == "other pages" else c.table
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy()  # noqa: E731
    ref = X.evict(bits(c.k), bits(c.v), c.table, lens, m.astype(np.float32), budget, recent, new)
    nl, nm, kept = run_evict(c, lens, mass, budget, recent, None if where == "in place" else new, in_place=where == "in place")
    assert nl.tolist() == ref[2].tolist() and np.array_equal(kept.cpu().numpy(), ref[4])
    assert np.array_equal(nm.cpu().numpy(), ref[3])
    if where != "other pages":  # slots behind the new length may hold anything
        for b, n in enumerate(ref[2]):
            for t in range(n, lens[b]):
                p = c.table[b][t // page]
                ref[0][p, :, t % page] = bits(c.k)[p, :, t % page]
                ref[1][p, :, t % page] = bits(c.v)[p, :, t % page]
    assert np.array_equal(bits(c.k), ref[0]) and np.array_equal(bits(c.v), ref[1])
    assert c.kv.check_device() == 0


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_sequences_longer_than_a_span(in_place):
    # 8192 masses are held at a time: lengths around that and past it, masses with many equal ones
    rng = np.random.default_rng(12)
    lens, page = [8192, 8193, 20000, 16500], 1024
    for budget, recent in ((8192, 0), (9000, 300), (100, 99)):
        c = Cached(rng, lens, 1, 1, 64, page, torch.float16, spare=-(-budget // page))
        m = rng.choice([0.0, 0.25, 1.0, 3.5], (4, c.table.shape[1] * page)).astype(np.float32)
        bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy()  # noqa: E731
        new = c.table if in_place else c.spare
        k0 = bits(c.k)
        nl, nm, kept = run_evict(c, lens, torch.from_numpy(m).cuda(), budget, recent, None if in_place else new, in_place=in_place)
        k1 = bits(c.k)
        for b, n in enumerate(lens):
            who = X.stays(m[b], n, budget, recent)
            assert nl[b] == len(who) and kept[b, :len(who)].tolist() == who and (kept[b, len(who):] == -1).all()
            assert np.array_equal(nm[b, :len(who)].cpu().numpy(), m[b][who]) and (nm[b, len(who):] == 0).all()
            who, at = np.array(who), np.arange(len(who))
            assert np.array_equal(k1[new[b][at // page], 0, at % page], k0[c.table[b][who // page], 0, who % page])
        assert c.kv.check_device() == 0


def test_evict_odd_masses():
    c = Cached(np.random.default_rng(2), [9, 9, 9], 2, 2, 64, 8, torch.float16)
    m = np.zeros((3, 16), dtype=np.float32)
    m[0, :9] = [NAN, 1, INF, -1, -INF, 0, -0.0, NAN, 2]
    m[1, :9] = NAN
    m[2, :9] = [1e-45, 0, -1e-45, 1e-38, 3e38, -3e38, 1e-45, 0, 0]
    for budget in range(1, 10):
        for recent in (0, 1):
            _, _, kept = run_evict(c, [9, 9, 9], torch.from_numpy(m).cuda(), budget, recent)
            for b in range(3):
                assert kept[b].tolist() == X.stays(m[b], 9, budget, recent), (budget, recent, b)


def test_evict_flags_lengths_and_pages():
    c = Cached(np.random.default_rng(6), [30, 30], 2, 2, 64, 16, torch.float16)
    mass = torch.rand(2, 32, device="cuda")
    nl, _, _ = run_evict(c, [30, 33], mass, 8, 2)
    assert nl.tolist() == [8, 8] and c.kv.check_device() == DEVICE_CHECK
    nl, _, _ = run_evict(c, [-1, 30], mass, 8, 2)
    assert nl.tolist() == [0, 8] and c.kv.check_device() == DEVICE_CHECK
    before = c.k.clone()
    good = c.table.copy()
    for bad in (-1, c.pages, 2 ** 31 - 1):
        c.table = good.copy()
        c.table[0, 0] = bad
        run_evict(c, [30, 0], mass, 20, 2)  # its first page is outside: those rows are neither read nor written
        assert c.kv.check_device() == DEVICE_CHECK
    c.table = good
    own = set(int(p) for p in c.table[0])
    for p in range(c.pages):
        if p not in own:
            assert torch.equal(c.k[p], before[p])


def test_a_cache_under_pressure_end_to_end():
    """A prompt goes through attention and into the cache, a decode step weighs its keys, half of them are evicted, and the
    next step attends over what is left; a 4-bit copy of the rest answers alike."""
    rng = np.random.default_rng(20)
    hq, hk, D, page, B = 8, 2, 64, 16, 3
    lens = [70, 33, 120]
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = off[-1]
    q, k, v = prompt_case(rng, T, hq, hk, D, torch.float16)
    out, lse, _ = run_prompt(q, k, v, off)
    check_prompt(q, k, v, off, out, lse)
    c = Cached(rng, [n + 2 * page for n in lens], hq, hk, D, page, torch.float16)
    slots = [int(c.table[b][t // page]) * page + t % page for b in range(B) for t in range(lens[b])]
    c.kv.append(k, v, ints(slots))
    # the last query of every prompt again, through the cache: the same result
    last = torch.tensor([z - 1 for z in off[1:]], device="cuda")
    q1, o1, l1 = q[last].contiguous(), torch.empty(B, hq, D, dtype=torch.float16, device="cuda"), torch.empty(B, hq, device="cuda")
    table, dl = ints(c.table), ints(lens)
    ws = torch.empty(c.kv.attend_workspace_size(B), dtype=torch.uint8, device="cuda")
    c.kv.attend(q1, table, dl, o1, ws, lse=l1)
    ref, rl, A, ds, n = S.attend(host(q1), host(c.k), host(c.v), c.table, lens, 1, D ** -0.5)
    off1 = (D + 16) * E32 * ds + (n + 16) * 2 * E32
    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -11 + 2 * off1 + n * E32)[..., None] * A
    close(o1, ref, bound)
    close(out[last], ref, bound)
    mass = torch.zeros(B, c.table.shape[1] * page, device="cuda")
    c.kv.weigh(q1, table, dl, l1, mass)
    assert np.allclose(host(mass).sum(1), hq, rtol=1e-3)  # every head's weights sum to 1
    m0, k0, v0 = mass.cpu().numpy().copy(), host(c.k), host(c.v)
    ews = torch.empty(c.kv.evict_workspace_size(B, 40), dtype=torch.uint8, device="cuda")
    c.kv.evict(table, dl, mass, 40, ews, recent=8)
    assert dl.tolist() == [40, 33, 40]
    c.kv.attend(q1, table, dl, o1, ws, lse=l1)
    kc, vc, nl, _, kept = X.evict(k0, v0, c.table, lens, m0, 40, 8, c.table)
    ref, rl, A, ds, n = S.attend(host(q1), kc, vc, c.table, nl, 1, D ** -0.5)
    off1 = (D + 16) * E32 * ds + (n + 16) * 2 * E32
    close(o1, ref, 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -11 + 2 * off1 + n * E32)[..., None] * A)
    # what is left in 4 bits
    kv4 = pw.KvCache4.empty(c.pages, hq, hk, page, D)
    n4 = c.pages * page
    kv4.append(c.k.transpose(1, 2).reshape(n4, hk, D), c.v.transpose(1, 2).reshape(n4, hk, D), torch.arange(n4, dtype=torch.int32, device="cuda"))
    w4 = torch.empty(kv4.attend_workspace_size(B), dtype=torch.uint8, device="cuda")
    o4 = torch.empty_like(o1)
    kv4.attend(q1, table, dl, o4, w4)
    k4, v4 = torch.empty(n4, hk, D, dtype=torch.float16, device="cuda"), torch.empty(n4, hk, D, dtype=torch.float16, device="cuda")
    kv4.load(torch.arange(n4, dtype=torch.int32, device="cuda"), k4, v4)
    paged = lambda a: host(a).reshape(c.pages, page, hk, D).transpose(0, 2, 1, 3)  # noqa: E731
    ref4, _, A4, ds4, _ = S.attend(host(q1), paged(k4), paged(v4), c.table, nl, 1, D ** -0.5)
    # the loaded keys are rounded once more: scores move by 2^-11 of their size
    close(o4, ref4, (2 * 2.0 ** -11 + 2 * (2.0 ** -11 * ds4))[..., None] * A4 + 2.0 ** -11 * np.abs(ref4) + 2.0 ** -20)
    # tokens are drawn from some logits, and scored
    logits = rand(rng, B, 1000, dtype=torch.float32, scale=2.0)
    check_logprobs(logits, host(logits).argmax(1), 3)
    assert c.kv.check_device() == 0 and kv4.check_device() == 0
