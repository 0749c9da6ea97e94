"""The calls around the layer on the GPU against the fp64 oracle: head norm and rotation, paged append, attention with
shared prefixes, draft verification.

Error bounds.  u is the output type's unit roundoff (2^-11 fp16, 2^-8 bf16), e = 2^-24 fp32's.
* rotation: an output is a sum of two products of fp32 values; norm (D products summed, a reciprocal square root of 2
  ulp, two products) and rotation make a relative error of at most (D + 16) e of |a| + |b| in front of the rounding.
* attention: a score is off by at most (D + 16) e times scale sum |q||k| (ds); exponential and sum add 8 e and n e; the
  weights are rounded to the heads' type (u), where fp16 weights of less than its smallest normal number are off by at
  most 2^-25 of the row's largest weight: out is off by u |out| + (u + 2 ((D + 16) e ds + (n + 16) 2e) + n 2^-24) A with
  A the weighted sum of |v| (tensor-core sums may truncate: 2e a step).  lse has no rounding to the type.
"""
import numpy as np
import pytest
import torch

import any_precision_expert_gb300 as pw
from oracle import pw_serve as S

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # 11 and 8 significant bits, rounded to nearest
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half the spacing of subnormal outputs
DEVICE_CHECK = 7


def host(t):
    return t.double().cpu().numpy()


def rand(rng, *shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype).cuda()


def cos_sin(maxpos, rot):
    inv = 10000.0 ** (-np.arange(rot // 2) * 2 / rot)
    ang = np.arange(maxpos)[:, None] * inv
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()


def rope_bound(x, w, eps, tab, pos, inter, dtype, D):
    ref = S.norm_rope(x, w, eps, tab, pos, inter)
    a = np.abs(S.norm_rope(x, w, eps, None, pos, inter))  # sizes of the turned pair: at most |a| + |b| over the head
    mag = np.maximum(a, a.max(-1, keepdims=True))
    return ref, UNIT[dtype] * np.abs(ref) + TINY[dtype] + (D + 16) * E32 * 2 * mag


def close(got, ref, bound, what=""):
    got = host(got)
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), f"{what}: {(err / np.maximum(bound, 1e-30)).max():.3g} of the bound"


# ---- norm and rotation ------------------------------------------------------

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm", [
    (1, 1, 1, 128, 128, False, True), (2, 32, 8, 128, 128, False, False), (7, 16, 16, 128, 64, False, True),
    (33, 22, 2, 64, 64, False, True), (5, 44, 4, 64, 32, True, False), (3, 5, 1, 64, 16, False, True),
    (4, 16, 1, 128, 96, False, True), (4, 6, 2, 128, 112, True, True), (2, 3, 3, 64, 0, False, True),
    (1201, 8, 2, 128, 128, True, True), (600, 20, 4, 64, 48, False, True)])
def test_rope_matches_oracle(dt, T, hq, hk, D, rot, inter, norm):
    rng = np.random.default_rng(T + hq + rot)
    dtype = TYPES[dt]
    qkv = rand(rng, T, (hq + 2 * hk) * D, dtype=dtype, scale=2.0)
    q, k = qkv[:, :hq * D].view(T, hq, D), qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    tab = cos_sin(500, rot) if rot else None
    pos = torch.from_numpy(rng.integers(0, 500, T).astype(np.int32)).cuda()
    qw, kw = (rand(rng, D, dtype=dtype), rand(rng, D, dtype=dtype)) if norm else (None, None)
    r = pw.Rotary(tab, qw, kw, eps=1e-5, interleaved=inter)
    qo = torch.full((T, hq, D), float("nan"), dtype=dtype, device="cuda")
    ko = torch.full((T, hk, D), float("nan"), dtype=dtype, device="cuda")
    pw.qk_norm_rope(r, q, k, pos, qo, ko)
    for x, w, y, what in ((q, qw, qo, "q"), (k, kw, ko, "k")):
        ref, bound = rope_bound(host(x), None if w is None else host(w), 1e-5, None if tab is None else host(tab),
                                pos.cpu().numpy(), inter, dtype, D)
        close(y, ref, bound, what)
    # one side alone, in place, inside the packed projection: the same bits, and nothing else changes
    before = qkv.clone()
    pw.qk_norm_rope(r, None, k, pos, None, k)
    assert torch.equal(k, ko)
    pw.qk_norm_rope(r, q, None, pos, q, None)
    assert torch.equal(q, qo)
    assert torch.equal(qkv[:, (hq + hk) * D:], before[:, (hq + hk) * D:])


def test_rope_positions_outside_the_table_are_clamped_and_flagged():
    rng = np.random.default_rng(0)
    q = rand(rng, 3, 4, 64, dtype=torch.float16)
    r, err = pw.Rotary(cos_sin(10, 64)), torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    pw.qk_norm_rope(r, q, None, torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda"), a, None, err=err)
    assert err.item() == 0
    pw.qk_norm_rope(r, q, None, torch.tensor([-5, 4, 10], dtype=torch.int32, device="cuda"), b, None, err=err)
    assert err.item() != 0 and torch.equal(a, b)
    pw.qk_norm_rope(r, q[:0], None, torch.zeros(0, dtype=torch.int32, device="cuda"), a[:0], None)  # no tokens


# ---- append -----------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hk,D,page,layout,withq", [
    (1, 8, 8, 128, 16, "head", True), (9, 32, 8, 128, 16, "token", True), (37, 44, 4, 64, 8, "head", False),
    (64, 16, 1, 64, 256, "token", True), (1030, 12, 4, 128, 32, "head", True)])
def test_append_matches_oracle(dt, T, hq, hk, D, page, layout, withq):
    rng = np.random.default_rng(T)
    dtype, pages = TYPES[dt], T // page + 4
    shape = (pages, hk, page, D) if layout == "head" else (pages, page, hk, D)
    kc, vc = rand(rng, *shape, dtype=dtype), rand(rng, *shape, dtype=dtype)
    kv_k, kv_v = (kc, vc) if layout == "head" else (kc.transpose(1, 2), vc.transpose(1, 2))
    k0, v0 = kv_k.clone(), kv_v.clone()
    qkv = rand(rng, T, (hq + 2 * hk) * D, dtype=dtype, scale=2.0)
    q, k, v = (x.view(T, -1, D) for x in qkv.split([hq * D, hk * D, hk * D], dim=1))
    v.view(torch.int16)[0, 0, :4] = torch.tensor([0x7e01, -1, 0x7c01, -32768], dtype=torch.int16)  # NaN bits stay
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 2:
        slots[1] = -1
    tab, pos = cos_sin(300, D), rng.integers(0, 300, T).astype(np.int32)
    qw, kw = rand(rng, D, dtype=dtype), rand(rng, D, dtype=dtype)
    r, cache = pw.Rotary(tab, qw, kw, eps=1e-6), pw.KvCache(kv_k, kv_v, n_heads=hq)
    qo = torch.empty_like(q) if withq else None
    sd, pd = torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda()
    cache.append(k, v, sd, rotary=r, positions=pd, q=q if withq else None, q_out=qo)
    ref, bound = rope_bound(host(k), host(kw), 1e-6, host(tab), pos, False, dtype, D)
    full = S.append(host(k0), ref, slots)
    touched = S.append(np.zeros(full.shape), bound, slots)
    close(kv_k, full, touched, "keys")  # untouched places: a bound of zero
    assert np.array_equal(kv_v.contiguous().view(torch.int16).cpu().numpy(),
                          S.append(v0.contiguous().view(torch.int16).cpu().numpy(),
                                   v.contiguous().view(torch.int16).cpu().numpy(), slots))
    if withq:
        close(qo, *rope_bound(host(q), host(qw), 1e-6, host(tab), pos, False, dtype, D), "q")
    assert cache.check_device() == 0
    # without norm and rotation keys are copied bit for bit
    cache.append(k, v, sd)
    assert torch.equal(kv_k, torch.from_numpy(S.append(host(kv_k), host(k), slots)).to(dtype).cuda())


def test_append_flags_slots_past_the_cache():
    kc = torch.zeros(2, 1, 8, 64, dtype=torch.float16, device="cuda")
    cache, k = pw.KvCache(kc, kc.clone(), n_heads=1), torch.ones(3, 1, 64, dtype=torch.float16, device="cuda")
    cache.append(k, k, torch.tensor([3, 16, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    assert cache.check_device() == DEVICE_CHECK and cache.check_device() == 0
    assert kc.sum().item() == 64 and cache.v.sum().item() == 64
    cache.append(k[:0], k[:0], torch.zeros(0, dtype=torch.int32, device="cuda"))


# ---- attention --------------------------------------------------------------

class Case:
    """A cache whose pages outside the sequences' own tokens hold NaN, with shuffled pages.  wide: a prefix table with room
    for a million tokens, so that groups of more than 64 rows take the tcgen05 kernel however short their prefixes are."""

    def __init__(self, rng, lens, plens, offsets, hq, hkv, D, page, dtype, q_len=1, layout="head", width=None, qscale=2.0,
                 wide=False):
        B = len(lens)
        need = [-(-max(0, n) // page) for n in list(plens) + list(lens)]
        pages = rng.permutation(sum(need) + 2)
        kc = np.full((len(pages), hkv, page, D), np.nan, dtype=np.float32)
        vc = kc.copy()
        width = max(need[len(plens):] + [0]) if width is None else width
        self.table = np.full((B, width), int(pages[-1]), dtype=np.int32)
        pwidth = (1 << 20) // page if wide else max(need[:len(plens)] + [0])
        self.ptable = np.full((len(plens), pwidth), int(pages[-1]), dtype=np.int32)
        at = 0
        for i, n in enumerate(list(plens) + list(lens)):
            row = self.ptable[i] if i < len(plens) else self.table[i - len(plens)]
            for t in range(n):
                p = pages[at + t // page]
                row[t // page] = p
                kc[p, :, t % page] = rng.standard_normal((hkv, D))
                vc[p, :, t % page] = rng.standard_normal((hkv, D)) * 3
            at += need[i]
        self.k, self.v = torch.from_numpy(kc).to(dtype).cuda(), torch.from_numpy(vc).to(dtype).cuda()
        if layout == "token":
            self.k, self.v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (self.k, self.v))
        self.q = rand(rng, B * q_len, hq, D, dtype=dtype, scale=qscale)
        self.lens, self.plens, self.offsets = lens, list(plens), offsets
        self.q_len, self.dtype, self.D, self.scale = q_len, dtype, D, D ** -0.5
        self.cache = pw.KvCache(self.k, self.v, n_heads=hq)

    def run(self, q=None, lse=True, ws=None, stream=None):
        q = self.q if q is None else q
        dev = {n: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for n, x in
               (("table", self.table), ("lens", self.lens), ("ptable", self.ptable), ("plens", self.plens))}
        off = None if self.offsets is None else torch.tensor(self.offsets, dtype=torch.int32, device="cuda")
        out = torch.full(q.shape, float("nan"), dtype=self.dtype, device="cuda")
        ls = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
        B, g = len(self.lens), len(self.plens)
        if ws is None:
            ws = torch.full((self.cache.attend_workspace_size(B, self.q_len, g),), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        self.cache.attend(q, dev["table"], dev["lens"], out, ws, q_len=self.q_len, scale=self.scale, lse=ls, stream=stream,
                          **(dict(prefix_table=dev["ptable"], prefix_lens=dev["plens"], group_offsets=off) if g else {}))
        torch.cuda.synchronize()
        return out, ls

    def check(self, out, lse, q=None):
        ref, rl, A, ds, n = S.attend(host(self.q if q is None else q), host(self.k), host(self.v), self.table, self.lens,
                                     self.q_len, self.scale, self.ptable, self.plens or None, self.offsets)
        u = UNIT[self.dtype]
        off = (self.D + 16) * E32 * ds + (n + 16) * 2 * E32
        close(out, ref, u * np.abs(ref) + TINY[self.dtype] + (u + 2 * off + n * 2.0 ** -24)[..., None] * A, "out")
        if lse is not None:
            got = host(lse)
            none = np.isneginf(rl)
            assert np.array_equal(np.isneginf(got), none)
            assert (np.abs(got[~none] - rl[~none]) <= (off + 4 * E32 * np.abs(rl))[~none]).all()
            assert not host(out)[none].any()


ATTEND = [
    # lens, plens, offsets, hq, hkv, D, page, q_len
    ([1], [], None, 1, 1, 128, 16, 1),
    ([0], [], None, 4, 2, 64, 16, 1),
    ([5, 0, 1, 64, 65], [], None, 8, 2, 128, 16, 1),
    ([3, 0, 17], [33], None, 16, 16, 128, 16, 1),
    ([0, 0], [1], None, 8, 8, 64, 8, 1),
    ([1, 2, 3], [0], None, 4, 1, 128, 8, 1),
    ([7, 130, 0, 2], [100, 0, 257], [0, 1, 1, 3], 22, 2, 64, 32, 1),     # an empty group, a sequence outside all
    ([40, 300, 129], [128], None, 14, 2, 128, 64, 1),
    ([5, 9, 200], [77], None, 8, 2, 128, 16, 5),
    ([5, 1, 0, 33], [64], None, 4, 4, 64, 8, 4),                          # fewer own tokens than queries
    ([2, 0], [], None, 2, 1, 128, 16, 5),                                 # rows that see nothing
    ([64, 70], [19], None, 4, 2, 64, 16, 64),
    ([10, 12, 90], [50], None, 128, 1, 64, 16, 1),                        # 128 query heads on one key head
    ([30, 4], [513], None, 96, 2, 128, 128, 3),
    ([3] * 70, [200], None, 8, 2, 128, 16, 1),                            # many rows a key head
    ([6] * 40, [300, 129], [0, 11, 40], 16, 4, 64, 16, 2),
    ([9] * 33, [140], None, 7, 1, 128, 1024, 3),
    ([2500, 1], [1100], None, 4, 4, 64, 256, 1),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attend_matches_oracle(i, wide, dt):
    lens, plens, off, hq, hkv, D, page, ql = ATTEND[i]
    if wide and not plens:
        pytest.skip("no prefix")
    c = Case(np.random.default_rng(i), lens, plens, off, hq, hkv, D, page, TYPES[dt], ql, wide=wide,
             layout="token" if i % 3 == 1 else "head")
    out, lse = c.run()
    c.check(out, lse)
    assert c.cache.check_device() == 0
    # the same bits again, with another workspace's contents and without lse
    again, _ = c.run(lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens,plens,off,hq,hkv,D,ql", [
    # more segments than CTAs, so that every CTA takes several: of many rows (groups of 80 and 40 rows a key head)
    ([9, 5] * 40, [150 + 7 * i for i in range(40)], [2 * i for i in range(40)] + [80], 64, 8, 64, 5),
    ([5] * 60, [300] * 12 + [64, 1, 0, 129, 128, 127, 2, 500], [3 * i for i in range(21)], 64, 16, 128, 5),
    # and of few
    ([i % 90 for i in range(400)], [], None, 16, 4, 64, 1),
    ([i % 70 for i in range(200)], [33], None, 12, 6, 128, 2),
    ([2 + i % 50 for i in range(120)], [40, 1], [0, 70, 120], 21, 3, 64, 2)])
def test_attend_several_segments_a_cta(lens, plens, off, hq, hkv, D, ql, wide):
    if wide and not plens:
        pytest.skip("no prefix")
    c = Case(np.random.default_rng(len(lens)), lens, plens, off, hq, hkv, D, 16, torch.float16, ql, wide=wide)
    out, lse = c.run()
    c.check(out, lse)
    assert c.cache.check_device() == 0
    assert torch.equal(out, c.run(lse=False)[0])


def test_attend_strided_queries_and_a_wide_table():
    rng = np.random.default_rng(50)
    c = Case(rng, [20, 3, 150], [90], None, 8, 2, 128, 16, torch.float16, width=40)
    packed = rand(rng, 3, 12 * 128, dtype=torch.float16, scale=2.0)
    q = packed[:, 256:256 + 1024].view(3, 8, 128)
    c.check(*c.run(q=q), q=q)
    swapped = rand(rng, 8, 3, 128, dtype=torch.float16).transpose(0, 1)
    c.check(*c.run(q=swapped), q=swapped)


@pytest.mark.parametrize("qscale", [0.0, 30.0])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attend_flat_and_peaked_scores(dt, qscale):
    for lens, wide in (([700, 33], False), ([20, 3] * 20, True)):
        c = Case(np.random.default_rng(8), lens, [400], None, 8, 2, 64, 16, TYPES[dt], qscale=qscale, wide=wide)
        c.check(*c.run())
        c.scale = -c.scale
        c.check(*c.run())


@pytest.mark.parametrize("ql,many", [(1, 1), (5, 1), (1, 80)])
def test_attend_scores_that_keep_growing(ql, many):
    # every key beats the ones before it by more than any threshold a running maximum may wait for
    c = Case(np.random.default_rng(9), [600] * many, [700], None, 4, 1, 64, 16, torch.float16, ql, wide=many > 1)
    c.q[:] = 0
    c.q[..., 0] = 8.0
    for row, n in [(c.ptable[0], 700)] + [(c.table[b], 600) for b in range(many)]:
        for t in range(n):
            c.k[int(row[t // 16]), :, t % 16, 0] = 0.25 * t
    c.check(*c.run())


def test_attend_infinite_scores_follow_the_definition():
    c = Case(np.random.default_rng(11), [40], [40], None, 2, 1, 64, 16, torch.float16)
    c.q[:, 0] = float("-inf")       # every score of head 0 is NaN or -inf: no weight is a number
    out, _ = c.run()
    ref = S.attend(host(c.q)[:, 1:], host(c.k), host(c.v), c.table, c.lens, 1, c.scale, c.ptable, c.plens)[0]
    assert np.abs(host(out)[:, 1:] - ref).max() < 0.02  # the neighbouring head is not disturbed


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,plens,hq,hkv,D,page,ql,wide", [
    ([40, 130, 3, 5, 300], [], 8, 2, 128, 16, 5, False),
    ([66, 2, 64], [30], 4, 4, 64, 8, 3, False),                    # four heads a stage
    ([129, 700], [50], 16, 1, 128, 64, 4, False),                  # 64 rows
    ([131] * 30, [300], 8, 2, 64, 16, 2, True),
    ([40, 140, 257], [], 8, 2, 128, 16, 17, False),                # suffixes in the tcgen05 kernel
    ([33, 190, 10], [20], 32, 2, 64, 16, 33, False),               # several row tiles
    ([64, 128, 129], [], 4, 2, 128, 256, 64, False)])
def test_attend_values_that_are_no_numbers_reach_only_the_queries_that_see_them(lens, plens, hq, hkv, D, page, ql, wide, dt):
    c = Case(np.random.default_rng(31), lens, plens, None, hq, hkv, D, page, TYPES[dt], ql, qscale=0.5, wide=wide)
    clean, lse = c.run()
    want = clean.clone()
    for b, n in enumerate(lens):
        for i, (t, x) in enumerate([(n - 1, float("nan")), (n - 1, float("-inf")), (n - ql + 1, float("inf")),
                                    (n - 1 - ql // 2, float("nan"))]):
            if t < 0:
                continue
            h, d = i % hkv, (37 * i + 5 + b) % D
            c.v[int(c.table[b, t // page]), h, t % page, d] = x
            first = max(0, t - n + ql)   # the first query that sees key t
            G = hq // hkv
            want[b * ql + first:(b + 1) * ql, h * G:(h + 1) * G, d] = x
    out, lse2 = c.run()
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(want, nan=7.0))
    assert torch.equal(lse, lse2)
    assert c.cache.check_device() == 0


@pytest.mark.parametrize("page", [10 ** 6, -1, 2 ** 31 - 1])
def test_attend_bad_prefix_pages_on_both_kernels(page):
    for lens, wide in (([20, 3], False), ([20, 3] * 20, True)):
        c = Case(np.random.default_rng(21), lens, [100], None, 8, 2, 128, 16, torch.bfloat16, wide=wide)
        c.ptable[0, 2] = page       # reads as zeros
        c.check(*c.run())
        assert c.cache.check_device() == DEVICE_CHECK


def test_attend_bad_tables_are_flagged_and_stay_inside():
    c = Case(np.random.default_rng(12), [40, 20], [30], None, 4, 2, 64, 16, torch.float16)
    good = c.run()[0]
    c.table[0, 1] = 10 ** 6         # reads as zeros
    out, lse = c.run()
    c.check(out, lse)
    assert torch.equal(out[1], good[1])
    assert c.cache.check_device() == DEVICE_CHECK and c.cache.check_device() == 0
    c.table[0, 1] = -7
    c.check(*c.run())
    assert c.cache.check_device() == DEVICE_CHECK
    d = Case(np.random.default_rng(13), [48, 16], [32], None, 4, 2, 64, 16, torch.float16)
    d.lens, d.plens = [10 ** 6, -4], [33]      # clamped to the tables' 48, 0 and 32 tokens
    d.check(*d.run())
    assert d.cache.check_device() == DEVICE_CHECK
    e = Case(np.random.default_rng(14), [20] * 5, [32, 16], [0, 2, 5], 4, 2, 64, 16, torch.float16)
    ref, _ = e.run()
    e.offsets = [-3, 2, 9]
    out, _ = e.run()
    assert torch.equal(ref, out) and e.cache.check_device() == DEVICE_CHECK
    e.offsets = [4, 2, 5]  # not ascending: flagged, finite, inside
    out, _ = e.run()
    assert torch.isfinite(out).all() and e.cache.check_device() == DEVICE_CHECK


@pytest.mark.parametrize("wide", [False, True])
def test_attend_on_a_side_stream_and_in_a_graph(wide):
    c = Case(np.random.default_rng(15), [100, 7, 300] * 4, [200], None, 32, 4, 128, 16, torch.float16, 2, wide=wide)
    want, wl = c.run()
    s = torch.cuda.Stream()
    got, _ = c.run(stream=s)
    assert torch.equal(want, got)
    dev = [torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for x in (c.table, c.lens, c.ptable, c.plens)]
    out, q = torch.zeros_like(want), torch.zeros_like(c.q)
    ws = torch.empty(c.cache.attend_workspace_size(12, 2, 1), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.cache.attend(q, dev[0], dev[1], out, ws, q_len=2, scale=c.scale, prefix_table=dev[2], prefix_lens=dev[3])
    q.copy_(c.q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    short = [max(2, n // 3) for n in c.lens]    # lengths are read on the device: the same graph serves others
    dev[1].copy_(torch.tensor(short, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    c.lens = short
    c.check(out, None)


@pytest.mark.parametrize("many", [1, 80])
def test_attend_scale_of_zero_is_the_mean(many):
    c = Case(np.random.default_rng(17), [50] * many, [70], None, 4, 1, 64, 16, torch.float16, layout="token", wide=many > 1)
    c.scale = 0.0
    c.check(*c.run())


@pytest.mark.parametrize("hkv", [4, 6, 3])
def test_cache_with_heads_outermost(hkv):
    c = Case(np.random.default_rng(18), [100, 3, 41], [60], None, 2 * hkv, hkv, 128, 16, torch.bfloat16)
    want = c.run()[0]
    c.k, c.v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c.k, c.v))  # [heads][pages][tokens]
    c.cache = pw.KvCache(c.k, c.v, n_heads=2 * hkv)
    out, lse = c.run()
    assert torch.equal(out, want)
    c.check(out, lse)


@pytest.mark.parametrize("hkv,D", [(8, 128), (2, 64), (1, 128)])
def test_attend_one_sequence_on_a_long_prefix(hkv, D):
    # every CTA holds a piece of every row
    c = Case(np.random.default_rng(19), [9], [9000], None, 5 * hkv, hkv, D, 128, torch.float16)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.equal(out, c.run(lse=False)[0])


def test_calls_follow_each_other_and_other_kernels():
    """Each call reads what the one before it in the stream wrote, with and without kernels of others between, many
    times over and from a captured graph (copies, fills and joined streams in front of the calls)."""
    rng = np.random.default_rng(20)
    B, H, hk, D, page = 3, 8, 2, 64, 16
    cache = pw.KvCache(*(torch.zeros(40, hk, page, D, dtype=torch.float16, device="cuda") for _ in range(2)), n_heads=H)
    r = pw.Rotary(cos_sin(600, D), *(rand(rng, D, dtype=torch.float16) for _ in range(2)))
    table = torch.arange(39, dtype=torch.int32, device="cuda").view(B, 13)
    ws = torch.empty(cache.attend_workspace_size(B, 1, 0), dtype=torch.uint8, device="cuda")
    steps = 100
    k, v = (rand(rng, steps, B, hk, D, dtype=torch.float16) for _ in range(2))
    q = rand(rng, steps, B, H, D, dtype=torch.float16)
    lens, pos = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    x, qo, out = (torch.zeros(B, H, D, dtype=torch.float16, device="cuda") for _ in range(3))
    kk, vv = (torch.zeros(B, hk, D, dtype=torch.float16, device="cuda") for _ in range(2))
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            kk.copy_(k.index_select(0, at)[0])
        vv.copy_(v.index_select(0, at)[0])
        x.copy_(q.index_select(0, at)[0])
        main.wait_stream(side)
        slots = table.gather(1, (at // page).expand(B, 1))[:, 0] * page + (at % page).to(torch.int32)
        pos.copy_(at.expand(B))
        cache.append(kk, vv, slots.to(torch.int32), rotary=r, positions=pos, q=x, q_out=qo)
        lens.add_(1)
        cache.attend(qo, table, lens, out, ws)
        cache.attend(out, table, lens, qo, ws)        # straight behind, on the same workspace
        pw.qk_norm_rope(r, qo, None, pos, qo, None)   # in place, straight behind
        pw.qk_norm_rope(r, qo, None, pos, out, None)
        at.add_(1)
        return out.clone()

    eager = []
    for _ in range(steps):
        eager.append(step())
    torch.cuda.synchronize()
    assert cache.check_device() == 0
    # each call alone, the device waited for in between
    for t in (cache.k, cache.v, lens, at):
        t.zero_()
    for i in range(steps):
        torch.cuda.synchronize()
        for n in range(B):
            pos[n] = i
        slots = (table[:, i // page] * page + i % page).to(torch.int32)
        cache.append(k[i], v[i], slots, rotary=r, positions=pos, q=q[i], q_out=qo)
        torch.cuda.synchronize()
        lens.fill_(i + 1)
        cache.attend(qo, table, lens, out, ws)
        torch.cuda.synchronize()
        cache.attend(out, table, lens, qo, ws)
        torch.cuda.synchronize()
        pw.qk_norm_rope(r, qo, None, pos, qo, None)
        torch.cuda.synchronize()
        pw.qk_norm_rope(r, qo, None, pos, out, None)
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i]), i
    for t in (cache.k, cache.v, lens, at):
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(steps):
        g.replay()
        assert torch.equal(got, eager[i]), i


def test_cache_offsets_past_32_bits():
    page, D = 64, 128
    pages = (5 << 30) // (page * D * 2)          # 5 GB of keys: element offsets past 2^31
    k = torch.zeros(pages, 1, page, D, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    cache = pw.KvCache(k, v, n_heads=2)
    T = 100
    rng = np.random.default_rng(16)
    rk, rv = rand(rng, T, 1, D, dtype=torch.float16), rand(rng, T, 1, D, dtype=torch.float16)
    table = torch.tensor([[pages - 1, pages - 9]], dtype=torch.int32, device="cuda")
    t = torch.arange(T, device="cuda")
    cache.append(rk, rv, (table[0].long()[t // page] * page + t % page).to(torch.int32))
    q, out = rand(rng, 1, 2, D, dtype=torch.float16), torch.empty(1, 2, D, dtype=torch.float16, device="cuda")
    ws = torch.empty(cache.attend_workspace_size(1, 1, 0), dtype=torch.uint8, device="cuda")
    cache.attend(q, table, torch.tensor([T], dtype=torch.int32, device="cuda"), out, ws)
    small = np.zeros((2, 1, page, D))
    small_v = small.copy()
    for i in range(T):
        small[i // page, :, i % page], small_v[i // page, :, i % page] = host(rk)[i], host(rv)[i]
    ref, _, A, ds, n = S.attend(host(q), small, small_v, np.array([[0, 1]]), [T], 1, D ** -0.5)
    off = (D + 16) * E32 * ds + (n + 16) * 2 * E32
    u = UNIT[torch.float16]
    close(out, ref, u * np.abs(ref) + TINY[torch.float16] + (u + 2 * off + n * 2.0 ** -24)[..., None] * A)
    assert cache.check_device() == 0


# ---- verification -----------------------------------------------------------

def verify(p, q, tok, n, u, e):
    B, K1, V = p.shape
    d = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in
         (p.astype(np.float32), q.astype(np.float32), tok.astype(np.int32), n.astype(np.int32), u.astype(np.float32),
          e.astype(np.float32))]
    out = torch.full((B, K1), 77, dtype=torch.int32, device="cuda")
    acc, err = torch.full((B,), 77, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pw.verify_draft(*d, out, acc, err=err)
    return out.cpu().numpy(), acc.cpu().numpy(), err.item()


def draws(rng, B, K, V, sharp=2.5, apart=0.7):
    l = rng.standard_normal((B, K + 1, V)) * sharp
    p = np.exp(l) / np.exp(l).sum(-1, keepdims=True)
    l = l[:, :K] + apart * rng.standard_normal((B, K, V))
    q = np.exp(l) / np.exp(l).sum(-1, keepdims=True)
    tok = (q / rng.exponential(size=q.shape)).argmax(-1) if K else np.zeros((B, 0))
    f = np.float32
    return p.astype(f), q.astype(f), tok, rng.integers(0, K + 1, B), rng.random((B, K)).astype(f), rng.exponential(size=(B, V)).astype(f)


@pytest.mark.parametrize("B,K,V", [(1, 0, 1), (1, 1, 1), (3, 4, 7), (2, 2, 1023), (5, 3, 4097), (2, 64, 130), (300, 1, 33),
                                   (4, 5, 50001), (64, 4, 32000), (1, 1, 262145)])
def test_verify_matches_oracle(B, K, V):
    a = draws(np.random.default_rng(B + V), B, K, V)
    out, acc, err = verify(*a)
    want, wacc = S.verify(*a)
    assert np.array_equal(acc, wacc) and np.array_equal(out, want) and err == 0


def test_verify_ties_zero_residuals_and_odd_values():
    rng = np.random.default_rng(3)
    V = 5000
    p, q, tok, n, u, e = draws(rng, 8, 2, V)
    n[:] = 2
    e[0] = 1.0
    p[0] = 0
    p[0, :, [4999, 1234, 77]] = 0.25       # equal quotients: the lowest index
    q[0] = 0.5
    p[1, 0] = q[1, 0]
    u[1, 0] = 1.0                          # refused with a residual of zero: from the target itself
    p[2] = 0                               # nothing at all: index 0
    p[3, :, 10] = np.nan                   # not a number: counts as 0
    p[4, 0, 4000] = np.inf
    q[5, :, ::2] = np.nan
    e[6, :3] = 0.0                         # infinite quotients: the first of them
    q[6] = 0
    p[7] = -p[7]
    out, acc, err = verify(p, q, tok, n, u, e)
    want, wacc = S.verify(p, q, tok, n, u, e)
    assert np.array_equal(acc, wacc) and np.array_equal(out, want) and err == 0
    assert out[0, 0] == 77 and out[2, 0] == 0 and out[6, 0] == 0 or acc[6] > 0


def test_verify_flags_bad_tokens_and_counts():
    a = list(draws(np.random.default_rng(4), 4, 3, 100))
    a[3][:] = 3
    a[2][0, 0], a[2][1, 1] = 100, -1
    out, acc, err = verify(*a)
    want, wacc = S.verify(*a)
    assert err != 0 and np.array_equal(acc, wacc) and np.array_equal(out, want) and acc[0] == 0 and acc[1] <= 1
    a = list(draws(np.random.default_rng(5), 4, 3, 100))
    a[3][:] = [-2, 9, 1, 2]
    out, acc, err = verify(*a)
    want, wacc = S.verify(*a)
    assert err != 0 and np.array_equal(acc, wacc) and np.array_equal(out, want)
