"""Refusals of prompt attention, token log probabilities, the 4-bit cache and eviction: every bad argument is answered on
the host, before anything is enqueued.  Runs without a GPU (host-simulated device, where an accepted call answers
PW_ERR_UNSUPPORTED)."""
import ctypes as C

import pytest
import torch

import any_precision_expert_gb300 as pw
from any_precision_expert_gb300 import _lib
from any_precision_expert_gb300._lib import AttendDesc, EvictDesc, Heads, Kv4Desc, KvDesc, LogprobDesc, PromptDesc, Rows, WeighDesc, lib

OK, INVALID, UNSUPPORTED, OOM = 0, 1, 2, 3
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def sim():
    lib.pw_testing_host_sim(1)
    yield
    lib.pw_testing_host_sim(0)


BUF = (C.c_char * 65536)()
P = (C.addressof(BUF) + 255) & ~255
Q, K = Rows(P, 1024, 128), Rows(P, 256, 128)
NAN, INF = float("nan"), float("inf")


def desc(cls, base, kw):
    return cls(**{**base, **kw})


def prompt(heads=(0, 8, 2, 128), **kw):
    d = desc(PromptDesc, dict(q=Q, k=K, v=K, out=Q, lse=P, tokens=4, offsets=P, batch=2, scale=0.1, err=P), kw)
    return lib.pw_prompt_attend(C.byref(Heads(*heads)), C.byref(d), None)


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, {}), (UNSUPPORTED, dict(lse=None, err=None)), (UNSUPPORTED, dict(tokens=0, q=Rows(), offsets=None)),
    (UNSUPPORTED, dict(batch=0, offsets=None)), (UNSUPPORTED, dict(k=Rows(P, 128, 0), heads=(0, 8, 1, 128))),
    (UNSUPPORTED, dict(tokens=1, k=Rows(P, 0, 128))), (UNSUPPORTED, dict(out=Rows(P, 2048, -128))), (INVALID, dict(q=Rows(P, 0, 128))),
    (INVALID, dict(tokens=-1)), (INVALID, dict(tokens=(1 << 20) + 1)), (INVALID, dict(batch=-1)), (UNSUPPORTED, dict(batch=4097)),
    (INVALID, dict(heads=(2, 8, 2, 128))), (UNSUPPORTED, dict(heads=(0, 8, 2, 96))), (UNSUPPORTED, dict(heads=(0, 258, 2, 128))),
    (INVALID, dict(heads=(0, 8, 3, 128))), (INVALID, dict(scale=NAN)), (INVALID, dict(scale=INF)), (INVALID, dict(offsets=None)),
    (INVALID, dict(offsets=P + 2)), (INVALID, dict(lse=P + 1)), (INVALID, dict(err=P + 2)), (INVALID, dict(q=Rows())),
    (INVALID, dict(v=Rows(P + 8, 256, 128))), (INVALID, dict(out=Rows(P, 1024, 4))), (INVALID, dict(k=Rows(P, 64, 128))),
    (INVALID, dict(v=Rows(P, 256, 0))), (INVALID, dict(v=Rows(P, 256, -128))), (INVALID, dict(k=Rows(P, 1 << 38, 128)))])
def test_prompt_arguments(want, kw):
    # an accepted call answers PW_ERR_UNSUPPORTED here; the shapes the library does not serve answer it as well
    assert prompt(**kw) == want


def logprobs(**kw):
    d = desc(LogprobDesc, dict(logits=P, dtype=2, row_stride=100, T=2, V=100, tokens=P, logprobs=P, entropy=P, n_top=5, top_ids=P,
                               top_logprobs=P, err=P), kw)
    return lib.pw_token_logprobs(C.byref(d), None)


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, {}), (UNSUPPORTED, dict(entropy=None, err=None, n_top=0, top_ids=None, top_logprobs=None)),
    (UNSUPPORTED, dict(T=0, logits=None, tokens=None)), (UNSUPPORTED, dict(dtype=0, logits=P + 2)), (UNSUPPORTED, dict(row_stride=0)),
    (INVALID, dict(dtype=3)), (INVALID, dict(dtype=-1)), (INVALID, dict(T=-1)), (INVALID, dict(T=(1 << 20) + 1)), (INVALID, dict(V=0)),
    (INVALID, dict(V=(1 << 24) + 1)), (INVALID, dict(n_top=-1)), (UNSUPPORTED, dict(n_top=33)), (INVALID, dict(V=4)),
    (INVALID, dict(logits=P + 2)), (INVALID, dict(dtype=1, logits=P + 1)), (INVALID, dict(logits=None)), (INVALID, dict(tokens=None)),
    (INVALID, dict(logprobs=None)), (INVALID, dict(top_ids=None)), (INVALID, dict(top_logprobs=None)), (INVALID, dict(tokens=P + 2)),
    (INVALID, dict(entropy=P + 1)), (INVALID, dict(top_ids=P + 2)), (INVALID, dict(err=P + 2))])
def test_logprobs_arguments(want, kw):
    assert logprobs(**kw) == want


def cache4(heads=(0, 8, 2, 128), page=16, pages=4, k=P, v=P, ks=P, vs=P, err=P):
    h = C.c_void_p()
    d = Kv4Desc(Heads(*heads), page, pages)
    return lib.pw_kv4_create(C.byref(d), k, v, ks, vs, err, C.byref(h)), h


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(page=8)), (OK, dict(page=1024)), (INVALID, dict(page=4)), (INVALID, dict(page=24)), (INVALID, dict(page=2048)),
    (INVALID, dict(pages=0)), (INVALID, dict(page=1024, pages=1 << 21)), (INVALID, dict(k=None)), (INVALID, dict(vs=None)),
    (INVALID, dict(ks=P + 8)), (INVALID, dict(v=P + 4)), (INVALID, dict(err=P + 1)), (UNSUPPORTED, dict(heads=(0, 8, 2, 32))),
    (INVALID, dict(heads=(2, 8, 2, 128)))])
def test_cache4_arguments(want, kw):
    st, h = cache4(**kw)
    assert st == want
    if st == OK:
        assert lib.pw_kv4_destroy(h) == OK
    assert lib.pw_kv4_destroy(None) == INVALID


def test_rows4_arguments():
    _, h = cache4()
    for f in (lib.pw_kv4_append, lib.pw_kv4_load):
        def call(h=h, slots=P, T=4, k=K, v=K):
            return f(h, slots, T, None if k is None else C.byref(k), None if v is None else C.byref(v), None)
        assert call() == UNSUPPORTED and call(T=0, slots=None, k=None, v=None) == UNSUPPORTED
        for kw in (dict(h=None), dict(slots=None), dict(slots=P + 2), dict(T=-1), dict(T=(1 << 20) + 1), dict(k=None), dict(v=None),
                   dict(k=Rows(P + 2, 256, 128)), dict(v=Rows(P, 4, 128))):
            assert call(**kw) == INVALID
    lib.pw_kv4_destroy(h)


def test_attend4_arguments():
    _, h = cache4()
    n = C.c_size_t(0)
    assert lib.pw_kv4_attend_workspace_size(h, 3, 1, C.byref(n)) == OK and n.value > 0
    for bad, want in (((-1, 1), INVALID), ((3, 0), INVALID), ((3, 65), INVALID), ((4097, 1), UNSUPPORTED)):
        assert lib.pw_kv4_attend_workspace_size(h, *bad, C.byref(C.c_size_t(0))) == want
    base = dict(q=Q, out=Q, lse=P, batch=3, q_len=1, scale=0.1, table=P, table_stride=4, lens=P, n_groups=0)

    def call(ws=P, size=None, h=h, **kw):
        d = desc(AttendDesc, base, kw)
        return lib.pw_kv4_attend(h, C.byref(d), ws, n.value if size is None else size, None)
    assert call() == UNSUPPORTED and call(lse=None) == UNSUPPORTED
    for want, kw in [(INVALID, dict(h=None)), (INVALID, dict(q_len=0)), (INVALID, dict(q_len=65)), (INVALID, dict(batch=-1)),
                     (INVALID, dict(scale=NAN)), (INVALID, dict(table=None)), (INVALID, dict(table_stride=-1)), (INVALID, dict(lens=None)),
                     (INVALID, dict(lens=P + 2)), (INVALID, dict(q=Rows())), (INVALID, dict(out=Rows(P, 3, 128))), (INVALID, dict(lse=P + 1)),
                     (INVALID, dict(n_groups=-1)), (UNSUPPORTED, dict(n_groups=1)), (INVALID, dict(ws=None)), (INVALID, dict(ws=P + 16)),
                     (OOM, dict(size=n.value - 1)), (INVALID, dict(table_stride=1 << 27))]:
        assert call(**kw) == want, kw
    lib.pw_kv4_destroy(h)


def cache():
    h = C.c_void_p()
    d = KvDesc(Heads(0, 8, 2, 128), 16, 4, 4096, 2048, 128)
    assert lib.pw_kv_create(C.byref(d), P, P, P, C.byref(h)) == OK
    return h


def test_weigh_arguments():
    h = cache()
    base = dict(q=Q, lse=P, batch=3, q_len=1, scale=0.1, decay=1.0, table=P, table_stride=4, lens=P, mass=P, out=P, mass_stride=64)

    def call(h=h, **kw):
        return lib.pw_kv_weigh(h, C.byref(desc(WeighDesc, base, kw)), None)
    for want, kw in [(UNSUPPORTED, {}), (UNSUPPORTED, dict(batch=0, q=Rows(), lens=None)), (INVALID, dict(h=None)), (INVALID, dict(batch=-1)),
                     (UNSUPPORTED, dict(batch=4097)), (INVALID, dict(q_len=0)), (INVALID, dict(q_len=65)), (INVALID, dict(scale=INF)),
                     (INVALID, dict(decay=NAN)), (INVALID, dict(lse=None)), (INVALID, dict(lse=P + 2)), (INVALID, dict(lens=None)),
                     (INVALID, dict(table=None)), (INVALID, dict(table_stride=-1)), (INVALID, dict(mass=None)), (INVALID, dict(out=None)),
                     (INVALID, dict(out=P + 2)), (INVALID, dict(mass_stride=-1)), (INVALID, dict(table_stride=1 << 27)),
                     (INVALID, dict(q=Rows(P, 1024, 3)))]:
        assert call(**kw) == want, kw
    lib.pw_kv_destroy(h)


def test_evict_arguments():
    h = cache()
    n = C.c_size_t(0)
    assert lib.pw_kv_evict_workspace_size(h, 3, 10, C.byref(n)) == OK
    for bad, want in (((-1, 10), INVALID), ((3, 0), INVALID), ((3, (1 << 24) + 1), INVALID), ((4097, 1), UNSUPPORTED)):
        assert lib.pw_kv_evict_workspace_size(h, *bad, C.byref(C.c_size_t(0))) == want
    base = dict(batch=3, budget=10, recent=2, table=P, table_stride=4, lens=P, mass=P, mass_stride=64, new_table=P, new_stride=1,
                new_lens=P, new_mass=P, kept=P)

    def call(h=h, ws=P, size=None, **kw):
        return lib.pw_kv_evict(h, C.byref(desc(EvictDesc, base, kw)), ws, n.value if size is None else size, None)
    for want, kw in [(UNSUPPORTED, {}), (UNSUPPORTED, dict(kept=None, recent=1000)), (INVALID, dict(h=None)), (INVALID, dict(batch=-1)),
                     (INVALID, dict(budget=0)), (INVALID, dict(recent=-1)), (INVALID, dict(table=None)), (INVALID, dict(new_table=None)),
                     (INVALID, dict(lens=None)), (INVALID, dict(new_lens=None)), (INVALID, dict(mass=None)), (INVALID, dict(new_mass=None)),
                     (INVALID, dict(kept=P + 1)), (INVALID, dict(new_stride=0)), (INVALID, dict(table_stride=-1)), (INVALID, dict(new_stride=-1)),
                     (INVALID, dict(mass_stride=-1)), (INVALID, dict(table_stride=1 << 27)), (INVALID, dict(ws=None)),
                     (INVALID, dict(ws=P + 4)), (OOM, dict(size=n.value - 1))]:
        assert call(**kw) == want, kw
    # what stays has to fit into the new table: the budget, or what the old one and the masses have room for
    assert call(budget=17, size=1 << 20) == INVALID
    assert call(budget=17, size=1 << 20, mass_stride=16) == UNSUPPORTED
    lib.pw_kv_destroy(h)


# ---- the Python calls ------------------------------------------------------------------

def z(*shape, dtype=F16):
    return torch.zeros(*shape, dtype=dtype)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def aligned(n):
    ws = torch.empty(n + 256, dtype=torch.uint8)
    return ws[-ws.data_ptr() % 256:]


def accepted(f, **kw):
    with pytest.raises(pw.PwError) as e:
        f(**kw)
    assert e.value.status == UNSUPPORTED


def kv16():
    k = z(4, 2, 16, 64)
    return pw.KvCache(k, k.clone(), n_heads=4)


CACHE4 = pw.KvCache4
CALLS = {
    "prompt": (lambda: pw.prompt_attend, dict(q=z(5, 4, 64), k=z(5, 2, 64), v=z(5, 2, 64), offsets=i32(3), out=z(5, 4, 64),
                                              lse=z(5, 4, dtype=torch.float32), err=i32(1))),
    "logprobs": (lambda: pw.token_logprobs, dict(logits=z(3, 50), tokens=i32(3), logprobs=z(3, dtype=torch.float32),
                                                 entropy=z(3, dtype=torch.float32), top_ids=i32(3, 4),
                                                 top_logprobs=z(3, 4, dtype=torch.float32), err=i32(1))),
    "append4": (lambda: CACHE4.empty(4, 4, 2, 16, 64, device="cpu").append, dict(k=z(5, 2, 64), v=z(5, 2, 64), slots=i32(5))),
    "load4": (lambda: CACHE4.empty(4, 4, 2, 16, 64, device="cpu").load, dict(k=z(5, 2, 64), v=z(5, 2, 64), slots=i32(5))),
    "attend4": (lambda: CACHE4.empty(4, 4, 2, 16, 64, device="cpu").attend,
                dict(q=z(3, 4, 64), table=i32(3, 2), lens=i32(3), out=z(3, 4, 64), ws=aligned(1 << 20), lse=z(3, 4, dtype=torch.float32))),
    "weigh": (lambda: kv16().weigh, dict(q=z(3, 4, 64), table=i32(3, 2), lens=i32(3), lse=z(3, 4, dtype=torch.float32),
                                         mass=z(3, 32, dtype=torch.float32), out=z(3, 32, dtype=torch.float32))),
    "evict": (lambda: kv16().evict, dict(table=i32(3, 2), lens=i32(3), mass=z(3, 32, dtype=torch.float32), budget=8, ws=aligned(4096),
                                         new_table=i32(3, 1), new_lens=i32(3), new_mass=z(3, 32, dtype=torch.float32), kept=i32(3, 8))),
}
OPTIONAL = {"lse", "err", "entropy", "out", "new_table", "new_lens", "new_mass", "kept"}


@pytest.mark.parametrize("name", CALLS)
def test_calls_hold_every_tensor_to_its_shape_type_and_place(name):
    make, args = CALLS[name]
    f = make()
    accepted(f, **args)
    for a, t in args.items():
        if not isinstance(t, torch.Tensor) or a == "ws":
            continue
        for bad in (t.to(torch.float64), t[:-1], t[None], "x", torch.empty_like(t, device="meta")):
            if a == "logits" and isinstance(bad, torch.Tensor) and bad.dtype == t.dtype and bad.dim() == 2 and not bad.is_meta:
                continue
            if a == "offsets" and isinstance(bad, torch.Tensor) and bad.dim() == 1 and bad.dtype == t.dtype and not bad.is_meta:
                continue
            with pytest.raises((ValueError, pw.PwError)) as e:
                f(**{**args, a: bad})
            assert not isinstance(e.value, pw.PwError) or e.value.status == INVALID, (a, bad)
        if a in OPTIONAL and not (name, a) in (("prompt", "out"), ("attend4", "out"), ("weigh", "lse")):
            accepted(f, **{**args, a: None})
    with pytest.raises((TypeError, ValueError, AttributeError)):
        f(**args, stream="x")


def test_calls_in_python_refuse_what_does_not_belong_together():
    _, a = CALLS["logprobs"]
    for k in ("top_ids", "top_logprobs"):
        with pytest.raises(ValueError):
            pw.token_logprobs(**{**a, k: None})
    with pytest.raises(ValueError):
        pw.token_logprobs(**{**a, "logits": z(50, 3).t()})
    with pytest.raises(ValueError):
        pw.token_logprobs(**{**a, "top_ids": i32(3, 8)[:, ::2]})
    f, a = CALLS["prompt"]
    for k in ("q", "k", "v", "out"):
        with pytest.raises(ValueError):
            pw.prompt_attend(**{**a, k: a[k].to(BF16)})
    with pytest.raises(pw.PwError):
        pw.prompt_attend(**{**a, "k": z(1, 2, 64).expand(5, 2, 64)})
    with pytest.raises(ValueError):
        CACHE4(z(4, 2, 16, 32, dtype=torch.uint8), z(4, 2, 16, 32, dtype=torch.uint8), z(4, 2, 16, 2, 2), z(4, 2, 16, 1, 2), 4)
    with pytest.raises(ValueError):
        CACHE4(z(4, 2, 32, 16, dtype=torch.uint8).transpose(2, 3), z(4, 2, 16, 32, dtype=torch.uint8), z(4, 2, 16, 2, 2), z(4, 2, 16, 2, 2), 4)
    with pytest.raises(ValueError):
        CACHE4.empty(4, 4, 2, 16, 64, dtype=torch.float32, device="cpu")
    kv = CACHE4.empty(4, 4, 2, 16, 64, device="cpu")
    kv.close()
    with pytest.raises(pw.PwError):
        kv.append(z(5, 2, 64), z(5, 2, 64), i32(5))
