"""Refusals of the calls around the layer: every bad argument is answered on the host, before anything is enqueued.
Runs without a GPU (host-simulated device, where an accepted call answers PW_ERR_UNSUPPORTED)."""
import ctypes as C

import pytest
import torch

import any_precision_expert_gb300 as pw
from any_precision_expert_gb300 import _lib
from any_precision_expert_gb300._lib import AttendDesc, Heads, KvDesc, RotaryDesc, Rows, lib

OK, INVALID, UNSUPPORTED, OOM = 0, 1, 2, 3


@pytest.fixture(autouse=True)
def sim():
    lib.pw_testing_host_sim(1)
    yield
    lib.pw_testing_host_sim(0)


BUF = (C.c_char * 65536)()
P = (C.addressof(BUF) + 255) & ~255


def rope(heads=(0, 8, 2, 128), rot=None, pos=P, T=4, q=(P, 1024, 128), k=(P, 256, 128), qo=(P, 1024, 128),
         ko=(P, 256, 128), err=None):
    r = RotaryDesc(**{**dict(cos_sin=P, max_pos=16, rot_dim=128, interleaved=0, q_weight=None, k_weight=None, eps=0.0),
                      **(rot or {})})
    rows = [None if a is None else C.byref(Rows(*a)) for a in (q, k, qo, ko)]
    h = Heads(*heads)
    return lib.pw_qk_norm_rope(C.byref(h), C.byref(r), pos, T, *rows, err, None)


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, {}), (UNSUPPORTED, dict(T=0)), (UNSUPPORTED, dict(q=None, qo=None)), (UNSUPPORTED, dict(k=None, ko=None)),
    (UNSUPPORTED, dict(rot=dict(rot_dim=0, cos_sin=None, max_pos=0), pos=None)),
    (INVALID, dict(T=-1)), (INVALID, dict(T=(1 << 20) + 1)), (INVALID, dict(heads=(2, 8, 2, 128))),
    (INVALID, dict(heads=(0, 8, 3, 128))), (INVALID, dict(heads=(0, 0, 1, 128))), (UNSUPPORTED, dict(heads=(0, 8, 2, 96))),
    (UNSUPPORTED, dict(heads=(0, 258, 2, 128))), (INVALID, dict(pos=None)), (INVALID, dict(pos=P + 2)),
    (INVALID, dict(rot=dict(rot_dim=8))), (INVALID, dict(rot=dict(rot_dim=144))), (INVALID, dict(rot=dict(rot_dim=-16))),
    (INVALID, dict(rot=dict(cos_sin=None))), (INVALID, dict(rot=dict(cos_sin=P + 4))), (INVALID, dict(rot=dict(max_pos=0))),
    (INVALID, dict(rot=dict(interleaved=2))), (INVALID, dict(rot=dict(q_weight=P + 2))),
    (INVALID, dict(rot=dict(eps=-1.0))), (INVALID, dict(rot=dict(eps=float("nan")))), (INVALID, dict(rot=dict(eps=float("inf")))),
    (INVALID, dict(q=None, k=None)), (INVALID, dict(qo=None)), (INVALID, dict(ko=None)),
    (INVALID, dict(q=(P + 2, 1024, 128))), (INVALID, dict(q=(P, 1023, 128))), (INVALID, dict(ko=(P, 256, 4))),
    (INVALID, dict(err=P + 1)),
])
def test_rope_arguments(want, kw):
    # an accepted call answers PW_ERR_UNSUPPORTED here; the shapes the library does not serve answer it as well
    assert rope(**kw) == want


def cache(heads=(0, 8, 2, 128), page=16, pages=4, strides=(2 * 16 * 128, 16 * 128, 128), k=P, v=P, err=P):
    h = C.c_void_p()
    d = KvDesc(Heads(*heads), page, pages, *strides)
    return lib.pw_kv_create(C.byref(d), k, v, err, C.byref(h)), h


@pytest.mark.parametrize("want,kw", [
    (OK, {}), (OK, dict(page=8)), (OK, dict(page=1024)), (INVALID, dict(page=4)), (INVALID, dict(page=2048)),
    (INVALID, dict(page=24)), (INVALID, dict(pages=0)), (INVALID, dict(pages=1 << 27)), (INVALID, dict(k=None)),
    (INVALID, dict(v=None)), (INVALID, dict(err=None)), (INVALID, dict(k=P + 8)), (INVALID, dict(err=P + 2)),
    (INVALID, dict(strides=(4096, 2048, 120))), (INVALID, dict(strides=(4100, 2048, 128))),
    (INVALID, dict(strides=(1 << 40, 2048, 128))), (UNSUPPORTED, dict(heads=(0, 8, 2, 256))),
])
def test_cache_arguments(want, kw):
    st, h = cache(**kw)
    assert st == want
    if st == OK:
        assert lib.pw_kv_destroy(h) == OK


def test_null_handles():
    n = C.c_size_t()
    assert lib.pw_kv_destroy(None) == INVALID
    assert lib.pw_kv_check_device(None, None) == INVALID
    assert lib.pw_kv_append(None, None, None, P, 1, None, None, None, None, None) == INVALID
    assert lib.pw_kv_attend(None, None, None, 0, None) == INVALID
    assert lib.pw_kv_attend_workspace_size(None, 1, 1, 0, C.byref(n)) == INVALID


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, {}), (UNSUPPORTED, dict(T=0, k=None, v=None, slots=None)), (INVALID, dict(T=-1)), (INVALID, dict(slots=None)),
    (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(v=(P, 256, 100))), (INVALID, dict(q=(P, 1024, 128))),
    (INVALID, dict(qo=(P, 1024, 128))), (UNSUPPORTED, dict(q=(P, 1024, 128), qo=(P, 1024, 128))),
])
def test_append_arguments(want, kw):
    st, h = cache()
    a = {**dict(T=2, slots=P, k=(P, 256, 128), v=(P, 256, 128), q=None, qo=None), **kw}
    rows = {n: None if a[n] is None else C.byref(Rows(*a[n])) for n in ("k", "v", "q", "qo")}
    assert lib.pw_kv_append(h, None, None, a["slots"], a["T"], rows["k"], rows["v"], rows["q"], rows["qo"], None) == want
    lib.pw_kv_destroy(h)


ROWS = (P, 1024, 128)


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, {}), (UNSUPPORTED, dict(batch=0)), (INVALID, dict(batch=-1)), (UNSUPPORTED, dict(batch=4097)),
    (INVALID, dict(q_len=0)), (INVALID, dict(q_len=65)), (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(q=Rows(None, 1024, 128))), (INVALID, dict(out=Rows(P + 2, 1024, 128))),
    (INVALID, dict(lens=None)), (INVALID, dict(table=None)), (UNSUPPORTED, dict(table=None, table_stride=0)),
    (INVALID, dict(table_stride=-1)), (INVALID, dict(table_stride=1 << 28)), (INVALID, dict(lse=P + 1)),
    (INVALID, dict(n_groups=-1)), (UNSUPPORTED, dict(n_groups=4097)), (UNSUPPORTED, dict(n_groups=0)),
    (INVALID, dict(prefix_lens=None)), (INVALID, dict(prefix_table=None)), (INVALID, dict(n_groups=2, group_offsets=None)),
    (INVALID, dict(ws=P + 16)), (INVALID, dict(ws=None)), (OOM, dict(ws_bytes=-1)),
])
def test_attend_arguments(want, kw):
    st, h = cache()
    d = dict(q=Rows(*ROWS), out=Rows(*ROWS), lse=None, batch=3, q_len=1, scale=1.0, table=P, table_stride=4, lens=P,
             n_groups=1, group_offsets=None, prefix_table=P, prefix_stride=4, prefix_lens=P)
    kw = dict(kw)
    ws, ws_bytes = kw.pop("ws", P), kw.pop("ws_bytes", None)
    d.update(kw)
    need = C.c_size_t()
    lib.pw_kv_attend_workspace_size(h, 3, 1, 1, C.byref(need))
    if ws_bytes is None:
        ws_bytes = max(need.value, 1 << 30)
    else:
        ws_bytes += need.value
    desc = AttendDesc(**d)
    assert lib.pw_kv_attend(h, C.byref(desc), ws, C.c_size_t(ws_bytes), None) == want
    lib.pw_kv_destroy(h)


@pytest.mark.parametrize("side", ["table_stride", "prefix_stride"])
def test_attend_keys_that_do_not_count_in_32_bits(side):
    st, h = cache()  # pages of 16
    for stride, want in (((1 << 27) - 1, INVALID), ((1 << 27) - 255, INVALID), ((1 << 27) - 256, UNSUPPORTED)):
        d = dict(q=Rows(*ROWS), out=Rows(*ROWS), lse=None, batch=1, q_len=1, scale=1.0, table=P, table_stride=4, lens=P,
                 n_groups=1, group_offsets=None, prefix_table=P, prefix_stride=4, prefix_lens=P)
        d[side] = stride
        desc = AttendDesc(**d)
        assert lib.pw_kv_attend(h, C.byref(desc), P, C.c_size_t(1 << 30), None) == want
    lib.pw_kv_destroy(h)


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, {}), (UNSUPPORTED, dict(B=0)), (UNSUPPORTED, dict(K=0, q=None, tokens=None, n=None, u=None)),
    (INVALID, dict(B=-1)), (INVALID, dict(B=65536)), (INVALID, dict(K=-1)), (INVALID, dict(K=65)), (INVALID, dict(V=0)),
    (INVALID, dict(V=(1 << 24) + 1)), (INVALID, dict(p=None)), (INVALID, dict(q=None)), (INVALID, dict(tokens=None)),
    (INVALID, dict(n=None)), (INVALID, dict(u=None)), (INVALID, dict(noise=None)), (INVALID, dict(out=None)),
    (INVALID, dict(accepted=None)), (INVALID, dict(p=P + 2)), (INVALID, dict(err=P + 3)),
])
def test_verify_arguments(want, kw):
    a = {**dict(p=P, q=P, tokens=P, n=P, u=P, noise=P, B=2, K=3, V=10, out=P, accepted=P, err=None), **kw}
    assert lib.pw_verify_draft(*[a[n] for n in ("p", "q", "tokens", "n", "u", "noise", "B", "K", "V", "out", "accepted",
                                                "err")], None) == want


def test_python_shape_checks():
    f16, kv = torch.float16, torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pw.KvCache(kv, kv.float(), n_heads=4)
    with pytest.raises(ValueError):
        pw.KvCache(kv.float(), kv.float(), n_heads=4)
    with pytest.raises(pw.PwError):
        pw.KvCache(kv, kv, n_heads=5)
    c = pw.KvCache(kv, kv.clone(), n_heads=4)
    k, s = torch.zeros(3, 2, 64, dtype=f16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        c.append(k, k[:2], s)
    with pytest.raises(ValueError):
        c.append(k, k, s.long())
    with pytest.raises(ValueError):
        c.append(k.transpose(1, 2).contiguous().transpose(1, 2), k, s)
    with pytest.raises(ValueError):
        c.append(k.bfloat16(), k, s)
    with pytest.raises(pw.PwError) as e:
        c.append(k, k, s)  # accepted; no device here
    assert e.value.status == UNSUPPORTED
    q, t = torch.zeros(3, 4, 64, dtype=f16), torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        c.attend(q, t, s, q, None, prefix_lens=s[:1])
    with pytest.raises(ValueError):
        c.attend(q[:, :2], t, s, q, None)
    with pytest.raises(ValueError):
        pw.Rotary(torch.zeros(8, 64, dtype=torch.float64))
    r = pw.Rotary(torch.zeros(8, 64), q_weight=torch.zeros(64))
    with pytest.raises(ValueError):
        pw.qk_norm_rope(r, q, None, s, q, None)  # the weight has another type
    with pytest.raises(ValueError):
        pw.verify_draft(torch.zeros(1, 2, 8), torch.zeros(1, 2, 8), s[None], s[:1], torch.zeros(1, 1), torch.zeros(1, 8),
                        t[:1], s[:1])
    c.close()
    c.close()
