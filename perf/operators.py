"""Measured cases of the serving operators beside the MoE layer.

A decode step that verifies drafted tokens runs four of them around the layer:

* ``rope``: RMS norm of every query and key head and the position rotation, in one pass;
* ``append``: the same on the way of new keys and values into a paged cache (and of the queries beside them);
* ``attend``: attention of a batch whose sequences share prefixes: paged prefix (read once for the group) plus each
  sequence's own paged suffix, one or several query tokens a sequence, causal among themselves;
* ``verify``: acceptance of drafted tokens and the draw of the next one from given random numbers.

``run`` computes them in elementary torch operations where ``own`` is false and through the package's entry points
where it is true.  Head layouts are those of hidden sizes 4096 (32 heads of 128), 2048 (16 heads of 128) and 2816 cut
into heads of 64 (44 query heads on 4), the layer configurations' sizes; vocabulary sizes are generic.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token of one sequence: the latency of the smallest call
        dict(name="rope-token", op="rope", T=1, hq=16, hkv=16, d=128, rot=128, inter=False, norm=True, dtype="f16"),
        # a mid-sized batch with partial, interleaved rotation and an odd group of 11 query heads a key head
        dict(name="rope-odd-333", op="rope", T=333, hq=44, hkv=4, d=64, rot=32, inter=True, norm=False, dtype="bf16"),
        # long prompts prepared at once
        dict(name="rope-prompt-16384", op="rope", T=16384, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, dtype="f16"),
        # one decode step of 64 sequences, small pages
        dict(name="append-decode-64", op="append", T=64, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, page=16, dtype="f16"),
        # one prompt of odd length, every query head with its own key head
        dict(name="append-prompt-8191", op="append", T=8191, hq=16, hkv=16, d=128, rot=128, inter=False, norm=True, page=64, dtype="bf16"),
        # a lone sequence behind a short system prompt: latency
        dict(name="attend-one", op="attend", B=1, ql=1, hq=16, hkv=16, d=128, groups=1, prefix=512, lo=40, hi=40, page=16, dtype="f16"),
        # a decode batch whose own contexts are long and ragged: bound by reading the suffixes
        dict(name="attend-decode-64", op="attend", B=64, ql=1, hq=32, hkv=8, d=128, groups=1, prefix=2048, lo=1, hi=4095, page=16, dtype="f16"),
        # five drafted positions a sequence behind an 8191-token document
        dict(name="attend-draft-24", op="attend", B=24, ql=5, hq=32, hkv=8, d=128, groups=1, prefix=8191, lo=5, hi=1500, page=64, dtype="bf16"),
        # four system prompts of different lengths, heads of 64 in groups of 11
        dict(name="attend-groups-48", op="attend", B=48, ql=1, hq=44, hkv=4, d=64, groups=4, prefix=6000, lo=3, hi=700, page=32, dtype="f16"),
        # many requests on one long document: bound by the prefix products
        dict(name="attend-prefix-256", op="attend", B=256, ql=1, hq=32, hkv=8, d=128, groups=1, prefix=32768, lo=1, hi=256, page=64, dtype="f16"),
        # a few sequences, four drafted tokens each
        dict(name="verify-4", op="verify", B=4, K=4, V=32000),
        # a large batch over a large vocabulary
        dict(name="verify-256", op="verify", B=256, K=4, V=131072),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "verify"])
    if op == "verify":
        V = _log(rng, 1000, 131072)
        return dict(op=op, B=_log(rng, 1, 256), K=rng.randint(0, 4), V=V)
    hq, hkv, d = rng.choice([(32, 8, 128), (16, 16, 128), (44, 4, 64), (32, 4, 128), (16, 1, 64), (20, 4, 128)])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("rope", "append"):
        T = _log(rng, 1, 16384 if hq * d <= 2048 or op == "rope" else 8191)
        case = dict(op=op, T=T, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2]), inter=rng.random() < 0.3,
                    norm=rng.random() < 0.6, dtype=dtype)
        if op == "append":
            case["page"] = rng.choice([8, 16, 32, 64, 128])
        return case
    B, ql = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
    # the prefix products cost at most those of 1024 rows a key head on 8 heads of 128 over 32768 keys, and the
    # suffixes at most 256 MB of keys and as many of values
    prefix = min(_log(rng, 1, 32768), max(1, (1024 * 8 * 128 * 32768) // (B * ql * hq * d)))
    hi = max(ql, min(_log(rng, 1, 8192), (256 << 20) // (B * hkv * d * 2)))
    groups = rng.choice([g for g in (1, 1, 2, 3, 4) if B % g == 0])
    return dict(op=op, B=B, ql=ql, hq=hq, hkv=hkv, d=d, groups=groups, prefix=prefix, lo=min(hi, ql + rng.randint(0, 3)),
                hi=hi, page=rng.choice([8, 16, 32, 64, 128]), dtype=dtype)


def _lens(case):
    """Suffix lengths, evenly spread over [lo, hi]; prefix lengths, from the full one down to half of it."""
    B, g = case["B"], case["groups"]
    lens = [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, B - 1) for i in range(B)]
    plens = [max(1, case["prefix"] - (case["prefix"] // 2) * i // max(1, g - 1)) for i in range(g)]
    return lens, plens


def _rotation(case, gen, dev):
    """cos | sin table [max_pos][rot] in fp32, and the norm weights."""
    rot, maxpos = case["rot"], 32768
    inv = 10000.0 ** (-torch.arange(0, rot // 2, dtype=torch.float64, device=dev) * 2 / rot)
    ang = torch.arange(maxpos, dtype=torch.float64, device=dev)[:, None] * inv[None]
    s = {"cos_sin": torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous(), "qw": None, "kw": None}
    if case["norm"]:
        dt = _DT[case["dtype"]]
        s["qw"] = (1 + 0.2 * torch.randn(case["d"], generator=gen, device=dev)).to(dt)
        s["kw"] = (1 + 0.2 * torch.randn(case["d"], generator=gen, device=dev)).to(dt)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2 + 1)
    host = torch.Generator().manual_seed(int(seed) * 2 + 1)
    s = {"case": case}
    if case["op"] == "verify":
        B, K, V = case["B"], case["K"], case["V"]
        logits = 2.5 * torch.randn(B, K + 1, V, generator=gen, device=dev)
        s["p"] = torch.softmax(logits, dim=-1)
        # the draft model: the target's logits, disturbed
        s["q"] = torch.softmax(logits[:, :K] + 0.7 * torch.randn(B, K, V, generator=gen, device=dev), dim=-1)
        del logits
        e = torch.empty(B, K, V, device=dev).exponential_(generator=gen)
        s["tokens"] = (s["q"] / e).argmax(dim=-1).to(torch.int32) if K else torch.zeros(B, 0, dtype=torch.int32, device=dev)
        del e
        s["n_draft"] = torch.randint(min(1, K), K + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        s["u"] = torch.rand(B, K, generator=gen, device=dev)
        s["noise"] = torch.empty(B, V, device=dev).exponential_(generator=gen)
        s["out"] = torch.empty(B, K + 1, dtype=torch.int32, device=dev)
        s["accepted"] = torch.empty(B, dtype=torch.int32, device=dev)
        return s
    dt, hq, hkv, d = _DT[case["dtype"]], case["hq"], case["hkv"], case["d"]

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    if case["op"] in ("rope", "append"):
        T = case["T"]
        # queries, keys and values as one projection leaves them: [T][(hq + 2 hkv) d]
        qkv = rand(T, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, :hq * d].view(T, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
        s.update(_rotation(case, gen, dev))
        s["pos"] = torch.randint(0, 32768, (T,), generator=gen, device=dev, dtype=torch.int32)
        s["q_out"] = torch.empty(T, hq, d, dtype=dt, device=dev)
        s["k_out"] = torch.empty(T, hkv, d, dtype=dt, device=dev)
        if case["op"] == "append":
            page = case["page"]
            pages = -(-T // page) + 7
            s["k_cache"] = rand(pages, hkv, page, d)
            s["v_cache"] = rand(pages, hkv, page, d)
            table = torch.randperm(pages, generator=host)
            t = torch.arange(T) + 3  # the first page is partly filled already
            s["slots"] = (table[t // page] * page + t % page).to(torch.int32).to(dev)
        if own:
            import any_precision_expert_gb300 as pw
            s["rotary"] = pw.Rotary(s["cos_sin"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, interleaved=case["inter"])
            if case["op"] == "append":
                s["kv"] = pw.KvCache(s["k_cache"], s["v_cache"], n_heads=hq)
        return s
    B, ql, page = case["B"], case["ql"], case["page"]
    lens, plens = _lens(case)
    order = torch.randperm(B, generator=host).tolist()
    lens = [lens[i] for i in order]
    need = [-(-n // page) for n in plens + lens]
    pages = torch.randperm(sum(need) + 1, generator=host).to(torch.int32)
    table = torch.zeros(B, max(1, max(need[len(plens):])), dtype=torch.int32)
    ptable = torch.zeros(len(plens), max(need[:len(plens)]), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        row = ptable[i] if i < len(plens) else table[i - len(plens)]
        row[:n] = pages[at:at + n]
        at += n
    s["k_cache"] = rand(len(pages), hkv, page, d)
    s["v_cache"] = rand(len(pages), hkv, page, d)
    s["table"], s["ptable"] = table.to(dev), ptable.to(dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["plens"] = torch.tensor(plens, dtype=torch.int32, device=dev)
    s["offsets"] = torch.arange(len(plens) + 1, dtype=torch.int32, device=dev) * (B // len(plens))
    s["q"] = rand(B * ql, hq, d, scale=2.0)  # peaked rather than flat weights
    s["scale"] = d ** -0.5
    s["out"] = torch.empty(B * ql, hq, d, dtype=dt, device=dev)
    s["lse"] = torch.empty(B * ql, hq, dtype=torch.float32, device=dev)
    if own:
        import any_precision_expert_gb300 as pw
        s["kv"] = pw.KvCache(s["k_cache"], s["v_cache"], n_heads=hq)
        s["ws"] = torch.empty(s["kv"].attend_workspace_size(B, ql, len(plens)), dtype=torch.uint8, device=dev)
    return s


def _norm_rotate(x, w, s):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * w.float()
    rot = s["case"]["rot"]
    cs = s["cos_sin"][s["pos"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if s["case"]["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, x[..., rot:]], dim=-1)


def _attend(s):
    c = s["case"]
    B, ql, hq, hkv, d, g = c["B"], c["ql"], c["hq"], c["hkv"], c["d"], c["groups"]
    G = hq // hkv
    q = s["q"].float().view(B, ql, hkv, G, d)
    minus = float("-inf")
    # the prefix, once a group: [g][hkv][rows][d] x [g][hkv][P][d]
    pk = s["k_cache"][s["ptable"].long()].float().transpose(2, 1).reshape(g, hkv, -1, d)
    pv = s["v_cache"][s["ptable"].long()].float().transpose(2, 1).reshape(g, hkv, -1, d)
    qp = q.view(g, B // g, ql, hkv, G, d).permute(0, 3, 1, 2, 4, 5).reshape(g, hkv, -1, d)
    seen = torch.arange(pk.shape[2], device=q.device) < s["plens"][:, None]
    sp = (qp @ pk.transpose(-1, -2) * s["scale"]).masked_fill(~seen[:, None, None], minus)
    # each sequence's own suffix, causal among its query tokens
    k = s["k_cache"][s["table"].long()].float().transpose(2, 1).reshape(B, hkv, -1, d)
    v = s["v_cache"][s["table"].long()].float().transpose(2, 1).reshape(B, hkv, -1, d)
    last = s["lens"][:, None] - ql + torch.arange(ql, device=q.device)
    seen = torch.arange(k.shape[2], device=q.device) <= last[..., None]
    qs = q.permute(0, 2, 1, 3, 4).reshape(B, hkv, ql * G, d)
    ss = (qs @ k.transpose(-1, -2) * s["scale"]).masked_fill(~seen.repeat_interleave(G, dim=1)[:, None], minus)

    def back(x):  # [g][hkv][B/g][ql][G][...] rows to the suffix's [B][hkv][ql G][...]
        x = x.view(g, hkv, B // g, ql * G, -1).permute(0, 2, 1, 3, 4)
        return x.reshape(B, hkv, ql * G, -1)

    m = torch.maximum(back(sp.amax(-1, keepdim=True)), ss.amax(-1, keepdim=True))
    m = torch.where(m == minus, torch.zeros_like(m), m)
    mp = m.view(g, B // g, hkv, ql * G, 1).permute(0, 2, 1, 3, 4).reshape(g, hkv, -1, 1)
    ep, es = (sp - mp).exp_(), (ss - m).exp_()
    total = back(ep.sum(-1, keepdim=True)) + es.sum(-1, keepdim=True)
    o = back(ep @ pv) + es @ v
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = m + total.log()

    def rows(x):  # [B][hkv][ql G][n] to [B ql][hq][n]
        return x.view(B, hkv, ql, G, -1).permute(0, 2, 1, 3, 4).reshape(B * ql, hq, -1)

    return {"out": rows(o).to(s["out"].dtype), "lse": rows(lse)[..., 0]}


def _verify(s):
    p, q, tok, u = s["p"], s["q"], s["tokens"].long(), s["u"]
    B, K, V = p.shape[0], q.shape[1], p.shape[2]
    at = torch.arange(K, device=p.device)
    pt = p[:, :K].gather(-1, tok[..., None])[..., 0]
    qt = q.gather(-1, tok[..., None])[..., 0]
    ok = (u * qt < pt) & (at < s["n_draft"][:, None])
    n = ok.long().cumprod(dim=1).sum(dim=1)
    row = p.gather(1, n[:, None, None].expand(B, 1, V))[:, 0]
    if K:
        less = q.gather(1, n.clamp(max=K - 1)[:, None, None].expand(B, 1, V))[:, 0]
        left = torch.where((n < s["n_draft"])[:, None], row - less, row).clamp(min=0)
        row = torch.where((left > 0).any(dim=1, keepdim=True), left, row)
    score = row / s["noise"]
    best = score.amax(dim=1, keepdim=True)
    ids = torch.arange(V, device=p.device)
    nxt = torch.where(score == best, ids, V).amin(dim=1)
    place = torch.arange(K + 1, device=p.device)
    drafted = torch.cat([tok, tok.new_zeros(B, 1)], dim=1)
    out = torch.where(place < n[:, None], drafted, torch.where(place == n[:, None], nxt[:, None], -1))
    return {"out": out.to(torch.int32), "accepted": n.to(torch.int32)}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import any_precision_expert_gb300 as pw
        if op == "rope":
            pw.qk_norm_rope(s["rotary"], s["q"], s["k"], s["pos"], s["q_out"], s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "append":
            s["kv"].append(s["k"], s["v"], s["slots"], rotary=s["rotary"], positions=s["pos"], q=s["q"], q_out=s["q_out"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "attend":
            s["kv"].attend(s["q"], s["table"], s["lens"], s["out"], s["ws"], q_len=s["case"]["ql"], scale=s["scale"],
                           prefix_table=s["ptable"], prefix_lens=s["plens"], group_offsets=s["offsets"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        pw.verify_draft(s["p"], s["q"], s["tokens"], s["n_draft"], s["u"], s["noise"], s["out"], s["accepted"])
        return {"out": s["out"], "accepted": s["accepted"]}
    if op == "rope":
        return {"q": _norm_rotate(s["q"], s["qw"], s).to(s["q"].dtype), "k": _norm_rotate(s["k"], s["kw"], s).to(s["k"].dtype)}
    if op == "append":
        page = s["case"]["page"]
        at, off = s["slots"].long() // page, s["slots"].long() % page
        s["k_cache"][at, :, off] = _norm_rotate(s["k"], s["kw"], s).to(s["k"].dtype)
        s["v_cache"][at, :, off] = s["v"]
        q = _norm_rotate(s["q"], s["qw"], s).to(s["q"].dtype)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return _attend(s) if op == "attend" else _verify(s)


def work(case):
    op = case["op"]
    if op == "verify":
        # one row of the target, one of the noise and, where a draft was refused (about half of them here), one of
        # the draft; a subtraction, a quotient and a comparison each
        n = case["B"] * case["V"]
        return {"bytes": n * 4 * 2.5, "flops": n * 3}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op in ("rope", "append"):
        heads = hq + (hkv if op == "rope" else 2 * hkv)
        n = case["T"] * d * heads
        table = case["T"] * case["rot"] * 4
        return {"bytes": n * 4 + table + case["T"] * (4 if op == "rope" else 8), "flops": 6 * case["T"] * d * (hq + hkv)}
    lens, plens = _lens(case)
    B, ql, g = case["B"], case["ql"], case["groups"]
    rows = B * ql * hq
    keys = sum(lens) + sum(plens)
    seen = sum(p * (B // g) for p in plens) * ql + sum(max(0, n - j) for n in lens for j in range(ql))
    return {"bytes": keys * hkv * d * 4 + rows * (d * 4 + 4), "flops": 4 * d * hq * seen}


def _exact_rotate(x, w, case, pos):
    """The rotation as products of complex numbers, angles from their definition in 64 bits through the fp32 table's values."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6).sqrt() * w.double()
    rot = case["rot"]
    half = rot // 2
    inv = 10000.0 ** (-torch.arange(0, half, dtype=torch.float64, device=x.device) * 2 / rot)
    ang = pos.double()[:, None] * inv[None]
    turn = torch.complex(ang.cos().float().double(), ang.sin().float().double())[:, None]
    head = x[..., :rot]
    pairs = head.unflatten(-1, (half, 2)) if case["inter"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn)
    y = z.flatten(-2) if case["inter"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _exact_rotate(s["q"], s["qw"], case, s["pos"]), "k": _exact_rotate(s["k"], s["kw"], case, s["pos"])}
    if case["op"] == "append":
        page, hkv, d = case["page"], case["hkv"], case["d"]
        kc = s["k_cache"].double().transpose(1, 2).reshape(-1, hkv, d)
        vc = s["v_cache"].double().transpose(1, 2).reshape(-1, hkv, d)
        kc.index_copy_(0, s["slots"].long(), _exact_rotate(s["k"], s["kw"], case, s["pos"]))
        vc.index_copy_(0, s["slots"].long(), s["v"].double())
        back = lambda c: c.view(-1, page, hkv, d).transpose(1, 2).contiguous()  # noqa: E731
        return {"q": _exact_rotate(s["q"], s["qw"], case, s["pos"]), "k_cache": back(kc), "v_cache": back(vc)}
    # attention one (sequence group, key head) at a time, then one (sequence, key head)
    B, ql, hq, hkv, d, g, page = (case[k] for k in ("B", "ql", "hq", "hkv", "d", "groups", "page"))
    G = hq // hkv
    out = torch.zeros(B * ql, hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B * ql, hq), float("-inf"), dtype=torch.float64, device=s["q"].device)
    plens, lens = s["plens"].tolist(), s["lens"].tolist()

    def keys(cache, row, n, h):
        return cache[row[:-(-n // page)].long(), h].reshape(-1, d)[:n].double()

    for b0 in range(0, B, B // g):
        gi = b0 // (B // g)
        for h in range(hkv):
            at = slice(b0 * ql, (b0 + B // g) * ql)
            q = s["q"][at, h * G:(h + 1) * G].double() * s["scale"]
            pk, pv = keys(s["k_cache"], s["ptable"][gi], plens[gi], h), keys(s["v_cache"], s["ptable"][gi], plens[gi], h)
            sc = q.reshape(-1, d) @ pk.T
            l = torch.logsumexp(sc, dim=-1)
            lse[at, h * G:(h + 1) * G] = l.view(-1, G)
            out[at, h * G:(h + 1) * G] = (torch.exp(sc - l[:, None]) @ pv).view(-1, G, d)
            del sc
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        kk = s["k_cache"][s["table"][b, :-(-n // page)].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :n].double()
        vv = s["v_cache"][s["table"][b, :-(-n // page)].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :n].double()
        q = s["q"][b * ql:(b + 1) * ql].double().view(ql, hkv, G, d) * s["scale"]
        sc = torch.einsum("jhgd,hnd->jhgn", q, kk)
        hidden = torch.arange(n, device=sc.device)[None] > (n - ql + torch.arange(ql, device=sc.device))[:, None]
        sc = sc.masked_fill(hidden[:, None, None], float("-inf"))
        top = sc.amax(-1).clamp(min=-1e300)
        w = torch.exp(sc - top[..., None])
        own_lse = (top + w.sum(-1).log()).reshape(ql, hq)
        o = torch.einsum("jhgn,hnd->jhgd", w, vv).reshape(ql, hq, d) / w.sum(-1).clamp(min=1e-300).reshape(ql, hq, 1)
        at = slice(b * ql, (b + 1) * ql)
        both = torch.logaddexp(lse[at], own_lse)
        out[at] = out[at] * torch.exp(lse[at] - both)[..., None] + o * torch.exp(own_lse - both)[..., None]
        lse[at] = both
    return {"out": out, "lse": lse}
