"""Measured cases of the operators for whole prompts, their scores and a cache that is short of memory.

* ``prompt``: causal attention of packed prompts over their own keys, grouped heads;
* ``logprobs``: log probabilities of given tokens, entropies and the best alternatives from rows of logits;
* ``append4``: keys and values into a paged cache held in 4 bits, and what that cache then stands for;
* ``attend4``: attention of a decode batch over such a cache;
* ``weigh``: attention weights of a step's queries added up by key;
* ``evict``: sequences cut to a budget of tokens, the heaviest and the latest, moved together into fewer pages.

``run`` computes them in elementary torch operations where ``own`` is false and through the package's entry points
where it is true.  Head layouts are those of hidden sizes 4096 (32 heads of 128), 2048 (16 heads of 128) and 2816 cut
into heads of 64 (44 query heads on 4), the layer configurations' sizes; vocabulary sizes are generic.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_MINUS = float("-inf")


def listed():
    return [
        # a batch of chat messages of very different lengths, prefilled together
        dict(name="prompt-chat-24", op="prompt", B=24, lo=1, hi=1111, hq=44, hkv=4, d=64, dtype="bf16"),
        # one long document
        dict(name="prompt-document-8191", op="prompt", B=1, lo=8191, hi=8191, hq=32, hkv=8, d=128, dtype="f16"),
        # a decode step that reports the sampled tokens' probabilities
        dict(name="logprobs-step-8", op="logprobs", T=8, V=32000, top=5, dtype="f32"),
        # a prompt scored token by token over a large vocabulary
        dict(name="logprobs-prompt-2047", op="logprobs", T=2047, V=131072, top=8, dtype="bf16"),
        # one decode step of 64 sequences
        dict(name="append4-decode-64", op="append4", T=64, hkv=8, d=128, page=16, dtype="f16"),
        # a prompt of odd length
        dict(name="append4-prompt-8191", op="append4", T=8191, hkv=16, d=128, page=64, dtype="bf16"),
        # a lone sequence with a long context: latency
        dict(name="attend4-one", op="attend4", B=1, ql=1, hq=32, hkv=4, d=128, lo=19327, hi=19327, page=64, dtype="bf16"),
        # a decode batch with long ragged contexts: bound by reading the cache
        dict(name="attend4-decode-64", op="attend4", B=64, ql=1, hq=32, hkv=8, d=128, lo=1, hi=8190, page=16, dtype="f16"),
        # three drafted positions of a few sequences
        dict(name="weigh-draft-5", op="weigh", B=5, ql=3, hq=44, hkv=4, d=64, lo=3, hi=1500, page=32, dtype="bf16"),
        # one decode step of a batch with long contexts
        dict(name="weigh-decode-64", op="weigh", B=64, ql=1, hq=32, hkv=8, d=128, lo=1, hi=4095, page=16, dtype="f16"),
        # few sequences that have grown past a small budget
        dict(name="evict-4", op="evict", B=4, hkv=4, d=64, lo=700, hi=1501, budget=512, recent=32, page=16, dtype="bf16"),
        # a batch halved when memory is short
        dict(name="evict-64", op="evict", B=64, hkv=8, d=128, lo=1000, hi=8190, budget=2048, recent=256, page=64, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(32, 8, 128), (16, 16, 128), (44, 4, 64), (32, 4, 128), (16, 1, 64), (20, 4, 128)]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "logprobs", "append4", "attend4", "weigh", "evict"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "logprobs":
        T, V = _log(rng, 1, 2047), _log(rng, 100, 131072)
        return dict(op=op, T=T, V=V, top=rng.choice([0, 1, 5, 20]), dtype=rng.choice(["f16", "bf16", "f32"] if T < 1000 else ["f16", "bf16"]))
    hq, hkv, d = rng.choice(_HEADS)
    if op == "prompt":
        B = _log(rng, 1, 200)
        # products of at most 8191^2 positions of 32 heads of 128, and at most 16384 tokens
        hi = min(_log(rng, 1, 8191), int((8191 ** 2 * 4096 / (B * hq * d)) ** 0.5), 16384 // B)
        return dict(op=op, B=B, lo=min(rng.choice([0, 1, 1, 64, hi]), hi), hi=hi, hq=hq, hkv=hkv, d=d, dtype=dtype)
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "append4":
        return dict(op=op, T=_log(rng, 1, 8191), hkv=hkv, d=d, page=page, dtype=dtype)
    B = _log(rng, 1, 256)
    ql = rng.choice([1, 1, 1, 2, 3, 5])
    values = {"attend4": 268, "weigh": 134, "evict": 72}[op] * 1000000  # of all keys
    hi = max(ql, min(_log(rng, 16, 32768), 2 * values // (B * hkv * d)))
    if op == "evict":
        hi = max(hi, 2)
        return dict(op=op, B=B, hkv=hkv, d=d, lo=rng.randint(1, hi), hi=hi, budget=max(1, int(hi * rng.uniform(0.1, 0.9))),
                    recent=rng.choice([0, 1, 16, 100]), page=page, dtype=dtype)
    return dict(op=op, B=B, ql=ql, hq=hq, hkv=hkv, d=d, lo=min(hi, ql + rng.randint(0, 3)), hi=hi, page=page, dtype=dtype)


def _lens(case):
    """Lengths, evenly spread over [lo, hi]."""
    B = case["B"]
    return [case["hi"] - (case["hi"] - case["lo"]) * i // max(1, B - 1) for i in range(B)]


def _quantise(x):
    """The 4-bit form of x [..., d]: codes, and the least value and step of every 32 values, both of x's type."""
    g = x.unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1), g.amax(-1)
    step = ((hi.float() - lo.float()) / 15).to(x.dtype)
    s = step.float()
    code = torch.where(s[..., None] > 0, (g.float() - lo.float()[..., None]) / s[..., None], torch.zeros_like(g, dtype=torch.float32))
    return code.round_().clamp_(0, 15).to(torch.uint8).flatten(-2), lo, step


def _values(code, lo, step):
    g = code.unflatten(-1, (-1, 32)).float()
    return g.mul_(step.float()[..., None]).add_(lo.float()[..., None]).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2 + 1)
    host = torch.Generator().manual_seed(int(seed) * 2 + 1)
    s = {"case": case}
    op, dt = case["op"], _DT[case["dtype"]]

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    if op == "logprobs":
        T, V = case["T"], case["V"]
        x = torch.randn(T, V, generator=gen, device=dev) * 2.5
        # every other row with a part of the vocabulary ruled out, as a grammar does
        x[1::2, : V // 7] = _MINUS
        noise = torch.empty(T, V, device=dev).exponential_(generator=gen)
        s["tokens"] = (x - noise.log_()).argmax(dim=-1).to(torch.int32)
        s["logits"] = x.to(dt)
        s["logprob"], s["entropy"] = torch.empty(T, device=dev), torch.empty(T, device=dev)
        if case["top"]:
            s["ids"] = torch.empty(T, case["top"], dtype=torch.int32, device=dev)
            s["tops"] = torch.empty(T, case["top"], device=dev)
        return s
    hkv, d = case["hkv"], case["d"]
    if op == "prompt":
        hq, lens = case["hq"], _lens(case)
        order = torch.randperm(len(lens), generator=host).tolist()
        s["lens"] = [lens[i] for i in order]
        ends = torch.tensor([0] + s["lens"]).cumsum(0)
        T = int(ends[-1])
        qkv = rand(T, (hq + 2 * hkv) * d, scale=1.4)  # as one projection leaves them
        s["q"] = qkv[:, :hq * d].view(T, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
        s["offsets"] = ends.to(torch.int32).to(dev)
        s["scale"] = d ** -0.5
        s["out"] = torch.empty(T, hq, d, dtype=dt, device=dev)
        s["lse"] = torch.empty(T, hq, device=dev)
        return s
    page = case["page"]
    if op == "append4":
        T = case["T"]
        s["k"], s["v"] = rand(T, hkv, d, scale=2.0), rand(T, hkv, d)
        pages = -(-T // page) + 7
        table = torch.randperm(pages, generator=host)
        t = torch.arange(T) + 3  # the first page is partly filled already
        s["slots"] = (table[t // page] * page + t % page).to(torch.int32).to(dev)
        if own:
            s["kv4"] = _cache4(pages, hkv, page, d, dt, hkv)
            s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    B, lens = case["B"], _lens(case)
    order = torch.randperm(B, generator=host).tolist()
    lens = [lens[i] for i in order]
    need = [-(-n // page) for n in lens]
    fresh = -(-min(case["budget"], case["hi"]) // page) if op == "evict" else 0  # pages a sequence moves to
    pages = torch.randperm(sum(need) + B * fresh + 1, generator=host).to(torch.int32)
    table = torch.zeros(B, max(1, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pages[at:at + n]
        at += n
    s["table"], s["lens"] = table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    k, v = rand(len(pages), hkv, page, d), rand(len(pages), hkv, page, d)
    if op == "attend4":
        hq, ql = case["hq"], case["ql"]
        s["q"] = rand(B * ql, hq, d, scale=2.0)
        s["scale"] = d ** -0.5
        s["out"] = torch.empty(B * ql, hq, d, dtype=dt, device=dev)
        s["lse"] = torch.empty(B * ql, hq, device=dev)
        if own:
            s["kv4"] = kv4 = _cache4(len(pages), hkv, page, d, dt, hq)
            n = len(pages) * page
            slots = torch.arange(n, dtype=torch.int32, device=dev)
            kt, vt = (x.transpose(1, 2).reshape(n, hkv, d) for x in (k, v))
            for i in range(0, n, 1 << 19):
                kv4.append(kt[i:i + (1 << 19)], vt[i:i + (1 << 19)], slots[i:i + (1 << 19)])
            s["ws"] = torch.empty(kv4.attend_workspace_size(B, ql), dtype=torch.uint8, device=dev)
        else:
            s["k4"], s["v4"] = _quantise(k), _quantise(v)
        return s
    s["k"], s["v"] = k, v
    cap = table.shape[1] * page
    # accumulated weights: heavy for a few keys, nothing yet for some
    mass = torch.empty(B, cap, device=dev).exponential_(generator=gen).square_()
    mass[torch.rand(B, cap, generator=gen, device=dev) < 0.1] = 0
    s["mass"], s["mass_out"] = mass, torch.zeros_like(mass)
    if op == "weigh":
        hq, ql = case["hq"], case["ql"]
        s["q"] = rand(B * ql, hq, d, scale=2.0)
        s["scale"], s["decay"] = d ** -0.5, 0.97
        lse = torch.empty(B * ql, hq, dtype=torch.float64, device=dev)
        for b, n in enumerate(lens):  # what attention has left
            kk = k[s["table"][b, :need[b]].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
            q = s["q"][b * ql:(b + 1) * ql].float().view(ql, hkv, hq // hkv, d)
            sc = torch.einsum("jhgd,hnd->jhgn", q, kk) * s["scale"]
            hidden = torch.arange(n, device=dev) > (n - ql + torch.arange(ql, device=dev))[:, None]
            lse[b * ql:(b + 1) * ql] = torch.logsumexp(sc.masked_fill(hidden[:, None, None], _MINUS).double(), -1).reshape(ql, hq)
        s["lse"] = lse.float()
    else:
        s["new_table"] = pages[sum(need):sum(need) + B * fresh].view(B, fresh).clone().to(dev)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
        s["kept"] = torch.empty(B, case["budget"], dtype=torch.int32, device=dev)
    if own:
        import any_precision_expert_gb300 as pw
        s["kv"] = pw.KvCache(k, v, n_heads=case.get("hq", hkv))
        if op == "evict":
            s["ws"] = torch.empty(s["kv"].evict_workspace_size(B, case["budget"]), dtype=torch.uint8, device=dev)
    return s


def _cache4(pages, hkv, page, d, dt, hq):
    import any_precision_expert_gb300 as pw
    codes = [torch.zeros(pages, hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    steps = [torch.zeros(pages, hkv, page, d // 32, 2, dtype=dt, device="cuda") for _ in range(2)]
    return pw.KvCache4(codes[0], codes[1], steps[0], steps[1], n_heads=hq)


def _prompt(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G, at = hq // hkv, 0
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    for n in s["lens"]:
        if n == 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool, device=out.device).triu_(1)
        step = max(1, min(hkv, (1 << 29) // (n * n * G)))  # key heads at a time
        for h in range(0, hkv, step):
            e = min(hkv, h + step)
            q = s["q"][at:at + n, h * G:e * G].float().view(n, e - h, G, d).permute(1, 2, 0, 3)
            k = s["k"][at:at + n, h:e].float().permute(1, 2, 0)[:, None]
            v = s["v"][at:at + n, h:e].float().permute(1, 0, 2)[:, None]
            sc = (q @ k).mul_(s["scale"]).masked_fill_(hidden, _MINUS)
            m = sc.amax(-1, keepdim=True)
            p = sc.sub_(m).exp_()
            total = p.sum(-1, keepdim=True)
            out[at:at + n, h * G:e * G] = ((p @ v) / total).permute(2, 0, 1, 3).reshape(n, -1, d).to(out.dtype)
            lse[at:at + n, h * G:e * G] = (m + total.log())[..., 0].permute(2, 0, 1).reshape(n, -1)
            del sc, p
        at += n
    return {"out": out, "lse": lse}


def _logprobs(s):
    x = s["logits"].float()
    T, V = x.shape
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp_()
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    entropy = (log_total - torch.where(e > 0, e * (x - m), torch.zeros_like(e)).sum(-1, keepdim=True) / total)[:, 0]
    del e
    r = {"logprob": (x.gather(1, s["tokens"].long()[:, None]) - m - log_total)[:, 0], "entropy": entropy}
    if s["case"]["top"]:
        ids = torch.arange(V, dtype=torch.int32, device=x.device)
        best, at = [], []
        left = x.clone()
        for _ in range(s["case"]["top"]):
            top = left.amax(-1, keepdim=True)
            i = torch.where(left == top, ids, V).amin(-1, keepdim=True)
            left.scatter_(1, i.long(), _MINUS)
            best.append(top - m - log_total)
            at.append(i)
        r["ids"], r["tops"] = torch.cat(at, 1).to(torch.int32), torch.cat(best, 1)
    return r


def _seen(s, B, ql, n):
    """[B][ql][n]: the keys that a query sees."""
    last = s["lens"][:, None] - ql + torch.arange(ql, device=s["lens"].device)
    return torch.arange(n, device=last.device) <= last[..., None]


def _attend4(s):
    c = s["case"]
    B, ql, hq, hkv, d = c["B"], c["ql"], c["hq"], c["hkv"], c["d"]
    G, t = hq // hkv, s["table"].long()

    def rows(x):
        return _values(*(y[t] for y in x)).transpose(2, 1).reshape(B, hkv, -1, d)

    k = rows(s["k4"])
    q = s["q"].float().view(B, ql, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, ql * G, d)
    sc = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    del k
    sc.masked_fill_(~_seen(s, B, ql, sc.shape[-1]).repeat_interleave(G, dim=1)[:, None], _MINUS)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ rows(s["v4"])) / total

    def back(x):
        return x.view(B, hkv, ql, G, -1).permute(0, 2, 1, 3, 4).reshape(B * ql, hq, -1)

    return {"out": back(o).to(s["out"].dtype), "lse": back(m + total.log())[..., 0]}


def _weigh(s):
    c = s["case"]
    B, ql, hq, hkv, d = c["B"], c["ql"], c["hq"], c["hkv"], c["d"]
    G = hq // hkv
    k = s["k"][s["table"].long()].float().transpose(2, 1).reshape(B, hkv, -1, d)
    q = s["q"].float().view(B, ql, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, ql * G, d)
    lse = s["lse"].view(B, ql, hkv, G).permute(0, 2, 1, 3).reshape(B, hkv, ql * G, 1)
    sc = (q @ k.transpose(-1, -2)).mul_(s["scale"]).sub_(lse)
    sc.masked_fill_(~_seen(s, B, ql, sc.shape[-1]).repeat_interleave(G, dim=1)[:, None], _MINUS)
    w = sc.exp_().sum(dim=(1, 2))
    held = torch.arange(w.shape[1], device=w.device) < s["lens"][:, None]
    return {"mass": torch.where(held, s["decay"] * s["mass"] + w, s["mass_out"])}


def _evict(s):
    c = s["case"]
    B, budget, recent, page, hkv, d = c["B"], c["budget"], c["recent"], c["page"], c["hkv"], c["d"]
    n = s["lens"].long()[:, None]
    cap = s["mass"].shape[1]
    at = torch.arange(cap, device=n.device)
    left = n.clamp(max=budget)
    # the latest first, then by weight; a stable sort leaves equal ones in order
    score = s["mass"].masked_fill(at >= n - min(recent, budget), float("inf")).masked_fill(at >= n, -1.0)
    order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :budget]
    place = torch.arange(order.shape[1], device=n.device)
    kept = torch.where(place < left, order, cap).sort(dim=1).values  # in their old order
    has = place < left
    src = kept.clamp(max=cap - 1)
    b, j = has.nonzero(as_tuple=True)
    old = src[b, j]
    p0, o0 = s["table"].long()[b, old // page], old % page
    p1, o1 = s["new_table"].long()[b, j // page], j % page
    s["k"][p1, :, o1] = s["k"][p0, :, o0]
    s["v"][p1, :, o1] = s["v"][p0, :, o0]
    mass = torch.zeros_like(s["mass"])
    mass[b, j] = s["mass"][b, old]
    ids = torch.full((B, budget), -1, dtype=torch.int32, device=n.device)
    ids[b, j] = old.to(torch.int32)
    return {"k": s["k"], "v": s["v"], "lens": left[:, 0].to(torch.int32), "mass": mass, "kept": ids}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import any_precision_expert_gb300 as pw
        if op == "prompt":
            pw.prompt_attend(s["q"], s["k"], s["v"], s["offsets"], s["out"], scale=s["scale"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "logprobs":
            pw.token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], top_ids=s.get("ids"),
                              top_logprobs=s.get("tops"))
            return {k: s[k] for k in ("logprob", "entropy", "ids", "tops") if k in s}
        if op == "append4":
            s["kv4"].append(s["k"], s["v"], s["slots"])
            s["kv4"].load(s["slots"], s["k_out"], s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if op == "attend4":
            s["kv4"].attend(s["q"], s["table"], s["lens"], s["out"], s["ws"], q_len=s["case"]["ql"], scale=s["scale"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "weigh":
            s["kv"].weigh(s["q"], s["table"], s["lens"], s["lse"], s["mass"], out=s["mass_out"], q_len=s["case"]["ql"],
                          scale=s["scale"], decay=s["decay"])
            return {"mass": s["mass_out"]}
        s["kv"].evict(s["table"], s["lens"], s["mass"], s["case"]["budget"], s["ws"], recent=s["case"]["recent"],
                      new_table=s["new_table"], new_lens=s["new_lens"], new_mass=s["mass_out"], kept=s["kept"])
        return {"k": s["k"], "v": s["v"], "lens": s["new_lens"], "mass": s["mass_out"], "kept": s["kept"]}
    if op == "append4":
        return {x: _values(*_quantise(s[x])).to(s[x].dtype) for x in ("k", "v")}
    return {"prompt": _prompt, "logprobs": _logprobs, "attend4": _attend4, "weigh": _weigh, "evict": _evict}[op](s)


def work(case):
    op = case["op"]
    if op == "logprobs":
        n = case["T"] * case["V"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["T"] * (12 + 8 * case["top"]), "flops": 5 * n}
    hkv, d = case["hkv"], case["d"]
    row4 = d // 2 + d // 8  # codes, least values and steps
    if op == "append4":
        n = 2 * case["T"] * hkv
        # written in 4 bits, then read back: values in, 4 bits out and in, values out
        return {"bytes": n * (4 * d + 2 * row4) + 8 * case["T"], "flops": 8 * n * d}
    lens = _lens(case)
    keys, B = sum(lens), case["B"]
    if op == "prompt":
        hq = case["hq"]
        return {"bytes": keys * (4 * hq * d + 4 * hkv * d + 4 * hq), "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    if op == "evict":
        left = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": keys * 4 + left * (8 * hkv * d + 8), "flops": keys}
    hq, ql = case["hq"], case["ql"]
    seen = sum(max(0, n - j) for n in lens for j in range(ql))
    if op == "weigh":
        return {"bytes": keys * (2 * hkv * d + 8) + B * ql * hq * (2 * d + 4), "flops": (2 * d + 2) * hq * seen}
    return {"bytes": keys * hkv * 2 * row4 + B * ql * hq * (4 * d + 4), "flops": 4 * d * hq * seen}


def _exact_cached(case, s, rows_of):
    """One sequence and key head at a time: scores in 64 bits [ql][G][n], and what `rows_of` makes of them."""
    B, ql, hq, hkv, d, page = (case[k] for k in ("B", "ql", "hq", "hkv", "d", "page"))
    G = hq // hkv
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-n // page)].long()
        hidden = torch.arange(n, device="cuda")[None] > (n - ql + torch.arange(ql, device="cuda"))[:, None]
        for h in range(hkv):
            k, v = rows_of(pages, h, n)
            q = s["q"][b * ql:(b + 1) * ql, h * G:(h + 1) * G].double()
            sc = (q.reshape(-1, d) @ k.T).view(ql, G, n) * s["scale"]
            yield b, h, sc.masked_fill(hidden[:, None], _MINUS), v


def _unquantised(x):
    """The values a 4-bit row stands for in 64 bits: steps and codes as they are defined, by 32 bit quotients."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    lo = g.min(-1, keepdim=True).values.float()
    step = ((g.max(-1, keepdim=True).values.float() - lo) / 15).to(x.dtype).float()
    code = torch.div(g.float() - lo, step).round()
    code = torch.where(step == 0, torch.zeros_like(code), code.clamp(0, 15))
    return (lo.double() + code.double() * step.double()).reshape(x.shape)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "logprobs":
        x, t = s["logits"], s["tokens"].long()
        T, top = x.shape[0], case["top"]
        r = {"logprob": torch.empty(T, dtype=torch.float64, device=x.device)}
        r["entropy"] = torch.empty_like(r["logprob"])
        if top:
            r["ids"], r["tops"] = None, torch.empty(T, top, dtype=torch.float64, device=x.device)
        for i in range(0, T, 128):
            y = x[i:i + 128].double()
            lp = y - torch.logsumexp(y, -1, keepdim=True)
            r["logprob"][i:i + 128] = lp.gather(1, t[i:i + 128, None])[:, 0]
            r["entropy"][i:i + 128] = -torch.xlogy(lp.exp(), lp.exp()).sum(-1)
            if top:
                r["tops"][i:i + 128] = lp.topk(top, dim=-1).values
        return r
    if op == "append4":
        return {x: _unquantised(s[x]) for x in ("k", "v")}
    if op == "prompt":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        G, at = hq // hkv, 0
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
        for n in s["lens"]:
            for h in range(hkv):
                k, v = s["k"][at:at + n, h].double(), s["v"][at:at + n, h].double()
                for i in range(0, n, 2048):  # rows at a time, up to the last key that they see
                    e = min(n, i + 2048)
                    q = s["q"][at + i:at + e, h * G:(h + 1) * G].double() * s["scale"]
                    sc = torch.einsum("ngd,md->gnm", q, k[:e])
                    sc += torch.full((e - i, e), _MINUS, dtype=torch.float64, device="cuda").triu(i + 1)
                    l = torch.logsumexp(sc, -1)
                    lse[at + i:at + e, h * G:(h + 1) * G] = l.T
                    out[at + i:at + e, h * G:(h + 1) * G] = torch.einsum("gnm,md->ngd", torch.exp(sc - l[..., None]), v[:e])
                    del sc
            at += n
        return {"out": out, "lse": lse}
    if op == "evict":
        return None  # rows are moved, not computed
    hkv, page, d, ql, G = case["hkv"], case["page"], case["d"], case["ql"], case["hq"] // case["hkv"]
    if op == "weigh":
        mass = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            mass[b, :n] = s["decay"] * s["mass"][b, :n].double()
        lse = s["lse"].double()
        for b, h, sc, _ in _exact_cached(case, s, lambda p, h, n: (s["k"][p, h].reshape(-1, d)[:n].double(), None)):
            l = lse[b * ql:(b + 1) * ql, h * G:(h + 1) * G]
            mass[b, :sc.shape[-1]] += torch.exp(sc - l[..., None]).sum(dim=(0, 1))
        return {"mass": mass}
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")

    def held(x, p, h, n):
        code, lo, step = (y[p, h] for y in x)
        g = code.reshape(-1, d // 32, 32).double() * step.reshape(-1, d // 32, 1).double() + lo.reshape(-1, d // 32, 1).double()
        return g.reshape(-1, d)[:n]

    for b, h, sc, v in _exact_cached(case, s, lambda p, h, n: (held(s["k4"], p, h, n), held(s["v4"], p, h, n))):
        l = torch.logsumexp(sc, -1)
        lse[b * ql:(b + 1) * ql, h * G:(h + 1) * G] = l
        out[b * ql:(b + 1) * ql, h * G:(h + 1) * G] = torch.exp(sc - l[..., None]) @ v
    return {"out": out, "lse": lse}
