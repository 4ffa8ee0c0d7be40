"""Cases of the paged FP8 cache operators: what is measured, and their plain form.

Two operators that a serving loop runs one after the other:

  append  the new keys and values of every sequence, their positions rotated
          on the way, quantised into the pages of an e4m3 cache with one
          power-of-two scale for each page and head (the queries of the same
          tokens are rotated in the same call);
  attend  attention of the new tokens' queries over those pages, causal, with
          an optional window and sinks.

Cache layout: codes [pages, Hkv, page, d], scales [pages, Hkv]; a sequence's
token t lies in row t mod page of page page_table[b, t // page].

`run` computes the plain form in elementary torch operations; with `own` set
it calls the library.
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LEAST = 2.0 ** -64  # the least scale a page can have


# ----------------------------------------------------------------- cases

def _append(name, B, n_lo, n_hi, kv_lo, kv_hi, H, Hkv, d, page, rd, dtype="bf16", inter=False):
    return {"name": name, "op": "append", "B": B, "n_lo": n_lo, "n_hi": n_hi, "kv_lo": kv_lo,
            "kv_hi": kv_hi, "H": H, "Hkv": Hkv, "d": d, "page": page, "rd": rd, "dtype": dtype,
            "interleaved": inter}


def _attend(name, B, n_lo, n_hi, kv_lo, kv_hi, H, Hkv, d, page, window=-1, sink=0):
    return {"name": name, "op": "attend", "B": B, "n_lo": n_lo, "n_hi": n_hi, "kv_lo": kv_lo,
            "kv_hi": kv_hi, "H": H, "Hkv": Hkv, "d": d, "page": page, "window": window,
            "sink": sink}


def listed():
    """kv_lo .. kv_hi is what the cache holds before the n_lo .. n_hi new tokens."""
    return [
        # a few interactive users, one new token each: all latency
        _append("append_decode_4", 4, 1, 1, 100, 2000, 32, 8, 128, 64, 128),
        # a full decode batch, pages partly filled
        _append("append_decode_256", 256, 1, 1, 1, 1500, 32, 8, 128, 64, 128),
        # a batch of prompts of odd lengths, some continuing inside a page
        _append("append_prompts_16", 16, 33, 1777, 0, 500, 32, 8, 128, 64, 128),
        # long prompts, fp32 projections, partial interleaved rotation, small pages
        _append("append_long_f32", 4, 7001, 8192, 0, 90, 16, 4, 64, 16, 32, "f32", True),
        # one user, a short context: all latency
        _attend("decode_1", 1, 1, 1, 999, 999, 32, 8, 128, 64),
        # an ordinary decode batch of ragged contexts
        _attend("decode_32", 32, 1, 1, 300, 8191, 32, 8, 128, 64),
        # the largest decode batch: long contexts
        _attend("decode_64_long", 64, 1, 1, 8000, 32767, 32, 8, 128, 128),
        # a sliding-window layer with null-logit sinks, small heads
        _attend("decode_window_128", 128, 1, 1, 5, 9000, 64, 8, 64, 16, 127, 2),
        # drafted tokens checked several at a time
        _attend("verify_32", 32, 3, 5, 1000, 16000, 32, 8, 128, 64, -1, 2),
        # prompts of odd lengths from nothing, with key-0 sinks
        _attend("prompts_16", 16, 61, 1500, 0, 0, 32, 8, 128, 64, -1, 1),
        # a chunk of a long prompt over what is cached already
        _attend("chunk_2048_of_32k", 1, 2048, 2048, 30720, 30720, 32, 8, 128, 64),
        # a whole long prompt, small heads, small pages
        _attend("prompt_8191", 1, 8191, 8191, 0, 0, 16, 4, 64, 32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    Hkv = rng.choice([1, 2, 4, 8, 8])
    G = rng.choice([1, 2, 4, 4, 5, 8])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if rng.random() < 0.4:
        if rng.random() < 0.5:  # one token each
            B, n_lo, n_hi = _log(rng, 1, 400), 1, 1
        else:  # prompts: about 30000 tokens at most
            n_hi = _log(rng, 2, 8192)
            B, n_lo = _log(rng, 1, max(1, 30000 // n_hi)), _log(rng, 1, n_hi)
        kv_hi = _log(rng, 1, max(1, min(4000, 400000 // B)))
        rd = rng.choice([d, d, d // 2, 16])
        return _append("", B, n_lo, n_hi, rng.randrange(kv_hi + 1), kv_hi, Hkv * G, Hkv, d, page,
                       rd, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.3) | {
                           "lens": rng.randrange(1 << 20)}
    window = rng.choice([-1, -1, _log(rng, 16, 4096)])
    sink = rng.choice([0, 0, 1, 2])
    if rng.random() < 0.65:  # decode, sometimes a few drafted tokens
        n_hi = rng.choice([1, 1, 1, 2, 4, 7])
        B = _log(rng, 1, 256)
        kv_hi = _log(rng, 16, max(17, min(32767, 1300000 // B)))
        return _attend("", B, 1, n_hi, rng.randrange(kv_hi), kv_hi, Hkv * G, Hkv, d, page, window,
                       sink) | {"lens": rng.randrange(1 << 20)}
    n_hi = _log(rng, 16, 4096)
    kv_hi = _log(rng, 1, 24000)
    B = _log(rng, 1, max(1, min(16, 40000000 // (n_hi * (kv_hi + n_hi)))))
    return _attend("", B, _log(rng, 1, n_hi), n_hi, rng.randrange(kv_hi), kv_hi, Hkv * G, Hkv, d,
                   page, window, sink) | {"lens": rng.randrange(1 << 20)}


def _lengths(case):
    """[(cached, new)] of the sequences: the extremes first, the others between."""
    r = random.Random(case.get("lens", 7))
    n = [case["n_hi"], case["n_lo"]] + [r.randint(case["n_lo"], case["n_hi"])
                                        for _ in range(case["B"])]
    kv = [case["kv_hi"], case["kv_lo"]] + [r.randint(case["kv_lo"], case["kv_hi"])
                                           for _ in range(case["B"])]
    return list(zip(kv, n))[: case["B"]]


def work(case):
    lens = _lengths(case)
    H, Hkv, d, page = case["H"], case["Hkv"], case["d"], case["page"]
    T = sum(n for _, n in lens)
    if case["op"] == "append":
        e = 4 if case["dtype"] == "f32" else 2
        pages = sum((kv + n - 1) // page - kv // page + 1 for kv, n in lens)
        # keys, values, queries and the table's rows in; codes, scales and queries out
        b = T * (2 * Hkv * d * e + 2 * H * d * e + case["rd"] * 4 + 2 * Hkv * d) + pages * Hkv * 8
        return {"bytes": b, "flops": T * (H + Hkv) * case["rd"] * 3 + 2 * T * Hkv * d * 2}
    w = case["window"]
    pairs = keys = 0
    for kv, n in lens:
        if w < 0:
            pairs += n * kv + n * (n + 1) // 2
            keys += kv + n
        else:
            pairs += sum(min(w + 1, kv + i + 1) for i in range(n))
            keys += min(kv + n, w + n)
    return {"bytes": keys * Hkv * d * 2 + keys // page * Hkv * 8 + T * H * (4 * d + 4),
            "flops": 4 * d * H * pairs}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    lens = _lengths(case)
    B, H, Hkv, d, page = case["B"], case["H"], case["Hkv"], case["d"], case["page"]
    T = sum(n for _, n in lens)
    longest = max(kv + n for kv, n in lens)
    width = -(-longest // page)
    used = [-(-(kv + n) // page) for kv, n in lens]
    pages = sum(used) + 3  # some pages belong to nobody
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    # a sequence's pages lie anywhere in the pool; entries behind its last page are never read
    starts = torch.tensor([0] + used).cumsum(0)
    at = starts[:-1, None] + torch.arange(width)
    at = torch.where(torch.arange(width) < torch.tensor(used)[:, None], at, 0)
    table = order[at.cuda()].contiguous()
    cu = torch.tensor([0] + [n for _, n in lens]).cumsum(0).to(torch.int32).cuda()
    total = torch.tensor([kv + n for kv, n in lens], dtype=torch.int32).cuda()

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    def filled(spread):
        """Pages of earlier tokens: codes of normal values, a scale that fits their largest."""
        codes = torch.empty(pages, Hkv, page, d, dtype=torch.uint8, device="cuda")
        scale = torch.empty(pages, Hkv, device="cuda")
        step = max(1, (1 << 27) // (Hkv * page * d))
        for a in range(0, pages, step):
            m = min(step, pages - a)
            x = normal(m, Hkv, page, d) * (spread * normal(m, Hkv, 1, 1)).exp()
            s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
            scale[a:a + m] = s
            codes[a:a + m] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes, scale

    st = dict(case=case, table=table, cu=cu, total=total, nmax=max(n for _, n in lens),
              lmax=longest)
    st["kc"], st["ks"] = filled(0.2)
    st["vc"], st["vs"] = filled(0.2)
    if case["op"] == "append":
        dt = DT[case["dtype"]]
        # one projection's output, as a model has it: queries, keys and values of a token in a row
        qkv = normal(T, H + 2 * Hkv, d, dtype=dt)
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        rd = case["rd"]
        freq = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
        angle = torch.arange(width * page, dtype=torch.float64, device="cuda")[:, None] * freq
        st["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    else:
        st["q"] = normal(T, H, d, dtype=torch.bfloat16)
        st["sinks"] = normal(H) if case["sink"] else None
    return st


# ----------------------------------------------------------------- plain form

def _positions(st):
    """Sequence and position of every new token."""
    t = torch.arange(st["q"].shape[0], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["cu"], t, right=True) - 1
    return b, st["total"][b] - st["cu"][b + 1] + t


def _rotate(x, rope, pos, rd, interleaved):
    x = x.float()
    cos, sin = rope[pos.long()][:, None, :].split(rd // 2, dim=2)
    if interleaved:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rd // 2], x[..., rd // 2: rd]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rd:]], -1)


def _pow2(amax):
    """The least power of two s, not below LEAST, with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    s = torch.ldexp(torch.ones_like(amax), torch.where(m > 0.875, e - 8, e - 9))
    return torch.where(amax > 0, s, 0.0).clamp_min(LEAST)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _store(codes, scale, x, pid, row, first_pid, kept):
    """Quantise the rows x [T, Hkv, d] into the pages; `first_pid` [B]: the page that
    each sequence's first new token goes to, `kept` [B]: that page held tokens before."""
    P, Hkv = scale.shape
    need = torch.zeros(P, Hkv, device="cuda").scatter_reduce(
        0, pid[:, None].expand(-1, Hkv), _pow2(x.abs().amax(2)), "amax")
    old = scale[first_pid]
    new = scale.clone()
    new[pid] = need[pid]
    new[first_pid] = torch.where(kept[:, None], torch.maximum(old, need[first_pid]),
                                 need[first_pid])
    ratio = torch.where(kept[:, None], old / new[first_pid], 1.0)
    held = codes[first_pid].view(torch.float8_e4m3fn).float() * ratio[:, :, None, None]
    codes[first_pid] = _e4m3(held)
    codes[pid, :, row] = _e4m3(x / new[pid][:, :, None])
    scale.copy_(new)


def _plain_append(st):
    c = st["case"]
    page = c["page"]
    b, pos = _positions(st)
    pid = st["table"][b, pos.long() // page].long()
    n = st["cu"].diff()
    p0 = st["total"] - n
    first = st["table"].gather(1, (p0 // page).long()[:, None])[:, 0].long()
    q = _rotate(st["q"], st["rope"], pos, c["rd"], c["interleaved"]).to(st["q"].dtype)
    k = _rotate(st["k"], st["rope"], pos, c["rd"], c["interleaved"])
    row = (pos % page).long()
    _store(st["kc"], st["ks"], k, pid, row, first, p0 % page > 0)
    _store(st["vc"], st["vs"], st["v"].float(), pid, row, first, p0 % page > 0)
    return q


def _dense(codes, scale, table, L):
    """The cached rows of every sequence, fp32 [B, Hkv, L, d]."""
    t = table.long()
    x = codes[t].view(torch.float8_e4m3fn).float() * scale[t][:, :, :, None, None]
    B, W, Hkv, page, d = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, W * page, d)[:, :, :L]


def _plain_attend(st):
    c = st["case"]
    B, H, Hkv, d, n, L = c["B"], c["H"], c["Hkv"], c["d"], st["nmax"], st["lmax"]
    G = H // Hkv
    k = _dense(st["kc"], st["ks"], st["table"], L)
    v = _dense(st["vc"], st["vs"], st["table"], L)
    T = st["q"].shape[0]
    b, pos = _positions(st)
    i = torch.arange(T, device="cuda", dtype=torch.int32) - st["cu"][b]
    q = torch.zeros(B, n, H, d, device="cuda")
    q[b, i.long()] = st["q"].float()
    q = q.reshape(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    s = (q @ k.transpose(2, 3)).mul_(d ** -0.5).view(B, Hkv, G, n, L)
    at = (st["total"] - st["cu"].diff())[:, None] + torch.arange(n, device="cuda")  # [B, n]
    j = torch.arange(L, device="cuda")
    seen = j <= at[:, :, None]
    if c["window"] >= 0:
        seen &= j >= at[:, :, None] - c["window"]
    sink = None if st["sinks"] is None else st["sinks"].view(Hkv, G, 1, 1)
    if c["sink"] == 1:
        s[..., :1] += sink
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    if c["sink"] == 2:
        m = torch.maximum(m, sink)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    if c["sink"] == 2:
        l = l + (sink - m).exp()
    o = (p.view(B, Hkv, G * n, L) @ v).view(B, Hkv, G, n, d) / l
    lse = m + l.log()
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H, d)[b, i.long()]
    lse = lse.permute(0, 3, 1, 2, 4).reshape(B, n, H)[b, i.long()]
    return o.to(st["q"].dtype), lse


# ----------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    if c["op"] == "append":
        if own:
            import windowed_attention_sinks_gb300 as sa

            q = sa.paged_fp8_append(st["k"], st["v"], st["kc"], st["vc"], st["ks"], st["vs"],
                                    st["table"], st["cu"], st["total"], cos_sin=st["rope"],
                                    interleaved=c["interleaved"], q=st["q"])
        else:
            q = _plain_append(st)
        return {"q": q, "k": st["kc"].view(torch.float8_e4m3fn), "k_scale": st["ks"],
                "v": st["vc"].view(torch.float8_e4m3fn), "v_scale": st["vs"]}
    if own:
        import windowed_attention_sinks_gb300 as sa

        o, lse = sa.paged_fp8_fwd(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"],
                                  st["cu"], st["total"], max_q_len=st["nmax"],
                                  window_left=c["window"], sinks=st["sinks"],
                                  sink_mode=c["sink"])
    else:
        o, lse = _plain_attend(st)
    return {"o": o, "lse": lse}


# ----------------------------------------------------------------- 64 bits

def _value(codes):
    """The values of e4m3 codes, from the format: sign, 4 exponent bits of bias 7, 3 of mantissa."""
    table = []
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        table.append((-x if c & 128 else x) if c & 127 != 127 else float("nan"))
    return torch.tensor(table, dtype=torch.float64, device="cuda")[codes.long()]


def _nearest(x):
    """The e4m3 value nearest to x (ties to the even one, at most 448)."""
    e = torch.frexp(x)[1].clamp_min(-5) - 1
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(st, case):
    H, Hkv, page, rd = case["H"], case["Hkv"], case["page"], case["rd"]
    lens = _lengths(case)
    table, at = st["table"].tolist(), 0
    half = rd // 2
    first = torch.arange(half) * 2 if case["interleaved"] else torch.arange(half)
    second = first + 1 if case["interleaved"] else first + half
    first, second = first.cuda(), second.cuda()

    def turned(x, p):
        c, s = st["rope"][p, :half].double()[:, None], st["rope"][p, half:].double()[:, None]
        y = x.clone()
        y[..., first] = x[..., first] * c - x[..., second] * s
        y[..., second] = x[..., first] * s + x[..., second] * c
        return y

    out = {"q": st["q"].double().clone(), "k": _value(st["kc"]), "k_scale": st["ks"].double(),
           "v": _value(st["vc"]), "v_scale": st["vs"].double()}
    for (kv, n), pages in zip(lens, table):
        p = torch.arange(kv, kv + n, device="cuda")
        out["q"][at:at + n] = turned(st["q"][at:at + n].double(), p)
        for name, rows in (("k", turned(st["k"][at:at + n].double(), p)),
                           ("v", st["v"][at:at + n].double())):
            codes, scale = out[name], out[name + "_scale"]
            lo = kv // page
            hi = (kv + n - 1) // page + 1
            ids = torch.tensor(pages[lo:hi], device="cuda")
            whole = torch.zeros((hi - lo) * page, Hkv, rows.shape[2], dtype=torch.float64,
                                device="cuda")
            whole[kv - lo * page: kv - lo * page + n] = rows
            amax = whole.view(hi - lo, page, Hkv, -1).abs().amax((1, 3))
            s = torch.exp2(torch.ceil(torch.log2(amax / 448))).clamp_min(LEAST)
            if kv % page:
                s[0] = torch.maximum(s[0], scale[ids[0]])
                codes[ids[0]] = _nearest(codes[ids[0]] * (scale[ids[0]] / s[0])[:, None, None])
            scale[ids] = s
            local = torch.arange(kv - lo * page, kv - lo * page + n, device="cuda")
            codes[ids[local // page], :, local % page] = _nearest(rows / s[local // page][..., None])
        at += n
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st, case)
    H, Hkv, page, d, w = case["H"], case["Hkv"], case["page"], case["d"], case["window"]
    G, at = H // Hkv, 0
    T = st["q"].shape[0]
    o = torch.empty(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, H, dtype=torch.float64, device="cuda")
    for b, (kv, n) in enumerate(_lengths(case)):
        L = kv + n
        ids = st["table"][b, : -(-L // page)].long()
        i = torch.arange(kv, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        hidden = (j > i) | ((j < i - w) if w >= 0 else (j < 0))
        for h in range(Hkv):
            k = (_value(st["kc"][ids, h]) * st["ks"][ids, h].double()[:, None, None]).view(-1, d)[:L]
            v = (_value(st["vc"][ids, h]) * st["vs"][ids, h].double()[:, None, None]).view(-1, d)[:L]
            for g in range(h * G, (h + 1) * G):
                s = st["q"][at:at + n, g].double() @ k.T / d ** 0.5
                if case["sink"] == 1:
                    s[:, 0] += st["sinks"][g].double()
                s[hidden] = float("-inf")
                if case["sink"] == 2:
                    extra = st["sinks"][g].double().expand(n, 1)
                    lse[at:at + n, g] = torch.logsumexp(torch.cat([s, extra], 1), 1)
                else:
                    lse[at:at + n, g] = torch.logsumexp(s, 1)
                o[at:at + n, g] = (s - lse[at:at + n, g, None]).exp() @ v
        at += n
    return {"o": o, "lse": lse}
