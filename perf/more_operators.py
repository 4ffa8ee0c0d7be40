"""Cases of the encoder-state operators: what is measured, and their plain form.

What a vision or speech model does with the states of its encoder, next to the
window attention inside that encoder:

  rope     queries and keys rotated by positions with several axes (time,
           height, width), each pair of columns by the axis it belongs to;
  cross    attention of each sequence's queries to encoder states of another
           length: prompts, single tokens, several beams over the same states;
  weights  what each state's key received of those queries' attention, added up
           over queries and the heads of its group;
  evict    the states that received little leave: a sequence keeps its `keep`
           heaviest rows of each KV head, the first and last ones always.

Layouts: q [T, H, d], k and v [S, Hkv, d] (slices of a projection, tokens a stride
apart); sequence b has the queries cu[b] .. cu[b + 1] - 1 and the states starts[b] ..
starts[b] + lens[b] - 1; weights [Hkv, S].

`run` computes the plain form in elementary torch operations; with `own` set
it calls the library.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------- cases

def _rope(name, kind, T, H, Hkv, d, rd, axes, dtype="bf16", inter=False, inverse=False):
    return {"name": name, "op": "rope", "kind": kind, "T": T, "H": H, "Hkv": Hkv, "d": d, "rd": rd,
            "axes": axes, "dtype": dtype, "interleaved": inter, "inverse": inverse}


def _states(name, op, B, n_lo, n_hi, l_lo, l_hi, H, Hkv, d, **more):
    return {"name": name, "op": op, "B": B, "n_lo": n_lo, "n_hi": n_hi, "l_lo": l_lo, "l_hi": l_hi,
            "H": H, "Hkv": Hkv, "d": d, **more}


def _cross(name, B, n_lo, n_hi, l_lo, l_hi, H, Hkv, d, sink=0, pad=False):
    return _states(name, "cross", B, n_lo, n_hi, l_lo, l_hi, H, Hkv, d, sink=sink, pad=pad)


def _weights(name, B, n_lo, n_hi, l_lo, l_hi, H, Hkv, d, add=False):
    return _states(name, "weights", B, n_lo, n_hi, l_lo, l_hi, H, Hkv, d, add=add, pad=False)


def _evict(name, B, l_lo, l_hi, Hkv, d, keep, first, last, dtype="bf16"):
    return _states(name, "evict", B, 0, 0, l_lo, l_hi, Hkv, Hkv, d, keep=keep, first=first,
                   last=last, dtype=dtype, pad=False)


def listed():
    """n_lo .. n_hi: queries of a sequence, l_lo .. l_hi: its encoder states."""
    return [
        # a decode step's tokens of a vision-language model: text behind images, all latency
        _rope("rope_decode_16", "text", 16, 32, 8, 128, 128, 3),
        # a batch of images of odd sizes through a vision encoder, height and width
        _rope("rope_images", "image", 14343, 16, 8, 128, 128, 2),
        # long video: time, height and width, partial rotation of neighbours, fp32, the
        # gradient's direction
        _rope("rope_video_f32", "video", 65521, 16, 16, 64, 48, 3, "f32", True, True),
        # one user asks about one image, a token at a time: all latency
        _cross("cross_decode_1", 1, 1, 1, 1601, 1601, 32, 8, 128),
        # a decode batch over images and videos of many sizes
        _cross("cross_decode_64", 64, 1, 1, 257, 6404, 32, 8, 128, 2),
        # beam search of a speech model, five hypotheses over each padded batch entry
        _cross("cross_beams_24", 24, 5, 5, 331, 1500, 16, 16, 64, 0, True),
        # text prompts of odd lengths beside images
        _cross("cross_prompts_16", 16, 17, 900, 257, 4100, 32, 8, 128, 2),
        # a long document against a long video: the largest
        _cross("cross_long", 1, 4097, 4097, 16411, 16411, 32, 8, 128),
        # the weights that one decode step adds
        _weights("weights_decode_64", 64, 1, 1, 257, 6404, 32, 8, 128, True),
        # the weights of whole prompts
        _weights("weights_prompts_8", 8, 100, 2000, 1000, 8000, 32, 8, 128),
        # a few videos down to 1024 rows each
        _evict("evict_8", 8, 3001, 8191, 8, 128, 1024, 16, 64),
        # many long ones, a quarter kept, small heads
        _evict("evict_64", 64, 1000, 16000, 4, 64, 4000, 4, 256),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "cross", "cross", "weights", "evict"])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 1, 2, 4, 4, 5, 8])
    d = rng.choice([64, 128, 128])
    lens = {"lens": rng.randrange(1 << 20)}
    if op == "rope":
        kind = rng.choice(["text", "image", "video"])
        T = _log(rng, 1, max(1, min(65000, 1500000 // (Hkv * (G + 1)))))
        return _rope("", kind, T, Hkv * G, Hkv, d, rng.choice([d, d, d // 2, 48, 16]),
                     2 if kind == "image" else 3, rng.choice(["bf16", "bf16", "f32"]),
                     rng.random() < 0.4, rng.random() < 0.3) | lens
    if op == "evict":
        l_hi = _log(rng, 2, 16000)
        B = _log(rng, 1, max(1, min(64, 60000000 // (2 * l_hi * Hkv * d))))
        keep = rng.randrange(1, l_hi + 1)
        first = rng.randrange(0, keep // 2 + 1)
        return _evict("", B, rng.randrange(l_hi), l_hi, Hkv, d, keep, first,
                      rng.randrange(0, keep - first + 1) // 2,
                      rng.choice(["bf16", "bf16", "f32"])) | lens
    n_hi = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 4096)])
    l_hi = _log(rng, 16, 16384)
    # at most as many rows and products as the largest case
    B = _log(rng, 1, max(1, min(128, 200000000 // (l_hi * Hkv * d),
                                150000000 // (n_hi * Hkv * G * d),
                                1600000000 // (n_hi * l_hi * Hkv * G))))
    n_lo, l_lo = _log(rng, 1, n_hi), rng.randrange(l_hi)
    if op == "weights":
        return _weights("", B, n_lo, n_hi, l_lo, l_hi, Hkv * G, Hkv, d, rng.random() < 0.5) | lens
    return _cross("", B, n_lo, n_hi, l_lo, l_hi, Hkv * G, Hkv, d, rng.choice([0, 0, 1, 2]),
                  rng.random() < 0.3) | lens


def _lengths(case):
    """[(queries, states)] of the sequences: the extremes first, the others between."""
    r = random.Random(case.get("lens", 7))
    n = [case["n_hi"], case["n_lo"]] + [r.randint(case["n_lo"], case["n_hi"])
                                        for _ in range(case["B"])]
    l = [case["l_hi"], case["l_lo"]] + [r.randint(case["l_lo"], case["l_hi"])
                                        for _ in range(case["B"])]
    return list(zip(n, l))[: case["B"]]


def work(case):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        e = 4 if case["dtype"] == "f32" else 2
        T, rd = case["T"], case["rd"]
        # queries and keys in and out, a position an axis
        return {"bytes": T * ((H + Hkv) * d * e * 2 + case["axes"] * 4),
                "flops": T * (H + Hkv) * rd * 3}
    lens = _lengths(case)
    T, S = sum(n for n, _ in lens), sum(l for _, l in lens)
    pairs = sum(n * l for n, l in lens)
    if case["op"] == "cross":
        return {"bytes": S * Hkv * d * 4 + T * H * (4 * d + 4), "flops": 4 * d * H * pairs}
    if case["op"] == "weights":
        return {"bytes": S * Hkv * (2 * d + 4 * (1 + case["add"])) + T * H * (2 * d + 4),
                "flops": 2 * d * H * pairs}
    e = 4 if case["dtype"] == "f32" else 2
    kept = sum(min(l, case["keep"]) for _, l in lens)
    # the weights in; kept keys and values in; the outputs, padded rows among them
    return {"bytes": Hkv * (S * 4 + kept * 2 * d * e + len(lens) * case["keep"] * (2 * d * e + 8)),
            "flops": S * Hkv}


# ----------------------------------------------------------------- inputs

def _grid(case, r):
    """Positions [axes, T] of text and of images or video frames of odd sizes, one after another."""
    T, axes = case["T"], case["axes"]
    if case["kind"] == "text":  # behind long contexts, the same on every axis
        at = [r.randrange(200000) for _ in range(T)]
        return torch.tensor([at] * axes, dtype=torch.int32)
    parts, have, t0 = [], 0, r.randrange(1000)
    while have < T:
        h, w = r.randrange(9, 73), r.randrange(9, 73)
        f = r.randrange(8, 64) if case["kind"] == "video" else 1
        p = torch.stack(torch.meshgrid(t0 + 25 * torch.arange(f), torch.arange(h), torch.arange(w),
                                       indexing="ij")).reshape(3, -1)
        parts.append(p)
        have += p.shape[1]
        t0 += 25 * f
    return torch.cat(parts, 1)[3 - axes:, :T].to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    st = dict(case=case)
    if case["op"] == "rope":
        r = random.Random(case.get("lens", 7) * 1000003 + seed)
        # one projection's output: queries, keys and values of a token in a row
        qkv = normal(case["T"], H + 2 * Hkv, d, dtype=DT[case["dtype"]])
        st["q"], st["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        st["pos"] = _grid(case, r).cuda()
        half, axes = case["rd"] // 2, case["axes"]
        st["freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        # video and text: a quarter of the pairs for time, the rest for height and width in
        # turns; images: height, then width
        i = torch.arange(half)
        axis = (i >= half // 2).int() if axes == 2 else torch.where(i < half // 4, 0, 1 + i % 2)
        st["axis"] = axis.to(torch.uint8).cuda()
        return st
    lens = _lengths(case)
    n, l = [a for a, _ in lens], [b for _, b in lens]
    T = sum(n)
    longest = max(l)
    starts = [b * longest for b in range(len(l))] if case["pad"] else \
        [sum(l[:b]) for b in range(len(l))]
    S = max(1, len(l) * longest if case["pad"] else sum(l))
    st.update(nmax=max(n), lmax=longest, S=S, T=T)
    st["cu"] = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32).cuda()
    st["starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
    st["lens"] = torch.tensor(l, dtype=torch.int32).cuda()
    dt = DT[case.get("dtype", "bf16")]
    kv = normal(S, 2 * Hkv, d, dtype=dt)  # one projection's output
    st["k"], st["v"] = kv[:, :Hkv], kv[:, Hkv:]
    if case["op"] == "evict":
        # sums over many queries: a few rows are heavy, some are equal (never attended)
        w = normal(Hkv, S).mul_(1.5).exp_()
        st["w"] = torch.where(normal(Hkv, S) > 1.2, 0.0, w)
        return st
    st["q"] = normal(T, H, d, dtype=dt) * 1.5
    st["sinks"] = normal(H) if case.get("sink") else None
    if case["op"] == "weights":
        st["lse"] = _plain_cross(st)[1]
        st["w"] = normal(Hkv, S).exp_() if case["add"] else torch.zeros(Hkv, S, device="cuda")
    return st


# ----------------------------------------------------------------- plain form

def _plain_rope(st):
    c = st["case"]
    rd, half = c["rd"], c["rd"] // 2
    angle = (st["pos"].double()[st["axis"].long()] * st["freq"].double()[:, None]).T
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin
    out = []
    for x in (st["q"], st["k"]):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:rd:2], y[..., 1:rd:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rd]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out.append(torch.cat([r, y[..., rd:]], -1).to(x.dtype))
    return {"q": out[0], "k": out[1]}


def _rows(st):
    """Sequence and place within it of every query; the states' rows [B, L] and which there are."""
    t = torch.arange(st["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["cu"], t, right=True) - 1
    i = (t - st["cu"][b]).long()
    j = torch.arange(st["lmax"], device="cuda")
    at = (st["starts"][:, None] + j).clamp_max(st["S"] - 1).long()
    return b, i, at, j < st["lens"][:, None]


def _scores(st, b, i, at):
    """Logits of the padded batch, [B, Hkv, G, n, L]."""
    c = st["case"]
    B, H, Hkv, d, n, L = c["B"], c["H"], c["Hkv"], c["d"], st["nmax"], st["lmax"]
    q = torch.zeros(B, n, H, d, device="cuda")
    q[b, i] = st["q"].float()
    q = q.reshape(B, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    k = st["k"][at].float().permute(0, 2, 3, 1)
    return (q @ k).mul_(d ** -0.5).view(B, Hkv, H // Hkv, n, L)


def _packed(x, b, i, H):
    """[B, Hkv, G, n, ...] to the packed [T, H, ...]."""
    x = x.movedim(3, 1)
    return x.reshape(x.shape[:2] + (H,) + x.shape[4:])[b, i]


def _plain_cross(st):
    c = st["case"]
    Hkv, G = c["Hkv"], c["H"] // c["Hkv"]
    b, i, at, there = _rows(st)
    sink = None if st["sinks"] is None else st["sinks"].view(Hkv, G, 1, 1)
    s = _scores(st, b, i, at)
    if c.get("sink") == 1:
        s[..., :1] += sink
    s.masked_fill_(~there[:, None, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full(s.shape[:-1] + (1,), -math.inf)
    if c.get("sink") == 2:
        m = torch.maximum(m, sink)
    # a sequence without states: no weight anywhere
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = p.sum(-1, keepdim=True)
    if c.get("sink") == 2:
        l = l + (sink - m).exp()
    v = st["v"][at].float().permute(0, 2, 1, 3)
    o = (p.flatten(2, 3) @ v).view(p.shape[:4] + (c["d"],)) / torch.where(l > 0, l, 1.0)
    lse = (m + l.log())[..., 0]
    return _packed(o, b, i, c["H"]).to(st["q"].dtype), _packed(lse, b, i, c["H"])


def _plain_weights(st):
    c = st["case"]
    Hkv, H = c["Hkv"], c["H"]
    b, i, at, there = _rows(st)
    s = _scores(st, b, i, at)
    lse = torch.full((c["B"], st["nmax"], H), math.inf, device="cuda")  # no query: no weight
    lse[b, i] = st["lse"]
    lse = lse.view(c["B"], -1, Hkv, H // Hkv).permute(0, 2, 3, 1)[..., None]
    w = s.sub_(lse).exp_().sum((2, 3))  # [B, Hkv, L]
    out = st["w"].clone()
    sum_, rows = w.movedim(1, 0)[:, there], at[there]
    out[:, rows] = out[:, rows] + sum_ if c["add"] else sum_
    return {"weights": out}


def _plain_evict(st):
    c = st["case"]
    B, Hkv, d, keep = c["B"], c["Hkv"], c["d"], c["keep"]
    L = st["lmax"]
    _, _, at, there = _rows(st)
    j = torch.arange(L, device="cuda")
    always = (j < c["first"]) | (j >= st["lens"][:, None] - c["last"])
    w = st["w"][:, at].movedim(1, 0)  # [B, Hkv, L]
    key = torch.where(w > 0, w, 0.0)
    key = torch.where(always[:, None], math.inf, key)
    key = torch.where(there[:, None], key, -1.0)
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = st["lens"].clamp_max(keep)
    m = order.shape[-1]
    slot = torch.arange(m, device="cuda")
    rows = torch.where(slot < kept[:, None, None], order, L).sort(dim=-1).values
    live = rows < L
    src = torch.where(live, rows, 0)
    full = torch.zeros(B, Hkv, keep, dtype=torch.int32, device="cuda") - 1
    full[..., :m] = torch.where(live, rows, -1).int()
    wout = torch.zeros(B, Hkv, keep, device="cuda")
    wout[..., :m] = torch.where(live, w.gather(2, src), 0.0)
    where = st["starts"][:, None, None] + src
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    out = {}
    for name in "kv":
        y = torch.zeros(B, keep, Hkv, d, dtype=st[name].dtype, device="cuda")
        y[:, :m] = torch.where(live[..., None], st[name][where.clamp_max(st["S"] - 1), head],
                               0.0).movedim(1, 2)
        out[name] = y.view(B * keep, Hkv, d)
    out["weights"] = wout.movedim(1, 0).reshape(Hkv, B * keep)
    out["rows"] = full.movedim(1, 0).reshape(Hkv, B * keep)
    out["starts"] = torch.arange(B, device="cuda", dtype=torch.int32) * keep
    out["lens"] = kept
    return out


# ----------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "cross":
            o, lse = _plain_cross(st)
            return {"o": o, "lse": lse}
        return {"rope": _plain_rope, "weights": _plain_weights, "evict": _plain_evict}[op](st)
    import windowed_attention_sinks_gb300 as sa

    if op == "rope":
        q, k = sa.rope_axes(st["q"], st["k"], st["pos"], st["freq"], st["axis"],
                            interleaved=c["interleaved"], inverse=c["inverse"])
        return {"q": q, "k": k}
    if op == "cross":
        o, lse = sa.cross_fwd(st["q"], st["k"], st["v"], st["cu"], st["starts"], st["lens"],
                              max_q_len=st["nmax"], sinks=st["sinks"], sink_mode=c["sink"])
        return {"o": o, "lse": lse}
    if op == "weights":
        w = st["w"].clone() if c["add"] else st["w"]
        return {"weights": sa.cross_key_weights(st["q"], st["k"], st["lse"], st["cu"],
                                                st["starts"], st["lens"], w,
                                                max_q_len=st["nmax"], accumulate=c["add"])}
    k, v, w, rows, starts, lens = sa.evict_keys(st["k"], st["v"], st["w"], st["starts"],
                                                st["lens"], c["keep"], first=c["first"],
                                                last=c["last"])
    return {"k": k, "v": v, "weights": w, "rows": rows, "starts": starts, "lens": lens}


# ----------------------------------------------------------------- 64 bits

def _exact_rope(st):
    """Each pair of columns as a complex number, multiplied by e^(i angle)."""
    c = st["case"]
    rd, half = c["rd"], c["rd"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    out = {}
    for name in ("q", "k"):
        x = st[name]
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for a in range(0, c["T"], 8192):
            part = x[a:a + 8192].double()
            z = part.clone()
            for axis in range(c["axes"]):
                mine = (st["axis"] == axis).nonzero()[:, 0]
                angle = st["pos"][axis, a:a + 8192].double()[:, None] * st["freq"][mine].double()
                turn = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle)
                pair = torch.complex(part[..., first[mine]], part[..., second[mine]])
                pair = pair * turn[:, None]
                z[..., first[mine]], z[..., second[mine]] = pair.real, pair.imag
            y[a:a + 8192] = z
        out[name] = y
    return out


def _exact_evict(st):
    c = st["case"]
    keep = c["keep"]
    wh, lens = st["w"].double().cpu().numpy(), st["lens"].tolist()
    S = c["B"] * keep
    k = torch.zeros(S, c["Hkv"], c["d"], dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    w = torch.zeros(c["Hkv"], S, dtype=torch.float64, device="cuda")
    rows = torch.full((c["Hkv"], S), -1, dtype=torch.int32, device="cuda")
    for b, (s, l) in enumerate(zip(st["starts"].tolist(), lens)):
        safe = set(range(min(l, c["first"]))) | set(range(max(0, l - c["last"]), l))
        for h in range(c["Hkv"]):
            x = wh[h, s:s + l].tolist()
            order = sorted(range(l), key=lambda j: (j not in safe, -x[j], j))
            kept = torch.tensor(sorted(order[:keep]), dtype=torch.long, device="cuda")
            to = slice(b * keep, b * keep + len(kept))
            k[to, h], v[to, h] = st["k"][s + kept, h].double(), st["v"][s + kept, h].double()
            w[h, to], rows[h, to] = st["w"][h, s + kept].double(), kept.int()
    return {"k": k, "v": v, "weights": w, "rows": rows,
            "starts": torch.tensor([b * keep for b in range(c["B"])], dtype=torch.int32),
            "lens": torch.tensor([min(l, keep) for l in lens], dtype=torch.int32)}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(st)
    if op == "evict":
        return _exact_evict(st)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    G, T = H // Hkv, st["T"]
    o = torch.zeros(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    w = st["w"].double() if op == "weights" else None
    t = 0
    for (n, l), s0 in zip(_lengths(case), st["starts"].tolist()):
        for h in range(Hkv):
            k = st["k"][s0:s0 + l, h].double()
            total = torch.zeros(l, dtype=torch.float64, device="cuda")
            for a in range(h * G, (h + 1) * G):
                x = st["q"][t:t + n, a].double() @ k.T / math.sqrt(d)
                if op == "weights":
                    total += (x - st["lse"][t:t + n, a, None].double()).exp().sum(0)
                    continue
                if case["sink"] == 1:
                    x[:, :1] += st["sinks"][a].double()
                if case["sink"] == 2:
                    extra = st["sinks"][a].double().expand(n, 1)
                    z = torch.logsumexp(torch.cat([x, extra], 1), 1)
                else:
                    z = torch.logsumexp(x, 1)
                lse[t:t + n, a] = z
                if l:
                    o[t:t + n, a] = (x - z[:, None]).exp() @ st["v"][s0:s0 + l, h].double()
            if op == "weights":
                w[h, s0:s0 + l] = total + (w[h, s0:s0 + l] if case["add"] else 0)
        t += n
    return {"weights": w} if op == "weights" else {"o": o, "lse": lse}
