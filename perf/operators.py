"""Cases that measure the attention operators: rotary positions over several
axes with the norms of queries and keys in the same pass, and attention over
packed sequences, each forward and backward.

With ``own`` false, ``run`` computes them in plain form: elementary torch
operations in 32 bits, rounded once at the end. With ``own`` true it makes the
library's calls. Sequence lengths are a text in the case ("80x80*4" is four
sequences of 6400 tokens), so that a case says all of its sizes.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # one new token for each of 8 requests of a captioning decoder: latency
        dict(name="rotary_tokens_bf16", op="rotary", dtype="bf16", grid="1x1x8", start=4096, q_heads=32, k_heads=8, dim=128, sections="24,20,20", layout="half", norm=True, fused=True),
        # the neck's feature maps (4 images of 80 x 80, 128 channels) as tokens of 2 heads
        dict(name="rotary_neck_f16", op="rotary", dtype="f16", grid="4x80x80", start=0, q_heads=2, k_heads=2, dim=64, sections="0,16,16", layout="blocks", norm=True, fused=True),
        # a clip of 8 frames of 64 x 64 patches: the largest forward
        dict(name="rotary_video_bf16", op="rotary", dtype="bf16", grid="8x64x64", start=0, q_heads=32, k_heads=8, dim=128, sections="24,20,20", layout="half", norm=True, fused=True),
        # training in float32 on odd sizes, neighbouring pairs, part of each head unrotated
        dict(name="rotary_bwd_odd_f32", op="rotary_backward", dtype="f32", grid="3x41x37", start=0, q_heads=12, k_heads=3, dim=80, sections="8,13,13", layout="interleaved", norm=True, fused=True),
        # training on 4 frames of 64 x 64 patches
        dict(name="rotary_bwd_video_bf16", op="rotary_backward", dtype="bf16", grid="4x64x64", start=0, q_heads=32, k_heads=8, dim=128, sections="24,20,20", layout="half", norm=True, fused=True),
        # one new token for each of 16 requests against prompts of different lengths in a cache
        dict(name="attn_token_bf16", op="attention", dtype="bf16", q="1*16", k="8192*3,7001,6400*2,5000,4097,4096*3,2500,1600,1024,129,1", slack=8192, q_heads=32, k_heads=8, dim=128, causal=True),
        # every pixel of the neck's feature map attends to its whole image
        dict(name="attn_neck_f16", op="attention", dtype="f16", q="80x80*4", k="80x80*4", slack=0, q_heads=2, k_heads=2, dim=64, causal=False),
        # a batch of packed prompts, from one token to long ones: the largest forward
        dict(name="attn_packed_bf16", op="attention", dtype="bf16", q="8192*2,6400,4096,2500,1600*2,1024,511,129,17,1", k="8192*2,6400,4096,2500,1600*2,1024,511,129,17,1", slack=0, q_heads=32, k_heads=8, dim=128, causal=True),
        # small feature maps in float32, shared key heads
        dict(name="attn_maps_f32", op="attention", dtype="f32", q="32x32,25x25,16x16*3,7x5", k="32x32,25x25,16x16*3,7x5", slack=0, q_heads=8, k_heads=4, dim=40, causal=False),
        # training on the large-channel maps: 16 images of 32 x 32, 512 channels as 8 heads
        dict(name="attn_bwd_largec_f16", op="attention_backward", dtype="f16", q="32x32*16", k="32x32*16", slack=0, q_heads=8, k_heads=8, dim=64, causal=False),
        # training on packed prompts with shared key heads: the largest backward
        dict(name="attn_bwd_packed_bf16", op="attention_backward", dtype="bf16", q="6400,4096,2500,1600,1024,511,129,17,1", k="6400,4096,2500,1600,1024,511,129,17,1", slack=0, q_heads=32, k_heads=8, dim=128, causal=True),
        # training in float32 on ragged lengths; the first rows of one sequence see no key
        dict(name="attn_bwd_ragged_f32", op="attention_backward", dtype="f32", q="700,333,90,1", k="700,401,50,9", slack=0, q_heads=6, k_heads=2, dim=72, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    group = rng.choice([1, 2, 3, 4, 8])
    k_heads = _log(rng, 1, 8)
    q_heads = k_heads * group
    dim = 8 * rng.randint(4, 16)
    if rng.random() < 0.4:
        op = rng.choice(["rotary", "rotary_backward"])
        # at most 8 x 64 x 64 tokens of 40 heads of 128 in 16 bits, for the backward half of that
        room = 8 * 64 * 64 * 40 * 128 // (2 if op == "rotary_backward" else 1) // (2 if dtype == "f32" else 1)
        tokens = _log(rng, 1, max(2, room // ((q_heads + k_heads) * dim)))
        h = _log(rng, 1, max(1, math.isqrt(tokens)))
        w = _log(rng, 1, max(1, math.isqrt(tokens)))
        pairs = rng.choice([dim // 2, dim // 2, rng.randint(3, dim // 2)])
        a = rng.randint(0, pairs // 2)
        b = rng.randint(0, pairs - a)
        return dict(op=op, dtype=dtype, grid="%dx%dx%d" % (max(1, tokens // (h * w)), h, w), start=_log(rng, 1, 4096) - 1, q_heads=q_heads, k_heads=k_heads, dim=dim, sections="%d,%d,%d" % (a, b, pairs - a - b), layout=rng.choice(["half", "interleaved", "blocks"]), norm=rng.random() < 0.7, fused=rng.random() < 0.7)
    op = rng.choice(["attention", "attention", "attention_backward"])
    # the score products of the largest listed cases (in float32 a fortieth of them)
    room = (2.6e11 if op == "attention" else 0.8e11) / (40 if dtype == "f32" else 1)
    if op == "attention" and rng.random() < 0.4:  # new tokens, one or a few for each request
        batch = _log(rng, 1, 32)
        most = 8192 * 8 // k_heads
        lens = [min(_log(rng, 1, 8192), max(1, most * 12 // batch)) for _ in range(batch)]
        new = rng.choice([1, 1, 1, rng.randint(2, 9)])
        return dict(op=op, dtype=dtype, q="%d*%d" % (new, batch), k=",".join(map(str, lens)), slack=rng.choice([0, max(lens) + rng.randint(0, 300)]), q_heads=q_heads, k_heads=k_heads, dim=dim, causal=True)
    causal = rng.random() < 0.5
    q, k, left = [], [], room / (dim * q_heads)
    for _ in range(_log(rng, 1, 16)):
        n = _log(rng, 1, min(8192, max(2, math.isqrt(int(max(4, left))))))
        m = n if rng.random() < 0.8 else max(1, n + rng.randint(-n // 2, n // 2))
        if n * m > left:
            break
        left -= n * m
        q.append(n)
        k.append(m)
    q, k = q or [64], k or [64]
    return dict(op=op, dtype=dtype, q=",".join(map(str, q)), k=",".join(map(str, k)), slack=0, q_heads=q_heads, k_heads=k_heads, dim=dim, causal=causal)


def _lengths(text):
    """"8192*2,32x32" -> [8192, 8192, 1024]"""
    out = []
    for part in text.split(","):
        size, _, times = part.partition("*")
        n = 1
        for f in size.split("x"):
            n *= int(f)
        out += [n] * int(times or 1)
    return out


def _grid(case):
    return [int(n) for n in case["grid"].split("x")]


def _sections(case):
    return [int(n) for n in case["sections"].split(",")]


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    if case["op"].startswith("rotary"):
        t, h, w = _grid(case)
        n = t * h * w
        if case["fused"]:  # one projection's output holds queries, keys and values
            qkv = _normal(g, n, hq + 2 * hk, d).to(dt)
            q, k = qkv[:, :hq], qkv[:, hq : hq + hk]
        else:
            q, k = _normal(g, n, hq, d).to(dt), _normal(g, n, hk, d).to(dt)
        i = torch.arange(n, device="cuda")
        positions = torch.stack([i // (h * w) + case["start"], i // w % h, i % w], 1).to(torch.int32).contiguous()
        sections = _sections(case)
        freq = torch.cat([10000.0 ** (-torch.arange(s, device="cuda", dtype=torch.float32) / max(s, 1)) for s in sections])
        s = dict(q=q, k=k, positions=positions, freq=freq, sections=sections, layout=case["layout"], norm=case["norm"], qw=None, kw=None)
        if case["norm"]:
            s["qw"] = (1 + 0.2 * _normal(g, d)).to(dt)
            s["kw"] = (1 + 0.2 * _normal(g, d)).to(dt)
        if case["op"] == "rotary_backward":
            s["gq"], s["gk"] = _normal(g, n, hq, d).to(dt), _normal(g, n, hk, d).to(dt)
    else:
        ql, kl = _lengths(case["q"]), _lengths(case["k"])
        room = [case["slack"] or n for n in kl]  # a cache has room for `slack` tokens of each request
        tq, tk = sum(ql), sum(room)
        starts = lambda ls: torch.tensor([sum(ls[:i]) for i in range(len(ls) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
        s = dict(q=_normal(g, tq, hq, d).to(dt), k=_normal(g, tk, hk, d).to(dt), v=_normal(g, tk, hk, d).to(dt), ql=ql, kl=kl, room=room, qs=starts(ql), ks=starts(room), kn=None)
        if case["slack"]:
            s["kn"] = torch.tensor(kl, dtype=torch.int32, device="cuda")
        s.update(causal=case["causal"], scale=d**-0.5)
        if case["op"] == "attention_backward":
            s["g"] = _normal(g, tq, hq, d).to(dt)
            s["out"], s["lse"] = _attention(s)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------- plain forms
def _pair_index(sections, layout, d, device):
    """Elements (lo, hi) of each of the d/2 pairs; those after the sections stay as they are."""
    p = sum(sections)
    i = torch.arange(p, device=device)
    if layout == "half":
        lo, hi = i, i + p
    elif layout == "interleaved":
        lo, hi = 2 * i, 2 * i + 1
    else:  # each section's own block, in halves
        size = torch.repeat_interleave(torch.tensor(sections, device=device), torch.tensor(sections, device=device), output_size=p)
        first = torch.repeat_interleave(torch.tensor([sum(sections[:a]) for a in range(len(sections))], device=device), torch.tensor(sections, device=device), output_size=p)
        lo, hi = i + first, i + first + size
    return lo, hi


def _rotate(x, s, sign):
    """x [tokens, heads, d] in 32 bits, each pair turned by sign * position * frequency."""
    sections = s["sections"]
    lo, hi = _pair_index(sections, s["layout"], x.shape[-1], x.device)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device), torch.tensor(sections, device=x.device), output_size=sum(sections))
    angle = sign * s["positions"].float()[:, axis] * s["freq"]
    c, z = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., lo], x[..., hi]
    y = x.clone()
    y[..., lo] = a * c - b * z
    y[..., hi] = b * c + a * z
    return y


def _normed(x, w, s):
    if not s["norm"]:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotary(s):
    return tuple(_rotate(_normed(s[x].float(), s[x + "w"], s), s, 1).to(s[x].dtype) for x in ("q", "k"))


def _rotary_backward_one(x, w, gy, s):
    g = _rotate(gy.float(), s, -1)
    if not s["norm"]:
        return g.to(x.dtype), None
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    n = xf * r
    gw = (g * n).sum((0, 1))
    g = g * w.float()
    return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(x.dtype), gw.to(w.dtype)


def _rotary_backward(s):
    gq, gqw = _rotary_backward_one(s["q"], s["qw"], s["gq"], s)
    gk, gkw = _rotary_backward_one(s["k"], s["kw"], s["gk"], s)
    out = {"q": gq, "k": gk}
    if s["norm"]:
        out.update(q_weight=gqw, k_weight=gkw)
    return out


def _batches(s):
    """The sequences as padded batches: all in one where their scores take at most 4 GB, else each alone."""
    ql, kl = s["ql"], s["kl"]
    n = len(ql)
    if n * max(ql) * max(kl) * s["q"].shape[1] <= 1 << 30:
        return [list(range(n))]
    return [[i] for i in range(n)]


def _padded(s, batch):
    """Rows of q and of k for a padded batch, and which (query, key) pairs see each other."""
    dev = s["q"].device
    ql = torch.tensor([s["ql"][i] for i in batch], device=dev)
    kl = torch.tensor([s["kl"][i] for i in batch], device=dev)
    i = torch.arange(max(s["ql"][b] for b in batch), device=dev)
    j = torch.arange(max(s["kl"][b] for b in batch), device=dev)
    qrow = torch.where(i < ql[:, None], s["qs"][batch[0] : batch[-1] + 1, None] + i, -1)
    krow = torch.where(j < kl[:, None], s["ks"][batch[0] : batch[-1] + 1, None] + j, -1)
    seen = (i < ql[:, None])[:, :, None] & (j < kl[:, None])[:, None]
    if s["causal"]:
        seen = seen & (j[None, None, :] <= i[None, :, None] + (kl - ql)[:, None, None])
    return qrow, krow, seen


def _heads(x, rows, groups=1):
    """[sequences, heads, rows, d] in 32 bits; rows of -1 are zero."""
    y = x[rows.clamp(min=0)].float() * (rows >= 0)[..., None, None]
    y = y.permute(0, 2, 1, 3)
    return y.repeat_interleave(groups, 1) if groups > 1 else y


def _attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    groups = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float32, device=q.device)
    lse = torch.full((q.shape[1], q.shape[0]), -math.inf, device=q.device)
    for batch in _batches(s):
        qrow, krow, seen = _padded(s, batch)
        p = _heads(q, qrow) @ _heads(k, krow, groups).transpose(-1, -2) * s["scale"]
        p = p.masked_fill_(~seen[:, None], -math.inf)
        m = p.amax(-1, keepdim=True).clamp(min=-3e38)
        p = torch.exp(p - m)
        total = p.sum(-1, keepdim=True)
        o = (p @ _heads(v, krow, groups)) / total.clamp(min=1e-38)
        at = qrow >= 0
        out[qrow[at]] = o.permute(0, 2, 1, 3)[at]
        lse[:, qrow[at]] = (m + torch.log(total))[..., 0].permute(0, 2, 1)[at].T
    return out.to(q.dtype), lse


def _attention_backward(s):
    q, k, v = s["q"], s["k"], s["v"]
    hk = k.shape[1]
    groups = q.shape[1] // hk
    gq, gk, gv = (torch.zeros(x.shape, dtype=torch.float32, device=x.device) for x in (q, k, v))
    for batch in _batches(s):
        qrow, krow, seen = _padded(s, batch)
        qh, kh, vh, gh = _heads(q, qrow), _heads(k, krow, groups), _heads(v, krow, groups), _heads(s["g"], qrow)
        delta = (gh * _heads(s["out"], qrow)).sum(-1, keepdim=True)
        lse = s["lse"][:, qrow.clamp(min=0)].permute(1, 0, 2)[..., None]
        p = torch.exp(qh @ kh.transpose(-1, -2) * s["scale"] - lse)
        p = p.masked_fill_(~seen[:, None], 0.0)
        shared = lambda x: x.unflatten(1, (hk, groups)).sum(2)  # noqa: E731
        dv = shared(p.transpose(-1, -2) @ gh)
        ds = p * (gh @ vh.transpose(-1, -2) - delta) * s["scale"]
        dq, dk = ds @ kh, shared(ds.transpose(-1, -2) @ qh)
        at, kt = qrow >= 0, krow >= 0
        gq[qrow[at]] = dq.permute(0, 2, 1, 3)[at]
        gk[krow[kt]] = dk.permute(0, 2, 1, 3)[kt]
        gv[krow[kt]] = dv.permute(0, 2, 1, 3)[kt]
    return {"q": gq.to(q.dtype), "k": gk.to(k.dtype), "v": gv.to(v.dtype)}


def _library(s):
    import modulated_deformable_convolution_gb300 as m

    op = s["op"]
    if op.startswith("rotary"):
        kw = dict(layout=s["layout"], norm=s["norm"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
        if op == "rotary":
            return m.rotary(s["q"], s["k"], s["positions"], s["freq"], s["sections"], **kw)
        g = m.rotary_backward(s["gq"], s["gk"], s["q"], s["k"], s["positions"], s["freq"], s["sections"], **kw)
        return g if s["norm"] else {"q": g["q"], "k": g["k"]}
    kw = dict(k_lengths=s["kn"], causal=s["causal"], scale=s["scale"])
    if op == "attention":
        return m.attention(s["q"], s["k"], s["v"], s["qs"], s["ks"], **kw)
    return m.attention_backward(s["g"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["qs"], s["ks"], **kw)


def run(state):
    if own:
        return _library(state)
    plain = {"rotary": _rotary, "rotary_backward": _rotary_backward, "attention": _attention, "attention_backward": _attention_backward}
    return plain[state["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    hq, hk, d, size = case["q_heads"], case["k_heads"], case["dim"], SIZES[case["dtype"]]
    if case["op"].startswith("rotary"):
        t, h, w = _grid(case)
        n = t * h * w
        values = n * (hq + hk) * d
        weights = 2 * d if case["norm"] else 0
        if case["op"] == "rotary":  # read x, write y; squares, scaling and rotation
            return {"bytes": 2 * values * size + 12 * n + weights * size, "flops": values * (7 if case["norm"] else 3)}
        # read the gradient (and x where it is normed), write the gradient of x (and of the weights)
        return {"bytes": (3 if case["norm"] else 2) * values * size + 12 * n + 2 * weights * size, "flops": values * (14 if case["norm"] else 3)}
    ql, kl = _lengths(case["q"]), _lengths(case["k"])
    pairs = 0
    for n, m in zip(ql, kl):
        if case["causal"]:  # row i sees max(0, min(m, i + 1 + m - n)) keys
            first = max(0, n - m)
            rows = n - first
            low = max(0, m - n) + 1
            pairs += rows * (low + low + rows - 1) // 2
        else:
            pairs += n * m
    qv, kv = sum(ql) * hq * d * size, sum(kl) * hk * d * size
    if case["op"] == "attention":
        return {"bytes": 2 * qv + 2 * kv + 4 * sum(ql) * hq, "flops": 4 * d * hq * pairs}
    return {"bytes": 4 * qv + 4 * kv + 4 * sum(ql) * hq, "flops": 10 * d * hq * pairs}


# ---------------------------------------------------------------- 64 bits
def _exact_rotary(case, s):
    """The pairs as complex numbers, in 64 bits."""
    sections, d = s["sections"], case["dim"]
    pos, freq = s["positions"].double(), s["freq"].double()
    turns = torch.cat([pos[:, a : a + 1] * freq[sum(sections[:a]) : sum(sections[: a + 1])] for a in range(len(sections))], 1)
    turn = torch.polar(torch.ones_like(turns), turns)[:, None]
    lo, hi = [], []
    at = 0
    for n in sections:
        for i in range(n):
            pair = {"half": (at + i, at + i + sum(sections)), "interleaved": (2 * (at + i), 2 * (at + i) + 1), "blocks": (2 * at + i, 2 * at + n + i)}[case["layout"]]
            lo.append(pair[0])
            hi.append(pair[1])
        at += n
    def rotated(x, by):
        y = x.clone()
        z = torch.complex(x[..., lo], x[..., hi]) * by
        y[..., lo], y[..., hi] = z.real, z.imag
        return y
    outs = {}
    for name in ("q", "k"):
        x = s[name].double()
        w = s[name + "w"].double() if case["norm"] else None
        length = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) if case["norm"] else None
        if case["op"] == "rotary":
            outs[name] = rotated(x / length * w if case["norm"] else x, turn)
        else:
            g = rotated(s["g" + name].double(), turn.conj())
            if case["norm"]:
                outs[name + "_weight"] = (g * x / length).sum((0, 1))
                g = g * w
                g = g / length - x * (g * x).sum(-1, keepdim=True) / (d * length**3)
            outs[name] = g
    return (outs["q"], outs["k"]) if case["op"] == "rotary" else outs


def _exact_attention(case, s):
    """One sequence and key head at a time, in 64 bits, softmax by the definition."""
    q, k, v = s["q"], s["k"], s["v"]
    hq, hk = case["q_heads"], case["k_heads"]
    n = hq // hk
    backward = case["op"] == "attention_backward"
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)
    gk, gv = torch.zeros_like(k, dtype=torch.float64), torch.zeros_like(v, dtype=torch.float64)
    a = b = 0
    for lq, lk, room in zip(s["ql"], s["kl"], s["room"]):
        hidden = torch.ones(lq, lk, dtype=torch.bool, device=q.device).triu(lk - lq + 1) if case["causal"] else None
        for h in range(hq):
            qd, kd, vd = q[a : a + lq, h].double(), k[b : b + lk, h // n].double(), v[b : b + lk, h // n].double()
            x = qd @ kd.T * s["scale"]
            if hidden is not None:
                x = torch.where(hidden, -math.inf, x)
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[:, None])
            if not backward:
                out[a : a + lq, h], lse[h, a : a + lq] = p @ vd, z
                continue
            gd = s["g"][a : a + lq, h].double()
            dp = gd @ vd.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
            out[a : a + lq, h] = ds @ kd
            gk[b : b + lk, h // n] += ds.T @ qd
            gv[b : b + lk, h // n] += p.T @ gd
        a, b = a + lq, b + room
    return {"q": out, "k": gk, "v": gv} if backward else (out, lse)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        return _exact_rotary(case, s)
    if work(case)["flops"] > 5e12:
        return None
    return _exact_attention(case, s)
