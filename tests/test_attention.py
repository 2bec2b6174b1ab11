"""Attention over packed sequences, forward and backward, against a plain
implementation in 64 bits.

Tolerances, derived from the arithmetic, with u the unit roundoff of the
tensors' type and e = 2^-24:
- a score is a sum of head_dim products in fp32 (tensor cores may drop the bits
  below the largest term's fp32 unit): off by (2 head_dim + 8) e of the sum of
  the products' magnitudes; a probability is off by that relatively, plus 16 e
  for the exponential, and by u more where it is rounded to the tensors' type;
- out = sum p v: that share of sum p |v|, and its own rounding, u |out|;
- delta = sum grad_out * out reads an out that is rounded: u sum |grad_out out|;
- ds = p (dp - delta) scale is rounded once more, u |ds|; the three sums take
  over their terms' errors, and the gradients are rounded, u |.|.
The sums over many terms add (64 + terms / 64) e of the magnitudes' sum."""
import ctypes
import math
import os

import pytest
import torch

import modulated_deformable_convolution_gb300 as mdcn
from modulated_deformable_convolution_gb300 import _abi

gpu = pytest.mark.gpu
U = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 2.0**-126, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-126}
E = 2.0**-24


class Problem:
    def __init__(self, dtype, ql, kl, hq, hk, d, causal, room=None, seed=0, fused=False, scale=None, gap=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.dtype, self.ql, self.kl, self.causal = dtype, list(ql), list(kl), causal
        self.room = list(room or kl)
        self.scale = d**-0.5 if scale is None else scale
        tq, tk = sum(ql) + gap, sum(self.room) + gap
        if fused:
            assert tq == tk
            qkv = rnd(tq, hq + 2 * hk, d).to(dtype)
            self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            self.q, self.k, self.v = (rnd(t, h, d).to(dtype) for t, h in ((tq, hq), (tk, hk), (tk, hk)))
        self.g = rnd(tq, hq, d).to(dtype)
        self.qs, self.ks = mdcn.sequence_starts(ql, "cpu"), mdcn.sequence_starts(self.room, "cpu")
        self.kn = torch.tensor(self.kl, dtype=torch.int32) if room else None

    def cuda(self, name):
        t = getattr(self, name)
        if t is None or t.is_contiguous():
            return None if t is None else t.cuda()
        base = t._base.cuda()
        return base.as_strided(t.shape, t.stride(), t.storage_offset())

    def kw(self):
        return dict(k_lengths=self.cuda("kn"), causal=self.causal, scale=self.scale)

    def forward(self):
        return mdcn.attention(self.cuda("q"), self.cuda("k"), self.cuda("v"), self.cuda("qs"), self.cuda("ks"), **self.kw())

    def backward(self, out, lse):
        return mdcn.attention_backward(self.cuda("g"), self.cuda("q"), self.cuda("k"), self.cuda("v"), out, lse, self.cuda("qs"), self.cuda("ks"), **self.kw())

    def reference(self):
        """Values and tolerances of out, lse and the gradients, in 64 bits on the CPU."""
        u, d = U[self.dtype], self.q.shape[2]
        hq, hk = self.q.shape[1], self.k.shape[1]
        n = hq // hk
        r = {x: torch.zeros(t.shape, dtype=torch.float64) for x, t in (("out", self.q), ("q", self.q), ("k", self.k), ("v", self.v))}
        tol = {x: torch.zeros_like(t) for x, t in r.items()}
        r["lse"] = torch.full((hq, self.q.shape[0]), -math.inf, dtype=torch.float64)
        tol["lse"] = torch.zeros_like(r["lse"])
        rounded = 0.0 if self.dtype == torch.float32 else u
        a = b = 0
        for lq, lk, room in zip(self.ql, self.kl, self.room):
            for h in range(hq):
                q, g = self.q[a:a + lq, h].double(), self.g[a:a + lq, h].double()
                k, v = self.k[b:b + lk, h // n].double(), self.v[b:b + lk, h // n].double()
                seen = torch.ones(lq, lk, dtype=torch.bool)
                if self.causal:
                    seen = torch.arange(lk)[None] <= torch.arange(lq)[:, None] + lk - lq
                s = (q @ k.T * self.scale).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(s, 1) if lk else torch.full((lq,), -math.inf, dtype=torch.float64)
                p = torch.exp(s - z.masked_fill(z == -math.inf, 0.0)[:, None])
                mag = (q.abs() @ k.abs().T * abs(self.scale)).masked_fill(~seen, 0.0)
                rel = (2 * d + 8) * E * mag + 16 * E  # of each probability, before rounding
                worst = rel.amax(1, keepdim=True) if lk else torch.zeros(lq, 1)
                rel = rel + worst  # its row's sum is off too
                add = (64 + lk / 64) * E
                o, av = p @ v, p @ v.abs()
                r["out"][a:a + lq, h], r["lse"][h, a:a + lq] = o, z
                tol["out"][a:a + lq, h] = u * o.abs() + (p * (rel + rounded + add)) @ v.abs()
                tol["lse"][h, a:a + lq] = worst[:, 0] + 4 * E * z.masked_fill(z == -math.inf, 0.0).abs() + 8 * E
                # backward
                dp, adp = g @ v.T, g.abs() @ v.abs().T
                delta, adelta = (g * o).sum(1, keepdim=True), (g * o).abs().sum(1, keepdim=True)
                ds = p * (dp - delta)
                eds = (rel + rounded) * ds.abs() + p * (2 * d + 8) * E * (adp + adelta) + p * u * adelta
                dsum = (64 + max(lq * n, lk) / 64) * E
                r["q"][a:a + lq, h] = ds @ k * self.scale
                tol["q"][a:a + lq, h] = ((eds + dsum * ds.abs()) @ k.abs()) * abs(self.scale)
                r["k"][b:b + lk, h // n] += ds.T @ q * self.scale
                tol["k"][b:b + lk, h // n] += ((eds + dsum * ds.abs()).T @ q.abs()) * abs(self.scale)
                r["v"][b:b + lk, h // n] += p.T @ g
                tol["v"][b:b + lk, h // n] += (p * (rel + rounded + dsum)).T @ g.abs()
            a, b = a + lq, b + room
        for x in ("q", "k", "v"):
            tol[x] += u * r[x].abs()
        for x in ("out", "q", "k", "v"):
            tol[x] = tol[x] * 1.02 + TINY[self.dtype] * (1 + max([1] + self.kl + self.ql))
        return r, tol

    def check(self, got, ref, tol, what):
        got = got.double().cpu()
        inf = torch.isinf(ref)
        assert torch.equal(got[inf], ref[inf]), what
        assert torch.isfinite(got[~inf]).all(), what
        over = ((got - ref).abs() - tol)[~inf]
        if over.numel():
            assert over.max() <= 0, f"{what}: beyond the tolerance by {over.max():.3e}"


def _run(p, backward=True):
    r, tol = p.reference()
    out, lse = p.forward()
    p.check(out, r["out"], tol["out"], "out")
    p.check(lse, r["lse"], tol["lse"], "lse")
    if backward:
        g = p.backward(r["out"].to(p.dtype).cuda(), r["lse"].float().cuda())
        for x in ("q", "k", "v"):
            p.check(g[x], r[x], tol[x], "grad_" + x)


BF, FH, FS = torch.bfloat16, torch.float16, torch.float32
CASES = [
    # dtype, query lengths, key lengths, q heads, k heads, head_dim, causal
    (BF, [1], [1], 1, 1, 64, True),
    (BF, [128], [128], 2, 1, 64, True),
    (FH, [127, 129, 1], [127, 129, 1], 2, 2, 64, False),
    (BF, [300, 0, 5, 257], [300, 0, 5, 257], 4, 2, 128, True),
    (FH, [64, 64, 200], [64, 64, 200], 3, 1, 40, True),
    (BF, [513], [513], 1, 1, 128, False),
    (BF, [100, 30], [37, 400], 4, 4, 80, True),     # the first rows of the first see no key
    (FH, [9, 20, 3], [0, 1, 130], 6, 2, 96, False),  # no keys at all
    (FH, [50, 3], [50, 700], 5, 1, 72, True),
    (BF, [260], [260], 7, 1, 128, True),            # 7 heads share a key head
    (FH, [70], [333], 40, 2, 8, False),             # 20 to a key head, 8 elements
    (BF, [33], [65], 64, 1, 128, True),             # 64 to a key head
    (FS, [65, 1, 130], [65, 1, 130], 2, 1, 64, True),
    (FS, [100, 30, 4], [37, 100, 0], 4, 2, 72, True),
    (FS, [64], [191], 3, 3, 128, False),
    (FS, [17], [70], 20, 1, 24, True),
]
IDS = [f"{i}_{str(c[0])[6:]}_{c[3]}over{c[4]}x{c[5]}" for i, c in enumerate(CASES)]


@gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_against_64_bits(case):
    _run(Problem(*case, seed=len(case[1])))


@gpu
@pytest.mark.parametrize("dtype,hq,hk,d,causal", [(BF, 4, 2, 64, True), (FH, 6, 1, 128, False), (FS, 2, 2, 40, True)])
def test_slices_of_one_projection(dtype, hq, hk, d, causal):
    _run(Problem(dtype, [130, 7, 66], [130, 7, 66], hq, hk, d, causal, fused=True, seed=5))


@gpu
@pytest.mark.parametrize("dtype", [BF, FH, FS])
@pytest.mark.parametrize("new", [1, 3])
def test_new_tokens_against_a_cache(dtype, new):
    """A few new tokens a request, against caches with room left over that
    holds NaN and infinities; enough keys that they are shared out."""
    kl = [1500, 1, 700, 129, 128, 0, 64]
    p = Problem(dtype, [new] * len(kl), kl, 8, 2, 64, True, room=[1600] * len(kl), seed=new)
    for i, n in enumerate(kl):
        p.k[1600 * i + n:1600 * (i + 1)] = math.nan
        p.v[1600 * i + n:1600 * (i + 1)] = math.inf if i % 2 else math.nan
    assert torch.isfinite(p.reference()[0]["out"]).all()
    _run(p)


@gpu
@pytest.mark.parametrize("d", [8, 16, 32, 48, 56, 88, 112, 128])
def test_float32_head_sizes_shared_out(d):
    """Each length of the float32 kernels' loops over a head, whole and with
    elements left over; keys and rows enough that both are shared out."""
    _run(Problem(FS, [70, 300], [530, 300], 4, 2, d, d % 16 == 0, seed=d))


@gpu
@pytest.mark.parametrize("d", range(8, 136, 8))
@pytest.mark.parametrize("dtype", [BF, FH])
def test_every_head_size_with_partial_tiles(dtype, d):
    """Row and key tiles of which some lanes of a warp have a row and others
    none: one to eight turns of the loops that read results out."""
    _run(Problem(dtype, [5, 131, 44], [133, 40, 44], 2, 1, d, d % 16 == 0, seed=d))


@gpu
@pytest.mark.parametrize("dtype,hq,hk,d,causal", [(BF, 8, 8, 64, True), (FH, 8, 8, 64, False), (BF, 8, 8, 128, False), (FH, 8, 8, 128, True), (BF, 24, 8, 72, True)])
def test_more_items_than_blocks(dtype, hq, hk, d, causal):
    """Some 500 work items with work for each of the tensor-core kernels, several
    to a block: what a block carries from one to the next, of one to three tiles
    each, with empty ones between them."""
    g = torch.Generator().manual_seed(d)
    ql = [0 if i % 9 == 4 else int(n) for i, n in enumerate(torch.randint(1, 300, (72,), generator=g))]
    kl = [max(0, n + int(e)) if i % 3 == 0 else n for i, (n, e) in enumerate(zip(ql, torch.randint(-40, 300, (72,), generator=g)))]
    p = Problem(dtype, ql, kl, hq, hk, d, causal, seed=d)
    assert sum(n > 0 for n in ql) * hk > 3 * 152 and sum(n > 0 for n in kl) * hk > 3 * 152
    _run(p)


@gpu
@pytest.mark.parametrize("dtype", [BF, FH, FS])
def test_heads_outermost(dtype):
    """Tensors stored [heads][tokens][head_dim]: the head's stride is the larger."""
    p = Problem(dtype, [150, 33], [150, 33], 4, 2, 64, True, seed=12)
    r, tol = p.reference()
    turned = {x: p.cuda(x).transpose(0, 1).contiguous().transpose(0, 1) for x in ("q", "k", "v", "g")}
    out, lse = torch.empty_like(turned["q"]), torch.empty(4, 183, device="cuda")
    assert out.stride(1) > out.stride(0)
    mdcn.attention(turned["q"], turned["k"], turned["v"], p.cuda("qs"), p.cuda("ks"), causal=True, out=out, lse=lse)
    p.check(out, r["out"], tol["out"], "out")
    p.check(lse, r["lse"], tol["lse"], "lse")
    g = mdcn.attention_backward(turned["g"], turned["q"], turned["k"], turned["v"], out, lse, p.cuda("qs"), p.cuda("ks"), causal=True)
    want = p.backward(out.contiguous(), lse)
    for x in ("q", "k", "v"):
        assert torch.equal(g[x], want[x]), x


def test_whole_warps_at_tensor_memory():
    """A load of results from tensor memory is the whole warp's, and the stores
    before it, in the loop's last turn, were those of the lanes that have a row: the
    warp meets before each."""
    csrc = os.path.join(os.path.dirname(_abi.__file__), "csrc")
    loads = 0
    for name in ("mdcn_attention_tc.cu", "mdcn_attention_tc_backward.cu"):
        with open(os.path.join(csrc, name)) as f:
            lines = [x.strip() for x in f]
        for i, line in enumerate(lines):
            if line.startswith("if (any) tmem_ld16("):
                loads += 1
                assert lines[i - 1].startswith("__syncwarp();"), (name, i + 1)
    assert loads == 4


@gpu
@pytest.mark.parametrize("dtype", [BF, FS])
def test_neighbours_do_not_leak(dtype):
    """What the next sequence holds (NaN, infinities) reaches no other."""
    p = Problem(dtype, [100, 50, 30], [100, 50, 30], 2, 1, 64, True, seed=2)
    want, wlse = p.forward()
    wg = p.backward(want, wlse)
    for t in (p.q, p.k, p.v, p.g):
        t[100:150] = math.nan
    p.v[101] = math.inf
    out, lse = p.forward()
    o2, l2 = want.clone(), wlse.clone()
    g = p.backward(o2, l2)
    keep = torch.ones(180, dtype=torch.bool, device="cuda")
    keep[100:150] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[:, keep], wlse[:, keep])
    for x in ("q", "k", "v"):
        assert torch.equal(g[x][keep], wg[x][keep]), x


@gpu
@pytest.mark.parametrize("dtype", [BF, FH, FS])
def test_large_scores(dtype):
    """Scores in the hundreds: probabilities of 0 and 1, a maximum that grows
    along the keys."""
    p = Problem(dtype, [140], [300], 2, 1, 64, False, seed=3, scale=4.0)
    p.k *= torch.linspace(0.1, 2.0, 300)[:, None, None].to(dtype)
    _run(p)
    p.scale = -1.0
    _run(p)


def _float16_gradient_tolerances(p, a, lq, b, lk, h, r):
    """Of one sequence's (queries a.., keys b..) query head h, without the slack
    that Problem.reference has for numbers below float16's normal ones: the
    gradients' own size decides. ds is held in float16 times a power of two
    that brings its bound |grad_out| |v| 2 to between 2^13 and 2^15, so that
    numbers below 2^-14 are off by 2^-25 of the scale at most, 2^-37 of the
    bound without it; p, kept times 2^8, by 2^-33."""
    u, d, n = U[FH], p.q.shape[2], p.q.shape[1] // p.k.shape[1]
    q, g, k, v = p.q[a:a + lq, h].double(), p.g[a:a + lq, h].double(), p.k[b:b + lk, h // n].double(), p.v[b:b + lk, h // n].double()
    s = q @ k.T * p.scale
    if p.causal:
        s = s.masked_fill(torch.arange(lk)[None] > torch.arange(lq)[:, None] + lk - lq, -math.inf)
    z = torch.logsumexp(s, 1, keepdim=True)
    w = torch.exp(s - z)
    rel = (2 * d + 8) * E * (q.abs() @ k.abs().T) * p.scale + 16 * E + E * z.abs()
    rel = rel + rel.amax(1, keepdim=True)
    o = r["out"][a:a + lq, h]
    dp, adp = g @ v.T, g.abs() @ v.abs().T
    delta, adelta = (g * o).sum(1, keepdim=True), (g * o).abs().sum(1, keepdim=True)
    ds = w * (dp - delta)
    group = slice(h // n * n, h // n * n + n)
    bound = p.g[a:a + lq, group].double().norm(dim=2).amax() * v.norm(dim=1).amax()
    # delta reads an out that is rounded: u of it, or 2^-25
    eds = (rel + u) * ds.abs() + w * ((2 * d + 8) * E * (adp + adelta) + u * adelta + 2.0**-25 * g.abs().sum(1, keepdim=True))
    eds = eds + (64 + max(lq * n, lk) / 64) * E * ds.abs() + 2.0**-37 * bound
    ev = w * (rel + u + (64 + lq * n / 64) * E) + 2.0**-33
    return eds @ k.abs() * p.scale, eds.T @ q.abs() * p.scale, ev.T @ g.abs()


@gpu
@pytest.mark.parametrize("lengths,d,causal,sizes,scale", [
    ([1500], 64, False, [0], None), ([1500], 64, False, [-10], None), ([1500], 128, True, [-13], None), ([1500], 40, True, [-16], None),
    ([700, 900, 600], 64, True, [-13, 0, -8], None),     # sequences whose gradients differ in size
    ([2] * 100, 64, False, [13] * 100, 1 / 32),          # ds beyond float16's largest number
    ([1000, 3], 64, False, [-14, 13], None),
])
def test_float16_gradients_of_any_size(lengths, d, causal, sizes, scale):
    """Gradients of size 2^-16 to 2^13: rounded as those of size 1 are."""
    p = Problem(FH, lengths, lengths, 4, 2, d, causal, seed=len(lengths), scale=scale)
    for i, size in enumerate(sizes):
        p.g[sum(lengths[:i]):sum(lengths[:i + 1])] *= 2.0**size
    assert torch.isfinite(p.g).all()
    r, _ = p.reference()
    tol = {x: 2.0**-25 + U[FH] * r[x].abs() for x in ("q", "k", "v")}
    a = 0
    for n in lengths:
        for h in range(4):
            eq, ek, ev = _float16_gradient_tolerances(p, a, n, a, n, h, r)
            tol["q"][a:a + n, h] += 1.02 * eq
            tol["k"][a:a + n, h // 2] += 1.02 * ek
            tol["v"][a:a + n, h // 2] += 1.02 * ev
        a += n
    assert all(r[x].abs().amax() < 65504 for x in r if x != "lse")
    g = p.backward(r["out"].to(FH).cuda(), r["lse"].float().cuda())
    for x in ("q", "k", "v"):
        p.check(g[x], r[x], tol[x], "grad_" + x)


@gpu
@pytest.mark.parametrize("dtype", [BF, FS])
def test_rows_of_no_sequence_stay(dtype):
    p = Problem(dtype, [40, 20], [40, 20], 2, 1, 64, True, gap=9)
    q, k, v = p.cuda("q"), p.cuda("k"), p.cuda("v")
    out, lse = torch.full_like(q, 7.0), torch.full((2, 69), 7.0, device="cuda")
    mdcn.attention(q, k, v, p.cuda("qs"), p.cuda("ks"), causal=True, out=out, lse=lse)
    assert (out[60:] == 7).all() and (lse[:, 60:] == 7).all() and (out[:60] != 7).any()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    g = [torch.full_like(t, 7.0) for t in (q, k, v)]
    mdcn.mdcn_attention_backward(p.cuda("g"), q, k, v, out, lse, p.cuda("qs"), p.cuda("ks"), *g, ws, causal=True)
    for t in g:
        assert (t[60:] == 7).all() and torch.isfinite(t[:60]).all()


@gpu
@pytest.mark.parametrize("dtype", [BF, FH, FS])
def test_deterministic_on_a_stream_and_status(dtype):
    p = Problem(dtype, [700, 130], [700, 130], 4, 2, 64, True, seed=9)
    q, k, v, g = (p.cuda(x) for x in ("q", "k", "v", "g"))
    qs, ks = p.cuda("qs"), p.cuda("ks")
    ws = torch.full((mdcn.mdcn_attention_workspace_size(q, k, v, q, qs, ks),), 255, dtype=torch.uint8, device="cuda")
    out, lse = mdcn.attention(q, k, v, qs, ks, causal=True, workspace=ws)
    assert mdcn.mdcn_query_status(ws) == (0, 0)
    grads = mdcn.attention_backward(g, q, k, v, out, lse, qs, ks, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            o2, l2 = mdcn.attention(q, k, v, qs, ks, causal=True)
            g2 = mdcn.attention_backward(g, q, k, v, o2, l2, qs, ks, causal=True)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    for x in grads:
        assert torch.equal(grads[x], g2[x]), x


@gpu
@pytest.mark.parametrize("dtype", [BF, FS])
def test_slices_of_starts_and_lengths(dtype):
    """Some of the sequences, by slices of the offsets and lengths of all, and
    rows of a longer lse."""
    p = Problem(dtype, [9, 20, 30, 5], [20, 20, 33, 7], 2, 1, 64, True, room=[40] * 4, seed=3)
    q, k, v, g, qs, ks, kn = (p.cuda(x) for x in ("q", "k", "v", "g", "qs", "ks", "kn"))
    out, lse = mdcn.attention(q, k, v, qs, ks, k_lengths=kn, causal=True)
    grads = mdcn.attention_backward(g, q, k, v, out, lse, qs, ks, k_lengths=kn, causal=True)
    longer = torch.cat([lse.new_zeros(1), lse.flatten()])[1:].view_as(lse)
    assert longer.data_ptr() % 16
    for b in range(4):
        rows, keys = slice(int(p.qs[b]), int(p.qs[b + 1])), slice(int(p.ks[b]), int(p.ks[b + 1]))
        o, z = mdcn.attention(q, k, v, qs[b:b + 2], ks[b:b + 2], k_lengths=kn[b:b + 1], causal=True)
        assert torch.equal(o[rows], out[rows]) and torch.equal(z[:, rows], lse[:, rows])
        one = mdcn.attention_backward(g, q, k, v, out, longer, qs[b:b + 2], ks[b:b + 2], k_lengths=kn[b:b + 1], causal=True)
        assert torch.equal(one["q"][rows], grads["q"][rows])
        assert torch.equal(one["k"][keys], grads["k"][keys]) and torch.equal(one["v"][keys], grads["v"][keys])


@gpu
def test_capture_in_a_graph():
    p = Problem(BF, [200, 56], [200, 56], 4, 2, 64, True, seed=4)
    q, k, v, qs, ks = (p.cuda(x) for x in ("q", "k", "v", "qs", "ks"))
    want, wlse = mdcn.attention(q, k, v, qs, ks, causal=True)
    out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mdcn.mdcn_attention_forward(q, k, v, qs, ks, out, lse, ws, causal=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@gpu
@pytest.mark.parametrize("dtype", [BF, FS])
def test_empty(dtype):
    e = Problem(dtype, [], [], 2, 1, 64, True)
    out, lse = e.forward()
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert {n: tuple(t.shape) for n, t in e.backward(out, lse).items()} == {"q": (0, 2, 64), "k": (0, 1, 64), "v": (0, 1, 64)}
    # keys without queries: their gradients are zero
    p = Problem(dtype, [0], [70], 2, 1, 64, False)
    out, lse = p.forward()
    g = p.backward(out, lse)
    assert (g["k"] == 0).all() and (g["v"] == 0).all()
    # queries without keys
    p = Problem(dtype, [5], [0], 2, 1, 64, False)
    out, lse = p.forward()
    assert (out == 0).all() and (lse == -math.inf).all()
    assert (p.backward(out, lse)["q"] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", [FS, FH])
def test_starts_out_of_range_are_clamped(dtype):
    """Offsets beyond the tensors read and write nothing outside them: what is
    left is attention over the clamped rows."""
    p = Problem(dtype, [64], [64], 2, 1, 64, False, seed=6)
    want, _ = p.forward()
    p.qs, p.ks = torch.tensor([-5, 1000], dtype=torch.int32), torch.tensor([-7, 900], dtype=torch.int32)
    out, _ = p.forward()
    assert torch.equal(out, want)


@gpu
def test_gradient_against_differences():
    """<gradient, direction> against the central difference of the 64-bit
    forward; the fp32 gradient's error is a few 1e-6 of the terms' magnitudes."""
    p = Problem(FS, [40, 9], [40, 30], 4, 2, 40, True, seed=8)
    out, lse = p.forward()
    grads = p.backward(out, lse)
    gen = torch.Generator().manual_seed(1)

    def loss(q, k, v):
        save = p.q, p.k, p.v
        p.q, p.k, p.v = q, k, v
        o = p.reference()[0]["out"]
        p.q, p.k, p.v = save
        return (o * p.g.double()).sum()

    base = [p.q.double(), p.k.double(), p.v.double()]
    for i, x in enumerate(("q", "k", "v")):
        step = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * step, base[i] - h * step
        diff = (loss(*up) - loss(*down)) / (2 * h)
        terms = grads[x].double().cpu() * step
        assert abs(terms.sum() - diff) <= 1e-5 * terms.abs().sum()


def _on_16_bytes(need):
    """A workspace of `need` bytes that starts on 16 but not on 32 bytes."""
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    first = (16 - ws.data_ptr()) % 32
    ws = ws[first:first + need]
    assert ws.data_ptr() % 32 == 16
    return ws


@gpu
@pytest.mark.parametrize("dtype", [BF, FH, FS])
@pytest.mark.parametrize("d", [40, 64, 128])
def test_workspace_on_16_bytes(dtype, d):
    """A workspace on the 16 bytes that are asked for and no more, with the
    work shared out, gives the bits of one on 256."""
    p = Problem(dtype, [2, 1, 3], [1500, 129, 700], 8, 2, d, True, room=[1600] * 3, seed=d)
    q, k, v, g, qs, ks, kn = (p.cuda(x) for x in ("q", "k", "v", "g", "qs", "ks", "kn"))
    kw = dict(k_lengths=kn, causal=True)
    want, wlse = mdcn.attention(q, k, v, qs, ks, **kw)
    need = mdcn.mdcn_attention_workspace_size(q, k, v, want, qs, ks, **kw)
    assert need > 256  # there are partial results
    out, lse = torch.empty_like(want), torch.empty_like(wlse)
    mdcn.mdcn_attention_forward(q, k, v, qs, ks, out, lse, _on_16_bytes(need), **kw)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    wg = mdcn.attention_backward(g, q, k, v, out, lse, qs, ks, **kw)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    need = mdcn.mdcn_attention_backward_workspace_size(g, q, k, v, out, lse, qs, ks, *grads, **kw)
    mdcn.mdcn_attention_backward(g, q, k, v, out, lse, qs, ks, *grads, _on_16_bytes(need), **kw)
    for got, x in zip(grads, ("q", "k", "v")):
        assert torch.equal(got, wg[x]), x


def test_dependent_kernels_wait_before_they_read():
    """Kernels that may start before the one ahead of them has ended wait for
    it, and hold no read-only load, which the compiler may move above the wait."""
    csrc = os.path.join(os.path.dirname(_abi.__file__), "csrc")
    kernels = 0
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            code = "\n".join(x.split("//")[0] for x in f.read().splitlines())
        if not name.endswith((".cu", ".cuh")) or "dependency_wait()" not in code and name != "mdcn_attention.cuh":
            continue
        for word in ("__ldg(", "__restrict__", "ld.global.nc"):
            assert word not in code, (name, word)
        for body in code.split("__global__")[1:]:
            kernels += 1
            assert "dependency_wait();" in body.split("\n}\n")[0], name
    assert kernels >= 11


# ---------------------------------------------------------------- refusals
FAKE = 0x7F0000000000  # never dereferenced: each call below fails validation first


@pytest.fixture(scope="module")
def lib():
    from modulated_deformable_convolution_gb300 import build

    build.build()
    return _abi.load()


def _dims(**kw):
    d = _abi.mdcn_attention_dims()
    d.batch, d.q_tokens, d.k_tokens, d.q_heads, d.k_heads, d.head_dim = 2, 10, 12, 4, 2, 64
    for n in ("q", "k", "v", "out", "grad_out", "grad_q", "grad_k", "grad_v"):
        s = getattr(d, n)
        s.token, s.head = 4 * 64, 64
    for k, v in kw.items():
        if k.endswith("_stride"):
            getattr(d, k[:-7]).token = v
        else:
            setattr(d, k, v)
    return d


def _fwd(lib, d, a=None, ptrs=None, dt=_abi.MDCN_BF16, nbytes=1 << 30):
    a = a or _abi.mdcn_attention_attrs(1, 0.125)
    p = ptrs or [FAKE + 256 * i for i in range(9)]
    return lib.mdcn_attention_forward(ctypes.byref(a), ctypes.byref(d), dt, *p, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), _abi.MDCN_ERR_SHAPE), (dict(batch=0), _abi.MDCN_ERR_SHAPE), (dict(q_heads=3), _abi.MDCN_ERR_SHAPE),
    (dict(k_heads=0), _abi.MDCN_ERR_SHAPE), (dict(q_tokens=-1), _abi.MDCN_ERR_SHAPE), (dict(head_dim=0), _abi.MDCN_ERR_SHAPE),
    (dict(head_dim=60), _abi.MDCN_ERR_UNSUPPORTED), (dict(head_dim=136), _abi.MDCN_ERR_UNSUPPORTED),
    (dict(q_heads=130, k_heads=2), _abi.MDCN_ERR_UNSUPPORTED), (dict(k_tokens=2**31), _abi.MDCN_ERR_UNSUPPORTED),
    (dict(q_stride=0), _abi.MDCN_ERR_SHAPE), (dict(out_stride=-8), _abi.MDCN_ERR_SHAPE), (dict(v_stride=260), _abi.MDCN_ERR_ALIGN),
])
def test_refuses_dims(lib, kw, status):
    assert _fwd(lib, _dims(**kw)) == status


def test_refuses_attrs_pointers_and_workspace(lib):
    d = _dims()
    for a in ((2, 1.0), (-1, 1.0), (0, math.inf), (0, math.nan)):
        assert _fwd(lib, d, _abi.mdcn_attention_attrs(*a)) == _abi.MDCN_ERR_ATTR
    assert _fwd(lib, d, dt=7) == _abi.MDCN_ERR_DTYPE
    p = [FAKE + 256 * i for i in range(9)]  # q k v q_starts k_starts k_lengths out lse workspace
    for i in (0, 1, 2, 3, 4, 6, 7, 8):
        q = list(p)
        q[i] = None
        assert _fwd(lib, d, ptrs=q) == _abi.MDCN_ERR_NULL, i
    for i in range(9):
        q = list(p)
        q[i] += 8
        assert _fwd(lib, d, ptrs=q) == _abi.MDCN_ERR_ALIGN, i
    assert _fwd(lib, d, nbytes=16) == _abi.MDCN_ERR_WORKSPACE
    n = ctypes.c_size_t()
    a = _abi.mdcn_attention_attrs(1, 0.125)
    assert lib.mdcn_attention_backward_workspace_size(ctypes.byref(a), ctypes.byref(d), _abi.MDCN_BF16, ctypes.byref(n)) == 0
    assert lib.mdcn_attention_backward_workspace_size(ctypes.byref(a), ctypes.byref(d), _abi.MDCN_BF16, None) == _abi.MDCN_ERR_NULL
    # grad_out q k v out lse q_starts k_starts k_lengths grad_q grad_k grad_v workspace
    p = [FAKE + 256 * i for i in range(13)]
    back = lambda p, n: lib.mdcn_attention_backward(ctypes.byref(a), ctypes.byref(d), _abi.MDCN_BF16, *p, n, None)  # noqa: E731
    assert back(p, n.value - 1) == _abi.MDCN_ERR_WORKSPACE
    for i in range(13):
        q = list(p)
        q[i] = None
        if i != 8:
            assert back(q, n.value) == _abi.MDCN_ERR_NULL, i
        q[i] = p[i] + 8
        assert back(q, n.value) == _abi.MDCN_ERR_ALIGN, i


def test_binding_refuses(lib):
    q = torch.zeros(4, 2, 64)
    s = mdcn.sequence_starts([4], "cpu")
    with pytest.raises(ValueError):
        mdcn.attention(q, q, q, s, s)  # not on a GPU


@gpu
def test_binding_refuses_on_gpu():
    p = Problem(BF, [8], [8], 4, 2, 64, True)
    q, k, v, qs = p.cuda("q"), p.cuda("k"), p.cuda("v"), p.cuda("qs")
    with pytest.raises(TypeError):
        mdcn.attention(q, k.float(), v, qs, qs)
    with pytest.raises(ValueError):
        mdcn.attention(q, k, v[:4], qs, qs)
    with pytest.raises(TypeError):
        mdcn.attention(q, k, v, qs.long(), qs)
    with pytest.raises(ValueError):
        mdcn.attention(q, k, v, qs, qs[:1])
    with pytest.raises(ValueError):
        mdcn.attention(q.transpose(1, 2), k, v, qs, qs)
    with pytest.raises(mdcn.MdcnError):
        mdcn.attention(q[:, :3], k, v, qs, qs)  # 3 heads over 2
    with pytest.raises(mdcn.MdcnError):
        mdcn.attention(q, k[:, :1].expand(8, 2, 64), v, qs, qs)  # a stride of 0
