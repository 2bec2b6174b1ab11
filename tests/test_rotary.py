"""Rotary positions over several axes with the norms of queries and keys,
forward and backward, against a plain implementation in 64 bits.

Tolerances, derived from the arithmetic (u = the output type's unit roundoff):
the output is rounded once (u * |ref|); before that the fp32 steps (mean
square, its root, weight, angle, two products) carry at most 32 units of 2^-24
of the pair's length, and an angle's 2^-24 of a turn is 2 pi of them. A
gradient of a weight is a sum of n terms in fp32, off by at most (64 + its
longest chain of additions) units of 2^-24 of the sum of their magnitudes."""
import ctypes
import math

import pytest
import torch

import modulated_deformable_convolution_gb300 as mdcn
from modulated_deformable_convolution_gb300 import _abi

gpu = pytest.mark.gpu
U = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 0.0, torch.float16: 2.0**-25, torch.bfloat16: 0.0}  # half the smallest subnormal
F32 = 2.0**-24


def _pairs(sections, layout):
    """(lo, hi, axis) of each pair, by the definition."""
    out, at, total = [], 0, sum(sections)
    for axis, n in enumerate(sections):
        for i in range(n):
            p = at + i
            lo, hi = {"half": (p, p + total), "interleaved": (2 * p, 2 * p + 1), "blocks": (2 * at + i, 2 * at + n + i)}[layout]
            out.append((lo, hi, axis))
        at += n
    return out


def _rotated(x, positions, freq, sections, layout, sign=1):
    y = x.clone()
    for p, (lo, hi, axis) in enumerate(_pairs(sections, layout)):
        t = sign * positions[:, axis].double() * freq[p].double()
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        y[..., lo] = x[..., lo] * c - x[..., hi] * s
        y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def _forward_ref(x, w, positions, freq, sections, layout, norm, eps):
    x = x.double()
    if norm:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
    return _rotated(x, positions, freq, sections, layout)


def _backward_ref(gy, x, w, positions, freq, sections, layout, norm, eps):
    g = _rotated(gy.double(), positions, freq, sections, layout, -1)
    if not norm:
        return g, None, None
    x = x.double()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    gw, size = (g * n).sum((0, 1)), (g * n).abs().sum((0, 1))
    gn = g if w is None else g * w.double()
    return r * (gn - n * (gn * n).mean(-1, keepdim=True)), gw, size


class Problem:
    def __init__(self, dtype, tokens, hq, hk, d, sections, layout, norm, weights=True, seed=0, fused=False, start=0, pad=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.sections, self.layout, self.norm, self.eps = sections, layout, norm, 1e-5
        qkv = rnd(tokens, hq + 2 * hk, d + pad).to(dtype)
        if fused:
            self.q, self.k = qkv[:, :hq, :d], qkv[:, hq:hq + hk, :d]
        else:
            self.q, self.k = qkv[:, :hq, :d].contiguous(), qkv[:, hq:hq + hk, :d].contiguous()
        self.qw = (1 + 0.3 * rnd(d)).to(dtype) if norm and weights else None
        self.kw = (1 + 0.3 * rnd(d)).to(dtype) if norm and weights else None
        self.pos = torch.randint(0, 97, (tokens, len(sections)), generator=g, dtype=torch.int32) + start
        self.freq = mdcn.rotary_frequencies(sections, device="cpu")
        self.gq, self.gk = rnd(tokens, hq, d).to(dtype), rnd(tokens, hk, d).to(dtype)
        self.dtype = dtype

    def cuda(self, name):
        t = getattr(self, name)
        if t is None:
            return None
        if t.is_contiguous():
            return t.cuda()
        base = torch.empty(t._base.shape, dtype=t.dtype, device="cuda")
        base.copy_(t._base)
        return base.as_strided(t.shape, t.stride(), t.storage_offset())

    def kw_args(self):
        return dict(layout=self.layout, norm=self.norm, q_weight=self.cuda("qw"), k_weight=self.cuda("kw"), eps=self.eps)

    def close(self, got, ref, scale):
        tol = U[self.dtype] * ref.abs() * 1.01 + 40 * F32 * scale + TINY[self.dtype]
        got = got.double().cpu()
        assert torch.isfinite(got).all()
        over = ((got - ref).abs() - tol).max() if got.numel() else torch.tensor(-1.0)
        assert over <= 0, f"beyond the tolerance by {over:.3e}"


def _length(ref):
    return ref.abs().amax(-1, keepdim=True).expand_as(ref) * math.sqrt(2)


CASES = [
    # dtype, tokens, hq, hk, d, sections, layout, norm
    (torch.float32, 5, 3, 1, 64, (16, 16), "half", True),
    (torch.float16, 33, 4, 2, 64, (0, 16, 16), "blocks", True),
    (torch.bfloat16, 17, 32, 8, 128, (24, 20, 20), "half", True),
    (torch.bfloat16, 1, 32, 8, 128, (24, 20, 20), "half", True),
    (torch.float32, 7, 12, 3, 80, (8, 13, 13), "interleaved", True),
    (torch.float16, 9, 5, 5, 72, (3, 8, 7), "half", True),      # odd sections, 36 of 72 elements rotated
    (torch.bfloat16, 9, 6, 2, 40, (5, 6), "blocks", False),
    (torch.float32, 4, 2, 2, 256, (32, 32, 32, 32), "half", True),
    (torch.float16, 6, 1, 1, 8, (1,), "interleaved", True),
    (torch.float32, 6, 2, 1, 16, (0, 0), "half", True),         # nothing rotates: norm alone
    (torch.bfloat16, 700, 7, 1, 120, (20, 20, 20), "interleaved", True),
    (torch.float32, 2, 300, 3, 24, (12,), "half", False),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}x{c[2]}+{c[3]}x{c[4]}_{c[6]}")
@pytest.mark.parametrize("fused", [False, True])
def test_forward(case, fused):
    p = Problem(*case, fused=fused)
    yq, yk = mdcn.rotary(p.cuda("q"), p.cuda("k"), p.cuda("pos"), p.cuda("freq"), p.sections, **p.kw_args())
    for got, x, w in ((yq, p.q, p.qw), (yk, p.k, p.kw)):
        ref = _forward_ref(x, w, p.pos, p.freq, p.sections, p.layout, p.norm, p.eps)
        p.close(got, ref, _length(ref))


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}_{c[1]}x{c[2]}+{c[3]}x{c[4]}_{c[6]}")
@pytest.mark.parametrize("fused", [False, True])
def test_backward(case, fused):
    p = Problem(*case, fused=fused)
    g = mdcn.rotary_backward(p.cuda("gq"), p.cuda("gk"), p.cuda("q"), p.cuda("k"), p.cuda("pos"), p.cuda("freq"), p.sections, **p.kw_args())
    for name, gy, x, w in (("q", p.gq, p.q, p.qw), ("k", p.gk, p.k, p.kw)):
        ref, gw, size = _backward_ref(gy, x, w, p.pos, p.freq, p.sections, p.layout, p.norm, p.eps)
        p.close(g[name], ref, _length(ref) + ref.abs().amax())
        if w is None:
            assert g[name + "_weight"] is None
        else:
            n = x.shape[0] * x.shape[1]
            tol = U[p.dtype] * gw.abs() * 1.01 + (64 + n) * F32 * size + TINY[p.dtype]
            assert ((g[name + "_weight"].double().cpu() - gw).abs() <= tol).all()


@gpu
def test_rows_off_16_bytes():
    """Strides and starts that break 16-byte alignment: the narrow loads."""
    p = Problem(torch.float16, 9, 3, 2, 40, (10, 10), "half", True, fused=True, pad=1)
    q = p.cuda("q")
    assert q.stride(1) % 8 != 0
    yq, yk = mdcn.rotary(q, p.cuda("k"), p.cuda("pos"), p.cuda("freq"), p.sections, **p.kw_args())
    for got, x, w in ((yq, p.q, p.qw), (yk, p.k, p.kw)):
        ref = _forward_ref(x, w, p.pos, p.freq, p.sections, p.layout, p.norm, p.eps)
        p.close(got, ref, _length(ref))


@gpu
def test_slices_of_positions():
    """A decoder's positions of one step after the other, rows of 12 bytes in one
    tensor, and frequencies and weights that start off 16 bytes."""
    p = Problem(torch.float16, 6, 3, 2, 48, (5, 8, 9), "half", True)
    pos, freq = p.cuda("pos"), torch.cat([torch.zeros(1), p.freq]).cuda()[1:]
    w = [torch.cat([torch.zeros(1, dtype=p.dtype), x]).cuda()[1:] for x in (p.qw, p.kw)]
    assert freq.data_ptr() % 16 and w[0].data_ptr() % 16
    q, k, gq, gk = (p.cuda(x) for x in ("q", "k", "gq", "gk"))
    kw = dict(layout=p.layout, norm=True, eps=p.eps)
    want = mdcn.rotary(q, k, pos, p.cuda("freq"), p.sections, q_weight=p.cuda("qw"), k_weight=p.cuda("kw"), **kw)
    wg = mdcn.rotary_backward(gq, gk, q, k, pos, p.cuda("freq"), p.sections, q_weight=p.cuda("qw"), k_weight=p.cuda("kw"), **kw)
    for t in range(6):
        at = pos[t:t + 1]
        got = mdcn.rotary(q[t:t + 1], k[t:t + 1], at, freq, p.sections, q_weight=w[0], k_weight=w[1], **kw)
        g = mdcn.rotary_backward(gq[t:t + 1], gk[t:t + 1], q[t:t + 1], k[t:t + 1], at, freq, p.sections, q_weight=w[0], k_weight=w[1], **kw)
        assert torch.equal(got[0], want[0][t:t + 1]) and torch.equal(got[1], want[1][t:t + 1])
        assert torch.equal(g["q"], wg["q"][t:t + 1]) and torch.equal(g["k"], wg["k"][t:t + 1])
    with pytest.raises(mdcn.MdcnError):  # the entry point itself takes what lies on 16 bytes
        mdcn.mdcn_rotary_forward(q[:1], None, pos[1:2], freq, p.sections, torch.empty_like(q[:1]), None)


@gpu
def test_large_positions_keep_precision():
    """Positions near 2^24: the angle is reduced from the exact product."""
    p = Problem(torch.float32, 64, 2, 1, 64, (16, 16), "half", False, start=2**24 - 200)
    yq, _ = mdcn.rotary(p.cuda("q"), None, p.cuda("pos"), p.cuda("freq"), p.sections, layout=p.layout)
    ref = _forward_ref(p.q, None, p.pos, p.freq, p.sections, p.layout, False, p.eps)
    p.close(yq, ref, _length(ref) * math.sqrt(2))


@gpu
def test_negative_positions_undo():
    p = Problem(torch.float32, 8, 2, 1, 64, (16, 16), "interleaved", False)
    y, _ = mdcn.rotary(p.cuda("q"), None, p.cuda("pos"), p.cuda("freq"), p.sections, layout=p.layout)
    x, _ = mdcn.rotary(y, None, -p.cuda("pos"), p.cuda("freq"), p.sections, layout=p.layout)
    p.close(x, p.q.double(), 2 * _length(p.q.double()))


@gpu
def test_in_place_and_no_keys():
    p = Problem(torch.bfloat16, 50, 6, 2, 64, (16, 16), "half", True)
    q, k = p.cuda("q"), p.cuda("k")
    want, _ = mdcn.rotary(q, None, p.cuda("pos"), p.cuda("freq"), p.sections, layout="half", norm=True, q_weight=p.cuda("qw"), eps=p.eps)
    yq, yk = mdcn.rotary(q, k, p.cuda("pos"), p.cuda("freq"), p.sections, q_out=q, k_out=k, **p.kw_args())
    assert yq.data_ptr() == q.data_ptr() and torch.equal(yq, want)
    ref = _forward_ref(p.k, p.kw, p.pos, p.freq, p.sections, p.layout, p.norm, p.eps)
    p.close(yk, ref, _length(ref))


@gpu
def test_zero_rows_and_no_tokens():
    """A head of zeros stays zero (and its gradient finite); no tokens give
    empty outputs and zero weight gradients."""
    p = Problem(torch.float32, 4, 2, 1, 64, (16, 16), "half", True)
    p.q[:] = 0
    yq, _ = mdcn.rotary(p.cuda("q"), p.cuda("k"), p.cuda("pos"), p.cuda("freq"), p.sections, **p.kw_args())
    assert (yq == 0).all()
    g = mdcn.rotary_backward(p.cuda("gq"), p.cuda("gk"), p.cuda("q"), p.cuda("k"), p.cuda("pos"), p.cuda("freq"), p.sections, **p.kw_args())
    ref, _, _ = _backward_ref(p.gq, p.q, p.qw, p.pos, p.freq, p.sections, p.layout, True, p.eps)
    p.close(g["q"], ref, _length(ref) + ref.abs().amax())
    e = Problem(torch.float32, 0, 2, 1, 64, (16, 16), "half", True)
    yq, yk = mdcn.rotary(e.cuda("q"), e.cuda("k"), e.cuda("pos"), e.cuda("freq"), e.sections, **e.kw_args())
    assert yq.shape == (0, 2, 64) and yk.shape == (0, 1, 64)
    g = mdcn.rotary_backward(e.cuda("gq"), e.cuda("gk"), e.cuda("q"), e.cuda("k"), e.cuda("pos"), e.cuda("freq"), e.sections, **e.kw_args())
    assert (g["q_weight"] == 0).all() and (g["k_weight"] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,sections,layout", [
    (80, (8, 13, 13), "interleaved"), (64, (3,), "interleaved"),  # neighbours, the last lanes in part or not at all
    (128, (16, 16), "half"), (128, (8, 16), "blocks"),             # runs of eight
    (72, (3, 8, 7), "half"), (40, (5, 6), "blocks"),               # anywhere
    (64, (0, 0), "half"),
])
def test_strays_in_elements_that_are_not_rotated(dtype, d, sections, layout):
    """Without norm an element past the rotated ones is copied, infinities and
    NaN too, and reaches no other."""
    p = Problem(dtype, 7, 3, 1, d, sections, layout, False)
    q = p.cuda("q")
    args = (p.cuda("pos"), p.cuda("freq"), p.sections)
    run = lambda x: mdcn.rotary(x, None, *args, layout=layout)[0]  # noqa: E731
    back = lambda x: mdcn.rotary_backward(x, None, None, None, *args, layout=layout)["q"]  # noqa: E731
    rotated = sorted(e for lo, hi, _ in _pairs(sections, layout) for e in (lo, hi))
    still = [e for e in range(d) if e not in rotated]
    for f in (run, back):
        want = f(q)
        assert torch.equal(want[..., still], q[..., still])
        x = q.clone()
        for i, e in enumerate(still):
            x[i % 7, i % 3, e] = (math.inf, -math.inf, math.nan)[i // 3 % 3]
        got = f(x)
        assert torch.equal(got[..., rotated], want[..., rotated])
        assert torch.equal(torch.nan_to_num(got[..., still], 7.0), torch.nan_to_num(x[..., still], 7.0))


@gpu
@pytest.mark.parametrize("q_weight", [True, False])
def test_weight_of_no_heads(q_weight):
    """A k without heads: its weight's gradient is an empty sum, whatever the
    workspace held."""
    p = Problem(torch.float16, 9, 3, 1, 40, (10, 10), "half", True)
    gq, q = p.cuda("gq"), p.cuda("q")
    none = torch.empty(9, 0, 40, dtype=p.dtype, device="cuda")
    kw = dict(layout=p.layout, norm=True, eps=p.eps, q_weight=p.cuda("qw") if q_weight else None)
    want = mdcn.rotary_backward(gq, None, q, None, p.cuda("pos"), p.cuda("freq"), p.sections, **kw)
    g, gw = torch.empty_like(q), [torch.full((40,), math.nan, dtype=p.dtype, device="cuda") for _ in range(2)]
    ws = torch.full((mdcn.mdcn_rotary_backward_workspace_size(gq, none, p.cuda("pos"), p.cuda("freq"), p.sections, norm=True),), 255, dtype=torch.uint8, device="cuda")
    mdcn.mdcn_rotary_backward(gq, none, q, none, p.cuda("pos"), p.cuda("freq"), p.sections, g, none, gw[0] if q_weight else None, gw[1], ws, k_weight=p.cuda("kw"), **kw)
    assert (gw[1] == 0).all() and torch.equal(g, want["q"])
    if q_weight:
        assert torch.equal(gw[0], want["q_weight"])


@gpu
def test_deterministic_and_on_a_stream():
    p = Problem(torch.bfloat16, 3001, 6, 2, 64, (16, 16), "half", True)
    args = (p.cuda("gq"), p.cuda("gk"), p.cuda("q"), p.cuda("k"), p.cuda("pos"), p.cuda("freq"), p.sections)
    kw = p.kw_args()
    first = mdcn.rotary_backward(*args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = mdcn.rotary_backward(*args, **kw)
    side.synchronize()
    for n in first:
        assert torch.equal(first[n], again[n]), n


@gpu
def test_gradient_against_differences():
    """<gradient, direction> against the central difference of the 64-bit
    forward, step 1e-5 (its own error about 1e-9); the fp32 gradient's error is
    a few 1e-7 of the sum of the terms' magnitudes."""
    p = Problem(torch.float32, 6, 3, 2, 40, (6, 9), "blocks", True)
    g = mdcn.rotary_backward(p.cuda("gq"), p.cuda("gk"), p.cuda("q"), p.cuda("k"), p.cuda("pos"), p.cuda("freq"), p.sections, **p.kw_args())
    gen = torch.Generator().manual_seed(3)
    for name, x, w, gy in (("q", p.q, p.qw, p.gq), ("k", p.k, p.kw, p.gk)):
        loss = lambda xx, ww: (gy.double() * _forward_ref(xx, ww, p.pos, p.freq, p.sections, p.layout, True, p.eps)).sum()  # noqa: E731,B023
        dx, dw = torch.randn(x.shape, generator=gen, dtype=torch.float64), torch.randn(w.shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        diff = (loss(x.double() + h * dx, w.double()) - loss(x.double() - h * dx, w.double())) / (2 * h)
        terms = g[name].double().cpu() * dx
        assert abs(terms.sum() - diff) <= 2e-6 * terms.abs().sum()
        diff = (loss(x.double(), w.double() + h * dw) - loss(x.double(), w.double() - h * dw)) / (2 * h)
        terms = g[name + "_weight"].double().cpu() * dw
        assert abs(terms.sum() - diff) <= 4e-6 * terms.abs().sum()


# ---------------------------------------------------------------- refusals
FAKE = 0x7F0000000000  # never dereferenced: each call below fails validation first


@pytest.fixture(scope="module")
def lib():
    from modulated_deformable_convolution_gb300 import build

    build.build()
    return _abi.load()


def _dims(**kw):
    d = _abi.mdcn_rotary_dims()
    d.tokens, d.q_heads, d.k_heads, d.head_dim, d.axes = 10, 4, 2, 64, 2
    d.sections[:] = (16, 16, 0, 0)
    for n in ("q", "k", "q_out", "k_out", "q_grad", "k_grad"):
        s = getattr(d, n)
        s.token, s.head = 8 * 64, 64
    for k, v in kw.items():
        if k == "sections":
            d.sections[:] = v
        elif k.endswith("_token"):
            getattr(d, k[:-6]).token = v
        else:
            setattr(d, k, v)
    return d


def _attrs(layout=0, norm=1, eps=1e-6):
    return _abi.mdcn_rotary_attrs(layout, norm, eps)


def _fwd(lib, a, d, ptrs=None, dt=_abi.MDCN_F16):
    p = [FAKE + 256 * i for i in range(8)] if ptrs is None else ptrs
    return lib.mdcn_rotary_forward(ctypes.byref(a), ctypes.byref(d), dt, *p, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), _abi.MDCN_ERR_SHAPE), (dict(q_heads=0), _abi.MDCN_ERR_SHAPE), (dict(k_heads=-1), _abi.MDCN_ERR_SHAPE),
    (dict(axes=0), _abi.MDCN_ERR_SHAPE), (dict(axes=5), _abi.MDCN_ERR_SHAPE), (dict(sections=(17, 16, 0, 0)), _abi.MDCN_ERR_SHAPE),
    (dict(sections=(-1, 16, 0, 0)), _abi.MDCN_ERR_SHAPE), (dict(sections=(8, 8, 1, 0)), _abi.MDCN_ERR_SHAPE),
    (dict(head_dim=60), _abi.MDCN_ERR_UNSUPPORTED), (dict(head_dim=264), _abi.MDCN_ERR_UNSUPPORTED),
    (dict(tokens=2**31), _abi.MDCN_ERR_UNSUPPORTED), (dict(q_token=0), _abi.MDCN_ERR_SHAPE), (dict(k_out_token=-64), _abi.MDCN_ERR_SHAPE),
    (dict(q_token=2**31), _abi.MDCN_ERR_UNSUPPORTED),
])
def test_refuses_dims(lib, kw, status):
    assert _fwd(lib, _attrs(), _dims(**kw)) == status


MOST = 2**31 - 2**17  # heads that the kernels can count


@pytest.mark.parametrize("q_heads,k_heads", [(MOST + 1, 0), (MOST, 1), (1, MOST), (2**31 - 1, 0), (2**30, 2**30 - 1), (2**30, 2**30)])
def test_refuses_more_heads_than_the_kernels_count(lib, q_heads, k_heads):
    d = _dims(q_heads=q_heads, k_heads=k_heads, head_dim=8, sections=(2, 2, 0, 0))
    assert _fwd(lib, _attrs(), d) == _abi.MDCN_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    size = lambda: lib.mdcn_rotary_backward_workspace_size(ctypes.byref(_attrs()), ctypes.byref(d), _abi.MDCN_F16, ctypes.byref(n))  # noqa: E731
    assert size() == _abi.MDCN_ERR_UNSUPPORTED
    d.q_heads, d.k_heads = MOST - 1, 1
    assert size() == _abi.MDCN_OK


def test_refuses_attrs_pointers_and_types(lib):
    d = _dims()
    for a in (_attrs(layout=3), _attrs(layout=-1), _attrs(norm=2), _attrs(eps=-1.0), _attrs(eps=math.inf), _attrs(eps=math.nan)):
        assert _fwd(lib, a, d) == _abi.MDCN_ERR_ATTR
    assert _fwd(lib, _attrs(norm=0), d) == _abi.MDCN_ERR_ATTR  # a weight without norm
    assert _fwd(lib, _attrs(), d, dt=3) == _abi.MDCN_ERR_DTYPE
    p = [FAKE + 256 * i for i in range(8)]
    for i in (0, 1, 2, 3, 6, 7):
        q = list(p)
        q[i] = None
        assert _fwd(lib, _attrs(), d, q) == _abi.MDCN_ERR_NULL
    for i in (2, 3, 4, 5):
        q = list(p)
        q[i] += 8
        assert _fwd(lib, _attrs(), d, q) == _abi.MDCN_ERR_ALIGN
    q = list(p)
    q[0] += 1
    assert _fwd(lib, _attrs(), d, q) == _abi.MDCN_ERR_ALIGN
    n = ctypes.c_size_t()
    assert lib.mdcn_rotary_backward_workspace_size(ctypes.byref(_attrs()), ctypes.byref(d), _abi.MDCN_F16, ctypes.byref(n)) == 0 and n.value > 0
    # grad_q_out, grad_k_out, q, k, positions, inv_freq, q_weight, k_weight, grad_q, grad_k, grad_q_weight, grad_k_weight, workspace
    p = [FAKE + 256 * i for i in range(13)]
    back = lambda p, n, a=_attrs(): lib.mdcn_rotary_backward(ctypes.byref(a), ctypes.byref(d), _abi.MDCN_F16, *p, n, None)  # noqa: E731
    assert back(p, n.value - 1) == _abi.MDCN_ERR_WORKSPACE
    assert back(p, n.value, _attrs(norm=0)) == _abi.MDCN_ERR_ATTR
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9, 10, 12):
        q = list(p)
        q[i] = None
        assert back(q, n.value) == _abi.MDCN_ERR_NULL, i


def test_binding_refuses(lib):
    q, pos, f = torch.zeros(4, 2, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError):
        mdcn.rotary(q, None, pos, f, (16, 16))  # not on a GPU
    with pytest.raises(ValueError):
        mdcn.rotary(q[0], None, pos, f, (16, 16))


@gpu
def test_binding_refuses_on_gpu():
    p = Problem(torch.float16, 8, 2, 1, 64, (16, 16), "half", True)
    q, k, pos, f = p.cuda("q"), p.cuda("k"), p.cuda("pos"), p.cuda("freq")
    with pytest.raises(TypeError):
        mdcn.rotary(q, k.float(), pos, f, p.sections)
    with pytest.raises(TypeError):
        mdcn.rotary(q, k, pos.long(), f, p.sections)
    with pytest.raises(ValueError):
        mdcn.rotary(q, k[:4], pos, f, p.sections)
    with pytest.raises(ValueError):
        mdcn.rotary(q, k, pos, f[:-1], p.sections)
    with pytest.raises(ValueError):
        mdcn.rotary(q.transpose(1, 2), None, pos, f, p.sections)
    with pytest.raises(ValueError):
        mdcn.rotary(q, k, pos, f, p.sections, layout="other")
    with pytest.raises(mdcn.MdcnError):
        mdcn.rotary(q, k, pos, f, p.sections, q_weight=p.cuda("qw"))  # a weight without norm
    with pytest.raises(mdcn.MdcnError):
        mdcn.rotary(q[:1].expand(8, 2, 64), k, pos, f, p.sections)  # a stride of 0
