"""The operators around the routed experts on the GPU, against plain evaluations in 64 bits.

Tolerances.  u = 2^-24 is fp32's rounding unit.  A sigmoid or softmax score is an exponential (at
most 2 ulp), an addition or a sum over a tree, and a division: relative error below 16 u; a weight
adds a sum of k and a division: below 32 u.  The choice compares c = score + bias in fp32, so an
expert can stand where 64 bits would not put it only when the two c differ by less than SLACK =
16 u * (1 + max|bias|) * 2.  Products of codes are exact integers: their fp32 outputs have to be
equal, bit by bit, to the same two fp32 multiplications."""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FLT_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def chord():
    import w4a16_int4_mixture_gb300 as m
    m.build()
    return m


# ------------------------------------------------------------------------------- router
def scores64(x, scoring):
    """-> (x with NaN as -inf and +inf as FLT_MAX, scores), float64."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, FLT_MAX)).astype(np.float64)
    with np.errstate(over="ignore", under="ignore"):
        if scoring == "sigmoid":
            return x, np.where(np.isneginf(x), 0.0, 1.0 / (1.0 + np.exp(-x)))
        top = np.max(x, 1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        e[np.isneginf(x)] = 0.0
        s = e.sum(1, keepdims=True)
        return x, e / np.where(s > 0, s, 1.0)


def group_scores(c, n_group, group_top):
    T, E = c.shape
    g = -np.sort(-c.reshape(T, n_group, E // n_group), axis=2)[:, :, :group_top]
    first = g[:, :, 0]
    rest = np.where(np.isneginf(g[:, :, 1:]), 0.0, g[:, :, 1:]).sum(2)
    return first + rest


def check_route(logits, bias, ids, w, k, scoring, n_group, topk_group, group_top, renorm, scale):
    x, s = scores64(logits, scoring)
    T, E = x.shape
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    c = np.where(np.isneginf(x), -np.inf, s + b)
    slack = 32 * U * (1 + np.abs(b).max())
    assert ids.shape == w.shape == (T, k) and ids.min() >= 0 and ids.max() < E
    gs = group_scores(c, n_group, group_top) if topk_group < n_group else None
    for t in range(T):
        row = ids[t]
        assert len(set(row.tolist())) == k, f"token {t}: an expert twice"
        allowed = np.ones(E, bool)
        if gs is not None:
            order = np.argsort(-gs[t], kind="stable")
            kept = set(order[:topk_group].tolist())
            edge = gs[t][order[topk_group - 1]]
            got = {int(e) // (E // n_group) for j, e in enumerate(row) if w[t, j] != 0}
            for g in got - kept:  # only a near tie may put another group in
                assert gs[t][g] >= edge - 2 * slack, f"token {t}: group {g}"
                kept = (kept - {min(kept - got, key=lambda q: gs[t][q])}) | {g}
            allowed = np.isin(np.arange(E) // (E // n_group), sorted(kept))
        key = np.where(allowed, c[t], -np.inf)
        n = min(k, int(np.sum(~np.isneginf(key))))
        # descending, nothing better left out
        assert np.all(np.diff(key[row[:n]]) <= slack), f"token {t}: order"
        left = np.setdiff1d(np.arange(E), row[:n])
        if n and left.size:
            assert key[left].max() <= key[row[:n]].min() + slack, f"token {t}: a better expert left"
        # slots that nothing can fill: the lowest ids not chosen, weight 0
        assert row[n:].tolist() == left[:k - n].tolist() and not w[t, n:].any(), f"token {t}: fill"
        sw = np.where(np.arange(k) < n, s[t][row], 0.0)
        if renorm:
            # the ratios of the scores, taken so that they survive where scores underflow in 64 bits
            if n:
                xc = x[t][row[:n]]
                m = min(xc.max(), 0.0) if scoring == "sigmoid" else xc.max()
                with np.errstate(over="ignore", under="ignore"):
                    e = np.exp(xc - m) if scoring == "softmax" else 1 / (np.exp(m) + np.exp(m - xc))
                sw[:n] = e / e.sum()
        tol = 32 * U * np.abs(scale * sw) + 1e-37
        assert np.all(np.abs(w[t] - scale * sw) <= tol), f"token {t}: weights"


def run_route(chord, logits, bias=None, **kw):
    ids, w = chord.moe_route(logits, bias=bias, **kw)
    torch.cuda.synchronize()
    a = dict(scoring="softmax", n_group=1, topk_group=1, group_top=2, renormalize=True, scale=1.0)
    a.update(kw)
    check_route(logits.float().cpu().numpy().astype(np.float64),
                None if bias is None else bias.cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(),
                a["k"], a["scoring"], a["n_group"], a["topk_group"], a["group_top"],
                a["renormalize"], a["scale"])
    return ids, w


ROUTES = [
    # T, E, k, scoring, bias, groups, kept, top, renorm, scale, type
    (1, 384, 8, "sigmoid", True, 1, 1, 2, True, 2.5, "f32"),
    (1, 1, 1, "softmax", False, 1, 1, 2, True, 1.0, "f32"),
    (5, 7, 7, "sigmoid", True, 1, 1, 2, False, 1.0, "bf16"),
    (33, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "bf16"),
    (33, 256, 8, "softmax", False, 8, 3, 1, True, 16.0, "f32"),
    (40, 160, 6, "softmax", True, 5, 2, 2, False, 1.0, "f16"),
    (64, 1024, 32, "sigmoid", False, 32, 5, 2, True, 1.0, "f32"),
    (64, 1023, 31, "softmax", True, 1, 1, 2, True, 1.0, "f32"),
    (70, 96, 12, "sigmoid", True, 12, 12, 2, True, 1.0, "f32"),
    (70, 96, 4, "sigmoid", False, 3, 1, 1, True, 0.0, "f16"),
    (70, 24, 3, "softmax", False, 24, 3, 2, True, 1.0, "f32"),
    (1217, 129, 9, "sigmoid", True, 1, 1, 2, True, -1.5, "f32"),
    (1300, 512, 16, "softmax", False, 2, 1, 2, False, 1.0, "bf16"),
    (2500, 384, 8, "sigmoid", True, 1, 1, 2, True, 2.5, "f32"),
]


@pytest.mark.parametrize("T,E,k,scoring,bias,G,tg,top,renorm,scale,dt", ROUTES)
def test_route(chord, T, E, k, scoring, bias, G, tg, top, renorm, scale, dt):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + E)
    x = (2 * torch.randn(T, E, device=DEV, generator=g)).to(TYPES[dt])
    b = 0.1 * torch.randn(E, device=DEV, generator=g) if bias else None
    run_route(chord, x, b, k=k, scoring=scoring, n_group=G, topk_group=tg, group_top=top,
              renormalize=renorm, scale=scale)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [(1, 1), (8, 3)])
def test_route_masked_and_extreme_logits(chord, scoring, groups):
    """Rows with no, one and few experts left, infinities, NaN, the type's lowest value, ties."""
    inf, nan, E, k = math.inf, math.nan, 64, 8
    rows = [[-inf] * E, [nan] * E, [-inf] * 40 + [1.0] + [-inf] * 23, [inf] * 3 + [0.0] * 61,
            [0.0] * E, [-0.0, 0.0] * 32, [-FLT_MAX] * E, [FLT_MAX] * E,
            [-inf] * 60 + [nan, 0.5, -100.0, 100.0], [1.0, nan, -inf, inf] * 16,
            [200.0] * 5 + [-200.0] * 59, [-200.0] * E, [float(-i) for i in range(E)]]
    x = torch.tensor(rows, device=DEV)
    b = torch.linspace(-0.25, 0.25, E, device=DEV)
    for bias in (None, b):
        run_route(chord, x, bias, k=k, scoring=scoring, n_group=groups[0], topk_group=groups[1])
        run_route(chord, x, bias, k=k, scoring=scoring, renormalize=False)
    if groups == (1, 1):  # (ties to the lower id)
        ids, _ = chord.moe_route(x, k, scoring=scoring)
        assert ids[4].tolist() == ids[5].tolist() == list(range(8))
        assert ids[2].tolist() == [40, 0, 1, 2, 3, 4, 5, 6]


def test_route_nan_bias_masks(chord):
    x = torch.randn(3, 16, device=DEV)
    b = torch.zeros(16, device=DEV)
    b[::2] = math.nan
    ids, w = chord.moe_route(x, 8, bias=b, scoring="sigmoid")
    assert (ids % 2 == 1).all() and (w > 0).all()


def test_route_strided_empty_and_out(chord):
    base = torch.randn(50, 200, device=DEV)
    x = base[::2, 3:131]
    ids, w = chord.moe_route(x, 4, scoring="sigmoid")
    ids2, w2 = chord.moe_route(x.contiguous(), 4, scoring="sigmoid",
                               out=(torch.empty(25, 4, dtype=torch.int32, device=DEV),
                                    torch.empty(25, 4, device=DEV)))
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    ids, w = chord.moe_route(base[:0], 4)
    assert tuple(ids.shape) == tuple(w.shape) == (0, 4)
    assert chord.moe_route_backward(w, base[:0], ids, w).shape == (0, 200)


def test_route_softmax_equals_route_align(chord):
    """Without bias and groups: the choice of chord_moe_route_align."""
    x = torch.randn(300, 384, device=DEV)
    ids, w = chord.moe_route(x, 8)
    ids2, w2, *_ = chord.moe_route_align(x, 8, 384)
    assert torch.equal(ids, ids2)
    assert ((w - w2).abs() <= 64 * U * w2).all()


# ----------------------------------------------------------------------- router's gradient
def backward64(g, x, ids, scoring, renorm, scale):
    """float64 autograd of the definition with the choice held."""
    x = torch.tensor(x, dtype=torch.float64, requires_grad=True)
    s = torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x, 1)
    w = s.gather(1, torch.tensor(ids, dtype=torch.int64))
    if renorm:
        w = w / w.sum(1, keepdim=True)
    ((scale * w) * torch.tensor(g, dtype=torch.float64)).sum().backward()
    return x.grad.numpy()


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,scale,dt", [(1, 384, 8, 2.5, "f32"), (37, 257, 6, 1.0, "f32"),
                                            (50, 8, 8, 1.0, "f32"), (1500, 384, 8, -0.5, "f32"),
                                            (9, 1024, 32, 1.0, "f32"), (130, 64, 1, 1.0, "bf16"),
                                            (2000, 100, 7, 2.5, "f16")])
def test_route_backward(chord, scoring, renorm, T, E, k, scale, dt):
    gen = torch.Generator(device="cuda").manual_seed(E + k)
    x = torch.randn(T, E, device=DEV, generator=gen).to(TYPES[dt])
    g = torch.randn(T, k, device=DEV, generator=gen)
    ids, w = chord.moe_route(x, k, scoring=scoring, renormalize=renorm, scale=scale)
    d = chord.moe_route_backward(g, x, ids, w, scoring=scoring, renormalize=renorm, scale=scale)
    ref = backward64(g.cpu().numpy(), x.double().cpu().numpy(), ids.cpu().numpy(), scoring, renorm, scale)
    got = d.double().cpu().numpy()
    assert d.dtype == x.dtype and got.shape == ref.shape
    # each entry is a few products of w (32 u) and a sum of k terms |g_j w_j| (16 u each way)
    gw = np.abs(g.cpu().numpy() * w.cpu().numpy()).sum(1, keepdims=True)
    wi = np.zeros((T, E))
    np.put_along_axis(wi, ids.cpu().numpy().astype(np.int64), np.abs(w.cpu().numpy()), 1)
    gmax = np.abs(g.cpu().numpy()).max(1, keepdims=True)
    tol = 128 * U * (wi * (gmax + gw / abs(scale)) + gw * (scores64(x.double().cpu().numpy(), "softmax")[1]))
    out_u = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -10}[dt]
    assert np.all(np.abs(got - ref) <= tol + out_u * np.abs(ref) + (2.0 ** -24 if dt == "f16" else 1e-37))


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_differences(chord, scoring, renorm):
    """Against central differences of the forward kernel itself, the choice unchanged by them.

    Step h = 2^-6 in x: truncation below h^2 * max third derivative (1 for these scores) * sum|g|,
    rounding 64 u * sum|g w| / h."""
    E, k, h, scale = 16, 4, 2.0 ** -6, 1.5
    x = torch.zeros(1, E, device=DEV)
    x[0, [3, 7, 9, 12]] = torch.tensor([2.0, 1.5, 1.0, 0.5], device=DEV)  # gaps far above 2 h
    x[0, 0] = -1.0
    g = torch.tensor([[0.7, -1.1, 0.4, 0.9]], device=DEV)
    kw = dict(scoring=scoring, renormalize=renorm, scale=scale)
    ids, w = chord.moe_route(x, k, **kw)
    d = chord.moe_route_backward(g, x, ids, w, **kw)[0].cpu().numpy()
    # one batch of 2 E perturbed rows
    step = h * torch.eye(E, device=DEV)
    rows = torch.cat([x + step, x - step])
    ids2, w2 = chord.moe_route(rows, k, **kw)
    assert torch.equal(ids2, ids.expand(2 * E, k))
    f = (w2.double() * g.double()).sum(1).cpu().numpy()
    num = (f[:E] - f[E:]) / (2 * h)
    tol = scale * float(g.abs().sum()) * (h * h + 64 * U / h)
    assert np.abs(d - num).max() <= tol


def test_route_backward_masked_slots_and_foreign_ids(chord):
    x = torch.full((2, 16), -math.inf, device=DEV)
    x[0, 3] = 1.0
    ids, w = chord.moe_route(x, 4, scoring="sigmoid")
    for scoring in ("sigmoid", "softmax"):
        for renorm in (True, False):
            d = chord.moe_route_backward(torch.ones(2, 4, device=DEV), x, ids, w, scoring=scoring,
                                         renormalize=renorm)
            assert torch.isfinite(d).all() and not d[1].any()
            assert not d[0, torch.arange(16, device=DEV) != 3].any()
    bad = torch.tensor([[3, -1, 16, 5]] * 2, dtype=torch.int32, device=DEV)
    d = chord.moe_route_backward(torch.ones(2, 4, device=DEV), torch.zeros(2, 16, device=DEV), bad,
                                 torch.full((2, 4), 0.25, device=DEV), scoring="sigmoid",
                                 renormalize=False)
    assert set(d.nonzero()[:, 1].tolist()) == {3, 5}


# ------------------------------------------------------------------------- quantisation
def quantize_ref(x):
    """The definition, each step one fp32 operation: bit-exact."""
    x = x.astype(np.float32)
    m = np.abs(x).max(1)
    bad, tiny = ~np.isfinite(x).all(1), m < np.float32(2.0 ** -100)
    m1 = np.where(bad | tiny, np.float32(1), m).astype(np.float32)
    inv = (np.float32(127) * (np.float32(1) / m1).astype(np.float32)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = np.rint((x * inv[:, None]).astype(np.float32))
    q[bad | tiny] = 0
    s = np.where(tiny, np.float32(0), (m1 / np.float32(127)).astype(np.float32))
    return q.astype(np.int8), np.where(bad, np.float32(np.nan), s).astype(np.float32)


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("T,K,pad", [(1, 1, 0), (3, 7, 0), (4, 64, 0), (5, 1003, 0), (7, 1000, 3),
                                     (2, 7168, 0), (400, 2048, 8), (2, 70001, 0)])
def test_quantize(chord, T, K, pad, dt):
    g = torch.Generator(device="cuda").manual_seed(K)
    x = (torch.randn(T, K + pad, device=DEV, generator=g) * 3).to(TYPES[dt])[:, pad:]
    q, s = chord.int8_quantize(x)
    assert q.dtype == torch.int8 and tuple(q.shape) == (T, K) and (T == 1 or q.stride(0) % 16 == 0)
    rq, rs = quantize_ref(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs)


def test_quantize_zero_tiny_and_not_finite_rows(chord):
    x = torch.randn(8, 40, device=DEV)
    x[0] = 0
    x[1] *= 1e-33
    x[2, 5] = math.inf
    x[3, 39] = math.nan
    x[4] = 0.01
    x[4, 7] = FLT_MAX
    x[5] = 2.0 ** -100
    x[6, 1] = -math.inf
    x[6, 2] = math.nan
    q, s = chord.int8_quantize(x)
    rq, rs = quantize_ref(x.cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("T,I,pad", [(1, 1, 0), (3, 100, 0), (5, 333, 1), (300, 2048, 0), (2, 40000, 4)])
def test_silu_mul_quantize(chord, T, I, pad, dt):
    """h is within 16 u of its value for |g| <= 16 (the exponential's argument is rounded), so a
    code is the nearest to 127 h / max|h| within 127 * 64 u + the rounding's half."""
    g = torch.Generator(device="cuda").manual_seed(I)
    gu = (2 * torch.randn(T, 2 * I + pad, device=DEV, generator=g)).to(TYPES[dt])[:, pad:]
    q, s = chord.int8_silu_mul_quantize(gu)
    v = gu.double().cpu().numpy()
    h = v[:, :I] / (1 + np.exp(-v[:, :I])) * v[:, I:]
    m = np.abs(h).max(1)
    assert np.all(np.abs(s.cpu().numpy() - m / 127) <= 64 * U * m / 127)
    assert np.abs(q.cpu().numpy() - 127 * h / m[:, None]).max() <= 0.5 + 127 * 128 * U


def test_silu_mul_quantize_extremes(chord):
    gu = torch.tensor([[-200.0, 200.0, 0.0, -FLT_MAX, 1.0, 2.0, 3.0, 4.0]], device=DEV)
    q, s = chord.int8_silu_mul_quantize(gu)
    assert q.tolist() == [[0, 127, 0, 0]] and abs(s.item() - 400 / 127) < 1e-5
    gu[0, 6] = math.inf  # 0 * inf
    q, s = chord.int8_silu_mul_quantize(gu)
    assert math.isnan(s.item()) and not q.any()


# ------------------------------------------------------------------------------ products
def codes(T, K, g, lo=-128, pad=0):
    ld = (K + 15) // 16 * 16 + pad
    return torch.randint(lo, 128, (T, ld), dtype=torch.int8, device=DEV, generator=g)[:, :K]


def product_ref(a, w):
    return (a.double().cpu() @ w.double().cpu().t()).numpy()  # exact: below 2^53


def scaled_ref(p, sa, sw):
    v = p.astype(np.float32) * sa.cpu().numpy()[:, None]
    return v.astype(np.float32) * sw.cpu().numpy()[None, :]


MATMULS = [(1, 1, 1), (1, 4096, 7168), (2, 3, 16), (3, 130, 17), (4, 64, 64), (5, 129, 127),
           (8, 1000, 2048), (9, 128, 128), (16, 256, 1024), (17, 100, 1025), (31, 257, 2049),
           (33, 1111, 1003), (64, 384, 4100), (65, 640, 512), (127, 200, 130), (128, 2048, 256),
           (129, 130, 3000), (200, 5000, 96), (300, 7168, 2048), (513, 777, 1500),
           (1000, 4096, 700), (1537, 1300, 2304), (160, 4096, 4500), (300, 2048, 6100),
           (384, 9700, 1100), (1150, 9700, 700)]


@pytest.mark.parametrize("T,N,K", MATMULS)
def test_matmul_is_exact(chord, T, N, K):
    g = torch.Generator(device="cuda").manual_seed(T + N + K)
    a, w = codes(T, K, g, pad=16 * (T % 2)), codes(N, K, g, pad=16 * (N % 3))
    sa, sw = torch.rand(T, device=DEV, generator=g) + 0.5, torch.rand(N, device=DEV, generator=g)
    y = chord.int8_matmul(a, sa, w, sw, out_dtype=torch.float32, flags=1)
    ref = scaled_ref(product_ref(a, w), sa, sw)
    assert np.array_equal(y.cpu().numpy(), ref)
    # 16-bit outputs: one rounding of the same value
    for dt in (torch.bfloat16, torch.float16):
        y = chord.int8_matmul(a, sa / 2 ** 20, w, sw, out_dtype=dt)
        want = torch.from_numpy(scaled_ref(product_ref(a, w), sa / 2 ** 20, sw)).to(dt)
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("T", [1, 7, 20, 70, 400])
@pytest.mark.parametrize("K", [1024, 4096, 20000])
def test_matmul_largest_sums(chord, T, K):
    """Codes at their ends, all of one sign: every partial sum is as large as it can be."""
    N = 140
    a = torch.full((T, (K + 15) // 16 * 16), -128, dtype=torch.int8, device=DEV)[:, :K]
    w = torch.full((N, (K + 15) // 16 * 16), -128, dtype=torch.int8, device=DEV)[:, :K]
    w[1::2] = 127
    w[::5, 1::2] = 127
    one_a, one_w = torch.ones(T, device=DEV), torch.ones(N, device=DEV)
    y = chord.int8_matmul(a, one_a, w, one_w, out_dtype=torch.float32)
    assert np.array_equal(y.cpu().numpy(), product_ref(a, w).astype(np.float32))


@pytest.mark.parametrize("T", [3, 50, 300])
@pytest.mark.parametrize("dt", sorted(TYPES))
def test_matmul_residual_strides_and_out(chord, T, dt):
    N, K = 333, 400
    g = torch.Generator(device="cuda").manual_seed(T)
    a, w = codes(T, K, g), codes(N, K, g)
    sa, sw = torch.rand(T, device=DEV, generator=g) / 4096, torch.rand(N, device=DEV, generator=g)
    r = torch.randn(T, N + 5, device=DEV, generator=g).to(TYPES[dt])[:, 2:2 + N]
    v = scaled_ref(product_ref(a, w), sa, sw).astype(np.float64)
    want = v + r.double().cpu().numpy()
    out = torch.zeros(T, N + 3, dtype=TYPES[dt], device=DEV)
    y = chord.int8_matmul(a, sa, w, sw, residual=r, out=out[:, 1:1 + N])
    assert y.data_ptr() == out[:, 1:].data_ptr()
    assert not out[:, 0].any() and not out[:, 1 + N:].any()
    # v is rounded twice in fp32, the sum once, then to the type
    tol = 4 * U * (np.abs(v) + np.abs(want)) + \
        {"f32": 0, "bf16": 2.0 ** -9, "f16": 2.0 ** -12}[dt] * 2 * np.abs(want)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)
    # in place: the residual is the output
    z = r.clone()
    chord.int8_matmul(a, sa, w, sw, residual=z, out=z)
    assert torch.equal(z, y)


def test_matmul_nan_scale_stays_in_its_row(chord):
    g = torch.Generator(device="cuda").manual_seed(0)
    for T in (4, 60, 260):
        x = torch.randn(T, 256, device=DEV, generator=g)
        x[2, 9] = math.nan
        w, ws = chord.int8_quantize(torch.randn(200, 256, device=DEV, generator=g))
        y = chord.int8_linear(x, w, ws)
        assert y[2].isnan().all() and torch.isfinite(y[torch.arange(T, device=DEV) != 2]).all()


def test_codes_past_the_row_are_ignored(chord):
    """Padding bytes between the rows hold anything; the last row may end its allocation."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for T, N, K in ((2, 40, 33), (30, 140, 130), (260, 300, 513)):
        ld = (K + 15) // 16 * 16
        a = codes(T, K, g)
        flat = torch.full((ld * (N - 1) + K,), 99, dtype=torch.int8, device=DEV)
        w = flat.as_strided((N, K), (ld, 1))
        w.copy_(codes(N, K, g))
        y = chord.int8_matmul(a, torch.ones(T, device=DEV), w, torch.ones(N, device=DEV),
                              out_dtype=torch.float32)
        assert np.array_equal(y.cpu().numpy(), product_ref(a, w).astype(np.float32))


@pytest.mark.parametrize("T,H,I,dt", [(1, 64, 32, "bf16"), (3, 250, 100, "f16"), (20, 1024, 384, "bf16"),
                                      (70, 512, 1000, "f32"), (300, 768, 640, "bf16")])
def test_linear_and_mlp_are_their_parts(chord, T, H, I, dt):
    """Bit-equal to quantise, product, quantise, product; and near the fp64 definition."""
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn(T, H, device=DEV, generator=g).to(TYPES[dt])
    w13, s13 = chord.int8_quantize(torch.randn(2 * I, H, device=DEV, generator=g) / H ** 0.5)
    w2, s2 = chord.int8_quantize(torch.randn(H, I, device=DEV, generator=g) / I ** 0.5)
    r = torch.randn(T, H, device=DEV, generator=g).to(TYPES[dt])
    q, qs = chord.int8_quantize(x)
    gu = chord.int8_matmul(q, qs, w13, s13, out_dtype=torch.float32)
    q2, qs2 = chord.int8_silu_mul_quantize(gu)
    want = chord.int8_matmul(q2, qs2, w2, s2, residual=r, out_dtype=x.dtype)
    assert torch.equal(chord.int8_mlp(x, w13, s13, w2, s2, residual=r, flags=1), want)
    y = r.clone()
    chord.int8_mlp(x, w13, s13, w2, s2, residual=y, out=y)
    assert torch.equal(y, want)
    lin = chord.int8_linear(x, w13, s13)
    assert torch.equal(lin, chord.int8_matmul(q, qs, w13, s13, out_dtype=x.dtype))
    # the definition without quantisation of the tokens: 8-bit steps of x and h are 1/127 of
    # their row's largest value, uniform errors of a half step add up like random signs
    x64 = x.double()
    g64 = x64 @ (w13.double() * s13.double()[:, None]).t()
    h64 = torch.nn.functional.silu(g64[:, :I]) * g64[:, I:]
    y64 = h64 @ (w2.double() * s2.double()[:, None]).t() + r.double()
    assert ((want.double() - y64).norm() / y64.norm()).item() <= 0.05


def test_offsets_past_32_bits(chord):
    """More than 2^32 elements in an operand or an output: the last rows are right."""
    g = torch.Generator(device="cuda").manual_seed(2)
    T, N, K = 140000, 32768, 64
    a, w = codes(T, K, g), codes(N, K, g)
    sa, sw = torch.rand(T, device=DEV, generator=g) / 4096, torch.rand(N, device=DEV, generator=g)
    y = chord.int8_matmul(a, sa, w, sw)
    for rows in (slice(0, 3), slice(T - 5, T)):
        want = torch.from_numpy(scaled_ref(product_ref(a[rows], w), sa[rows], sw)).bfloat16()
        assert torch.equal(y[rows].cpu(), want)
    del y
    x = torch.zeros((1 << 22) + 9, 1024, dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn(3, 1024, device=DEV, generator=g).bfloat16()
    q, s = chord.int8_quantize(x)
    rq, rs = quantize_ref(x[-3:].float().cpu().numpy())
    assert np.array_equal(q[-3:].cpu().numpy(), rq) and np.array_equal(s[-3:].cpu().numpy(), rs)
    ids, w = chord.moe_route(x, 8, scoring="sigmoid")
    ids3, w3 = chord.moe_route(x[-3:].clone(), 8, scoring="sigmoid")
    assert torch.equal(ids[-3:], ids3) and torch.equal(w[-3:], w3)
    d = chord.moe_route_backward(torch.ones_like(w), x, ids, w, scoring="softmax", renormalize=False)
    d3 = chord.moe_route_backward(torch.ones_like(w3), x[-3:].clone(), ids3, w3, scoring="softmax",
                                  renormalize=False)
    assert torch.equal(d[-3:], d3)


def test_empty_batches(chord):
    w, s = chord.int8_quantize(torch.randn(48, 32, device=DEV))
    x = torch.zeros(0, 32, device=DEV)
    q, qs = chord.int8_quantize(x)
    assert tuple(q.shape) == (0, 32) and qs.numel() == 0
    assert tuple(chord.int8_linear(x, w, s).shape) == (0, 48)
    assert tuple(chord.int8_matmul(q, qs, w, s).shape) == (0, 48)


def test_refusals_on_device(chord):
    w, s = chord.int8_quantize(torch.randn(48, 32, device=DEV))
    x = torch.zeros(4, 32, device=DEV)
    with pytest.raises(ValueError, match="16-byte"):
        chord.int8_linear(x, w.contiguous().view(-1)[1:1 + 31 * 32].view(31, 32), s[:31].clone())
    with pytest.raises(ValueError, match="disagree"):
        chord.int8_linear(torch.zeros(4, 16, device=DEV), w, s)
    with pytest.raises(ValueError, match="overlap"):
        chord.int8_linear(torch.zeros(1, 32, device=DEV).expand(4, 32), w, s)
    with pytest.raises(ValueError, match="contiguous"):
        chord.moe_route(torch.zeros(8, 4, device=DEV).t(), 2)
    with pytest.raises(ValueError):
        chord.int8_linear(x, w, s[:47])
    with pytest.raises(ValueError, match="residual"):
        chord.int8_linear(x, w, s, residual=torch.zeros(4, 47, device=DEV))
    with pytest.raises(TypeError):
        chord.int8_linear(x, w, s, residual=torch.zeros(4, 48, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError, match="scoring"):
        chord.moe_route(x, 2, scoring="relu")
    with pytest.raises(chord.ChordError):
        chord.moe_route(x, 33)
    with pytest.raises(chord.ChordError):
        chord.int8_linear(x, w, s, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    odd = torch.randint(-9, 9, (5, 33), dtype=torch.int8, device=DEV)
    with pytest.raises(ValueError, match="16-byte"):
        chord.int8_matmul(odd, torch.ones(5, device=DEV), odd, torch.ones(5, device=DEV))
    rows = chord.int8_rows(odd)
    y = chord.int8_matmul(rows, torch.ones(5, device=DEV), rows, torch.ones(5, device=DEV),
                          out_dtype=torch.float32)
    assert np.array_equal(y.cpu().numpy(), product_ref(odd, odd).astype(np.float32))


def test_other_stream_and_graph(chord):
    """Calls on a side stream, and captured in a graph and replayed on new inputs."""
    g = torch.Generator(device="cuda").manual_seed(5)
    w13, s13 = chord.int8_quantize(torch.randn(256, 384, device=DEV, generator=g) / 20)
    w2, s2 = chord.int8_quantize(torch.randn(384, 128, device=DEV, generator=g) / 11)
    for T in (3, 40, 200):
        x = torch.randn(T, 384, device=DEV, generator=g)
        want = chord.int8_mlp(x, w13, s13, w2, s2)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = chord.int8_mlp(x, w13, s13, w2, s2)
            ids, w = chord.moe_route(x, 8, scoring="sigmoid")
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        static = torch.zeros_like(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = chord.int8_mlp(static, w13, s13, w2, s2)
            i2, w2_ = chord.moe_route(static, 8, scoring="sigmoid")
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(i2, ids) and torch.equal(w2_, w)


def test_mixture_block(chord):
    """Router, routed experts and shared expert together, against the parts and fp64."""
    import fp64_ref  # noqa: F401  (the routed layer has its own fp64 tests)
    from w4a16_int4_mixture_gb300 import synth
    from gpu_util import dev_tensor, weights_to

    s = synth.workload("tiny")
    inp = synth.make_inputs(s)
    x = dev_tensor(inp.x, DEV, True)
    wts = weights_to(inp, DEV)
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(s.T, s.E_global, device=DEV, generator=g)
    bias = 0.05 * torch.randn(s.E_global, device=DEV, generator=g)
    w13, s13 = chord.int8_quantize(torch.randn(256, s.H, device=DEV, generator=g) / s.H ** 0.5)
    w2, s2 = chord.int8_quantize(torch.randn(s.H, 128, device=DEV, generator=g) / 128 ** 0.5)
    kw = dict(bias=bias, scoring="sigmoid", n_group=2, topk_group=1, scale=2.5)
    y = chord.moe_block(x, logits, s.k, wts, (w13, s13, w2, s2), flags=2, **kw)
    ids, w = chord.moe_route(logits, s.k, **kw)
    routed = chord.w4a16_moe(x, ids, w, *wts, E_global=s.E_global, flags=2)
    assert torch.equal(y, chord.int8_mlp(x, w13, s13, w2, s2, residual=routed))
    packed = chord.prepack_weights(*wts)
    assert torch.equal(chord.moe_block(x, logits, s.k, packed, flags=2, **kw), routed)


def test_threads_on_one_stream(chord):
    """Two host threads whose calls' launches mix on one stream do not share a workspace."""
    import threading

    g = torch.Generator(device="cuda").manual_seed(8)
    w13, s13 = chord.int8_quantize(torch.randn(256, 384, device=DEV, generator=g) / 20)
    w2, s2 = chord.int8_quantize(torch.randn(384, 128, device=DEV, generator=g) / 11)
    xs = [torch.randn(40, 384, device=DEV, generator=g) for _ in range(2)]
    want = [chord.int8_mlp(x, w13, s13, w2, s2) for x in xs]
    got = [[], []]

    def calls(i):
        for _ in range(200):
            got[i].append(chord.int8_mlp(xs[i], w13, s13, w2, s2))

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 200 and all(torch.equal(y, want[i]) for y in got[i])
