"""Router losses and their gradient, layer norm, 4-bit weights and the expert FFN over them, on a
GPU, each against a plain implementation in 64 bits.

Tolerances are bounds from the arithmetic, stated where they are formed: U = 2^-24 is the largest
relative error of one fp32 rounding, HALF[dtype] that of the result's one rounding."""
import ctypes
import math

import pytest
import torch

from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = math.inf


@pytest.fixture(scope="module")
def moe():
    from expert_ffn_layer_router_b200 import moe as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=dev())


def assert_within(got, ref, tol, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what + ": not finite"
    over = (got - ref).abs() - tol
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0.0, "%s: over its bound by %.3g" % (what, worst)


def status(moe, layer):
    return moe.moe_get_device_status(layer.ws)


# ----------------------------------------------------------------------------------------------
# Router losses
# ----------------------------------------------------------------------------------------------
def balance_reference(logits, ids, keep, k, renorm, grad_losses, grad_w):
    """Losses, counts, probs, dlogits in 64 bits from the formulas, and the magnitude of the terms
    each dlogits element is made of."""
    T, E = logits.shape
    L = logits.double()[keep]
    I = ids.long()[keep]
    n = L.shape[0]
    p = torch.softmax(L, 1)
    lse = torch.logsumexp(L, 1)
    ok = (I >= 0) & (I < E)
    one = torch.zeros(n, E, dtype=torch.float64, device=dev())
    one.scatter_add_(1, I.clamp(0, E - 1), ok.double())
    counts = one.sum(0)
    d = max(n, 1)
    f, P = counts / (d * k), p.sum(0) / d
    losses = torch.stack([E * (f * P).sum(), (lse ** 2).sum() / d])
    gb, gz = (0.0, 0.0) if grad_losses is None else grad_losses.double().tolist()
    a = (gb * E / d * f)[None, :].expand(n, E).clone()
    mag = a.abs()
    if grad_w is not None:
        dw = grad_w.double()[keep] * ok
        m = dw.abs()
        if renorm:
            pk = torch.gather(p, 1, I.clamp(0, E - 1)) * ok
            S = pk.sum(1, keepdim=True)
            m = (m + (m * pk).sum(1, keepdim=True) / S) / S
            dw = (dw - (dw * pk).sum(1, keepdim=True) / S) / S
        dw, m = dw * ok, m * ok                      # a bad id has no weight
        a.scatter_add_(1, I.clamp(0, E - 1), dw)
        mag = mag.scatter_add(1, I.clamp(0, E - 1), m)
    zt = 2 * gz / d * lse[:, None]
    dl = torch.zeros(T, E, dtype=torch.float64, device=dev())
    dl[keep] = p * (a - (p * a).sum(1, keepdim=True)) + zt * p
    terms = torch.zeros_like(dl)
    terms[keep] = p * (mag + (p * mag).sum(1, keepdim=True) + zt.abs())
    return losses, torch.cat([counts, torch.tensor([float(n)], device=dev())]), P, dl, terms


def balance_bound(logits, keep):
    """Relative error of a probability, in units of U: the rounding of L - max (|L - max| U in the
    exponent), exp within 2 ulp (4 U), the sum over the row (a lane's 32 terms and 5 tree steps),
    the reciprocal and the product; twice that for the products and sums made from it."""
    L = logits.double()[keep]
    L = torch.where(torch.isfinite(L), L, L.new_zeros(()))
    span = (L.amax(1) - L.amin(1)).max().item() if L.numel() else 0.0
    return 2 * (span + 4 + 37 + 4)


CASES = [  # T, E, k, mask, renorm, grad_w
    (1, 4, 1, None, False, False),
    (1, 1, 1, None, True, True),
    (7, 5, 2, "some", False, True),
    (33, 8, 8, None, True, True),
    (20, 16, 16, "some", True, True),
    (64, 64, 8, None, False, False),
    (50, 32, 32, None, True, True),
    (513, 60, 6, "some", False, True),
    (1000, 257, 3, "some", True, True),
    (4097, 64, 6, "some", True, True),
    (300, 384, 4, None, False, True),
    (200, 1000, 32, "some", True, True),
    (1500, 1024, 2, None, False, False),
    (20000, 128, 8, "some", True, True),
    (64, 64, 8, "all", False, True),
    (4000, 64, 8, "all", True, True),
    (9, 64, 2, "one", True, True),
]


@pytest.mark.parametrize("T,E,k,mask,renorm,grad_w", CASES)
def test_balance_loss_and_gradient(moe, T, E, k, mask, renorm, grad_w):
    g = gen(T * 1000 + E)
    logits = 3 * randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    keep = torch.ones(T, dtype=torch.bool, device=dev())
    if mask == "some":
        keep = torch.rand(T, generator=g, device=dev()) < 0.7
    elif mask:
        keep[:] = False
        if mask == "one":
            keep[T // 2] = True
    # What the mask leaves out may hold anything.
    bad = [math.nan, INF, -INF]
    logits[~keep] = torch.tensor([bad[i % 3] for i in range(E)], device=dev())
    ids[~keep] = 2 ** 30
    gl = torch.tensor([0.7, -0.3], device=dev())
    gw = randn(g, T, k) if grad_w else None
    layer = moe.MoELayer(T, 64, 64, E, k, flags=moe.FLAG_RENORMALIZE if renorm else 0)
    m = None if mask is None else keep.to(torch.uint8)
    losses, counts, probs = layer.balance_loss(logits, ids, mask=m)
    dl = layer.route_backward(logits, ids, counts, gl, gw, mask=m)
    ref = balance_reference(logits, ids, keep, k, renorm, gl, gw)
    b = balance_bound(logits, keep)
    # Sums over tokens: a thread adds at most T / 36 terms and 64 partial sums follow.
    bt = b + T / 36 + 64
    assert torch.equal(counts.double(), ref[1])
    assert_within(probs, ref[2], 2 * bt * U * ref[2], "probs")
    lse_max = ref[0][1].item() ** 0.5 + 1
    assert_within(losses, ref[0], 4 * bt * U * (ref[0] + torch.tensor([0.0, lse_max],
                                                                      device=dev())), "losses")
    # (renormalised weights divide by S: two more divisions and two sums of k terms)
    assert_within(dl, ref[3], (4 * b + 64) * U * ref[4] + 1e-37, "dlogits")
    assert status(moe, layer) == 0
    assert (dl[~keep] == 0).all()
    # Each part alone, and both runs the same bits.
    if grad_w:
        only = layer.route_backward(logits, ids, grad_w=gw, mask=m)
        r = balance_reference(logits, ids, keep, k, renorm, None, gw)
        assert_within(only, r[3], (4 * b + 64) * U * r[4] + 1e-37, "dlogits of the weights alone")
    again = layer.balance_loss(logits, ids, mask=m) + (
        layer.route_backward(logits, ids, counts, gl, gw, mask=m),)
    for x, y in zip(again, (losses, counts, probs, dl)):
        assert torch.equal(x, y)


def test_balance_excluded_experts_and_wide_logits(moe):
    """-infinity logits are experts a token cannot take; far-apart logits underflow cleanly."""
    T, E, k = 257, 40, 2
    g = gen(5)
    logits = 60 * randn(g, T, E)
    logits[:, 3] = -INF
    logits[5, :39] = -INF
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    keep = torch.ones(T, dtype=torch.bool, device=dev())
    layer = moe.MoELayer(T, 64, 64, E, k)
    losses, counts, probs = layer.balance_loss(logits, ids)
    gl = torch.tensor([1.0, 1.0], device=dev())
    dl = layer.route_backward(logits, ids, counts, gl)
    ref = balance_reference(logits, ids, keep, k, False, gl, None)
    b = balance_bound(logits, keep)
    assert_within(losses, ref[0], 4 * (b + 64) * U * ref[0], "losses")
    assert_within(probs, ref[2], 2 * (b + 64) * U * ref[2] + 1e-37, "probs")
    assert_within(dl, ref[3], (4 * b + 64) * U * ref[4] + 1e-37, "dlogits")
    assert (dl[:, 3] == 0).all() and probs[3] == 0


def test_balance_gradient_against_differences(moe):
    """dlogits . v against the central difference of the losses the forward gives.  With step h the
    losses (about 1 and 17, forward error below 4 b U of that) give the difference to 8 b U loss /
    (2 h); the third-order term is below h^2 times the losses (derivatives of softmax terms are
    bounded by a few times the value for |v| <= 1)."""
    T, E, k = 48, 24, 3
    g = gen(9)
    logits = randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    layer = moe.MoELayer(T, 64, 64, E, k)
    keep = torch.ones(T, dtype=torch.bool, device=dev())
    b = balance_bound(logits, keep) + 64
    h = 2.0 ** -5
    v = torch.sign(randn(g, T, E))
    for part in range(2):
        gl = torch.zeros(2, device=dev())
        gl[part] = 1.0
        losses, counts, _ = layer.balance_loss(logits, ids)
        dl = layer.route_backward(logits, ids, counts, gl)
        up = layer.balance_loss(logits + h * v, ids)[0][part].double()
        dn = layer.balance_loss(logits - h * v, ids)[0][part].double()
        got = (dl.double() * v).sum()
        tol = 8 * b * U * losses[part] / (2 * h) + h * h * losses[part]
        assert abs((up - dn) / (2 * h) - got) <= tol
        assert abs(got) > 4 * tol or part == 0


def test_balance_bad_and_repeated_ids(moe):
    T, E, k = 40, 16, 4
    g = gen(3)
    logits = randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    ids[7] = ids[7, 0]                               # the same expert four times
    ids[9, 2] = ids[9, 1]
    gl, gw = torch.tensor([0.5, 0.25], device=dev()), randn(g, T, k)
    keep = torch.ones(T, dtype=torch.bool, device=dev())
    b = balance_bound(logits, keep)
    for flags in (0, moe.FLAG_RENORMALIZE):
        layer = moe.MoELayer(T, 64, 64, E, k, flags=flags)
        for bad in (False, True):
            if bad:
                ids[3, 1], ids[11, 0] = -1, E
            losses, counts, probs = layer.balance_loss(logits, ids)
            code = status(moe, layer)
            moe.moe_reset_device_status(layer.ws)
            dl = layer.route_backward(logits, ids, counts, gl, gw)
            assert code == status(moe, layer) == (moe.DEV_BAD_INDEX if bad else 0)
            ref = balance_reference(logits, ids, keep, k, flags != 0, gl, gw)
            assert torch.equal(counts.double(), ref[1])
            assert_within(dl, ref[3], (4 * b + 64) * U * ref[4] + 1e-37, "dlogits")
        ids[3, 1], ids[11, 0] = 0, 0


def test_balance_unaligned_rows_and_no_tokens(moe):
    """Logits and dlogits that start off a 16-byte boundary, and T = 0."""
    T, E, k = 100, 64, 2
    g = gen(4)
    store, out = randn(g, T * E + 1), torch.full((T * E + 2,), 7.0, device=dev())
    logits = store[1:].view(T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    layer = moe.MoELayer(T, 64, 64, E, k)
    losses, counts, probs = layer.balance_loss(logits, ids)
    gl = torch.tensor([0.5, 0.25], device=dev())
    moe.moe_route_backward(layer.p, logits, ids, counts, out[1:], layer.ws, grad_losses=gl)
    aligned = logits.clone()
    l2, c2, p2 = layer.balance_loss(aligned, ids)
    d2 = layer.route_backward(aligned, ids, counts, gl)
    keep = torch.ones(T, dtype=torch.bool, device=dev())
    b = balance_bound(logits, keep)
    assert torch.equal(counts, c2)
    assert_within(probs, p2, 4 * (b + 64) * U * p2, "probs")
    assert_within(out[1:-1].view(T, E), d2, 8 * b * U, "dlogits")
    assert out[0] == 7.0 and out[-1] == 7.0
    none = moe.MoELayer(0, 64, 64, E, k)
    e = torch.empty(0, E, device=dev())
    i = torch.empty(0, k, dtype=torch.int32, device=dev())
    losses, counts, probs = none.balance_loss(e, i)
    assert (losses == 0).all() and (counts == 0).all() and (probs == 0).all()
    assert none.route_backward(e, i, counts, gl).shape == (0, E)


# ----------------------------------------------------------------------------------------------
# Layer norm
# ----------------------------------------------------------------------------------------------
def norm_reference(x, gamma, beta, eps, dy=None, dres=None):
    x, ga, be = x.double(), gamma.double(), beta.double()
    mu = x.mean(1, keepdim=True)
    rs = 1 / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + eps)
    xh = (x - mu) * rs
    r = dict(y=ga * xh + be, mean=mu[:, 0], rstd=rs[:, 0], xh=xh)
    if dy is not None:
        dy = dy.double()
        gy = dy * ga
        r["dgamma"], r["dbeta"] = (dy * xh).sum(0), dy.sum(0)
        r["dx"] = rs * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
        r["terms"] = rs * (gy.abs() + gy.abs().mean(1, keepdim=True) +
                           xh.abs() * (gy * xh).abs().mean(1, keepdim=True))
        r["sg"], r["sb"] = (dy * xh).abs().sum(0), dy.abs().sum(0)
        if dres is not None:
            r["dx"] = r["dx"] + dres.double()
            r["terms"] = r["terms"] + dres.double().abs()
    return r


def check_norm(layer, x, gamma, beta, eps, dy, dres):
    T, d = x.shape
    half = HALF[x.dtype]
    y, mean, rstd = layer.layer_norm(x, gamma, beta, eps)
    r = norm_reference(x, gamma, beta, eps, dy, dres)
    # A row sum: at most 40 additions behind one another (a lane's elements, the lanes, the warps;
    # d / 512 more in very wide rows), of terms of mean magnitude A.  The mean's error m moves xh
    # by m rstd; the variance's relative error is that of its sum plus twice m / std, and rstd's
    # half of it.
    n = (40 + max(0, d // 512 - 32)) * U
    A = x.double().abs().mean(1)
    em = n * A + U * r["mean"].abs()
    assert_within(mean, r["mean"], em + 1e-37, "mean")
    es = 2 * n + 4 * U + (em * r["rstd"]) ** 2 + 4 * em * r["rstd"]
    assert_within(rstd, r["rstd"], es * r["rstd"], "rstd")
    exh = (es + 4 * U)[:, None] * r["xh"].abs() + (em * r["rstd"])[:, None] + \
        U * (x.double().abs() * r["rstd"][:, None])
    ey = gamma.double().abs() * exh + 2 * U * r["y"].abs()
    assert_within(y, r["y"], ey + half * (r["y"].abs() + ey) + 1e-37, "y")
    dx, dgamma, dbeta = layer.layer_norm_backward(dy, x, gamma, mean, rstd, dres=dres)
    # dx: n and exh enter each of its terms at most twice (the row's largest |xh| bounds the mean
    # of g xh's error).
    rel = 2 * n + 8 * U + 2 * es[:, None]
    gy = (dy.double() * gamma.double()).abs()
    shift = r["rstd"][:, None] * (exh * (gy * r["xh"].abs()).mean(1, keepdim=True) +
                                  r["xh"].abs() * (gy * exh).mean(1, keepdim=True))
    ed = rel * r["terms"] + 2 * shift
    assert_within(dx, r["dx"], ed + half * (r["dx"].abs() + ed) + 1e-37, "dx")
    # Parameter sums: rows per thread, then at most 8 row groups and 300 / 8 + 8 partial rows.
    depth = (T / 8 + 64 + 8) * U
    eg = depth * r["sg"] + (dy.double().abs() * exh).sum(0)
    assert_within(dgamma, r["dgamma"], eg + 1e-37, "dgamma")
    assert_within(dbeta, r["dbeta"], depth * r["sb"] + 1e-37, "dbeta")
    a = layer.layer_norm_backward(dy, x, gamma, mean, rstd, dres=dres)
    for u, v in zip(a, (dx, dgamma, dbeta)):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 2), (5, 3), (1, 33), (9, 64), (64, 100), (2, 504),
                                 (700, 512), (33, 513), (17, 1000), (5, 1024), (300, 1408),
                                 (65, 2048), (7, 2049), (2400, 256), (11, 4096), (4, 5000),
                                 (3, 8192), (3, 8193), (2, 16384), (2, 16385), (3, 20000),
                                 (40, 16392)])
def test_layer_norm(moe, dtype, T, d):
    g = gen(T * 31 + d)
    x = (randn(g, T, d) * 2 + randn(g, T, 1)).to(DT[dtype])
    gamma, beta = 1 + 0.2 * randn(g, d), randn(g, d)
    dy = randn(g, T, d).to(DT[dtype])
    dres = randn(g, T, d).to(DT[dtype]) if (T + d) % 2 else None
    layer = moe.MoELayer(T, d, 64, 1, 1, dtype=dtype)
    check_norm(layer, x, gamma, beta, 1e-5, dy, dres)


def test_layer_norm_hard_rows(moe):
    """Constant rows (variance 0), rows far off zero, rows of the type's small and large values."""
    T, d = 6, 768
    g = gen(2)
    for dtype in ("bf16", "f32"):
        x = randn(g, T, d)
        x[0] = 3.0
        x[1] = 0.0
        x[2] = 100.0 + x[2]
        x[3] *= 1e-6
        x[4] *= 1e6
        x = x.to(DT[dtype])
        dy = randn(g, T, d).to(DT[dtype])
        layer = moe.MoELayer(T, d, 64, 1, 1, dtype=dtype)
        gamma, beta = randn(g, d), randn(g, d)
        check_norm(layer, x, gamma, beta, 1e-5, dy, None)
        y = layer.layer_norm(x, gamma, beta, 1e-5)[0]
        assert torch.equal(y[0], beta.to(DT[dtype]))


@pytest.mark.parametrize("d", [60, 768, 8200])
def test_layer_norm_variance_overflow(moe, d):
    """A row whose variance passes float32's range: rstd 0, y = beta and dx = dres, at every width;
    the other rows do not see it."""
    T = 5
    g = gen(d)
    for dtype in ("bf16", "f32"):
        x = randn(g, T, d)
        x[2] *= 1e25
        x = x.to(DT[dtype])
        gamma, beta = randn(g, d), randn(g, d)
        dy, dres = randn(g, T, d).to(DT[dtype]), randn(g, T, d).to(DT[dtype])
        layer = moe.MoELayer(T, d, 64, 1, 1, dtype=dtype)
        y, mean, rstd = layer.layer_norm(x, gamma, beta)
        assert rstd[2] == 0 and torch.equal(y[2], beta.to(DT[dtype]))
        dx, dg, db = layer.layer_norm_backward(dy, x, gamma, mean, rstd, dres)
        assert torch.equal(dx[2], dres[2]) and torch.isfinite(dg).all() and torch.isfinite(db).all()
        keep = torch.tensor([0, 1, 3, 4], device=dev())
        rest = moe.MoELayer(4, d, 64, 1, 1, dtype=dtype).layer_norm(x[keep], gamma, beta)
        assert torch.equal(y[keep], rest[0]) and torch.equal(rstd[keep], rest[2])


def test_layer_norm_unaligned_and_no_rows(moe):
    """Pointers off the 16-byte boundary take the one-element loads; T = 0 clears the sums."""
    T, d = 20, 512
    g = gen(8)
    for dtype in ("bf16", "f32"):
        dt = DT[dtype]
        store = [randn(g, T * d + 1).to(dt) for _ in range(3)]
        x, dy, dres = (s[1:].view(T, d) for s in store)
        pg, pb = randn(g, d + 1), randn(g, d + 1)
        check_norm(moe.MoELayer(T, d, 64, 1, 1, dtype=dtype), x, pg[1:], pb[1:], 1e-3, dy, dres)
    layer = moe.MoELayer(0, d, 64, 1, 1, dtype="f32")
    e, v = torch.empty(0, d, device=dev()), torch.empty(0, device=dev())
    dx, dg, db = layer.layer_norm_backward(e, e, pg[:d], v, v)
    assert dx.shape == (0, d) and (dg == 0).all() and (db == 0).all()


def test_layer_norm_gradient_against_differences(moe):
    """sum(dx v) and the parameter gradients against central differences of sum(y w), formed in 64
    bits from fp32 outputs: y's error is below 2^-20 for these values (|xh| < 5), so the difference
    is good to 2 T d 2^-20 max|w| / (2 h) in the worst case; its third-order term is below h^2
    times the sum of |terms|."""
    T, d = 4, 96
    g = gen(6)
    x, gamma, beta = randn(g, T, d), 1 + 0.1 * randn(g, d), randn(g, d)
    w = randn(g, T, d)
    layer = moe.MoELayer(T, d, 64, 1, 1, dtype="f32")
    y, mean, rstd = layer.layer_norm(x, gamma, beta)
    dx, dg, db = layer.layer_norm_backward(w, x, gamma, mean, rstd)
    h = 2.0 ** -4

    def value(x_, g_, b_):
        return (layer.layer_norm(x_, g_, b_)[0].double() * w.double()).sum()

    noise = (w.double().abs().sum() * 2.0 ** -20 / h).item()
    for at, grad in ((0, dx), (1, dg), (2, db)):
        v = torch.sign(grad)
        up, dn = [x, gamma, beta], [x, gamma, beta]
        up[at], dn[at] = up[at] + h * v, dn[at] - h * v
        diff = ((value(*up) - value(*dn)) / (2 * h)).item()
        want = (grad.double() * v).sum().item()
        third = 0.0 if at else 4 * h * h * w.double().abs().sum().item()
        assert abs(diff - want) <= noise + third
        assert want > 2 * noise


# ----------------------------------------------------------------------------------------------
# 4-bit weights
# ----------------------------------------------------------------------------------------------
def quantize_reference(W, group, zeros):
    """(nibbles - 8, scale, zero) as [E, N, K], [E, G, N]: the definition in float32 steps
    (7 and 15 through their float32 reciprocals)."""
    E, N, K = W.shape
    w = W.float()
    q, scale, zero = torch.empty_like(w), [], []
    for k0 in range(0, K, group):
        v = w[:, :, k0:k0 + group]
        if zeros:
            lo, hi = v.amin(2), v.amax(2)
            s = ((hi - lo) * torch.tensor(1.0 / 15.0, device=dev())).to(torch.bfloat16).float()
            z = (lo + 8.0 * s).to(torch.bfloat16).float()
        else:
            m = v.abs().amax(2)
            s = (m * torch.tensor(1.0 / 7.0, device=dev())).to(torch.bfloat16).float()
            z = torch.zeros_like(s)
        t = torch.round((v - z[..., None]) / s[..., None]).clamp(-8, 7)
        q[:, :, k0:k0 + group] = torch.where(s[..., None] > 0, t, torch.zeros_like(t))
        scale.append(s)
        zero.append(z)
    return q, torch.stack(scale, 1), torch.stack(zero, 1)


def unpack(words, K):
    """Nibbles - 8 [E, N, K] from the words, column by column as the header states the order."""
    k = torch.arange(K, device=words.device)
    word = (k // 128) * 16 + 4 * ((k % 32) // 8) + (k % 128) // 32
    i = k % 8
    return ((words.long()[:, :, word] >> (4 * (4 * (i % 2) + i // 2))) & 15) - 8


def values(w):
    """A W4Weights' values in 64 bits."""
    per = [torch.zeros(1)] * 2
    for n, t in enumerate((w.scale, w.zero)):
        if t is not None:
            per[n] = t.double().transpose(1, 2).repeat_interleave(w.group, 2)[:, :, :w.K]
    v = unpack(w.q, w.K).double() * per[0]
    return v if w.zero is None else v + per[1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("E,N,K,group", [(1, 1, 64, 32), (2, 3, 64, 128), (3, 32, 128, 64),
                                         (2, 64, 192, 128), (1, 100, 576, 32), (2, 96, 1472, 64),
                                         (5, 33, 1024, 128), (1, 640, 2048, 32)])
def test_quantize_and_back(moe, dtype, zeros, E, N, K, group):
    g = gen(E * 7 + N + K)
    W = randn(g, E, N, K) / 8 + (0.05 if zeros else 0.0)
    W[0, 0, :32] = 0.0                                    # a group of zeros (group 32), or its part
    W[0, N - 1] = 0.25                                    # a constant row
    W[-1, N // 2] *= 1e-30                                # tiny scales
    W[-1, N // 3] = torch.round(W[-1, N // 3] * 16) / 16   # many exact halves of a step
    W = W.to(DT[dtype]).contiguous()
    w = moe.quantize_w4(W, group, zeros=zeros)
    q, s, z = quantize_reference(W, group, zeros)
    assert torch.equal(w.scale.float(), s)
    if zeros:
        assert torch.equal(w.zero.float(), z)
    assert torch.equal(unpack(w.q, K).float(), q)
    # Words past K hold 8 in every nibble.
    C = -(-K // 128)
    assert torch.equal(unpack(w.q, C * 128)[:, :, K:], torch.zeros(E, N, C * 128 - K, device=dev(),
                                                                  dtype=torch.int64))
    back = moe.dequantize_w4(w)
    assert torch.equal(back, values(w).to(torch.float32).to(torch.bfloat16))


def test_quantize_leaves_what_is_behind(moe):
    """Nothing outside the outputs is written (guards around each)."""
    E, N, K, group = 2, 35, 192, 64
    g = gen(1)
    W = randn(g, E, N, K).to(torch.bfloat16)
    nq, ns = E * N * 32, E * 3 * N
    q = torch.full((nq + 64,), -7, dtype=torch.int32, device=dev())
    s = torch.full((ns + 64,), -7.0, dtype=torch.bfloat16, device=dev())
    z = s.clone()
    moe.moe_quantize_packed(W, E, N, K, group, q, s, z)
    for t in (q[nq:], s[ns:], z[ns:]):
        assert (t == -7).all()
    out = torch.full((E * N * K + 64,), -7.0, dtype=torch.bfloat16, device=dev())
    c = moe.W4(q.data_ptr(), s.data_ptr(), z.data_ptr(), group)
    moe.moe_dequantize_packed(c, E, N, K, out)
    assert (out[E * N * K:] == -7).all()


def test_offsets_past_32_bits(moe):
    """More than 2^31 elements: the last rows and experts come out like small tensors do."""
    g = gen(77)
    E, N, K = 9, 65536, 4096
    W = torch.zeros(E, N, K, dtype=torch.bfloat16, device=dev())
    last = (randn(g, 1, 64, K) / 64).to(torch.bfloat16)
    W[-1, -64:] = last[0]
    w, small = moe.quantize_w4(W, 128), moe.quantize_w4(last, 128)
    assert torch.equal(w.q[-1, -64:], small.q[0])
    assert torch.equal(w.scale[-1, :, -64:], small.scale[0])
    del W
    back = moe.dequantize_w4(w)
    assert torch.equal(back[-1, -64:], moe.dequantize_w4(small)[0])
    assert (back[0, :64] == 0).all()
    del back, w
    T, d = 270000, 8192
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=dev())
    x[-8:] = randn(g, 8, d).to(torch.bfloat16)
    ga, be = randn(g, d), randn(g, d)
    layer, few = moe.MoELayer(T, d, 64, 1, 1), moe.MoELayer(8, d, 64, 1, 1)
    y, mean, rstd = layer.layer_norm(x, ga, be)
    ys, ms, rs = few.layer_norm(x[-8:].contiguous(), ga, be)
    assert torch.equal(y[-8:], ys) and torch.equal(mean[-8:], ms) and torch.equal(rstd[-8:], rs)
    dx = layer.layer_norm_backward(y, x, ga, mean, rstd)[0]
    assert torch.equal(dx[-8:], few.layer_norm_backward(ys, x[-8:].contiguous(), ga, ms, rs)[0])


# ----------------------------------------------------------------------------------------------
# Expert FFN over 4-bit weights
# ----------------------------------------------------------------------------------------------
def make_experts(moe, g, E, F1, F, d, groups, zeros):
    def weights(n, k, group):
        W = (randn(g, E, n, k) / math.sqrt(k)).to(torch.bfloat16)
        return moe.quantize_w4(W, group, zeros=zeros)
    return weights(F1, d, groups[0]), weights(d, F, groups[1])


def ffn_reference(x, offsets, rowtok, W1, b1, W2, b2, gated, copy):
    """Y in 64 bits, and its bound.  Of h: the fp32 sums, at most K / 16 + 32 accumulations behind
    one another, each good to 2 U of the running magnitude (the tensor cores cut what they align),
    and for `copy` (weights first read back to bfloat16) half a bfloat16 step of every weight.  Of a:
    h's error (the slope of SiLU is below 1.1), SiLU's own (below 2^-20), and the rounding of a to
    bfloat16.  Of y the same with a in x's place, and its own rounding."""
    off = offsets.tolist()
    h2 = HALF[torch.bfloat16]
    d, F = W2.N, W2.K
    v1, v2 = values(W1), values(W2)
    Y = torch.zeros(off[-1], d, dtype=torch.float64, device=dev())
    tol = torch.zeros_like(Y)

    def product(a, ea, w, b):
        K = a.shape[1]
        y = a @ w.T + (0 if b is None else b.double())
        mag = a.abs() @ w.abs().T
        return y, ea @ w.abs().T + ((K / 16 + 32) * 2 * U + (h2 if copy else 0)) * mag + \
            2 * U * y.abs()

    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        xe = x[rowtok[lo:hi].long()].double()
        h, eh = product(xe, torch.zeros_like(xe), v1[e], None if b1 is None else b1[e])
        s = torch.nn.functional.silu(h[:, :F])
        es = 1.1 * eh[:, :F] + 2.0 ** -20 * s.abs()
        if gated:
            u, eu = h[:, F:], eh[:, F:]
            a, ea = s * u, es * (u.abs() + eu) + s.abs() * eu + 2 * U * (s * u).abs()
        else:
            a, ea = s, es
        ea = ea + h2 * (a.abs() + ea)
        y, ey = product(a, ea, v2[e], None if b2 is None else b2[e])
        Y[lo:hi], tol[lo:hi] = y, ey + h2 * (y.abs() + ey)
    return Y, tol


def routing(g, T, E, k, kind):
    """offsets, rowtok of a dropless routing: random, or all tokens on the first k experts."""
    if kind == "hot":
        ids = torch.arange(k, device=dev()).expand(T, k).reshape(-1)
    else:
        ids = torch.topk(randn(g, T, E), k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev())
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0).to(torch.int32)
    return offsets, (order // k).to(torch.int32)


FFN = [  # T, d, F, E, k, groups, zeros, gated, kind
    (1, 64, 64, 1, 1, (32, 32), False, False, "random"),
    (1, 256, 128, 64, 8, (128, 64), True, False, "random"),
    (3, 192, 128, 4, 2, (128, 32), False, True, "random"),
    (5, 320, 384, 6, 2, (64, 128), True, True, "random"),
    (17, 128, 192, 3, 1, (32, 128), True, False, "hot"),
    (33, 448, 64, 5, 2, (64, 32), False, False, "hot"),
    (64, 2048, 1024, 16, 4, (64, 64), False, False, "random"),
    (65, 1472, 128, 9, 3, (128, 128), True, False, "random"),
    (100, 1024, 512, 300, 2, (32, 64), False, False, "random"),
    (129, 512, 1408, 8, 3, (128, 32), True, True, "random"),
    (64, 256, 256, 1, 1, (64, 64), True, False, "hot"),
    (65, 256, 256, 1, 1, (64, 64), True, False, "hot"),      # above the rows the direct path takes
    (700, 512, 384, 6, 2, (32, 128), False, True, "random"),
    (1100, 320, 192, 4, 2, (64, 64), True, False, "hot"),
]


@pytest.mark.parametrize("T,d,F,E,k,groups,zeros,gated,kind", FFN)
def test_expert_ffn_w4(moe, T, d, F, E, k, groups, zeros, gated, kind):
    g = gen(T + d + F)
    F1 = 2 * F if gated else F
    W1, W2 = make_experts(moe, g, E, F1, F, d, groups, zeros)
    b1, b2 = 0.1 * randn(g, E, F1), 0.1 * randn(g, E, d)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets, rowtok = routing(g, T, E, k, kind)
    layer = moe.MoELayer(T, d, F, E, k, flags=moe.FLAG_GATED if gated else 0, w4=True)
    copy = T * k > 64 * E
    for bias in (True, False):
        bb = (b1, b2) if bias else (None, None)
        Y = layer.expert_ffn_w4(x, offsets, rowtok, W1, bb[0], W2, bb[1])
        ref, tol = ffn_reference(x, offsets, rowtok, W1, bb[0], W2, bb[1], gated, copy)
        assert_within(Y, ref, tol, "Y")
        assert status(moe, layer) == 0
        assert torch.equal(Y, layer.expert_ffn_w4(x, offsets, rowtok, W1, bb[0], W2, bb[1]))


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 24, 25, 31, 32, 33, 40, 64, 65])
def test_expert_ffn_w4_row_counts(moe, rows):
    """Every number of rows around the tile widths, beside empty experts and a full one."""
    T, d, F, E = 96, 256, 128, 5
    g = gen(rows)
    W1, W2 = make_experts(moe, g, E, F, F, d, (64, 32), False)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets = torch.tensor([0, 0, rows, rows, rows + 3, rows + 3], dtype=torch.int32, device=dev())
    rowtok = torch.zeros(T * 1, dtype=torch.int32, device=dev())
    rowtok[:rows + 3] = torch.randint(0, T, (rows + 3,), generator=g, device=dev()).to(torch.int32)
    layer = moe.MoELayer(T, d, F, E, 1, w4=True)
    Y = torch.full((T, d), 5.0, dtype=torch.bfloat16, device=dev())
    moe.moe_expert_ffn_packed(layer.p, x, offsets, rowtok, W1.c, None, W2.c, None, Y, layer.ws)
    ref, tol = ffn_reference(x, offsets, rowtok, W1, None, W2, None, False, False)
    assert_within(Y[:rows + 3], ref, tol, "Y")
    assert (Y[rows + 3:] == 5.0).all(), "rows behind the last one were written"


def test_expert_ffn_w4_bad_offsets_and_rows(moe):
    T, d, F, E, k = 32, 128, 64, 4, 2
    g = gen(11)
    W1, W2 = make_experts(moe, g, E, F, F, d, (32, 32), False)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets, rowtok = routing(g, T, E, k, "random")
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    for change in ((0, 1), (E, T * k + 1), (2, -5)):
        bad = offsets.clone()
        bad[change[0]] = change[1]
        Y = torch.full((T * k, d), 5.0, dtype=torch.bfloat16, device=dev())
        moe.moe_expert_ffn_packed(layer.p, x, bad, rowtok, W1.c, None, W2.c, None, Y, layer.ws)
        assert status(moe, layer) == moe.DEV_BAD_INDEX
        assert (Y == 5.0).all()
        moe.moe_reset_device_status(layer.ws)
    bad = rowtok.clone()
    bad[3], bad[20] = T, -1
    Y = layer.expert_ffn_w4(x, offsets, bad, W1, None, W2, None)
    assert status(moe, layer) == moe.DEV_BAD_INDEX
    xz = torch.cat([x, torch.zeros(1, d, dtype=x.dtype, device=dev())])
    bad[3] = bad[20] = T                              # the row of zeros
    ref, tol = ffn_reference(xz, offsets, bad, W1, None, W2, None, False, False)
    assert_within(Y, ref, tol, "rows with a bad index")


@pytest.mark.parametrize("T", [32, 300])                # read directly; read back first
def test_expert_ffn_w4_offsets_whose_difference_wraps(moe, T):
    """Offsets 2^31 apart and more are seen to decrease: nothing is read or written.  (After the
    check of the order, an expert of a wrapped row count has no rows.)"""
    d, F, E, k = 128, 64, 4, 2
    g = gen(12)
    W1, W2 = make_experts(moe, g, E, F, F, d, (32, 32), False)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets, rowtok = routing(g, T, E, k, "random")
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    for inner in ((2000000000, -2000000000, 5), (2 ** 31 - 1, -2 ** 31, 0)):
        bad = offsets.clone()
        bad[1:4] = torch.tensor(inner, dtype=torch.int32)
        Y = torch.full((T * k, d), 5.0, dtype=torch.bfloat16, device=dev())
        moe.moe_expert_ffn_packed(layer.p, x, bad, rowtok, W1.c, None, W2.c, None, Y, layer.ws)
        assert status(moe, layer) == moe.DEV_BAD_INDEX
        assert (Y == 5.0).all()
        moe.moe_reset_device_status(layer.ws)


def test_expert_ffn_w4_infinities_stay_in_their_rows(moe):
    T, d, F, E, k = 16, 256, 128, 2, 1
    g = gen(12)
    W1, W2 = make_experts(moe, g, E, F, F, d, (64, 64), True)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets, rowtok = routing(g, T, E, k, "random")
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    clean = layer.expert_ffn_w4(x, offsets, rowtok, W1, None, W2, None)
    x[5, 7] = INF
    x[6, 1] = math.nan
    Y = layer.expert_ffn_w4(x, offsets, rowtok, W1, None, W2, None)
    hit = (rowtok == 5) | (rowtok == 6)
    assert torch.equal(Y[~hit], clean[~hit])
    assert not torch.isfinite(Y[hit]).all(1).any()


# ----------------------------------------------------------------------------------------------
# The operators together
# ----------------------------------------------------------------------------------------------
def block_inputs(g, T, d, F, E, dtype="bf16"):
    dt = DT[dtype]
    return dict(x=randn(g, T, d).to(dt), Wr=0.1 * randn(g, d, E), br=0.1 * randn(g, E),
                gamma=1 + 0.1 * randn(g, d), beta=0.1 * randn(g, d),
                b1=0.1 * randn(g, E, F), b2=0.1 * randn(g, E, d))


def block_reference(x, y, rt, ffn, W2N):
    """out in 64 bits under the block's own routing, from its normed rows y; ffn gives (Y, bound)
    of rows y sorted by (expert, token)."""
    T, k = rt["ids_out"].shape
    E = rt["counts_out"].numel() // 2
    keep = rt["drop_out"].reshape(-1) == 0
    pair = torch.nonzero(keep)[:, 0]
    ids = rt["ids_out"].reshape(-1).long()[pair]
    order = pair[torch.sort(ids, stable=True).indices]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev())
    offsets[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0).to(torch.int32)
    Y, tol = ffn(y, offsets, (order // k).to(torch.int32))
    w = rt["w_out"].reshape(-1).double()[order][:, None]
    out, bound = x.double(), torch.zeros(T, W2N, dtype=torch.float64, device=dev())
    out = out.index_add(0, order // k, w * Y)
    bound = bound.index_add(0, order // k, w * (tol + 8 * U * Y.abs()))
    h2 = HALF[x.dtype]
    return out, bound + h2 * (out.abs() + bound) + 4 * U * x.double().abs()


@pytest.mark.parametrize("T,E,k,C", [(1, 8, 2, INF), (64, 16, 4, INF), (200, 8, 2, 1.0),
                                     (1500, 8, 2, 1.25)])
def test_block_with_norm_and_w4(moe, T, E, k, C):
    """Norm, router, dispatch, 4-bit experts and combine in one call, under decoding and prefill
    sizes, with capacity drops."""
    d, F = 256, 192
    g = gen(T)
    i = block_inputs(g, T, d, F, E)
    W1, W2 = make_experts(moe, g, E, F, F, d, (64, 32), True)
    layer = moe.MoELayer(T, d, F, E, k, C, w4=True)
    out, rt = layer.forward_block(i["x"], i["Wr"], i["br"], W1, i["b1"], W2, i["b2"],
                                  norm=(i["gamma"], i["beta"], 1e-5))
    assert status(moe, layer) == 0
    y, mean, rstd = layer.layer_norm(i["x"], i["gamma"], i["beta"], 1e-5)
    for key, t in (("y", y), ("mean", mean), ("rstd", rstd)):
        assert torch.equal(rt[key], t)
    logits = layer.router_logits(y, i["Wr"], i["br"])
    assert torch.equal(rt["logits_out"], logits)
    r = layer.route(logits)
    for key in ("ids", "w", "slot", "drop", "counts"):
        assert torch.equal(rt[key + "_out"], r[key]), key
    copy = layer.max_rows > 64 * E
    ref, tol = block_reference(
        i["x"], y, rt, lambda rows, off, tok: ffn_reference(rows, off, tok, W1, i["b1"], W2,
                                                            i["b2"], False, copy), d)
    assert_within(out, ref, tol, "out")
    # The stages one by one give the same bits.
    offs, rowtok, _ = layer.dispatch(r["ids"], r["slot"])
    Y = layer.expert_ffn_w4(y, offs, rowtok, W1, i["b1"], W2, i["b2"])
    assert torch.equal(out, layer.combine(i["x"], Y, r["w"], r["ids"], r["slot"], offs))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_without_extras_is_the_forward(moe, dtype):
    T, d, F, E, k = 130, 128, 64, 4, 2
    g = gen(21)
    i = block_inputs(g, T, d, F, E, dtype)
    W1 = (randn(g, E, F, d) / 12).to(DT[dtype])
    W2 = (randn(g, E, d, F) / 8).to(DT[dtype])
    layer = moe.MoELayer(T, d, F, E, k, 1.0, dtype)
    args = (i["x"], i["Wr"], i["br"], W1, i["b1"], W2, i["b2"])
    assert torch.equal(layer.forward_block(*args)[0], layer.forward(*args))
    out, rt = layer.forward_block(*args, norm=(i["gamma"], i["beta"], 1e-6))
    r = layer.route(rt["logits_out"])
    offs, rowtok, _ = layer.dispatch(r["ids"], r["slot"])
    Y = layer.expert_ffn(rt["y"], offs, rowtok, W1, i["b1"], W2, i["b2"])
    assert torch.equal(out, layer.combine(i["x"], Y, r["w"], r["ids"], r["slot"], offs))


def test_router_training_step(moe):
    """Norm, logits, losses; their gradient back through the logits' product and the norm, against
    64-bit autograd of the whole chain.  The middle product runs in 64 bits here, so the bounds of
    the two kernels are what is left: dlogits' relative 1e-5 of its row terms (see above), carried
    through linear maps, and the norm's outputs (relative 2^-20)."""
    T, d, E, k = 600, 192, 24, 3
    g = gen(31)
    i = block_inputs(g, T, d, 64, E, "f32")
    layer = moe.MoELayer(T, d, 64, E, k, dtype="f32")
    y, mean, rstd = layer.layer_norm(i["x"], i["gamma"], i["beta"])
    logits = layer.router_logits(y, i["Wr"], i["br"])
    ids = layer.route(logits)["ids"]
    gl = torch.tensor([1.0, 0.1], device=dev())
    losses, counts, _ = layer.balance_loss(logits, ids)
    dl = layer.route_backward(logits, ids, counts, gl)
    dy = (dl.double() @ i["Wr"].double().T).float()
    dx, dg, db = layer.layer_norm_backward(dy, i["x"], i["gamma"], mean, rstd)

    p = [t.double().requires_grad_(True) for t in (i["x"], i["gamma"], i["beta"])]
    mu = p[0].mean(1, keepdim=True)
    xh = (p[0] - mu) / torch.sqrt(((p[0] - mu) ** 2).mean(1, keepdim=True) + 1e-5)
    L = (xh * p[1] + p[2]) @ i["Wr"].double() + i["br"].double()
    pr = torch.softmax(L, 1)
    f = torch.bincount(ids.long().reshape(-1), minlength=E).double() / (T * k)
    loss = E * (f * pr.mean(0)).sum() + 0.1 * (torch.logsumexp(L, 1) ** 2).mean()
    want = torch.autograd.grad(loss, p)
    assert abs(losses[0] + 0.1 * losses[1] - loss) < 1e-5 * loss
    for got, ref in zip((dx, dg, db), want):
        assert (got.double() - ref).norm() <= 1e-4 * ref.norm()


# ----------------------------------------------------------------------------------------------
# Streams, graphs, refusals
# ----------------------------------------------------------------------------------------------
def all_operators(moe, layer, i, W1, W2, offsets, rowtok, logits, ids, dy, W, stream=None):
    gl = i["gl"]
    losses, counts, probs = layer.balance_loss(logits, ids, stream=stream)
    dl = layer.route_backward(logits, ids, counts, gl, stream=stream)
    y, mean, rstd = layer.layer_norm(i["x"], i["gamma"], i["beta"], stream=stream)
    back = layer.layer_norm_backward(dy, i["x"], i["gamma"], mean, rstd, stream=stream)
    Y = layer.expert_ffn_w4(y, offsets, rowtok, W1, i["b1"], W2, i["b2"], stream=stream)
    q = moe.quantize_w4(W, 64, zeros=True, stream=stream)
    return (losses, counts, probs, dl, y, mean, rstd, *back, Y, q.q, q.scale, q.zero,
            moe.dequantize_w4(q, stream=stream))


@pytest.mark.parametrize("T", [48, 2000])
def test_streams_and_graphs(moe, T):
    """The operators on a stream of their own, and captured into a graph that is replayed on new
    inputs, give the bits of the plain calls."""
    d, F, E, k = 256, 128, 8, 2
    g = gen(41)
    i = block_inputs(g, T, d, F, E)
    i["gl"] = torch.tensor([0.5, 0.25], device=dev())
    W1, W2 = make_experts(moe, g, E, F, F, d, (64, 32), False)
    logits = randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    offsets, rowtok = routing(g, T, E, k, "random")
    dy, W = randn(g, T, d).to(torch.bfloat16), randn(g, 2, 96, 192)
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    args = (moe, layer, i, W1, W2, offsets, rowtok, logits, ids, dy, W)
    want = all_operators(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = all_operators(*args, stream=side)
    raw = all_operators(*args, stream=side.cuda_stream)
    side.synchronize()
    for a, b, c in zip(want, got, raw):
        assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = all_operators(*args)
    for seed in (1, 2):
        g2 = gen(seed)
        logits.copy_(randn(g2, T, E))
        i["x"].copy_(randn(g2, T, d))
        dy.copy_(randn(g2, T, d))
        W.copy_(randn(g2, 2, 96, 192))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(all_operators(*args), kept):
            assert torch.equal(a, b)


def test_two_graphs_share_a_workspace(moe):
    """Graphs captured over one workspace and replayed in turn, with plain calls between them, do not
    disturb each other."""
    T, d, F, E, k = 3000, 128, 128, 16, 2
    g = gen(43)
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    W1, W2 = make_experts(moe, g, E, F, F, d, (64, 64), False)
    logits = [randn(g, T, E) for _ in range(2)]
    ids = [torch.topk(x, k, dim=1).indices.to(torch.int32) for x in logits]
    x = [randn(g, T, d).to(torch.bfloat16) for _ in range(2)]
    ga = 1 + 0.1 * randn(g, d)
    route = [routing(g, T, E, k, "random") for _ in range(2)]

    def work(i):
        y, mean, rstd = layer.layer_norm(x[i], ga, ga)
        return (*layer.balance_loss(logits[i], ids[i]),
                *layer.layer_norm_backward(y, x[i], ga, mean, rstd),
                layer.expert_ffn_w4(y, *route[i], W1, None, W2, None))

    want = [work(0), work(1)]
    graphs, kept = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            kept.append(work(i))
    for i in (0, 1, 1, 0):
        for t in kept[i]:
            t.zero_()
        graphs[i].replay()
        for a, b in zip(work(1 - i), want[1 - i]):
            assert torch.equal(a, b)
        for a, b in zip(kept[i], want[i]):
            assert torch.equal(a, b)


def test_wrong_tensors_are_refused(moe):
    """Types, shapes, devices and layouts that a call does not take raise before anything runs."""
    T, d, F, E, k = 16, 128, 64, 4, 2
    g = gen(51)
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    x = randn(g, T, d).to(torch.bfloat16)
    ga = randn(g, d)
    logits = randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    W1, W2 = make_experts(moe, g, E, F, F, d, (32, 32), False)
    offsets, rowtok = routing(g, T, E, k, "random")
    y, mean, rstd = layer.layer_norm(x, ga, ga)
    gl = torch.ones(2, device=dev())
    _, counts, _ = layer.balance_loss(logits, ids)
    wide = randn(g, T, 2 * d).to(torch.bfloat16)
    calls = [
        lambda: layer.layer_norm(x.float(), ga, ga),
        lambda: layer.layer_norm(x[:8], ga, ga),
        lambda: layer.layer_norm(wide[:, :d], ga, ga),
        lambda: layer.layer_norm(x.cpu(), ga, ga),
        lambda: layer.layer_norm(x, ga.double(), ga),
        lambda: layer.layer_norm(x, ga, ga, eps=-1.0),
        lambda: layer.layer_norm(x, ga, ga, eps=math.nan),
        lambda: layer.layer_norm_backward(y, x, ga, mean[:3], rstd),
        lambda: layer.layer_norm_backward(y, x, ga, mean, rstd, dres=y.float()),
        lambda: moe.moe_layer_norm(layer.p, x, ga, ga, 1e-5, x, mean, rstd),
        lambda: layer.balance_loss(logits.half(), ids),
        lambda: layer.balance_loss(logits, ids.long()),
        lambda: layer.balance_loss(logits.t().contiguous().t(), ids),
        lambda: layer.balance_loss(logits, ids, mask=torch.ones(T, device=dev())),
        lambda: layer.route_backward(logits, ids),
        lambda: layer.route_backward(logits, ids, None, gl),
        lambda: layer.route_backward(logits, ids, counts[:E], gl),
        lambda: moe.moe_route_backward(layer.p, logits, ids, counts, logits, layer.ws, gl),
        lambda: layer.expert_ffn_w4(x, offsets, rowtok, W2, None, W1, None),
        lambda: layer.expert_ffn_w4(x, offsets, rowtok, x, None, W2, None),
        lambda: layer.expert_ffn_w4(x, offsets, rowtok[:5], W1, None, W2, None),
        lambda: layer.expert_ffn_w4(x.float(), offsets, rowtok, W1, None, W2, None),
        lambda: moe.MoELayer(T, d, F, E, k, dtype="f32", w4=True),
        lambda: moe.W4Weights(W1.q, W1.scale, K=d, group=48),
        lambda: moe.W4Weights(W1.q, W1.scale, K=d, group=64),
        lambda: moe.quantize_w4(x, 32),
        lambda: moe.quantize_w4(randn(g, 1, 4, 64), 48),
        lambda: moe.quantize_w4(randn(g, 1, 4, 65), 32),
        lambda: moe.quantize_w4(randn(g, 1, 64, 64).transpose(1, 2), 32),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(moe.MoeError):
            call()
            pytest.fail("call %d was not refused" % n)
    small = torch.zeros(8, dtype=torch.int64, device=dev())
    with pytest.raises(moe.MoeError):
        moe.moe_layer_norm_backward(layer.p, y, x, ga, mean, rstd, torch.empty_like(x), ga, ga, small)
    big = moe.MoELayer(2000, d, F, E, k)                  # its workspace has no room for the copy
    with pytest.raises(moe.MoeError):
        big.expert_ffn_w4(randn(g, 2000, d).to(torch.bfloat16), offsets,
                          torch.zeros(4000, dtype=torch.int32, device=dev()), W1, None, W2, None)
