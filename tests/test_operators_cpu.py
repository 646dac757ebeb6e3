"""Host-side checks of the router-loss, layer-norm and 4-bit calls: argument errors return before
anything is launched (no GPU needed), and workspace sizes."""
import ctypes
import math

import pytest

from expert_ffn_layer_router_b200 import build as lib_build


@pytest.fixture(scope="module")
def moe():
    lib_build.build()
    from expert_ffn_layer_router_b200 import moe as m
    return m


FAKE = ctypes.c_void_p(1 << 20)                     # never dereferenced: every call is refused
FAKE2 = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40


def prob(moe, **kw):
    a = dict(T=16, d=64, F=64, E=4, k=2, C=math.inf, dtype=1, flags=0)
    a.update(kw)
    return ctypes.byref(moe.Problem(*a.values()))


BAD = [dict(k=5), dict(E=0), dict(T=-1), dict(d=0), dict(dtype=5), dict(flags=16), dict(C=-1.0)]


@pytest.mark.parametrize("bad", BAD)
def test_malformed_problems(moe, bad):
    L, p, w = moe.lib(), prob(moe, **bad), ctypes.byref(moe.W4(1 << 20, 1 << 20, None, 32))
    n = ctypes.c_size_t()
    assert L.moe_workspace_size_packed(p, ctypes.byref(n)) == 1
    assert L.moe_layer_norm(p, FAKE, FAKE, FAKE, 1e-5, FAKE2, FAKE, FAKE, None) == 1
    assert L.moe_layer_norm_backward(p, *[FAKE] * 6, FAKE2, FAKE, FAKE, FAKE, BIG, None) == 1
    assert L.moe_balance_loss(p, *[FAKE] * 7, BIG, None) == 1
    assert L.moe_route_backward(p, *[FAKE] * 6, FAKE2, FAKE, BIG, None) == 1
    assert L.moe_expert_ffn_packed(p, FAKE, FAKE, FAKE, w, None, w, None, FAKE, FAKE, BIG, None) == 1
    assert L.moe_forward_block(p, FAKE, None, FAKE, None, FAKE, FAKE, None, None, None, None,
                               FAKE2, *[None] * 6, FAKE, BIG, None) == 1


def test_layer_norm_refusals(moe):
    L, p = moe.lib(), prob(moe)
    good = [FAKE, FAKE, FAKE, 1e-5, FAKE2, FAKE, FAKE]
    for i in (0, 1, 2, 4, 5, 6):
        a = list(good)
        a[i] = None
        assert L.moe_layer_norm(p, *a, None) == 1
    for eps in (-1e-9, math.nan, math.inf):
        assert L.moe_layer_norm(p, FAKE, FAKE, FAKE, eps, FAKE2, FAKE, FAKE, None) == 1
    assert L.moe_layer_norm(p, FAKE, FAKE, FAKE, 1e-5, FAKE, FAKE, FAKE, None) == 1     # y = x
    wide = prob(moe, d=(1 << 30) + 1)
    assert L.moe_layer_norm(wide, FAKE, FAKE, FAKE, 1e-5, FAKE2, FAKE, FAKE, None) == 2
    assert L.moe_layer_norm_backward(wide, *[FAKE] * 5, None, FAKE2, FAKE, FAKE, FAKE, BIG,
                                     None) == 2
    good = [FAKE] * 5 + [None, FAKE2, FAKE, FAKE]
    for i in (0, 1, 2, 3, 4, 6, 7, 8):
        a = list(good)
        a[i] = None
        assert L.moe_layer_norm_backward(p, *a, FAKE, BIG, None) == 1
    for i in (0, 1, 5):                                                              # dx aliases
        a = list(good)
        a[i] = FAKE2
        assert L.moe_layer_norm_backward(p, *a, FAKE, BIG, None) == 1
    assert L.moe_layer_norm_backward(p, *good, None, 0, None) == 3
    assert L.moe_layer_norm_backward(p, *good, FAKE, 512, None) == 3
    assert L.moe_layer_norm_backward(p, *good, ODD, BIG, None) == 3


def test_router_loss_refusals(moe):
    L, p = moe.lib(), prob(moe)
    good = [FAKE, FAKE, None, FAKE, FAKE, FAKE]
    for i in (0, 1, 3, 4, 5):
        a = list(good)
        a[i] = None
        assert L.moe_balance_loss(p, *a, FAKE, BIG, None) == 1
    assert L.moe_balance_loss(p, *good, None, 0, None) == 3
    rb = L.moe_route_backward
    #            logits ids mask counts grad_losses grad_w dlogits
    assert rb(p, FAKE, FAKE, None, FAKE, None, None, FAKE2, FAKE, BIG, None) == 1  # no gradient
    assert rb(p, FAKE, FAKE, None, None, FAKE, None, FAKE2, FAKE, BIG, None) == 1  # no counts
    assert rb(p, FAKE, None, None, FAKE, None, FAKE, FAKE2, FAKE, BIG, None) == 1  # no ids
    assert rb(p, None, FAKE, None, FAKE, FAKE, None, FAKE2, FAKE, BIG, None) == 1
    assert rb(p, FAKE, FAKE, None, FAKE, FAKE, None, None, FAKE, BIG, None) == 1
    assert rb(p, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, BIG, None) == 1   # aliases
    assert rb(p, FAKE, FAKE, None, FAKE, FAKE, None, FAKE2, None, 0, None) == 3


def test_packed_weight_refusals(moe):
    L = moe.lib()
    quant = L.moe_quantize_packed
    for bad in (dict(dtype=2), dict(E=0), dict(N=0), dict(K=0), dict(group=16), dict(group=0),
                dict(W=None), dict(q=None), dict(scale=None), dict(W=ODD), dict(q=ODD),
                dict(scale=ODD), dict(zero=ODD)):
        a = dict(W=FAKE, dtype=1, E=2, N=32, K=64, group=32, q=FAKE, scale=FAKE, zero=None)
        a.update(bad)
        assert quant(*a.values(), None) == 1, bad
    assert quant(FAKE, 1, 2, 32, 65, 32, FAKE, FAKE, None, None) == 2
    assert quant(FAKE, 1, 2, 32 * 65535 + 1, 64, 32, FAKE, FAKE, None, None) == 2
    W = lambda *a: ctypes.byref(moe.W4(*a))                                    # noqa: E731
    ok = W(1 << 20, 1 << 20, None, 64)
    for bad in (W(None, 1 << 20, None, 64), W(1 << 20, None, None, 64), W(1 << 20, 1 << 20, None, 63),
                W((1 << 20) + 4, 1 << 20, None, 64), W(1 << 20, 1 << 20, (1 << 20) + 2, 64)):
        assert L.moe_dequantize_packed(bad, 1, 32, 64, FAKE, None) == 1
        for pair in ((bad, ok), (ok, bad)):
            assert L.moe_expert_ffn_packed(prob(moe), FAKE, FAKE, FAKE, pair[0], None, pair[1], None,
                                           FAKE, FAKE, BIG, None) == 1
    assert L.moe_dequantize_packed(ok, 1, 32, 96, FAKE, None) == 2
    ffn = L.moe_expert_ffn_packed
    assert ffn(prob(moe, dtype=0), FAKE, FAKE, FAKE, ok, None, ok, None, FAKE, FAKE, BIG, None) == 2
    assert ffn(prob(moe, d=96), FAKE, FAKE, FAKE, ok, None, ok, None, FAKE, FAKE, BIG, None) == 2
    assert ffn(prob(moe, E=1024, F=1 << 21), FAKE, FAKE, FAKE, ok, None, ok, None, FAKE, FAKE, BIG,
               None) == 2
    assert ffn(prob(moe, flags=4), FAKE, FAKE, FAKE, ok, None, ok, None, FAKE, FAKE, BIG, None) == 2
    for i in (0, 1, 2, 7):
        a = [FAKE, FAKE, FAKE, ok, None, ok, None, FAKE]
        a[i if i < 3 else 7] = None
        assert ffn(prob(moe), *a, FAKE, BIG, None) == 1
    assert ffn(prob(moe), ODD, FAKE, FAKE, ok, None, ok, None, FAKE, FAKE, BIG, None) == 1
    assert ffn(prob(moe), FAKE, FAKE, FAKE, ok, ODD, ok, None, FAKE, FAKE, BIG, None) == 1
    assert ffn(prob(moe), FAKE, FAKE, FAKE, ok, None, ok, None, FAKE, FAKE, 1024, None) == 3


def test_block_refusals(moe):
    L, p = moe.lib(), prob(moe)
    q = ctypes.byref(moe.W4(1 << 20, 1 << 20, None, 64))

    def call(W1=None, W2=None, Q1=None, Q2=None, x=FAKE, out=FAKE2, norm=None, p=p, ws=FAKE,
             n=BIG):
        return L.moe_forward_block(p, x, norm, FAKE, None, W1, W2, Q1, Q2, None, None, out,
                                   *[None] * 6, ws, n, None)

    assert call() == 1                                       # no weights
    assert call(W1=FAKE) == 1
    assert call(W1=FAKE, W2=FAKE, Q1=q, Q2=q) == 1           # both kinds
    assert call(Q1=q) == 1 and call(Q2=q) == 1               # half of a pair
    assert call(W1=FAKE, Q2=q) == 1
    assert call(W1=FAKE, W2=FAKE, x=None) == 1
    assert call(W1=FAKE, W2=FAKE, out=FAKE) == 1             # out = x
    assert call(W1=FAKE, W2=FAKE, ws=None, n=0) == 3
    assert call(Q1=q, Q2=q, p=prob(moe, dtype=0)) == 2
    for bad in (dict(gamma=None), dict(beta=None), dict(eps=-1.0), dict(y=None), dict(mean=None),
                dict(rstd=None), dict(y=1 << 20), dict(y=1 << 21), dict(y=(1 << 22) + 2)):
        a = dict(gamma=1 << 20, beta=1 << 20, eps=1e-5, y=1 << 22, mean=1 << 20, rstd=1 << 20)
        a.update(bad)
        assert call(W1=FAKE, W2=FAKE, norm=ctypes.byref(moe.Norm(*a.values()))) == 1, bad


def test_workspace_sizes(moe):
    """The 4-bit workspace holds one bfloat16 copy of the larger weight exactly when an expert's
    average share passes 64 rows."""
    for T, d, F, E, k, flags in ((64, 2048, 1024, 64, 8, 0), (64, 64, 64, 2, 2, 0),
                                 (65, 64, 64, 2, 2, 0), (4096, 2048, 1408, 64, 6, 0),
                                 (500, 256, 128, 4, 2, 4)):
        p = moe.problem(T, d, F, E, k, math.inf, "bf16", flags)
        plain, packed = moe.moe_workspace_size(p), moe.moe_workspace_size_packed(p)
        copy = E * d * max(F * (2 if flags else 1), F) * 2
        assert packed - plain == (0 if T * k <= 64 * E else -(-copy // 256) * 256)
    n = ctypes.c_size_t()
    L = moe.lib()
    assert L.moe_workspace_size_packed(prob(moe, dtype=0), ctypes.byref(n)) == 2
    assert L.moe_workspace_size_packed(prob(moe, d=96), ctypes.byref(n)) == 2
    assert L.moe_workspace_size_packed(prob(moe), None) == 1


def test_packed_weight_size_limits(moe):
    """Sizes past what the tiles of a weight are counted in are refused, in every call that would
    walk them."""
    L, n = moe.lib(), ctypes.c_size_t()
    w = ctypes.byref(moe.W4(1 << 20, 1 << 20, None, 64))
    rows, cols = 32 * 65535, 1 << 30
    assert L.moe_quantize_packed(FAKE, 1, 1, 32, cols + 64, 64, FAKE, FAKE, None, None) == 2
    assert L.moe_quantize_packed(FAKE, 1, 65536, 32, 64, 64, FAKE, FAKE, None, None) == 2
    assert L.moe_dequantize_packed(w, 1, 32, cols + 64, FAKE, None) == 2
    assert L.moe_dequantize_packed(w, 1, rows + 1, 64, FAKE, None) == 2
    for size in (dict(F=rows + 32), dict(d=rows + 32), dict(F=(rows + 64) // 2, flags=4)):
        for T in (16, 4096):                         # (directly; after reading back)
            a = dict(T=T, E=1, k=1)
            a.update(size)
            a = {key: -(-v // 128) * 128 if key in "dF" else v for key, v in a.items()}
            p = prob(moe, **a)
            assert L.moe_workspace_size_packed(p, ctypes.byref(n)) == 2
            assert L.moe_expert_ffn_packed(p, FAKE, FAKE, FAKE, w, None, w, None, FAKE, FAKE, BIG,
                                           None) == 2
            assert L.moe_forward_block(p, FAKE, None, FAKE, None, None, None, w, w, None, None,
                                       FAKE2, *[None] * 6, FAKE, BIG, None) == 2


def test_cpu_tensors_are_refused(moe):
    """Tensors in host memory never reach a kernel."""
    import torch
    w = moe.W4Weights(torch.zeros(4, 64, 16, dtype=torch.int32),
                      torch.zeros(4, 1, 64, dtype=torch.bfloat16), K=64, group=64)
    x, f = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(64)
    ids, logits = torch.zeros(16, 2, dtype=torch.int32), torch.zeros(16, 4)
    rows, counts = torch.zeros(32, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    layer = moe.MoELayer(16, 64, 64, 4, 2, device="cpu", w4=True)
    m = torch.zeros(16)
    for call in (lambda: moe.quantize_w4(torch.zeros(1, 32, 64), 32), lambda: moe.dequantize_w4(w),
                 lambda: layer.balance_loss(logits, ids),
                 lambda: layer.route_backward(logits, ids, grad_w=torch.zeros(16, 2)),
                 lambda: layer.layer_norm(x, f, f),
                 lambda: layer.layer_norm_backward(x, x, f, m, m),
                 lambda: layer.expert_ffn_w4(x, counts, rows, w, None, w, None),
                 lambda: layer.forward_block(x, torch.zeros(64, 4), None, w, None, w, None)):
        with pytest.raises(moe.MoeError, match="CUDA device"):
            call()
