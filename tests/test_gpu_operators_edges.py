"""The operators around the layer at their edges: after errors of the data, at extreme values, over
every split of the 4-bit products, beside each other on threads.  (Helpers and bounds are those of the
operators' main tests.)"""
import math

import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_operators import (U, assert_within, ffn_reference, gen,  # noqa: F401
                                      make_experts, moe, randn, routing, status, unpack)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------------------------
# What an error of the data leaves alone
# ----------------------------------------------------------------------------------------------
def test_waits_go_on_after_a_bad_index(moe):
    """A recorded bad index ends no wait: one that nothing arrives on still runs for its limit, and
    its timeout replaces the index error; a later index error does not replace the timeout."""
    layer = moe.MoELayer(40, 64, 64, 4, 2)
    logits, ids = randn(gen(1), 40, 4), torch.zeros(40, 2, dtype=torch.int32, device=dev())
    ids[3, 1] = 4
    layer.balance_loss(logits, ids)
    assert status(moe, layer) == moe.DEV_BAD_INDEX
    moe.moe_selftest_wait_timeout(layer.ws, 20000)
    assert status(moe, layer) == moe.DEV_TIMEOUT
    layer.balance_loss(logits, ids)
    assert status(moe, layer) == moe.DEV_TIMEOUT


@pytest.mark.parametrize("T", [64, 1024])                # read directly; read back first
def test_expert_ffn_w4_after_a_bad_index(moe, T):
    """A status word that already holds a bad index (here the router losses') and one bad row do not
    cost any other row."""
    d, F, E, k = 2048, 1024, 64, 8
    g = gen(61)
    W1, W2 = make_experts(moe, g, E, F, F, d, (64, 64), False)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets, rowtok = routing(g, T, E, k, "random")
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    clean = layer.expert_ffn_w4(x, offsets, rowtok, W1, None, W2, None)
    logits = randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    ids[3, 1] = E
    layer.balance_loss(logits, ids)
    assert status(moe, layer) == moe.DEV_BAD_INDEX
    bad = rowtok.clone()
    bad[77] = T
    rest = torch.arange(T * k, device=dev()) != 77
    for _ in range(20):
        Y = torch.full_like(clean, 7.0)
        moe.moe_expert_ffn_packed(layer.p, x, offsets, bad, W1.c, None, W2.c, None, Y, layer.ws)
        assert torch.equal(Y[rest], clean[rest])


@pytest.mark.parametrize("T", [64, 1024])
def test_expert_ffn_w4_under_a_timeout_and_after(moe, T):
    """With a timeout in the status word a call ends (its waits may give up, its output is not used);
    once the word is cleared, the next one gives the bits of the first."""
    d, F, E, k = 2048, 1024, 64, 8
    g = gen(62)
    W1, W2 = make_experts(moe, g, E, F, F, d, (32, 128), True)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets, rowtok = routing(g, T, E, k, "random")
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    clean = layer.expert_ffn_w4(x, offsets, rowtok, W1, None, W2, None)
    moe.moe_selftest_wait_timeout(layer.ws, 1000)
    for _ in range(3):
        layer.expert_ffn_w4(x, offsets, rowtok, W1, None, W2, None)
    assert status(moe, layer) == moe.DEV_TIMEOUT
    moe.moe_reset_device_status(layer.ws)
    assert torch.equal(layer.expert_ffn_w4(x, offsets, rowtok, W1, None, W2, None), clean)
    assert status(moe, layer) == 0


@pytest.mark.parametrize("kind", ["w4", "bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [30, 700])
def test_rows_of_a_bad_token_index_are_those_of_zeros(moe, kind, gated, T):
    """A rowtok entry outside [0, T) gives the row that a token of zeros gives, bit for bit, whatever
    the tiles held before; the other rows do not see it."""
    d, F, E, k = 256, 128, 3, 2
    g = gen(63)
    layer = moe.MoELayer(T, d, F, E, k, dtype="f32" if kind == "f32" else "bf16",
                         flags=moe.FLAG_GATED if gated else 0, w4=kind == "w4")
    dt, F1 = layer.torch_dtype, 2 * F if gated else F
    b1, b2 = randn(g, E, F1), randn(g, E, d)
    if kind == "w4":
        W1, W2 = make_experts(moe, g, E, F1, F, d, (64, 32), False)
        ffn = layer.expert_ffn_w4
    else:
        W1, W2 = (randn(g, E, F1, d) / 16).to(dt), (randn(g, E, d, F) / 11).to(dt)
        ffn = layer.expert_ffn
    x = randn(g, T, d).to(dt)
    x[T - 1] = 0
    offsets, rowtok = routing(g, T, E, k, "random")
    hit = torch.rand(T * k, generator=g, device=dev()) < 0.05
    hit[[0, T, T * k - 1]] = True
    zero = torch.where(hit, T - 1, rowtok)
    want = ffn(x, offsets, zero, W1, b1, W2, b2)
    ffn(torch.full_like(x, 3.0), offsets, rowtok, W1, b1, W2, b2)
    assert status(moe, layer) == 0
    for index in (T, -1, 2 ** 31 - 1, -2 ** 31):
        got = ffn(x, offsets, torch.where(hit, index, rowtok), W1, b1, W2, b2)
        assert torch.equal(got, want)
        assert status(moe, layer) == moe.DEV_BAD_INDEX


def renormalised_reference(logits, ids, grad_w):
    """The renormalised weights' part of dlogits in 64 bits, from w = softmax over the named logits,
    and the magnitude of its terms.  Ids outside [0, E) are left out."""
    T, E = logits.shape
    I = ids.long()
    ok = (I >= 0) & (I < E)
    L = torch.gather(logits.double(), 1, I.clamp(0, E - 1)).masked_fill(~ok, -math.inf)
    top = L.amax(1, keepdim=True)
    u = torch.where(L > -math.inf, torch.exp(L - torch.where(top > -math.inf, top, 0.0)), 0.0)
    w = u / u.sum(1, keepdim=True).clamp(min=1e-300)
    dw = grad_w.double() * ok
    term = w * (dw - (w * dw).sum(1, keepdim=True))
    mag = w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
    out, terms = (torch.zeros(T, E, dtype=torch.float64, device=dev()) for _ in range(2))
    out.scatter_add_(1, I.clamp(0, E - 1), term * ok)
    terms.scatter_add_(1, I.clamp(0, E - 1), mag * ok)
    return out, terms


@pytest.mark.parametrize("gap", [0, 60, 85, 95, 100, 120, 1000, 1e30])
@pytest.mark.parametrize("E,k", [(8, 2), (30, 5), (64, 6), (128, 8), (400, 32)])
def test_renormalised_gradient_far_below_the_maximum(moe, gap, E, k):
    """Named experts `gap` below the row's maximum: their weights are a softmax of their own, with
    finite gradients.  w's relative error: the rounding of L - top (|L - top| < 20 here; at 1e30 the
    logits are equal), exp within 2 ulp (4 U), sums of k terms, reciprocal and products: at most 2 (20
    + 4 + k + 4) U in each of the two terms."""
    T = 41
    g = gen(E + k)
    logits = 2 * randn(g, T, E)
    ids = torch.argsort(torch.rand(T, E, generator=g, device=dev()), 1)[:, :k].contiguous().to(torch.int32)
    named = torch.zeros(T, E, dtype=torch.bool, device=dev()).scatter_(1, ids.long(), True)
    named[5] = False                                        # (a row that names its maximum too)
    logits = torch.where(named, logits - gap, logits).float()
    ids[7, 0] = E                                           # left out
    ids[9, 1] = ids[9, 0]                                   # named twice
    logits[11, ids[11, 0].long()] = -math.inf               # weight 0
    logits[12, ids[12].long()] = -math.inf                  # no weights at all
    if gap == 1e30:
        logits[11] = -1e30                                  # (with the row's maximum a named one too)
        logits[11, ids[11, 0].long()] = -math.inf
    grad_w = randn(g, T, k)
    layer = moe.MoELayer(T, 64, 64, E, k, flags=moe.FLAG_RENORMALIZE)
    got = layer.route_backward(logits, ids, grad_w=grad_w)
    assert status(moe, layer) == moe.DEV_BAD_INDEX
    want, terms = renormalised_reference(logits, ids, grad_w)
    assert_within(got, want, 4 * (20 + 8 + k) * U * terms + 1e-37, "dlogits")
    assert (got[12] == 0).all() and (got[~named & (torch.arange(T, device=dev()) != 5)[:, None]] == 0).all()
    # The losses' gradient is added to it.
    gl = torch.tensor([0.7, -0.3], device=dev())
    live = logits.clone()
    live[12] = 0                                            # (a row needs one finite logit)
    _, counts, _ = layer.balance_loss(live, ids)
    alone = layer.route_backward(live, ids, counts, gl)
    both = layer.route_backward(live, ids, counts, gl, grad_w)
    want, terms = renormalised_reference(live, ids, grad_w)
    assert_within(both, alone.double() + want, 4 * (20 + 8 + k) * U * terms + 2 * U * alone.abs().double() +
                  1e-37, "dlogits with the losses")


def test_layers_on_threads(moe):
    """Layers of different numbers of experts (and so of different shared-memory sizes), each on a
    thread and a stream of its own at once, give the bits that they give alone."""
    import threading
    T, d, F, k = 48, 128, 128, 2
    jobs = []
    for n, E in enumerate((1024, 3, 700, 40, 1000, 8)):
        g = gen(70 + n)
        layer = moe.MoELayer(T, d, F, E, k, flags=moe.FLAG_GATED if n % 2 else 0, w4=True)
        W1, W2 = make_experts(moe, g, E, 2 * F if n % 2 else F, F, d, ((32, 64, 128)[n % 3], 32), n < 3)
        x, logits = randn(g, T, d).to(torch.bfloat16), randn(g, T, E)
        ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        jobs.append((layer, x, routing(g, T, E, k, "random"), W1, W2, logits, ids, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(job):
        layer, x, route, W1, W2, logits, ids, stream = job
        return [(layer.expert_ffn_w4(x, *route, W1, None, W2, None, stream=stream),
                 *layer.balance_loss(logits, ids, stream=stream)) for _ in range(20)]

    got, start = [None] * len(jobs), threading.Barrier(len(jobs))

    def run(n):
        start.wait()
        got[n] = work(jobs[n])

    threads = [threading.Thread(target=run, args=(n,)) for n in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for job, results in zip(jobs, got):
        want = work(job)[0]
        torch.cuda.synchronize()
        for r in results:
            for a, b in zip(r, want):
                assert torch.equal(a, b)
        assert status(moe, job[0]) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_quantize_keeps_what_is_not_finite_in_its_group(moe, dtype, zeros, group, value):
    """A NaN or an infinity makes its own group's values not finite and changes no other group."""
    E, N, K = 2, 35, 576
    g = gen(80)
    W = randn(g, E, N, K).to(dtype)
    clean = moe.quantize_w4(W, group, zeros=zeros)
    hit = torch.rand(E, N, K, generator=g, device=dev()) < 0.002
    hit[1, 34, 575] = hit[0, 0, 0] = True
    w = moe.quantize_w4(torch.where(hit, torch.full_like(W, value), W), group, zeros=zeros)
    G = -(-K // group)
    in_group = torch.nn.functional.pad(hit, (0, G * group - K)).view(E, N, G, group).any(3)
    keep = ~in_group.transpose(1, 2)
    assert keep.any() and not keep.all()
    assert torch.equal(w.scale[keep], clean.scale[keep])
    assert not torch.isfinite(w.scale[~keep]).any()
    if zeros:
        assert torch.equal(w.zero[keep], clean.zero[keep])
    cols = in_group.repeat_interleave(group, 2)[:, :, :K]
    back, want = moe.dequantize_w4(w), moe.dequantize_w4(clean)
    assert torch.equal(back[~cols], want[~cols])
    assert not torch.isfinite(back[cols]).any()
    # The words past K, whose nibbles are 8, hold the same bits.
    past = torch.arange(16 * (-(-K // 128)), device=dev())
    first = 128 * (past // 16) + 32 * (past % 4) + 8 * (past % 16 // 4)
    assert (w.q[:, :, first >= K] == -0x77777778).all()


def stage_times(moe, call):
    """Milliseconds of the six stages of call() (its seven events' gaps), the host well ahead."""
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(moe.STAGE_EVENTS)]
    for e in ev:
        e.record()                                          # (creates the handle)
    torch.cuda.synchronize()
    torch.cuda._sleep(2000000)
    moe.moe_set_stage_events(ev)
    try:
        call()
    finally:
        moe.moe_set_stage_events(None)
    torch.cuda.synchronize()
    return [ev[i].elapsed_time(ev[i + 1]) for i in range(6)]


def median(values):
    return sorted(values)[len(values) // 2]


@pytest.mark.parametrize("T,d,F,k", [(256, 2048, 2048, 8), (4096, 1024, 1024, 4)])   # direct; read back
def test_block_stages_of_packed_products(moe, T, d, F, k):
    """A block over 4-bit weights records its two products, of the same weight bytes and flops, as two
    stages (neither below a fifth of their sum)."""
    E = 32
    g = gen(90)
    layer = moe.MoELayer(T, d, F, E, k, w4=True)
    W1, W2 = make_experts(moe, g, E, F, F, d, (64, 64), False)
    x, Wr = randn(g, T, d).to(torch.bfloat16), randn(g, d, E) / 32
    t = [stage_times(moe, lambda: layer.forward_block(x, Wr, None, W1, None, W2, None))
         for _ in range(7)]
    assert 0.2 < median([v[4] / (v[3] + v[4]) for v in t]) < 0.8


def test_block_stages_hold_the_norm(moe):
    """The norm runs after the first event: with it the first stage is longer by the norm's time (at
    least half of what the norm takes alone)."""
    T, d, E = 30000, 4096, 2
    g = gen(91)
    layer = moe.MoELayer(T, d, 64, E, 1, 0.01)
    x, Wr, ga = randn(g, T, d).to(torch.bfloat16), randn(g, d, E) / 64, randn(g, d)
    W1, W2 = (randn(g, E, 64, d) / 64).to(x.dtype), (randn(g, E, d, 64) / 8).to(x.dtype)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    alone, plain, normed = [], [], []
    for _ in range(7):
        torch.cuda.synchronize()
        torch.cuda._sleep(2000000)
        a.record()
        layer.layer_norm(x, ga, ga)
        b.record()
        torch.cuda.synchronize()
        alone.append(a.elapsed_time(b))
        for times, norm in ((plain, None), (normed, (ga, ga, 1e-5))):
            times.append(stage_times(moe, lambda: layer.forward_block(x, Wr, None, W1, None, W2, None,
                                                                      norm=norm))[0])
    assert median(normed) - median(plain) >= 0.5 * median(alone)


@pytest.mark.parametrize("C", [0.01, 2.0])               # scratch larger than H and Y; smaller
def test_training_calls_beside_a_prepared_router(moe, C):
    """The losses' and the norm's scratch shares the workspace with a forward and with the router's
    prepared terms: neither call's results change for the other's."""
    T, d, F, E, k = 3000, 512, 64, 16, 2
    g = gen(95)
    layer = moe.MoELayer(T, d, F, E, k, C, flags=moe.FLAG_ROUTER_PREPARED)
    plain = moe.MoELayer(T, d, F, E, k, C)
    x, Wr, ga = randn(g, T, d).to(torch.bfloat16), randn(g, d, E) / 23, randn(g, d)
    W1, W2 = (randn(g, E, F, d) / 23).to(x.dtype), (randn(g, E, d, F) / 8).to(x.dtype)
    moe.moe_prepare_router(layer.p, Wr, layer.ws)
    y, mean, rstd = layer.layer_norm(x, ga, ga)
    logits = randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    want = plain.forward(x, Wr, None, W1, None, W2, None)
    losses, grads = plain.balance_loss(logits, ids), plain.layer_norm_backward(y, x, ga, mean, rstd)
    for _ in range(2):
        for a, b in zip(layer.balance_loss(logits, ids), losses):
            assert torch.equal(a, b)
        for a, b in zip(layer.layer_norm_backward(y, x, ga, mean, rstd), grads):
            assert torch.equal(a, b)
        assert torch.equal(layer.forward(x, Wr, None, W1, None, W2, None), want)


# ----------------------------------------------------------------------------------------------
# Every split of the 4-bit products
# ----------------------------------------------------------------------------------------------
def k_split(E, max_rows, K, N):
    """Warps that share a unit's K, as the products choose them: 2, 4 or 8."""
    lks = 1
    while lks < 3 and (256 << lks) <= K and min(E, max_rows) * (N // 32) < 148 * (8 >> lks):
        lks += 1
    return 1 << lks


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,d,F,E,k,gated,splits", [
    (1, 2048, 128, 8, 2, False, (8, 2)), (1, 2048, 256, 8, 2, True, (8, 2)),
    (1, 576, 640, 8, 2, False, (4, 4)), (1, 576, 640, 8, 2, True, (4, 4)),
    (20, 1472, 1408, 4, 2, False, (8, 8)), (20, 1472, 1408, 4, 2, True, (4, 8)),
    (20, 1472, 512, 4, 2, True, (8, 4)), (33, 960, 768, 5, 1, False, (4, 4)),
    (7, 1024, 2048, 3, 3, True, (4, 8)), (64, 512, 1152, 8, 4, False, (4, 8)),
    (50, 1088, 384, 30, 5, True, (2, 2))])
def test_expert_ffn_w4_splits(moe, T, d, F, E, k, gated, splits, group, zeros):
    """Both products, plain and gated, at every split of K, with ragged last steps, for every group
    size and with and without offsets."""
    g = gen(T + d + F + group)
    F1 = 2 * F if gated else F
    assert (k_split(E, T * k, d, F1), k_split(E, T * k, F, d)) == splits
    W1, W2 = make_experts(moe, g, E, F1, F, d, (group, group), zeros)
    b1, b2 = 0.1 * randn(g, E, F1), 0.1 * randn(g, E, d)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets, rowtok = routing(g, T, E, k, "random")
    layer = moe.MoELayer(T, d, F, E, k, flags=moe.FLAG_GATED if gated else 0, w4=True)
    Y = layer.expert_ffn_w4(x, offsets, rowtok, W1, b1, W2, b2)
    ref, tol = ffn_reference(x, offsets, rowtok, W1, b1, W2, b2, gated, False)
    assert_within(Y, ref, tol, "Y")
    assert status(moe, layer) == 0
    assert torch.equal(Y, layer.expert_ffn_w4(x, offsets, rowtok, W1, b1, W2, b2))


@pytest.mark.parametrize("d,F,gated,splits", [
    (256, 128, False, (2, 2)), (256, 128, True, (2, 2)), (576, 640, False, (4, 4)),
    (576, 640, True, (4, 4)), (1472, 1408, False, (8, 8)), (1472, 896, True, (8, 4))])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 7, 8, 9, 12, 13, 15, 16, 17, 24, 25, 31, 32, 33, 63, 64])
def test_expert_ffn_w4_row_counts_of_each_split(moe, d, F, gated, splits, rows):
    """Numbers of rows around the row tiles of each split (16, 8 and 4 rows), beside empty experts and
    a full one; rows behind the last one stay as they were."""
    T, E = 96, 5
    g = gen(rows + d)
    F1 = 2 * F if gated else F
    assert (k_split(E, T, d, F1), k_split(E, T, F, d)) == splits
    W1, W2 = make_experts(moe, g, E, F1, F, d, (64, 32), rows % 2 == 0)
    x = randn(g, T, d).to(torch.bfloat16)
    offsets = torch.tensor([0, 0, rows, rows, rows + 3, rows + 3], dtype=torch.int32, device=dev())
    rowtok = torch.zeros(T, dtype=torch.int32, device=dev())
    rowtok[:rows + 3] = torch.randint(0, T, (rows + 3,), generator=g, device=dev()).to(torch.int32)
    layer = moe.MoELayer(T, d, F, E, 1, flags=moe.FLAG_GATED if gated else 0, w4=True)
    Y = torch.full((T, d), 5.0, dtype=torch.bfloat16, device=dev())
    moe.moe_expert_ffn_packed(layer.p, x, offsets, rowtok, W1.c, None, W2.c, None, Y, layer.ws)
    ref, tol = ffn_reference(x, offsets, rowtok, W1, None, W2, None, gated, False)
    assert_within(Y[:rows + 3], ref, tol, "Y")
    assert (Y[rows + 3:] == 5.0).all()


def test_block_over_packed_weights_without_rows(moe):
    """A capacity of zero keeps no pair: the block leaves x as it is; so does a batch of no tokens."""
    d, F, E, k = 128, 64, 4, 2
    g = gen(97)
    W1, W2 = make_experts(moe, g, E, F, F, d, (32, 64), True)
    Wr, ga = randn(g, d, E), randn(g, d)
    for T, C in ((40, 0.0), (0, 1.0)):
        x = randn(g, T, d).to(torch.bfloat16)
        layer = moe.MoELayer(T, d, F, E, k, C, w4=True)
        out, r = layer.forward_block(x, Wr, None, W1, None, W2, None, norm=(ga, ga, 1e-5))
        assert torch.equal(out, x) and (r["drop_out"] == 1).all()
        assert status(moe, layer) == 0


def test_read_back_of_every_scale(moe):
    """Every bfloat16 scale (subnormal ones, infinities and NaN too) times every nibble is the float32
    product rounded once; with an offset the float32 fused sum rounded once."""
    bits = torch.arange(65536, device=dev(), dtype=torch.int32).to(torch.int16)
    scale = bits.view(torch.bfloat16)
    q = torch.zeros(1, 65536, 16, dtype=torch.int32, device=dev())
    q[:] = torch.tensor([0x76543210, -0x01234568], dtype=torch.int32, device=dev()).repeat(8)
    side = scale.view(1, 1, 65536).contiguous()
    for zero in (None, side.flip(2).contiguous(), torch.full_like(side, 0.37)):
        w = moe.W4Weights(q, side, zero, K=128, group=128)
        # In 64 bits the product is exact, and the sum exact or, with terms more than 2^41 apart, one
        # that rounds like the larger term alone.
        v = unpack(q, 128).double() * scale.double().view(1, -1, 1)
        if zero is not None:
            v = v + zero.double().view(1, -1, 1)
        want = v.float().to(torch.bfloat16)
        got = moe.dequantize_w4(w)
        same = (got == want) | (got.isnan() & want.isnan())
        assert same.all()


# ----------------------------------------------------------------------------------------------
# Long sums, against bounds of the depth they have
# ----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,E,k,groups", [(1 << 21, 8, 2, 64), (1 << 20, 64, 6, 64), (1 << 18, 1024, 4, 8)])
def test_balance_loss_of_many_tokens(moe, T, E, k, groups):
    """Large batches: 256 blocks of `groups` tokens at a time, so a lane adds T / (256 groups)
    probabilities behind one another; the lanes, warps (16), cluster (8) and clusters (32) follow, at
    most 64 more."""
    g = gen(E)
    logits = 2 * randn(g, T, E)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    layer = moe.MoELayer(T, 64, 64, E, k, 0.001)
    losses, counts, probs = layer.balance_loss(logits, ids)
    P, z, span = torch.zeros(E, dtype=torch.float64, device=dev()), 0.0, 0.0
    for L in logits.split(1 << 16):
        L = L.double()
        lse = torch.logsumexp(L, 1)
        P += torch.exp(L - lse[:, None]).sum(0)
        z += (lse ** 2).sum()
        span = max(span, (L.amax(1) - L.amin(1)).max().item())
    n = torch.bincount(ids.reshape(-1).long(), minlength=E)
    P, z = P / T, z / T
    assert torch.equal(counts.long(), torch.cat([n, torch.tensor([T], device=dev())]))
    # A probability's own error as in the operators' main tests, and the sum over the tokens.
    b = 2 * (span + 45) + T // (256 * groups) + 64
    assert_within(probs, P, b * U * P, "probs")
    bal = E * (n.double() / (T * k) * P).sum()
    # (sum over the experts: a thread's one or two, 5 tree steps, the warps; lse's error is that of the
    # exponentials' sum plus its own two roundings, twice in its square)
    assert_within(losses[:1], bal[None], (b + 64) * U * bal, "balance loss")
    assert_within(losses[1:], z[None], (2 * (span + 45) / z ** 0.5 + b + 8) * 2 * U * z, "z-loss")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,depth", [(200000, 512, 200000 // (296 * 8) + 64),
                                       (50000, 4096, 50000 // 296 + 64),
                                       (20000, 8200, 20000 // 16 + 64)])
def test_layer_norm_parameter_sums_of_many_rows(moe, dtype, T, d, depth):
    """dgamma and dbeta: a thread adds its rows behind one another (of 296 blocks and the rows a block
    has in flight; a sixteenth of all rows past 8192 columns), then the blocks' partial rows."""
    g = gen(d)
    x, dy = randn(g, T, d).to(dtype), randn(g, T, d).to(dtype)
    gamma = randn(g, d)
    mean, rstd = x.float().mean(1), 1 / x.float().std(1)
    layer = moe.MoELayer(T, d, 64, 1, 1, dtype="f32" if dtype == torch.float32 else "bf16")
    _, dgamma, dbeta = layer.layer_norm_backward(dy, x, gamma, mean, rstd)
    ref = [torch.zeros(d, dtype=torch.float64, device=dev()) for _ in range(4)]
    for r in range(0, T, 8192):
        s = slice(r, r + 8192)
        xh = (x[s].double() - mean[s, None].double()) * rstd[s, None].double()
        y = dy[s].double()
        for acc, v in zip(ref, (y * xh, (y * xh).abs(), y, y.abs())):
            acc += v.sum(0)
    # (x - mean) rstd: two roundings.
    assert_within(dgamma, ref[0], (depth + 3) * U * ref[1], "dgamma")
    assert_within(dbeta, ref[2], depth * U * ref[3], "dbeta")
