"""The operators around the layer at their edges: after errors of the data, at extreme values, over
every split of the 4-bit products, beside each other on threads.  (Helpers and bounds are those of the
operators' main tests.)"""
import math

import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_operators import gen, make_experts, moe, randn, routing, status  # noqa: F401

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
