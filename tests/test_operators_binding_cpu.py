"""The binding's side of the calls around the layer, on host tensors (no GPU needed): what it keeps
between calls, and what it refuses."""
import pytest
import torch

from expert_ffn_layer_router_b200 import build as lib_build


@pytest.fixture(scope="module")
def moe():
    lib_build.build()
    from expert_ffn_layer_router_b200 import moe as m
    return m


def packed(moe, E=4, N=64, K=192, group=64, zeros=True):
    side = (E, -(-K // group), N)
    return moe.W4Weights(torch.zeros(E, N, 16 * (-(-K // 128)), dtype=torch.int32),
                         torch.zeros(side, dtype=torch.bfloat16),
                         torch.zeros(side, dtype=torch.bfloat16) if zeros else None, K=K, group=group)


@pytest.mark.parametrize("name", ["q", "scale", "zero"])
def test_packed_weights_follow_their_tensors(moe, name):
    """The addresses a call gets are those of the tensors at the call: a tensor cannot be replaced
    behind them, and one that was given other storage in place is followed or refused."""
    w = packed(moe)
    t = getattr(w, name)
    assert (w.c.q, w.c.scale, w.c.zero, w.c.group) == (w.q.data_ptr(), w.scale.data_ptr(),
                                                       w.zero.data_ptr(), 64)
    with pytest.raises(AttributeError):
        setattr(w, name, t.clone())
    moved = t.clone()
    t.set_(moved)
    assert getattr(w.c, name) == moved.data_ptr()
    t.resize_(1)
    with pytest.raises(moe.MoeError):
        w.c
    assert packed(moe, zeros=False).c.zero is None


def test_packed_weights_are_checked(moe):
    q, s = torch.zeros(2, 32, 16, dtype=torch.int32), torch.zeros(2, 2, 32, dtype=torch.bfloat16)
    ok = moe.W4Weights(q, s, K=128, group=64)
    assert (ok.E, ok.N, ok.K, ok.group) == (2, 32, 128, 64)
    for args, kw in (((None, s), {}), ((q[0], s), {}), ((q, None), {}), ((q, s.float()), {}),
                     ((q, s, s[:1]), {}), ((q.long(), s), {}), ((q, s), dict(group=32)),
                     ((q, s), dict(K=64)), ((q, s), dict(K=256)), ((q.transpose(0, 1), s), {})):
        with pytest.raises(moe.MoeError):
            moe.W4Weights(*args, **{**dict(K=128, group=64), **kw})


class FakeGuard:
    depth = 0

    def __init__(self, *a):
        pass

    def __enter__(self):
        FakeGuard.depth += 1

    def __exit__(self, *exc):
        FakeGuard.depth -= 1
        return False


class FakeStream:
    cuda_stream = 1 << 20

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_streams_that_cannot_be_used(moe, monkeypatch):
    """A stream of another device than the tensors', or something that is no stream, is refused (the
    work would have run on another stream than the caller ordered), and the current device and stream
    are what they were."""
    monkeypatch.setattr(torch.cuda, "device", FakeGuard)
    monkeypatch.setattr(torch.cuda, "stream", FakeGuard)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 77, raising=False)
    dev = torch.device("cuda", 0)
    for stream in (FakeStream(1), "stream", 1.5, object()):
        with pytest.raises(moe.MoeError):
            with moe._on(dev, stream):
                pass
        assert FakeGuard.depth == 0
    with moe._on(dev, FakeStream(0)) as handle:
        assert handle == 77 and FakeGuard.depth == 2
    assert FakeGuard.depth == 0


def test_arguments_of_another_kind(moe):
    """What is no tensor, no 4-bit weight or of a type that a call does not take raises the library's
    error before anything is read (half-precision weights would have been read as float32)."""
    half = torch.zeros(1, 32, 64, dtype=torch.float16)
    q, s = torch.zeros(1, 32, 16, dtype=torch.int32), torch.zeros(1, 2, 32, dtype=torch.bfloat16)
    layer = moe.MoELayer(16, 64, 64, 4, 2, device="cpu", w4=True)
    x, f = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(64)
    w, counts = packed(moe, N=64, K=64), torch.zeros(5, dtype=torch.int32)
    calls = [lambda: moe.moe_quantize_packed(half, 1, 32, 64, 32, q, s, None, 0),
             lambda: moe.moe_quantize_packed(half.double(), 1, 32, 64, 32, q, s, None, 0),
             lambda: moe.quantize_w4(half, 32), lambda: moe.quantize_w4(None, 32),
             lambda: moe.dequantize_w4(q), lambda: moe.dequantize_w4(None)]
    calls += [lambda r=r: layer.expert_ffn_w4(x, counts, r, w, None, w, None)
              for r in (None, [0] * 32, torch.zeros(32))]
    calls += [lambda n=n: layer.forward_block(x, torch.zeros(64, 4), None, w, None, w, None, norm=n)
              for n in (f, (f, f), (f, None, 1e-5), (None, f, 1e-5))]
    for n, call in enumerate(calls):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.MOE_ERR_INVALID_ARG, n
        assert "CUDA device" not in str(e.value), n


@pytest.mark.parametrize("args,size", [
    ((64, 2048, 1024, 64, 8, float("inf"), "bf16", 0), 4237824),
    ((16384, 2048, 1408, 64, 6, 1.0, "bf16", 0), 690587648),
    ((65536, 4096, 1024, 128, 8, 1.0, "bf16", 4), 5447879936),
    ((1, 2048, 1024, 64, 8, float("inf"), "bf16", 0), 1101568),
    ((8, 4, 8, 4, 1, 1.25, "f32", 0), 36864),
    ((4096, 512, 256, 1024, 2, 1.25, "f32", 0), 67269632)])
def test_layers_pay_nothing_for_training_scratch(moe, args, size):
    """The scratch of the losses and of the norm's parameter gradients lies over the forward's: a
    layer's workspace is what the forward alone needs."""
    assert moe.moe_workspace_size(moe.problem(*args)) == size
