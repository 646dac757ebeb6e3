"""The layer's operators around the router and the experts' products, each in its plain form and
through the library, with the cases they are measured on.

  balance   the router's training step: load-balance loss, router z-loss and per-expert counts, then
            their gradient (and that of the k routing weights) with respect to the logits
  ffn_w4    the expert FFN over 4-bit weights with group scales, W1 and W2
  quant_w4  quantising weights to that format and reading them back
  norm      the layer norm in front of the layer, forward or forward and backward

The 4-bit format of a weight [E, N, K]: 32-bit words q [E, N, 16 * ceil(K / 128)]; word 4 t + j of a
row's 128-column chunk c holds the columns 128 c + 32 j + 8 t + i, i = 0..7, column i in bits
4 (4 (i % 2) + i // 2) and up; scales (and optional offsets) [E, ceil(K / group), N] bfloat16; the
value is scale * (nibble - 8) + offset.  Columns past K hold 8.
"""
import math

import torch

own = False

EPS = 1e-5


# ----------------------------------------------------------------------------------------------
# Cases.  The sizes are those of the library's own workloads (64 experts of width 2048 x 1024 in
# decoding, 2048 x 1408 in training, 128 experts and 65,536 tokens of width 4096 in prefill).
# ----------------------------------------------------------------------------------------------
def listed():
    return [
        # A micro-batch of 64 tokens: launch latency counts.
        dict(name="balance_t64", op="balance", T=64, E=64, k=8, mask=False, grad_w=False,
             renorm=False),
        # A padded training batch (a quarter of the rows masked, NaN in them).
        dict(name="balance_t16384_masked", op="balance", T=16384, E=64, k=6, mask=True,
             grad_w=False, renorm=False),
        # A large batch whose router also learns through its renormalised top-k weights.
        dict(name="balance_t65536_grad_w", op="balance", T=65536, E=128, k=8, mask=False,
             grad_w=True, renorm=True),
        # One decoded token: eight experts are read.
        dict(name="ffn_w4_t1", op="ffn_w4", T=1, d=2048, F=1024, E=64, k=8, group=128,
             zeros=False, gated=False),
        # A decoding batch: every expert's weights are read for a handful of rows.
        dict(name="ffn_w4_t64", op="ffn_w4", T=64, d=2048, F=1024, E=64, k=8, group=64,
             zeros=False, gated=False),
        # A gated layer with offsets and small groups, ragged rows, an odd number of K chunks.
        dict(name="ffn_w4_t129_gated", op="ffn_w4", T=129, d=2048, F=1408, E=64, k=6, group=32,
             zeros=True, gated=True),
        # A prompt of 4096 tokens over the same weights.
        dict(name="ffn_w4_t4096", op="ffn_w4", T=4096, d=2048, F=1408, E=64, k=6, group=128,
             zeros=False, gated=False),
        # Quantising a decoding layer's W1 from bfloat16.
        dict(name="quant_w4_e64", op="quant_w4", E=64, N=1024, K=2048, group=64, zeros=False,
             dtype="bf16"),
        # Two experts' float32 master weights, with offsets, K not a multiple of the chunk.
        dict(name="quant_w4_e2_f32", op="quant_w4", E=2, N=2048, K=1472, group=128, zeros=True,
             dtype="f32"),
        # The norm of a decoding batch.
        dict(name="norm_t64", op="norm", T=64, d=2048, dtype="bf16", train=False, res=False),
        # A float32 training step with an odd number of rows.
        dict(name="norm_t4099_f32", op="norm", T=4099, d=1408, dtype="f32", train=True,
             res=False),
        # The prefill width over a whole batch, backward pass with the residual's gradient.
        dict(name="norm_t65536", op="norm", T=65536, d=4096, dtype="bf16", train=True, res=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "ffn_w4", "ffn_w4", "quant_w4", "norm"])
    if op == "balance":
        E = _log(rng, 4, 256)
        T = min(_log(rng, 1, 65536), 65536 * 128 // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), mask=rng.random() < 0.5,
                    grad_w=rng.random() < 0.5, renorm=rng.random() < 0.5)
    if op == "ffn_w4":
        E = _log(rng, 4, 64)
        return dict(op=op, T=_log(rng, 1, 4096 if rng.random() < 0.25 else 256),
                    d=64 * _log(rng, 4, 32), F=128 * _log(rng, 1, 11), E=E,
                    k=rng.randint(1, min(6, E)), group=rng.choice([32, 64, 128]),
                    zeros=rng.random() < 0.5, gated=rng.random() < 0.5)
    if op == "quant_w4":
        return dict(op=op, E=_log(rng, 1, 64), N=32 * _log(rng, 1, 32), K=64 * _log(rng, 1, 32),
                    group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f32"]))
    return dict(op=op, T=_log(rng, 1, 16384), d=_log(rng, 16, 8192),
                dtype=rng.choice(["bf16", "f32"]), train=rng.random() < 0.7,
                res=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _weights(g, E, N, K, dtype):
    return (torch.randn(E, N, K, generator=g, device="cuda") / math.sqrt(K)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    c = case
    s = {"case": dict(c)}
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        logits = randn(T, E) + 0.5 * randn(E)
        s["ids"] = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        s["mask"] = None
        if c["mask"]:
            keep = torch.rand(T, generator=g, device="cuda") >= 0.25
            s["mask"] = keep.to(torch.uint8)
            logits[~keep] = math.nan
        s["logits"] = logits
        s["grad_losses"] = torch.tensor([0.01, 0.001], device="cuda")
        s["grad_w"] = randn(T, k) / math.sqrt(T) if c["grad_w"] else None
    elif c["op"] == "ffn_w4":
        T, d, F, E, k = c["T"], c["d"], c["F"], c["E"], c["k"]
        F1 = 2 * F if c["gated"] else F
        s["x"] = randn(T, d).to(torch.bfloat16)
        ids = torch.topk(randn(T, E), k, dim=1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        s["rowtok"] = (order // k).to(torch.int32)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0).to(torch.int32)
        s["w1"] = _quantize_plain(_weights(g, E, F1, d, torch.bfloat16), c["group"], c["zeros"])
        s["w2"] = _quantize_plain(_weights(g, E, d, F, torch.bfloat16), c["group"], c["zeros"])
        s["b1"] = 0.02 * randn(E, F1)
        s["b2"] = 0.02 * randn(E, d)
    elif c["op"] == "quant_w4":
        s["W"] = _weights(g, c["E"], c["N"], c["K"], _dt(c["dtype"]))
    else:
        T, d = c["T"], c["d"]
        s["x"] = (randn(T, d) * (0.5 + torch.rand(T, 1, generator=g, device="cuda")) +
                  0.3 * randn(T, 1)).to(_dt(c["dtype"]))
        s["gamma"] = 1.0 + 0.1 * randn(d)
        s["beta"] = 0.1 * randn(d)
        if c["train"]:
            s["dy"] = randn(T, d).to(_dt(c["dtype"]))
            s["dres"] = randn(T, d).to(_dt(c["dtype"])) if c["res"] else None
    if own:
        s["layer"] = _layer(c)
    return s


def _layer(c):
    """The layer object a program keeps: the problem's description and its workspace."""
    from expert_ffn_layer_router_b200 import moe
    if c["op"] == "balance":
        return moe.MoELayer(c["T"], 64, 64, c["E"], c["k"],
                            flags=moe.FLAG_RENORMALIZE if c["renorm"] else 0)
    if c["op"] == "ffn_w4":
        return moe.MoELayer(c["T"], c["d"], c["F"], c["E"], c["k"],
                            flags=moe.FLAG_GATED if c["gated"] else 0, w4=True)
    if c["op"] == "norm":
        return moe.MoELayer(c["T"], c["d"], 64, 1, 1, dtype=c["dtype"])
    return None


# ----------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from expert_ffn_layer_router_b200 import moe
    c, layer = s["case"], s["layer"]
    if c["op"] == "balance":
        losses, counts, probs = layer.balance_loss(s["logits"], s["ids"], mask=s["mask"])
        dlogits = layer.route_backward(s["logits"], s["ids"], counts,
                                       grad_losses=s["grad_losses"], grad_w=s["grad_w"],
                                       mask=s["mask"])
        return dict(losses=losses, counts=counts, probs=probs, dlogits=dlogits)
    if c["op"] == "ffn_w4":
        F1 = 2 * c["F"] if c["gated"] else c["F"]
        W1 = moe.W4Weights(*s["w1"], K=c["d"], group=c["group"])
        W2 = moe.W4Weights(*s["w2"], K=c["F"], group=c["group"])
        assert W1.N == F1
        return dict(Y=layer.expert_ffn_w4(s["x"], s["offsets"], s["rowtok"], W1, s["b1"], W2,
                                          s["b2"]))
    if c["op"] == "quant_w4":
        w = moe.quantize_w4(s["W"], c["group"], zeros=c["zeros"])
        return dict(W=moe.dequantize_w4(w), scale=w.scale, zero=w.zero)
    y, mean, rstd = layer.layer_norm(s["x"], s["gamma"], s["beta"], EPS)
    out = dict(y=y, mean=mean, rstd=rstd)
    if c["train"]:
        out["dx"], out["dgamma"], out["dbeta"] = layer.layer_norm_backward(
            s["dy"], s["x"], s["gamma"], mean, rstd, dres=s["dres"])
    return out


def _plain(s):
    return {"balance": _plain_balance, "ffn_w4": _plain_ffn, "quant_w4": _plain_quant,
            "norm": _plain_norm}[s["case"]["op"]](s)


def _plain_balance(s):
    c, ids = s["case"], s["ids"].long()
    T, E, k = c["T"], c["E"], c["k"]
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    L = torch.where(keep[:, None], s["logits"], 0.0)
    kf = keep.float()[:, None]
    m = L.amax(1, keepdim=True)
    u = torch.exp(L - m)
    Z = u.sum(1, keepdim=True)
    p = u / Z * kf
    lse = (m + torch.log(Z)) * kf
    n = keep.sum()
    n1 = n.clamp(min=1).float()
    counts = torch.zeros(E, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, ids.reshape(-1), keep[:, None].expand(T, k).reshape(-1).long())
    f = counts.float() / (n1 * k)
    P = p.sum(0) / n1
    losses = torch.stack([E * (f * P).sum(), lse.square().sum() / n1])
    # Gradient with respect to the probabilities, then through the softmax.
    gb, gz = s["grad_losses"][0], s["grad_losses"][1]
    dp = (gb * E / n1 * f)[None, :].expand(T, E)
    if s["grad_w"] is not None:
        dw = s["grad_w"]
        if c["renorm"]:
            pk = torch.gather(p, 1, ids)
            S = torch.where(keep[:, None], pk.sum(1, keepdim=True), 1.0)
            dw = (dw - (dw * pk).sum(1, keepdim=True) / S) / S
        dp = dp.scatter_add(1, ids, dw)
    dl = p * (dp - (p * dp).sum(1, keepdim=True)) + 2.0 * gz / n1 * lse * p
    return dict(losses=losses, counts=torch.cat([counts, n[None]]).to(torch.int32), probs=P,
                dlogits=torch.where(keep[:, None], dl, 0.0))


def _chunks(K):
    return (K + 127) // 128


def _per_group(v, K, group):
    """[E, groups, N] -> [E, N, K]: each column's scale or offset."""
    return v.float().transpose(1, 2).repeat_interleave(group, 2)[:, :, :K]


def _quantize_plain(W, group, zeros):
    """(words, scales, offsets or None) of W [E, N, K]; scales and offsets are rounded to bfloat16
    before the values are divided by them."""
    E, N, K = W.shape
    G = (K + group - 1) // group
    w = W.float()
    wp = torch.cat([w, w.new_zeros(E, N, G * group - K)], 2).view(E, N, G, group)
    in_row = (torch.arange(G * group, device=W.device) < K).view(G, group)
    if zeros:
        lo = torch.where(in_row, wp, math.inf).amin(3)
        hi = torch.where(in_row, wp, -math.inf).amax(3)
        scale = ((hi - lo) / 15.0).to(torch.bfloat16)
        zero = (lo + 8.0 * scale.float()).to(torch.bfloat16)
    else:
        scale = (wp.abs().amax(3) / 7.0).to(torch.bfloat16)
        zero = None
    sc = scale.float()[..., None]
    wz = wp - zero.float()[..., None] if zeros else wp
    q = torch.where(sc > 0, torch.round(wz / sc), 0.0).clamp(-8, 7)
    q = (q.view(E, N, G * group)[:, :, :K] + 8).to(torch.uint8)
    C = _chunks(K)
    q = torch.cat([q, q.new_full((E, N, C * 128 - K), 8)], 2)
    q = q.view(E, N, C, 4, 4, 4, 2).permute(0, 1, 2, 4, 3, 6, 5)    # [.., c, t, j, i % 2, i // 2]
    q = q.reshape(E, N, C * 16, 4, 2).long()                        # bytes of two nibbles
    byte = (q[..., 0] | (q[..., 1] << 4)).to(torch.uint8).contiguous()
    words = byte.view(torch.int32).view(E, N, C * 16)
    return (words, scale.transpose(1, 2).contiguous(),
            zero.transpose(1, 2).contiguous() if zeros else None)


def _nibbles(words, K):
    """[E, N, 16 C] words -> [E, N, K] values - 8 in float32."""
    E, N, W = words.shape
    sh = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    v = (words[..., None] >> sh) & 15
    v = v.view(E, N, W // 16, 4, 4, 2, 4).permute(0, 1, 2, 4, 3, 6, 5).reshape(E, N, W * 8)
    return v[:, :, :K].float() - 8.0


def _dequantize_plain(words, scale, zero, K, group):
    w = _nibbles(words, K) * _per_group(scale, K, group)
    return w if zero is None else w + _per_group(zero, K, group)


def _plain_ffn(s):
    c = s["case"]
    d, F, E, G = c["d"], c["F"], c["E"], c["group"]
    R = s["rowtok"].numel()
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    act = torch.nonzero(n)[:, 0]                     # the experts that have rows
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), n, output_size=R)
    slot = torch.arange(R, device="cuda") - s["offsets"].long()[e]
    at = (torch.cumsum(n > 0, 0) - 1)[e]
    xp = torch.zeros(act.numel(), int(n.max()), d, device="cuda")
    xp[at, slot] = s["x"].float()[s["rowtok"].long()]

    def values(w, K):
        return _dequantize_plain(*(None if v is None else v[act] for v in w), K, G)

    h = torch.bmm(xp, values(s["w1"], d).transpose(1, 2)) + s["b1"][act][:, None, :]
    if c["gated"]:
        a = h[..., :F] / (1.0 + torch.exp(-h[..., :F])) * h[..., F:]
    else:
        a = h / (1.0 + torch.exp(-h))
    y = torch.bmm(a, values(s["w2"], F).transpose(1, 2)) + s["b2"][act][:, None, :]
    return dict(Y=y[at, slot].to(torch.bfloat16))


def _plain_quant(s):
    c = s["case"]
    words, scale, zero = _quantize_plain(s["W"], c["group"], c["zeros"])
    w = _dequantize_plain(words, scale, zero, c["K"], c["group"])
    return dict(W=w.to(torch.bfloat16), scale=scale, zero=zero)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt(xc.square().mean(1, keepdim=True) + EPS)
    xh = xc * rstd
    out = dict(y=(xh * s["gamma"] + s["beta"]).to(s["x"].dtype), mean=mean[:, 0], rstd=rstd[:, 0])
    if c["train"]:
        dy = s["dy"].float()
        out["dgamma"] = (dy * xh).sum(0)
        out["dbeta"] = dy.sum(0)
        gy = dy * s["gamma"]
        dx = (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True)) * rstd
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        out["dx"] = dx.to(s["x"].dtype)
    return out


# ----------------------------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        b = 2 * T * E * 4 + T * k * 4 + E * 8
        b += T if c["mask"] else 0
        b += T * k * 4 if c["grad_w"] else 0
        return {"bytes": b, "flops": 12 * T * E}
    if c["op"] == "ffn_w4":
        T, d, F, E, k, G = c["T"], c["d"], c["F"], c["E"], c["k"], c["group"]
        F1 = 2 * F if c["gated"] else F
        # Experts that get at least one of T uniform top-k choices.
        active = E * (1.0 - (1.0 - k / E) ** T)
        sides = 2 * (2 if c["zeros"] else 1)
        per = (F1 * d + d * F) / 2 + sides * (F1 * -(-d // G) + d * -(-F // G)) + 4 * (F1 + d)
        return {"bytes": active * per + 2 * T * d + 2 * T * k * d + 4 * T * k,
                "flops": 2 * T * k * (F1 * d + d * F)}
    if c["op"] == "quant_w4":
        E, N, K, G = c["E"], c["N"], c["K"], c["group"]
        size = 2 if c["dtype"] == "bf16" else 4
        n = E * N * K
        side = E * N * -(-K // G) * 2 * (2 if c["zeros"] else 1)
        # The words are written by one call and read by the other.
        return {"bytes": n * size + 2 * (n / 2 + side) + 2 * n, "flops": 4 * n}
    size = 2 if c["dtype"] == "bf16" else 4
    n = c["T"] * c["d"]
    b = 2 * n * size + 8 * c["T"] + 8 * c["d"]
    f = 8 * n
    if c["train"]:
        # x again: the forward's is another pass of the program, long before this one.
        b += (3 + (1 if c["res"] else 0)) * n * size + 8 * c["T"] + 12 * c["d"]
        f += 14 * n
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------------------------------------
# The same results in 64 bits, from the definitions
# ----------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "ffn_w4": _exact_ffn, "quant_w4": _exact_quant,
            "norm": _exact_norm}[case["op"]](s)


def _exact_balance(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    rows = (torch.arange(T, device="cuda") if s["mask"] is None
            else torch.nonzero(s["mask"])[:, 0])
    n = rows.numel()
    L = s["logits"][rows].double().requires_grad_(True)
    ids = s["ids"][rows].long()
    one_hot = torch.zeros(n, E, dtype=torch.float64, device="cuda").scatter_(1, ids, 1.0)
    cnt = one_hot.sum(0)
    lse = torch.logsumexp(L, 1)
    p = torch.exp(L - lse[:, None])
    d = max(n, 1)
    P = p.sum(0) / d
    bal = E * torch.dot(cnt / (d * k), P)
    z = (lse ** 2).sum() / d
    g = s["grad_losses"].double()
    total = g[0] * bal + g[1] * z
    if s["grad_w"] is not None:
        w = torch.gather(p, 1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        total = total + (w * s["grad_w"][rows].double()).sum()
    dl = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    dl[rows] = torch.autograd.grad(total, L)[0]
    counts = torch.cat([cnt, torch.tensor([float(n)], device="cuda").double()]).to(torch.int32)
    return dict(losses=torch.stack([bal, z]).detach(), counts=counts, probs=P.detach(),
                dlogits=dl)


def _exact_values(w, e, K, group):
    """Expert e's [N, K] weights, column by column position."""
    words, scale, zero = w
    k = torch.arange(K, device="cuda")
    j, t, i = (k % 128) // 32, (k % 32) // 8, k % 8
    word = (k // 128) * 16 + 4 * t + j
    nib = (words[e].long()[:, word] >> (4 * (4 * (i % 2) + i // 2))) % 16
    v = (nib - 8).double() * scale[e].double()[k // group, :].T
    return v if zero is None else v + zero[e].double()[k // group, :].T


def _exact_ffn(s):
    c = s["case"]
    off = s["offsets"].tolist()
    Y = torch.zeros(off[-1], c["d"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        xe = s["x"][s["rowtok"][lo:hi].long()].double()
        h = xe @ _exact_values(s["w1"], e, c["d"], c["group"]).T + s["b1"][e].double()
        if c["gated"]:
            a = torch.nn.functional.silu(h[:, :c["F"]]) * h[:, c["F"]:]
        else:
            a = torch.nn.functional.silu(h)
        Y[lo:hi] = a @ _exact_values(s["w2"], e, c["F"], c["group"]).T + s["b2"][e].double()
    return dict(Y=Y)


def _exact_quant(s):
    c = s["case"]
    K, group = c["K"], c["group"]
    W = s["W"].double()
    out, scale, zero = torch.empty_like(W), [], []
    for k0 in range(0, K, group):
        w = W[:, :, k0:k0 + group]
        if c["zeros"]:
            lo, hi = w.min(2).values, w.max(2).values
            sc = ((hi - lo) / 15).to(torch.bfloat16).double()
            zr = (lo + 8 * sc).to(torch.bfloat16).double()
        else:
            sc = (w.abs().max(2).values / 7).to(torch.bfloat16).double()
            zr = torch.zeros_like(sc)
        step = torch.where(sc > 0, sc, 1.0)[..., None]
        q = torch.clamp(torch.round((w - zr[..., None]) / step), -8, 7)
        out[:, :, k0:k0 + group] = q * sc[..., None] + zr[..., None]
        scale.append(sc)
        zero.append(zr)
    return dict(W=out, scale=torch.stack(scale, 1),
                zero=torch.stack(zero, 1) if c["zeros"] else None)


def _exact_norm(s):
    c = s["case"]
    T, d = c["T"], c["d"]
    ga, be = s["gamma"].double(), s["beta"].double()
    out = dict(y=torch.empty(T, d, dtype=torch.float64, device="cuda"),
               mean=torch.empty(T, dtype=torch.float64, device="cuda"),
               rstd=torch.empty(T, dtype=torch.float64, device="cuda"))
    if c["train"]:
        out.update(dx=torch.empty(T, d, dtype=torch.float64, device="cuda"),
                   dgamma=torch.zeros_like(ga), dbeta=torch.zeros_like(be))
    for t in range(0, T, 8192):                      # blocks of rows bound the 64-bit copies
        r = slice(t, min(t + 8192, T))
        x = s["x"][r].double().requires_grad_(True)
        ga_, be_ = ga.clone().requires_grad_(True), be.clone().requires_grad_(True)
        mu = x.sum(1) / d
        var = ((x - mu[:, None]) ** 2).sum(1) / d
        rs = (var + EPS) ** -0.5
        y = ga_ * (x - mu[:, None]) * rs[:, None] + be_
        out["y"][r], out["mean"][r], out["rstd"][r] = y.detach(), mu.detach(), rs.detach()
        if c["train"]:
            dx, dg, db = torch.autograd.grad((y * s["dy"][r].double()).sum(), (x, ga_, be_))
            out["dx"][r] = dx + (s["dres"][r].double() if s["dres"] is not None else 0.0)
            out["dgamma"] += dg
            out["dbeta"] += db
    return out
