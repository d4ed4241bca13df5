"""Layer norm over the channels of [B, C, L], 8-bit activation checkpoints, and the backward passes
that read them: the cases that are timed, their plain forms in elementary torch operations, and
the calls a user makes of this package for the same work.

The 8-bit checkpoint of a tensor [B, C, L]: blocks of 32 values along the row (the L positions of
a channel; the C channels when L is 1), int8 codes, and one byte s a block that holds the biased
exponent of the block's step 2^(s - 127).  The step is the smallest power of two at which the
block's largest magnitude still rounds to a code of at most 127.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


# ---------------------------------------------------------------- the cases

def _norm(name, op, dtype, B, C, L):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "C": C, "L": L}


def listed():
    return [
        # one token through the norm in front of a layer of 512 channels: latency
        _norm("norm_token_bf16", "norm", "bf16", 1, 512, 1),
        # the input of the fp32 usage layer (16 x 512 channels, length 128)
        _norm("norm_usage_f32", "norm", "f32", 16, 512, 128),
        # the input of the depthwise layer: 65.5 million values
        _norm("norm_depthwise_bf16", "norm", "bf16", 8, 512, 16000),
        # gradients at the usage layer's output length, an odd one, from the fp32 input
        _norm("norm_grad_usage_f32", "norm_grad", "f32", 16, 512, 83),
        # gradients of the modulated layer's norm from its 8-bit checkpoint
        _norm("norm_grad_modulated_bf16", "norm_grad_checkpoint", "bf16", 16, 256, 4096),
        # the same at the large layer's input: 268 million values
        _norm("norm_grad_large_bf16", "norm_grad_checkpoint", "bf16", 32, 1024, 8192),
        # a training step's norm: forward that keeps 8 bits a value, then the backward
        _norm("norm_train_depthwise_bf16", "norm_train", "bf16", 8, 512, 16000),
        # the same in fp16 at odd sizes
        _norm("norm_train_odd_f16", "norm_train", "f16", 3, 381, 1001),
        # an activation kept in 8 bits and read back
        _norm("checkpoint_modulated_bf16", "checkpoint", "bf16", 16, 256, 4096),
        _norm("checkpoint_odd_f32", "checkpoint", "f32", 5, 333, 1601),
        # the depthwise layer's backward from the checkpoint of its input
        {"name": "conv_grad_depthwise_bf16", "op": "conv_grad", "dtype": "bf16", "B": 8, "C": 512,
         "L": 16000, "C_out": 512, "K": 3, "stride": 1, "padding": 64, "dilation": 64,
         "groups": 512, "offset_groups": 512, "unconstrained": True, "mask": False,
         "affine": False, "spread": 4.0},
        # the modulated layer's backward; its input is the norm's output, rebuilt from the
        # checkpoint of the normalised values
        {"name": "conv_grad_modulated_bf16", "op": "conv_grad", "dtype": "bf16", "B": 16, "C": 256,
         "L": 4096, "C_out": 256, "K": 5, "stride": 1, "padding": 2, "dilation": 1, "groups": 1,
         "offset_groups": 8, "unconstrained": False, "mask": True, "affine": True, "spread": 1.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm_grad_checkpoint", "norm_train", "checkpoint",
                     "conv_grad", "conv_grad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "norm_train" and dtype == "f32":
        dtype = "bf16"
    B = _log_int(rng, 1, 32)
    if op != "conv_grad":
        C = _log_int(rng, 48, 1024)
        L = _log_int(rng, 1, 16384)
        if rng.random() < 0.5:
            L = max(8, L // 8 * 8)
        while B * C * L > 1 << 26:
            L = max(1, L // 2)
        return {"op": op, "dtype": dtype, "B": B, "C": C, "L": L}
    K = rng.randint(2, 6)
    dilation = rng.choice([1, 2, 7, 64])
    stride = rng.choice([1, 1, 2])
    mask = rng.random() < 0.5
    unconstrained = rng.random() < 0.5
    padding = dilation * (K - 1) // 2
    if rng.random() < 0.6:      # depthwise, offsets of each channel's own
        C = C_out = groups = offset_groups = _log_int(rng, 16, 512)
        L = _log_int(rng, 64, 16000)
    else:
        groups = rng.choice([1, 2])
        offset_groups = rng.choice([1, 2, 4])
        C = 16 * rng.randint(1, 16)
        C_out = 16 * rng.randint(1, 16)
        L = _log_int(rng, 64, 2048)
    if rng.random() < 0.5:
        L = max(64, L // 8 * 8)
    while B * C * L * K > 1 << 26 and B > 1:
        B = B // 2
    return {"op": op, "dtype": dtype, "B": B, "C": C, "L": L, "C_out": C_out, "K": K,
            "stride": stride, "padding": padding, "dilation": dilation, "groups": groups,
            "offset_groups": offset_groups, "unconstrained": unconstrained, "mask": mask,
            "affine": rng.random() < 0.5, "spread": round(rng.uniform(0.5, 4.0), 2)}


def _l_out(case):
    return (case["L"] + 2 * case["padding"] - case["dilation"] * (case["K"] - 1) - 1) \
        // case["stride"] + 1


def work(case):
    e = SIZE[case["dtype"]]
    n, tokens = case["B"] * case["C"] * case["L"], case["B"] * case["L"]
    packed = n + n / BLOCK
    weights = 2 * case["C"] * e
    op = case["op"]
    if op == "norm":
        return {"bytes": 2 * n * e + 8 * tokens + weights, "flops": 9 * n}
    if op == "norm_grad":
        return {"bytes": 3 * n * e + 8 * tokens + 1.5 * weights, "flops": 14 * n}
    if op == "norm_grad_checkpoint":
        return {"bytes": 2 * n * e + packed + 4 * tokens + 1.5 * weights, "flops": 13 * n}
    if op == "norm_train":
        return {"bytes": 4 * n * e + 8 * tokens + 2.5 * weights, "flops": 25 * n}
    if op == "checkpoint":
        return {"bytes": 2 * n * e, "flops": 4 * n}
    Lo, K = _l_out(case), case["K"]
    taps = case["B"] * case["offset_groups"] * Lo * K
    w = case["C_out"] * case["C"] // case["groups"] * K
    heads = 2 if case["mask"] else 1
    moved = packed + n * e + 2 * heads * taps * e + case["B"] * case["C_out"] * Lo * e \
        + 2 * w * e + case["C_out"] * e
    cols = case["B"] * case["C"] * Lo * K
    return {"bytes": moved, "flops": 4 * cols * (case["C_out"] // case["groups"]) + 12 * cols}


# ---------------------------------------------------------------- inputs

def _pack_plain(x):
    """(codes, scales) of x [B, C, L] by the rule of this file's first lines."""
    top = 142 if x.dtype == torch.float16 else 254      # no step past the type's largest value
    rows = x.float().transpose(1, 2) if x.shape[2] == 1 else x.float()
    n = rows.shape[2]
    pad = -n % BLOCK
    blocks = torch.nn.functional.pad(rows, (0, pad)).unflatten(2, (-1, BLOCK))
    bits = blocks.abs().amax(3).view(torch.int32)
    s = (((bits + 0x10000) >> 23).clamp(max=top) - 6).clamp(min=1)
    inverse = ((254 - s) << 23).view(torch.float32)
    codes = (blocks * inverse[..., None]).round().clamp(-127, 127)
    bad = bits >= 0x7F800000
    codes = torch.where(bad[..., None], 0.0, codes).to(torch.int8).flatten(2)[:, :, :n]
    scales = torch.where(bad, 255, s).to(torch.uint8)
    if x.shape[2] == 1:
        codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
    return codes.contiguous(), scales.contiguous()


def _steps(scales, shape, dtype):
    """The step of every value of a checkpoint of `shape`."""
    axis = 1 if shape[2] == 1 else 2
    s = scales.to(torch.int32)
    step = torch.where(s == 255, math.nan, (s << 23).view(torch.float32)).to(dtype)
    return step.repeat_interleave(BLOCK, axis).narrow(axis, 0, shape[axis])


def _values(codes, scales):
    """What a checkpoint stands for, in float32."""
    return codes.float() * _steps(scales, codes.shape, torch.float32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = TYPES[case["dtype"]]
    B, C, L = case["B"], case["C"], case["L"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    state = {"case": case}
    op = case["op"]
    # activations: channels of different scale and offset, as a trained layer's output has
    spread = torch.exp(0.5 * randn(1, C, 1))
    x = (randn(B, C, L) * spread + 0.5 * randn(1, C, 1)).to(T)
    gamma = (1 + 0.1 * randn(C)).to(T)
    beta = (0.1 * randn(C)).to(T)
    if op == "checkpoint":
        return {**state, "x": x}
    if op in ("norm", "norm_train", "norm_grad"):
        state.update(x=x)
    if op in ("norm", "norm_train", "norm_grad", "norm_grad_checkpoint"):
        state.update(gamma=gamma)
    if op in ("norm", "norm_train"):
        state.update(beta=beta)
    if op != "norm" and op != "conv_grad":
        state.update(gy=randn(B, C, L).to(T))
    if op in ("norm_grad", "norm_grad_checkpoint"):
        mean = x.float().mean(1)
        var = (x.float() - mean[:, None]).square().mean(1)
        rstd = 1 / (var + EPS).sqrt()
        state.update(mean=mean, rstd=rstd)
    if op == "norm_grad_checkpoint":
        v = (x.float() - mean[:, None]) * rstd[:, None]
        state["codes"], state["scales"] = _pack_plain(v)
        state.pop("mean")
    if op == "conv_grad":
        K, G, Lo = case["K"], case["offset_groups"], _l_out(case)
        state["codes"], state["scales"] = _pack_plain(x)
        state["gamma"], state["beta"] = (gamma, beta) if case["affine"] else (None, None)
        state["offsets"] = (randn(B, G, Lo, K) * case["spread"]).to(T)
        state["mask"] = torch.sigmoid(randn(B, G, Lo, K)).to(T) if case["mask"] else None
        fan = C // case["groups"] * K
        state["weight"] = (randn(case["C_out"], C // case["groups"], K) / math.sqrt(fan)).to(T)
        state["gout"] = randn(B, case["C_out"], Lo).to(T)
    return state


# ---------------------------------------------------------------- plain forms

def _norm_plain(x, gamma, beta):
    """y, mean, rstd and the normalised values."""
    x32 = x.float()
    mean = x32.mean(1)
    d = x32 - mean[:, None]
    rstd = 1 / (d.square().mean(1) + EPS).sqrt()
    v = d * rstd[:, None]
    y = v * gamma.float()[:, None] + beta.float()[:, None]
    return y.to(x.dtype), mean, rstd, v


def _norm_grad_plain(v, rstd, gamma, gy):
    g32 = gy.float()
    d = g32 * gamma.float()[:, None]
    gx = rstd[:, None] * (d - d.mean(1, keepdim=True) - v * (d * v).mean(1, keepdim=True))
    return {"x": gx.to(gy.dtype), "gamma": (g32 * v).sum((0, 2)).to(gy.dtype),
            "beta": g32.sum((0, 2)).to(gy.dtype)}


def _conv_input(state, values):
    """The convolution's input: the checkpoint's values, through the norm's weights if it has
    them, rounded to the layer's type as the forward's input was."""
    if state["gamma"] is not None:
        values = values * state["gamma"].to(values.dtype)[:, None] \
            + state["beta"].to(values.dtype)[:, None]
    return values.to(state["gout"].dtype)


def _positions(case, offsets):
    """fp32 tap positions [B, G, L_out, K] before any clamp, and each tap's receptive field."""
    Lo, K = offsets.shape[2:]
    start = torch.arange(Lo, device=offsets.device) * case["stride"] - case["padding"]
    base = start[:, None] + torch.arange(K, device=offsets.device) * case["dilation"]
    first = start.float()[:, None]
    return base.float() + offsets.float(), first, first + float(case["dilation"] * (K - 1))


def _conv_grad_plain(state):
    case = state["case"]
    B, C, L, G = case["B"], case["C"], case["L"], case["offset_groups"]
    K, Lo, groups = case["K"], _l_out(case), case["groups"]
    T = state["gout"].dtype
    x = _conv_input(state, _values(state["codes"], state["scales"])).float()
    raw, lo, hi = _positions(case, state["offsets"])
    pos = raw if case["unconstrained"] else torch.minimum(torch.maximum(raw, lo), hi)
    i0 = pos.floor()
    f = (pos - i0)[:, :, None]                                   # [B, G, 1, Lo, K]
    m = state["mask"].float()[:, :, None] if case["mask"] else torch.ones_like(f)
    per = C // G
    xg = x.view(B, G, per, L)

    def at(i):
        """(index, whether inside) of integer positions, for every channel of the group."""
        inside = ((i >= 0) & (i <= L - 1))[:, :, None]
        index = i.clamp(0, L - 1).long()[:, :, None].expand(B, G, per, Lo, K).reshape(B, G, per, -1)
        return index, inside

    at0, in0 = at(i0)
    at1, in1 = at(i0 + 1)
    x0 = xg.gather(3, at0).view(B, G, per, Lo, K) * in0
    x1 = xg.gather(3, at1).view(B, G, per, Lo, K) * in1
    v = (1 - f) * x0 + f * x1
    w = state["weight"].float().view(groups, -1, C // groups, K)
    go = state["gout"].float().view(B, groups, -1, Lo)
    dv = torch.einsum("gock,bgol->bgclk", w, go).reshape(B, G, per, Lo, K)
    cols = (m * v).reshape(B, groups, C // groups, Lo, K)
    grads = {"weight": torch.einsum("bgol,bgclk->gock", go, cols).reshape(state["weight"].shape),
             "bias": go.sum((0, 3)).flatten()}
    gx = torch.zeros(B, G, per, L, device=x.device)
    gx.scatter_add_(3, at0, (m * (1 - f) * dv * in0).reshape(B, G, per, -1))
    gx.scatter_add_(3, at1, (m * f * dv * in1).reshape(B, G, per, -1))
    grads["x"] = gx.view(B, C, L)
    goff = (m * (x1 - x0) * dv).sum(2)
    if not case["unconstrained"]:
        goff = goff * ((raw >= lo) & (raw <= hi))
    grads["offsets"] = goff
    if case["mask"]:
        grads["mask"] = (v * dv).sum(2)
    return {k: t.to(T) for k, t in grads.items()}


# ---------------------------------------------------------------- one pass

def _run_own(state):
    import deformable_convolution_dcn1d_b200 as dcn
    case = state["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd, _ = dcn.dcn1d_layer_norm_forward(state["x"], state["gamma"], state["beta"],
                                                        EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        return dcn.dcn1d_layer_norm_backward(state["x"], state["gamma"], state["mean"],
                                             state["rstd"], state["gy"])
    if op == "norm_grad_checkpoint":
        kept = dcn.Checkpoint8(state["codes"], state["scales"])
        return dcn.dcn1d_layer_norm_backward(kept, state["gamma"], None, state["rstd"],
                                             state["gy"])
    if op == "norm_train":
        y, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(state["x"], state["gamma"],
                                                           state["beta"], EPS, checkpoint=True)
        grads = dcn.dcn1d_layer_norm_backward(kept, state["gamma"], None, rstd, state["gy"])
        return {"y": y, "mean": mean, "rstd": rstd, **grads}
    if op == "checkpoint":
        kept = dcn.dcn1d_checkpoint_pack(state["x"])
        return dcn.dcn1d_checkpoint_unpack(kept, dtype=state["x"].dtype)
    kept = dcn.Checkpoint8(state["codes"], state["scales"])
    return dcn.dcn1d_backward_checkpoint(kept, state["offsets"], state["mask"], state["weight"],
                                         state["gout"], case["stride"], case["padding"],
                                         case["dilation"], case["groups"], case["offset_groups"],
                                         case["unconstrained"], gamma=state["gamma"],
                                         beta=state["beta"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        y, mean, rstd, _ = _norm_plain(state["x"], state["gamma"], state["beta"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        v = (state["x"].float() - state["mean"][:, None]) * state["rstd"][:, None]
        return _norm_grad_plain(v, state["rstd"], state["gamma"], state["gy"])
    if op == "norm_grad_checkpoint":
        return _norm_grad_plain(_values(state["codes"], state["scales"]), state["rstd"],
                                state["gamma"], state["gy"])
    if op == "norm_train":
        y, mean, rstd, v = _norm_plain(state["x"], state["gamma"], state["beta"])
        kept = _values(*_pack_plain(v))
        return {"y": y, "mean": mean, "rstd": rstd,
                **_norm_grad_plain(kept, rstd, state["gamma"], state["gy"])}
    if op == "checkpoint":
        return _values(*_pack_plain(state["x"])).to(state["x"].dtype)
    return _conv_grad_plain(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _two_to(e):
    """2^e in 64 bits, exactly, for whole e (a library's power may be off in the last bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _kept_exact(v, largest_exponent):
    """The values that the checkpoint of v (64 bits) stands for."""
    rows = v.transpose(1, 2) if v.shape[2] == 1 else v
    out = torch.empty_like(rows)
    n = rows.shape[2]
    for at in range(0, n, BLOCK):           # block by block along the row
        part = rows[:, :, at:at + BLOCK]
        top = part.abs().amax(2, keepdim=True)
        # the smallest e with rne(top / 2^e) <= 127, at least -126
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -200))) - 6
        e = torch.where(torch.round(top / _two_to(e)) > 127, e + 1, e)
        step = _two_to(e.clamp(-126, largest_exponent))
        out[:, :, at:at + BLOCK] = torch.round(part / step).clamp(-127, 127) * step
    return out.transpose(1, 2) if v.shape[2] == 1 else out


def _norm_exact(x, gamma, beta):
    mean = x.mean(1, keepdim=True)
    rstd = ((x * x).mean(1, keepdim=True) - mean * mean + EPS) ** -0.5
    v = (x - mean) * rstd
    return gamma[:, None] * v + beta[:, None], mean[:, 0], rstd[:, 0], v


def _norm_grad_exact(v, rstd, gamma, gy):
    C = v.shape[1]
    first = torch.einsum("bcl,c->bl", gy, gamma) / C
    second = torch.einsum("bcl,bcl,c->bl", gy, v, gamma) / C
    gx = gy * gamma[:, None]
    gx = (gx - first[:, None] - v * second[:, None]) * rstd[:, None]
    return {"x": gx, "gamma": torch.einsum("bcl,bcl->c", gy, v), "beta": gy.sum(2).sum(0)}


def _conv_exact(state):
    """By differentiating the forward, written out in 64 bits with positions in fp32."""
    case = state["case"]
    B, C, L, G = case["B"], case["C"], case["L"], case["offset_groups"]
    K, Lo, groups = case["K"], _l_out(case), case["groups"]
    step = _steps(state["scales"], state["codes"].shape, torch.float64)
    x = _conv_input(state, state["codes"].double() * step).double().requires_grad_()
    off = state["offsets"].double().requires_grad_()
    w = state["weight"].double().requires_grad_()
    mask = state["mask"].double().requires_grad_() if case["mask"] else None
    raw, lo, hi = _positions(case, state["offsets"])
    pos = raw.double() + (off - off.detach())
    if not case["unconstrained"]:
        pos = torch.clamp(pos, lo.double().expand_as(pos), hi.double().expand_as(pos))
    cell = pos.detach().floor()
    frac = pos - cell
    # the signal between zeros: cell -1 and cell L are the first and last zero
    line = torch.nn.functional.pad(x, (2, 2)).view(B, G, C // G, L + 4)
    index = (cell.clamp(-2, L) + 2).long()[:, :, None].expand(B, G, C // G, Lo, K).flatten(3)
    left = line.gather(3, index).view(B, G, C // G, Lo, K)
    right = line.gather(3, index + 1).view(B, G, C // G, Lo, K)
    cols = torch.lerp(left, right, frac[:, :, None].expand_as(left))
    if mask is not None:
        cols = cols * mask[:, :, None]
    cols = cols.reshape(B, groups, C // groups, Lo, K)
    go = state["gout"].double().view(B, groups, -1, Lo)
    total = (torch.einsum("bgclk,gock->bgol", cols, w.view(groups, -1, C // groups, K)) * go).sum()
    names = ["x", "offsets", "weight"] + (["mask"] if case["mask"] else [])
    leaves = [x, off, w] + ([mask] if case["mask"] else [])
    grads = dict(zip(names, torch.autograd.grad(total, leaves)))
    grads["bias"] = go.sum((0, 3)).flatten()
    return grads


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "conv_grad":
        return _conv_exact(state)
    if op == "checkpoint":
        return _kept_exact(state["x"].double(), 9 if case["dtype"] == "f16" else 121)
    if op == "norm_grad_checkpoint":
        v = state["codes"].double() * _steps(state["scales"], state["codes"].shape, torch.float64)
        return _norm_grad_exact(v, state["rstd"].double(), state["gamma"].double(),
                                state["gy"].double())
    x, gamma = state["x"].double(), state["gamma"].double()
    if op == "norm_grad":
        rstd = state["rstd"].double()
        v = (x - state["mean"].double()[:, None]) * rstd[:, None]
        return _norm_grad_exact(v, rstd, gamma, state["gy"].double())
    y, mean, rstd, v = _norm_exact(x, gamma, state["beta"].double())
    out = {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_train":
        out.update(_norm_grad_exact(_kept_exact(v, 121), rstd, gamma, state["gy"].double()))
    return out
