"""Host-side tests of the layer norm and 8-bit checkpoint entry points (no GPU): invalid
arguments return their status code before anything is launched, workspace sizes, and the
binding's own refusals."""
import ctypes
import math

import pytest
import torch

import deformable_convolution_dcn1d_b200 as dcn
from test_abi_host import FAKE, T

F32, BF16, F16, I8, U8 = 0, 1, 2, 3, 4
B, C, L = 2, 6, 40


def r(t):
    return None if t is None else ctypes.byref(t)


def run(name, a, order):
    lib = dcn.load()
    args = [r(a[k]) if isinstance(a[k], (dcn.Dcn1dTensor, type(None))) else a[k] for k in order]
    return getattr(lib, name)(*args)


def norm_args(**over):
    a = dict(x=T((B, C, L), BF16), gamma=T((C,), BF16), beta=T((C,), BF16), eps=1e-5,
             y=T((B, C, L), BF16, 2 * FAKE), mean=T((B, L)), rstd=T((B, L)), codes=T((B, C, L), I8),
             scales=T((B, C, 2), U8), stream=None)
    a.update(over)
    return a


NORM = ["x", "gamma", "beta", "eps", "y", "mean", "rstd", "codes", "scales", "stream"]

BAD_NORM = [
    ("null x", dict(x=None), 1),
    ("null y", dict(y=None), 1),
    ("null x data", dict(x=T((B, C, L), BF16, data=None)), 1),
    ("codes without scales", dict(scales=None), 1),
    ("scales without codes", dict(codes=None), 1),
    ("integer x", dict(x=T((B, C, L), I8)), 2),
    ("y of another type", dict(y=T((B, C, L), F32)), 2),
    ("gamma of another type", dict(gamma=T((C,), F32)), 2),
    ("mean not fp32", dict(mean=T((B, L), BF16)), 2),
    ("codes not int8", dict(codes=T((B, C, L), U8)), 2),
    ("scales not uint8", dict(scales=T((B, C, 2), I8)), 2),
    ("x of two dimensions", dict(x=T((B, C), BF16)), 3),
    ("no channels", dict(x=T((B, 0, L), BF16), y=T((B, 0, L), BF16)), 3),
    ("negative length", dict(x=T((B, C, -1), BF16)), 3),
    ("y shape", dict(y=T((B, C, L + 1), BF16)), 3),
    ("gamma shape", dict(gamma=T((C + 1,), BF16)), 3),
    ("beta shape", dict(beta=T((L,), BF16)), 3),
    ("rstd shape", dict(rstd=T((L, B))), 3),
    ("scales shape", dict(scales=T((B, C, 1), U8)), 3),
    ("codes shape", dict(codes=T((B, L, C), I8)), 3),
    ("negative eps", dict(eps=-1e-5), 4),
    ("NaN eps", dict(eps=math.nan), 4),
    ("infinite eps", dict(eps=math.inf), 4),
    ("y in x's place", dict(x=T((B, C, L), BF16, FAKE + 64), y=T((B, C, L), BF16, FAKE + 64)), 4),
    ("too many positions", dict(x=T((1 << 16, 1, 1 << 16), BF16)), 5),
    ("too many channels", dict(x=T((1, 1 << 31, 1), BF16)), 5),
]


@pytest.mark.parametrize("name,over,code", BAD_NORM, ids=[b[0] for b in BAD_NORM])
def test_norm_forward_refusals(name, over, code):
    assert run("dcn1d_layer_norm_forward", norm_args(**over), NORM) == code
    assert dcn.dcn1d_last_launch_count() == 0


def test_single_token_checkpoints_have_blocks_along_the_channels():
    one = dict(x=T((B, 70, 1), BF16), y=T((B, 70, 1), BF16), gamma=None, beta=None,
               mean=None, rstd=None, codes=T((B, 70, 1), I8))
    assert run("dcn1d_layer_norm_forward", norm_args(**one, scales=T((B, 70, 1), U8)), NORM) == 3
    empty = dict(one, x=T((0, 70, 1), BF16, data=None), y=T((0, 70, 1), BF16, data=None),
                 codes=T((0, 70, 1), I8, data=None), scales=T((0, 3, 1), U8, data=None))
    assert run("dcn1d_layer_norm_forward", norm_args(**empty), NORM) == 0
    assert dcn.dcn1d_last_launch_count() == 0


def grad_args(**over):
    a = dict(x=T((B, C, L), BF16, 2 * FAKE), gamma=T((C,), BF16), mean=T((B, L)), rstd=T((B, L)),
             codes=None, scales=None, gy=T((B, C, L), BF16, 3 * FAKE), gx=T((B, C, L), BF16),
             ggamma=T((C,), BF16), gbeta=T((C,), BF16), ws=None, bytes=0, stream=None)
    a.update(over)
    return a


GRAD = ["x", "gamma", "mean", "rstd", "codes", "scales", "gy", "gx", "ggamma", "gbeta"]
KEPT = dict(x=None, mean=None, codes=T((B, C, L), I8), scales=T((B, C, 2), U8))

BAD_GRAD = [
    ("no values at all", dict(x=None, mean=None), 1),
    ("x without mean", dict(mean=None), 1),
    ("no rstd", dict(rstd=None), 1),
    ("no grad_y", dict(gy=None), 1),
    ("codes alone", dict(KEPT, scales=None), 1),
    ("both x and a checkpoint", dict(codes=T((B, C, L), I8), scales=T((B, C, 2), U8)), 4),
    ("a checkpoint and a mean", dict(KEPT, mean=T((B, L))), 4),
    ("grad_x in grad_y's place", dict(gy=T((B, C, L), BF16, FAKE)), 4),
    ("grad_x in x's place", dict(x=T((B, C, L), BF16, FAKE)), 4),
    ("x of another type", dict(x=T((B, C, L), F16)), 2),
    ("grad_x of another type", dict(gx=T((B, C, L), F32)), 2),
    ("rstd of 16 bits", dict(rstd=T((B, L), BF16)), 2),
    ("x shape", dict(x=T((B, C, L - 1), BF16)), 3),
    ("grad_gamma shape", dict(ggamma=T((L,), BF16)), 3),
    ("scales shape", dict(KEPT, scales=T((B, 2, C), U8)), 3),
    ("too many positions", dict(gy=T((1 << 16, 1, 1 << 16), BF16)), 5),
]


@pytest.mark.parametrize("name,over,code", BAD_GRAD, ids=[b[0] for b in BAD_GRAD])
def test_norm_backward_refusals(name, over, code):
    a = grad_args(**over)
    assert run("dcn1d_layer_norm_backward_workspace_size", a, GRAD) == -code
    a.update(ws=FAKE, bytes=1 << 40)
    assert run("dcn1d_layer_norm_backward", a, GRAD + ["ws", "bytes", "stream"]) == code
    assert dcn.dcn1d_last_launch_count() == 0


@pytest.mark.parametrize("kept", [False, True])
def test_norm_backward_workspace(kept):
    a = grad_args(**(KEPT if kept else {}))
    need = run("dcn1d_layer_norm_backward_workspace_size", a, GRAD)
    assert need >= 2 * C * 4
    full = GRAD + ["ws", "bytes", "stream"]
    assert run("dcn1d_layer_norm_backward", dict(a, ws=None, bytes=0), full) == 1
    assert run("dcn1d_layer_norm_backward", dict(a, ws=FAKE, bytes=need - 1), full) == 4
    assert run("dcn1d_layer_norm_backward", dict(a, ws=FAKE + 16, bytes=need + 256), full) == 4
    only_x = dict(a, ggamma=None, gbeta=None)
    assert run("dcn1d_layer_norm_backward_workspace_size", only_x, GRAD) == 0


def ck_args(**over):
    a = dict(x=T((B, C, L), F16), codes=T((B, C, L), I8), scales=T((B, C, 2), U8), gamma=None,
             beta=None, out=T((B, C, L), F16), stream=None)
    a.update(over)
    return a


BAD_CK = [
    ("null codes", dict(codes=None), 1),
    ("null scales", dict(scales=None), 1),
    ("null scales data", dict(scales=T((B, C, 2), U8, data=None)), 1),
    ("codes type", dict(codes=T((B, C, L), F32)), 2),
    ("codes shape", dict(codes=T((B, C, L + 1), I8)), 3),
    ("scales shape", dict(scales=T((B, C, 3), U8)), 3),
    ("scales of two dimensions", dict(scales=T((B * C, 2), U8)), 3),
]


@pytest.mark.parametrize("name,over,code", BAD_CK, ids=[b[0] for b in BAD_CK])
def test_checkpoint_refusals(name, over, code):
    a = ck_args(**over)
    assert run("dcn1d_checkpoint_pack", a, ["x", "codes", "scales", "stream"]) == code
    assert run("dcn1d_checkpoint_unpack", a,
               ["codes", "scales", "gamma", "beta", "out", "stream"]) == code
    assert dcn.dcn1d_last_launch_count() == 0


def test_unpack_refuses_weights_of_another_type_or_size():
    order = ["codes", "scales", "gamma", "beta", "out", "stream"]
    assert run("dcn1d_checkpoint_unpack", ck_args(gamma=T((C,), F32)), order) == 2
    assert run("dcn1d_checkpoint_unpack", ck_args(beta=T((C + 1,), F16)), order) == 3
    assert run("dcn1d_checkpoint_unpack", ck_args(out=T((B, C, L), I8)), order) == 2


def conv_args(**over):
    K, og = 3, 2
    a = dict(codes=T((B, C, L), I8), scales=T((B, C, 2), U8), gamma=T((C,), BF16),
             beta=T((C,), BF16), off=T((B, og, L, K), BF16), mask=None, w=T((C, C, K), BF16),
             gout=T((B, C, L), BF16), stride=1, pl=1, pr=1, dilation=1, groups=1, og=og, unc=0,
             gx=T((B, C, L), BF16), goff=T((B, og, L, K), BF16), gmask=None,
             gw=T((C, C, K), BF16), gb=T((C,), BF16), ws=None, bytes=0, stream=None)
    a.update(over)
    return a


CONV = ["codes", "scales", "gamma", "beta", "off", "mask", "w", "gout", "stride", "pl", "pr",
        "dilation", "groups", "og", "unc", "gx", "goff", "gmask", "gw", "gb"]

BAD_CONV = [
    ("null codes", dict(codes=None), 1),
    ("null scales", dict(scales=None), 1),
    ("null grad_out", dict(gout=None), 1),
    ("codes type", dict(codes=T((B, C, L), BF16)), 2),
    ("gamma type", dict(gamma=T((C,), F32)), 2),
    ("weight type", dict(w=T((C, C, 3), F32)), 2),
    ("codes of two dimensions", dict(codes=T((B, C * L), I8)), 3),
    ("scales shape", dict(scales=T((B, C, 1), U8)), 3),
    ("beta shape", dict(beta=T((C - 1,), BF16)), 3),
    ("grad_out length", dict(gout=T((B, C, L - 1), BF16)), 3),
    ("mask gradient without a mask", dict(gmask=T((B, 2, L, 3), BF16)), 4),
    ("stride 0", dict(stride=0), 4),
]


@pytest.mark.parametrize("name,over,code", BAD_CONV, ids=[b[0] for b in BAD_CONV])
def test_backward_checkpoint_refusals(name, over, code):
    a = conv_args(**over)
    assert run("dcn1d_backward_checkpoint_workspace_size", a, CONV) == -code
    a.update(ws=FAKE, bytes=1 << 40)
    assert run("dcn1d_backward_checkpoint", a, CONV + ["ws", "bytes", "stream"]) == code
    assert dcn.dcn1d_last_launch_count() == 0


def test_backward_checkpoint_workspace():
    a = conv_args()
    need = run("dcn1d_backward_checkpoint_workspace_size", a, CONV)
    assert need > 0
    full = CONV + ["ws", "bytes", "stream"]
    assert run("dcn1d_backward_checkpoint", a, full) == 1
    assert run("dcn1d_backward_checkpoint", dict(a, ws=FAKE, bytes=need - 1), full) == 4
    assert run("dcn1d_backward_checkpoint", dict(a, ws=FAKE + 1, bytes=need + 256), full) == 4


def test_binding_refuses_host_tensors_and_unknown_gradients():
    x = torch.zeros(1, 4, 8)
    s = torch.zeros(1, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dcn.dcn1d_layer_norm_forward(x)
    with pytest.raises(ValueError, match="CUDA"):
        dcn.dcn1d_checkpoint_pack(x)
    with pytest.raises(ValueError, match="unknown gradients"):
        dcn.dcn1d_layer_norm_backward(x, None, s, s, x, wanted=("x", "weight"))
    with pytest.raises(ValueError, match="unknown gradients"):
        dcn.dcn1d_backward_checkpoint((x, x), x, None, x, x, wanted=("gamma",))


def test_batches_past_the_gemm_grid_are_the_fused_depthwise_kernels_only():
    b, c, l = 70, 1000, 8
    a = dict(codes=T((b, c, l), I8), scales=T((b, c, 1), U8), gamma=None, beta=None,
             off=T((b, c, l, 3), BF16), w=T((c, 1, 3), BF16), gout=T((b, c, l), BF16), groups=c,
             og=c, gx=T((b, c, l), BF16), goff=T((b, c, l, 3), BF16), gw=T((c, 1, 3), BF16),
             gb=T((c,), BF16))
    assert run("dcn1d_backward_checkpoint_workspace_size", conv_args(**a), CONV) > 0
    shared = dict(a, og=500, off=T((b, 500, l, 3), BF16), goff=T((b, 500, l, 3), BF16))
    assert run("dcn1d_backward_checkpoint_workspace_size", conv_args(**shared), CONV) == -5
