"""The depthwise layer's backward pass from a checkpoint (GPU), element by element against the
64-bit form and the bounds of depthwise_ref.py: rows of one position, what lies past the end of
a row, and gradients of very different size in one row."""
import pytest
import torch

import depthwise_ref as D
import deformable_convolution_dcn1d_b200 as dcn

pytestmark = pytest.mark.gpu

TOL = {"torch.float32": 1e-5, "torch.bfloat16": 2e-2, "torch.float16": 5e-3}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(T, B, C, L, K, stride=1, padding=0, dilation=1, mask=True, seed=1, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    Lo = (L + 2 * padding - dilation * (K - 1) - 1) // stride + 1

    def randn(*shape):
        return torch.randn(*shape, generator=g)
    t = {"x": randn(B, C, L) * torch.exp(randn(1, C, 1)), "off": randn(B, C, Lo, K) * spread,
         "mask": torch.sigmoid(randn(B, C, Lo, K)) if mask else None, "w": randn(C, 1, K),
         "gout": randn(B, C, Lo)}
    return {k: None if v is None else v.to(T).cuda() for k, v in t.items()}


def run(t, stride, padding, dilation, unconstrained, gamma=None, beta=None, kept=None, **k):
    C = t["w"].shape[0]
    kept = dcn.dcn1d_checkpoint_pack(t["x"]) if kept is None else kept
    got = dcn.dcn1d_backward_checkpoint(kept, t["off"], t["mask"], t["w"], t["gout"], stride, padding,
                                        dilation, C, C, unconstrained, gamma=gamma, beta=beta, **k)
    return kept, got


def check(t, stride=1, padding=0, dilation=1, unconstrained=True, gamma=None, beta=None):
    kept, got = run(t, stride, padding, dilation, unconstrained, gamma, beta)
    x = dcn.dcn1d_checkpoint_unpack(kept, gamma, beta, dtype=t["gout"].dtype)
    ref, bound, _ = D.backward(x, t["off"], t["mask"], t["w"], t["gout"], stride, padding, dilation,
                               unconstrained)
    assert set(got) == set(ref)
    for n, g in got.items():
        assert g.shape == ref[n].shape and g.dtype == t["gout"].dtype
        assert torch.equal(g.isfinite(), ref[n].isfinite()), n
        ok = ref[n].isfinite()
        err = (g.double() - ref[n]).abs()
        room = bound[n]
        if n == "x":   # one fixed-point unit serves a row: compared with the tensor's largest
            room = TOL[str(g.dtype)] * ref[n][ok].abs().max()
        bad = ok & ~(err <= room)
        assert not bad.any(), (n, int(bad.sum()), (err / room)[bad].max().item())
    return got


@pytest.mark.parametrize("affine", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("mask", [False, True], ids=["", "mask"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("B,C,K,padding,dilation", [(3, 70, 3, 1, 1), (2, 32, 3, 2, 2), (1, 1, 1, 0, 1),
                                                    (4, 513, 5, 4, 2)])
def test_rows_of_one_position(B, C, K, padding, dilation, dt, mask, affine):
    """L = 1: the checkpoint's blocks run along the channels, a channel's step is its block's."""
    T = TYPES[dt]
    t = make(T, B, C, 1, K, 1, padding, dilation, mask)
    gamma, beta = (t["x"][0, :, 0] * 0.5 + 1, t["x"][-1, :, 0] * 0.25) if affine else (None, None)
    check(t, 1, padding, dilation, True, gamma, beta)
    check(t, 1, padding, dilation, False, gamma, beta)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("L,K,dilation,stride", [(140, 2, 64, 1), (333, 3, 64, 1), (640, 2, 64, 2)])
def test_bad_values_past_the_last_output(L, K, dilation, stride, dt, bad):
    """Lanes past the end of a row touch nothing: neither a marked block of x that only they
    would reach, nor sites of grad_x from a bad mask at the last position or a bad weight."""
    T = TYPES[dt]
    t = make(T, 2, 3, L, K, stride, 0, dilation, mask=True)
    t["off"].zero_()
    Lo = t["off"].shape[2]
    # x behind what tap 0 of the last output reads is marked, from the next block on
    after = ((Lo - 1) * stride // 32 + 1) * 32
    t["x"][0, 0, after:] = bad
    check(t, stride, 0, dilation)
    t = make(T, 2, 3, L, K, stride, 0, dilation, mask=True)
    t["off"].zero_()
    t["mask"][1, 2, -1] = bad
    got = check(t, stride, 0, dilation)
    assert (~got["x"][1, 2].isfinite()).sum() <= 2 * K
    assert got["x"][0].isfinite().all() and got["x"][1, :2].isfinite().all()
    t = make(T, 2, 3, L, K, stride, 0, dilation, mask=True)
    t["off"].zero_()
    t["w"][1, 0, 0] = bad
    check(t, stride, 0, dilation)


@pytest.mark.parametrize("dt", TYPES)
def test_far_offsets_at_the_last_positions(dt):
    """Offsets of the last positions that reach back into the signal are not taken along by the
    lanes behind them."""
    t = make(TYPES[dt], 2, 3, 301, 3, 1, 1, 1, mask=True)
    t["off"][:, :, -2:] -= 150
    check(t, 1, 1, 1, True)
