"""The depthwise layer's backward pass from a checkpoint (GPU), element by element against the
64-bit form and the bounds of depthwise_ref.py: rows of one position, what lies past the end of
a row, and gradients of very different size in one row."""
import pytest
import torch

import depthwise_ref as D
import deformable_convolution_dcn1d_b200 as dcn
from gpu_util import TOL, norm_err

pytestmark = pytest.mark.gpu

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
        ok = ref[n].to(g.dtype).isfinite()      # a value past the type's range is an infinity in it
        assert torch.equal(g.isfinite(), ok), n
        err = (g.double() - ref[n]).abs()
        bad = ok & ~(err <= bound[n])
        assert not bad.any(), (n, int(bad.sum()), (err / bound[n])[bad].max().item())
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


@pytest.mark.parametrize("unconstrained", [True, False])
@pytest.mark.parametrize("mask", [False, True], ids=["", "mask"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("B,C,L,K,stride,padding,dilation", [
    (2, 5, 1600, 3, 1, 64, 64), (3, 4, 333, 5, 2, 3, 3), (1, 3, 4000, 9, 1, 4, 1), (2, 3, 77, 1, 1, 0, 1),
    (2, 2, 16000, 2, 1, 1, 1), (5, 7, 8, 4, 1, 2, 1), (1, 2, 2, 2, 1, 1, 1)])
def test_every_gradient(B, C, L, K, stride, padding, dilation, dt, mask, unconstrained):
    t = make(TYPES[dt], B, C, L, K, stride, padding, dilation, mask, spread=3.0)
    check(t, stride, padding, dilation, unconstrained)


SPIKE = {"f32": 2.0 ** 40, "bf16": 2.0 ** 40, "f16": 2.0 ** 15}


@pytest.mark.parametrize("masked", [False, True], ids=["", "masked"])
@pytest.mark.parametrize("dt", TYPES)
def test_a_spike_leaves_the_rest_of_its_row_alone(dt, masked):
    """One output gradient far above the others, with and without a mask of zero that takes it
    out again: every other site keeps the precision of its own contributions."""
    T = TYPES[dt]
    t = make(T, 2, 3, 1000, 3, 1, 1, 1, mask=masked, spread=0.5)
    if dt == "f16":
        t["gout"] *= 2.0 ** -8
    t["gout"][0, 1, 500] = SPIKE[dt]
    if masked:
        t["mask"][0, 1, 500] = 0
    check(t, 1, 1, 1, True)
    t["off"].zero_()        # whole positions: the neighbours of the spike's sites get nothing of it
    check(t, 1, 1, 1, True)


@pytest.mark.parametrize("dt", TYPES)
def test_quiet_stretches_keep_their_precision(dt):
    """Stretches of a row whose gradients lie 2^-6 apart, down to 2^-54 (fp16: 2^-12 in all):
    each element within the bound of its own contributions."""
    T = TYPES[dt]
    t = make(T, 1, 3, 1280, 3, 1, 1, 1, mask=True, spread=0.7)
    lower = 2.0 ** -((1 if dt == "f16" else 6) * (torch.arange(1280) // 128).double())
    t["gout"] = (t["gout"].double() * lower.cuda()).to(T)
    check(t, 1, 1, 1, True)
    t["gout"] *= 2.0 ** (10 if dt == "f16" else 90)
    check(t, 1, 1, 1, False)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients_near_the_ends_of_the_range(dt):
    T = TYPES[dt]
    for scale in (2.0 ** -120, 2.0 ** -96, 2.0 ** -60, 2.0 ** 110):
        t = make(T, 1, 3, 300, 3, 1, 1, 1, mask=False)
        t["gout"] = (t["gout"].double() * scale).to(T)
        check(t, 1, 1, 1, True)


@pytest.mark.parametrize("dt", TYPES)
def test_many_contributions_at_one_site(dt):
    """More of the largest kind than a word's sum takes: added again in fp32."""
    T = TYPES[dt]
    t = make(T, 2, 3, 700, 3, 1, 1, 1, mask=False)
    t["off"].copy_(100.25 - torch.arange(700, device="cuda")[:, None] - torch.arange(-1, 2, device="cuda"))
    t["gout"].fill_(1.0)
    t["w"].fill_(1.0)
    check(t, 1, 1, 1, True)


@pytest.mark.parametrize("L,K,dt,mask", [(15000, 3, "bf16", False), (9000, 5, "f32", True)])
def test_equal_calls_give_equal_bits(L, K, dt, mask):
    t = make(TYPES[dt], 2, 64, L, K, 1, K // 2, 1, mask, spread=4.0)
    kept, first = run(t, 1, K // 2, 1, True)
    for _ in range(5):
        _, again = run(t, 1, K // 2, 1, True, kept=kept)
        for n in first:
            assert torch.equal(first[n], again[n]), n


# rows around the ends of what shared memory holds: with the staged stores, without them, and
# without the sites' own units (fp32 additions)
@pytest.mark.parametrize("L,K,dt,mask", [
    (34000, 2, "bf16", False), (34900, 9, "f16", True), (37500, 3, "bf16", True), (38600, 2, "bf16", False),
    (22000, 9, "f32", True), (26500, 3, "f32", False), (28000, 2, "f32", True), (29000, 2, "f32", False)])
def test_rows_near_the_limit(L, K, dt, mask):
    t = make(TYPES[dt], 1, 3, L, K, 1, K // 2, 1, mask, spread=2.0)
    if L in (38600, 29000):     # past the limit: the checkpoint is unpacked, other kernels run
        _, got = run(t, 1, K // 2, 1, True)
        x = dcn.dcn1d_checkpoint_unpack(dcn.dcn1d_checkpoint_pack(t["x"]), dtype=TYPES[dt])
        ref = D.backward(x, t["off"], t["mask"], t["w"], t["gout"], 1, K // 2, 1, True)[0]
        for n, g in got.items():
            assert norm_err(g.double().cpu().numpy(), ref[n].cpu().numpy()) <= TOL[dt], n
        return
    check(t, 1, K // 2, 1, True)
