"""Layer norm (GPU) of values whose variance a sum about a badly chosen value would lose: a few
channels far from the others, among them those that the kernels look at first, against the
64-bit form within norm_ref's bounds, which are those of a sum of squares about the mean."""
import pytest
import torch

import deformable_convolution_dcn1d_b200 as dcn
import norm_ref as R
from test_gpu_norm import check_kept, within

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# aligned rows (whole and short tiles, one block and a cluster), unaligned rows, single tokens
SHAPES = [(2, 512, 64), (1, 4096, 128), (1, 16384, 64), (2, 4096, 8), (40, 512, 512), (1, 4100, 33),
          (2, 512, 41), (1, 9001, 8), (3, 4096, 1), (1, 20000, 1)]
FIRST = {"one": [0], "four": [0, 32, 64, 96], "spread": list(range(0, 512, 16)), "last": [511]}


def make(shape, T, rows, size, seed=2, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) + mean
    x[:, rows] += size * (1 + 0.1 * torch.randn(x[:, rows].shape, generator=g))
    return x.to(T).cuda()


def check(x, eps=1e-5):
    y, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(x, eps=eps, checkpoint=True)
    ry, rm, rr, rv = R.norm(x, None, None, eps)
    bm, br, bv = R.norm_bounds(x, None, None, eps)
    within(mean, rm, bm, "mean")
    within(rstd, rr, br, "rstd")
    within(y, ry, R.y_bound(ry, rv, bv, None, x.dtype), "y")
    check_kept(kept, x, eps)
    again = dcn.dcn1d_layer_norm_forward(x, eps=eps)
    assert torch.equal(again[0], y) and torch.equal(again[1], mean) and torch.equal(again[2], rstd)
    return y, mean, rstd


@pytest.mark.parametrize("first", FIRST)
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_outlying_channels(shape, dt, first):
    for size in (30.0, 300.0, -3000.0):
        check(make(shape, TYPES[dt], FIRST[first], size))


# tiles enough for every SM, so that one block walks all channels of a position
MANY_TILES = [(10, 4096, 512), (5, 16384, 1024), (160, 4096, 24), (160, 2000, 31)]


@pytest.mark.parametrize("shape", SHAPES + MANY_TILES, ids=str)
def test_rstd_is_as_close_as_a_sum_about_the_mean(shape):
    """Typical errors, not the worst case.  A position's values lie in 32 chains or more, of
    m = C / 32 additions; an outlier may hold all of the sum in one of them.  m roundings of
    either sign, uniform in half a step u, add up to sqrt(m / 3) u, six times that in all but
    one of 10^9; the variance may have taken that three times and rstd takes half: 9 sqrt(C / 96)
    u, and 10 u for the joins, the division, the root and what else is rounded once."""
    for rows in FIRST.values():
        x = make(shape, torch.float32, rows, 300.0)
        rstd = dcn.dcn1d_layer_norm_forward(x)[2].double()
        ref = R.norm(x, None, None, 1e-5)[2]
        room = (9 * (shape[1] / 96) ** 0.5 + 10) * R.U
        assert ((rstd / ref - 1).abs() <= room).all(), (rows, (rstd / ref - 1).abs().max().item() / R.U)


@pytest.mark.parametrize("shape", [(2, 512, 64), (1, 4096, 128), (2, 512, 41), (1, 9001, 8)], ids=str)
def test_a_position_does_not_depend_on_its_neighbours(shape):
    """Positions that take their sums again leave the others' results as they are, bit for bit."""
    L = shape[2]
    x = make(shape, torch.float32, FIRST["four"], 300.0)
    quiet = make(shape, torch.float32, [5], 0.5, seed=3)
    mixed = quiet.clone()
    mixed[:, :, 1::3] = x[:, :, 1::3]
    a = check(quiet)
    b = check(mixed)
    keep = torch.arange(L) % 3 != 1
    assert torch.equal(a[0][:, :, keep], b[0][:, :, keep])
    assert torch.equal(a[2][:, keep], b[2][:, keep])


def test_outliers_on_a_large_mean():
    for shape in ((1, 4096, 64), (2, 512, 41)):
        check(make(shape, torch.float32, FIRST["four"], 300.0, mean=4096.0))
