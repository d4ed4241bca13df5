"""Layer norm over the channels and its gradients (GPU) against the 64-bit forms of
norm_ref.py, element by element within bounds counted from the roundings made."""
import pytest
import torch

import deformable_convolution_dcn1d_b200 as dcn
import norm_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# one channel, one position, sizes around the 32-value blocks and the 64-position tiles,
# channels around the slices that one block holds, rows that start off every alignment
SHAPES = [(1, 1, 1), (1, 512, 1), (3, 33, 1), (5, 1024, 1), (70, 96, 1), (2, 4100, 1),
          (1, 1, 5), (2, 7, 2), (3, 64, 8), (2, 48, 31), (2, 256, 32), (2, 37, 33),
          (1, 512, 64), (2, 130, 65), (3, 512, 83), (2, 260, 128), (1, 381, 1001),
          (1, 1030, 40), (1, 2056, 72), (1, 9001, 8), (1, 16, 4096), (4, 256, 200),
          (1, 26001, 33), (1, 20000, 1),
          (2, 70, 50), (3, 200, 36), (1, 40, 14), (3000, 1000, 1), (700, 64, 1), (900, 3000, 1)]
# the memory that 16-byte accesses need is not there: rows start one element further on
SHIFTED = [(2, 96, 1), (2, 40, 64), (1, 256, 72)]


def make(shape, T, seed, shift=0, affine=True):
    B, C, L = shape
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, C, L, generator=g) * torch.exp(0.7 * torch.randn(1, C, 1, generator=g))
    x = x + torch.randn(1, C, 1, generator=g)
    gy = torch.randn(B, C, L, generator=g)
    gamma = 1 + 0.3 * torch.randn(C, generator=g)
    beta = torch.randn(C, generator=g)

    def dev(t):
        flat = torch.empty(t.numel() + shift, dtype=T, device="cuda")
        out = flat[shift:].view(t.shape)
        out.copy_(t)
        return out
    x, gy = dev(x), dev(gy)
    return x, gy, (dev(gamma) if affine else None), (dev(beta) if affine else None)


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), err[bad].max().item(),
                           (err / bound)[bad].max().item())


def check_forward(shape, T, shift=0, affine=True, eps=1e-5, seed=0):
    x, _, gamma, beta = make(shape, T, seed, shift, affine)
    y, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(x, gamma, beta, eps)
    assert kept is None and y.dtype == T and mean.dtype == rstd.dtype == torch.float32
    ry, rm, rr, rv = R.norm(x, gamma, beta, eps)
    bm, br, bv = R.norm_bounds(x, gamma, beta, eps)
    within(mean, rm, bm, "mean")
    within(rstd, rr, br, "rstd")
    within(y, ry, R.y_bound(ry, rv, bv, gamma, T), "y")
    return x, y, mean, rstd, gamma, beta


def check_kept(kept, x, eps=1e-5):
    """The checkpoint of the normalised values, each within half a step of v and its error."""
    _, _, _, v = R.norm(x, None, None, eps)
    _, _, bv = R.norm_bounds(x, None, None, eps)
    r, b = R.rows_of(v), R.rows_of(bv)
    n = r.shape[1]
    pad = (0, -n % 32)
    amax = torch.nn.functional.pad(r.abs(), pad).unflatten(1, (-1, 32)).amax(2)
    off = torch.nn.functional.pad(b, pad).unflatten(1, (-1, 32)).amax(2)
    e = kept.scales.reshape(r.shape[0], -1).int() - 127
    assert (e >= R.step_exponent(amax - off, 121)).all()
    assert (e <= R.step_exponent(amax + off, 121)).all()
    step = R.two_to(e).repeat_interleave(32, 1)[:, :n]
    assert (kept.codes.abs().int() <= 127).all()
    within(R.rows_of(R.values(*kept)), r, step / 2 + b, "checkpoint")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dt):
    T = TYPES[dt]
    x, y, mean, rstd, gamma, beta = check_forward(shape, T)
    y2, m2, r2, kept = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True)
    assert torch.equal(y, y2) and torch.equal(mean, m2) and torch.equal(rstd, r2)
    check_kept(kept, x)
    y3, m3, r3, _ = dcn.dcn1d_layer_norm_forward(x, gamma, beta, stats=False)
    assert m3 is None and r3 is None and torch.equal(y, y3)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHIFTED, ids=str)
def test_forward_off_alignment(shape, dt):
    x, y, mean, rstd, gamma, beta = check_forward(shape, TYPES[dt], shift=1)
    out = torch.full((x.numel() + 3,), 7.0, dtype=x.dtype, device="cuda")
    got, *_, kept = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True,
                                                 out=out[1:-2].view(shape))
    assert torch.equal(got, y) and (out[0] == 7).all() and (out[-2:] == 7).all()
    check_kept(kept, x)


@pytest.mark.parametrize("shape", [(2, 65, 1), (2, 65, 40)], ids=str)
def test_weights_may_be_absent_one_by_one(shape):
    x, _, gamma, beta = make(shape, torch.float32, 3)
    for g, b in ((gamma, None), (None, beta), (None, None)):
        ry, _, _, rv = R.norm(x, g, b, 1e-5)
        bv = R.norm_bounds(x, g, b, 1e-5)[2]
        y = dcn.dcn1d_layer_norm_forward(x, g, b)[0]
        within(y, ry, R.y_bound(ry, rv, bv, g, torch.float32), (g is None, b is None))


@pytest.mark.parametrize("shape", [(3, 40, 1), (2, 40, 70)], ids=str)
def test_equal_channels_and_a_large_mean(shape):
    # equal channels: v is 0 up to the rounding of the mean, rstd = 1 / sqrt(eps)
    x = torch.full(shape, 3.0, device="cuda")
    y, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(x, eps=1e-5, checkpoint=True)
    assert torch.equal(mean, torch.full_like(mean, 3.0)) and (y == 0).all()
    assert (dcn.dcn1d_checkpoint_unpack(kept) == 0).all() and (kept.scales == 1).all()
    # a mean 4096 times the deviation: squares of x would lose the variance in fp32
    g = torch.Generator().manual_seed(1)
    x = (4096 + torch.randn(shape, generator=g)).cuda()
    y, mean, rstd, _ = dcn.dcn1d_layer_norm_forward(x)
    ry, rm, rr, rv = R.norm(x, None, None, 1e-5)
    bm, br, bv = R.norm_bounds(x, None, None, 1e-5)
    within(mean, rm, bm, "mean")
    within(rstd, rr, br, "rstd")
    within(y, ry, R.y_bound(ry, rv, bv, None, torch.float32), "y")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("shape", [(2, 70, 1), (2, 48, 100), (2, 40, 64)], ids=str)
def test_bad_values_stay_at_their_position(shape, bad):
    x, _, gamma, beta = make(shape, torch.float32, 5)
    clean = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True)
    x[1, 3, shape[2] // 2] = bad
    y, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True)
    hit = torch.zeros(shape[0], shape[2], dtype=torch.bool, device="cuda")
    hit[1, shape[2] // 2] = True
    assert torch.equal(y.isnan(), hit[:, None].expand(shape))
    assert torch.equal(torch.where(hit[:, None], 0.0, y), torch.where(hit[:, None], 0.0, clean[0]))
    # the checkpoint: the blocks that hold the position read back NaN, no other
    v = dcn.dcn1d_checkpoint_unpack(kept)
    if shape[2] == 1:
        block = hit[:, None].expand(shape)
    else:
        at = shape[2] // 2 // 32 * 32
        block = torch.zeros(shape, dtype=torch.bool, device="cuda")
        block[1, :, at:at + 32] = True
    assert torch.equal(v.isnan(), block)


def grads_of(x, gy, gamma, kept, eps=1e-5):
    """(gradients, their references and bounds) from x or from the checkpoint."""
    T = gy.dtype
    _, mean, rstd, k = dcn.dcn1d_layer_norm_forward(x, gamma, None, eps, checkpoint=kept)
    got = dcn.dcn1d_layer_norm_backward(k if kept else x, gamma, None if kept else mean, rstd, gy)
    rs = rstd.double()
    if kept:
        v, e_v = R.values(*k), torch.zeros((), dtype=torch.float64, device="cuda")
    else:   # the kernel's v has two roundings, of x - mean and of the product
        v = (x.double() - mean.double()[:, None]) * rs[:, None]
        e_v = 2.02 * R.U * v.abs()
    return got, R.norm_grads(v, rs, gamma, gy), R.grad_bounds(v, e_v, rs, gamma, gy, T)


@pytest.mark.parametrize("kept", [False, True], ids=["x", "checkpoint"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dt, kept):
    x, gy, gamma, _ = make(shape, TYPES[dt], 11)
    got, ref, bound = grads_of(x, gy, gamma, kept)
    for n in dcn.NORM_GRADS:
        assert got[n].dtype == gy.dtype
        within(got[n], ref[n], bound[n], n)


@pytest.mark.parametrize("kept", [False, True], ids=["x", "checkpoint"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHIFTED, ids=str)
def test_backward_off_alignment(shape, dt, kept):
    x, gy, gamma, _ = make(shape, TYPES[dt], 12, shift=1)
    got, ref, bound = grads_of(x, gy, gamma, kept)
    for n in dcn.NORM_GRADS:
        within(got[n], ref[n], bound[n], n)


@pytest.mark.parametrize("shape", [(40, 96, 1), (3, 130, 70), (6, 256, 640)], ids=str)
def test_backward_subsets_and_equal_bits(shape):
    x, gy, gamma, _ = make(shape, torch.bfloat16, 13)
    _, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(x, gamma, checkpoint=True)
    for src, m in ((x, mean), (kept, None)):
        full = dcn.dcn1d_layer_norm_backward(src, gamma, m, rstd, gy)
        for wanted in (("x",), ("gamma",), ("beta",), ("x", "beta"), ("gamma", "beta"), ()):
            part = dcn.dcn1d_layer_norm_backward(src, gamma, m, rstd, gy, wanted=wanted)
            assert set(part) == set(wanted)
            for n in wanted:
                assert torch.equal(part[n], full[n]), (wanted, n)


def test_backward_without_gamma():
    x, gy, _, _ = make((2, 70, 50), torch.float32, 14)
    got, ref, bound = grads_of(x, gy, None, False)
    for n in dcn.NORM_GRADS:
        within(got[n], ref[n], bound[n], n)


def test_gradient_against_differences():
    """grad_x along a random direction against central differences of the 64-bit forward:
    the difference quotient is off by O(h^2) < 1e-8 here, the fp32 gradient by its bound."""
    x, gy, gamma, beta = make((2, 40, 33), torch.float32, 15)
    got, _, bound = grads_of(x, gy, gamma, False)
    u = torch.randn(x.shape, dtype=torch.float64, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(3))
    h = 1e-5
    f = [(R.norm(x.double() + s * h * u, gamma, beta, 1e-5)[0] * gy.double()).sum()
         for s in (1, -1)]
    slope = (f[0] - f[1]) / (2 * h)
    # mean and rstd that the gradient was given are themselves rounded: 2^-24 and the
    # forward's bound of each, in every term
    bm, br, bv = R.norm_bounds(x, gamma, beta, 1e-5)
    rstd = R.norm(x, gamma, beta, 1e-5)[2]
    given = (got["x"].double().abs() * (br / rstd)[:, None] + 4 * bv * rstd[:, None]
             * (gy.double() * gamma.double()[:, None]).abs().mean(1, keepdim=True)).abs()
    room = ((bound["x"] + given) * u.abs()).sum() + 1e-6
    assert abs((got["x"].double() * u).sum() - slope) <= room


def test_empty_inputs():
    for shape in ((0, 8, 5), (3, 8, 0), (0, 8, 1)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(x, checkpoint=True)
        assert y.shape == shape and kept.codes.shape == shape
        assert dcn.dcn1d_last_launch_count() == 0
        got = dcn.dcn1d_layer_norm_backward(x, None, mean, rstd, x)
        assert (got["gamma"] == 0).all() and (got["beta"] == 0).all()


def test_more_than_2_31_elements():
    # 2^31 + 2^22 values: offsets pass 32 bits; checked at both ends
    B, C, L = 1026, 512, 4096
    x = torch.empty(B, C, L, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(4)
    x[0].normal_(generator=g)
    x[1:] = x[0]
    x[-1] *= -1
    y, mean, rstd, kept = dcn.dcn1d_layer_norm_forward(x, checkpoint=True)
    assert torch.equal(y[0], y[-2]) and torch.equal(y[0], -y[-1])
    assert torch.equal(kept.codes[0], -kept.codes[-1])
    assert torch.equal(kept.scales[0], kept.scales[-1])
    back = dcn.dcn1d_checkpoint_unpack(kept, dtype=torch.bfloat16)
    assert torch.equal(back[0], -back[-1])
    got = dcn.dcn1d_layer_norm_backward(kept, None, None, rstd, x, wanted=("x",))["x"]
    assert torch.equal(got[0], -got[-1]) and torch.equal(got[0], got[-2])
    v = R.values(kept.codes[:1], kept.scales[:1])
    ref = R.norm_grads(v, rstd[:1].double(), None, x[:1])
    bound = R.grad_bounds(v, torch.zeros_like(v), rstd[:1].double(), None, x[:1], x.dtype)
    within(got[:1], ref["x"], bound["x"], "x")


def test_streams_and_a_replayed_graph():
    x, gy, gamma, beta = make((2, 128, 200), torch.bfloat16, 16)
    want = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True)
    wantg = dcn.dcn1d_layer_norm_backward(want[3], gamma, None, want[2], gy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True, stream=s)
    gotg = dcn.dcn1d_layer_norm_backward(got[3], gamma, None, got[2], gy, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[3].codes, want[3].codes)
    for n in dcn.NORM_GRADS:
        assert torch.equal(gotg[n], wantg[n])
    # two graphs that share no scratch, replayed on two streams at once with new inputs
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True)
            b = dcn.dcn1d_layer_norm_backward(f[3], gamma, None, f[2], gy)
        graphs.append(graph)
        outs.append((f, b))
    x.copy_(x.flip(2))
    gy.copy_(gy.flip(2))
    want = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=True)
    wantg = dcn.dcn1d_layer_norm_backward(want[3], gamma, None, want[2], gy)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for f, b in outs:
        assert torch.equal(f[0], want[0]) and torch.equal(f[3].scales, want[3].scales)
        for n in dcn.NORM_GRADS:
            assert torch.equal(b[n], wantg[n])


def test_given_outputs_and_workspace():
    x, gy, gamma, beta = make((2, 64, 48), torch.float16, 17)
    kept = dcn.Checkpoint8(torch.empty(x.shape, dtype=torch.int8, device="cuda"),
                           torch.empty(2, 64, 2, dtype=torch.uint8, device="cuda"))
    out = torch.empty_like(x)
    y, mean, rstd, k = dcn.dcn1d_layer_norm_forward(x, gamma, beta, checkpoint=kept, out=out)
    assert y is out and k.codes is kept.codes
    gx = torch.empty_like(x)
    want = dcn.dcn1d_layer_norm_backward(kept, gamma, None, rstd, gy)
    with pytest.raises(ValueError, match="workspace"):
        dcn.dcn1d_layer_norm_backward(kept, gamma, None, rstd, gy,
                                      workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")   # NaN bits
    got = dcn.dcn1d_layer_norm_backward(kept, gamma, None, rstd, gy, grads={"x": gx}, workspace=ws)
    assert got["x"] is gx
    for n in dcn.NORM_GRADS:
        assert torch.equal(got[n], want[n])
    with pytest.raises(dcn.Dcn1dError):
        dcn.dcn1d_layer_norm_backward(x, gamma, None, rstd, gy)   # x without its mean
    with pytest.raises(ValueError, match="contiguous"):
        dcn.dcn1d_layer_norm_forward(x.transpose(1, 2))
