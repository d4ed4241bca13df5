"""8-bit checkpoints (GPU): codes and step bytes equal to the 64-bit rule's, what is read
back exact, and the convolution's backward pass from a checkpoint."""
import pytest
import torch

import deformable_convolution_dcn1d_b200 as dcn
import norm_ref as R
import oracle
import workloads as W
from gpu_util import TOL, norm_err

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SHAPES = [(1, 1, 1), (2, 31, 1), (3, 512, 1), (1, 1, 7), (2, 5, 32), (3, 7, 33), (2, 16, 64),
          (1, 3, 1601), (4, 64, 200), (2, 9, 2048), (1, 2, 40001)]


def make(shape, T, seed=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape[:2] + (1,), generator=g))
    flat = torch.empty(x.numel() + shift, dtype=T, device="cuda")
    out = flat[shift:].view(shape)
    out.copy_(x)
    return out


def check(x):
    kept = dcn.dcn1d_checkpoint_pack(x)
    codes, scales = R.pack(x)
    assert torch.equal(kept.scales, scales)
    assert torch.equal(kept.codes, codes)
    v = R.values(codes, scales)
    for T in TYPES.values():
        got = dcn.dcn1d_checkpoint_unpack(kept, dtype=T)
        assert torch.equal(got.isnan(), v.isnan())
        assert torch.equal(got.nan_to_num(), v.float().to(T).nan_to_num())
    return kept, v


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_pack_and_unpack_are_exact(shape, dt, shift):
    kept, v = check(make(shape, TYPES[dt], 1, shift))
    again = dcn.dcn1d_checkpoint_pack(dcn.dcn1d_checkpoint_unpack(kept))
    assert torch.equal(dcn.dcn1d_checkpoint_unpack(again), v.float())


@pytest.mark.parametrize("dt", TYPES)
def test_blocks_at_the_ends_of_the_range(dt):
    T = TYPES[dt]
    f = torch.finfo(T)
    sub = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dt]
    x = torch.zeros(1, 9, 70, dtype=T, device="cuda")
    x[0, 0, :3] = torch.tensor([f.max, -f.max, f.max / 3], dtype=T)
    x[0, 1, 33] = f.tiny
    x[0, 2, ::5] = sub
    x[0, 3, 40] = float("nan")
    x[0, 4, 69] = float("inf")
    x[0, 5, 0] = -float("inf")
    x[0, 6] = 127.5
    x[0, 7] = -127.0
    kept, v = check(x)
    finite = torch.isfinite(dcn.dcn1d_checkpoint_unpack(kept, dtype=T))
    bad = torch.zeros(1, 9, 70, dtype=torch.bool, device="cuda")
    bad[0, 3, 32:64] = bad[0, 4, 64:] = bad[0, 5, :32] = True
    assert torch.equal(finite, ~bad)
    assert torch.equal(v.isnan(), bad)


@pytest.mark.parametrize("shape", [(2, 33, 1), (3, 20, 45), (2, 24, 64)], ids=str)
@pytest.mark.parametrize("dt", TYPES)
def test_unpack_through_weights(shape, dt):
    T = TYPES[dt]
    kept = dcn.dcn1d_checkpoint_pack(make(shape, T, 2))
    g = torch.Generator("cuda").manual_seed(5)
    gamma = torch.randn(shape[1], device="cuda", generator=g).to(T)
    beta = torch.randn(shape[1], device="cuda", generator=g).to(T)
    v = R.values(*kept).float()
    for a, b in ((gamma, beta), (gamma, None), (None, beta)):
        want = v if a is None else v * a.float()[:, None]      # one rounding each in fp32
        want = want if b is None else want + b.float()[:, None]
        got = dcn.dcn1d_checkpoint_unpack(kept, a, b, dtype=T)
        assert torch.equal(got, want.to(T))


def test_outputs_given_and_empty():
    x = make((2, 6, 50), torch.bfloat16)
    want = dcn.dcn1d_checkpoint_pack(x)
    out = dcn.Checkpoint8(torch.empty_like(want.codes), torch.empty_like(want.scales))
    got = dcn.dcn1d_checkpoint_pack(x, out=out)
    assert got.codes is out.codes and torch.equal(got.codes, want.codes)
    back = torch.empty_like(x)
    assert dcn.dcn1d_checkpoint_unpack(got, out=back) is back
    for shape in ((0, 4, 9), (2, 4, 0)):
        k = dcn.dcn1d_checkpoint_pack(torch.empty(shape, device="cuda"))
        assert dcn.dcn1d_last_launch_count() == 0
        assert dcn.dcn1d_checkpoint_unpack(k).shape == shape
    with pytest.raises(ValueError, match="B, C, L"):
        dcn.dcn1d_checkpoint_pack(x[0])


# dtype, B, C_in, C_out, K, L, s, p, d, groups, og, mask, unconstrained, offset scale
CONV = {
    "dense_bf16_mask": ("bf16", 2, 64, 64, 5, 264, 1, 2, 1, 1, 8, True, False, 3.0),
    "dense_f16_g2": ("f16", 2, 32, 48, 3, 130, 2, 1, 2, 2, 2, False, True, 2.0),
    "dense_f32": ("f32", 2, 48, 32, 4, 203, 2, 1, 1, 1, 2, False, False, 2.0),
    "depthwise_f32": ("f32", 2, 16, 16, 3, 300, 1, 8, 8, 16, 16, False, True, 4.0),
    "depthwise_f32_mask": ("f32", 3, 9, 9, 4, 97, 1, 2, 1, 9, 9, True, False, 2.0),
    "depthwise_bf16": ("bf16", 2, 24, 24, 3, 520, 1, 64, 64, 24, 24, False, True, 4.0),
    "depthwise_bf16_mask_stride": ("bf16", 2, 16, 16, 5, 333, 2, 3, 3, 16, 16, True, True, 3.0),
    "depthwise_f16": ("f16", 1, 40, 40, 2, 1000, 1, 1, 2, 40, 40, True, False, 1.0),
    "depthwise_one_tap": ("f32", 2, 8, 8, 1, 77, 1, 0, 1, 8, 8, True, True, 40.0),
    "depthwise_nine_taps": ("bf16", 1, 12, 12, 9, 400, 1, 8, 2, 12, 12, False, False, 2.0),
    "depthwise_shared_offsets": ("bf16", 2, 16, 16, 3, 200, 1, 1, 1, 16, 4, True, False, 2.0),
    "depthwise_lout_1": ("f32", 3, 6, 6, 8, 8, 1, 0, 1, 6, 6, False, False, 2.0),
    "depthwise_many_rows": ("bf16", 70, 1000, 1000, 3, 8, 1, 1, 1, 1000, 1000, False, False, 1.0),
    "depthwise_wide_padding": ("f32", 1, 2, 2, 3, 50, 1, 60000, 1, 2, 2, True, True, 2.0),
    "depthwise_long_rows_f32": ("f32", 1, 2, 2, 3, 20000, 1, 1, 1, 2, 2, False, True, 2.0),
    "depthwise_long_rows": ("f16", 1, 3, 3, 2, 32001, 1, 0, 1, 3, 3, True, False, 1.0),
    "depthwise_far": ("f32", 2, 5, 5, 3, 300, 1, 1, 1, 5, 5, True, True, 400.0),
}
NAMES = {"x": "grad_x", "offsets": "grad_offsets", "mask": "grad_mask", "weight": "grad_weight",
         "bias": "grad_bias"}


def conv_case(key, seed=7):
    dt, B, Ci, Co, K, L, s, p, d, G, og, mask, unc, sc = CONV[key]
    L_out = oracle.out_length(L, K, s, p, d)
    w, t = W.small_case(seed, B=B, C_in=Ci, C_out=Co, K=K, stride=s, padding=p, dilation=d,
                        groups=G, offset_groups=og, L_in=L, L_out=L_out, dtype=dt, mask=mask,
                        unconstrained=unc, off_scale=sc)
    g = torch.Generator().manual_seed(seed + 1)
    T = t["x"].dtype
    gout = torch.randn(B, Co, L_out, generator=g).to(T)
    gamma = (1 + 0.3 * torch.randn(Ci, generator=g)).to(T)
    beta = torch.randn(Ci, generator=g).to(T)
    t = {k: (v.cuda() if v is not None else None) for k, v in t.items()}
    return w, t, gout.cuda(), gamma.cuda(), beta.cuda()


def conv_args(w):
    return (w.stride, w.padding, w.dilation, w.groups, w.offset_groups, w.unconstrained)


@pytest.mark.parametrize("affine", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("key", CONV)
def test_conv_backward_from_a_checkpoint(key, affine):
    w, t, gout, gamma, beta = conv_case(key)
    kept = dcn.dcn1d_checkpoint_pack(t["x"])
    gamma, beta = (gamma, beta) if affine else (None, None)
    got = dcn.dcn1d_backward_checkpoint(kept, t["offsets"], t["mask"], t["weight"], gout,
                                        *conv_args(w), gamma=gamma, beta=beta)
    x = dcn.dcn1d_checkpoint_unpack(kept, gamma, beta, dtype=t["x"].dtype)
    cpu = [None if v is None else v.cpu() for v in (x, t["offsets"], t["mask"], t["weight"], gout)]
    ref = oracle.backward(*cpu, *conv_args(w))
    assert set(got) == set(dcn.GRADS) - (set() if w.mask else {"mask"})
    for n, g in got.items():
        assert g.dtype == gout.dtype
        err = norm_err(g.double().cpu().numpy(), ref[NAMES[n]])
        assert err <= TOL[w.dtype], (n, err)


@pytest.mark.parametrize("key", ["depthwise_bf16_mask_stride", "dense_bf16_mask"])
def test_conv_backward_subsets(key):
    """Every subset against the full call: rounded alike, so apart by one rounding of the
    type where fp32 additions came in another order."""
    w, t, gout, _, _ = conv_case(key)
    kept = dcn.dcn1d_checkpoint_pack(t["x"])

    def run(**k):
        return dcn.dcn1d_backward_checkpoint(kept, t["offsets"], t["mask"], t["weight"], gout,
                                             *conv_args(w), **k)
    full = run()
    for wanted in (("x",), ("offsets",), ("mask",), ("weight",), ("bias",), ("offsets", "mask"),
                   ("x", "weight", "bias")):
        part = run(wanted=wanted)
        assert set(part) == set(wanted)
        for n in wanted:
            a, b = part[n].double(), full[n].double()
            room = 2 * R.half_step(gout.dtype) * b.abs() + 1e-5 * b.abs().max()
            assert ((a - b).abs() <= room).all(), n


def test_conv_backward_of_an_empty_batch():
    w, t, gout, _, _ = conv_case("depthwise_bf16")
    kept = dcn.dcn1d_checkpoint_pack(t["x"][:0])
    got = dcn.dcn1d_backward_checkpoint(kept, t["offsets"][:0], None, t["weight"], gout[:0],
                                        *conv_args(w))
    assert (got["weight"] == 0).all() and (got["bias"] == 0).all() and got["x"].shape[0] == 0


@pytest.mark.parametrize("key", ["depthwise_bf16", "dense_bf16_mask"])
def test_a_training_step_from_one_checkpoint(key):
    """Norm, convolution, and both backward passes from the one checkpoint that the norm
    kept; against 64-bit autograd of the same step whose saved values are the checkpoint's.
    Also captured into a graph and replayed on new inputs."""
    w, t, gout, gamma, beta = conv_case(key)
    a = conv_args(w)
    h = t["x"]
    h.mul_(1.7).add_(0.3)

    def step():
        y, _, rstd, kept = dcn.dcn1d_layer_norm_forward(h, gamma, beta, checkpoint=True)
        z = dcn.dcn1d_forward(y, t["offsets"], t["mask"], t["weight"], t["bias"], *a)
        gc = dcn.dcn1d_backward_checkpoint(kept, t["offsets"], t["mask"], t["weight"], gout, *a,
                                           gamma=gamma, beta=beta)
        gn = dcn.dcn1d_layer_norm_backward(kept, gamma, None, rstd, gc["x"])
        return y, z, rstd, kept, gc, gn

    def check(y, z, rstd, kept, gc, gn):
        v = R.values(*kept)
        x = (v.float() * gamma.float()[:, None] + beta.float()[:, None]).to(y.dtype)
        # what the checkpoint stands for is within its step of what the forward used
        step_of = R.two_to(kept.scales.int() - 127).repeat_interleave(32, 2)[:, :, :h.shape[2]]
        room = step_of * gamma.double().abs()[:, None] + 2 * R.half_step(y.dtype) * (
            y.double().abs() + 1)
        assert ((x.double() - y.double()).abs() <= room).all()
        cpu = [None if q is None else q.cpu() for q in (x, t["offsets"], t["mask"], t["weight"],
                                                        gout)]
        ref = oracle.backward(*cpu, *a)
        for n, g in gc.items():
            assert norm_err(g.double().cpu().numpy(), ref[NAMES[n]]) <= TOL[w.dtype], n
        rn = R.norm_grads(v, rstd.double(), gamma, gc["x"])
        bn = R.grad_bounds(v, torch.zeros_like(v), rstd.double(), gamma, gc["x"], y.dtype)
        for n in dcn.NORM_GRADS:
            assert ((gn[n].double() - rn[n]).abs() <= bn[n]).all(), n

    check(*step())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    h.copy_(h.flip(0) * 0.5)
    gout.copy_(gout.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    check(*out)


@pytest.mark.parametrize("K,og", [(3, 16), (5, 4)])
def test_far_and_bad_offsets_read_nothing_outside(K, og):
    """Offsets that leave the signal by far, infinities and NaN: no access out of range (the
    rows around the gradients keep their fill), and finite offsets' gradients stay right."""
    w, t, gout, _, _ = conv_case("depthwise_f32" if og == 16 else "depthwise_shared_offsets")
    off = t["offsets"]
    off[0, 0, :4] = torch.tensor([1e6, -1e6, 3.0e38], device="cuda").to(off.dtype)[
        torch.arange(off.shape[3], device="cuda") % 3]
    kept = dcn.dcn1d_checkpoint_pack(t["x"])
    wide = torch.full((t["x"].numel() + 64,), 7.0, dtype=gout.dtype, device="cuda")
    gx = wide[32:-32].view(t["x"].shape)
    got = dcn.dcn1d_backward_checkpoint(kept, off, t["mask"], t["weight"], gout, *conv_args(w),
                                        grads={"x": gx})
    assert (wide[:32] == 7).all() and (wide[-32:] == 7).all()
    assert all(torch.isfinite(g).all() for g in got.values())
    off[0, 0, :4] = float("nan")
    off[0, 0, 4:6] = float("inf")
    got = dcn.dcn1d_backward_checkpoint(kept, off, t["mask"], t["weight"], gout, *conv_args(w),
                                        grads={"x": gx})
    assert (wide[:32] == 7).all() and (wide[-32:] == 7).all()
    # the batches that hold no such offset are untouched by it
    clean = dcn.dcn1d_backward_checkpoint(
        dcn.Checkpoint8(kept.codes[1:], kept.scales[1:]), off[1:].contiguous(),
        None if t["mask"] is None else t["mask"][1:].contiguous(), t["weight"], gout[1:],
        *conv_args(w), wanted=("x", "offsets"))
    for n in ("x", "offsets"):
        a, b = got[n][1:].double(), clean[n].double()
        assert ((a - b).abs() <= 2 * R.half_step(gout.dtype) * b.abs()
                + 1e-5 * b.abs().max()).all(), n


@pytest.mark.parametrize("dt,C,L,K,mask", [("bf16", 3, 700, 3, False), ("f16", 2, 1200, 2, True),
                                          ("f32", 3, 700, 3, True), ("bf16", 2, 5000, 5, True)])
def test_many_taps_at_one_site(dt, C, L, K, mask):
    """Every tap of a row samples near position 100, so thousands of equal contributions meet
    at two sites; the oracle adds them in 64 bits.  Position and fraction are exact in the
    type (offsets are whole multiples of 1/4 up to L in fp32, rounded by the type before)."""
    T = TYPES[dt]
    l = torch.arange(L)[:, None]
    k = torch.arange(K)[None]
    off = (100.25 - (l + k)).to(T).expand(2, C, L, K).contiguous()
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, C, L, generator=g).to(T)
    w = torch.ones(C, 1, K).to(T)
    gout = torch.ones(2, C, L + K - 1).to(T)[:, :, :L].contiguous()
    m = torch.full((2, C, L, K), 0.5).to(T) if mask else None
    args = (1, (0, K - 1), 1, C, C, True)
    kept = dcn.dcn1d_checkpoint_pack(x.cuda())
    dev = [None if t is None else t.cuda() for t in (off, m, w, gout)]
    got = dcn.dcn1d_backward_checkpoint(kept, *dev, *args)
    back = dcn.dcn1d_checkpoint_unpack(kept, dtype=T).cpu()
    ref = oracle.backward(back, off, m, w, gout, *args)
    for n, t in got.items():
        assert norm_err(t.double().cpu().numpy(), ref[NAMES[n]]) <= TOL[dt], n


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt", TYPES)
def test_bad_gradients_reach_their_sites_only(dt, bad):
    T = TYPES[dt]
    C, L, K = 4, 200, 3
    g = torch.Generator().manual_seed(8)
    x = torch.randn(2, C, L, generator=g).to(T).cuda()
    off = (0.5 * torch.randn(2, C, L, K, generator=g)).to(T).cuda()
    w = (1 + torch.rand(C, 1, K, generator=g)).to(T).cuda()
    gout = torch.randn(2, C, L, generator=g).to(T).cuda()
    kept = dcn.dcn1d_checkpoint_pack(x)
    args = (1, 1, 1, C, C, False)
    clean = dcn.dcn1d_backward_checkpoint(kept, off, None, w, gout, *args)
    gout[1, 2, 90] = bad
    got = dcn.dcn1d_backward_checkpoint(kept, off, None, w, gout, *args)
    hit = ~torch.isfinite(got["x"])
    assert hit[1, 2, 88:93].any() and hit.sum() == hit[1, 2, 88:93].sum()
    a, b = got["x"][~hit].double(), clean["x"][~hit].double()
    assert ((a - b).abs() <= 2 * R.half_step(T) * b.abs() + 1e-5 * b.abs().max()).all()
    touched = ~torch.isfinite(got["offsets"])
    assert touched[1, 2, 90].any() and touched.sum() == touched[1, 2, 90].sum()


@pytest.mark.parametrize("dt", TYPES)
def test_gradients_of_very_different_size_in_one_row(dt):
    """Output gradients from 1 down to 2^-9 in stretches of a row: the small ones' grad_x is
    compared on its own.  Fixed point of unit M 2^-22 leaves them 13 bits and more of their
    own largest, below half a step of bf16 (2^-8) and fp16 (2^-11)."""
    T = TYPES[dt]
    C, L, K = 3, 1024, 3
    g = torch.Generator().manual_seed(9)
    x = torch.randn(1, C, L, generator=g).to(T)
    off = torch.zeros(1, C, L, K).to(T)
    w = torch.ones(C, 1, K).to(T)
    size = 2.0 ** -(torch.arange(L) // 128 * 9 // 7).double()
    gout = (torch.randn(1, C, L, generator=g).double() * size).to(T)
    args = (1, 1, 1, C, C, False)
    kept = dcn.dcn1d_checkpoint_pack(x.cuda())
    got = dcn.dcn1d_backward_checkpoint(kept, off.cuda(), None, w.cuda(), gout.cuda(), *args,
                                        wanted=("x",))["x"].double().cpu()
    ref = torch.from_numpy(oracle.backward(dcn.dcn1d_checkpoint_unpack(kept, dtype=T).cpu(), off,
                                           None, w, gout, *args)["grad_x"])
    M = gout.double().abs().amax()
    # three contributions a site and its neighbours' zeros: six roundings to the unit
    unit = M * (2.0 ** -22 if dt != "f32" else 2.0 ** -28)
    fp32 = 4 * R.U * ref.abs().amax() if dt == "f32" else 0.0
    room = R.half_step(T) * ref.abs() + 6 * unit + fp32
    for at in range(0, L, 128):
        part = slice(at + 2, at + 126)
        assert ((got - ref)[:, :, part].abs() <= room[:, :, part]).all(), at


@pytest.mark.parametrize("key", ["depthwise_bf16_mask_stride", "dense_bf16_mask"])
def test_calls_from_two_threads_on_their_own_streams(key):
    """Two host threads, a stream each, many calls at once: scratch is a call's own, so every
    result is the one of a quiet device (apart by one rounding where dense fp32 atomics came in
    another order)."""
    import threading
    w, t, gout, gamma, beta = conv_case(key)
    kept = dcn.dcn1d_checkpoint_pack(t["x"])

    def step(stream=None):
        k = dcn.dcn1d_checkpoint_pack(t["x"], stream=stream)
        return k, dcn.dcn1d_backward_checkpoint(k, t["offsets"], t["mask"], t["weight"], gout,
                                                *conv_args(w), gamma=gamma, beta=beta,
                                                stream=stream)
    _, want = step()
    torch.cuda.synchronize()
    results, errors = [], []

    def work():
        try:
            s = torch.cuda.Stream()
            out = [step(s) for _ in range(20)]
            s.synchronize()
            results.extend(out)
        except Exception as e:   # a thread's failure must reach the test
            errors.append(e)
    threads = [threading.Thread(target=work) for _ in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and len(results) == 40
    for k, got in results:
        assert torch.equal(k.codes, kept.codes) and torch.equal(k.scales, kept.scales)
        for n, g in got.items():
            a, b = g.double(), want[n].double()
            room = 2 * R.half_step(gout.dtype) * b.abs() + 1e-5 * b.abs().max()
            assert ((a - b).abs() <= room).all(), n
            if key.startswith("depthwise"):
                assert torch.equal(g, want[n]), n


def test_a_given_stream():
    x = make((1, 4, 40), torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k = dcn.dcn1d_checkpoint_pack(x, stream=s)
    v = dcn.dcn1d_checkpoint_unpack(k, stream=s)
    s.synchronize()
    assert torch.equal(v, dcn.dcn1d_checkpoint_unpack(dcn.dcn1d_checkpoint_pack(x)))
