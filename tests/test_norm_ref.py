"""The 64-bit forms that the GPU tests compare with: their gradients against autograd and
central differences, and the checkpoint's rules on values worked out by hand (CPU)."""
import pytest
import torch

import norm_ref as R


def test_norm_gradients_against_autograd_and_differences():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(3, 7, 5, generator=g, dtype=torch.float64).requires_grad_()
    gamma = torch.randn(7, generator=g, dtype=torch.float64).requires_grad_()
    beta = torch.randn(7, generator=g, dtype=torch.float64).requires_grad_()
    gy = torch.randn(3, 7, 5, generator=g, dtype=torch.float64)
    y, mean, rstd, v = R.norm(x, gamma, beta, 1e-5)
    want = torch.autograd.grad((y * gy).sum(), (x, gamma, beta))
    got = R.norm_grads(v.detach(), rstd.detach(), gamma.detach(), gy)
    for n, w in zip(("x", "gamma", "beta"), want):
        assert torch.allclose(got[n], w, rtol=1e-12, atol=1e-12), n
    # along a random direction, central differences (error h^2 ~ 1e-10)
    u = torch.randn(3, 7, 5, generator=g, dtype=torch.float64)
    h = 1e-5
    with torch.no_grad():
        f = [(R.norm(x + s * h * u, gamma, beta, 1e-5)[0] * gy).sum() for s in (1, -1)]
    assert abs((f[0] - f[1]) / (2 * h) - (got["x"] * u).sum()) < 1e-7


def test_norm_matches_the_library_layer_norm_in_64_bits():
    x = torch.randn(2, 9, 4, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    want = torch.nn.functional.layer_norm(x.transpose(1, 2), (9,), eps=1e-3).transpose(1, 2)
    assert torch.allclose(R.norm(x, None, None, 1e-3)[0], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("amax,exponent", [
    (64.0, 0), (127.0, 0), (127.25, 0), (127.5, 1), (128.0, 1), (1.0, -6), (0.0, -126),
    (2.0 ** -130, -126), (3.4028234663852886e38, 121), (1.99, -6), (1.9921875, -5)])
def test_step_of_a_block(amax, exponent):
    assert R.step_exponent(torch.tensor(amax, dtype=torch.float64), 121).item() == exponent


def test_pack_by_hand():
    x = torch.zeros(1, 2, 34)
    x[0, 0, :4] = torch.tensor([127.0, -63.5, 0.5, 1.5])   # step 1: ties go to even
    x[0, 0, 32] = -0.25                                     # a block of two: step 2^-8
    x[0, 1, 5] = float("nan")
    codes, scales = R.pack(x)
    assert codes[0, 0, :5].tolist() == [127, -64, 0, 2, 0]
    assert scales[0].tolist() == [[127, 127 - 8], [255, 1]]
    assert codes[0, 0, 32].item() == -64
    back = R.values(codes, scales)
    assert back[0, 0, 32].item() == -0.25 and back[0, 1, :32].isnan().all()
    assert (back[0, 1, 32:] == 0).all()


def test_half_float_blocks_saturate_inside_the_type():
    x = torch.full((1, 1, 3), 65504.0, dtype=torch.float16)
    v = R.values(*R.pack(x))
    assert (v == 127 * 512.0).all() and torch.isfinite(v.half()).all()


@pytest.mark.parametrize("shape", [(2, 3, 65), (2, 70, 1), (1, 1, 1), (3, 5, 31)])
def test_pack_error_and_repacking(shape):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(2))
    codes, scales = R.pack(x)
    n = shape[1] if shape[2] == 1 else shape[2]
    assert scales.shape[1 if shape[2] == 1 else 2] == -(-n // 32)
    v = R.values(codes, scales)
    step = R.two_to(scales.reshape(-1, -(-n // 32)).int() - 127).repeat_interleave(32, 1)[:, :n]
    assert ((R.rows_of(v) - R.rows_of(x.double())).abs() <= step / 2).all()
    again = R.values(*R.pack(v))
    assert torch.equal(again, v)
