"""Ranges of the output head's inputs on the GPU: activations of 4-bit products from the smallest to the
largest bfloat16 numbers, and buffers of the cross entropy past 2^32 bytes.

4-bit products: (48 + n / 32) u of sum |s| (c + |z|) |x|, u = 2^-23 (24 accumulator steps in a group, 3 to
apply zero point and scale, n / 32 groups, 16 warps to add).  The kernel keeps 2^-16 of every sum, so
that a rounding is at least 2^-150 there, 2^-134 of y: in n / 32 groups of at most 27 of them.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -23
BF = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def nq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from binary_rank_linear_02_b200 import nq as mod

    return mod


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [3.3e38, 1e37, 1e36, 1e20, 1e-20, 1e-30, 1e-36, 1e-39])
def test_q4_activations_of_any_size(nq, size, group, zeros):
    """Whole groups of one sign, so that their sums are as large as they can be, and mixed ones."""
    m, n, batch = 97, 1024, 4
    g = torch.Generator(device="cuda").manual_seed(21)
    codes = torch.randint(0, 16, (m, n), device="cuda", generator=g, dtype=torch.uint8)
    scales = ((torch.rand(m, n // group, device="cuda", generator=g) + 0.5) * (2.0 ** -14 if size > 1 else 4.0)).half()
    z = (torch.rand(m, n // group, device="cuda", generator=g) * 15).half() if zeros else None
    x = (torch.rand(batch, n, device="cuda", generator=g) * size).bfloat16()
    x[1] = size
    x[2, ::2] *= -1
    x[3, 1::3] = 0.0
    assert torch.isfinite(x).all()
    y = nq.q4_linear_fwd(x, nq.pack_q4(codes), scales, m, n, group, zeros=z)
    c = codes.double()
    zz = z.double().repeat_interleave(group, 1) if zeros else torch.full_like(c, 8.0)
    s = scales.double().repeat_interleave(group, 1)
    ref = x.double() @ ((c - zz) * s).T
    mag = x.double().abs() @ ((c + zz) * s).T
    assert torch.all(ref.abs() < 3e38)
    assert torch.all((y.double() - ref).abs() <= (48 + n / 32) * U * mag + n / 32 * 27 * 2.0 ** -134 * 4.0)
