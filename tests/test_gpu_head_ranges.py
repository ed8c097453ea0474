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


@pytest.mark.parametrize("tokens", [5, 128, 129, 400])
@pytest.mark.parametrize("gap", [3.0, 9.0, 14.0, 30.0])
def test_cross_entropy_gradients_of_sure_tokens(nq, tokens, gap):
    """Tokens whose label's logit is `gap` above what the others add up to, so that p - 1 is a small
    difference: the gradients are within the bound that the header states (which is checked as
    stated, with p from the lse that the forward gave), and so are those of hopeless tokens."""
    vocab, d = 500, 256
    g = torch.Generator(device="cuda").manual_seed(31)
    W = (torch.randn(vocab, d, device="cuda", generator=g) / 16).bfloat16()
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    h = (W[labels.long()].float() * gap * 2 + torch.randn(tokens, d, device="cuda", generator=g) * 0.3).bfloat16()
    labels[1::4] = (labels[1::4] + 1) % vocab  # hopeless
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    _, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    hd, Wd, dl = h.double(), W.double(), dloss.double()[:, None]
    z = hd @ Wd.T
    ez = (d / 16 + 16) * U * (hd.abs() @ Wd.abs().T)
    p = torch.exp(z - lse.double()[:, None])
    dz = p * dl
    dz[torch.arange(tokens, device="cuda"), labels.long()] -= dl[:, 0]
    r = 2.0 ** -16 if tokens <= 128 else 2.0 ** -8
    edz = r * dz.abs() + dl * (p * (2 * ez + 2.0 ** -18) + 2.0 ** -23)
    for got, e, x, b, terms in ((dh, edz, dz, Wd, vocab), (dW, edz.T, dz.T, hd, tokens)):
        ref = x @ b
        bound = e @ b.abs() + (terms / 8 + 32) * U * (x.abs() @ b.abs()) + BF * ref.abs()
        assert torch.all((got.double() - ref).abs() <= bound * (1 + 2.0 ** -6) + 1e-38)


def test_cross_entropy_head_past_four_gigabytes(nq):
    """A head, and its gradient, of more than 2^32 bytes: classes at both ends."""
    tokens, vocab, d = 20, 1 << 20, 2056
    g = torch.Generator(device="cuda").manual_seed(32)
    W = torch.empty(vocab, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g) * (1.0 / 64)
    h = torch.randn(tokens, d, device="cuda", generator=g).bfloat16()
    labels = torch.tensor([0, 1, vocab - 1, vocab - 2, vocab // 2, -100] + [vocab - 3] * 14, device="cuda", dtype=torch.int32)
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    hd, dl = h.double(), torch.where(labels >= 0, dloss, 0.0).double()[:, None]
    total = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    want = torch.zeros(tokens, d, dtype=torch.float64, device="cuda")
    slack = torch.zeros_like(want)
    worst = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    for v0 in range(0, vocab, 1 << 16):
        Wd = W[v0:v0 + (1 << 16)].double()
        z = hd @ Wd.T
        total += z.exp().sum(1)
        ez = (d / 16 + 16) * U * (hd.abs() @ Wd.abs().T)
        worst = torch.maximum(worst, ez.amax(1))
        p = torch.exp(z - lse.double()[:, None])
        dz = p * dl
        for i, v in enumerate(labels.tolist()):
            if v0 <= v < v0 + (1 << 16):
                dz[i, v - v0] -= dl[i, 0]
        edz = 2.0 ** -16 * dz.abs() + dl * (p * (2 * ez + 2.0 ** -18) + 2.0 ** -23 * (dz < 0))
        want += dz @ Wd
        slack += edz @ Wd.abs() + (vocab / 8 + 32) * U * (dz.abs() @ Wd.abs())
        if v0 in (0, vocab // 2, vocab - (1 << 16)):
            ref = dz.T @ hd
            bound = edz.T @ hd.abs() + (tokens / 8 + 32) * U * (dz.T.abs() @ hd.abs()) + BF * ref.abs()
            assert torch.all((dW[v0:v0 + (1 << 16)].double() - ref).abs() <= bound * (1 + 2.0 ** -6) + 1e-38)
    ref = total.log()
    assert torch.all((lse.double() - ref).abs() <= worst + (vocab / 32 + 64 + ref.abs()) * U)
    assert torch.all((dh.double() - want).abs() <= (slack + BF * want.abs()) * (1 + 2.0 ** -6) + 1e-38)


def test_cross_entropy_tokens_past_four_gigabytes(nq):
    """Hidden states, and their gradient, of more than 2^32 bytes: tokens at both ends."""
    tokens, vocab, d = 270000, 300, 8200
    g = torch.Generator(device="cuda").manual_seed(33)
    h = torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    W = (torch.randn(vocab, d, device="cuda", generator=g) / 64).bfloat16()
    labels = torch.randint(-1, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    dh, _ = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss, need_dW=False)
    Wd = W.double()
    for at in (0, 131000, 261860, tokens - 300):  # (2^31 elements are passed in row 261888)
        rows = slice(at, at + 300)
        hd, counted = h[rows].double(), labels[rows] >= 0
        dl = torch.where(counted, dloss[rows], 0.0).double()[:, None]
        z = hd @ Wd.T
        ez = (d / 16 + 16) * U * (hd.abs() @ Wd.abs().T)
        ref = torch.logsumexp(z, 1)
        off = ez.amax(1) + (vocab / 32 + 64 + ref.abs()) * U
        assert torch.all((lse[rows].double() - ref).abs() <= off)
        picked = z.gather(1, labels[rows].clamp_min(0).long()[:, None])[:, 0]
        want = torch.where(counted, ref - picked, 0.0)
        assert torch.all((loss[rows].double() - want).abs() <= 2 * off + U * picked.abs())
        p = torch.exp(z - lse[rows].double()[:, None])
        dz = p * dl
        dz[torch.arange(300, device="cuda")[counted], labels[rows][counted].long()] -= dl[counted, 0]
        edz = 2.0 ** -8 * dz.abs() + dl * (p * (2 * ez + 2.0 ** -18) + 2.0 ** -23)
        ref = dz @ Wd
        bound = edz @ Wd.abs() + (vocab / 8 + 32) * U * (dz.abs() @ Wd.abs()) + BF * ref.abs()
        assert torch.all((dh[rows].double() - ref).abs() <= bound * (1 + 2.0 ** -6) + 1e-38)


@pytest.mark.parametrize("tokens,vocab,d,kind", [
    (129, 1, 8, "even"), (129, 700, 72, "even"), (200, 5, 264, "even"), (256, 32, 1000, "one"), (257, 1000, 64, "even"),
    (300, 40, 136, "even"), (600, 40, 520, "even"), (600, 5000, 200, "some"), (1000, 3001, 256, "some"), (2050, 700, 136, "even"),
    (1100, 300, 264, "one"), (4100, 40000, 64, "some"), (3000, 257, 1032, "few")])
def test_cross_entropy_labels_are_kept_apart(nq, tokens, vocab, d, kind):
    """Above 128 tokens dz is bfloat16 but at the labels, whose rest is added in fp32 (off by 2^-24 of the
    entry beside the logits' error): to dh each token's own, to dW those of a class's tokens, none, a few,
    or more than are kept in registers (4) and than are looked for at a time (32)."""
    g = torch.Generator(device="cuda").manual_seed(41)
    h = torch.randn(tokens, d, device="cuda", generator=g).bfloat16()
    W = (torch.randn(vocab, d, device="cuda", generator=g) * (1.6 / d ** 0.5)).bfloat16()
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    if kind == "some":  # classes of one, two, ... tokens beside each other
        labels[: tokens // 4] = labels[: tokens // 4] % 20
    if kind == "few":  # three classes far apart
        labels = torch.tensor([0, vocab // 2, vocab - 1], device="cuda", dtype=torch.int32)[labels % 3]
    if kind == "one":
        labels[:] = vocab - 1
    labels[3::11] = -100
    labels[5::13] = vocab  # do not count either
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    counted = (labels >= 0) & (labels < vocab)
    hd, Wd = h.double(), W.double()
    dl = torch.where(counted, dloss, 0.0).double()[:, None]
    z = hd @ Wd.T
    ez = (d / 16 + 16) * U * (hd.abs() @ Wd.abs().T)
    p = torch.exp(z - lse.double()[:, None])
    dz = p * dl
    rows = torch.arange(tokens, device="cuda")[counted]
    at = labels[counted].long()
    dz[rows, at] -= dl[counted, 0]
    stored = 2.0 ** -8 * dz.abs()
    stored[rows, at] = 2.0 ** -23 * dz[rows, at].abs()
    edz = stored + dl * (p * (2 * ez + 2.0 ** -18) + 2.0 ** -23)
    for got, e, x, b, terms in ((dh, edz, dz, Wd, vocab), (dW, edz.T, dz.T, hd, tokens)):
        ref = x @ b
        bound = e @ b.abs() + (terms / 8 + 32) * U * (x.abs() @ b.abs()) + BF * ref.abs()
        assert torch.all((got.double() - ref).abs() <= bound * (1 + 2.0 ** -6) + 1e-38)
    alone, none = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss, need_dW=False)
    assert torch.equal(alone, dh)
    none, alone = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss, need_dh=False)
    assert torch.equal(alone, dW)


@pytest.mark.parametrize("tokens,vocab,d", [(129, 2000, 512), (300, 5003, 520), (1000, 3001, 1024), (2050, 700, 136)])
def test_cross_entropy_gradients_lose_little_beside_their_rounding(nq, tokens, vocab, d):
    """dh's and dW's relative error in the norm: that of rounding them to bfloat16 (below 2^-9, about 0.29 of a
    step of 2^-7, as errors spread evenly) and little more, since what bfloat16 dz adds is its classes'
    beside the labels': below 2^-8 sqrt(sum p^2) of the norm, with sum p^2 of these logits below 0.05."""
    g = torch.Generator(device="cuda").manual_seed(42)
    h = torch.randn(tokens, d, device="cuda", generator=g).bfloat16()
    W = (torch.randn(vocab, d, device="cuda", generator=g) * (1.6 / d ** 0.5)).bfloat16()
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.5
    _, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    got = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    p = torch.softmax(h.double() @ W.double().T, 1)
    assert float((p * p).sum(1).mean()) < 0.05
    dz = p * dloss.double()[:, None]
    dz[torch.arange(tokens, device="cuda"), labels.long()] -= dloss.double()
    for x, ref in zip(got, (dz @ W.double(), dz.T @ h.double())):
        rounded = (ref.bfloat16().double() - ref).norm()
        assert float((x.double() - ref).norm()) <= float(1.1 * rounded + 2.0 ** -8 * 0.05 ** 0.5 * 0.5 * ref.norm())


@pytest.mark.parametrize("tokens,kept", [(262144, True), (262400, False)])
def test_cross_entropy_many_tokens_of_few_classes(nq, tokens, kept):
    """dW of so many tokens per class: up to 2^18 of them dz is two parts (off by 2^-16), beyond it is one."""
    vocab, d = 100, 16
    g = torch.Generator(device="cuda").manual_seed(43)
    h = torch.randn(tokens, d, device="cuda", generator=g).bfloat16()
    W = torch.randn(vocab, d, device="cuda", generator=g).bfloat16()
    labels = torch.randint(-1, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    _, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    hd, Wd = h.double(), W.double()
    dl = torch.where(labels >= 0, dloss, 0.0).double()[:, None]
    z = hd @ Wd.T
    ez = (d / 16 + 16) * U * (hd.abs() @ Wd.abs().T)
    p = torch.exp(z - lse.double()[:, None])
    dz = p * dl
    rows = torch.arange(tokens, device="cuda")[labels >= 0]
    at = labels[rows].long()
    dz[rows, at] -= dl[rows, 0]
    stored = 2.0 ** -8 * dz.abs()
    stored[rows, at] = 2.0 ** -16 * dz[rows, at].abs()
    other = dl * (p * (2 * ez + 2.0 ** -18) + 2.0 ** -23)
    for got, e, x, b, terms in ((dh, stored + other, dz, Wd, vocab),
                                (dW, ((2.0 ** -16 if kept else 2.0 ** -8) * dz.abs() + other).T, dz.T, hd, tokens)):
        ref = x @ b
        bound = e @ b.abs() + (terms / 8 + 32) * U * (x.abs() @ b.abs()) + BF * ref.abs()
        assert torch.all((got.double() - ref).abs() <= bound * (1 + 2.0 ** -6) + 1e-38)


@pytest.mark.parametrize("tokens,vocab", [(20, 300), (128, 300), (200, 1000), (200, 100), (600, 2000), (600, 500)])
def test_cross_entropy_of_an_infinite_weight(nq, tokens, vocab):
    """A token whose weight is infinite: its dz is infinite, +inf or -inf at its label, and dW what that times
    its h is, not NaN (a second part of dz has nothing of an infinity); the other tokens' dh are as without it."""
    d = 72
    g = torch.Generator(device="cuda").manual_seed(44)
    h = torch.randn(tokens, d, device="cuda", generator=g).bfloat16()
    W = (torch.randn(vocab, d, device="cuda", generator=g) * 0.1).bfloat16()
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    labels[5] = 7
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    _, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    plain, _ = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    dloss[5] = float("inf")
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    sign = torch.ones(vocab, device="cuda")
    sign[7] = -1.0
    assert torch.all(h[5] != 0)
    assert torch.equal(dW.float(), sign[:, None] * h[5].float()[None, :] * float("inf"))
    others = torch.arange(tokens, device="cuda") != 5
    assert torch.equal(dh[others], plain[others])
