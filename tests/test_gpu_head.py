"""The output head on the GPU, through the binding, against plain computations in 64 bits:
products with 4-bit weights, the distillation loss against a teacher's top logits with its
gradient, and the cross entropy of a dense head with its gradients.

Tolerances.  u = 2^-23 (a truncated fp32 step; a rounded one is half of it).
  * 4-bit products: exact products c x; 24 accumulator steps within a group (the sum of x takes
    fewer), 3 to apply zero point and scale, at most n / 32 groups and 16 warps to add: with
    sums of c x and of z x taken apart, (48 + n / 32) u of sum |s| (c + |z|) |x| bounds them.
  * distillation: a thread adds V / 512 exponentials one after another, 9 tree steps and a few
    joins follow; an exponential is off by 2 u and by its argument's rounding (|argument| u,
    arguments up to 40 where it matters): the relative error of a sum is below
    (V / 512 + 64) u =: e.  loss: T^2 (2 e + u |loss| / T^2); gradient: 3 e of
    dloss T (p (sum q + q_rest) + q_rest p / p_rest) and u of dloss T q; a bfloat16 result
    half a step more, 2^-8 |dz|.
  * cross entropy: z is off by (d / 16 + 16) u of sum_j |h_j W_vj| =: ez; sums of exponentials
    by (V / 32 + 64) u at most; lse and loss by the largest ez of their row plus that plus
    u (|lse| + |z_label|).  dz: relative 2^-8 (bfloat16) + 2 ez + 32 u of dloss p; products:
    (terms / 16 + 16) u of the sum of magnitudes; results 2^-8.
"""
import math

import numpy as np
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


# ------------------------------------------------------------------ 4-bit products

def q4_case(m, n, group, batch, zeros, seed):
    g = gen(seed)
    codes = torch.randint(0, 16, (m, n), device="cuda", generator=g, dtype=torch.uint8)
    scales = ((torch.rand(m, n // group, device="cuda", generator=g) + 0.5) * 0.02).half()
    z = (torch.rand(m, n // group, device="cuda", generator=g) * 15).half() if zeros else None
    x = randn(g, batch, n)
    x[:, ::97] *= 300.0
    return codes, scales, z, x.bfloat16()


def q4_check(y, codes, scales, z, x, n, group):
    c = codes.double()
    zz = z.double().repeat_interleave(group, 1) if z is not None else torch.full_like(c, 8.0)
    s = scales.double().repeat_interleave(group, 1)
    ref = x.double() @ ((c - zz) * s).T
    mag = x.double().abs() @ ((c + zz.abs()) * s.abs()).T
    assert torch.all((y.double() - ref).abs() <= (48 + n / 32) * U * mag)


Q4_SHAPES = [
    (1, 128, 32, 1, False), (1, 128, 128, 2, True), (16, 128, 64, 1, True), (17, 256, 64, 8, True),
    (15, 384, 128, 3, False), (513, 384, 32, 9, True), (512, 512, 128, 1, False), (33, 640, 64, 17, False),
    (100, 8192, 32, 3, True), (2049, 1152, 32, 1, True), (4096, 4096, 128, 8, False), (32001, 512, 64, 2, True),
    (28672, 1024, 128, 5, True), (260, 2176, 128, 16, True),
    (301, 1408, 128, 4, True), (77, 11008, 128, 2, True), (53, 2176, 64, 3, False), (95, 2176, 32, 1, True),
    (300, 8320, 32, 8, True), (3000, 28672, 64, 8, True), (70, 28672, 32, 3, False), (5000, 66048, 128, 1, True),
]


@pytest.mark.parametrize("m,n,group,batch,zeros", Q4_SHAPES)
def test_q4_matches_reference(nq, m, n, group, batch, zeros):
    codes, scales, z, x = q4_case(m, n, group, batch, zeros, 1000 + m + n)
    y = nq.q4_linear_fwd(x, nq.pack_q4(codes), scales, m, n, group, zeros=z)
    assert y.shape == (batch, m)
    q4_check(y, codes, scales, z, x, n, group)


# Matrices of an odd number of 128-column blocks beside even ones, several tiles of a narrow one to
# a stage, one, three and four stages a tile with the last one full, half full and of a single block.
Q4_BLOCKS = [
    (40, 128, 64, 8, True), (4800, 128, 32, 8, True), (5000, 384, 32, 2, True), (2500, 896, 128, 4, False),
    (700, 2048, 64, 1, True), (333, 4224, 128, 1, False), (650, 6272, 64, 8, True), (2400, 1920, 32, 7, False),
]


@pytest.mark.parametrize("m,n,group,batch,zeros", Q4_BLOCKS)
def test_q4_blocks_of_a_stage(nq, m, n, group, batch, zeros):
    codes, scales, z, x = q4_case(m, n, group, batch, zeros, 4000 + m + n)
    w = nq.pack_q4(codes)
    y = nq.q4_linear_fwd(x, w, scales, m, n, group, zeros=z)
    q4_check(y, codes, scales, z, x, n, group)
    assert torch.equal(y, nq.q4_linear_fwd(x, w, scales, m, n, group, zeros=z))


def test_q4_pack_device_equals_host(nq):
    codes = torch.randint(0, 16, (37, 133), device="cuda", generator=gen(5), dtype=torch.uint8)
    got = nq.pack_q4(codes)
    assert np.array_equal(got.cpu().numpy().view(np.uint32), nq.pack_q4(codes.cpu().numpy()))
    codes[36, 132] = 16
    with pytest.raises(nq.NQError) as e:
        nq.pack_q4(codes)
    assert e.value.status == nq.NQ_ERR_VALUE


def test_q4_tokens_do_not_touch_each_other(nq):
    """Each token alone gives the same bits, beside tokens of NaN and infinity too; repeats agree."""
    m, n, group = 300, 1280, 64
    codes, scales, z, x = q4_case(m, n, group, 8, True, 7)
    w = nq.pack_q4(codes)
    y = nq.q4_linear_fwd(x, w, scales, m, n, group, zeros=z)
    assert torch.equal(y, nq.q4_linear_fwd(x, w, scales, m, n, group, zeros=z))
    x2 = x.clone()
    x2[1] = float("nan")
    x2[6] = float("inf")
    y2 = nq.q4_linear_fwd(x2, w, scales, m, n, group, zeros=z)
    for b in range(8):
        assert torch.equal(nq.q4_linear_fwd(x[b], w, scales, m, n, group, zeros=z)[0], y[b])
        if b not in (1, 6):
            assert torch.equal(y2[b], y[b])
    assert not torch.isfinite(y2[1]).any()


def test_q4_writes_its_rows_only(nq):
    m, n, group, batch = 77, 256, 32, 3
    codes, scales, z, x = q4_case(m, n, group, batch, False, 8)
    whole = torch.full((batch + 2, m), 7.0, device="cuda")
    nq.q4_linear_fwd(x, nq.pack_q4(codes), scales, m, n, group, y=whole[:batch])
    assert torch.all(whole[batch:] == 7.0)
    q4_check(whole[:batch], codes, scales, z, x, n, group)


def test_q4_codes_past_four_gigabytes(nq):
    """The last rows of a matrix whose codes pass 2^32 bytes."""
    m, n, group = 140000, 65536, 128
    w = torch.randint(-(1 << 31), 1 << 31, (m, n // 8), device="cuda", generator=gen(9), dtype=torch.int32)
    scales = ((torch.rand(m, n // group, device="cuda", generator=gen(10)) + 0.5) * 0.02).half()
    x = randn(gen(11), 2, n).bfloat16()
    y = nq.q4_linear_fwd(x, w, scales, m, n, group)
    rows = torch.tensor([0, 1, 65535, 131071, 131072, m - 2, m - 1], device="cuda")
    codes = ((w[rows][:, :, None] >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).reshape(len(rows), n)
    q4_check(y[:, rows], codes, scales[rows], None, x, n, group)


# ------------------------------------------------------------------ distillation

def distill_reference(logits, ids, teacher, lse, vocab, t, dloss):
    """Loss and gradient from the definitions, 64 bits; also the magnitude that the gradient's
    error is measured by."""
    z = logits[:, :vocab].double() / t
    tokens, k = ids.shape
    loss = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    grad = torch.zeros_like(z)
    mag = torch.zeros_like(z)
    for i in range(tokens):
        ok = (ids[i] >= 0) & (ids[i] < vocab)
        if not ok.any():
            continue
        at, u = ids[i][ok].long(), teacher[i][ok].double() / t
        logq = u - (lse[i].double() if lse is not None else torch.logsumexp(u, 0))
        q = logq.exp()
        logp = torch.log_softmax(z[i], 0)
        p = logp.exp()
        live = q > 0
        loss[i] = (q[live] * (logq[live] - logp[at][live])).sum()
        out = torch.ones(vocab, dtype=torch.bool, device="cuda")
        out[at] = False
        dq = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, at, q)
        rest = torch.zeros((), dtype=torch.float64, device="cuda")
        share = torch.zeros_like(p)
        if lse is not None and out.any() and torch.isfinite(z[i][out]).any():
            rest = (1 - q.sum()).clamp_min(0)
            log_rest = torch.logsumexp(logp[out], 0)
            if rest > 0:
                loss[i] += rest * (rest.log() - log_rest)
            share = torch.where(out, (logp - log_rest).exp() * rest, torch.zeros_like(p))
        tot = q.sum() + rest
        grad[i] = dloss[i].double() * t * (p * tot - dq - share)
        mag[i] = dloss[i].double().abs() * t * (p * tot + share + dq)
    return loss * t * t, grad, mag


def distill_case(tokens, vocab, pitch, k, rest, t, dtype, seed, spread=2.5):
    g = gen(seed)
    full = torch.zeros(tokens, pitch, device="cuda")
    full[:, :vocab] = randn(g, tokens, vocab) * spread
    if pitch > vocab:
        full[:, vocab:] = float("nan")  # what lies behind a row's classes is not read
    logits = full.to(dtype)
    teacher = full[:, :vocab] + randn(g, tokens, vocab)
    top, ids = torch.topk(teacher, k, dim=1)
    lse = torch.logsumexp(teacher.double() / t, 1).float() if rest else None
    ids = ids.int()
    for i in range(0, tokens, 3):  # fewer entries in some rows, none in the first
        ids[i, (i * 5) % (k + 1):] = -1
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    return logits, ids.contiguous(), top.contiguous(), lse, dloss


def distill_check(nq, logits, ids, teacher, lse, vocab, t, dloss, dtype):
    loss, grad, mag = distill_reference(logits, ids, teacher, lse, vocab, t, dloss)
    e = (vocab / 512 + 64) * U
    tol = t * t * 2 * e + U * loss.abs()
    got = nq.distill_topk_fwd(logits, ids, teacher, vocab, temperature=t, teacher_lse=lse)
    assert torch.all((got.double() - loss).abs() <= tol)
    dz, loss2 = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=dtype)
    assert torch.all((loss2.double() - loss).abs() <= tol)
    assert dz.dtype == dtype and dz.shape == logits.shape
    half = BF if dtype == torch.bfloat16 else U
    assert torch.all((dz[:, :vocab].double() - grad).abs() <= 3 * e * mag + half * grad.abs() + 1e-38)
    assert torch.all(dz[:, vocab:] == 0)
    return dz, got


DISTILL = [
    (1, 1, 1, 1, False, 1.0), (2, 7, 7, 3, True, 2.0), (3, 8, 16, 8, True, 1.0), (3, 9, 9, 1, False, 4.0),
    (5, 100, 101, 20, True, 0.5), (4, 1001, 1001, 64, False, 1.0), (7, 4099, 4224, 50, True, 2.0),
    (5, 32000, 32000, 256, True, 1.0), (4, 50257, 50304, 33, False, 2.0), (3, 128001, 128001, 1024, True, 1.5),
    (2, 262144, 262144, 8, True, 1.0), (300, 515, 515, 5, True, 1.0), (2, 1 << 20, 1 << 20, 9, True, 1.0),
    (200, 20003, 20003, 7, False, 1.0), (160, 70001, 70001, 11, True, 2.0),
]


@pytest.mark.parametrize("tokens,vocab,pitch,k,rest,t", DISTILL)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_distill_matches_reference(nq, tokens, vocab, pitch, k, rest, t, dtype, grad):
    case = distill_case(tokens, vocab, pitch, k, rest, t, dtype, 2000 + vocab)
    logits, ids, teacher, lse, dloss = case
    distill_check(nq, logits, ids, teacher, lse, vocab, t, dloss, grad)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_gradient_against_differences(nq, rest):
    """The kernel's gradient along a direction against central differences of the 64-bit loss:
    the third derivative of the loss is of order 1, so steps of 1e-4 leave about 1e-8."""
    t, vocab = 2.0, 513
    logits, ids, teacher, lse, dloss = distill_case(6, vocab, vocab, 12, rest, t, torch.float32, 31)
    dz, _ = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=torch.float32)
    way = randn(gen(32), 6, vocab).double()
    step = 1e-4
    up = distill_reference(logits.double() + step * way, ids, teacher, lse, vocab, t, dloss)[0]
    down = distill_reference(logits.double() - step * way, ids, teacher, lse, vocab, t, dloss)[0]
    want = dloss.double() * (up - down) / (2 * step)
    got = (dz.double() * way).sum(1)
    scale = (dz.double() * way).abs().sum(1)
    assert torch.all((got - want).abs() <= 1e-6 + 3e-5 * scale)


def test_distill_rows_without_entries(nq):
    """No entry (-1, ids out of range): loss 0 and gradient 0, whatever the logits hold."""
    vocab = 300
    logits = torch.full((4, vocab), float("nan"), device="cuda")
    logits[1] = float("inf")
    logits[2] = float("-inf")
    logits[3] = 1.0
    ids = torch.tensor([[-1, -1], [vocab, 1 << 30], [-(1 << 31), -5], [-1, vocab]], dtype=torch.int32, device="cuda")
    teacher = torch.full((4, 2), float("nan"), device="cuda")
    for lse in (None, torch.zeros(4, device="cuda")):
        assert torch.all(nq.distill_topk_fwd(logits, ids, teacher, vocab, teacher_lse=lse) == 0)
        dz, loss = nq.distill_topk_bwd(logits, ids, teacher, vocab, torch.ones(4, device="cuda"), teacher_lse=lse,
                                       dtype=torch.float32)
        assert torch.all(loss == 0) and torch.all(dz == 0)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_masked_and_extreme_logits(nq, rest):
    """Classes masked with -inf or the type's lowest value, logits near the top of the range,
    rows in which one class has all the mass, teacher entries of -inf, absent entries of NaN."""
    t, vocab, k = 1.0, 777, 6
    for dtype in (torch.float32, torch.bfloat16):
        logits, ids, teacher, lse, dloss = distill_case(9, vocab, vocab, k, rest, t, dtype, 41)
        ids[:] = torch.topk(logits.float(), k, dim=1).indices.int()
        logits[1, 400:] = float("-inf")
        ids[1] = torch.tensor([1, 2, 3, 30, 200, 399], device="cuda", dtype=torch.int32)
        logits[2, 100:500] = torch.finfo(dtype).min
        ids[2] = torch.tensor([1, 2, 3, 30, 99, 600], device="cuda", dtype=torch.int32)
        logits[3] += 3000.0
        logits[4, 5] = 200.0
        ids[4, 0] = 5
        ids[4, 1:] = torch.tensor([6, 7, 8, 9, 10], device="cuda", dtype=torch.int32)
        teacher[5, 2] = float("-inf")
        ids[6, 3] = -1
        teacher[6, 3] = float("nan")
        logits[7] = 0.25
        dz, _ = distill_check(nq, logits, ids, teacher, lse, vocab, t, dloss, torch.float32)
        assert torch.all(dz[1, 400:] == 0)


def test_distill_listed_twice_and_whole_vocabulary(nq):
    """An id listed again adds its mass; a list that names every class leaves no rest."""
    vocab, k = 40, 40
    logits, ids, teacher, lse, dloss = distill_case(4, vocab, vocab, k, True, 1.0, torch.float32, 43)
    ids[:] = torch.arange(vocab, device="cuda", dtype=torch.int32)
    teacher[:] = randn(gen(44), 4, k)
    lse = torch.logsumexp(teacher.double(), 1).float()
    distill_check(nq, logits, ids, teacher, lse, vocab, 1.0, dloss, torch.float32)
    ids[1] = ids[1] // 2  # every class twice, half of them never
    ids[2] = 7            # one class forty times
    ids[3, 20:] = ids[3, :20]
    distill_check(nq, logits, ids, teacher, lse + 0.5, vocab, 1.0, dloss, torch.float32)
    distill_check(nq, logits, ids, teacher, None, vocab, 1.0, dloss, torch.float32)


def test_distill_repeats_bit_for_bit_and_per_row(nq):
    logits, ids, teacher, lse, dloss = distill_case(33, 5003, 5003, 40, True, 2.0, torch.float32, 47)
    ids[5, 10:20] = ids[5, 0]
    a = nq.distill_topk_bwd(logits, ids, teacher, 5003, dloss, temperature=2.0, teacher_lse=lse)
    b = nq.distill_topk_bwd(logits, ids, teacher, 5003, dloss, temperature=2.0, teacher_lse=lse)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_distill_past_four_billion_elements(nq):
    """Rows whose offset passes 2^32 elements."""
    tokens, vocab, k = 33600, 128000, 4
    logits = torch.zeros(tokens, vocab, dtype=torch.bfloat16, device="cuda")
    last = [0, 16777, 33554, 33555, tokens - 1]
    for i in last:
        logits[i] = randn(gen(50 + i), vocab).bfloat16()
    ids = torch.randint(0, vocab, (tokens, k), device="cuda", generator=gen(48), dtype=torch.int32)
    teacher = randn(gen(49), tokens, k)
    dloss = torch.ones(tokens, device="cuda")
    dz, loss = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss)
    ref, grad, mag = distill_reference(logits[last], ids[last], teacher[last], None, vocab, 1.0, dloss[last])
    e = (vocab / 512 + 64) * U
    assert torch.all((loss[last].double() - ref).abs() <= 2 * e + U * ref.abs())
    assert torch.all((dz[last].double() - grad).abs() <= 3 * e * mag + BF * grad.abs())


# ------------------------------------------------------------------ cross entropy

def xent_case(tokens, vocab, d, seed, spread=1.6):
    g = gen(seed)
    h = randn(g, tokens, d).bfloat16()
    W = (randn(g, vocab, d) * (spread / math.sqrt(d))).bfloat16()
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    if tokens > 2:
        labels[::5] = -100
        labels[1] = vocab - 1
        labels[2] = 0
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    return h, W, labels, dloss


def xent_check_forward(nq, h, W, labels):
    vocab, d = W.shape
    loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    z = h.double() @ W.double().T
    ez = (d / 16 + 16) * U * (h.double().abs() @ W.double().abs().T)
    ref = torch.logsumexp(z, 1)
    counted = (labels >= 0) & (labels < vocab)
    picked = z.gather(1, torch.where(counted, labels, 0).long()[:, None])[:, 0]
    tol = ez.amax(1) + (vocab / 32 + 64) * U + U * (ref.abs() + picked.abs())
    assert torch.all((lse.double() - ref).abs() <= tol)
    assert torch.all((loss.double() - torch.where(counted, ref - picked, torch.zeros_like(ref))).abs() <= 2 * tol)
    assert torch.all(loss[~counted] == 0)
    return lse, z, ez, counted


def xent_check(nq, h, W, labels, dloss):
    tokens, d = h.shape
    vocab = W.shape[0]
    lse, z, ez, counted = xent_check_forward(nq, h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    dl = torch.where(counted, dloss.double(), 0.0)[:, None]
    p = torch.exp(z - lse.double()[:, None]) * dl
    dz = p.clone()
    rows = torch.arange(tokens, device="cuda")[counted]
    dz[rows, labels[counted].long()] -= dl[counted, 0]
    edz = BF * dz.abs() + (2 * ez + 32 * U) * p.abs() + U * dl.abs()
    Wd, hd = W.double(), h.double()
    ref = dz @ Wd
    bound = edz @ Wd.abs() + (vocab / 16 + 16) * U * (dz.abs() @ Wd.abs()) + BF * ref.abs() * (1 + BF) + BF * (edz @ Wd.abs())
    assert dh.shape == h.shape and dh.dtype == torch.bfloat16
    assert torch.all((dh.double() - ref).abs() <= bound + 1e-38)
    ref = dz.T @ hd
    bound = edz.T @ hd.abs() + (tokens / 16 + 16) * U * (dz.abs().T @ hd.abs()) + BF * ref.abs() * (1 + BF) + BF * (edz.T @ hd.abs())
    assert dW.shape == W.shape and dW.dtype == torch.bfloat16
    assert torch.all((dW.double() - ref).abs() <= bound + 1e-38)
    return lse, dh, dW


XENT = [
    (1, 1, 8), (1, 2, 64), (2, 100, 72), (3, 127, 16), (127, 128, 64), (128, 129, 128), (129, 1000, 200),
    (64, 257, 512), (255, 511, 264), (257, 513, 1000), (300, 5003, 520), (1, 32000, 4096), (8, 50257, 1024),
    (1000, 3001, 2048), (2050, 700, 136),
]


@pytest.mark.parametrize("tokens,vocab,d", XENT)
def test_cross_entropy_matches_reference(nq, tokens, vocab, d):
    xent_check(nq, *xent_case(tokens, vocab, d, 3000 + tokens + vocab + d))
    nq.device_status()


# Sums over d in one part, two and three; K blocks fewer than a tile's accumulators (up to 64
# tokens four, up to 128 two); last column tiles of 1, 128, 129 and 255 classes, with labels in them.
XENT_PARTS = [
    (257, 385, 3008), (300, 513, 3136), (385, 767, 5200), (17, 300, 8), (40, 513, 136), (64, 130, 1040), (65, 700, 72),
    (128, 257, 264), (144, 260, 64), (270, 128, 8),
]


@pytest.mark.parametrize("tokens,vocab,d", XENT_PARTS)
def test_cross_entropy_parts_of_a_sum(nq, tokens, vocab, d):
    h, W, labels, dloss = xent_case(tokens, vocab, d, 5000 + tokens + vocab + d)
    labels[4] = vocab - 1 - (vocab - 1) % 128  # the first class of the last half tile
    xent_check(nq, h, W, labels, dloss)
    nq.device_status()


@pytest.mark.parametrize("tokens,vocab,d", [(1, 1000, 64), (3, 129, 8), (8, 5003, 520), (16, 513, 264), (17, 257, 1000),
                                            (64, 300, 128), (65, 513, 72), (127, 1000, 264), (128, 700, 136)])
def test_cross_entropy_few_tokens_round_once(nq, tokens, vocab, d):
    """Up to 128 tokens dz passes through two bf16 parts: what the first leaves, at most BF of dz, is
    rounded to the second, so dz is off by BF^2 of itself; the fp32 sums have the terms of both."""
    h, W, labels, dloss = xent_case(tokens, vocab, d, 6000 + tokens + vocab + d)
    lse, z, ez, counted = xent_check_forward(nq, h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    dl = torch.where(counted, dloss.double(), 0.0)[:, None]
    p = torch.exp(z - lse.double()[:, None]) * dl
    dz = p.clone()
    rows = torch.arange(tokens, device="cuda")[counted]
    dz[rows, labels[counted].long()] -= dl[counted, 0]
    edz = BF * BF * dz.abs() + (2 * ez + 32 * U) * p.abs() + U * dl.abs()
    for got, a, b, terms in ((dh, (edz, dz), W.double(), vocab), (dW, (edz.T, dz.T), h.double(), tokens)):
        ref = a[1] @ b
        before = a[0] @ b.abs() + (terms / 8 + 32) * U * (1 + 2 * BF) * (a[1].abs() @ b.abs())
        assert torch.all((got.double() - ref).abs() <= before * (1 + BF) + BF * ref.abs() + 1e-38)


def test_cross_entropy_more_than_one_piece(nq):
    """dz of 4100 tokens and 40000 classes does not fit its scratch: the vocabulary in pieces."""
    assert nq.lib().nq_linear_cross_entropy_scratch_bytes(4100, 40000, 64, 1) < 2 * 4100 * 40000
    xent_check(nq, *xent_case(4100, 40000, 64, 61))


def test_cross_entropy_large_logits(nq):
    """Logits of some hundreds: the maximum is taken out, confident and hopeless tokens both."""
    xent_check(nq, *xent_case(70, 900, 256, 62, spread=90.0))


def test_cross_entropy_gradient_against_differences(nq):
    """dh along a direction against central differences of the 64-bit loss (dh is bfloat16:
    2^-8 of the terms' magnitudes, twice)."""
    h, W, labels, dloss = xent_case(40, 333, 96, 63)
    _, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    counted = labels >= 0

    def total(hd, Wd):
        logp = torch.log_softmax(hd @ Wd.T, 1)
        picked = logp.gather(1, labels.clamp_min(0).long()[:, None])[:, 0]
        return -(picked * dloss.double() * counted).sum()

    hd, Wd, step = h.double(), W.double(), 1e-4
    for seed, which in ((64, "h"), (65, "W")):
        way = randn(gen(seed), *(h.shape if which == "h" else W.shape)).double()
        at = (lambda s: total(hd + s * way, Wd)) if which == "h" else (lambda s: total(hd, Wd + s * way))
        want = (at(step) - at(-step)) / (2 * step)
        got = ((dh if which == "h" else dW).double() * way)
        assert abs(float(got.sum() - want)) <= 2 * BF * float(got.abs().sum()) * 2 + 1e-6


def test_cross_entropy_no_token_counts(nq):
    h, W, labels, dloss = xent_case(50, 300, 64, 66)
    for label in (-100, 300, 1 << 30):
        labels[:] = label
        loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
        assert torch.all(loss == 0) and torch.isfinite(lse).all()
        dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, torch.full_like(dloss, float("nan")))
        assert torch.all(dh == 0) and torch.all(dW == 0)


def test_cross_entropy_no_tokens(nq):
    W = randn(gen(67), 10, 64).bfloat16()
    h = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    labels = torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty(0, device="cuda")
    loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    assert loss.shape == lse.shape == (0,)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, e, e)
    assert dh.shape == (0, 64) and torch.all(dW == 0)


def test_cross_entropy_one_gradient_alone_and_repeats(nq):
    h, W, labels, dloss = xent_case(200, 1500, 320, 68)
    loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss)
    a, none = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss, need_dW=False)
    assert none is None and torch.equal(a, dh)
    none, b = nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss, need_dh=False)
    assert none is None and torch.equal(b, dW)
    again = nq.linear_cross_entropy_fwd(h, W, labels)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


def test_cross_entropy_small_scratch_is_refused(nq):
    h, W, labels, dloss = xent_case(20, 200, 64, 69)
    L = nq.lib()
    loss = torch.zeros(20, device="cuda")
    need = L.nq_linear_cross_entropy_scratch_bytes(20, 200, 64, 0)
    scratch = torch.zeros(need, dtype=torch.uint8, device="cuda")
    f = L.nq_linear_cross_entropy_fwd
    args = [t.data_ptr() for t in (h, W, labels)] + [20, 200, 64, loss.data_ptr(), loss.data_ptr(), scratch.data_ptr()]
    assert f(*args, need - 1, 0) == nq.NQ_ERR_NOMEM
    assert torch.all(loss == 0)


# ------------------------------------------------------------------ streams, graphs

def test_head_on_two_streams_at_once(nq):
    """The head's calls share no workspace: two streams at the same time give what one gives."""
    cases = [(xent_case(300, 4000, 512, 70 + i), q4_case(2000, 1024, 64, 4, True, 72 + i),
              distill_case(64, 9000, 9000, 16, True, 2.0, torch.float32, 74 + i)) for i in range(2)]

    def go(case):
        (h, W, labels, dl), (codes, scales, z, x), (logits, ids, teacher, tl, dloss) = case
        w = case_packed[id(case)]
        loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
        dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dl)
        y = nq.q4_linear_fwd(x, w, scales, 2000, 1024, 64, zeros=z)
        dz, dist = nq.distill_topk_bwd(logits, ids, teacher, 9000, dloss, temperature=2.0, teacher_lse=tl)
        return loss, lse, dh, dW, y, dz, dist

    case_packed = {id(c): nq.pack_q4(c[1][0]) for c in cases}
    alone = [go(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = go(cases[i])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(alone[i], got[i]):
            assert torch.equal(a, b)


def test_head_on_another_stream_than_the_current(nq):
    """A call that is given another stream than the current one, which is busy when it comes: its
    scratch and its results are not the current stream's memory, which is given out and filled
    again while the call still waits."""
    h, W, labels, dl = xent_case(300, 4000, 512, 76)
    codes, scales, z, x = q4_case(2000, 1024, 64, 4, True, 77)
    w = nq.pack_q4(codes)
    logits, ids, teacher, tl, dloss = distill_case(64, 9000, 9000, 16, True, 2.0, torch.float32, 78)

    def go(stream=None):
        loss, lse = nq.linear_cross_entropy_fwd(h, W, labels, stream=stream)
        dh, dW = nq.linear_cross_entropy_bwd(h, W, labels, lse, dl, stream=stream)
        y = nq.q4_linear_fwd(x, w, scales, 2000, 1024, 64, zeros=z, stream=stream)
        dz, dist = nq.distill_topk_bwd(logits, ids, teacher, 9000, dloss, temperature=2.0, teacher_lse=tl, stream=stream)
        return loss, lse, dh, dW, y, dz, dist

    want = go()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = go(side.cuda_stream)
        sizes = [nq.lib().nq_linear_cross_entropy_scratch_bytes(300, 4000, 512, b) for b in (0, 1)]
        filled = [torch.full((s,), 0x7F, dtype=torch.uint8, device="cuda") for s in sizes]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        assert all(torch.all(f == 0x7F) for f in filled)
        del filled


def test_head_on_the_default_stream_from_another(nq):
    """stream=0 names the default stream, whichever is current."""
    h, W, labels, dl = xent_case(60, 700, 128, 79)
    loss, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = nq.linear_cross_entropy_fwd(h, W, labels, stream=0)
        grads = nq.linear_cross_entropy_bwd(h, W, labels, lse, dl, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
    for a, b in zip(grads, nq.linear_cross_entropy_bwd(h, W, labels, lse, dl)):
        assert torch.equal(a, b)


def test_head_in_captured_graphs(nq):
    """Two graphs that hold the head's calls, replayed in turn with new inputs and with larger
    eager calls in between."""
    def step(s):
        loss, lse = nq.linear_cross_entropy_fwd(s["h"], s["W"], s["labels"])
        dh, dW = nq.linear_cross_entropy_bwd(s["h"], s["W"], s["labels"], lse, s["dl"])
        y = nq.q4_linear_fwd(s["x"], s["wq"], s["scales"], 500, 512, 128)
        ids = s["ids"]
        dz, dist = nq.distill_topk_bwd(y, ids, s["teacher"], 500, s["dloss"])
        return loss, lse, dh, dW, y, dz, dist

    def state(seed, tokens):
        h, W, labels, dl = xent_case(tokens, 800, 128, seed)
        codes, scales, _, x = q4_case(500, 512, 128, 4, False, seed + 1)
        ids = torch.randint(0, 500, (4, 6), device="cuda", generator=gen(seed + 2), dtype=torch.int32)
        return dict(h=h, W=W, labels=labels, dl=dl, x=x, wq=nq.pack_q4(codes), scales=scales, ids=ids,
                    teacher=randn(gen(seed + 3), 4, 6), dloss=torch.ones(4, device="cuda"))

    states = [state(80, 130), state(90, 60)]
    graphs, outs = [], []
    for s in states:
        step(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(s))
        graphs.append(graph)
    for turn in range(3):
        for s in states:
            s["h"].copy_(randn(gen(100 + turn), *s["h"].shape).bfloat16())
            s["x"].copy_(randn(gen(200 + turn), *s["x"].shape).bfloat16())
        xent_check(nq, *xent_case(600, 900, 64, 300 + turn))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for s, out in zip(states, outs):
            for a, b in zip(step(s), out):
                assert torch.equal(a, b)


# ------------------------------------------------------------------ together, as they are used

def test_refinement_step_of_a_factorised_head(nq):
    """A factorised head padded to a multiple of 128 classes: logits by nq_lowrank_linear_fwd,
    the distillation gradient of them, and from it the head's input, scale and factor gradients:
    against the same step in 64 bits with the same rounded dy."""
    from binary_rank_linear_02_b200 import synth

    vocab, m, n, r, tokens, k = 1000, 1024, 512, 256, 96, 16
    Us, Vs = synth.signs(m, r, 5, "U"), synth.signs(n, r, 5, "V")
    dev = torch.device("cuda")
    Upk = nq.pack_signs(torch.from_numpy(Us).to(dev))
    Vpk = nq.pack_signs(torch.from_numpy(np.ascontiguousarray(Vs.T)).to(dev))
    UpkT, VpkT = nq.transpose_signs(Upk, m, r), nq.transpose_signs(Vpk, r, n)
    s1 = torch.from_numpy(synth.scales_f16(m, 5, "s1").view(np.int16)).to(dev)
    s2 = torch.from_numpy(synth.scales_f16(n, 5, "s2").view(np.int16)).to(dev)
    x = torch.from_numpy(synth.activations_bf16(tokens, n, 5).view(np.int16)).to(dev)
    y = nq.lowrank_linear_fwd(x, Upk, Vpk, s1, s2, m, n, r)

    teacher_full = y[:, :vocab] + randn(gen(6), tokens, vocab)
    teacher, ids = torch.topk(teacher_full, k, dim=1)
    lse = torch.logsumexp(teacher_full.double(), 1).float()
    ids = ids.int()
    ids[3] = -1
    dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")
    dy, loss = nq.distill_topk_bwd(y, ids, teacher, vocab, dloss, teacher_lse=lse)
    ref_loss, grad, mag = distill_reference(y, ids, teacher, lse, vocab, 1.0, dloss)
    e = (vocab / 512 + 64) * U
    assert torch.all((loss.double() - ref_loss).abs() <= 2 * e + U * ref_loss.abs())
    assert torch.all((dy[:, :vocab].double() - grad).abs() <= 3 * e * mag + BF * grad.abs())
    assert torch.all(dy[:, vocab:] == 0)

    dx = nq.lowrank_linear_bwd_input(dy, UpkT, VpkT, s1, s2, m, n, r)
    ds1, ds2 = nq.lowrank_linear_bwd_scales(x, dy, Upk, Vpk, UpkT, VpkT, s1, s2, m, n, r)
    dU, dV = nq.lowrank_linear_bwd_factors(x, dy, Vpk, UpkT, s1, s2, m, n, r)
    torch.cuda.synchronize()
    a, b = s1.view(torch.float16).double(), s2.view(torch.float16).double()
    Ud, Vd = torch.from_numpy(Us).to(dev).double(), torch.from_numpy(Vs).to(dev).double()
    xd, dyd = x.view(torch.bfloat16).double(), dy.double()
    t, u = (xd * b) @ Vd, (dyd * a) @ Ud
    want = (u @ Vd.T) * b
    assert torch.all((dx.double() - want).abs() <= 2e-3 * want.abs().amax(1, keepdim=True) + 1e-30)
    z = t @ Ud.T
    assert torch.all((ds1.double() - (dyd * z).sum(0)).abs() <= 2e-3 * (dyd.abs() * z.abs().amax(1, keepdim=True)).sum(0))
    want = a[:, None] * (dyd.T @ t)
    assert torch.all((dU.double() - want).abs() <= 2e-3 * a[:, None] * (dyd.abs() * t.abs().amax(1, keepdim=True)).sum(0)[:, None])


def test_dense_head_gradient_into_the_layer_below(nq):
    """Cross entropy of a dense head over the output of a factorised layer: dh, as it comes, is
    the dy of that layer's input gradient."""
    from binary_rank_linear_02_b200 import synth

    vocab, d, n, r, tokens = 777, 256, 384, 128, 40
    dev = torch.device("cuda")
    Us, Vs = synth.signs(d, r, 9, "U"), synth.signs(n, r, 9, "V")
    Upk = nq.pack_signs(torch.from_numpy(Us).to(dev))
    Vpk = nq.pack_signs(torch.from_numpy(np.ascontiguousarray(Vs.T)).to(dev))
    s1 = torch.from_numpy(synth.scales_f16(d, 9, "s1").view(np.int16)).to(dev)
    s2 = torch.from_numpy(synth.scales_f16(n, 9, "s2").view(np.int16)).to(dev)
    x = torch.from_numpy(synth.activations_bf16(tokens, n, 9).view(np.int16)).to(dev)
    h = nq.rms_normalize_bf16(nq.lowrank_linear_fwd(x, Upk, Vpk, s1, s2, d, n, r)).view(torch.bfloat16)
    _, W, labels, dloss = xent_case(tokens, vocab, d, 10)
    lse, dh, dW = xent_check(nq, h, W, labels, dloss)
    dx = nq.lowrank_linear_bwd_input(dh, nq.transpose_signs(Upk, d, r), nq.transpose_signs(Vpk, r, n), s1, s2, d, n, r)
    torch.cuda.synchronize()
    a, b = s1.view(torch.float16).double(), s2.view(torch.float16).double()
    Ud, Vd = torch.from_numpy(Us).to(dev).double(), torch.from_numpy(Vs).to(dev).double()
    want = ((dh.double() * a) @ Ud @ Vd.T) * b
    assert torch.all((dx.double() - want).abs() <= 2e-3 * want.abs().amax(1, keepdim=True) + 1e-30)


def test_serving_step_with_a_four_bit_head(nq):
    """A decode step's end: a factorised layer, its RMS-normalised bfloat16 output (from the
    grouped call), and the 4-bit head's logits of it; scored against a teacher's top logits."""
    from binary_rank_linear_02_b200 import synth

    d, n, r, vocab, tokens = 512, 256, 128, 1003, 3
    dev = torch.device("cuda")
    Us, Vs = synth.signs(d, r, 12, "U"), synth.signs(n, r, 12, "V")
    Upk = nq.pack_signs(torch.from_numpy(Us).to(dev))
    Vpk = nq.pack_signs(torch.from_numpy(np.ascontiguousarray(Vs.T)).to(dev))
    s1 = torch.from_numpy(synth.scales_f16(d, 12, "s1").view(np.int16)).to(dev)
    s2 = torch.from_numpy(synth.scales_f16(n, 12, "s2").view(np.int16)).to(dev)
    x = torch.from_numpy(synth.activations_bf16(tokens, n, 12).view(np.int16)).to(dev)
    y = torch.empty(tokens, d, device="cuda")
    h = torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda")
    nq.lowrank_linear_fwd_grouped_ex([(x, Upk, Vpk, s1, s2, y, d, n, r, None, h)], tokens)
    codes, scales, z, _ = q4_case(vocab, d, 64, 1, True, 13)
    logits = nq.q4_linear_fwd(h, nq.pack_q4(codes), scales, vocab, d, 64, zeros=z)
    q4_check(logits, codes, scales, z, h, d, 64)
    teacher, ids = torch.topk(logits + randn(gen(14), tokens, vocab), 10, dim=1)
    ids = ids.int()
    distill_check(nq, logits, ids, teacher, None, vocab, 1.0, torch.ones(tokens, device="cuda"), torch.bfloat16)
