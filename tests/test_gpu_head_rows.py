"""The distillation's kernel over many rows: its CTAs (up to three per SM, 444 on 148 SMs) go from
row to row with three rows' sums and lists in turns, so from 1333 tokens on places are used again.
Every row is compared with the definitions in 64 bits.

Tolerances, u = 2^-23.  A row is shared by 256 threads.  A thread adds 16 values with 6 roundings one
after another (u / 2 each), at a row's end 8 values with 4: below V / 512 u for V classes.  An
exponential is off by 2 u and by its argument's two roundings, |argument| u, arguments (base 2) up to
24 where a term matters.  A running maximum that rises, and each of the 5 joins across the lanes,
costs an exponential and a product, 4 u; a thread's maximum rises some 8 times.  Warps are joined in
64 bits.  A sum's relative error e is below (V / 512 + 2 + 24 + 52) u; taken: (V / 512 + 96) u.
loss: T^2 2 e and u |loss|; gradient: 3 e of the magnitude of its terms (the sum, the exponential
and the factors), and the result's rounding.
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


def case(tokens, vocab, pitch, k, rest, t, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.zeros(tokens, pitch, device="cuda")
    full[:, :vocab] = torch.randn(tokens, vocab, device="cuda", generator=g) * 2.5
    full[:, vocab:] = float("nan")
    teacher = full[:, :vocab] + torch.randn(tokens, vocab, device="cuda", generator=g)
    top, ids = torch.topk(teacher, k, dim=1)
    lse = torch.logsumexp(teacher.double() / t, 1).float() if rest else None
    kept = torch.randint(0, 2 * k + 1, (tokens,), device="cuda", generator=g)  # half of the rows are short, some empty
    ids = torch.where(torch.arange(k, device="cuda")[None, :] < kept[:, None], ids, -1).int().contiguous()
    if k > 3:
        ids[::7, 2] = ids[::7, 0]  # listed twice
    dloss = torch.rand(tokens, device="cuda", generator=g) + 0.1
    return full.to(dtype), ids, top.contiguous(), lse, dloss


def reference(logits, ids, teacher, lse, vocab, t, dloss):
    z = logits[:, :vocab].double() / t
    ok = (ids >= 0) & (ids < vocab)
    at = torch.where(ok, ids, 0).long()
    u = torch.where(ok, teacher.double() / t, -torch.inf)
    some = ok.any(1)
    shift = lse.double() if lse is not None else torch.where(some, torch.logsumexp(u, 1), torch.zeros_like(u[:, 0]))
    logq = u - shift[:, None]
    q = torch.where(ok, logq.exp(), 0.0)
    logp = torch.log_softmax(z, 1)
    p = logp.exp()
    loss = torch.where(q > 0, q * (logq - logp.gather(1, at)), 0.0).sum(1)
    dq = torch.zeros_like(p).scatter_add_(1, at, q)
    out = torch.zeros_like(p).scatter_add_(1, at, ok.double()) == 0
    rest = torch.zeros_like(shift)
    share = torch.zeros_like(p)
    if lse is not None:
        there = out.any(1)
        log_rest = torch.logsumexp(torch.where(out, logp, -torch.inf), 1)
        rest = torch.where(there, (1 - q.sum(1)).clamp_min(0), 0.0)
        loss = loss + torch.where(rest > 0, rest * (rest.clamp_min(1e-300).log() - log_rest), 0.0)
        # p_v / p_rest is a softmax of the classes outside the list (of logits of -1e20, p_v and p_rest
        # differ by less than 64 bits of their logarithms hold)
        share = torch.where(there[:, None], torch.softmax(torch.where(out, z, -torch.inf), 1), 0.0) * rest[:, None]
    tot = (q.sum(1) + rest)[:, None]
    w = (dloss.double() * t)[:, None]
    grad, mag = w * (p * tot - dq - share), w * (p * tot + dq + share)
    return (torch.where(some, loss * t * t, 0.0), torch.where(some[:, None], grad, 0.0),
            torch.where(some[:, None], mag, 0.0))


ROWS = [  # tokens, vocab, pitch, k, temperature, element type of the logits
    (1332, 500, 500, 64, 1.0, torch.float32), (1333, 500, 500, 64, 2.0, torch.float32),
    (1333, 9, 9, 4, 1.0, torch.bfloat16), (4096, 9, 11, 9, 1.0, torch.float32),
    (4096, 777, 777, 200, 2.0, torch.float32), (4096, 777, 896, 1, 1.0, torch.bfloat16),
    (2000, 515, 515, 256, 1.0, torch.bfloat16), (3001, 1100, 1100, 1024, 4.0, torch.float32),
    (4096, 4099, 4224, 50, 2.0, torch.float32), (4096, 4099, 4099, 256, 1.0, torch.bfloat16),
    (900, 9000, 9000, 64, 1.0, torch.float32), (2221, 9001, 9001, 16, 2.0, torch.float32),
    (1500, 32000, 32000, 256, 1.0, torch.bfloat16), (1400, 20011, 20096, 64, 2.0, torch.float32),
    (700, 60001, 60001, 128, 1.0, torch.float32),
]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("tokens,vocab,pitch,k,t,dtype", ROWS)
def test_distill_many_rows(nq, tokens, vocab, pitch, k, t, dtype, rest):
    logits, ids, teacher, lse, dloss = case(tokens, vocab, pitch, k, rest, t, dtype, 7000 + tokens + vocab + k)
    loss, grad, mag = reference(logits, ids, teacher, lse, vocab, t, dloss)
    e = (vocab / 512 + 96) * U
    tol = t * t * 2 * e + U * loss.abs()
    got = nq.distill_topk_fwd(logits, ids, teacher, vocab, temperature=t, teacher_lse=lse)
    nq.device_status()
    assert torch.all((got.double() - loss).abs() <= tol)
    assert torch.equal(got, nq.distill_topk_fwd(logits, ids, teacher, vocab, temperature=t, teacher_lse=lse))
    for out, half in ((torch.float32, U), (torch.bfloat16, BF)):
        dz, loss2 = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=out)
        nq.device_status()
        assert torch.all((loss2.double() - loss).abs() <= tol)
        assert torch.all((dz[:, :vocab].double() - grad).abs() <= 3 * e * mag + half * grad.abs() + 1e-38)
        assert torch.all(dz[:, vocab:] == 0)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_rows_alone_and_among_others(nq, rest):
    """A row's loss and gradient are the same bits whatever is before and after it."""
    vocab, t = 1016, 2.0  # (rows begin on 16-byte boundaries, alone as among others)
    logits, ids, teacher, lse, dloss = case(2700, vocab, vocab, 40, rest, t, torch.float32, 77)

    def both(s):
        f = nq.distill_topk_fwd(logits[s], ids[s].clone(), teacher[s].clone(), vocab, temperature=t,
                                teacher_lse=None if lse is None else lse[s].clone())
        return (f, *nq.distill_topk_bwd(logits[s], ids[s].clone(), teacher[s].clone(), vocab, dloss[s].clone(),
                                        temperature=t, teacher_lse=None if lse is None else lse[s].clone()))

    whole = both(slice(None))
    for i in (0, 443, 444, 1331, 1332, 1333, 1776, 2220, 2699):
        for a, b in zip(whole, both(slice(i, i + 1))):
            assert torch.equal(a[i:i + 1], b)
    nq.device_status()


MASKS = [-1e4, -65504.0, -1e9, -1e10, -3e10, -1e12, -1e20, -1e29, -1e30, -3e38]


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", MASKS)
def test_distill_finite_masks(nq, value, dtype, rest):
    """Masked classes hold some large negative number: they have no part in the row, whether a few
    are masked, or all but a few, or all that are not listed; a row begins with masked or other classes."""
    vocab, t, k, tokens = 5003, 1.0, 12, 24
    logits, ids, teacher, lse, dloss = case(tokens, vocab, vocab, k, rest, t, dtype, 501)
    g = torch.Generator(device="cuda").manual_seed(502)
    ids = torch.randint(0, 2500, (tokens, k), device="cuda", generator=g, dtype=torch.int32)
    for i in range(tokens):
        if i % 4 == 0:
            logits[i, 2500:] = value
        elif i % 4 == 1:
            logits[i, 2500:4990] = value
            logits[i, ::2] = value
            ids[i] |= 1
        elif i % 4 == 2:
            logits[i, 1:] = value
            ids[i] = 0
        else:
            kept = logits[i, ids[i].long()].clone()
            logits[i] = value
            logits[i, ids[i].long()] = kept
    if rest:  # a teacher whose mass is all but in its list (what is masked here has next to none there)
        lse = torch.logsumexp(teacher.double() / t, 1).float() + 1e-3
    loss, grad, mag = reference(logits, ids, teacher, lse, vocab, t, dloss)
    e = (vocab / 512 + 96) * U
    got = nq.distill_topk_fwd(logits, ids, teacher, vocab, temperature=t, teacher_lse=lse)
    dz, loss2 = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=torch.float32)
    for x in (got, loss2):
        assert torch.all((x.double() - loss).abs() <= t * t * 2 * e + U * loss.abs())
    assert torch.all((dz.double() - grad).abs() <= 3 * e * mag + U * grad.abs() + 1e-38)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("t", [2.0 ** -28, 2.0 ** -20, 2.0 ** -13])
def test_distill_small_temperatures(nq, t, rest):
    """logits / temperature of up to 5e9: a rounding of it would be a power of two of its own.  (Powers
    of two: the temperature reaches the kernel as fp32.)"""
    vocab = 2003
    logits, ids, teacher, lse, dloss = case(40, vocab, vocab, 8, rest, 1.0, torch.float32, 503)
    # differences of a few temperatures between some of the classes, so that a row has several terms
    g = torch.Generator(device="cuda").manual_seed(504)
    logits = torch.randn(40, vocab, device="cuda", generator=g) * 3 * t
    logits[1::2, ::3] += 20.0  # two levels, far from each other
    logits[3::4] -= 7.0
    if rest:
        lse = torch.logsumexp(teacher.double() / t, 1).float()
        teacher = torch.full_like(teacher, -t)
        lse = torch.full_like(lse, 1.5)
    else:
        teacher = teacher * t
    loss, grad, mag = reference(logits, ids, teacher, lse, vocab, t, dloss)
    e = (vocab / 512 + 96) * U
    got = nq.distill_topk_fwd(logits, ids, teacher, vocab, temperature=t, teacher_lse=lse)
    dz, loss2 = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=torch.float32)
    for x in (got, loss2):
        assert torch.all((x.double() - loss).abs() <= t * t * 2 * e + U * loss.abs())
    assert torch.all((dz.double() - grad).abs() <= 3 * e * mag + U * grad.abs() + 1e-38)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [-1e20, -3e38, 3e38, 1e12, -1e6])
def test_distill_rows_at_one_large_value(nq, value, dtype, rest):
    """Rows whose mask leaves nothing but its own value, which is a uniform distribution, and rows
    of which a half is left at it."""
    vocab, t, k, tokens = 2047, 2.0, 8, 9
    logits, ids, teacher, lse, dloss = case(tokens, vocab, vocab, k, rest, t, dtype, 505)
    logits[:] = value
    logits[::3, 1000:] = -1e30 if value > -1e30 else float("-inf")
    ids[::3] = ids[::3] % 1000
    if rest:
        lse = torch.logsumexp(teacher.double() / t, 1).float() + 0.2
    loss, grad, mag = reference(logits, ids, teacher, lse, vocab, t, dloss)
    e = (vocab / 512 + 96) * U
    got = nq.distill_topk_fwd(logits, ids, teacher, vocab, temperature=t, teacher_lse=lse)
    dz, loss2 = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=torch.float32)
    for x in (got, loss2):
        assert torch.all((x.double() - loss).abs() <= t * t * 2 * e + U * loss.abs())
    assert torch.all((dz.double() - grad).abs() <= 3 * e * mag + U * grad.abs() + 1e-38)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_lists_of_repeated_ids(nq, rest):
    """Lists in which every class stands several times, next to itself and far from it: against the
    definitions, and the same bits each time (the order of no sum is left to the lanes' speed)."""
    vocab, t, k, tokens = 300, 1.0, 1024, 600
    logits, _, _, _, dloss = case(tokens, vocab, vocab, 1, rest, t, torch.float32, 506)
    g = torch.Generator(device="cuda").manual_seed(507)
    ids = torch.randint(-2, vocab, (tokens, k), device="cuda", generator=g, dtype=torch.int32)
    ids[::2, 1::2] = ids[::2, ::2]
    teacher = torch.randn(tokens, k, device="cuda", generator=g)
    lse = torch.logsumexp(teacher.double() / t, 1).float() + 0.3 if rest else None
    loss, grad, mag = reference(logits, ids, teacher, lse, vocab, t, dloss)
    e = (vocab / 512 + 96) * U
    first = None
    for _ in range(30):
        got = nq.distill_topk_fwd(logits, ids, teacher, vocab, temperature=t, teacher_lse=lse)
        dz, loss2 = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=torch.float32)
        if first is None:
            first = got, dz, loss2
            # (a sum of up to k masses per class beside the terms' own rounding)
            assert torch.all((got.double() - loss).abs() <= t * t * 2 * e + U * loss.abs())
            assert torch.all((dz.double() - grad).abs() <= 3 * e * mag + U * grad.abs() + 1e-38)
        for a, b in zip(first, (got, dz, loss2)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("t", [2.0 ** -126, 2.0 ** 40])
def test_distill_temperatures_at_the_ends(nq, t, rest):
    """Each row's largest logit has all the mass, or all classes have the same."""
    vocab = 777
    logits, ids, teacher, _, dloss = case(30, vocab, vocab, 6, rest, 1.0, torch.float32, 508)
    teacher = torch.randn(30, 6, device="cuda", generator=torch.Generator(device="cuda").manual_seed(509)) * t
    lse = torch.full((30,), 2.5, device="cuda") if rest else None
    loss, grad, mag = reference(logits, ids, teacher, lse, vocab, t, dloss)
    e = (vocab / 512 + 96) * U
    dz, got = nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, temperature=t, teacher_lse=lse, dtype=torch.float32)
    # (fp32 numbers below 2^-126 are 2^-149 apart: a result there is rounded by up to 2^-150, which no
    # multiple of it bounds; a gradient's factors there, of which there are some, may be flushed to 0)
    assert torch.all((got.double() - loss).abs() <= t * t * 2 * e + U * loss.abs() + 2.0 ** -150)
    assert torch.all((dz.double() - grad).abs() <= 3 * e * mag + U * grad.abs() + 2.0 ** -126)
