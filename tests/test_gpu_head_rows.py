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
        share = torch.where(out & there[:, None], (logp - log_rest[:, None]).exp() * rest[:, None], 0.0)
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
