"""Waits of the output head's kernels that give up: the call ends, with the copies that it has in
flight landed, the status is reported once, and the same call is right afterwards.

The limit is a microsecond of GPU time, and the work that is waited for is far longer than that.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from binary_rank_linear_02_b200 import nq as mod

    return mod


def gives_up_and_recovers(nq, call, always=True):
    want = call()
    nq.device_status()
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        assert nq.nq_selftest_head_wait_limit(1000) == nq.NQ_OK
        try:
            call()
        finally:
            assert nq.nq_selftest_head_wait_limit(0) == nq.NQ_OK
        status = nq.nq_device_status(stream)
        assert status == nq.NQ_ERR_TIMEOUT or not always and status == nq.NQ_OK
        assert nq.nq_device_status(stream) == nq.NQ_OK
        for a, b in zip(want, call()):
            assert torch.equal(a, b)
        nq.device_status()


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("tokens,vocab", [(3, 1 << 20), (500, 200001)])
def test_distill_gives_up(nq, tokens, vocab, rest):
    g = torch.Generator(device="cuda").manual_seed(11)
    logits = torch.randn(tokens, vocab, device="cuda", generator=g)
    ids = torch.randint(0, vocab, (tokens, 7), device="cuda", generator=g, dtype=torch.int32)
    teacher = torch.randn(tokens, 7, device="cuda", generator=g)
    lse = torch.full((tokens,), 4.0, device="cuda") if rest else None
    dloss = torch.ones(tokens, device="cuda")
    gives_up_and_recovers(nq, lambda: (nq.distill_topk_fwd(logits, ids, teacher, vocab, teacher_lse=lse),))
    gives_up_and_recovers(nq, lambda: nq.distill_topk_bwd(logits, ids, teacher, vocab, dloss, teacher_lse=lse))



def test_q4_gives_up(nq):
    """The kernel's own waits are a few microseconds long; here x lies in managed memory that the host
    has just written, so that its pages come over first, while the fetching warp waits."""
    import ctypes

    import numpy as np

    m, n, group, batch = 100, 1 << 20, 128, 8
    g = torch.Generator(device="cuda").manual_seed(12)
    w = torch.randint(-(1 << 31), 1 << 31, (m, n // 8), device="cuda", generator=g, dtype=torch.int32)
    scales, zeros = (torch.rand(m, n // group, device="cuda", generator=g).half() for _ in range(2))
    x = torch.randn(batch, n, device="cuda", generator=g).bfloat16()
    bits = x.view(torch.int16).cpu().numpy()
    runtime = ctypes.CDLL("libcudart.so.12")
    at = ctypes.c_void_p()
    assert runtime.cudaMallocManaged(ctypes.byref(at), ctypes.c_size_t(bits.nbytes), ctypes.c_uint(1)) == 0
    try:
        there = np.ctypeslib.as_array(ctypes.cast(at, ctypes.POINTER(ctypes.c_int16)), bits.shape)

        def call():
            there[:] = bits
            y = torch.empty(batch, m, device="cuda")
            assert nq.lib().nq_q4_linear_fwd(at.value, w.data_ptr(), scales.data_ptr(), zeros.data_ptr(), m, n, group,
                                             batch, y.data_ptr(), torch.cuda.current_stream().cuda_stream) == nq.NQ_OK
            torch.cuda.synchronize()
            return (y,)

        assert torch.equal(call()[0], nq.q4_linear_fwd(x, w, scales, m, n, group, zeros=zeros))
        gives_up_and_recovers(nq, call)
    finally:
        torch.cuda.synchronize()
        runtime.cudaFree(at)


@pytest.mark.parametrize("tokens,vocab,d", [(40, 700, 1 << 18), (200, 300, 1 << 17), (300, 520, 1 << 17), (1000, 3000, 1 << 15)])
def test_cross_entropy_gives_up(nq, tokens, vocab, d):
    """Epilogues that wait for a long sum: hundreds of microseconds."""
    g = torch.Generator(device="cuda").manual_seed(13)
    h = torch.randn(tokens, d, device="cuda", generator=g).bfloat16()
    W = (torch.randn(vocab, d, device="cuda", generator=g) / d ** 0.5).bfloat16()
    labels = torch.randint(0, vocab, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    dloss = torch.ones(tokens, device="cuda")
    _, lse = nq.linear_cross_entropy_fwd(h, W, labels)
    gives_up_and_recovers(nq, lambda: nq.linear_cross_entropy_bwd(h, W, labels, lse, dloss))
    # (above 256 tokens the forward's sums are taken in parts, whose waits may be too short to give up)
    gives_up_and_recovers(nq, lambda: nq.linear_cross_entropy_fwd(h, W, labels), always=tokens <= 256)
