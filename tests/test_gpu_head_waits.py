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


def test_head_status_leaves_the_workspace_alone(nq):
    """The head shares no workspace: reading and clearing the status of a call that gave up does not
    reach into the arrival counters of the factorised layers' calls under way on another stream."""
    import numpy as np

    from binary_rank_linear_02_b200 import synth

    m, n, r = 4096, 4096, 1024
    dev = torch.device("cuda")
    Us, Vs = synth.signs(m, r, 3, "U"), synth.signs(n, r, 3, "V")
    Upk = nq.pack_signs(torch.from_numpy(Us).to(dev))
    Vpk = nq.pack_signs(torch.from_numpy(np.ascontiguousarray(Vs.T)).to(dev))
    s1 = torch.from_numpy(synth.scales_f16(m, 3, "s1").view(np.int16)).to(dev)
    s2 = torch.from_numpy(synth.scales_f16(n, 3, "s2").view(np.int16)).to(dev)
    xs = [torch.from_numpy(synth.activations_bf16(b, n, 3).view(np.int16)).to(dev) for b in (1, 5, 40)]
    want = [nq.lowrank_linear_fwd(x, Upk, Vpk, s1, s2, m, n, r) for x in xs]
    vocab = 1 << 20
    logits = torch.zeros(3, vocab, device="cuda")
    ids, teacher = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, 1, device="cuda")
    loss = torch.empty(3, device="cuda")
    head, layers = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    try:
        for _ in range(10):
            assert nq.nq_selftest_head_wait_limit(1000) == nq.NQ_OK
            nq.distill_topk_fwd(logits, ids, teacher, vocab, loss=loss, stream=head.cuda_stream)
            with torch.cuda.stream(layers):
                got = [[nq.lowrank_linear_fwd(x, Upk, Vpk, s1, s2, m, n, r) for x in xs] for _ in range(20)]
            assert nq.nq_device_status(head.cuda_stream) == nq.NQ_ERR_TIMEOUT
            torch.cuda.synchronize()
            assert nq.nq_device_status(0) == nq.NQ_OK
            for y in got:
                for a, b in zip(want, y):
                    assert torch.equal(a, b)
    finally:
        nq.nq_selftest_head_wait_limit(0)
