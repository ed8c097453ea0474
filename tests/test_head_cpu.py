"""The output head's entry points without a GPU: host packing of 4-bit codes, scratch sizes,
the argument errors found on the host, and the binding's checks of types and shapes."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def nq():
    from binary_rank_linear_02_b200 import build

    build.build()
    from binary_rank_linear_02_b200 import nq as mod

    return mod


@pytest.fixture(scope="module")
def ptrs():
    buf = np.zeros(1 << 17, dtype=np.uint8)
    base = (buf.ctypes.data + 255) // 256 * 256
    return [base + 4096 * i for i in range(10)], buf


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (5, 9), (2, 128), (7, 31)])
def test_host_pack_q4(nq, rows, cols):
    codes = np.random.default_rng(rows * 100 + cols).integers(0, 16, (rows, cols)).astype(np.uint8)
    got = nq.pack_q4(codes)
    want = np.zeros((rows, (cols + 7) // 8), dtype=np.uint32)
    for i in range(rows):
        for j in range(cols):
            want[i, j // 8] |= np.uint32(int(codes[i, j]) << (4 * (j % 8)))
    assert np.array_equal(got, want)


def test_host_pack_q4_errors(nq):
    out = np.zeros((1, 1), dtype=np.uint32)
    codes = np.array([[1, 16]], dtype=np.uint8)
    f = nq.lib().nq_pack_q4
    assert f(codes.ctypes.data, 1, 2, out.ctypes.data, 0) == nq.NQ_ERR_VALUE
    assert f(0, 1, 2, out.ctypes.data, 0) == nq.NQ_ERR_NULL
    assert f(codes.ctypes.data, 1, 2, 0, 0) == nq.NQ_ERR_NULL
    assert f(codes.ctypes.data, -1, 2, out.ctypes.data, 0) == nq.NQ_ERR_SHAPE
    assert f(codes.ctypes.data, 1, 0, out.ctypes.data, 0) == nq.NQ_OK
    with pytest.raises(TypeError):
        nq.pack_q4(codes.astype(np.int32))


def test_q4_argument_errors(nq, ptrs):
    p, _ = ptrs
    f = nq.lib().nq_q4_linear_fwd
    good = dict(m=16, n=128, group=128, batch=1)

    def call(a=p[0], w=p[1], s=p[2], z=0, y=p[3], **kw):
        v = {**good, **kw}
        return f(a, w, s, z, v["m"], v["n"], v["group"], v["batch"], y, 0)

    assert call(batch=-1) == nq.NQ_ERR_BATCH
    assert call(batch=65535 * 8 + 1) == nq.NQ_ERR_BATCH
    assert call(m=0) == nq.NQ_ERR_SHAPE
    assert call(n=64) == nq.NQ_ERR_SHAPE
    assert call(n=0) == nq.NQ_ERR_SHAPE
    assert call(n=1 << 21) == nq.NQ_ERR_SHAPE
    for group in (0, 16, 48, 256, -32):
        assert call(group=group) == nq.NQ_ERR_SHAPE
    assert call(batch=0) == nq.NQ_OK
    for name in "awsy":
        assert call(**{name: 0}) == nq.NQ_ERR_NULL
    assert call(a=p[0] + 2) == nq.NQ_ERR_ALIGN
    assert call(z=p[4] + 8) == nq.NQ_ERR_ALIGN
    assert call() == nq.NQ_ERR_PTRKIND  # host memory


def test_distill_argument_errors(nq, ptrs):
    p, _ = ptrs
    L = nq.lib()
    base = dict(lt=nq.NQ_F32, ld=100, tokens=2, vocab=100, k=4, t=1.0, gt=nq.NQ_BF16, logits=p[0], ids=p[1],
                teacher=p[2], lse=0, dloss=p[3], loss=p[4], dl=p[5])

    def fwd(**kw):
        v = {**base, **kw}
        return L.nq_distill_topk_fwd(v["logits"], v["lt"], v["ld"], v["ids"], v["teacher"], v["lse"], v["tokens"],
                                     v["vocab"], v["k"], v["t"], v["loss"], 0)

    def bwd(**kw):
        v = {**base, **kw}
        return L.nq_distill_topk_bwd(v["logits"], v["lt"], v["ld"], v["ids"], v["teacher"], v["lse"], v["dloss"],
                                     v["tokens"], v["vocab"], v["k"], v["t"], v["loss"], v["dl"], v["gt"], 0)

    for f in (fwd, bwd):
        assert f(tokens=-1) == nq.NQ_ERR_BATCH
        assert f(tokens=1 << 31) == nq.NQ_ERR_BATCH
        assert f(vocab=0) == nq.NQ_ERR_SHAPE
        assert f(ld=99) == nq.NQ_ERR_SHAPE
        assert f(vocab=(1 << 20) + 1, ld=1 << 21) == nq.NQ_ERR_SHAPE
        assert f(k=0) == nq.NQ_ERR_SHAPE
        assert f(k=1025) == nq.NQ_ERR_SHAPE
        assert f(lt=2) == nq.NQ_ERR_VALUE
        for t in (0.0, -1.0, float("inf"), float("nan")):
            assert f(t=t) == nq.NQ_ERR_VALUE
        assert f(tokens=0) == nq.NQ_OK
        for name in ("logits", "ids", "teacher"):
            assert f(**{name: 0}) == nq.NQ_ERR_NULL
            assert f(**{name: p[6] + 4}) == nq.NQ_ERR_ALIGN
        assert f() == nq.NQ_ERR_PTRKIND
    assert fwd(loss=0) == nq.NQ_ERR_NULL
    assert bwd(gt=7) == nq.NQ_ERR_VALUE
    assert bwd(dl=0) == nq.NQ_ERR_NULL
    assert bwd(dloss=0) == nq.NQ_ERR_NULL
    assert bwd(loss=0) == nq.NQ_ERR_PTRKIND  # the loss is optional here


def test_cross_entropy_argument_errors(nq, ptrs):
    p, _ = ptrs
    L = nq.lib()
    base = dict(tokens=2, vocab=100, d=64, h=p[0], w=p[1], labels=p[2], loss=p[3], lse=p[4], dloss=p[5], dh=p[6],
                dw=p[7], scratch=p[8], size=1 << 40)

    def fwd(**kw):
        v = {**base, **kw}
        return L.nq_linear_cross_entropy_fwd(v["h"], v["w"], v["labels"], v["tokens"], v["vocab"], v["d"], v["loss"],
                                             v["lse"], v["scratch"], v["size"], 0)

    def bwd(**kw):
        v = {**base, **kw}
        return L.nq_linear_cross_entropy_bwd(v["h"], v["w"], v["labels"], v["lse"], v["dloss"], v["tokens"],
                                             v["vocab"], v["d"], v["dh"], v["dw"], v["scratch"], v["size"], 0)

    for f in (fwd, bwd):
        assert f(tokens=-1) == nq.NQ_ERR_BATCH
        assert f(tokens=(1 << 24) + 1) == nq.NQ_ERR_BATCH
        for bad in (0, 4, 12, -8, (1 << 20) + 8):
            assert f(d=bad) == nq.NQ_ERR_SHAPE
        assert f(vocab=0) == nq.NQ_ERR_SHAPE
        assert f(vocab=(1 << 20) + 1) == nq.NQ_ERR_SHAPE
        for name in ("h", "w", "labels", "lse", "scratch"):
            assert f(**{name: 0}) == nq.NQ_ERR_NULL
            assert f(**{name: p[9] + 8}) == nq.NQ_ERR_ALIGN
        assert f() == nq.NQ_ERR_PTRKIND
    assert fwd(tokens=0) == nq.NQ_OK
    assert fwd(loss=0) == nq.NQ_ERR_NULL
    assert bwd(dh=0, dw=0) == nq.NQ_OK  # nothing to compute
    assert bwd(tokens=0, dw=0) == nq.NQ_OK
    assert bwd(tokens=0) == nq.NQ_ERR_PTRKIND  # zeros would be written to host memory


def test_cross_entropy_scratch_bytes(nq):
    f = nq.lib().nq_linear_cross_entropy_scratch_bytes
    assert f(-1, 100, 64, 0) == -1
    assert f(1, 100, 60, 1) == -1
    assert f(0, 100, 64, 1) == 0
    for tokens, vocab, d in ((1, 1, 8), (4096, 32000, 4096), (1000, 128256, 8192), (1 << 20, 1 << 20, 64)):
        fwd, bwd = f(tokens, vocab, d, 0), f(tokens, vocab, d, 1)
        assert fwd >= 8 * tokens and bwd >= 2 * tokens
        # the logits are never kept: a piece of dz and the shares of dh's sums are bounded
        assert bwd <= max(256 << 20, 2 * 256 * tokens) + max(256 << 20, 4 * tokens * d) + 1024


def test_binding_refuses_wrong_types_and_shapes(nq):
    import torch

    x = torch.zeros(1, 128, dtype=torch.bfloat16)
    w = torch.zeros(4, 16, dtype=torch.int32)
    s = torch.zeros(4, 1, dtype=torch.float16)
    with pytest.raises(TypeError):
        nq.q4_linear_fwd(x.float(), w, s, 4, 128, 128)
    with pytest.raises(TypeError):
        nq.q4_linear_fwd(x, w, s.float(), 4, 128, 128)
    with pytest.raises(ValueError):
        nq.q4_linear_fwd(x, w, s, 5, 128, 128)
    with pytest.raises(ValueError):
        nq.q4_linear_fwd(x, w, s, 4, 128, 64)
    logits = torch.zeros(3, 50)
    ids = torch.zeros(3, 2, dtype=torch.int32)
    teacher = torch.zeros(3, 2)
    with pytest.raises(TypeError):
        nq.distill_topk_fwd(logits.double(), ids, teacher, 50)
    with pytest.raises(TypeError):
        nq.distill_topk_fwd(logits, ids.long(), teacher, 50)
    with pytest.raises(ValueError):
        nq.distill_topk_fwd(logits, ids, teacher[:2], 50)
    with pytest.raises(nq.NQError):  # more classes than columns
        nq.distill_topk_fwd(logits, ids, teacher, 51)
    with pytest.raises(ValueError):
        nq.distill_topk_bwd(logits, ids, teacher, 50, torch.zeros(2))
    h, W = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nq.linear_cross_entropy_fwd(h, W, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        nq.linear_cross_entropy_fwd(h.float(), W, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        nq.linear_cross_entropy_fwd(h, W[:, :32].contiguous(), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(nq.NQError):
        nq.linear_cross_entropy_fwd(h, W, torch.zeros(3, dtype=torch.int32))  # host memory
