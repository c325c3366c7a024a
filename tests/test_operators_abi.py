"""What the operators for rounded layers refuse, checked before any device is
touched, through the C ABI; and the sizes of their workspaces."""
import ctypes
import os

import pytest

from two_sided_gptq_amd import bakron

F = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bakron.LIB_PATH):
        from two_sided_gptq_amd import build
        build.build()
    return bakron.load()


def refused(lib, rc, word, code=1):
    assert rc == code, rc
    assert word in lib.bakron_last_error(), lib.bakron_last_error()


def test_fp8_quantize(lib):
    def call(X=F, type=1, rows=4, cols=256, ldx=256, br=1, Q=F, ldq=256, s=F):
        return lib.bakron_fp8_quantize(X, type, rows, cols, ldx, br, Q, ldq, s, None, None)
    refused(lib, call(X=None), b"non-NULL")
    refused(lib, call(Q=None), b"non-NULL")
    refused(lib, call(s=None), b"non-NULL")
    refused(lib, call(type=3), b"type")
    refused(lib, call(rows=0), b"sizes")
    refused(lib, call(cols=-1), b"sizes")
    refused(lib, call(rows=(1 << 22) + 1), b"sizes")
    refused(lib, call(ldx=255), b"stride")
    refused(lib, call(ldq=128), b"stride")
    refused(lib, call(ldx=1 << 40), b"stride")
    refused(lib, call(br=64), b"block_rows")
    refused(lib, call(X=ODD), b"misaligned")


def test_fp8_from_codes(lib):
    def call(codes=F, zeros=None, m=4, n=64, kind=0, bits=4, Q=F, ldq=64):
        return lib.bakron_fp8_from_codes(codes, zeros, m, n, kind, bits, Q, ldq, None)
    refused(lib, call(codes=None), b"non-NULL")
    refused(lib, call(m=0), b"sizes")
    refused(lib, call(ldq=63), b"stride")
    refused(lib, call(bits=8), b"exact")
    refused(lib, call(kind=2), b"exact")
    refused(lib, call(kind=1), b"zeros")
    refused(lib, call(zeros=F), b"zeros")


def test_fp8_matmul(lib):
    def call(X=F, ldx=256, sx=F, W=F, ldw=256, sw=F, kind=0, rows=4, N=64, K=256, groups=1, off=None, Y=F, yt=1,
             ldy=64):
        return lib.bakron_fp8_matmul(X, ldx, sx, W, ldw, sw, kind, rows, N, K, groups, off, Y, yt, ldy, None,
                                     F, 1 << 40, None)
    for name in ("X", "sx", "W", "sw", "Y"):
        refused(lib, call(**{name: None}), b"non-NULL")
    refused(lib, call(kind=2), b"scale")
    for size in ("rows", "N", "K"):
        refused(lib, call(**{size: 0}), b"sizes")
        refused(lib, call(**{size: (1 << 24) + 1}), b"sizes")
    refused(lib, call(groups=0), b"groups")
    refused(lib, call(groups=5000, off=F), b"groups")
    refused(lib, call(groups=2), b"offsets")
    refused(lib, call(ldx=255), b"ldx")
    refused(lib, call(ldw=255), b"ldw")
    refused(lib, call(ldy=63), b"ldy")
    refused(lib, call(yt=0), b"type")
    refused(lib, call(Y=ODD), b"misaligned")
    need = lib.bakron_fp8_matmul_workspace_size(64, 64, 8192, 1)
    assert need > 0 and lib.bakron_fp8_matmul_workspace_size(0, 64, 64, 1) == 0
    def small(ws, size):
        return lib.bakron_fp8_matmul(F, 8192, F, F, 8192, F, 0, 64, 64, 8192, 1, None, F, 1, 64, None, ws, size, None)
    refused(lib, small(F, 4096), b"workspace", 2)
    refused(lib, small(None, need), b"workspace", 2)
    refused(lib, small(ctypes.c_void_p(4096 + 8), need), b"workspace", 2)


@pytest.mark.parametrize("name", ["bakron_grouped_matmul", "bakron_grouped_matmul_grad_x",
                                  "bakron_grouped_matmul_grad_w"])
def test_grouped_matmul(lib, name):
    def call(A=F, type=1, lda=512, B=F, ldb=512, rows=4, N=64, K=256, groups=2, off=F, Y=F, yt=1, ldy=512):
        return getattr(lib, name)(A, type, lda, B, ldb, rows, N, K, groups, off, Y, yt, ldy, None, F, 1 << 40, None)
    for p in ("A", "B", "Y"):
        refused(lib, call(**{p: None}), b"non-NULL")
        refused(lib, call(**{p: ODD}), b"misaligned")
    refused(lib, call(type=0), b"type")
    refused(lib, call(yt=2), b"type")
    for size in ("rows", "N", "K"):
        refused(lib, call(**{size: 0}), b"sizes")
    refused(lib, call(off=None), b"offsets")
    refused(lib, call(groups=0), b"groups")
    for ld in ("lda", "ldb", "ldy"):
        refused(lib, call(**{ld: 32}), b"stride")
    refused(lib, call(rows=1 << 24, N=1 << 24), b"tiles")


def test_token_logprobs(lib):
    def call(x=F, type=0, rows=4, vocab=1000, ld=1000, t=F, k=5, lp=F, lse=F, e=F, tl=F, ti=F, ws=F, size=1 << 30):
        return lib.bakron_token_logprobs(x, type, rows, vocab, ld, t, k, lp, lse, e, tl, ti, None, ws, size, None)
    for p in ("x", "t", "lp", "lse", "e", "tl", "ti"):
        refused(lib, call(**{p: None}), b"non-NULL")
    refused(lib, call(type=3), b"type")
    refused(lib, call(rows=0), b"sizes")
    refused(lib, call(vocab=(1 << 21) + 1, ld=1 << 22), b"sizes")
    refused(lib, call(ld=999), b"stride")
    refused(lib, call(k=65), b"k must")
    refused(lib, call(k=-1), b"k must")
    refused(lib, call(vocab=3, k=4), b"k must")
    refused(lib, call(x=ctypes.c_void_p(4098)), b"misaligned")
    need = lib.bakron_token_logprobs_workspace_size(4, 100000, 5)
    assert need > 0 and lib.bakron_token_logprobs_workspace_size(10000, 1000, 5) == 0
    assert lib.bakron_token_logprobs_workspace_size(4, 100, 101) == 0
    refused(lib, call(vocab=100000, ld=100000, size=need - 1), b"workspace", 2)
    refused(lib, call(vocab=100000, ld=100000, ws=None), b"workspace", 2)
    refused(lib, call(vocab=100000, ld=100000, ws=ctypes.c_void_p(4096 + 8)), b"workspace", 2)


def test_token_logprobs_grad(lib):
    def call(x=F, type=0, rows=4, vocab=1000, ld=1000, t=F, lse=F, e=F, g=F, gh=F, d=F, ldd=1000):
        return lib.bakron_token_logprobs_grad(x, type, rows, vocab, ld, t, lse, e, g, gh, d, ldd, None, None)
    for p in ("x", "t", "lse", "g", "d"):
        refused(lib, call(**{p: None}), b"non-NULL")
    refused(lib, call(e=None), b"entropy")
    refused(lib, call(type=9), b"type")
    refused(lib, call(vocab=0), b"sizes")
    refused(lib, call(ld=10), b"stride")
    refused(lib, call(ldd=10), b"stride")
    refused(lib, call(d=ODD), b"misaligned")


def test_binding_refuses_tensors_that_do_not_fit():
    """Tensors off the GPU, of other types or shapes raise BakronError; no call is made."""
    import torch
    x = torch.zeros(4, 256)
    with pytest.raises(bakron.BakronError):
        bakron.fp8_quantize(x)
    with pytest.raises(bakron.BakronError):
        bakron.fp8_from_codes(torch.zeros(4, 4, dtype=torch.int8))
    q = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(bakron.BakronError):
        bakron.fp8_matmul(q, torch.ones(2, 4), q, torch.ones(4))
    b = x.bfloat16()
    for w, off in ((torch.zeros(2, 8, 256).bfloat16(), None), (torch.zeros(2, 8, 128).bfloat16(), torch.zeros(3).int()),
                   (torch.zeros(8, 256).bfloat16(), None)):
        with pytest.raises(bakron.BakronError):
            bakron.grouped_matmul(b, w, off)
    with pytest.raises(bakron.BakronError):
        bakron.grouped_matmul_grad(torch.zeros(4, 9).bfloat16(), b, torch.zeros(1, 8, 256).bfloat16())
    with pytest.raises(bakron.BakronError):
        bakron.token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(bakron.BakronError):
        bakron.token_logprobs_grad(x, torch.zeros(4, dtype=torch.int64), None, None, None)
