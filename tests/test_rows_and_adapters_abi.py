"""What the operators around a rounded layer's products refuse, checked before any device is
touched, through the C ABI; and the sizes of their workspaces."""
import ctypes
import os
import re

import pytest

from two_sided_gptq_amd import bakron

F = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bakron.LIB_PATH):
        from two_sided_gptq_amd import build
        build.build()
    return bakron.load()


def refused(lib, rc, word, code=1):
    assert rc == code, rc
    assert word in lib.bakron_last_error(), lib.bakron_last_error()


def test_the_binding_has_what_the_header_declares(lib):
    with open(os.path.join(ROOT, "include", "bakron.h")) as f:
        names = set(re.findall(r"^(?:int32_t|size_t|const char \*)\s*\*?(bakron_\w+)\(", f.read(), re.M))
    assert names == set(bakron.EXPORTS)
    for n in names:
        assert getattr(lib, n).argtypes is not None


def test_group_sort(lib):
    def call(ids=F, bits=64, n=100, groups=8, off=F, order=F, slots=F, ws=None, size=0):
        return lib.bakron_group_sort(ids, bits, n, groups, off, order, slots, None, ws, size, None)
    for a in ("ids", "off", "order", "slots"):
        refused(lib, call(**{a: None}), b"non-NULL")
    refused(lib, call(bits=16), b"id_bits")
    refused(lib, call(n=0), b"size")
    refused(lib, call(n=(1 << 24) + 1), b"size")
    refused(lib, call(groups=0), b"groups")
    refused(lib, call(groups=4097), b"groups")
    refused(lib, call(ids=ctypes.c_void_p(4100)), b"misaligned")
    need = lib.bakron_group_sort_workspace_size(100000, 8)
    assert need > 0
    refused(lib, call(n=100000), b"workspace", 2)
    refused(lib, call(n=100000, ws=F, size=need - 1), b"workspace", 2)
    refused(lib, call(n=100000, ws=ctypes.c_void_p(4096 + 128), size=need), b"workspace", 2)
    assert lib.bakron_group_sort_workspace_size(0, 8) == 0
    assert lib.bakron_group_sort_workspace_size(1 << 60, 8) == 0
    assert lib.bakron_group_sort_workspace_size(100, -1) == 0
    for n in (1, 4096, 4097, 1 << 20, (1 << 20) + 1, 1 << 24):
        for g in (1, 1024, 1025, 4096):
            assert lib.bakron_group_sort_workspace_size(n, g) <= 1 << 28


def rows_refusals(lib, call, pointers, strides, typed):
    for p in pointers:
        refused(lib, call(**{p: None}), b"non-NULL")
    refused(lib, call(type=3), b"type")
    for bad in (dict(tokens=0), dict(k=0), dict(k=65), dict(cols=0), dict(tokens=1 << 24, k=2), dict(tokens=1 << 62),
                dict(cols=(1 << 24) + 1), dict(tokens=-5)):
        refused(lib, call(**bad), b"sizes")
    refused(lib, call(groups=0), b"groups")
    refused(lib, call(groups=4097), b"groups")
    for s in strides:
        refused(lib, call(**{s: 63}), b"stride")
        refused(lib, call(**{s: (1 << 32) + 1}), b"stride")
    for p in typed:
        refused(lib, call(**{p: ODD}), b"misaligned")


def test_group_gather(lib):
    def call(X=F, type=1, tokens=10, k=2, cols=64, ldx=64, slots=F, groups=4, off=F, out=F, ldo=64):
        return lib.bakron_group_gather(X, type, tokens, k, cols, ldx, slots, groups, off, out, ldo, None, None)
    rows_refusals(lib, call, ("X", "slots", "off", "out"), ("ldx", "ldo"), ("X", "out"))


def test_group_gather_fp8(lib):
    def call(X=F, type=0, tokens=10, k=2, cols=64, ldx=64, slots=F, groups=4, off=F, Q=F, ldq=64, s=F):
        return lib.bakron_group_gather_fp8(X, type, tokens, k, cols, ldx, slots, groups, off, Q, ldq, s, None, None)
    rows_refusals(lib, call, ("X", "slots", "off", "Q", "s"), ("ldx", "ldq"), ("X",))


def test_group_combine(lib):
    def call(Y=F, type=2, tokens=10, k=2, cols=64, ldy=64, slots=F, groups=4, off=F, w=None, out=F, ldo=64):
        return lib.bakron_group_combine(Y, type, tokens, k, cols, ldy, slots, groups, off, w, out, ldo, None, None)
    rows_refusals(lib, call, ("Y", "slots", "off", "out"), ("ldy", "ldo"), ("Y", "out"))


def test_group_combine_grad(lib):
    def call(d=F, ldd=64, Y=F, type=2, tokens=10, k=2, cols=64, ldy=64, slots=F, groups=4, off=F, w=F, dY=F, lddy=64,
             dw=F):
        return lib.bakron_group_combine_grad(d, ldd, Y, type, tokens, k, cols, ldy, slots, groups, off, w, dY, lddy, dw,
                                             None, None)
    rows_refusals(lib, call, ("d", "Y", "slots", "off", "w", "dY", "dw"), ("ldd", "ldy", "lddy"), ("d", "Y", "dY"))


def sizes_refusals(lib, call):
    for bad in (dict(rows=0), dict(N=0), dict(K=-1), dict(rows=(1 << 24) + 1), dict(N=1 << 40)):
        refused(lib, call(**bad), b"sizes")
    refused(lib, call(rank=0), b"rank")
    refused(lib, call(rank=257), b"rank")
    refused(lib, call(groups=0), b"groups")
    refused(lib, call(groups=4097), b"groups")
    refused(lib, call(rows=1 << 24, N=1 << 24), b"too many tiles")
    refused(lib, call(groups=4096, K=1 << 24), b"too many tiles")
    refused(lib, call(off=None, groups=2), b"offsets")
    refused(lib, call(type=0), b"type")
    refused(lib, call(type=3), b"type")


def test_adapter_matmul(lib):
    need = lib.bakron_adapter_matmul_workspace_size(20, 64, 128, 16, 3)
    assert need > 0

    def call(X=F, type=1, ldx=128, A=F, B=F, rows=20, N=64, K=128, rank=16, groups=3, off=F, base=F, ldb=64, out=F,
             ot=1, ldo=64, ws=None, size=0):
        return lib.bakron_adapter_matmul(X, type, ldx, A, B, rows, N, K, rank, groups, off, None, None, base, ldb, out,
                                         ot, ldo, None, ws, size, None)
    for p in ("X", "A", "B", "out"):
        refused(lib, call(**{p: None}), b"non-NULL")
    sizes_refusals(lib, call)
    refused(lib, call(ldx=127), b"ldx")
    refused(lib, call(ldo=63), b"ldo")
    refused(lib, call(ldb=63), b"ldb")
    refused(lib, call(ldb=65), b"base in place")
    refused(lib, call(ot=2), b"type")
    refused(lib, call(X=ODD), b"misaligned")
    refused(lib, call(out=ctypes.c_void_p(4098), ot=0), b"misaligned")
    refused(lib, call(), b"workspace", 2)
    refused(lib, call(ws=F, size=need - 1), b"workspace", 2)
    refused(lib, call(ws=ctypes.c_void_p(4096 + 64), size=need), b"workspace", 2)


def test_adapter_matmul_grad(lib):
    need = lib.bakron_adapter_matmul_grad_workspace_size(20, 64, 128, 16, 3)
    assert need > 0

    def call(dY=F, lddy=64, X=F, type=1, ldx=128, A=F, B=F, rows=20, N=64, K=128, rank=16, groups=3, off=F, base=None,
             ldb=128, dX=F, xt=1, lddx=128, dA=F, dB=F, wt=0, ws=None, size=0):
        return lib.bakron_adapter_matmul_grad(dY, lddy, X, type, ldx, A, B, rows, N, K, rank, groups, off, None, None,
                                              base, ldb, dX, xt, lddx, dA, dB, wt, None, ws, size, None)
    for p in ("dY", "A", "B"):
        refused(lib, call(**{p: None}), b"non-NULL")
    refused(lib, call(dX=None, dA=None, dB=None), b"non-NULL")
    refused(lib, call(dA=None), b"together")
    refused(lib, call(X=None), b"need X")
    sizes_refusals(lib, call)
    refused(lib, call(lddy=63), b"lddy")
    refused(lib, call(ldx=127), b"ldx")
    refused(lib, call(lddx=127), b"lddx")
    refused(lib, call(base=F, ldb=127), b"ldb")
    refused(lib, call(base=F, ldb=129), b"base in place")
    refused(lib, call(xt=2), b"type")
    refused(lib, call(wt=2), b"type")
    refused(lib, call(dB=ctypes.c_void_p(4098)), b"misaligned")
    refused(lib, call(ws=F, size=need - 1), b"workspace", 2)


def test_adapter_workspaces_stay_small(lib):
    """Places in whole tiles of the rank's values, three times in the backward pass, and partial sums
    of the weights' gradients for about as many chunks as fill the GPU."""
    for rows in (1, 17, 1000, 100000):
        for groups in (1, 7, 64, 4096):
            for rank in (1, 16, 100, 256):
                for n, k in ((64, 64), (4096, 14336), (14336, 4096)):
                    places = (rows // 16 + groups + 2) * 4 * 16 * (-(-rank // 16) * 16) * 4
                    assert lib.bakron_adapter_matmul_workspace_size(rows, n, k, rank, groups) <= 8 * places + (1 << 20)
                    chunks = rank * (n + k) * 4 * (groups + 600)
                    assert lib.bakron_adapter_matmul_grad_workspace_size(rows, n, k, rank, groups) <= 4 * places + chunks + (1 << 20)
    assert lib.bakron_adapter_matmul_workspace_size(0, 1, 1, 1, 1) == 0
    assert lib.bakron_adapter_matmul_grad_workspace_size(1 << 62, 1 << 62, 1, 1, 1) == 0


def test_verify_drafts(lib):
    def call(p=F, ldp=1000, q=F, ldq=1000, type=0, batch=4, drafts=3, vocab=1000, d=F, u=F, v=F, acc=F, tok=F, ws=None,
             size=0):
        return lib.bakron_verify_drafts(p, ldp, q, ldq, type, batch, drafts, vocab, d, u, v, acc, tok, None, ws, size, None)
    for p in ("p", "v", "acc", "tok", "d", "u"):
        refused(lib, call(**{p: None}), b"non-NULL")
    refused(lib, call(type=3), b"type")
    for bad in (dict(batch=0), dict(batch=(1 << 20) + 1), dict(drafts=-1), dict(drafts=65), dict(vocab=0),
                dict(vocab=(1 << 24) + 1)):
        refused(lib, call(**bad), b"sizes")
    refused(lib, call(ldp=999), b"ldp")
    refused(lib, call(ldq=999), b"ldq")
    refused(lib, call(p=ODD), b"misaligned")
    refused(lib, call(q=ctypes.c_void_p(4098)), b"misaligned")
    big = 1 << 17
    need = lib.bakron_verify_drafts_workspace_size(4, 3, big)
    assert 0 < need <= 1 << 20
    refused(lib, call(vocab=big, ldp=big, ldq=big), b"workspace", 2)
    refused(lib, call(vocab=big, ldp=big, ldq=big, ws=F, size=need - 1), b"workspace", 2)
    for batch in (1, 63, 64, 128, 255, 256, 1 << 20):
        for vocab in (1, 1000, 50001, 1 << 24):
            assert lib.bakron_verify_drafts_workspace_size(batch, 4, vocab) <= 1 << 20
    assert lib.bakron_verify_drafts_workspace_size(0, 4, 1000) == 0
    assert lib.bakron_verify_drafts_workspace_size(1, -4, 1000) == 0
