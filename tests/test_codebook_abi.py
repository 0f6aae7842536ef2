"""The codebook operators' C ABI on the CPU: exported symbols and the refusals (nothing here launches a kernel)."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "flashkm_codebook.h")

EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    import exact_means_clustering_amd as km
    return km._lib


def at(i, off=0):
    """The i-th of a set of distinct, aligned addresses far apart; never dereferenced: validation fails first."""
    return ctypes.c_void_p((i + 1 << 36) + off)


def err(lib):
    return lib.kmeans_last_error().decode()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"KM_API\s+[\w\s\*]+?\b(kmeans_\w+)\s*\(", text))
    assert names == {"kmeans_embed", "kmeans_embed_grad", "kmeans_embed_grad_workspace_bytes", "kmeans_balance",
                     "kmeans_balance_grad", "kmeans_balance_workspace_bytes"}
    for n in names:
        assert hasattr(lib, n), n


def embed(lib, table=at(0), tdt=BF16, N=10, K=20, D=64, B=1, ids=at(1), out=at(2), odt=BF16):
    return lib.kmeans_embed(table, tdt, N, K, D, B, ids, 1.0, out, odt, None)


@pytest.mark.parametrize("kw, code, word", [
    (dict(tdt=3), EUNSUPPORTED, "table dtype"),
    (dict(odt=-1), EUNSUPPORTED, "out dtype"),
    (dict(K=0), EINVAL, "K=0"),
    (dict(B=0), EINVAL, "B=0"),
    (dict(N=-1), EINVAL, "N=-1"),
    (dict(N=1 << 31), EINVAL, "B*N"),
    (dict(N=1 << 62, B=4), EINVAL, "B*N"),
    (dict(N=1 << 30, B=2), EINVAL, "B*N"),
    (dict(K=1 << 30, B=2), EINVAL, "B*K"),
    (dict(D=0), EUNSUPPORTED, "D=0"),
    (dict(D=(1 << 20) + 1), EUNSUPPORTED, "D="),
    (dict(table=None), EINVAL, "table"),
    (dict(ids=None), EINVAL, "ids"),
    (dict(out=None), EINVAL, "out"),
    (dict(table=at(0, 1)), EINVAL, "misaligned pointer: table"),
    (dict(tdt=F32, table=at(0, 2)), EINVAL, "misaligned pointer: table"),
    (dict(ids=at(1, 2)), EINVAL, "misaligned pointer: ids"),
    (dict(odt=F32, out=at(2, 2)), EINVAL, "misaligned pointer: out"),
    (dict(out=at(0)), EINVAL, "out overlaps table"),
    (dict(out=at(0, 20 * 64 * 2 - 2)), EINVAL, "out overlaps table"),
    (dict(out=at(1, 32)), EINVAL, "out overlaps ids"),
])
def test_embed_refusals(lib, kw, code, word):
    assert embed(lib, **kw) == code
    assert word in err(lib)


def test_embed_of_no_rows_is_nothing(lib):
    assert embed(lib, N=0, ids=None, out=None) == 0


def grad(lib, dout=at(0), idt=BF16, N=1000, K=20, D=64, B=1, ids=at(1), acc=0, g=at(2), gdt=F32, ws=at(3), wb=1 << 30):
    return lib.kmeans_embed_grad(dout, idt, N, K, D, B, ids, 1.0, acc, g, gdt, ws, wb, None)


@pytest.mark.parametrize("kw, code, word", [
    (dict(idt=9), EUNSUPPORTED, "dout dtype"),
    (dict(gdt=9), EUNSUPPORTED, "grad dtype"),
    (dict(K=-5), EINVAL, "K=-5"),
    (dict(N=1 << 33), EINVAL, "B*N"),
    (dict(D=-1), EUNSUPPORTED, "D=-1"),
    (dict(wb=16), EWORKSPACE, "workspace too small"),
    (dict(ws=None), EINVAL, "workspace"),
    (dict(ws=at(3, 64)), EINVAL, "256-byte"),
    (dict(dout=None), EINVAL, "dout"),
    (dict(ids=None), EINVAL, "ids"),
    (dict(g=None), EINVAL, "grad"),
    (dict(g=at(2, 2)), EINVAL, "misaligned pointer: grad"),
    (dict(g=at(0, 64)), EINVAL, "grad overlaps dout"),
    (dict(g=at(3)), EINVAL, "grad overlaps workspace"),
    (dict(ids=at(3, 256)), EINVAL, "workspace overlaps ids"),
])
def test_embed_grad_refusals(lib, kw, code, word):
    assert grad(lib, **kw) == code
    assert word in err(lib)


def test_embed_grad_of_no_rows_accumulated_is_nothing(lib):
    assert grad(lib, N=0, dout=None, ids=None, acc=1) == 0
    assert grad(lib, N=0, dout=None, ids=None, acc=1, ws=None, wb=0) == 0


def test_few_rows_need_no_workspace(lib):
    # 256 bytes stand for none; a misaligned or overlapping one is then of no consequence, other faults still are
    assert lib.kmeans_embed_grad_workspace_bytes(256, 20, 64, 1) == 256
    assert lib.kmeans_embed_grad_workspace_bytes(257, 20, 64, 1) > 256
    assert lib.kmeans_balance_workspace_bytes(32, 8, 1, 2) == 256
    assert grad(lib, N=10, ws=None, wb=0, dout=None) == EINVAL and "dout" in err(lib)
    assert balance(lib, N=10, ws=None, wb=0, labels=None) == EINVAL and "labels" in err(lib)


def test_workspace_sizes(lib):
    f, g = lib.kmeans_embed_grad_workspace_bytes, lib.kmeans_balance_workspace_bytes
    assert f(10, 0, 64, 1) == 0 and f(10, 20, 0, 1) == 0 and f(1 << 31, 20, 64, 1) == 0 and f(10, 20, 64, 0) == 0
    assert g(10, 0, 1, 1) == 0 and g(10, 20, 1, 0) == 0 and g(1 << 30, 20, 1, 2) == 0 and g(-1, 20, 1, 1) == 0
    for n in (0, 1, 1000, 1 << 20):
        assert f(n, 20, 64, 1) > 0 and f(n, 20, 64, 1) % 256 == 0
        assert g(n, 20, 1, 2) > 0 and g(n, 20, 1, 2) % 256 == 0
    # linear in the rows (and the row length), not in rows x entries
    assert f(1 << 23, 65536, 128, 1) < 128 * (1 << 23)
    assert g(1 << 20, 1024, 1, 1) < (1 << 20) * 1024 // 8


def balance(lib, x=at(0), dt=F16, N=10000, K=20, B=1, labels=at(1), S=2, valid=at(2), loss=at(3), counts=at(4), prob=at(5),
            lse=at(6), coef=at(7), ws=at(8), wb=1 << 30):
    return lib.kmeans_balance(x, dt, N, K, B, labels, S, valid, loss, counts, prob, lse, coef, ws, wb, None)


@pytest.mark.parametrize("kw, code, word", [
    (dict(dt=3), EUNSUPPORTED, "dtype"),
    (dict(K=0), EINVAL, "K=0"),
    (dict(B=-1), EINVAL, "B=-1"),
    (dict(B=(1 << 22) + 1, N=1), EINVAL, "B=4194305"),
    (dict(S=0), EINVAL, "S=0"),
    (dict(N=1 << 28, S=8), EINVAL, "B*N*S"),
    (dict(N=-7), EINVAL, "N=-7"),
    (dict(wb=0), EWORKSPACE, "workspace too small"),
    (dict(ws=None), EINVAL, "workspace"),
    (dict(ws=at(8, 4)), EINVAL, "256-byte"),
    (dict(x=None), EINVAL, "logits"),
    (dict(labels=None), EINVAL, "labels"),
    (dict(loss=None), EINVAL, "loss"),
    (dict(counts=None), EINVAL, "counts"),
    (dict(prob=None), EINVAL, "prob"),
    (dict(lse=None), EINVAL, "lse"),
    (dict(coef=None), EINVAL, "coef"),
    (dict(x=at(0, 1)), EINVAL, "misaligned pointer: logits"),
    (dict(lse=at(6, 2)), EINVAL, "misaligned pointer: lse"),
    (dict(coef=at(5)), EINVAL, "prob overlaps coef"),
    (dict(lse=at(0, 16)), EINVAL, "lse overlaps logits"),
    (dict(valid=at(8, 16)), EINVAL, "workspace overlaps valid"),
])
def test_balance_refusals(lib, kw, code, word):
    assert balance(lib, **kw) == code
    assert word in err(lib)


def bgrad(lib, x=at(0), dt=BF16, N=10, K=20, B=1, lse=at(1), coef=at(2), dloss=at(3), out=at(4)):
    return lib.kmeans_balance_grad(x, dt, N, K, B, lse, coef, dloss, out, None)


@pytest.mark.parametrize("kw, code, word", [
    (dict(dt=4), EUNSUPPORTED, "dtype"),
    (dict(K=0), EINVAL, "K=0"),
    (dict(N=1 << 31), EINVAL, "B*N"),
    (dict(x=None), EINVAL, "logits"),
    (dict(lse=None), EINVAL, "lse"),
    (dict(coef=None), EINVAL, "coef"),
    (dict(dloss=None), EINVAL, "dloss"),
    (dict(out=None), EINVAL, "dlogits"),
    (dict(out=at(0)), EINVAL, "dlogits overlaps logits"),
    (dict(out=at(4, 1)), EINVAL, "misaligned pointer: dlogits"),
])
def test_balance_grad_refusals(lib, kw, code, word):
    assert bgrad(lib, **kw) == code
    assert word in err(lib)


def test_balance_grad_of_no_rows_is_nothing(lib):
    assert bgrad(lib, N=0, x=None, lse=None, out=None) == 0


def test_binding_refuses_what_is_not_on_the_gpu():
    import exact_means_clustering_amd as km
    t, ids = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: km.embed(t, ids), lambda: km.embed_grad(torch.zeros(3, 8), ids, 4),
                 lambda: km.balance(torch.zeros(3, 4), ids),
                 lambda: km.balance_grad(torch.zeros(3, 4), (torch.zeros(3), torch.zeros(4)), torch.zeros(1))):
        with pytest.raises(km.KMeansError, match="CUDA tensor"):
            call()
    with pytest.raises(km.KMeansError, match="32 bits"):
        km.embed_grad_workspace_bytes(10, 1 << 32, 64)


@pytest.mark.parametrize("N, K", [(1, (1 << 31) - 1), (1, (1 << 31) - 8), (1, (1 << 31) - 31), (100, (1 << 31) - 2),
                                  (129, (1 << 31) - 2049), (64, 20001)])
def test_balance_workspace_at_the_largest_k(lib, N, K):
    # longer rows: column sums of every chunk of 64 rows, a term of the loss for every 32 columns, two values a row
    need = -(-N // 64) * K * 4 + -(-K // 32) * 8 + N * 8
    assert need <= lib.kmeans_balance_workspace_bytes(N, K, 1, 1) <= need + 8 * 256


@pytest.mark.parametrize("name", ["embed", "embed_grad", "balance", "balance_grad"])
def test_binding_shows_its_stream_argument(name):
    import inspect

    import exact_means_clustering_amd as km
    fn = getattr(km, name)
    p = inspect.signature(fn).parameters["stream"]
    assert p.kind is inspect.Parameter.KEYWORD_ONLY and p.default is None
    assert "stream" in fn.__doc__
