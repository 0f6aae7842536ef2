"""The training operators' C ABI on the CPU: exported symbols, the AdamW table and the refusals (nothing here launches a
kernel)."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "flashkm_train.h")

EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
F32, F16, BF16 = 0, 1, 2
SOFTMAX, SIGMOID = 0, 1


@pytest.fixture(scope="module")
def lib():
    import exact_means_clustering_amd as km
    return km._lib


def at(i, off=0):
    """The i-th of a set of distinct, aligned addresses far apart; never dereferenced: validation fails first."""
    return ctypes.c_void_p((i + 1 << 42) + off)


def err(lib):
    return lib.kmeans_last_error().decode()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"KM_API\s+[\w\s\*]+?\b(kmeans_\w+)\s*\(", text))
    assert names == {"kmeans_route", "kmeans_route_grad", "kmeans_adamw", "kmeans_adamw_table", "kmeans_adamw_chunks",
                     "kmeans_adamw_table_bytes"}
    for n in names:
        assert hasattr(lib, n), n


def route(lib, x=at(0), dt=BF16, N=10, K=16, bias=at(1), score=SOFTMAX, G=4, keep=2, best=2, S=3, renorm=1, valid=at(2),
          ids=at(3), w=at(4), z=at(5)):
    return lib.kmeans_route(x, dt, N, K, bias, score, G, keep, best, S, renorm, 1.0, valid, ids, w, z, None)


@pytest.mark.parametrize("kw, code, word", [
    (dict(dt=3), EUNSUPPORTED, "dtype 3"),
    (dict(score=2), EUNSUPPORTED, "score 2"),
    (dict(score=-1), EUNSUPPORTED, "score -1"),
    (dict(N=-1), EINVAL, "N=-1"),
    (dict(N=1 << 31), EINVAL, "N=2147483648"),
    (dict(K=0), EINVAL, "K=0"),
    (dict(S=0), EINVAL, "S=0"),
    (dict(S=17), EINVAL, "S=17"),
    (dict(K=260, G=1, keep=1, S=65), EUNSUPPORTED, "S=65"),
    (dict(G=0), EINVAL, "groups=0"),
    (dict(G=3), EINVAL, "groups=3"),
    (dict(G=-4), EINVAL, "groups=-4"),
    (dict(K=260, G=65), EUNSUPPORTED, "groups=65"),
    (dict(keep=0), EINVAL, "top_groups=0"),
    (dict(keep=5), EINVAL, "top_groups=5"),
    (dict(best=0), EINVAL, "group_best=0"),
    (dict(best=3), EINVAL, "group_best=3"),
    (dict(x=None), EINVAL, "logits"),
    (dict(ids=None), EINVAL, "ids"),
    (dict(w=None), EINVAL, "weights"),
    (dict(z=None), EINVAL, "chosen"),
    (dict(x=at(0, 1)), EINVAL, "misaligned pointer: logits"),
    (dict(bias=at(1, 2)), EINVAL, "misaligned pointer: bias"),
    (dict(ids=at(3, 2)), EINVAL, "misaligned pointer: ids"),
    (dict(w=at(3, 8)), EINVAL, "ids overlaps weights"),
    (dict(z=at(0, 16)), EINVAL, "chosen overlaps logits"),
    (dict(w=at(1, 60)), EINVAL, "weights overlaps bias"),
    (dict(ids=at(2, 8)), EINVAL, "ids overlaps valid"),
])
def test_route_refusals(lib, kw, code, word):
    assert route(lib, **kw) == code
    assert word in err(lib)


def test_route_of_no_rows_is_nothing(lib):
    assert route(lib, N=0, x=None, valid=None, ids=None, w=None, z=None) == 0
    assert route(lib, N=0, x=None, ids=None, w=None, z=None, S=0) == EINVAL


def grad(lib, x=at(0), dt=F16, N=10, K=16, ids=at(1), z=at(2), dw=at(3), S=3, score=SOFTMAX, renorm=1, acc=0, out=at(4)):
    return lib.kmeans_route_grad(x, dt, N, K, ids, z, dw, S, score, renorm, 1.0, acc, out, None)


@pytest.mark.parametrize("kw, code, word", [
    (dict(dt=7), EUNSUPPORTED, "dtype 7"),
    (dict(score=5), EUNSUPPORTED, "score 5"),
    (dict(N=1 << 40), EINVAL, "N="),
    (dict(K=-3), EINVAL, "K=-3"),
    (dict(S=0), EINVAL, "S=0"),
    (dict(S=20), EINVAL, "S=20"),
    (dict(K=100, S=70), EUNSUPPORTED, "S=70"),
    (dict(renorm=0, x=None), EINVAL, "logits"),
    (dict(z=None), EINVAL, "chosen"),
    (dict(ids=None), EINVAL, "ids"),
    (dict(dw=None), EINVAL, "dweights"),
    (dict(out=None), EINVAL, "dlogits"),
    (dict(out=at(4, 1)), EINVAL, "misaligned pointer: dlogits"),
    (dict(renorm=0, x=at(4)), EINVAL, "dlogits overlaps logits"),
    (dict(out=at(3, 64)), EINVAL, "dlogits overlaps dweights"),
    (dict(z=at(4, 4)), EINVAL, "dlogits overlaps chosen"),
])
def test_route_grad_refusals(lib, kw, code, word):
    assert grad(lib, **kw) == code
    assert word in err(lib)


def test_route_grad_takes_what_it_reads(lib):
    # (no rows: nothing is launched) logits only for softmax without renormalise, chosen only otherwise
    assert grad(lib, N=0, x=None, ids=None, z=None, dw=None, out=None) == 0
    assert grad(lib, renorm=0, z=None, dw=None) == EINVAL and "dweights" in err(lib)
    assert grad(lib, score=SIGMOID, renorm=0, x=None, dw=None) == EINVAL and "dweights" in err(lib)


def tensors(km, n=3, size=1000, bits=32, masters=False, **changes):
    """n tensors at addresses far apart; changes: {field: {index: value}}."""
    ts = (km._AdamWTensor * n)()
    for i, t in enumerate(ts):
        names = ["param", "grad", "exp_avg", "exp_avg_sq"] + ["master"] * masters
        names += ["exp_avg_scale", "exp_avg_sq_scale"] * (bits == 8)
        for k, name in enumerate(names):
            setattr(t, name, at(10 * i + k).value)
        t.numel, t.decay = size, 1.0
    for name, by in changes.items():
        for i, v in by.items():
            setattr(ts[i], name, v)
    return ts


def table(lib, ts, pdt=F32, gdt=F32, bits=32, room=None):
    need = lib.kmeans_adamw_table_bytes(ts, len(ts))
    buf = torch.zeros(max(1, need), dtype=torch.uint8)
    return lib.kmeans_adamw_table(ts, len(ts), pdt, gdt, bits, buf.data_ptr(), need if room is None else room), buf


@pytest.mark.parametrize("kw, code, word", [
    (dict(pdt=3), EUNSUPPORTED, "param dtype 3"),
    (dict(gdt=-2), EUNSUPPORTED, "grad dtype -2"),
    (dict(bits=16), EUNSUPPORTED, "bits=16"),
    (dict(room=64), EWORKSPACE, "table too small"),
    (dict(ch=dict(numel={1: -1})), EINVAL, "tensor 1: numel=-1"),
    (dict(ch=dict(numel={1: 1 << 40})), EINVAL, "tensor 1: numel"),
    (dict(ch=dict(param={2: None})), EINVAL, "tensor 2: param must be non-null"),
    (dict(ch=dict(grad={0: None})), EINVAL, "tensor 0: grad must be non-null"),
    (dict(ch=dict(exp_avg={0: None})), EINVAL, "exp_avg must be non-null"),
    (dict(ch=dict(exp_avg_sq={1: None})), EINVAL, "exp_avg_sq must be non-null"),
    (dict(bits=8), EINVAL, "exp_avg_scale must be non-null"),
    (dict(ch=dict(param={0: at(0).value + 2})), EINVAL, "misaligned pointer: param"),
    (dict(ch=dict(exp_avg={0: at(2).value + 1})), EINVAL, "misaligned pointer: exp_avg"),
    (dict(ch=dict(decay={0: -1.0})), EINVAL, "decay"),
    (dict(ch=dict(decay={0: float("nan")})), EINVAL, "decay"),
    (dict(ch=dict(master={1: at(99).value}), pdt=BF16), EINVAL, "for every tensor or for none"),
    (dict(masters=True), EINVAL, "needs no master"),
    # the same tensor twice, a parameter inside another's state, a gradient that is a parameter
    (dict(ch=dict(param={1: at(0).value})), EINVAL, "overlaps"),
    (dict(ch=dict(param={1: at(2).value + 3996})), EINVAL, "overlaps exp_avg of tensor 0"),
    (dict(ch=dict(grad={1: at(0).value + 64})), EINVAL, "overlaps"),
    (dict(ch=dict(exp_avg={0: at(3).value})), EINVAL, "overlaps"),
])
def test_adamw_table_refusals(lib, kw, code, word):
    import exact_means_clustering_amd as km
    kw = dict(kw)
    ts = tensors(km, masters=kw.pop("masters", False), **kw.pop("ch", {}))
    assert table(lib, ts, **kw)[0] == code
    assert word in err(lib)


def test_adamw_table(lib):
    import exact_means_clustering_amd as km
    ts = tensors(km, size=5000)
    ts[1].numel = 0
    ts[1].param = ts[1].grad = None                                  # a tensor without elements needs no memory
    assert lib.kmeans_adamw_chunks(ts, 3) == 4                       # 4096 elements each
    assert lib.kmeans_adamw_table_bytes(ts, 3) % 256 == 0
    rc, buf = table(lib, ts)
    assert rc == 0
    item = buf[:3 * 80].view(3, 80)
    words = item.contiguous().view(torch.int64).view(3, 10)
    assert words[0, 0] == ts[0].param and words[2, 3] == ts[2].exp_avg and words[2, 7] == 5000
    assert words[:, 8].tolist() == [0, 2, 2]                         # first chunks
    assert buf[256:256 + 16].view(torch.int32).tolist() == [0, 0, 2, 2]
    # gradients may be one array
    ts[2].grad = ts[0].grad
    assert table(lib, ts)[0] == 0
    # neighbours touch and do not overlap
    ts[2].param = ts[0].param + 20000
    assert table(lib, ts)[0] == 0
    for n, ok in ((0, 0), (-1, 0), ((1 << 20) + 1, 0)):
        assert lib.kmeans_adamw_table_bytes(ts, n) == ok and lib.kmeans_adamw_chunks(ts, n) == -1
    assert lib.kmeans_adamw_table_bytes(None, 2) == 0 and "tensors" in err(lib)
    assert lib.kmeans_adamw_table(ts, 3, F32, F32, 32, None, 1 << 20) == EINVAL


def step(lib, t=at(0), n=3, chunks=4, pdt=F32, gdt=F32, bits=32, masters=0, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, k=1,
         lr_at=None, k_at=None, gs=None, skip=None):
    return lib.kmeans_adamw(t, n, chunks, pdt, gdt, bits, masters, lr, b1, b2, eps, wd, k, lr_at, k_at, gs, skip, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw, code, word", [
    (dict(pdt=5), EUNSUPPORTED, "param dtype"),
    (dict(gdt=5), EUNSUPPORTED, "grad dtype"),
    (dict(bits=4), EUNSUPPORTED, "bits=4"),
    (dict(n=0), EINVAL, "count=0"),
    (dict(chunks=-1), EINVAL, "chunks=-1"),
    (dict(chunks=1 << 31), EINVAL, "chunks="),
    (dict(masters=1), EINVAL, "master"),
    (dict(b1=1.0), EINVAL, "beta1"),
    (dict(b1=NAN), EINVAL, "beta1"),
    (dict(b2=-0.1), EINVAL, "beta2"),
    (dict(eps=-1e-8), EINVAL, "eps"),
    (dict(eps=INF), EINVAL, "eps"),
    (dict(lr=INF), EINVAL, "lr"),
    (dict(wd=NAN), EINVAL, "weight_decay"),
    (dict(k=0), EINVAL, "step=0"),
    (dict(t=None), EINVAL, "table"),
    (dict(t=at(0, 128)), EINVAL, "256-byte"),
    (dict(lr_at=at(1, 2)), EINVAL, "lr_at"),
    (dict(k_at=at(1, 4)), EINVAL, "step_at"),
    (dict(gs=at(1, 1)), EINVAL, "grad_scale_at"),
])
def test_adamw_refusals(lib, kw, code, word):
    assert step(lib, **kw) == code
    assert word in err(lib)


def test_adamw_of_nothing_is_nothing(lib):
    assert step(lib, chunks=0) == 0


def test_binding_refuses_what_is_not_on_the_gpu():
    import exact_means_clustering_amd as km
    x, i, f = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    m, v, _ = km.adamw_states([x])
    for call in (lambda: km.route(x, 2), lambda: km.route_grad(x, i, f, f), lambda: km.adamw_plan([x], [x], m, v)):
        with pytest.raises(km.KMeansError, match="CUDA tensor"):
            call()
    with pytest.raises(km.KMeansError, match="empty"):
        km.adamw_plan([], [], [], [])
    with pytest.raises(km.KMeansError, match="grads must have 1"):
        km.adamw_plan([x], [], m, v)
    with pytest.raises(km.KMeansError, match="bits=16"):
        km.adamw_states([x], 16)
    with pytest.raises(km.KMeansError, match="adamw_plan"):
        km.adamw(None, lr=1e-3, step=1)


def test_states():
    import exact_means_clustering_amd as km
    ps = [torch.zeros(3, 100, dtype=torch.bfloat16), torch.zeros(0), torch.zeros(256), torch.zeros(())]
    m, v, s = km.adamw_states(ps)
    assert s is None and all(a.shape == p.shape and a.dtype == torch.float32 for p, a in zip(ps, m)) and len(v) == 4
    m, v, s = km.adamw_states(ps, bits=8)
    assert [a.dtype for a in m] == [torch.float8_e4m3fn] * 4 and [a.dtype for a in v] == [torch.float8_e5m2] * 4
    assert [t.numel() for t in s[0]] == [t.numel() for t in s[1]] == [2, 0, 1, 1]


@pytest.mark.parametrize("name", ["route", "route_grad", "adamw"])
def test_binding_shows_its_stream_argument(name):
    import inspect

    import exact_means_clustering_amd as km
    fn = getattr(km, name)
    p = inspect.signature(fn).parameters["stream"]
    assert p.kind is inspect.Parameter.KEYWORD_ONLY and p.default is None
    assert "stream" in fn.__doc__
