"""Refusals of the AdamW step with stochastic rounding, without a GPU."""

import inspect

import pytest

from tests.test_train_abi import EINVAL, EUNSUPPORTED, F32, INF, NAN, at, err, lib, table, tensors  # noqa: F401 (a fixture)


def step(lib, t=at(0), n=3, chunks=4, pdt=F32, gdt=F32, bits=8 | 256, masters=0, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, k=1,  # noqa: F811
         lr_at=None, k_at=None, gs=None, skip=None):
    return lib.kmeans_adamw(t, n, chunks, pdt, gdt, bits, masters, lr, b1, b2, eps, wd, k, lr_at, k_at, gs, skip, None)


@pytest.mark.parametrize("kw, code, word", [
    (dict(bits=32 | 256), EUNSUPPORTED, "bits=288"),
    (dict(bits=256), EUNSUPPORTED, "bits=256"),
    (dict(bits=8 | 512), EUNSUPPORTED, "bits=520"),
    (dict(pdt=5), EUNSUPPORTED, "param dtype"),
    (dict(n=0), EINVAL, "count=0"),
    (dict(chunks=-1), EINVAL, "chunks=-1"),
    (dict(masters=1), EINVAL, "master"),
    (dict(b2=1.0), EINVAL, "beta2"),
    (dict(eps=INF), EINVAL, "eps"),
    (dict(lr=NAN), EINVAL, "lr"),
    (dict(k=0), EINVAL, "step=0"),
    (dict(t=None), EINVAL, "table"),
    (dict(k_at=at(1, 4)), EINVAL, "step_at"),
])
def test_refusals(lib, kw, code, word):  # noqa: F811
    assert step(lib, **kw) == code
    assert word in err(lib)


def test_a_table_is_that_of_8_bits(lib):  # noqa: F811
    import exact_means_clustering_amd as km
    ts = tensors(km, bits=8)
    assert table(lib, ts, bits=8)[0] == 0
    assert table(lib, ts, bits=8 | 256)[0] == EUNSUPPORTED and "bits=264" in err(lib)


def test_nothing_is_nothing(lib):  # noqa: F811
    assert step(lib, chunks=0) == 0


def test_the_binding_says_which_rounding():
    import exact_means_clustering_amd as km
    p = inspect.signature(km.adamw).parameters
    assert p["rounding"].default == "nearest"
    assert "stochastic" in km.adamw.__doc__ and "frozen" in km.adamw.__doc__
