"""The weight objects: what they hand out is the caller's, and holds no addresses."""
import copy
import dataclasses
import pickle

import pytest
import torch

from quantized_linear_layers_nf4_b200.build import build


@pytest.fixture(scope="module")
def nf4():
    build()
    import quantized_linear_layers_nf4_b200 as m
    return m


def _weight(nf4, kind):
    n, k = 8, 128
    wq = torch.arange(n * k // 2).to(torch.uint8)
    if kind == "int4":  # on the host, which its constructor refuses
        w = object.__new__(nf4.Int4Weight)
        w.__dict__.update(n=n, k=k, group=64, wq=wq, scale=torch.ones(2, n), zero=None)
        return w
    return nf4.NF4Weight(n, k, wq, torch.zeros(n * k // 64, dtype=torch.int8), torch.ones(1), torch.zeros(1), kind)


@pytest.mark.parametrize("kind", ["nf4", "fp4", "int4"])
def test_a_struct_is_the_callers(nf4, kind):
    w = _weight(nf4, kind)
    want = bytes(w.struct())
    mine = w.struct()
    assert mine.wq == w.wq.data_ptr() and mine.n == w.n
    mine.n, mine.wq, mine.magic = 5, 0, 0
    assert bytes(w.struct()) == want
    assert bytes(w._struct_ref()[1]) == want
    w._struct_ref()
    assert w.struct() is not w._struct_ref()[1]


@pytest.mark.parametrize("kind", ["nf4", "fp4", "int4"])
def test_what_a_weight_holds_is_its_fields(nf4, kind):
    w = _weight(nf4, kind)
    w._struct_ref()
    names = [f.name for f in dataclasses.fields(w)]
    assert list(vars(w)) == names
    again = pickle.loads(pickle.dumps(vars(w)))
    assert all(torch.equal(again[i], v) if isinstance(v, torch.Tensor) else again[i] == v for i, v in vars(w).items())
    for other in (copy.copy(w), copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert list(vars(other)) == names
        st = other._struct_ref()[1]
        assert st.wq == other.wq.data_ptr() and st.k == other.k
    # a weight whose tensor is another one points to that
    if kind != "int4":
        w.wq = w.wq.clone()
        assert w._struct_ref()[1].wq == w.wq.data_ptr() == w.struct().wq


def test_an_integer_weight_stays_frozen(nf4):
    w = _weight(nf4, "int4")
    w._struct_ref()
    with pytest.raises(dataclasses.FrozenInstanceError):
        w.n = 3
    with pytest.raises(dataclasses.FrozenInstanceError):
        w._kept = None
