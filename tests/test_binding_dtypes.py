"""The type that the binding tells the libraries for the tensors of a call, where the caller gives
none: bfloat16 or float32, the same for all of them, and a refusal otherwise (the kernels would
read past the end of narrower tensors).  No GPU: everything is refused or recorded before a
library is called."""
import numpy as np
import pytest
import torch

import top_kv_routing_b200 as msa
from top_kv_routing_b200 import abi

BF16, F32 = torch.bfloat16, torch.float32
OTHERS = [torch.float16, torch.float64, torch.float8_e4m3fn, torch.int32, torch.uint8]


def _t(dtype):
    return None if dtype is None else torch.zeros(64).to(dtype)


def _append(q, k, v, **kw):
    ints = np.zeros(8, np.int32)
    return msa.msa_paged_append(_t(q), _t(k), _t(v), ints, 1, 1, 1, 1, 1, 128, _t(BF16), 1, 16, ints, 1, ints, None, 0,
                                1e6, None if q is None else _t(BF16), stream=0, **kw)


def _pool(k, v, kr, **kw):
    longs = np.zeros(2, np.int64)
    return msa.msa_pool_blocks(_t(k), _t(v), _t(kr), longs, longs, 1, 1, 1, 128, 64, 1e6, stream=0, **kw)


def _route(q, **kw):
    z = np.zeros(16, np.uint16)
    return msa.msa_route_topk(_t(q), [0, 1], z, np.zeros(2, np.int64), 1, 1, 1, 32, 8, 128, 4, np.zeros(4, np.int32),
                              np.zeros(4, np.float32), np.zeros(256, np.uint8), stream=0, **kw)


@pytest.fixture
def told(monkeypatch):
    """The types that reach the libraries, in place of the calls."""
    seen = []

    class Recorder:
        def __init__(self, at):
            self.at = at

        def __call__(self, *args):
            seen.append(args[self.at])
            return 0

    monkeypatch.setattr(abi.paged_lib, "msa_paged_append", Recorder(3))
    monkeypatch.setattr(abi.pool_lib, "msa_pool_blocks", Recorder(3))
    monkeypatch.setattr(abi.route_lib, "msa_route_topk", Recorder(1))
    return seen


@pytest.mark.parametrize("dtype,code", [(BF16, msa.MSA_BF16), (F32, msa.MSA_F32)])
def test_types_that_the_calls_take(told, dtype, code):
    _append(dtype, dtype, dtype)
    _append(None, dtype, dtype)
    _pool(dtype, dtype, dtype)
    _pool(None, None, dtype)
    _route(dtype)
    assert told == [code] * 5


@pytest.mark.parametrize("other", OTHERS)
def test_other_types_are_refused(told, other):
    for call, args in ((_append, (other, other, other)), (_append, (BF16, BF16, other)), (_append, (other, F32, F32)),
                       (_append, (None, other, BF16)), (_pool, (other, other, other)), (_pool, (F32, F32, other)),
                       (_pool, (None, None, other)), (_route, (other,))):
        with pytest.raises(msa.MsaError) as e:
            call(*args)
        assert e.value.status == msa.MSA_ERR_UNSUPPORTED and str(other) in str(e.value)
    assert told == []


def test_tensors_of_two_types_are_refused(told):
    for call, args in ((_append, (BF16, F32, F32)), (_append, (F32, F32, BF16)), (_append, (F32, BF16, F32)),
                       (_append, (None, BF16, F32)), (_pool, (F32, BF16, F32)), (_pool, (BF16, None, F32))):
        with pytest.raises(msa.MsaError) as e:
            call(*args)
        assert e.value.status == msa.MSA_ERR_INVALID_ARG
    assert told == []


def test_a_type_that_is_given_is_told_as_it_is(told):
    _append(BF16, BF16, BF16, in_dtype=msa.MSA_F32)
    _pool(F32, F32, F32, in_dtype=msa.MSA_BF16)
    _route(BF16, q_dtype=7)
    assert told == [msa.MSA_F32, msa.MSA_BF16, 7]
