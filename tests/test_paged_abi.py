"""The paged-batch library without a GPU: exported symbols, prototypes, constants, and every
argument the host checks must refuse (before anything reaches a device)."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from test_abi import ROOT, _declared, _expected_ctype, _prototypes

HEADER = "msa_paged.h"


@pytest.fixture(scope="module")
def msa():
    import top_kv_routing_b200 as m
    return m


def test_library_exports_declared_symbols(msa):
    path = os.path.join(msa.LIB_DIR, "libmsa_paged.so")
    assert path in msa.loaded_libraries()
    names = _declared(HEADER)
    assert len(names) == 5
    out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True, check=True).stdout
    exported = set(line.split()[-1] for line in out.splitlines() if line.strip())
    assert not [n for n in names if n not in exported]


def test_binding_argtypes_follow_the_header_prototypes(msa):
    checked = 0
    for name, params in _prototypes(HEADER).items():
        fn = getattr(msa.paged_lib, name)
        if fn.argtypes is None:
            continue
        assert len(fn.argtypes) == len(params), name
        for got, par in zip(fn.argtypes, params):
            want = _expected_ctype(par)
            assert got == want or (want is ctypes.c_void_p and issubclass(got, ctypes._Pointer)), (name, par)
        checked += 1
    assert checked >= 4


def test_constants_match_the_headers(msa):
    text = open(os.path.join(ROOT, "include", "msa_common.h")).read()
    assert msa.MSA_DEVERR_BAD_PAGE == int(re.search(r"#define MSA_DEVERR_BAD_PAGE (\d+)u", text).group(1))
    bits = [int(v) for v in re.findall(r"#define MSA_DEVERR_\w+ (\d+)u", text)]
    assert len(set(bits)) == len(bits) and all(b & (b - 1) == 0 for b in bits)
    text = open(os.path.join(ROOT, "include", HEADER)).read()
    assert msa.MSA_PAGED_MAX_SEQS == int(re.search(r"#define MSA_PAGED_MAX_SEQS (\d+)", text).group(1))


def _aligned(n=64):
    raw = np.zeros(n + 16, np.uint8)
    at = (-raw.ctypes.data) % 16
    return raw[at:at + n]


Z, I = _aligned(), np.zeros(8, np.int32)
APPEND = dict(q=Z, k_new=Z, v_new=Z, q_offsets=I, n_tokens=4, n_seqs=2, n_layers=1, n_q_heads=8, n_kv_heads=2,
              head_dim=128, kv_pages=Z, n_pages=3, page_size=16, page_table=I, max_pages=2, seq_len=I,
              pos_offset=None, rope_pos_offset=0, rope_theta=1e6, q_rot=Z, in_dtype=1, stream=0)


@pytest.mark.parametrize("change", [
    dict(k_new=None), dict(v_new=None), dict(q_offsets=None), dict(seq_len=None), dict(kv_pages=None),
    dict(page_table=None), dict(q=None), dict(q_rot=None), dict(head_dim=64), dict(n_q_heads=6),
    dict(n_q_heads=32), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=17, n_q_heads=17), dict(n_tokens=0),
    dict(n_seqs=0), dict(n_seqs=1025), dict(n_layers=0), dict(n_layers=65536), dict(n_pages=0), dict(page_size=8),
    dict(page_size=48), dict(page_size=512), dict(max_pages=0), dict(max_pages=1 << 27), dict(rope_theta=1.0),
    dict(rope_theta=float("nan")), dict(rope_theta=float("inf")), dict(q=Z[2:]), dict(k_new=Z[8:]),
    dict(v_new=Z[4:]), dict(kv_pages=Z[2:]), dict(q_rot=Z[2:]), dict(q_stride=1020), dict(k_stride=255),
    dict(k_stride=260), dict(v_stride=-256), dict(q_stride=1028),
])
def test_append_refuses(msa, change):
    with pytest.raises(msa.MsaError) as e:
        msa.msa_paged_append(**{**APPEND, **change})
    assert e.value.status == msa.MSA_ERR_INVALID_ARG and str(e.value).split(": ")[-1]


def test_append_refuses_other_types(msa):
    with pytest.raises(msa.MsaError) as e:
        msa.msa_paged_append(**{**APPEND, "in_dtype": 7})
    assert e.value.status == msa.MSA_ERR_UNSUPPORTED


ATTEND = dict(q=Z, q_offsets=I, n_tokens=4, n_seqs=2, n_layers=1, n_q_heads=8, n_kv_heads=2, head_dim=128, mem_kv=Z,
              mem_len=I, max_mem_chunks=4, group_offsets=I, n_groups=1, kv_pages=Z, n_pages=3, page_size=16,
              page_table=I, max_pages=2, seq_len=I, softmax_scale=0.1, out=Z, workspace=_aligned(1 << 12), stream=0)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q_offsets=None), dict(seq_len=None), dict(out=None), dict(workspace=None), dict(kv_pages=None),
    dict(page_table=None), dict(mem_kv=None), dict(mem_len=None), dict(group_offsets=None), dict(max_mem_chunks=0),
    dict(n_groups=-1), dict(n_groups=3), dict(head_dim=64), dict(n_q_heads=10), dict(n_q_heads=32), dict(n_tokens=0),
    dict(n_seqs=2000), dict(n_layers=0), dict(page_size=20), dict(n_pages=0), dict(max_pages=0),
    dict(softmax_scale=0.0), dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")),
    dict(softmax_scale=float("inf")), dict(q=Z[2:]), dict(mem_kv=Z[2:]), dict(out=Z[2:]), dict(kv_pages=Z[2:]),
    dict(workspace=_aligned(1 << 12)[1:]),
])
def test_attend_refuses(msa, change):
    with pytest.raises(msa.MsaError) as e:
        msa.msa_shared_attend(**{**ATTEND, **change})
    assert e.value.status == msa.MSA_ERR_INVALID_ARG and str(e.value).split(": ")[-1]


def test_attend_refuses_a_small_workspace(msa):
    with pytest.raises(msa.MsaError) as e:
        msa.msa_shared_attend(**ATTEND)
    assert e.value.status == msa.MSA_ERR_CAPACITY


def test_workspace_size_refuses(msa):
    for args in ((0, 1, 0, 1, 8, 2), (1, 0, 0, 1, 8, 2), (1, 1, 2, 1, 8, 2), (1, 1, 0, 1, 7, 2), (1, 1, 0, 0, 8, 2)):
        with pytest.raises(msa.MsaError) as e:
            msa.msa_shared_attend_workspace_size(*args)
        assert e.value.status == msa.MSA_ERR_INVALID_ARG
