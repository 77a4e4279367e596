"""Refusals of the operators between the projections, before any device work."""
import ctypes

import pytest

import q4_q8_int8_gb300 as mmq
from q4_q8_int8_gb300 import build as mmq_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    mmq_build.build()
    return mmq.load_library()


def rope(**change):
    p = mmq.mmq_qk_norm_rope_t(0x10000, 0x20000, 0x30000, 0x40000, None, None, 0x50000, 0x60000, 0x70000, 0x80000,
                               6 * 64, 3, 100, 10, 4, 1, 64, 64, (ctypes.c_int32 * 4)(32), 0, mmq.MMQ_TYPE_F16, 1e-6)
    for k, v in change.items():
        setattr(p, k, (ctypes.c_int32 * 4)(*v) if k == "sections" else v)
    return mmq.mmq_qk_norm_rope(p, None)


@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(q=None), dict(k_cache=None), dict(v_cache=None), dict(positions=None), dict(slots=None),
    dict(cos_table=None), dict(sin_table=None), dict(tokens=-1), dict(tokens=2 ** 31), dict(n_slots=-1),
    dict(heads=0), dict(kv_heads=0), dict(head_dim=60), dict(head_dim=264), dict(head_dim=8), dict(rot=72),
    dict(rot=60), dict(rot=-8), dict(ld=6 * 64 - 4), dict(ld=6 * 64 + 2), dict(type=mmq.MMQ_TYPE_F32), dict(type=-1),
    dict(sections=(31,)), dict(sections=(33, -1)), dict(sections=(16, 8, 4, 8)), dict(table_rows=-1)])
def test_rope_refuses_arguments(change):
    assert rope(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("name,by", [("qkv", 8), ("q", 8), ("k_cache", 2), ("v_cache", 8), ("q_weight", 4),
                                     ("k_weight", 8), ("cos_table", 4), ("sin_table", 4), ("positions", 2), ("slots", 1)])
def test_rope_refuses_alignment(name, by):
    assert rope(**{name: 0x90000 + by}) == mmq.MMQ_ERR_ALIGN


def test_null_structs():
    assert mmq.load_library().mmq_qk_norm_rope(None, None) == mmq.MMQ_ERR_ARG
