"""The few-token operators where their ranges end: tables, batches, value ranges, streams.

Inputs and 64-bit forms are those of test_gpu_serve.py and serve_ref.py.
"""
import pytest
import torch

import serve_ref as ref
import w4a4_mxfp4_post_b200 as kq
from test_gpu_serve import Plan, attend, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["native", "python"])
def either_binding(request, monkeypatch):
    """For what the binding does: its native part, and the Python calls."""
    if request.param == "python":
        monkeypatch.setattr(kq, "_native", lambda: False)
    else:
        assert kq._native(), "the binding's native part is not built"


def test_tables_whose_rows_share_memory_are_refused(cuda_device, either_binding):
    """An expanded table would be read past its end; its copy is taken."""
    p = Plan([40, 40, 40], [2, 2, 2], 2, 64, 16, seed=1)
    p.table = p.table[:1].expand(3, -1)
    q = normal(6, 8, 64, key=1)
    before = [t.clone() for t in p.cache]
    for table in (p.table, p.table[0].as_strided((3, p.table.shape[1]), (1, 1))):
        with pytest.raises(ValueError, match="overlap"):
            kq.mx_paged_attention(q, *p.cache, table, p.cud, p.lensd)
        with pytest.raises(ValueError, match="overlap"):
            kq.mx_cache_read(*p.cache, table, p.cud, 6)
        with pytest.raises(ValueError, match="overlap"):
            kq.mx_cache_write(q[:, :2], q[:, 2:4], *p.cache, table, p.cud, p.lensd)
    assert all(torch.equal(a, b) for a, b in zip(before, p.cache))
    p.table = p.table.contiguous()
    attend(p, q, max_new=2)


def test_a_single_sequence_with_any_row_stride(cuda_device, either_binding):
    p = Plan([70], [3], 2, 64, 16, seed=2)
    q = normal(3, 8, 64, key=2)
    want = attend(p, q, max_new=3)
    for stride in (0, 1, 1000):
        p.table = p.table.as_strided(p.table.shape, (stride, 1))
        assert torch.equal(attend(p, q, max_new=3), want)
