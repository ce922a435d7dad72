"""The few-token operators' binding, without a GPU: what it packs for the library and what it refuses."""
import pytest
import torch

import w4a4_mxfp4_post_b200 as kq

CPU = torch.device("cpu")


class Cuda(torch.Tensor):
    """A host tensor that passes for one on the device, for checks that look no further."""

    is_cuda = True


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def batch_of(table, lens=True):
    B = table.shape[0]
    packed, n = kq._batch(table.as_subclass(Cuda), i32(B + 1), i32(B) if lens else None, CPU)
    assert n == B
    return dict(zip(("table", "stride", "pages", "cu", "lens", "batch"), kq._BATCH.unpack(packed)))


@pytest.mark.parametrize("lens", [True, False])
def test_block_table_row_strides(lens):
    """The library gets the tensor's own distance of rows: never one that leads outside of it."""
    wide = i32(4, 9)
    assert batch_of(wide, lens)["stride"] == 9
    got = batch_of(wide[:, 2:7], lens)
    assert got["stride"] == 9 and got["pages"] == 5
    assert batch_of(wide[::2, :3], lens)["stride"] == 18
    # a single row's stride is never used, whatever it is
    assert batch_of(wide[:1, :5].as_strided((1, 5), (0, 1)), lens)["stride"] >= 5
    assert batch_of(i32(5).as_strided((1, 5), (2, 1)), lens)["stride"] >= 5
    # rows that share memory: the largest place that stride 5 reaches would be 19 of 5
    for shared in (i32(1, 5).expand(4, -1), i32(12).as_strided((3, 5), (3, 1)), i32(8).unfold(0, 5, 1), i32(1, 1).expand(2, -1)):
        with pytest.raises(ValueError, match="overlap"):
            batch_of(shared, lens)
