"""The few-token operators' binding, without a GPU: what it packs for the library and what it refuses."""
import ctypes
import os
import subprocess

import pytest
import torch

import w4a4_mxfp4_post_b200 as kq
from w4a4_mxfp4_post_b200 import build as kbuild

CPU = torch.device("cpu")
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kq.lib()


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


def test_attention_rows_end_before_32_bits(L):
    """The rows of a kv head are counted in 32 bits, to the end of the item behind the last: more are refused, by the size query too."""
    cache, seqs = kq._CACHE.pack(16, 16, 16, 16, 4, 2, 16, 64), kq._BATCH.pack(16, 3, 3, 16, 16, 2)
    most = (1 << 31) - (1 << 10)
    for T, hq in (((1 << 31) - 1, 2), (most + 1, 2), (most // 2 + 1, 4)):
        assert L.mx_paged_attention(P(16), 256, 64, cache, seqs, 1.0, 1, P(16), T, hq, 1, P(16), 1 << 62, None) == -2
        assert "2^31 - 2^10" in L.kq_last_error().decode()
        assert L.mx_attention_workspace(T, hq, 2, 64, 1) == -1
    # (the last that is taken fails the next check)
    assert L.mx_paged_attention(None, 256, 64, cache, seqs, 1.0, 1, P(16), most, 2, 1, P(16), 1 << 62, None) == -1
    assert L.mx_attention_workspace(most, 2, 2, 64, 1) > 0
    for bad in ((1 << 31, 2, 2, 64, 0), (1 << 62, 1 << 62, 2, 64, 1), (4, 1 << 40, 2, 64, 1), (4, 1 << 17, 1 << 17, 64, 1)):
        assert L.mx_attention_workspace(*bad) == -1


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """build() into tmp_path with compilers that only write their output; `failing` maps a compiler to what it raises."""
    calls, failing = [], {}

    def run(cmd, check):
        name = os.path.basename(cmd[0])
        calls.append(name)
        if name in failing:
            raise failing[name]
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(name)

    monkeypatch.setattr(kbuild.subprocess, "run", run)
    monkeypatch.setattr(kbuild, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(kbuild, "binding_path", lambda: str(tmp_path / "binding.so"))
    return calls, failing, tmp_path


def test_build_makes_the_library_and_the_binding(compilers):
    calls, _, tmp = compilers
    assert kbuild.build() == kbuild.LIB and calls == ["nvcc", "g++"]
    assert (tmp / "lib.so").read_text() == "nvcc" and (tmp / "binding.so").read_text() == "g++"
    assert kbuild.build() == kbuild.LIB and len(calls) == 2                  # nothing is stale
    kbuild.build(force=True)
    assert len(calls) == 4


@pytest.mark.parametrize("error", [subprocess.CalledProcessError(1, ["g++"]), FileNotFoundError("g++")], ids=["fails", "missing"])
def test_build_makes_the_library_without_the_binding(compilers, error):
    """The library needs nvcc alone: where the native part of the binding does not compile, it is left out, and no older one stays."""
    calls, failing, tmp = compilers
    (tmp / "binding.so").write_text("older")
    failing["g++"] = error
    with pytest.warns(UserWarning, match="left out"):
        assert kbuild.build(force=True) == kbuild.LIB
    assert (tmp / "lib.so").exists() and not (tmp / "binding.so").exists() and calls == ["nvcc", "g++"]


def test_build_without_torch_metadata(compilers, monkeypatch):
    from importlib.metadata import PackageNotFoundError

    def no_metadata():
        raise PackageNotFoundError("torch")

    monkeypatch.setattr(kbuild, "binding_path", no_metadata)
    with pytest.warns(UserWarning, match="left out"):
        assert kbuild.build(force=True) == kbuild.LIB and compilers[2].joinpath("lib.so").exists()


def test_build_fails_without_the_library(compilers):
    compilers[1]["nvcc"] = subprocess.CalledProcessError(1, ["nvcc"])
    with pytest.raises(subprocess.CalledProcessError):
        kbuild.build(force=True)


@pytest.mark.parametrize("why", ["absent", "no metadata", "no binary"])
def test_calls_without_the_native_binding(L, monkeypatch, tmp_path, why):
    """Where it was not built or does not load, the Python binding does the calls: found out once, and said."""
    from importlib.metadata import PackageNotFoundError

    asked = []

    def path():
        asked.append(1)
        if why == "no metadata":
            raise PackageNotFoundError("torch")
        if why == "no binary":
            (tmp_path / "binding.so").write_text("not a shared object")
        return str(tmp_path / "binding.so")

    monkeypatch.setattr(kbuild, "binding_path", path)
    monkeypatch.setattr(kq, "_native_module", None)
    if why == "absent":
        assert kq._native() is False
    else:
        with pytest.warns(UserWarning, match="does not load"):
            assert kq._native() is False
    assert kq._native() is False and len(asked) == 1
    with pytest.raises(ValueError, match="CUDA"):            # as the Python binding says it
        kq.mxf4_gemv(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))


def test_strides_of_one_token_or_head_are_not_read(L):
    """The stride of a dimension of size 1 may be anything: these calls fail the check behind the strides'."""
    seqs = kq._BATCH.pack(16, 3, 3, 16, 16, 2)
    one, two = (kq._CACHE.pack(16, 16, 16, 16, 4, heads, 16, 64) for heads in (1, 2))
    for cache, T, st, sh in ((two, 1, 132, 64), (two, 1, -1, 64), (one, 4, 128, 3), (one, 1, 1, 1)):
        assert L.mx_cache_write(P(16), st, sh, None, st, sh, 0, cache, seqs, T, None) == -1
        assert L.mx_cache_write(P(16), 128, 64, P(8), st, sh, 0, cache, seqs, T, None) == -3
        heads = 1 if cache == one else 4
        assert L.mx_paged_attention(P(16), st, sh, cache, seqs, 1.0, 1, None, T, heads, 1, P(16), 1 << 40, None) == -1
    for cache, T, st, sh in ((two, 2, 132, 64), (two, 1, 128, 3), (one, 2, 132, 64)):
        assert L.mx_cache_write(P(16), st, sh, None, 128, 64, 0, cache, seqs, T, None) == -3
        assert L.mx_paged_attention(P(16), st, sh, cache, seqs, 1.0, 1, None, T, 4, 1, P(16), 1 << 40, None) == -3
