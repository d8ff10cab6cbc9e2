"""Paged KV cache on the host: what the calls allow beyond the refusals of test_paged_host.py, the build,
and rules of the kernels' source.  No call here reaches a kernel."""
import os

import pytest
import torch

import fp8_quantization_amax_b200 as fq
from fp8_quantization_amax_b200 import build

CSRC = os.path.join(os.path.dirname(os.path.abspath(fq.__file__)), "csrc")


# ------------------------------------------------------------------ kernels' source

@pytest.mark.parametrize("name", ["kv_plan.cu", "kv_append.cu", "attention.cu", "kv_pages.cuh", "dequantize.cu", "quantize.cu",
                                  "fp8q_device.cuh", "gemm_sm100.cu", "gemm_mx_sm100.cu"])
def test_dependent_kernels_use_no_read_only_loads(name):
    """A kernel launched as a programmatic dependent lives while the one before it still writes its inputs:
    the read-only path (memory that nobody writes meanwhile) is not for them."""
    with open(os.path.join(CSRC, name)) as f:
        code = "\n".join(line.split("//")[0] for line in f)
    assert "__ldg" not in code and "ld.global.nc" not in code
    if name != "gemm_sm100.cu":                      # (there: pointers of the cooperative launch, no dependent)
        assert "__restrict__" not in code


# ------------------------------------------------------------------ rotation table

def test_rope_turns_defaults_follow_the_kind():
    """`high` left out: 4 turns for the smooth kind, 32 for the ramp (the value of the paper it follows)."""
    for kind, high in ((fq.ROPE_SMOOTH, 4.0), (fq.ROPE_RAMP, 32.0)):
        got, gain = fq.rope_turns(128, 500000.0, kind, 8.0)
        want, same = fq.rope_turns(128, 500000.0, kind, 8.0, 8192.0, 1.0, high)
        assert torch.equal(got, want) and gain == same
        other, _ = fq.rope_turns(128, 500000.0, kind, 8.0, 8192.0, 1.0, 36.0 - high)
        assert not torch.equal(got, other)


# ------------------------------------------------------------------ build

def test_c_library_is_built_where_the_python_calls_cannot_be(monkeypatch, tmp_path):
    """No C++ compiler: libfp8q.so is linked, then the failure is raised; an older _torch_calls.so is gone."""
    build.build()
    lib, calls = tmp_path / "lib.so", tmp_path / "calls.so"
    calls.write_bytes(b"of another header")
    os.utime(calls, (1, 1))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "CALLS", str(calls))
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="torch_calls"):
        build.build()
    assert lib.stat().st_size > 1 << 20 and not calls.exists()
    monkeypatch.setenv("CXX", str(tmp_path / "missing"))
    lib.unlink()
    with pytest.raises(FileNotFoundError):
        build.build()
    assert lib.stat().st_size > 1 << 20
