"""Paged KV cache on the host: what the calls allow beyond the refusals of test_paged_host.py, the build,
and rules of the kernels' source.  No call here reaches a kernel."""
import os

import pytest
import torch

import fp8_quantization_amax_b200 as fq
from fp8_quantization_amax_b200 import build
from test_paged_host import append_args, attention_args, pages

CSRC = os.path.join(os.path.dirname(os.path.abspath(fq.__file__)), "csrc")


# ------------------------------------------------------------------ refusals

def cache_status(**kw):
    """Status of an append and an attention that have nothing to do, so that the cache alone decides."""
    L, cache = fq.lib(), pages(**kw)
    got = {L.fp8_kv_append(*append_args(cache, tokens=0)), L.fp8_attention_paged(*attention_args(cache, batch=0))}
    assert len(got) == 1
    return got.pop()


@pytest.mark.parametrize("single,change,status", [
    ("head", {}, 0), ("token", {}, 0), ("page", {}, 0), ("head", dict(page_stride=1 << 35), 2),
    ("token", dict(page_stride=1 << 35), 2), ("page", dict(token_stride=1 << 33), 2),
])
@pytest.mark.parametrize("unused", [-(1 << 46), -16, 0, 8, 1 << 50])
def test_strides_of_single_entries_are_not_used(single, change, status, unused):
    """Neither refused nor, negative, counted against the others' span."""
    d = {"head": dict(heads=1), "token": dict(page_size=1), "page": dict(num_pages=1)}[single]
    assert cache_status(**{**d, single + "_stride": unused, **change}) == status


@pytest.mark.parametrize("page,token,head,status", [
    (2048, 128, 64, 0), (2048, 64, 1024, 0), (64, 512, 256, 0), (64, 256, 4096, 0), (4096, 256, 128, 0), (8192, 80, 4096, 0),
    (2048, 64, 64, 1), (2048, 128, 128, 1), (2048, 64, 960, 1), (1024, 128, 64, 1), (128, 128, 64, 1), (64, 240, 64, 1),
    (64, 256, 4000, 1), (2032, 128, 64, 1),
])
def test_layouts_whose_places_overlap_are_refused(page, token, head, status):
    """4 pages of 16 tokens of 2 heads of 64, whichever order the dimensions lie in."""
    assert cache_status(page_stride=page, token_stride=token, head_stride=head) == status
    places = sorted(p * page + t * token + h * head for p in range(4) for t in range(16) for h in range(2))
    assert status == int(any(b - a < 64 for a, b in zip(places, places[1:])))


@pytest.mark.parametrize("fmt", [2, -1, 1 << 32, (1 << 32) + 1, -(1 << 40)])
def test_formats_that_are_none_are_refused(fmt):
    """Not cut to 32 bits first, which made 2^32 the format 0."""
    k, s = torch.empty((4, 16, 2, 64), dtype=torch.uint8), torch.empty(2)
    x, n = torch.empty((3, 2, 64), dtype=torch.bfloat16), torch.empty(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="fmt"):
        fq.fp8_attention_paged(x, k, k, s, s, torch.empty((3, 5), dtype=torch.int32), n, fmt)
    with pytest.raises(ValueError, match="fmt"):
        fq.fp8_kv_append(None, x, x, n.long(), k, k, s, s, fmt)


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


# ------------------------------------------------------------------ division of the attention's work

@pytest.mark.parametrize("n", [-1, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 64])
def test_attention_split_refuses_lengths_that_no_call_has(n):
    """Tokens are counted in an int up to 2^31 - 65: beyond, the count of tiles itself would overflow."""
    assert fq.check_attention_split([5, n], 0, 0, 148) == -1
    assert fq.check_attention_split([n, 5], 100, 4, 148) == -1


# ------------------------------------------------------------------ rotation table

def test_rope_turns_defaults_follow_the_kind():
    """`high` left out: 4 turns for the smooth kind, 32 for the ramp (the value of the paper it follows)."""
    for kind, high in ((fq.ROPE_SMOOTH, 4.0), (fq.ROPE_RAMP, 32.0)):
        got, gain = fq.rope_turns(128, 500000.0, kind, 8.0)
        want, same = fq.rope_turns(128, 500000.0, kind, 8.0, 8192.0, 1.0, high)
        assert torch.equal(got, want) and gain == same
        other, _ = fq.rope_turns(128, 500000.0, kind, 8.0, 8192.0, 1.0, 36.0 - high)
        assert not torch.equal(got, other)


@pytest.mark.parametrize("kind", [fq.ROPE_PLAIN, fq.ROPE_LINEAR, fq.ROPE_SMOOTH])
def test_rope_turns_refuses_frequencies_beyond_doubles(kind):
    with pytest.raises(fq.Fp8qError) as e:
        fq.rope_turns(256, 5e-324, kind, 2.0)
    assert e.value.status == 1
    turns, _ = fq.rope_turns(256, 1e-300, kind, 2.0)         # the largest frequency is 10^297 and finite
    assert turns.numel() == 128


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
