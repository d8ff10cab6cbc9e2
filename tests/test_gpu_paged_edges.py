"""GPU tests of the paged KV cache where its calls can go wrong without a fault: what an earlier kernel
leaves in shared memory, weights far below the largest, pages that were given away.

References and tolerances as in test_gpu_paged.py; what differs is derived beside each check.
"""
import numpy as np
import pytest
import torch

import fp8_quantization_amax_b200 as fq
from helpers import dev_bf16
from test_gpu_paged import append_case, bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    assert torch.cuda.is_available()
    assert fq.device_status() == 0
    yield
    assert fq.device_status() == 0


# ------------------------------------------------------------------ append

def nan_in_shared_memory():
    """A call that leaves the NaN word 0xFFFFFFFF in some 200 KB of every SM's shared memory: attention
    copies codes of 0xFF and scales of NaN through it, one block to an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    codes = torch.full((1, 16, 8, 128), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((8, 16), -1, dtype=torch.int32, device="cuda").view(torch.float32)
    table = torch.zeros((sms, 8), dtype=torch.int32, device="cuda")
    lens = torch.full((sms,), 128, dtype=torch.int32, device="cuda")
    q = dev_bf16(bf16(np.random.default_rng(0), sms, 8, 128))
    return lambda: fq.fp8_attention_paged(q, codes, codes, scales, scales, table, lens, 0, 3)


@pytest.mark.parametrize("d", [16, 32, 48, 80, 96, 112, 160, 192, 240])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_after_nan_in_shared_memory(d, interleaved, monkeypatch):
    """Norm and a scale per token, heads that do not fill a power of two: the places past head_dim count as zeros
    whatever an earlier kernel left behind."""
    before, append = nan_in_shared_memory(), fq.fp8_kv_append

    def after_nan(*a, **kw):
        before()
        return append(*a, **kw)
    monkeypatch.setattr(fq, "fp8_kv_append", after_nan)
    for rot in (0, d // 2 // 8 * 8, d):
        append_case(d + rot, 700, 3, 3, d, 24, 0, 3, rot, interleaved, True)
