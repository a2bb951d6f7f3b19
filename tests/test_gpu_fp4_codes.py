"""The 4-bit writer's rows are the definition's, byte by byte: codes (with the sign of a value that becomes 0),
scales and k_rope."""
import numpy as np
import pytest
import torch

from tests.test_gpu_fp4cache import pack_rows, rows_of_many_ranges

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_04_b200 import mla as m
    return m


def written(mla, kv):
    n = len(kv)
    pool = torch.full((-(-n // 64), 64, 416), 0xAB, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.kv_quantize_fp4(kv.to(DEV), torch.arange(n, dtype=torch.int32, device=DEV), pool, status)
    assert status.item() == 0
    return pool.reshape(-1, 416)[:n].cpu().numpy()


@pytest.mark.parametrize("n", [1, 64, 1001, 9001])
def test_rows_of_many_ranges(mla, n):
    kv = rows_of_many_ranges(n, 3 * n)
    kv[n // 4, 64:96] = -kv[n // 4, 64:96].abs()
    kv[n // 4, 96:128] = torch.tensor([0.0, -0.0]).repeat(16).to(torch.bfloat16)          # a scale of 0
    np.testing.assert_array_equal(written(mla, kv), pack_rows(kv))


def test_signs_of_zeros_and_small_values(mla):
    """Values that round to 0, the ties between 0 and 0.5 among them, under one scale."""
    kv = torch.zeros((4, 576))
    kv[:, 0:512:32] = 6.0                                                                  # scale 1
    kv[0, 1:32] = torch.linspace(-0.3, 0.3, 31)
    kv[1, 1:5] = torch.tensor([0.25, -0.25, 0.2490234375, -0.2490234375])
    kv[2, 1:512:32], kv[2, 2:512:32] = -0.0, -1e-30
    kv[3, :512] = -1e-38                                                                   # a scale of 0
    kv = kv.to(torch.bfloat16)
    got = written(mla, kv)
    np.testing.assert_array_equal(got, pack_rows(kv))
    assert got[2, 0] >> 4 == 8 and got[2, 1] & 15 == 8


@pytest.mark.parametrize("exponent", [-24, -23, -20, -14])
def test_subnormal_scales(mla, exponent):
    """Scales with few bits left: quotients up to 9 before they are cut at 6."""
    g = torch.Generator().manual_seed(-exponent)
    kv = (torch.randn((200, 576), generator=g) * 2.0 ** exponent * 8).to(torch.bfloat16)
    np.testing.assert_array_equal(written(mla, kv), pack_rows(kv))


def test_raw_stream_handles(mla):
    """A call given a stream as a number makes its own tensors on that stream too."""
    kv = rows_of_many_ranges(500, 5).to(DEV)
    pool = torch.zeros((8, 64, 416), dtype=torch.uint8, device=DEV)
    slots = torch.arange(500, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mla.kv_quantize_fp4(kv, slots, pool, stream=side.cuda_stream)
    back = mla.kv_dequantize_fp4(pool, slots, stream=side.cuda_stream)
    side.synchronize()
    want = mla.kv_dequantize_fp4(pool, slots)
    torch.cuda.synchronize()
    assert torch.equal(back, want)
