"""Page summaries at the ends of what a page can hold, against the float64 definition, bit by bit."""
import numpy as np
import pytest
import torch

from oracle import fp4 as F

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_04_b200 import mla as m
    return m


def summarize(mla, pool, kind="bf16"):
    nb = pool.shape[0]
    codes = torch.full((nb, 576), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((nb,), -1.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.summarize_pages(pool, torch.arange(nb, dtype=torch.int32, device=DEV), codes, scales, kind, status)
    return codes.cpu().numpy(), scales.cpu().numpy(), status.item()


@pytest.mark.parametrize("low", [-133, -130, -127, -126, -124, -121, -100])
def test_tiny_pages(mla, low):
    """bf16 values down to the subnormals: 127 over the largest sum would leave the range of a double."""
    g = torch.Generator().manual_seed(-low)
    pool = torch.zeros((6, 64, 576))
    pool[1:3] = torch.randint(-3, 4, (2, 64, 576), generator=g).float() * 2.0 ** low
    pool[3, :, :40] = 2.0 ** low                      # every row the same, and zero columns
    pool[4, 7, 3] = -(2.0 ** low)                     # one value alone
    pool[5, :, 0], pool[5, :, 1], pool[5, :, 2] = 2.0 ** (low + 1), 2.0 ** low, -(2.0 ** low)   # 63.5 goes to 64
    pool = pool.to(torch.bfloat16)
    codes, scales, status = summarize(mla, pool.to(DEV))
    want, want_scales = F.code8(pool.double().numpy().sum(1) / 64)
    assert status == 0
    np.testing.assert_array_equal(codes, want.astype(np.int8))
    np.testing.assert_array_equal(scales, want_scales)


def test_pages_of_the_largest_values(mla):
    pool = torch.zeros((3, 64, 576), dtype=torch.bfloat16)
    top = torch.finfo(torch.bfloat16).max
    pool[0] = top
    pool[1, :, ::3], pool[1, :, 1::3] = -top, 2.0 ** 127
    pool[2, 5] = top
    codes, scales, status = summarize(mla, pool.to(DEV))
    want, want_scales = F.code8(pool.double().numpy().sum(1) / 64)
    assert status == 0
    np.testing.assert_array_equal(codes, want.astype(np.int8))
    np.testing.assert_array_equal(scales, want_scales)


@pytest.mark.parametrize("exponent", [-126, -140, -149])
def test_tiny_fp8_scales(mla, exponent):
    """FP8 rows with the smallest scales, beside k_rope of the same size."""
    from tests.test_gpu_fp8cache import dequant_rows
    g = np.random.default_rng(-exponent)
    rows = np.zeros((2 * 64, 656), dtype=np.uint8)
    rows[:, :512] = g.integers(0, 0x7E, (128, 512)) | (g.integers(0, 2, (128, 512)) << 7)
    rows[:, 512:528] = np.full((128, 4), 2.0 ** exponent, dtype=np.float32).view(np.uint8)
    rope = torch.full((128, 64), 2.0 ** max(exponent, -133)).to(torch.bfloat16)
    rows[:, 528:] = rope.view(torch.uint8).numpy().reshape(128, 128)
    values = dequant_rows(rows).reshape(2, 64, 576)
    codes, scales, status = summarize(mla, torch.from_numpy(rows.reshape(2, 64, 656)).to(DEV), "fp8")
    want, want_scales = F.code8(values.sum(1) / 64)
    assert status == 0
    np.testing.assert_array_equal(codes, want.astype(np.int8))
    np.testing.assert_array_equal(scales, want_scales)
