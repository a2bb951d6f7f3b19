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


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kind,where,value", [
    ("bf16", 0, INF), ("bf16", 575, NAN), ("bf16", 300, -INF), ("fp8", "code", 0x7F), ("fp8", "code", 0xFF),
    ("fp8", "scale", NAN), ("fp8", "scale", -INF), ("fp8", "rope", INF), ("fp4", "scale", INF), ("fp4", "scale", NAN),
    ("fp4", "rope", NAN)])
@pytest.mark.parametrize("row", [0, 17, 63])
def test_pages_that_are_not_finite_are_reported(mla, kind, where, value, row):
    """One Inf or NaN among the page's values: CACHE_RANGE, codes 0 and a scale of NaN; other pages are as ever."""
    g = torch.Generator().manual_seed(row)
    kv = torch.randn((3, 64, 576), generator=g).to(torch.bfloat16).to(DEV)
    pool = kv if kind == "bf16" else (mla.fp8_pool_from if kind == "fp8" else mla.fp4_pool_from)(kv)
    good_codes, good_scales, status = summarize(mla, pool, kind)
    assert status == 0
    if kind == "bf16":
        pool[1, row, where] = value
    elif where == "code":
        pool[1, row, 77] = value
    else:
        raw = pool[1, row].cpu().numpy()
        at, dtype = {("fp8", "scale"): (520, np.float32), ("fp4", "scale"): (270, np.float16)}.get((kind, where), (0, None))
        if where == "rope":
            raw[-2:] = torch.tensor([value]).to(torch.bfloat16).view(torch.uint8).numpy()
        else:
            raw[at:at + np.dtype(dtype).itemsize] = np.frombuffer(dtype(value).tobytes(), np.uint8)
        pool[1, row] = torch.from_numpy(raw).to(DEV)
    codes, scales, status = summarize(mla, pool, kind)
    assert status == mla.STATUS_CACHE_RANGE
    assert np.all(codes[1] == 0) and np.isnan(scales[1])
    np.testing.assert_array_equal(codes[[0, 2]], good_codes[[0, 2]])
    np.testing.assert_array_equal(scales[[0, 2]], good_scales[[0, 2]])


def test_a_page_without_a_summary_is_chosen_last(mla):
    """A scale of NaN: the page loses against every scored one, and is reported by nobody (its writer was)."""
    T, H, k, nb = 64 * 40, 8, 12, 40
    g = torch.Generator().manual_seed(2)
    pool = (torch.randn((nb, 64, 576), generator=g) + torch.randn((nb, 1, 576), generator=g)).to(torch.bfloat16)
    att = mla.SparseAttention(1, 1, H, nb, nb, k)
    codes, scales = torch.zeros((nb, 576), dtype=torch.int8, device=DEV), torch.zeros(nb, device=DEV)
    dev = pool.to(DEV)
    mla.summarize_pages(dev, torch.arange(nb, dtype=torch.int32, device=DEV), codes, scales)
    q = torch.randn((1, H, 576), generator=g).to(torch.bfloat16).to(DEV)
    args = (q[..., :512].contiguous(), q[..., 512:].contiguous(), dev, codes, scales,
            torch.arange(nb, dtype=torch.int32, device=DEV)[None].contiguous(), torch.tensor([T], dtype=torch.int32, device=DEV))
    before = att.run(*args).pages[0].tolist()
    lost = before[4]
    scales[lost] = float("nan")
    res = att.run(*args)
    after = res.pages[0].tolist()
    assert res.status.item() == 0 and lost not in after and len(set(after)) == k
    assert set(before) - {lost} <= set(after)
    scales[:] = float("nan")
    assert att.run(*args).pages[0].tolist() == list(range(k - 1)) + [nb - 1]
