"""Accuracy of the 4-bit attention where scores are large: the two halves of a row's 576 columns are
scored apart and exchanged in fp16, and added in fp32.

The bound of a test is that of its inputs.  The cached values are exact here (scales are powers of
two), and so are the queries in fp16.  With partial scores p0, p1 of a key in log2 units, each
rounded to fp16 (2^-11 at worst), a weight's logarithm is off by at most
    eps = ln 2 * 2^-11 * max_t (|p0| + |p1|)          (+ 2^-20 |s|: fp32 sums and the exponential)
so that a column of the output moves by at most (exp(2 eps) - 1) * sum_t w_t |c_t - o|.  P in fp16
adds 2^-11 sum_t w_t |c_t| and, for weights below its smallest normal number, 2^-25 max |c| a key;
the output's rounding to bf16 2^-8 |o|.  The LSE moves by at most eps (and its own fp32 arithmetic)."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4 as F

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
LN2 = math.log(2.0)


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_04_b200 import mla as m
    return m


def exact_rows(T, seed):
    """Rows whose 4-bit form is themselves: values of the E2M1 grid, every group reaching 6."""
    g = np.random.default_rng(seed)
    rows = np.zeros((T, 576))
    rows[:, :512] = F.e2m1_values(g.integers(0, 16, (T, 512)).astype(np.uint8)) / 4
    rows[:, 0:512:32] = np.where(g.integers(0, 2, (T, 16)) > 0, 1.5, -1.5)
    rows[:, 512:] = torch.from_numpy(g.standard_normal((T, 64))).to(torch.bfloat16).double().numpy()
    return rows


def attend(mla, q, rows, scale, clusters=7):
    T, H = len(rows), q.shape[0]
    nb = -(-T // 64)
    padded = torch.zeros((nb * 64, 576), dtype=torch.bfloat16)
    padded[:T] = torch.from_numpy(rows).to(torch.bfloat16)
    codes, scales = F.quantize(padded[:, :512].double().numpy())
    packed = F.pack(codes, scales, padded[:, 512:].contiguous().view(torch.uint8).numpy())
    assert np.array_equal(F.dequantize_rows(packed)[:T], rows)
    pool = torch.from_numpy(packed.reshape(nb, 64, 416)).to(DEV)
    dims = mla.make_dims(1, 1, H, nb, nb, scale)
    plan, slots = mla.plan(dims, [T], clusters)
    plan = torch.from_numpy(plan).to(DEV)
    o_part, lse_part = torch.empty(max(slots, 1) * H * 512, device=DEV), torch.empty(max(slots, 1) * H, device=DEV)
    out, lse = torch.empty((1, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((1, H), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    qb = torch.from_numpy(q).to(torch.bfloat16)
    assert np.array_equal(qb.double().numpy(), q)
    mla.decode_attn_fp4cache(dims, qb[None, :, :512].contiguous().to(DEV), qb[None, :, 512:].contiguous().to(DEV), pool,
                             torch.arange(nb, dtype=torch.int32, device=DEV)[None].contiguous(),
                             torch.tensor([T], dtype=torch.int32, device=DEV), plan, clusters, o_part, lse_part, out,
                             lse, status)
    if slots:
        mla.combine(dims, plan, o_part, lse_part, out, lse)
    return out[0].double().cpu().numpy(), lse[0].double().cpu().numpy(), status.item()


def halves(q, rows):
    """Column sets of the two CTAs: 256 latent and 32 RoPE columns each."""
    own = [np.r_[256 * r:256 * r + 256, 512 + 32 * r:512 + 32 * r + 32] for r in range(2)]
    return [q[:, c] @ rows[:, c].T for c in own]


def check(got, lse, q, rows, scale, exact_partials=False):
    """Largest error of the output as a share of its bound."""
    p = [h * scale / LN2 for h in halves(q, rows)]
    s = (p[0] + p[1]) * LN2
    w = np.exp(s - s.max(1, keepdims=True))
    l = w.sum(1, keepdims=True)
    w /= l
    c = rows[:, :512]
    o = w @ c
    rounded = 0.0 if exact_partials else 2.0 ** -11
    eps = LN2 * (rounded * (np.abs(p[0]) + np.abs(p[1])) + 2.0 ** -20 * (1 + np.abs(p[0] + p[1]))).max(1)
    spread = np.stack([(w[h][:, None] * np.abs(c - o[h])).sum(0) for h in range(len(q))])
    bound = np.expm1(2 * eps)[:, None] * spread + 2.0 ** -11 * (w @ np.abs(c)) + len(rows) * 2.0 ** -25 * np.abs(c).max()
    bound = bound + 2.0 ** -8 * (np.abs(o) + bound)
    share = np.abs(got - o) / bound
    assert share.max() <= 1, (share.max(), np.abs(got - o).max())
    want_lse = s.max(1) + np.log(l[:, 0])
    assert np.all(np.abs(lse - want_lse) <= eps + 2.0 ** -18 * (1 + np.abs(want_lse)))
    return share.max()


@pytest.mark.parametrize("factor", [1, 3, 10, 30, 200])
@pytest.mark.parametrize("T", [130, 1000])
def test_peaked_softmax_stays_within_its_bound(mla, factor, T):
    rows = exact_rows(T, T)
    g = torch.Generator().manual_seed(factor)
    q = (torch.randn((16, 576), generator=g) * factor).to(torch.bfloat16).double().numpy()
    scale = 1 / math.sqrt(192)
    got, lse, status = attend(mla, q, rows, scale)
    assert status == 0
    check(got, lse, q, rows, scale)


@pytest.mark.parametrize("size", [1.0, 8.0, 64.0])
def test_halves_that_cancel(mla, size):
    """Partials of opposite sign and up to hundreds in size, whose sum is small."""
    rows = exact_rows(700, 3)
    rows[:, 256:512] = rows[:, :256]
    g = torch.Generator().manual_seed(5)
    a = (torch.randn((16, 256), generator=g) * size).to(torch.bfloat16).double().numpy()
    q = np.zeros((16, 576))
    q[:, :256], q[:, 256:512] = a, -a
    q[:, 0::64] += np.sign(a[:, :1]) * 0.5
    q = torch.from_numpy(q).to(torch.bfloat16).double().numpy()
    scale = 1 / math.sqrt(192)
    got, lse, status = attend(mla, q, rows, scale)
    assert status == 0
    check(got, lse, q, rows, scale)


@pytest.mark.parametrize("big", [16.0, 64.0, 512.0, 4096.0])
def test_the_sum_of_the_halves_is_not_rounded(mla, big):
    """One half the same large number for every key, the other small: both exact in fp16, their sum is not."""
    T, scale = 600, LN2
    rows = np.zeros((T, 576))
    rows[:, 0:512:32] = 6.0                                   # the scale of every group is 1
    rows[:, 257:272] = F.e2m1_values(np.random.default_rng(1).integers(0, 16, (T, 15)).astype(np.uint8))
    q = np.zeros((4, 576))
    q[:, 0] = big / 8                                          # p0 = 0.75 big
    for h in range(4):
        q[h, 257 + h] = 2.0 ** -(4 + h)                        # |p1| <= 6 / 16
    got, lse, status = attend(mla, q, rows, scale)
    assert status == 0
    check(got, lse, q, rows, scale, exact_partials=True)


@pytest.mark.parametrize("case", ["queries", "all keys", "one key", "up"])
def test_partials_that_leave_fp16(mla, case):
    """Above the range, or below it for every key: reported.  One key below it has no weight, as it should."""
    T = 300
    rows = np.zeros((T, 576))
    rows[:, 0:512:32] = 6.0
    q = np.zeros((4, 576))
    q[:, 40] = 1.0
    if case == "queries":
        q[2, 0] = -2.0 ** 20                     # beyond fp16: -inf times 6 for every key
    elif case == "all keys":
        q[2, 0] = -2.0 ** 15                     # -196608 in log2 units
    elif case == "one key":
        rows[77, 33] = 6.0
        q[2, 33] = -2.0 ** 15
    else:
        q[2, 0] = 2.0 ** 15
    got, lse, status = attend(mla, q, rows, LN2)
    assert status == (0 if case == "one key" else mla.STATUS_SCORE_RANGE)
    if case == "one key":
        check(got, lse, q, rows, LN2, exact_partials=True)
    q[2, [0, 33]] = -2.0 ** 13                   # -49152: in range
    got, lse, status = attend(mla, q, rows, LN2)
    assert status == 0
    check(got, lse, q, rows, LN2, exact_partials=True)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_other_caches_report_rows_below_fp16(mla, kind):
    T, H = 200, 4
    kv = torch.zeros((4, 64, 576), dtype=torch.bfloat16)
    kv[..., 0] = 4.0
    pool = kv.to(DEV) if kind == "bf16" else mla.fp8_pool_from(kv.to(DEV))
    dims = mla.make_dims(1, 1, H, 4, 4, LN2)
    plan, slots = mla.plan(dims, [T], 3)
    plan = torch.from_numpy(plan).to(DEV)
    o_part, lse_part = torch.empty(max(slots, 1) * H * 512, device=DEV), torch.empty(max(slots, 1) * H, device=DEV)
    out, status = torch.empty((1, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    fn = mla.decode_attn if kind == "bf16" else mla.decode_attn_fp8cache
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None].contiguous()
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    for size, want in ((-2.0 ** 12, 0), (-2.0 ** 15, mla.STATUS_SCORE_RANGE), (2.0 ** 15, mla.STATUS_SCORE_RANGE)):
        q = torch.zeros((1, H, 512), dtype=torch.bfloat16, device=DEV)
        q[0, 1, 0] = size
        status.zero_()
        fn(dims, q, q[..., 64:128].contiguous(), pool, table, lens, plan, 3, o_part, lse_part, out, status=status)
        assert status.item() == want
