"""The 4-bit latent cache on the GPU against the float64 oracle (oracle/fp4.py).

The writer is compared code by code and scale by scale; the reader's bf16 rows bit by bit (code x
scale is exact in fp32, so the one rounding to bf16 is that of the float64 value).  The
attention reads pools that the oracle packed, never the CUDA writer.  Its operands: rows
widened to fp16 (relative error 2^-11), q_lat in fp16 (2^-11), P in fp16 (2^-11), partial
scores in fp16 in log2 units (|x| below 32 in these unit-variance workloads: 2^-7 x ln 2 at
worst on a logit, typically a tenth of it, and averaging over keys); o_lat is rounded to bf16 (2^-8 at worst, 1.7e-3 in
relative Frobenius).  The sum in quadrature stays below the bounds of the other caches' tests,
5e-3 relative Frobenius and 2e-2 absolute, and 2e-2 on the LSE."""
import numpy as np
import pytest
import torch

from head_latent_attention_04_b200 import workloads as W
from oracle import fp4 as F
from oracle import mla_oracle as O
from tests.gpu_helpers import check_out

pytestmark = pytest.mark.gpu

ROW4 = 416
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_04_b200 import mla as m
    return m


def pack_rows(rows: torch.Tensor) -> np.ndarray:
    """bf16 [n][576] -> uint8 [n][416] by the oracle."""
    codes, scales = F.quantize(rows[:, :512].double().numpy())
    return F.pack(codes, scales, rows[:, 512:].contiguous().view(torch.uint8).numpy().reshape(len(rows), 128))


def oracle_pool(w, poison_rows=None):
    rows = w.kv_pool.reshape(-1, 576)
    pool = np.concatenate([pack_rows(rows[r:r + 16384]) for r in range(0, len(rows), 16384)])
    if poison_rows is not None:
        pool[poison_rows, :256] = 0x77
        pool[poison_rows, 256:288] = np.frombuffer(np.full(16, np.nan, np.float16).tobytes(), np.uint8)
        nan = torch.full((64,), float("nan"), dtype=torch.bfloat16).view(torch.uint8).numpy()
        pool[poison_rows, 288:] = nan
    return torch.from_numpy(pool.reshape(w.num_blocks, 64, ROW4))


def oracle_rows4(w, pool4, b, heads=None):
    T = int(w.seq_lens[b])
    ids = np.asarray(w.block_table[b, :-(-T // 64)], dtype=np.int64)
    cache = F.dequantize_rows(pool4.numpy()[ids].reshape(-1, ROW4)[:T])
    rows = slice(b * w.s_q, (b + 1) * w.s_q)
    return O.mla_decode(w.q_nope[rows].double().numpy(), w.q_rope[rows].double().numpy(), [cache],
                        w.w_uk.double().numpy(), w.w_uv.double().numpy(), w.s_q, heads=heads)


def run_fp4(mla, w, pool4, num_clusters=None):
    wd = w.to(DEV)
    bt = torch.as_tensor(w.block_table, dtype=torch.int32, device=DEV)
    dec = mla.Decoder(w.seq_lens, w.s_q, w.n_heads, w.max_blocks, w.num_blocks, DEV, num_clusters=num_clusters,
                      kv_cache="fp4")
    res = dec.run(wd.q_nope, wd.q_rope, pool4.to(DEV), bt, wd.w_uk, wd.w_uv)
    torch.cuda.synchronize()
    return dec, res


def full_check(mla, w, num_clusters=None, poison_rows=None):
    pool4 = oracle_pool(w, poison_rows)
    dec, res = run_fp4(mla, w, pool4, num_clusters)
    assert res.status.item() == 0
    for b in range(w.B):
        ref = oracle_rows4(w, pool4, b)
        rows = slice(b * w.s_q, (b + 1) * w.s_q)
        check_out(res.o_lat[rows], ref["o_lat"])
        check_out(res.out[rows], ref["out"])
        np.testing.assert_allclose(res.lse[rows].cpu().numpy(), ref["lse"], rtol=0, atol=2e-2)
    return dec, res


# ------------------------------------------------------------------ rows in and out
def rows_of_many_ranges(n, seed):
    kv = torch.randn((n, 576), generator=torch.Generator().manual_seed(seed))
    kv[:, :512] *= 10.0 ** torch.linspace(-6, 4, n)[:, None]          # subnormal scales to large ones
    kv[n // 2, 32:64] = 0                                             # an all-zero group
    kv[n // 3, :512] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]).repeat(64)   # every tie
    kv[n // 3, 64:512] *= -1
    return kv.to(torch.bfloat16)


@pytest.mark.parametrize("n", [1, 3, 333])
def test_quantize_and_dequantize_are_exact(mla, n):
    nb = 8
    kv = rows_of_many_ranges(n, 7 + n)
    slots = torch.from_numpy(np.random.default_rng(3).permutation(nb * 64)[:n].astype(np.int32))
    pool = torch.full((nb, 64, ROW4), 0xAB, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.kv_quantize_fp4(kv.to(DEV), slots.to(DEV), pool, status)
    back = mla.kv_dequantize_fp4(pool, slots.to(DEV), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    got = pool.reshape(-1, ROW4).cpu().numpy()
    s = slots.numpy()
    want = pack_rows(kv)
    assert np.array_equal(got[s, 256:], want[:, 256:])                # scales and k_rope, bit by bit
    assert np.array_equal(F.e2m1_values(F.unpack(got[s])[0]), F.e2m1_values(F.unpack(want)[0]))
    assert np.all(np.delete(got, s, axis=0) == 0xAB)
    exact = torch.from_numpy(F.dequantize_rows(want)).to(torch.bfloat16)
    assert torch.equal(back.cpu(), exact)


def test_padding_is_skipped_and_bad_slots_are_reported(mla):
    kv = rows_of_many_ranges(6, 1).to(DEV)
    pool = torch.full((2, 64, ROW4), 0x11, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([-1, 5, -1, 127, -1, -1], dtype=torch.int32, device=DEV)
    mla.kv_quantize_fp4(kv, slots, pool, status)
    out = torch.full((6, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    mla.kv_dequantize_fp4(pool, slots, out, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    p = pool.reshape(-1, ROW4).cpu().numpy()
    assert np.all(np.delete(p, [5, 127], axis=0) == 0x11) and np.array_equal(p[[5, 127], 256:], pack_rows(kv.cpu())[[1, 3], 256:])
    assert torch.all(out[[0, 2, 4, 5]] == 3.0) and not torch.any(torch.all(out[[1, 3]] == 3.0, 1))
    before = pool.clone()
    bad = torch.tensor([-2, 128, 2 ** 31 - 1, -1, -1, -1], dtype=torch.int32, device=DEV)
    mla.kv_quantize_fp4(kv, bad, pool, status)
    assert status.item() == mla.STATUS_BAD_BLOCK and torch.equal(pool, before)
    status.zero_()
    out.fill_(3.0)
    mla.kv_dequantize_fp4(pool, bad, out, status)
    assert status.item() == mla.STATUS_BAD_BLOCK and torch.all(out == 3.0)


@pytest.mark.parametrize("n", [4097, 8288, 8289, 16301])
def test_long_calls_are_exact_too(mla, n):
    """Both forms of the row kernels, one and four rows a thread: padding, bad slots and a ragged end."""
    nb = 300
    kv = rows_of_many_ranges(n, n)
    rng = np.random.default_rng(n)
    s = rng.permutation(nb * 64)[:n].astype(np.int32)
    s[rng.permutation(n)[:97]] = -1
    s[[0, n - 1]] = -1
    live = s >= 0
    pool = torch.full((nb, 64, ROW4), 0xAB, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.from_numpy(s).to(DEV)
    mla.kv_quantize_fp4(kv.to(DEV), slots, pool, status)
    back = torch.full((n, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    mla.kv_dequantize_fp4(pool, slots, back, status)
    assert status.item() == 0
    got, want = pool.reshape(-1, ROW4).cpu().numpy(), pack_rows(kv)
    assert np.array_equal(got[s[live], 256:], want[live, 256:])
    assert np.array_equal(F.e2m1_values(F.unpack(got[s[live]])[0]), F.e2m1_values(F.unpack(want[live])[0]))
    assert np.all(np.delete(got, s[live], axis=0) == 0xAB)
    exact = torch.from_numpy(F.dequantize_rows(want)).to(torch.bfloat16)
    exact[~torch.from_numpy(live)] = 3.0
    assert torch.equal(back.cpu(), exact)
    slots[n // 2] = nb * 64
    mla.kv_quantize_fp4(kv.to(DEV), slots, pool, status)
    assert status.item() == mla.STATUS_BAD_BLOCK


@pytest.mark.parametrize("value", [65536.0, 1e30, float("inf"), float("nan"), float("-inf")])
def test_values_beyond_fp16_are_flagged_and_stay_finite(mla, value):
    kv = rows_of_many_ranges(4, 2)
    kv[2, 130] = value
    pool = torch.zeros((1, 64, ROW4), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.kv_quantize_fp4(kv.to(DEV), torch.arange(4, dtype=torch.int32, device=DEV), pool, status)
    assert status.item() == mla.STATUS_CACHE_RANGE
    got = pool.reshape(-1, ROW4)[:4].cpu().numpy()
    assert np.array_equal(got[[0, 1, 3], 256:], pack_rows(kv[[0, 1, 3]])[:, 256:])
    assert np.all(np.isfinite(F.unpack(got)[1].astype(np.float64))) and F.unpack(got)[1].max() <= 10912
    kv[2, 130] = 65280.0                                               # the largest bf16 that is in range
    status.zero_()
    mla.kv_quantize_fp4(kv.to(DEV), torch.arange(4, dtype=torch.int32, device=DEV), pool, status)
    assert status.item() == 0 and np.array_equal(pool.reshape(-1, ROW4)[:4].cpu().numpy()[:, 256:], pack_rows(kv)[:, 256:])


def test_rows_written_and_read_back_at_once_many_times(mla):
    """Every pass writes other values to the same slots and reads them back, with nothing between
    the launches, on a stream of its own: the reader never sees the pass before."""
    pool = torch.zeros((64, 64, ROW4), dtype=torch.uint8, device=DEV)
    slots = torch.randperm(64 * 64, generator=torch.Generator().manual_seed(0))[:3000].to(torch.int32).to(DEV)
    base = torch.randint(1, 7, (3000, 576), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        with torch.cuda.stream(side):
            kv = torch.where(base > 3, float(6 << i % 8), 0.0).to(torch.bfloat16) * (1 if i % 2 else -1)
            kv[:, ::32] = float(6 << i % 8)                # every group reaches 6 x a power of two: exact
        mla.kv_quantize_fp4(kv, slots, pool, stream=side)
        got.append((kv, mla.kv_dequantize_fp4(pool, slots, stream=side)))
    torch.cuda.synchronize()
    for kv, back in got:
        assert torch.equal(back, kv)


def test_empty_calls(mla):
    pool = torch.zeros((1, 64, ROW4), dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    mla.kv_quantize_fp4(torch.zeros((0, 576), dtype=torch.bfloat16, device=DEV), none, pool)
    assert mla.kv_dequantize_fp4(pool, none).shape == (0, 576)


# ------------------------------------------------------------------ attention
def test_tiny(mla):
    full_check(mla, W.preset_workload("tiny"))


@pytest.mark.parametrize("clusters", [1, 3, 74, 148])
def test_split_counts(mla, clusters):
    full_check(mla, W.make_workload(3, 1, 32, [700, 64, 1000], seed=11, pool="permuted"), num_clusters=clusters)


@pytest.mark.parametrize("lens", [[1], [64], [65], [1, 2, 3, 127, 128, 129, 191], [5000]])
def test_ragged_lengths(mla, lens):
    full_check(mla, W.make_workload(len(lens), 1, 128, lens, seed=sum(lens) + 1, pool="scattered:1.5"), num_clusters=4)


@pytest.mark.parametrize("H", [1, 33, 100])
def test_head_counts(mla, H):
    full_check(mla, W.make_workload(2, 1, H, [300, 90], seed=H + 2, pool="permuted"))


@pytest.mark.parametrize("s_q,lens,clusters", [(2, [2, 3, 65, 66, 200], 74), (4, [4, 200, 4100], 7), (8, [8, 71, 900], 5)])
def test_drafts(mla, s_q, lens, clusters):
    full_check(mla, W.make_workload(len(lens), s_q, 128, lens, seed=s_q * 5 + clusters, pool="permuted"),
               num_clusters=clusters)


@pytest.mark.parametrize("s_q,lens,clusters", [(1, [65, 130, 1, 200, 64], 5), (2, [66, 129, 2], 74)])
def test_non_finite_rows_never_leak(mla, s_q, lens, clusters):
    """Page tails and unused blocks hold NaN scales and NaN k_rope."""
    w = W.make_workload(len(lens), s_q, 128, lens, seed=91 + s_q, pool="scattered:3")
    used = np.zeros((w.num_blocks, 64), dtype=bool)
    for b in range(w.B):
        T = int(w.seq_lens[b])
        for p in range(-(-T // 64)):
            used[int(w.block_table[b, p]), :min(64, T - 64 * p)] = True
    full_check(mla, w, num_clusters=clusters, poison_rows=~used.reshape(-1))


def test_unevenly_scaled_groups(mla):
    """Groups of very different ranges, as outlier channels make them."""
    w = W.make_workload(2, 1, 128, [400, 77], seed=5, pool="permuted")
    w.kv_pool[..., :512] *= 2.0 ** (torch.arange(512) // 32 % 5 - 3).float()
    full_check(mla, w.__class__(**{**w.__dict__, "kv_pool": w.kv_pool.to(torch.bfloat16)}))


@pytest.mark.parametrize("name,heads", [("v2_4k", list(range(3, 128, 8))), ("long128k", list(range(5, 128, 16)))])
def test_full_size(mla, name, heads):
    w = W.preset_workload(name)
    pool4 = mla.fp4_pool_from(w.kv_pool.to(DEV)).cpu()
    dec, res = run_fp4(mla, w, pool4)
    again = res.o_lat.clone()
    assert res.status.item() == 0 and dec.num_slots > 0
    ref = oracle_rows4(w, pool4, 1, heads=heads)
    check_out(res.o_lat[1:2][:, heads], ref["o_lat"])
    _, res2 = run_fp4(mla, w, pool4)
    assert torch.equal(res2.o_lat, again)                              # the same bits every run


def test_bad_block_stale_length_and_wrong_plan_are_reported(mla):
    w = W.make_workload(3, 1, 16, [100, 200, 300], seed=3, pool="permuted")
    pool4 = oracle_pool(w).to(DEV)
    wd = w.to(DEV)
    bt = torch.as_tensor(w.block_table, dtype=torch.int32, device=DEV)
    dec = mla.Decoder(w.seq_lens, 1, 16, w.max_blocks, w.num_blocks, DEV, kv_cache="fp4")
    good = dec.run(wd.q_nope, wd.q_rope, pool4, bt, wd.w_uk, wd.w_uv).o_lat.clone()
    bad = bt.clone()
    bad[1, 1] = w.num_blocks
    dec.run(wd.q_nope, wd.q_rope, pool4, bad, wd.w_uk, wd.w_uv)
    assert dec.status.item() == mla.STATUS_BAD_BLOCK
    dec.status.zero_()
    dec.seq_lens_dev[1] = 201
    r = dec.run(wd.q_nope, wd.q_rope, pool4, bt, wd.w_uk, wd.w_uv)
    assert dec.status.item() == mla.STATUS_BAD_SEQLEN
    assert torch.all(r.o_lat[1] == 0) and torch.all(r.lse[1] == float("-inf"))
    assert torch.equal(r.o_lat[[0, 2]], good[[0, 2]])
    dec.status.zero_()
    dec.plan_dev[0] = 0
    dec.run(wd.q_nope, wd.q_rope, pool4, bt, wd.w_uk, wd.w_uv)
    assert dec.status.item() & mla.STATUS_BAD_PLAN
    with pytest.raises(ValueError, match="bf16 cache"):
        dec.run(wd.q_nope, wd.q_rope, pool4, bt, wd.w_uk, wd.w_uv, draft_masks=bt)


def test_a_plan_that_splits_rows_needs_the_workspaces(mla):
    w = W.make_workload(1, 1, 16, [3000], seed=3, pool="permuted")
    pool4 = oracle_pool(w).to(DEV)
    dec = mla.Decoder(w.seq_lens, 1, 16, w.max_blocks, w.num_blocks, DEV, kv_cache="fp4")
    assert dec.num_slots > 0
    bt = torch.as_tensor(w.block_table, dtype=torch.int32, device=DEV)
    q = torch.zeros((1, 16, 512), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 7.0)
    for o_part, lse_part in ((None, None), (dec.o_part, None), (None, dec.lse_part)):
        dec.status.zero_()
        mla.decode_attn_fp4cache(dec.dims, q, q[..., :64].contiguous(), pool4, bt, dec.seq_lens_dev, dec.plan_dev,
                                 dec.num_clusters, o_part, lse_part, out, status=dec.status)
        assert dec.status.item() == mla.STATUS_BAD_PLAN and torch.all(out == 7.0)


def test_graphed_and_streamed_steps_on_the_4_bit_cache(mla):
    w = W.make_workload(3, 2, 32, [700, 64, 1000], seed=17, pool="permuted")
    pool4 = oracle_pool(w)
    dec, res = run_fp4(mla, w, pool4)
    want = res.out.clone()
    wd, pool = w.to(DEV), pool4.to(DEV)
    for make in (mla.GraphedStep, mla.StreamedDecoder):
        step = make(dec, pool, wd.w_uk, wd.w_uv)
        if make is mla.GraphedStep:
            step.q_nope.copy_(w.q_nope), step.q_rope.copy_(w.q_rope)
            step.block_table.copy_(torch.as_tensor(w.block_table))
            assert torch.equal(step.run(), want.cpu())
        else:
            for qn, qr, bt in step.host_in:
                qn.copy_(w.q_nope), qr.copy_(w.q_rope), bt.copy_(torch.as_tensor(w.block_table))
            ids = [step.submit() for _ in range(2)]
            for i in ids:
                assert torch.equal(step.wait(i), want.cpu())
    assert dec.status.item() == 0


def test_queries_beyond_fp16_are_reported(mla):
    w = W.make_workload(1, 1, 16, [100], seed=3, pool="permuted")
    pool4 = oracle_pool(w).to(DEV)
    wd = w.to(DEV)
    bt = torch.as_tensor(w.block_table, dtype=torch.int32, device=DEV)
    dec = mla.Decoder(w.seq_lens, 1, 16, w.max_blocks, w.num_blocks, DEV, kv_cache="fp4")
    dec.run((wd.q_nope.float() * 1e6).to(torch.bfloat16), wd.q_rope, pool4, bt, wd.w_uk, wd.w_uv)
    assert dec.status.item() & mla.STATUS_SCORE_RANGE


def test_wait_time_out_returns_and_the_context_recovers(mla):
    w = W.make_workload(3, 1, 128, [3000, 1000, 77], seed=67, pool="permuted")
    pool4 = oracle_pool(w)
    try:
        mla.set_wait_limit_ns(1)
        for _ in range(2):
            _, res = run_fp4(mla, w, pool4, num_clusters=4)
            assert res.status.item() & mla.STATUS_TIMEOUT
    finally:
        mla.set_wait_limit_ns(0)
    full_check(mla, w, num_clusters=4)


def test_wrong_shapes_are_refused(mla):
    w = W.make_workload(1, 1, 16, [100], seed=3, pool="permuted")
    dec = mla.Decoder(w.seq_lens, 1, 16, w.max_blocks, w.num_blocks, DEV, kv_cache="fp4")
    wd = w.to(DEV)
    bt = torch.as_tensor(w.block_table, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="kv_pool_fp4"):
        dec.run(wd.q_nope, wd.q_rope, wd.kv_pool, bt, wd.w_uk, wd.w_uv)
    pool = torch.zeros((w.num_blocks, 64, ROW4), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="block_table"):
        dec.run(wd.q_nope, wd.q_rope, pool, bt.long(), wd.w_uk, wd.w_uv)
    with pytest.raises(ValueError, match="contiguous"):
        mla.kv_quantize_fp4(torch.zeros((4, 1152), dtype=torch.bfloat16, device=DEV)[:, ::2],
                            torch.zeros(4, dtype=torch.int32, device=DEV), pool)
    with pytest.raises(ValueError, match="tensors of one call"):
        mla.kv_quantize_fp4(torch.zeros((4, 576), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32, device=DEV), pool)
