"""Block tables, slot maps and plans made on the GPU: whole numbers, compared bit by bit with the
oracle's request-by-request loop and with the host planner."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def check_tables(mla, cached, new, width, n_free, head=0, max_new=None, free=None, num_blocks=None, in_place=False):
    rng = np.random.default_rng(len(cached) + sum(new) % 1000)
    held = [-(-max(c, 0) // 64) if c <= width * 64 else 0 for c in cached]
    total = sum(held) + n_free
    num_blocks = num_blocks or max(total, 1)
    ids = rng.permutation(max(total, 1)).tolist()
    table = [[-7] * width for _ in cached]
    at = 0
    for b, h in enumerate(held):
        table[b][:h] = ids[at:at + h]
        at += h
    free = ids[at:at + n_free] if free is None else free
    max_new = sum(new) + 3 if max_new is None else max_new
    want = F.build_tables(cached, new, table, free, head, max_new)
    c, h, t = i32(cached), i32([head]), i32(table)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = mla.BatchTables.empty(len(cached), max_new)
    if in_place:
        out.seq_lens, out.free_head = c, h
    r = mla.build_tables(c, i32(new), t, i32(free), h, max_new, num_blocks, out, status)
    torch.cuda.synchronize()
    assert t.tolist() == want[0]
    assert (r.seq_lens.tolist(), r.cu_new.tolist()) == want[1:3]
    assert r.slots.tolist() == want[3] and r.positions.tolist() == want[4]
    assert r.free_head.item() == want[5]
    assert (status.item() == mla.STATUS_NO_SPACE) == want[6] and status.item() in (0, mla.STATUS_NO_SPACE)
    return r


@pytest.mark.parametrize("cached,new", [
    ([0], [0]), ([0], [1]), ([63], [1]), ([64], [1]), ([63], [2]), ([0], [200]),
    ([10, 0, 64, 127, 128, 5], [1, 1, 1, 1, 1, 1]),
    ([10, 0, 64, 127, 128, 5], [0, 300, 0, 65, 1, 0]),
    ([0] * 7, [0] * 7),
])
def test_small(mla, cached, new):
    check_tables(mla, cached, new, 9, 20, head=2)
    check_tables(mla, cached, new, 9, 20, in_place=True)


@pytest.mark.parametrize("B,hi", [(1023, 3), (1024, 3), (1025, 3), (5000, 2), (40, 3000), (3, 40000), (2100, 70)])
def test_many_requests_and_long_prompts(mla, B, hi):
    rng = np.random.default_rng(B)
    cached = rng.integers(0, 500, B).tolist()
    new = rng.integers(0, hi + 1, B).tolist()
    check_tables(mla, cached, new, 8 + hi // 64 + 2, 64 * B + sum(new) // 64)


@pytest.mark.parametrize("kw", [
    dict(n_free=3), dict(n_free=0), dict(n_free=40, max_new=700), dict(n_free=40, max_new=0),
    dict(n_free=40, head=38), dict(n_free=40, head=40), dict(n_free=40, head=41), dict(n_free=40, head=-1),
])
def test_requests_that_do_not_fit(mla, kw):
    cached = [10, 64, 0, 100, 500, 7, -5, 600, 3, 64]
    new = [1, 1, 130, 27, 100, 0, 2, 41, -3, 63]
    check_tables(mla, cached, new, 10, **{"max_new": 2000, **kw})


@pytest.mark.parametrize("max_new", [20000, 100000])
def test_wide_slot_maps_leave_the_same_answers(mla, max_new):
    """Long slot maps take a launch of their own; ends inside a tile, and a request too many."""
    check_tables(mla, [70] * 30, [333] * 30, 40, 400, max_new=max_new)
    check_tables(mla, [70] * 30 + [64 * 40 - 1], [333] * 30 + [5], 40, 400, max_new=max_new)
    check_tables(mla, [70] * 30, [1333] * 30, 40, 400, max_new=max_new)


@pytest.mark.parametrize("max_new", [7167, 7168, 7169, 8193])
def test_slot_maps_around_the_second_launch(mla, max_new):
    check_tables(mla, [70] * 30, [233] * 30, 40, 400, max_new=max_new)             # 6990 tokens
    check_tables(mla, [63, 0, 128], [max_new - 5, 0, 5], 140, 300, max_new=max_new)   # full to the last slot


def test_bad_blocks_are_reported(mla):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = i32([[3, 99, -1], [-4, -1, -1]])
    r = mla.build_tables(i32([100, 5]), i32([1, 1]), table, i32([7]), i32([0]), 4, 8, status=status)
    assert status.item() == mla.STATUS_BAD_BLOCK and r.slots.tolist() == [-1] * 4 and r.positions.tolist() == [100, 5, -1, -1]
    status.zero_()
    r = mla.build_tables(i32([64]), i32([2]), table[:1].contiguous(), i32([8]), i32([0]), 2, 8, status=status)
    assert status.item() == mla.STATUS_BAD_BLOCK and r.slots.tolist() == [-1, -1] and r.free_head.item() == 1


def test_refusals(mla):
    c = i32([1, 2])
    table = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="new_lens"):
        mla.build_tables(c, i32([1]), table, i32([1]), i32([0]), 4, 8)
    with pytest.raises(ValueError, match="block_table"):
        mla.build_tables(c, c, table[:1].contiguous(), i32([1]), i32([0]), 4, 8)
    with pytest.raises(ValueError, match="cached_lens"):
        mla.build_tables(c.long(), c, table, i32([1]), i32([0]), 4, 8)
    with pytest.raises(ValueError, match="contiguous"):
        mla.build_tables(c, c, torch.zeros((2, 6), dtype=torch.int32, device=DEV)[:, ::2], i32([1]), i32([0]), 4, 8)
    with pytest.raises(mla.MlaError):
        mla.build_tables(c, c, table, i32([1]), i32([0]), 4, 0)


# ------------------------------------------------------------------ plans
def same_plan(mla, lens, s_q, C, causal=True, H=128):
    dims = mla.make_dims(len(lens), s_q, H, max(1, max(-(-t // 64) for t in lens)), 10 ** 6, causal=causal)
    want, _ = mla.plan(dims, lens, C)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    buf = torch.full((len(want),), -9, dtype=torch.int32, device=DEV)
    got = mla.plan_device(dims, i32(lens), C, buf, status)
    assert status.item() == 0
    np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("lens,s_q,C", [
    ([4096] * 32, 1, 74), ([256, 256], 1, 74), ([131072] * 4, 1, 74), ([1], 1, 74), ([1], 1, 1), ([64, 65], 1, 4096),
    ([1, 64, 65, 127, 128, 129, 5000], 1, 5), ([2, 3, 64, 65, 66, 4097, 130], 2, 74), ([2, 3, 64, 65, 66, 4097, 130], 2, 1),
    ([3, 64, 65, 5000, 130], 3, 74), ([8, 9, 700, 64], 8, 5), ([4, 4100], 4, 3), ([8, 2 ** 21], 8, 148),
])
@pytest.mark.parametrize("causal", [True, False])
def test_plan_equals_the_host_planner(mla, lens, s_q, C, causal):
    same_plan(mla, lens, s_q, C, causal)


@pytest.mark.parametrize("seed", range(8))
def test_random_plans_equal_the_host_planner(mla, seed):
    rng = np.random.default_rng(seed)
    B = int(rng.choice([3, 50, 400, 1024, 1025, 3000]))
    s_q = int(rng.integers(1, 9))
    lens = rng.integers(s_q, int(rng.choice([80, 3000, 200000])), size=B).tolist()
    same_plan(mla, lens, s_q, int(rng.integers(1, 300)), bool(seed & 1), H=int(rng.integers(1, 129)))


def test_largest_batch(mla):
    same_plan(mla, (np.arange(65536) % 777 + 1).tolist(), 1, 148)
    same_plan(mla, (np.arange(8192) % 777 + 8).tolist(), 8, 148)


@pytest.mark.parametrize("s_q", [1, 3])
def test_padded_and_bad_rows_get_no_items(mla, s_q):
    lens = [500, 0, 70, 0, 4000, 0, 0]
    keep = [b for b, t in enumerate(lens) if t]
    dims = mla.make_dims(len(lens), s_q, 16, 80, 1000)
    C = 9
    plan = mla.plan_device(dims, i32(lens), C).cpu().numpy()
    dense, ns = mla.plan(mla.make_dims(len(keep), s_q, 16, 80, 1000), [lens[b] for b in keep], C)
    I = dense[2]
    assert plan[2] == I and plan[3] == ns and plan[4] == len(lens) * s_q and plan[7] == len(lens)
    off = 16 + C + 1
    assert np.array_equal(plan[16:off], dense[16:off])
    got, want = plan[off:off + 8 * I].reshape(-1, 8), dense[off:off + 8 * I].reshape(-1, 8).copy()
    want[:, 6] = [keep[b] * s_q + qi for b, qi in want[:, :2]]
    want[:, 0] = [keep[b] for b in want[:, 0]]
    assert np.array_equal(got, want)
    rows = plan[plan[10]:plan[10] + plan[4] + 1]
    assert np.all(np.diff(rows).reshape(-1, s_q)[[1, 3, 5, 6]] == 0) and rows[-1] == ns
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = list(lens)
    bad[1], bad[3], bad[5] = 80 * 64 + 1, -4, s_q - 1
    again = mla.plan_device(dims, i32(bad), C, status=status).cpu().numpy()
    assert status.item() == mla.STATUS_BAD_SEQLEN and np.array_equal(again, plan)


def test_no_rows_at_all(mla):
    dims = mla.make_dims(5, 2, 16, 80, 1000)
    plan = mla.plan_device(dims, i32([0] * 5), 9).cpu().numpy()
    assert plan[2] == 0 and plan[3] == 0 and np.all(plan[16:26] == 0) and np.all(plan[plan[10]:] == 0)


def test_small_plan_buffer_is_refused(mla):
    dims = mla.make_dims(2, 1, 16, 8, 100)
    with pytest.raises(mla.MlaError, match=f"status {mla.MLA_ERR_WORKSPACE_TOO_SMALL}"):
        mla.plan_device(dims, i32([5, 6]), 9, torch.zeros(20, dtype=torch.int32, device=DEV))
