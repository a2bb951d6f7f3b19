"""Page summaries, page selection and attention over the selection, against oracle/fp4.py and the
float64 attention oracle.  Summaries and selections are compared bit by bit: both sides work
from exact sums, exact quotients and whole-number dot products (only the one rounding to
fp32 that the definition names).  The attention's tolerances are those of the cache kinds' tests."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4 as F
from tests.gpu_helpers import check_out

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_04_b200 import mla as m
    return m


def drifting_pool(nb, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((nb, 64, 576), generator=g) + 0.5 * torch.randn((nb, 1, 576), generator=g)
    return x.to(torch.bfloat16)


def pool_of_kind(mla, pool, kind):
    """(device pool of that kind, its values float64 [nb][64][576])."""
    from tests.test_gpu_fp8cache import dequant_rows
    if kind == "bf16":
        return pool.to(DEV), pool.double().numpy()
    p = (mla.fp8_pool_from if kind == "fp8" else mla.fp4_pool_from)(pool.to(DEV))
    flat = p.cpu().numpy().reshape(-1, p.shape[-1])
    return p, (dequant_rows(flat) if kind == "fp8" else F.dequantize_rows(flat)).reshape(-1, 64, 576)


def summaries(values):
    codes, scales = F.code8(values.sum(1) / 64)
    return codes.astype(np.int8), scales


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("nb", [1, 37, 500])
def test_summaries_are_exact(mla, kind, nb):
    pool = drifting_pool(nb, nb)
    pool[nb // 2, :, 100:200] *= 1e-6
    if nb > 1:
        pool[1] = 0                                           # amax 0
        pool[nb - 1] *= 1e3
    p, values = pool_of_kind(mla, pool, kind)
    codes = torch.full((nb, 576), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((nb,), -1.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    order = torch.from_numpy(np.random.default_rng(nb).permutation(nb).astype(np.int32)).to(DEV)
    mla.summarize_pages(p, order, codes, scales, kind, status)
    assert status.item() == 0
    want_codes, want_scales = summaries(values)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_codes)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)


@pytest.mark.parametrize("spread", [4, 5, 6, 12, 24])
def test_fp4_summaries_of_scales_far_apart(mla, spread):
    """Rows whose scales differ by up to 2^spread: up to 2^5 within 16 rows the sums are kept in fp32,
    beyond in fp64; zero and subnormal scales among them."""
    nb = 40
    pool = drifting_pool(nb, spread).float()
    g = torch.Generator().manual_seed(spread)
    pool[..., :512] *= 2.0 ** (-torch.randint(0, spread + 1, (nb, 64, 1), generator=g).float())
    pool[3, 5:9] = 0
    pool[4, 17, :64] *= 2.0 ** -20
    p, values = pool_of_kind(mla, pool.to(torch.bfloat16), "fp4")
    codes = torch.zeros((nb, 576), dtype=torch.int8, device=DEV)
    scales = torch.zeros((nb,), device=DEV)
    mla.summarize_pages(p, torch.arange(nb, dtype=torch.int32, device=DEV), codes, scales, "fp4")
    want_codes, want_scales = summaries(values)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_codes)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)


def test_summary_ties_skips_and_bad_blocks(mla):
    pool = torch.zeros((4, 64, 576))
    pool[2, :, 0], pool[2, :, 1], pool[2, :, 2] = 2.0, 1.0, -1.0      # 63.5 goes to 64
    p = pool.to(torch.bfloat16).to(DEV)
    codes = torch.full((4, 576), 5, dtype=torch.int8, device=DEV)
    scales = torch.full((4,), 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.summarize_pages(p, torch.tensor([-1, 2, 2], dtype=torch.int32, device=DEV), codes, scales, status=status)
    assert status.item() == 0 and codes[2, :4].tolist() == [127, 64, -64, 0]
    assert torch.all(codes[[0, 1, 3]] == 5) and scales.tolist() == [5, 5, np.float32(2 / 127), 5]
    mla.summarize_pages(p, torch.tensor([4, -2], dtype=torch.int32, device=DEV), codes, scales, status=status)
    assert status.item() == mla.STATUS_BAD_BLOCK and torch.all(codes[[0, 1, 3]] == 5)
    mla.summarize_pages(p, torch.zeros(0, dtype=torch.int32, device=DEV), codes, scales)


class Batch:
    """A batch with random tables over a drifting pool, its summaries and queries."""

    def __init__(self, mla, lens, s_q, H, k, kind="bf16", n_first=1, n_recent=1, causal=True, seed=0, width=None):
        rng = np.random.default_rng(seed)
        pages = [-(-t // 64) for t in lens]
        self.width = width or max(max(pages), 1)
        self.nb = sum(pages) + 3
        perm = rng.permutation(self.nb)
        self.table = np.full((len(lens), self.width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.lens, self.s_q, self.H, self.k, self.causal = lens, s_q, H, k, causal
        self.n_first, self.n_recent = n_first, n_recent
        self.pool, self.values = pool_of_kind(mla, drifting_pool(self.nb, seed + 1), kind)
        self.codes, self.scales = summaries(self.values)
        g = torch.Generator().manual_seed(seed + 2)
        N = len(lens) * s_q
        self.q_lat = torch.randn((N, H, 512), generator=g).to(torch.bfloat16)
        self.q_rope = torch.randn((N, H, 64), generator=g).to(torch.bfloat16)
        self.att = mla.SparseAttention(len(lens), s_q, H, self.width, self.nb, k, n_first, n_recent, kv_cache=kind,
                                       causal=causal)

    def device_args(self):
        return (self.q_lat.to(DEV), self.q_rope.to(DEV), self.pool, torch.from_numpy(self.codes).to(DEV),
                torch.from_numpy(self.scales).to(DEV), torch.from_numpy(self.table).to(DEV),
                torch.tensor(self.lens, dtype=torch.int32, device=DEV))

    def kv_len(self, n):
        b, i = divmod(n, self.s_q)
        T = self.lens[b]
        return 0 if T == 0 else (T - self.s_q + 1 + i if self.causal else T)

    def want(self, n):
        kv = self.kv_len(n)
        if kv == 0:
            return [], 0
        ids = self.table[n // self.s_q, :-(-kv // 64)]
        q = torch.cat([self.q_lat[n], self.q_rope[n]], 1).double().numpy()
        chosen = F.select(q, self.codes[ids], self.scales[ids], kv, self.k, self.n_first, self.n_recent)
        return chosen, len(chosen) * 64 - (-(-kv // 64) * 64 - kv)

    def check(self, res, attention=True):
        pages, table, lens = res.pages.cpu().numpy(), res.table.cpu().numpy(), res.lens.cpu().numpy()
        for n in range(len(self.lens) * self.s_q):
            chosen, length = self.want(n)
            pad = [-1] * (self.k - len(chosen))
            assert pages[n].tolist() == chosen + pad and lens[n] == length, n
            blocks = self.table[n // self.s_q, chosen] if chosen else np.zeros(0, np.int32)
            assert table[n].tolist() == blocks.tolist() + pad
            if not attention or not chosen:
                continue
            keys = self.values[blocks].reshape(-1, 576)[:length]
            q = torch.cat([self.q_lat[n], self.q_rope[n]], 1).double().numpy()
            s = q @ keys.T / math.sqrt(192.0)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            check_out(res.o_lat[n], p / p.sum(1, keepdims=True) @ keys[:, :512])
            np.testing.assert_allclose(res.lse[n].cpu().numpy(), (m + np.log(p.sum(1, keepdims=True)))[:, 0], rtol=0, atol=2e-2)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("lens,s_q,H,k,first,recent", [
    ([1], 1, 128, 4, 1, 1), ([64 * 5], 1, 128, 4, 1, 1), ([64 * 5 + 1, 64, 63, 700], 1, 16, 4, 0, 1),
    ([5000, 9000, 333], 2, 128, 17, 1, 2), ([64 * 130 + 7], 1, 33, 5, 2, 3), ([20000, 8, 4100], 8, 100, 3, 1, 1),
    ([3000, 100], 4, 1, 1, 0, 1), ([3000, 100], 1, 128, 2, 1, 1),
])
def test_selection_and_attention(mla, kind, lens, s_q, H, k, first, recent):
    bt = Batch(mla, lens, s_q, H, k, kind, first, recent, seed=sum(lens) + k)
    res = bt.att.run(*bt.device_args())
    assert res.status.item() == 0
    bt.check(res)


def test_more_pages_than_a_pass_of_the_selection(mla):
    """2500 pages: several tiles a block, several chunks of the ordered pass."""
    bt = Batch(mla, [64 * 2500 - 5, 64 * 1025], 1, 64, 40, n_first=2, n_recent=4, seed=4)
    bt.check(bt.att.run(*bt.device_args()))


def test_many_rows_share_a_block(mla):
    """More rows than SMs: a block walks every tile of its row."""
    bt = Batch(mla, [64 * 260 + 3, 900, 64 * 300] + [700] * 60, 3, 5, 12, seed=9)
    bt.check(bt.att.run(*bt.device_args()), attention=False)


def test_equal_scores_take_the_lowest_pages(mla):
    bt = Batch(mla, [64 * 300], 1, 16, 9, seed=5)
    ids = bt.table[0]
    bt.codes[ids] = 0
    bt.codes[ids[[7, 100, 250]]] = bt.codes[ids[7]] + (np.arange(576) % 3 - 1).astype(np.int8) * 50
    bt.scales[:] = 0.01
    bt.check(bt.att.run(*bt.device_args()), attention=False)
    bt.scales[:] = 0
    res = bt.att.run(*bt.device_args())
    assert res.pages[0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 299]
    bt.check(res, attention=False)


def test_quantised_queries_tie_and_tiny_values(mla):
    """Query values on the half-way points of the 8-bit form, zeros, and magnitudes near the end of fp32."""
    bt = Batch(mla, [64 * 200, 64 * 90], 1, 128, 10, seed=6)
    x = bt.q_lat.float()
    x[0, :, ::2] = torch.sign(x[0, :, ::2]) * 0.5
    x[0, :, 1] = 1.0
    x[0, 3] = 0
    x[1] *= 1e-30
    bt.q_lat = x.to(torch.bfloat16)
    r = bt.q_rope.float()
    r[0, 3] = 0
    r[1] *= 1e-30
    bt.q_rope = r.to(torch.bfloat16)
    bt.check(bt.att.run(*bt.device_args()), attention=False)


def test_non_causal_rows_see_every_page(mla):
    bt = Batch(mla, [64 * 30 + 9, 200], 3, 16, 6, causal=False, seed=8)
    bt.check(bt.att.run(*bt.device_args()))


def test_padded_and_bad_rows_are_left_as_they_were(mla):
    bt = Batch(mla, [64 * 30, 0, 500, 0], 2, 16, 6, "fp4", seed=8)
    bt.att.o_lat.fill_(7.0)
    bt.att.lse.fill_(7.0)
    res = bt.att.run(*bt.device_args())
    assert res.status.item() == 0
    bt.check(res)
    assert torch.all(res.o_lat[[2, 3, 6, 7]] == 7.0) and torch.all(res.lse[[2, 3, 6, 7]] == 7.0)
    args = list(bt.device_args())
    args[6] = torch.tensor([64 * 30, 1, 500, bt.width * 64 + 1], dtype=torch.int32, device=DEV)
    res = bt.att.run(*args)
    assert res.status.item() == mla.STATUS_BAD_SEQLEN
    bt.check(res)


def test_bad_blocks_are_scored_last_and_reported(mla):
    bt = Batch(mla, [64 * 30], 1, 16, 6, seed=8)
    args = list(bt.device_args())
    before = bt.att.run(*args).pages[0].tolist()
    victim = before[2]
    args[5][0, victim] = bt.nb
    res = bt.att.run(*args)
    assert res.status.item() == mla.STATUS_BAD_BLOCK and victim not in res.pages[0].tolist()


def test_selection_does_not_depend_on_the_batch(mla):
    lens = [64 * 150 + 5, 64 * 70, 9000, 64 * 33 + 1]
    bt = Batch(mla, lens, 1, 64, 8, seed=12)
    args = bt.device_args()
    res = bt.att.run(*args)
    for n in range(4):
        one = mla.SparseAttention(1, 1, 64, bt.width, bt.nb, 8)
        r = one.run(args[0][n:n + 1], args[1][n:n + 1], *args[2:5], args[5][n:n + 1], args[6][n:n + 1])
        assert torch.equal(r.pages[0], res.pages[n])


def test_refusals(mla):
    bt = Batch(mla, [700], 1, 16, 4, seed=1)
    args = bt.device_args()
    with pytest.raises(ValueError, match="codes"):
        bt.att.run(args[0], args[1], args[2], args[3].float(), *args[4:])
    with pytest.raises(ValueError, match="seq_lens"):
        bt.att.run(*args[:6], args[6].long())
    with pytest.raises(ValueError, match="kv_pool"):
        bt.att.run(args[0], args[1], args[2].float(), *args[3:])
    with pytest.raises(ValueError, match="q_lat"):
        bt.att.run(args[0][:, :8].contiguous(), *args[1:])


# ------------------------------------------------------------------ the set together
def test_a_captured_serving_step_follows_growing_requests(mla):
    """Tables -> rows into the 4-bit cache -> summaries -> page-sparse and full attention, with the
    plans made on the device: captured once, replayed while requests grow over page borders,
    one finishes (length 0: a padded row) and the lengths stay on the GPU."""
    B, H, width, k, C = 3, 16, 12, 4, 74
    nb = B * width + 1
    cached = torch.tensor([0, 0, 0], dtype=torch.int32, device=DEV)
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    free = torch.from_numpy(np.random.default_rng(0).permutation(nb).astype(np.int32)).to(DEV)
    head = torch.zeros(1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cap = 640
    out = mla.BatchTables.empty(B, cap)
    out.seq_lens, out.free_head = cached, head
    pool = torch.zeros((nb, 64, 416), dtype=torch.uint8, device=DEV)
    kv = torch.zeros((cap, 576), dtype=torch.bfloat16, device=DEV)
    codes, scales = torch.zeros((nb, 576), dtype=torch.int8, device=DEV), torch.zeros(nb, device=DEV)
    q_lat, q_rope = (torch.zeros((B, H, d), dtype=torch.bfloat16, device=DEV) for d in (512, 64))
    dims = mla.make_dims(B, 1, H, width, nb)
    plan_bytes, o_bytes, l_bytes = mla.plan_size(dims, C)
    plan = torch.zeros(plan_bytes // 4, dtype=torch.int32, device=DEV)
    o_part, lse_part = torch.empty(o_bytes // 4, device=DEV), torch.empty(l_bytes // 4, device=DEV)
    o_full = torch.zeros((B, H, 512), dtype=torch.bfloat16, device=DEV)
    att = mla.SparseAttention(B, 1, H, width, nb, k, kv_cache="fp4", num_clusters=C)

    def step():
        mla.build_tables(cached, new, table, free, head, cap, nb, out, status)
        mla.kv_quantize_fp4(kv, out.slots, pool, status)
        mla.summarize_pages(pool, free, codes, scales, "fp4", status)      # every page of the pool: simple, small here
        sparse = att.run(q_lat, q_rope, pool, codes, scales, table, cached)
        mla.plan_device(dims, cached, C, plan, status)
        mla.decode_attn_fp4cache(dims, q_lat, q_rope, pool, table, cached, plan, C, o_part, lse_part, o_full, None, status)
        mla.combine(dims, plan, o_part, lse_part, o_full)
        return sparse

    g = torch.Generator().manual_seed(1)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        sparse = step()                                                    # no requests yet: nothing to do
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            sparse = step()
    held = [np.zeros((0, 576)) for _ in range(B)]
    lens = [0] * B
    for add in ([130, 0, 5], [1, 64, 59], [1, 300, 1], [200, 1, 0], [1, 1, 1], [0, 200, 70]):
        rows = torch.randn((sum(add), 576), generator=g).to(torch.bfloat16)
        codes_, s_ = F.quantize(rows[:, :512].double().numpy())
        packed = F.pack(codes_, s_, rows[:, 512:].contiguous().view(torch.uint8).numpy().reshape(-1, 128))
        vals = F.dequantize_rows(packed)
        at = 0
        for b in range(B):
            held[b] = np.concatenate([held[b], vals[at:at + add[b]]])
            at += add[b]
            lens[b] += add[b]
        kv[:sum(add)] = rows.to(DEV)
        new.copy_(torch.tensor(add, dtype=torch.int32))
        q_lat.copy_(torch.randn((B, H, 512), generator=g).to(torch.bfloat16))
        q_rope.copy_(torch.randn((B, H, 64), generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0 and att.status.item() == 0 and cached.tolist() == lens
        pages, slens = sparse.pages.cpu().numpy(), sparse.lens.tolist()
        for b in range(B):
            if lens[b] == 0:
                assert slens[b] == 0 and torch.all(o_full[b] == 0)
                continue
            q = torch.cat([q_lat[b], q_rope[b]], 1).double().cpu().numpy()

            def attend(keys):
                s = q @ keys.T / math.sqrt(192.0)
                p = np.exp(s - s.max(1, keepdims=True))
                return p / p.sum(1, keepdims=True) @ keys[:, :512]
            check_out(o_full[b], attend(held[b]))
            count = -(-lens[b] // 64)
            padded = np.zeros((count * 64, 576))
            padded[:lens[b]] = held[b]
            pc, ps = summaries(padded.reshape(count, 64, 576))
            chosen = F.select(q, pc, ps, lens[b], k, 1, 1)
            assert pages[b].tolist() == chosen + [-1] * (k - len(chosen))
            keys = np.concatenate([held[b][64 * p:64 * p + 64] for p in chosen])
            assert slens[b] == len(keys)
            check_out(sparse.o_lat[b], attend(keys))


def test_another_stream_and_two_objects_at_once(mla):
    """Two selections on two streams do not touch one another's buffers."""
    a = Batch(mla, [64 * 150 + 5, 4000], 1, 64, 8, "fp4", seed=21)
    b = Batch(mla, [64 * 90, 64 * 300 + 1, 77], 2, 128, 16, "bf16", seed=22)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    args_a, args_b = a.device_args(), b.device_args()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(sa):
            ra = a.att.run(*args_a)
        rb = b.att.run(*args_b, stream=sb)
    torch.cuda.synchronize()
    a.check(ra)
    b.check(rb)
