"""A captured serving step over the life of requests: they start, grow over page borders, have drafts
rejected, end, and give their blocks and their row to another one."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4 as F
from tests.gpu_helpers import check_out
from tests.test_gpu_pages import summaries

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_04_b200 import mla as m
    return m


def test_requests_end_and_drafts_are_rejected_under_one_graph(mla):
    """Tables -> rows into the 4-bit cache -> summaries -> page-sparse and full attention, captured once; after
    every replay each block of the pool is free or held by one row."""
    B, H, width, k, C, cap = 3, 16, 9, 3, 74, 400
    nb = 17
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    cached, new, held, head, status = i32([0] * B), i32([0] * B), i32([0] * B), i32([0]), i32([0])
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    free = torch.full((nb,), -1, dtype=torch.int32, device=DEV)
    every = torch.arange(nb, dtype=torch.int32, device=DEV)
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
        mla.build_tables(cached, new, table, free, head, cap, nb, out, status, held_pages=held)
        mla.kv_quantize_fp4(kv, out.slots, pool, status)
        mla.summarize_pages(pool, every, codes, scales, "fp4", status)
        sparse = att.run(q_lat, q_rope, pool, codes, scales, table, cached)
        mla.plan_device(dims, cached, C, plan, status)
        mla.decode_attn_fp4cache(dims, q_lat, q_rope, pool, table, cached, plan, C, o_part, lse_part, o_full, None, status)
        mla.combine(dims, plan, o_part, lse_part, o_full, status=status)
        return sparse

    g = torch.Generator().manual_seed(3)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            sparse = step()

    blocks = list(range(nb))                             # free blocks, as the host keeps them
    keys = [np.zeros((0, 576)) for _ in range(B)]        # each request's rows as the cache holds them
    ended = [0] * B
    # per step: new tokens, how many of them are kept, requests that end after it
    life = [([130, 63, 5], [130, 63, 5], []), ([2, 2, 60], [1, 1, 60], []), ([8, 8, 8], [1, 0, 8], []),
            ([8, 8, 200], [2, 1, 200], [1]), ([70, 0, 8], [70, 0, 0], []), ([1, 300, 8], [1, 300, 1], [0]),
            ([65, 4, 8], [65, 1, 0], [2]), ([8, 8, 100], [0, 0, 100], []), ([8, 1, 1], [8, 1, 1], [0, 1, 2]),
            ([64, 128, 1], [64, 128, 1], [])]
    for add, kept, end in life:
        free[:len(blocks)] = i32(blocks)
        free[len(blocks):] = -1
        head.zero_()
        lens = [len(x) + a for x, a in zip(keys, add)]
        rows = torch.randn((sum(add), 576), generator=g).to(torch.bfloat16)
        c, s = F.quantize(rows[:, :512].double().numpy())
        packed = F.pack(c, s, rows[:, 512:].contiguous().view(torch.uint8).numpy().reshape(-1, 128))
        vals, at = F.dequantize_rows(packed), 0
        now = []
        for b in range(B):
            now.append(np.concatenate([keys[b], vals[at:at + add[b]]]))
            at += add[b]
        kv[:sum(add)] = rows.to(DEV)
        new.copy_(torch.tensor(add, dtype=torch.int32))
        q_lat.copy_(torch.randn((B, H, 512), generator=g).to(torch.bfloat16))
        q_rope.copy_(torch.randn((B, H, 64), generator=g).to(torch.bfloat16))
        o_full.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0 and att.status.item() == 0 and cached.tolist() == lens
        blocks = blocks[head.item():]
        rows_of = [table[b, :held[b]].tolist() for b in range(B)]
        assert sorted(blocks + sum(rows_of, [])) == list(range(nb))          # no block lost or held twice
        pages, slens = sparse.pages.cpu().numpy(), sparse.lens.tolist()
        for b in range(B):
            if lens[b] == 0:
                assert slens[b] == 0 and torch.all(o_full[b] == 9.0)          # a row that has ended: left as it was
                ended[b] += 1
                continue
            q = torch.cat([q_lat[b], q_rope[b]], 1).double().cpu().numpy()

            def attend(rows):
                x = q @ rows.T / math.sqrt(192.0)
                p = np.exp(x - x.max(1, keepdims=True))
                return p / p.sum(1, keepdims=True) @ rows[:, :512]
            check_out(o_full[b], attend(now[b]))
            count = -(-lens[b] // 64)
            padded = np.zeros((count * 64, 576))
            padded[:lens[b]] = now[b]
            pc, ps = summaries(padded.reshape(count, 64, 576))
            chosen = F.select(q, pc, ps, lens[b], k, 1, 1)
            assert pages[b].tolist() == chosen + [-1] * (k - len(chosen))
            part = np.concatenate([now[b][64 * p:64 * p + 64] for p in chosen])
            assert slens[b] == len(part)
            check_out(sparse.o_lat[b], attend(part))
        for b in range(B):
            keys[b] = now[b][:len(keys[b]) + kept[b]]
            if b in end:
                blocks += rows_of[b]
                keys[b] = keys[b][:0]
                held[b] = 0
        cached.copy_(i32([len(x) for x in keys]))
    assert ended == [0, 1, 0]
