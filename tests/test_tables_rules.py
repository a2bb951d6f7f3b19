"""The admission rules of build_tables by hand, on the oracle (CPU) and on the GPU."""
import pytest
import torch

from oracle import fp4 as F


def on_gpu(cached, new, table, free, head, max_new, num_blocks):
    from head_latent_attention_04_b200 import mla
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = i32(table)
    r = mla.build_tables(i32(cached), i32(new), t, i32(free), i32([head]), max_new, num_blocks, status=status)
    torch.cuda.synchronize()
    assert status.item() in (0, mla.STATUS_NO_SPACE)
    return (t.tolist(), r.seq_lens.tolist(), r.cu_new.tolist(), r.slots.tolist(), r.positions.tolist(),
            r.free_head.item(), status.item() == mla.STATUS_NO_SPACE)


# (cached, new, table, free, head, max_new) and what comes out
CASES = {
    # a long prompt that gets no blocks takes no room in the slot map from the decoding requests behind it
    "refused for blocks, the next one goes on": (
        ([0, 63], [640, 1], [[-1] * 10, [4] + [-1] * 9], [7], 0, 640),
        ([[-1] * 10, [4] + [-1] * 9], [0, 64], [0, 0, 1], [4 * 64 + 63] + [-1] * 639, [63] + [-1] * 639, 0, True)),
    # refused for blocks, then one that would not fit the map beside it, then one that does not fit at all
    "the map is filled by those that get blocks": (
        ([0, 10, 20, 30], [128, 3, 2, 1], [[-1, -1], [5, -1], [6, -1], [8, -1]], [7], 0, 5),
        ([[-1, -1], [5, -1], [6, -1], [8, -1]], [0, 13, 22, 30], [0, 0, 3, 5, 5],
         [330, 331, 332, 404, 405], [10, 11, 12, 20, 21], 0, True)),
    # a request refused for the map keeps its place in front: no later one gets tokens
    "refused for the map": (
        ([10, 20, 30], [3, 4, 1], [[5, -1], [6, -1], [8, -1]], [7], 0, 5),
        ([[5, -1], [6, -1], [8, -1]], [13, 20, 30], [0, 3, 3, 3], [330, 331, 332, -1, -1], [10, 11, 12, -1, -1], 0, True)),
}


@pytest.mark.parametrize("name", CASES)
def test_admission_by_hand(name):
    args, want = CASES[name]
    assert F.build_tables(*args) == want


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_admission_by_hand_on_the_gpu(name):
    args, want = CASES[name]
    assert on_gpu(*args, num_blocks=16) == want


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_admission_of_large_batches(seed):
    """More requests than one chunk, some refused for their blocks and some for the slot map."""
    import random
    rng = random.Random(seed)
    B = rng.choice([700, 1024, 1500, 2500])
    cached = [rng.choice([0, 63, 64, 100, -1, 200]) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 1, 2, 70, 300]) for _ in range(B)]
    width = 6
    held = [-(-max(c, 0) // 64) for c in cached]
    ids = list(range(sum(held) + B))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free = ids[at:at + rng.choice([5, B // 3, B])]
    max_new = rng.choice([B // 2, 3 * B, 9000])
    assert on_gpu(cached, new, table, free, 0, max_new, len(ids)) == F.build_tables(cached, new, table, free, 0, max_new)


# ------------------------------------------------------------------ lengths that fall (rejected drafts)
def test_a_page_of_rejected_drafts_is_kept_by_hand():
    """63 cached, two drafts, one rejected, two drafts again: page 1 gets one block, once."""
    table, held = [[4, -1, -1]], [1]
    table, lens, _, slots, _, head, bad = F.build_tables([63], [2], table, [7, 8, 9], 0, 2, held)
    assert (table, lens, slots, head, held, bad) == ([[4, 7, -1]], [65], [4 * 64 + 63, 7 * 64], 1, [2], False)
    table, lens, _, slots, _, head, bad = F.build_tables([64], [2], table, [7, 8, 9], head, 2, held)
    assert (table, lens, slots, head, held, bad) == ([[4, 7, -1]], [66], [7 * 64, 7 * 64 + 1], 1, [2], False)
    assert F.build_tables([64], [2], [[4, 7, -1]], [7, 8, 9], 1, 2)[0] == [[4, 8, -1]]      # without the count: 7 is lost


def draft_steps(seed, B, width, steps, max_draft):
    """Per step (new tokens, tokens kept of them) of requests that end now and then; None: ends."""
    import random
    rng = random.Random(seed)
    for _ in range(steps):
        yield [rng.randint(0, max_draft) for _ in range(B)], [rng.random() for _ in range(B)], \
              [rng.random() < 0.03 for _ in range(B)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,max_draft,start", [(1, 3, 62), (7, 8, 0), (40, 8, 50), (1100, 70, 0), (5, 2000, 0)])
def test_lengths_that_fall_lose_no_block(B, max_draft, start):
    """Drafts are written and mostly rejected; blocks of requests that end return to the list.  Every
    block is held by one row or is free, and the answers are the oracle's."""
    from head_latent_attention_04_b200 import mla
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    width = 8 + max_draft * 3 // 64
    nb = B * width
    lens, held = [0] * B, [0] * B
    table = [[-1] * width for _ in range(B)]
    free = list(range(nb))
    cached, dev_held, dev_table = i32(lens), i32(held), i32(table)
    first = [start] * B
    for step, (new, kept, ends) in enumerate([(first, [1.0] * B, [False] * B)] + list(draft_steps(B, B, width, 14, max_draft))):
        new = [min(n, width * 64 - c) for n, c in zip(new, lens)]
        free_dev, head = i32(free), i32([0])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = mla.build_tables(cached, i32(new), dev_table, free_dev, head, sum(new) + 2, nb, status=status,
                             held_pages=dev_held)
        want = F.build_tables(lens, new, table, free, 0, sum(new) + 2, held)
        table = want[0]
        assert dev_table.tolist() == table and r.seq_lens.tolist() == want[1] and r.slots.tolist() == want[3]
        assert r.free_head.item() == want[5] and dev_held.tolist() == held and status.item() == 0 and not want[6]
        free = free[want[5]:]
        for b in range(B):                                   # some of the new tokens are rejected, some requests end
            lens[b] = lens[b] + int(new[b] * kept[b])
            if ends[b] or lens[b] > (width - 2) * 64:
                free += table[b][:held[b]]
                lens[b] = held[b] = 0
        used = [blk for b in range(B) for blk in table[b][:held[b]]]
        assert sorted(used + free) == list(range(nb)), step
        cached.copy_(i32(lens)), dev_held.copy_(i32(held))


@pytest.mark.gpu
def test_held_pages_in_a_captured_step_and_out_of_range():
    from head_latent_attention_04_b200 import mla
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cached, new, held, head = i32([63, 10]), i32([2, 2]), i32([0, 9]), i32([0])
    table, free, status = i32([[4, -1, -1], [5, -1, -1]]), i32([7, 8, 9]), i32([0])
    out = mla.BatchTables.empty(2, 4)
    out.free_head = head
    mla.build_tables(cached, new, table, free, head, 4, 16, out, status, held_pages=held)
    assert status.item() == mla.STATUS_NO_SPACE              # row 1 claims more pages than the table has
    assert table.tolist() == [[4, 7, -1], [5, -1, -1]] and held.tolist() == [2, 9] and out.seq_lens.tolist() == [65, 10]
    status.zero_(), held.copy_(i32([2, 0])), cached.copy_(i32([63, 10]))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        mla.build_tables(cached, new, table, free, head, 4, 16, out, status, held_pages=held)
    for lens, want_held, want_head in ([63, 10], [2, 1], 1), ([64, 63], [2, 2], 2), ([63, 62], [2, 2], 2):
        cached.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert held.tolist() == want_held and head.item() == want_head and status.item() == 0
    assert table.tolist() == [[4, 7, -1], [5, 8, -1]]
    with pytest.raises(ValueError, match="held_pages"):
        mla.build_tables(cached, new, table, free, head, 4, 16, out, status, held_pages=held[:1].contiguous())


def test_held_pages_alignment_is_checked():
    from head_latent_attention_04_b200 import mla
    A = 0x1000
    args = [2, A, A, 4, A, A + 2, A, 8, A, 8, 16, A, A, A, A, A, None, None]
    assert mla._lib.mla_build_tables_held(*args) == 1 and b"held_pages" in mla._lib.mla_last_error_string()
