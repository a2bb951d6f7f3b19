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
