"""Cases of the long-context serving operators, with their plain forms.

Five operators are measured, in the order in which a serving step uses them:

* ``tables``  block tables, slot maps and the split-KV plan made on the GPU from
  request lengths (``mla.build_tables``, ``mla.plan_device``);
* ``append``  new cache rows written to a 4-bit latent cache and read back
  (``mla.kv_quantize_fp4``, ``mla.kv_dequantize_fp4``);
* ``attend``  absorbed MLA attention over the 4-bit cache
  (``mla.decode_attn_fp4cache``, ``mla.combine``);
* ``summary`` the 8-bit summaries of full cache pages (``mla.summarize_pages``);
* ``sparse``  attention of each query over the pages a cheap score picks
  (``mla.select_pages``, ``mla.plan_device``, then the attention of the cache's kind).

Formulas.  A cached token is a row [c (512) | r (64)].  The 4-bit row keeps c in
sixteen groups of 32 columns: s = fp16(amax / 6), code = E2M1(c / s) rounded to
nearest even and saturated at 6; r stays bf16.  Row bytes: 256 codes (column 2i
in the low nibble of byte i) | 16 fp16 scales | 64 bf16.  A page's summary is the
mean of its 64 rows m, in 8 bits: scale = fp32(amax / 127), code = rint(127 m / amax).
A query's score of a page is fp32(max_h((qcode_h . pcode) * qscale_h) * pscale) with
qcode, qscale the same 8-bit form of [q_lat | q_rope]; the first ``n_first`` and
the last ``n_recent`` pages are always taken, then the highest scores, ties to the lowest
page, up to k pages.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAGE, D_C, D_R, ROW = 64, 512, 64, 576
GROUP, FP4_ROW = 32, 416
CLUSTERS = 74                       # two-CTA clusters of a 148-SM card, what the plans are cut for
SCALE = 1.0 / math.sqrt(128 + 64)
PLAN_MAGIC, PLAN_HEADER, PLAN_ITEM, PLAN_ITEM_COST = 0x314C414D, 16, 8, 5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 32 requests: the per-step bookkeeping of a decode batch
        {"name": "tables decode", "op": "tables", "B": 32, "s_q": 1, "cached_min": 4000, "cached_max": 4191,
         "new_min": 1, "new_max": 1, "heads": 128},
        # a mixed batch: long chunks of prompts and drafts side by side, about a million new tokens
        {"name": "tables prompts", "op": "tables", "B": 509, "s_q": 2, "cached_min": 2, "cached_max": 30000,
         "new_min": 0, "new_max": 4096, "heads": 128},
        # the rows of one decode step of 32 requests
        {"name": "append step", "op": "append", "n": 32, "blocks": 4096, "pad": 0},
        # a prompt of odd length, in a batch padded to a fixed size
        {"name": "append prompt", "op": "append", "n": 16301, "blocks": 4096, "pad": 83},
        # two short requests and 16 heads: what a small tensor-parallel shard sees, launch latency counts
        {"name": "attend tiny", "op": "attend", "B": 2, "s_q": 1, "heads": 16, "len_min": 256, "len_max": 256},
        # the decode batch of 32 requests at 4K context
        {"name": "attend batch", "op": "attend", "B": 32, "s_q": 1, "heads": 128, "len_min": 4096, "len_max": 4096},
        # four requests at 128K context: every row split over the whole card
        {"name": "attend long", "op": "attend", "B": 4, "s_q": 1, "heads": 128, "len_min": 131072, "len_max": 131072},
        # 128 ragged requests with one drafted token each, the largest batch
        {"name": "attend drafts", "op": "attend", "B": 128, "s_q": 2, "heads": 128, "len_min": 294, "len_max": 32768},
        # the pages that a step's requests have just filled, 4-bit cache
        {"name": "summary step", "op": "summary", "n": 61, "cache": "fp4"},
        # all pages of 512K tokens of prompts, bf16 cache
        {"name": "summary prompt", "op": "summary", "n": 8192, "cache": "bf16"},
        # four requests at 128K context attending to 2K tokens each, bf16 cache
        {"name": "sparse long", "op": "sparse", "B": 4, "s_q": 1, "heads": 128, "len_min": 131072, "len_max": 131072,
         "k": 32, "n_first": 1, "n_recent": 1, "cache": "bf16"},
        # 61 ragged requests with one drafted token each over a 4-bit cache, some shorter than the selection
        {"name": "sparse drafts", "op": "sparse", "B": 61, "s_q": 2, "heads": 128, "len_min": 1000, "len_max": 65536,
         "k": 65, "n_first": 1, "n_recent": 2, "cache": "fp4"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend", "summary", "sparse"])
    heads = rng.choice([128, 128, 64, rng.randint(1, 128)])
    if op == "tables":
        lo = _log_int(rng, 8, 20000)
        return {"op": op, "B": _log_int(rng, 1, 500), "s_q": rng.randint(1, 8), "cached_min": lo,
                "cached_max": lo + rng.randint(0, 10000), "new_min": rng.randint(0, 1),
                "new_max": _log_int(rng, 1, 4000), "heads": heads}
    if op == "append":
        n = _log_int(rng, 1, 16384)
        return {"op": op, "n": n, "blocks": rng.randint(256, 4096), "pad": rng.choice([0, rng.randint(1, 100)])}
    if op == "summary":
        cache = rng.choice(["bf16", "fp4"])
        return {"op": op, "n": _log_int(rng, 1, 8192), "cache": cache}
    s_q = rng.choice([1, 1, 2, 3, 4])
    hi = _log_int(rng, 64, 131072)
    lo = max(s_q, int(hi * rng.choice([1.0, 0.5, 0.02])))
    B = _log_int(rng, 1, max(1, min(128, 700000 // hi // s_q)))
    if op == "attend":
        return {"op": op, "B": B, "s_q": s_q, "heads": heads, "len_min": lo, "len_max": hi}
    n_first, n_recent = rng.randint(0, 3), rng.randint(1, 4)
    return {"op": op, "B": B, "s_q": s_q, "heads": heads, "len_min": lo, "len_max": hi,
            "k": n_first + n_recent + _log_int(rng, 1, 128), "n_first": n_first, "n_recent": n_recent,
            "cache": rng.choice(["bf16", "fp4"])}


def _lens(case, key="len", tag="len"):
    """The request lengths of a case: log-uniform between its bounds, both bounds present."""
    lo, hi = case[key + "_min"], case[key + "_max"]
    rng = random.Random(f"{tag} {lo} {hi} {case['B']}")
    out = []
    for b in range(case["B"]):
        if lo < 1:
            out.append(rng.randint(lo, hi))
        else:
            out.append(_log_int(rng, lo, hi))
    out[0] = hi
    if case["B"] > 1:
        out[-1] = lo
    return out


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _cache_rows(gen, blocks, drift):
    """bf16 pages [blocks][64][576]; with ``drift`` the rows of a page share an offset, as
    neighbouring tokens do, so that pages differ in what they hold."""
    pool = torch.empty((blocks, PAGE, ROW), dtype=torch.bfloat16, device="cuda")
    for p0 in range(0, blocks, 2048):
        p1 = min(blocks, p0 + 2048)
        x = torch.randn((p1 - p0, PAGE, ROW), generator=gen, device="cuda")
        if drift:
            x = 0.9 * x + 0.45 * torch.randn((p1 - p0, 1, ROW), generator=gen, device="cuda")
        pool[p0:p1] = x.to(torch.bfloat16)
    return pool


def _fp4_round(a):
    """|x| in units of the scale -> the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    fine, mid, coarse = torch.round(a * 2) / 2, torch.round(a), torch.round(a / 2) * 2
    return torch.where(a < 2, fine, torch.where(a < 4, mid, coarse)).clamp(max=6.0)


def _fp4_codes(values):
    """Values of the 4-bit grid (signed) -> codes 0 .. 15."""
    a = values.abs()
    mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4))
    return mag.to(torch.uint8) + 8 * torch.signbit(values).to(torch.uint8)


def _fp4_pack(rows):
    """bf16 rows [..., 576] -> 4-bit rows uint8 [..., 416], for the pools that a case starts from."""
    lead = rows.shape[:-1]
    c = rows[..., :D_C].float().reshape(-1, D_C // GROUP, GROUP)
    s = (c.abs().amax(-1, keepdim=True) / 6).to(torch.float16)
    sf = s.float()
    v = torch.where(sf > 0, _fp4_round((c / sf).abs()), torch.zeros_like(c))
    codes = _fp4_codes(torch.copysign(v, c)).reshape(-1, D_C)
    out = torch.empty((codes.shape[0], FP4_ROW), dtype=torch.uint8, device=rows.device)
    out[:, :256] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    out[:, 256:288] = s.reshape(-1, 16).contiguous().view(torch.uint8)
    out[:, 288:] = rows[..., D_C:].reshape(-1, D_R).contiguous().view(torch.uint8)
    return out.reshape(*lead, FP4_ROW)


def _fp4_pool(pool):
    out = torch.empty((pool.shape[0], PAGE, FP4_ROW), dtype=torch.uint8, device=pool.device)
    for p0 in range(0, pool.shape[0], 512):
        out[p0:p0 + 512] = _fp4_pack(pool[p0:p0 + 512])
    return out


def _paged(case, gen, drift):
    lens = _lens(case)
    pages = [(t + PAGE - 1) // PAGE for t in lens]
    total = sum(pages)
    max_blocks = max(pages)
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["B"], max_blocks), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    pool = _cache_rows(gen, total, drift)
    if case.get("cache", "fp4") == "fp4":
        pool = _fp4_pool(pool)
    N, H = case["B"] * case["s_q"], case["heads"]
    return dict(lens_host=lens, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), table=table, pool=pool,
                q_lat=_randn(gen, N, H, D_C), q_rope=_randn(gen, N, H, D_R))


def _summaries(pool, kind):
    """The 8-bit summaries of a whole pool (codes int8 [blocks][576], scales fp32 [blocks])."""
    codes = torch.empty((pool.shape[0], ROW), dtype=torch.int8, device=pool.device)
    scales = torch.empty(pool.shape[0], dtype=torch.float32, device=pool.device)
    for p0 in range(0, pool.shape[0], 256):
        part = pool[p0:p0 + 256]
        rows = part.double() if kind == "bf16" else _fp4_values(part)
        m = rows.sum(1) / PAGE
        amax = m.abs().amax(-1, keepdim=True)
        codes[p0:p0 + 256] = torch.where(amax > 0, torch.round(m * 127 / amax), torch.zeros_like(m)).to(torch.int8)
        scales[p0:p0 + 256] = (amax[:, 0] / 127).float()
    return codes, scales


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "tables":
        B, s_q = case["B"], case["s_q"]
        cached, new = _lens(case, "cached", "cached"), _lens(case, "new", "new")
        cached = [max(t, s_q) for t in cached]
        held = [(t + PAGE - 1) // PAGE for t in cached]
        need = [(t + n + PAGE - 1) // PAGE - h for t, n, h in zip(cached, new, held)]
        blocks = sum(held) + sum(need) + 97
        max_blocks = max(h + n for h, n in zip(held, need)) + 3
        perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = perm[at:at + h]
            at += h
        as_dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        return dict(cached=as_dev(cached), new=as_dev(new), table=table, free=perm[at:].contiguous(),
                    head=as_dev([11]), blocks=blocks, max_new=sum(new) + 5)
    if op == "append":
        n, pad, blocks = case["n"], case["pad"], case["blocks"]
        kv = _randn(gen, n + pad, ROW)
        slots = torch.randperm(blocks * PAGE, generator=gen, device="cuda")[:n + pad].to(torch.int32)
        if pad:
            slots[n:] = -1
        return dict(kv=kv, slots=slots, pool=torch.zeros((blocks, PAGE, FP4_ROW), dtype=torch.uint8, device="cuda"))
    if op == "summary":
        pool = _cache_rows(gen, case["n"], True)
        if case["cache"] == "fp4":
            pool = _fp4_pool(pool)
        blocks = torch.randperm(case["n"], generator=gen, device="cuda").to(torch.int32)
        return dict(pool=pool, blocks=blocks)
    st = _paged(case, gen, op == "sparse")
    if op == "sparse":
        st["codes"], st["scales"] = _summaries(st["pool"], case["cache"])
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    op = case["op"]
    if not own:
        if op == "append":
            st["out"] = torch.zeros((case["n"] + case["pad"], ROW), dtype=torch.bfloat16, device="cuda")
        return st
    from head_latent_attention_04_b200 import mla
    H = case.get("heads", 0)
    if op == "tables":
        st["dims"] = mla.make_dims(case["B"], case["s_q"], H, st["table"].shape[1], st["blocks"])
    if op == "append":
        st["out"] = torch.zeros((case["n"] + case["pad"], ROW), dtype=torch.bfloat16, device="cuda")
    if op == "summary":
        st["codes"] = torch.zeros((case["n"], ROW), dtype=torch.int8, device="cuda")
        st["scales"] = torch.zeros(case["n"], dtype=torch.float32, device="cuda")
    if op == "attend":
        N, blocks = case["B"] * case["s_q"], st["pool"].shape[0]
        st["dims"] = dims = mla.make_dims(case["B"], case["s_q"], H, st["table"].shape[1], blocks)
        plan, slots = mla.plan(dims, st["lens_host"], CLUSTERS)
        st["plan"], st["slots"] = torch.from_numpy(plan).cuda(), slots
        st["o_part"] = torch.empty(max(slots, 1) * H * D_C, dtype=torch.float32, device="cuda")
        st["lse_part"] = torch.empty(max(slots, 1) * H, dtype=torch.float32, device="cuda")
        st["o_lat"] = torch.empty((N, H, D_C), dtype=torch.bfloat16, device="cuda")
    if op == "sparse":
        st["decoder"] = mla.SparseAttention(case["B"], case["s_q"], H, st["table"].shape[1], st["pool"].shape[0],
                                            k=case["k"], n_first=case["n_first"], n_recent=case["n_recent"],
                                            kv_cache=case["cache"], num_clusters=CLUSTERS)
    return st


# ------------------------------------------------------------------ the pass
def run(st):
    return (_run_own if own else _run_plain)[st["case"]["op"]](st)


def _own_tables(st):
    from head_latent_attention_04_b200 import mla
    t = mla.build_tables(st["cached"], st["new"], st["table"], st["free"], st["head"], st["max_new"], st["blocks"])
    plan = mla.plan_device(st["dims"], t.seq_lens, CLUSTERS)
    return st["table"], t.seq_lens, t.cu_new, t.slots, t.positions, t.free_head, plan


def _own_append(st):
    from head_latent_attention_04_b200 import mla
    mla.kv_quantize_fp4(st["kv"], st["slots"], st["pool"])
    return mla.kv_dequantize_fp4(st["pool"], st["slots"], st["out"])


def _own_attend(st):
    from head_latent_attention_04_b200 import mla
    mla.decode_attn_fp4cache(st["dims"], st["q_lat"], st["q_rope"], st["pool"], st["table"], st["lens"], st["plan"],
                             CLUSTERS, st["o_part"], st["lse_part"], st["o_lat"])
    if st["slots"] > 0:
        mla.combine(st["dims"], st["plan"], st["o_part"], st["lse_part"], st["o_lat"])
    return st["o_lat"]


def _own_summary(st):
    from head_latent_attention_04_b200 import mla
    codes, scales = mla.summarize_pages(st["pool"], st["blocks"], st["codes"], st["scales"],
                                        kv_cache=st["case"]["cache"])
    return codes * scales[:, None]


def _own_sparse(st):
    r = st["decoder"].run(st["q_lat"], st["q_rope"], st["pool"], st["codes"], st["scales"], st["table"], st["lens"])
    return r.pages, r.lens, r.o_lat


_run_own = {"tables": _own_tables, "append": _own_append, "attend": _own_attend, "summary": _own_summary,
            "sparse": _own_sparse}


# ------------------------------------------------------------------ plain forms
def _plain_plan(B, s_q, heads, max_blocks, seq_lens):
    """The split-KV plan as int32 words: rows laid end to end, each after five virtual pages,
    cut into equal ranges; one group of ranges for each query position."""
    dev, N = seq_lens.device, B * s_q
    groups = s_q if CLUSTERS >= s_q else 1
    per = CLUSTERS // groups
    T = seq_lens.long()
    qi = torch.arange(s_q, device=dev)
    kv = (T[:, None] - s_q + 1 + qi[None]).reshape(-1)
    pages = (kv + PAGE - 1) // PAGE
    pieces = []
    for g in range(groups):
        rows = torch.arange(N, device=dev)[g::groups] if groups > 1 else torch.arange(N, device=dev)
        cost = pages[rows] + PLAN_ITEM_COST
        r1 = cost.cumsum(0)
        r0 = r1 - pages[rows]
        cut = torch.arange(per + 1, device=dev) * r1[-1] // per
        a = torch.maximum(cut[None, :-1], r0[:, None])
        e = torch.minimum(cut[None, 1:], r1[:, None])
        i, c = torch.nonzero(a < e, as_tuple=True)
        pieces.append(torch.stack([g * per + c, rows[i], a[i, c] - r0[i], e[i, c] - r0[i]], 1))
    pieces = torch.cat(pieces)
    cluster, row = pieces[:, 0], pieces[:, 1]
    count = torch.bincount(row, minlength=N)
    slot_end = torch.where(count > 1, count, 0).cumsum(0)
    slot_begin = torch.cat([slot_end.new_zeros(1), slot_end])
    items = torch.zeros((pieces.shape[0], PLAN_ITEM), dtype=torch.long, device=dev)
    items[:, 0], items[:, 1] = row // s_q, row % s_q
    items[:, 2:4] = pieces[:, 2:4]
    items[:, 4] = kv[row]
    first = torch.ones_like(row, dtype=torch.bool)          # pieces of a row are neighbours
    first[1:] = row[1:] != row[:-1]
    at = torch.arange(row.shape[0], device=dev)
    rank = at - torch.where(first, at, 0).cummax(0).values
    items[:, 5] = torch.where(count[row] > 1, slot_begin[row] + rank, -1)
    items[:, 6] = row
    begin = torch.cat([row.new_zeros(1), torch.bincount(cluster, minlength=CLUSTERS).cumsum(0)])
    words = PLAN_HEADER + CLUSTERS + 1 + (CLUSTERS + N) * PLAN_ITEM + N + 1
    off_items = PLAN_HEADER + CLUSTERS + 1
    off_rows = off_items + items.numel()
    plan = torch.zeros(words, dtype=torch.long, device=dev)
    head = [PLAN_MAGIC, CLUSTERS, items.shape[0], 0, N, heads, s_q, B, PLAN_HEADER, off_items, off_rows,
            off_rows + N + 1, max_blocks, 1]
    plan[:len(head)] = torch.tensor(head, device=dev)
    plan[3] = slot_end[-1]
    plan[PLAN_HEADER:off_items] = begin
    plan[off_items:off_rows] = items.reshape(-1)
    plan[off_rows:off_rows + N + 1] = slot_begin
    return plan.to(torch.int32)


def _plain_tables(st):
    case, table = st["case"], st["table"]
    cached, new = st["cached"].long(), st["new"].long()
    held = (cached + PAGE - 1) // PAGE
    total = cached + new
    need = (total + PAGE - 1) // PAGE - held
    before = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=table.device)[None]
    take = (col >= held[:, None]) & (col < (held + need)[:, None])
    index = st["head"].long() + before[:, None] + col - held[:, None]
    table[:] = torch.where(take, st["free"][index.clamp(0, st["free"].shape[0] - 1)], table)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    tok = torch.arange(st["max_new"], device=table.device)
    b = torch.searchsorted(cu[1:], tok, right=True).clamp(max=case["B"] - 1)
    pos = cached[b] + tok - cu[b]
    live = tok < cu[-1]
    page = torch.where(live, pos // PAGE, 0)
    slots = torch.where(live, table[b, page].long() * PAGE + pos % PAGE, -1)
    i32 = lambda x: x.to(torch.int32)
    plan = _plain_plan(case["B"], case["s_q"], case["heads"], table.shape[1], total)
    return (table, i32(total), i32(cu), i32(slots), i32(torch.where(live, pos, -1)),
            i32(st["head"].long() + need.sum()), plan)


def _fp4_values(rows):
    """4-bit rows uint8 [..., 416] -> their values, float64 [..., 576]."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                        device=rows.device)
    byte = rows[..., :256].long()
    codes = torch.stack([byte & 15, byte >> 4], -1).reshape(*rows.shape[:-1], D_C // GROUP, GROUP)
    s = rows[..., 256:288].contiguous().view(torch.float16).double()
    c = (grid[codes] * s[..., None]).reshape(*rows.shape[:-1], D_C)
    r = rows[..., 288:].contiguous().view(torch.bfloat16).double()
    return torch.cat([c, r], -1)


def _plain_append(st):
    live = st["slots"] >= 0
    where = st["slots"][live].long()
    flat = st["pool"].view(-1, FP4_ROW)
    flat[where] = _fp4_pack(st["kv"][live])
    st["out"][live] = _fp4_values(flat[where]).to(torch.bfloat16)
    return st["out"]


def _plain_rows(pool, ids, kind):
    rows = pool[ids.long()]
    rows = rows.reshape(-1, rows.shape[-1])
    return rows.float() if kind == "bf16" else _fp4_values(rows).float()


def _plain_attention(q_lat, q_rope, rows, lens):
    """Queries [n][h][*] over keys ``rows`` [t][576]; query i sees keys below lens[i]."""
    q = torch.cat([q_lat, q_rope], -1).float()
    s = (q.reshape(-1, ROW) @ rows.t()).reshape(*q.shape[:2], -1) * SCALE
    hidden = torch.arange(rows.shape[0], device=rows.device)[None] >= lens[:, None]
    s = s.masked_fill(hidden[:, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p.reshape(-1, p.shape[-1]) @ rows[:, :D_C]).reshape(*q.shape[:2], D_C)
    return (o / p.sum(-1, keepdim=True)).to(torch.bfloat16)


def _plain_attend(st):
    case = st["case"]
    s_q = case["s_q"]
    out = torch.empty_like(st["q_lat"])
    for b, T in enumerate(st["lens_host"]):
        rows = _plain_rows(st["pool"], st["table"][b, :(T + PAGE - 1) // PAGE], "fp4")[:T]
        n = slice(b * s_q, (b + 1) * s_q)
        lens = torch.arange(T - s_q + 1, T + 1, device=rows.device)
        out[n] = _plain_attention(st["q_lat"][n], st["q_rope"][n], rows, lens)
    return out


def _plain_summary(st):
    pool, codes = st["pool"], torch.empty((st["case"]["n"], ROW), dtype=torch.float32, device="cuda")
    for i in range(0, st["case"]["n"], 256):
        ids = st["blocks"][i:i + 256].long()
        part = pool[ids]
        rows = part.double() if st["case"]["cache"] == "bf16" else _fp4_values(part)
        m = rows.sum(1) / PAGE
        amax = m.abs().amax(-1, keepdim=True)
        c = torch.where(amax > 0, torch.round(m * 127 / amax), torch.zeros_like(m))
        codes[ids] = c.float() * (amax / 127).float()
    return codes


def _plain_select(st):
    """Pages [N][k] (-1 behind the last) and the tokens they hold, for every query row."""
    case = st["case"]
    k, s_q = case["k"], case["s_q"]
    q = torch.cat([st["q_lat"], st["q_rope"]], -1).double()
    amax = q.abs().amax(-1, keepdim=True)
    qcode = torch.where(amax > 0, torch.round(q * 127 / amax), torch.zeros_like(q)).float()
    qscale = (amax / 127).float().double()
    pages = torch.full((q.shape[0], k), -1, dtype=torch.int32, device=q.device)
    lens = torch.zeros(q.shape[0], dtype=torch.int32, device=q.device)
    for b, T in enumerate(st["lens_host"]):
        ids = st["table"][b, :(T + PAGE - 1) // PAGE].long()
        pcode, pscale = st["codes"][ids].float(), st["scales"][ids].double()
        for i in range(s_q):
            n, kv = b * s_q + i, T - s_q + 1 + i
            np_ = (kv + PAGE - 1) // PAGE
            take = torch.arange(np_, device=q.device)
            if np_ > k:
                dot = (qcode[n] @ pcode[:np_].t()).double()         # whole numbers below 2^24
                score = ((dot * qscale[n]).amax(0) * pscale[:np_]).float()
                score[:case["n_first"]] = float("inf")
                score[np_ - case["n_recent"]:] = float("inf")
                take = torch.sort(score, descending=True, stable=True).indices[:k].sort().values
            pages[n, :take.shape[0]] = take.to(torch.int32)
            lens[n] = (take.shape[0] - 1) * PAGE + kv - (np_ - 1) * PAGE
    return pages, lens


def _plain_sparse(st):
    pages, lens = _plain_select(st)
    s_q = st["case"]["s_q"]
    out = torch.empty_like(st["q_lat"])
    count = (lens + PAGE - 1) // PAGE
    for n, c in enumerate(count.tolist()):
        rows = _plain_rows(st["pool"], st["table"][n // s_q, pages[n, :c].long()], st["case"]["cache"])
        out[n] = _plain_attention(st["q_lat"][n:n + 1], st["q_rope"][n:n + 1], rows, lens[n:n + 1])[0]
    return pages, lens, out


_run_plain = {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend, "summary": _plain_summary,
              "sparse": _plain_sparse}


# ------------------------------------------------------------------ work
def work(case):
    """Bytes each read or written once, and the multiplications and additions of the formulas."""
    op = case["op"]
    if op == "tables":
        B, s_q = case["B"], case["s_q"]
        cached, new = _lens(case, "cached", "cached"), _lens(case, "new", "new")
        need = sum((max(t, s_q) + n + PAGE - 1) // PAGE - (max(t, s_q) + PAGE - 1) // PAGE for t, n in zip(cached, new))
        plan = PLAN_HEADER + CLUSTERS + 1 + (CLUSTERS + B * s_q) * PLAN_ITEM + B * s_q + 1
        return {"bytes": 4 * (2 * B + 2 * need + 2 * B + 2 + 2 * (sum(new) + 5) + plan + 2), "flops": 0}
    if op == "append":
        n = case["n"]
        return {"bytes": n * (ROW * 2 + FP4_ROW + ROW * 2) + 4 * (n + case["pad"]), "flops": 3 * n * D_C}
    row = ROW * 2 if case.get("cache", "fp4") == "bf16" else FP4_ROW
    if op == "summary":
        n = case["n"]
        return {"bytes": n * (PAGE * row + 4 + ROW * 4), "flops": n * ROW * PAGE}
    H, s_q = case["heads"], case["s_q"]
    N = case["B"] * s_q
    lens = _lens(case)
    io = N * H * (ROW + D_C) * 2
    if op == "attend":
        pairs = sum(T - s_q + 1 + i for T in lens for i in range(s_q))
        return {"bytes": sum(lens) * row + io, "flops": 2 * pairs * H * (ROW + D_C)}
    k = case["k"]
    pairs = scored = cells = keys = 0
    for T in lens:
        longest = 0
        for i in range(s_q):
            kv = T - s_q + 1 + i
            pages = (kv + PAGE - 1) // PAGE
            seen = (min(pages, k) - 1) * PAGE + kv - (pages - 1) * PAGE
            pairs += seen
            longest = max(longest, seen)
            if pages > k:
                scored += pages
        keys += longest
        if (T + PAGE - 1) // PAGE > k:
            cells += (T + PAGE - 1) // PAGE
    return {"bytes": keys * row + io + cells * (ROW + 4) + 8 * N * k,
            "flops": 2 * pairs * H * (ROW + D_C) + 2 * scored * H * ROW}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "tables":
        return _exact_tables(case, st)
    if op == "append":
        out = torch.zeros((case["n"] + case["pad"], ROW), dtype=torch.float64, device="cuda")
        n = case["n"]
        x = st["kv"][:n, :D_C].double().reshape(n, 16, GROUP)
        scale = (x.abs().max(dim=2, keepdim=True).values / 6).to(torch.float16).double()
        out[:n, :D_C] = (_nearest_fp4(x / scale.clamp(min=1e-30)) * scale).reshape(n, D_C).to(torch.bfloat16)
        out[:n, D_C:] = st["kv"][:n, D_C:]
        return out
    if op == "summary":
        pool = st["pool"]
        out = torch.empty((case["n"], ROW), dtype=torch.float64, device="cuda")
        for i in range(0, case["n"], 128):
            part = pool[i:i + 128]
            mean = (part.double() if case["cache"] == "bf16" else _wide(part)).mean(dim=1)
            top = mean.abs().max(dim=1, keepdim=True).values
            out[i:i + 128] = (mean / top * 127).round() * (top / 127).float().double()
        return out
    N, s_q = case["B"] * case["s_q"], case["s_q"]
    out = torch.empty((N, case["heads"], D_C), dtype=torch.float64, device="cuda")
    if op == "attend":
        for b, T in enumerate(st["lens_host"]):
            keys = _wide(st["pool"][st["table"][b, :-(-T // PAGE)].long()]).reshape(-1, ROW)
            for i in range(s_q):
                n = b * s_q + i
                out[n] = _exact_row(st["q_lat"][n], st["q_rope"][n], keys[:T - s_q + 1 + i])
        return out
    pages = torch.full((N, case["k"]), -1, dtype=torch.int32)
    lens = torch.zeros(N, dtype=torch.int32)
    for n in range(N):
        b, kv = n // s_q, st["lens_host"][n // s_q] - s_q + 1 + n % s_q
        count = -(-kv // PAGE)
        ids = st["table"][b, :count].long()
        chosen = list(range(count))
        if count > case["k"]:
            q = torch.cat([st["q_lat"][n], st["q_rope"][n]], 1).double()
            top = q.abs().max(dim=1, keepdim=True).values.clamp(min=1e-300)
            score = (q * 127 / top).round() @ st["codes"][ids].double().t() * (top / 127).float().double()
            score = (score.max(dim=0).values * st["scales"][ids].double()).float().tolist()
            middle = range(case["n_first"], count - case["n_recent"])
            best = sorted(middle, key=lambda p: (-score[p], p))[:case["k"] - case["n_first"] - case["n_recent"]]
            chosen = sorted(list(range(case["n_first"])) + best + list(range(count - case["n_recent"], count)))
        pages[n, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        lens[n] = len(chosen) * PAGE - (count * PAGE - kv)
        rows = st["pool"][ids[torch.tensor(chosen, device="cuda")]]
        keys = (rows.double() if case["cache"] == "bf16" else _wide(rows)).reshape(-1, ROW)
        out[n] = _exact_row(st["q_lat"][n], st["q_rope"][n], keys[:int(lens[n])])
    return pages.cuda(), lens.cuda(), out


def _nearest_fp4(x):
    """Nearest value of the 4-bit grid, ties to the value whose code is even."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    a = x.abs()
    up = torch.zeros_like(a)
    for i in range(7):
        border = (grid[i] + grid[i + 1]) / 2
        up += ((a > border) if i % 2 == 0 else (a >= border)).double() * (grid[i + 1] - grid[i])
    return up * x.sign()


def _wide(rows):
    """4-bit rows -> float64, byte by byte through a table of both nibbles."""
    v = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    both = torch.tensor([[v[i & 15], v[i >> 4]] for i in range(256)], dtype=torch.float64, device=rows.device)
    flat = rows.reshape(-1, FP4_ROW)
    c = both[flat[:, :256].int()].reshape(-1, 16, GROUP)
    c *= flat[:, 256:288].clone().view(torch.float16)[:, :, None]
    r = flat[:, 288:].clone().view(torch.bfloat16).double()
    return torch.cat([c.reshape(-1, D_C), r], 1).reshape(*rows.shape[:-1], ROW)


def _exact_row(q_lat, q_rope, keys):
    logit = (q_lat.double() @ keys[:, :D_C].t() + q_rope.double() @ keys[:, D_C:].t()) / math.sqrt(192.0)
    return torch.softmax(logit, dim=1) @ keys[:, :D_C]


def _exact_tables(case, st):
    """The same lists, made request by request."""
    B, s_q = case["B"], case["s_q"]
    table = st["table"].tolist()
    cached, new, free = st["cached"].tolist(), st["new"].tolist(), st["free"].tolist()
    head = int(st["head"])
    total, cu, slots, positions = [], [0], [], []
    for b in range(B):
        for page in range(-(-cached[b] // PAGE), -(-(cached[b] + new[b]) // PAGE)):
            table[b][page] = free[head]
            head += 1
        for t in range(cached[b], cached[b] + new[b]):
            slots.append(table[b][t // PAGE] * PAGE + t % PAGE)
            positions.append(t)
        total.append(cached[b] + new[b])
        cu.append(len(slots))
    slots += [-1] * (st["max_new"] - len(slots))
    positions += [-1] * (st["max_new"] - len(positions))
    groups = s_q if CLUSTERS >= s_q else 1
    per = CLUSTERS // groups
    pieces = []                                    # (cluster, row, first page, end page)
    for g in range(groups):
        rows = [n for n in range(B * s_q) if groups == 1 or n % s_q == g]
        kv = {n: total[n // s_q] - s_q + 1 + n % s_q for n in rows}
        line = sum(-(-kv[n] // PAGE) + PLAN_ITEM_COST for n in rows)
        at, c = 0, 0
        for n in rows:
            at += PLAN_ITEM_COST
            p, end = 0, -(-kv[n] // PAGE)
            while p < end:
                while (c + 1) * line // per <= at + p:
                    c += 1
                q = min(end, (c + 1) * line // per - at)
                pieces.append((g * per + c, n, p, q))
                p = q
            at += end
    parts = [0] * (B * s_q)
    for piece in pieces:
        parts[piece[1]] += 1
    slot_begin = [0]
    for m in parts:
        slot_begin.append(slot_begin[-1] + (m if m > 1 else 0))
    words = PLAN_HEADER + CLUSTERS + 1 + (CLUSTERS + B * s_q) * PLAN_ITEM + B * s_q + 1
    off_items = PLAN_HEADER + CLUSTERS + 1
    off_rows = off_items + len(pieces) * PLAN_ITEM
    plan = [PLAN_MAGIC, CLUSTERS, len(pieces), slot_begin[-1], B * s_q, case["heads"], s_q, B, PLAN_HEADER, off_items,
            off_rows, off_rows + B * s_q + 1, len(table[0]), 1, 0, 0]
    plan += [sum(1 for piece in pieces if piece[0] < c) for c in range(CLUSTERS + 1)]
    used = [0] * (B * s_q)
    for _, n, p, q in pieces:
        slot = slot_begin[n] + used[n] if parts[n] > 1 else -1
        used[n] += 1
        plan += [n // s_q, n % s_q, p, q, total[n // s_q] - s_q + 1 + n % s_q, slot, n, 0]
    plan += slot_begin
    plan += [0] * (words - len(plan))
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return dev(table), dev(total), dev(cu), dev(slots), dev(positions), dev([head]), dev(plan)
