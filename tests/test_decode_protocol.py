"""The barrier protocol of the decode attention kernels, run as a model on the CPU.

A kernel's roles are warps that wait for and complete phases of shared-memory barriers.  A wait
names a parity only, so it is lost for good when its barrier moves on two phases before
the waiting warp looks: nothing may let one role lap another on a barrier.  The model
below has the roles of one pair of CTAs, page by page, with the barriers and conditions of
decode_attn.cu and decode_attn_fp4.cu (the barriers' counts are read from the sources), and
runs them in many orders, among them those that hold one role back as long as any other can move.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "head_latent_attention_04_b200", "csrc")
SOFT, STAGES_RAW, ITEMS = 2, 4, [3, 1, 7, 2, 9]        # softmax actors (of 8 warps), pages of each work item


def source(kernel):
    return open(os.path.join(CSRC, kernel + ".cu")).read()


def barriers_named(kernel, name):
    """Barriers that struct Bars holds under a name (an array's length, 1 for a single one)."""
    bars = source(kernel).split("struct Bars {")[1].split("};")[0]
    m = re.search(rf"\b{name}(?:\[(\w+)\])?\s*[,;]", re.sub(r"//.*", "", bars))
    return int(m.group(1)) if m.group(1) else 1


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, "an arrival too many"
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Cta:
    def __init__(self, stages, p_full):
        self.kv_full = [Bar(1) for _ in range(stages)]
        self.kv_empty = [Bar(1) for _ in range(stages)]
        self.raw_full = [Bar(1) for _ in range(STAGES_RAW)]
        self.raw_empty = [Bar(1) for _ in range(STAGES_RAW)]
        self.q_full, self.q_empty, self.s_full, self.s_read, self.own_full = (Bar(1) for _ in range(5))
        self.own_free, self.x_recv, self.x_sendok = Bar(SOFT + 1), Bar(1), Bar(SOFT)
        self.p_full = [Bar(SOFT) for _ in range(p_full)]
        self.o_full = [Bar(1) for _ in range(2)]
        self.o_done, self.o_free = Bar(1), Bar(SOFT)
        self.scores = None      # page whose partial scores S, the own tile and the peer tile hold
        self.p = [None, None]   # page whose P the buffer holds
        self.peer_tile = None


def roles(me, peer, stages, widens, rescales):
    """Generators that yield the (barrier, parity) they wait for."""
    pages = [(it, j, n) for it, n in enumerate(ITEMS) for j in range(n)]
    total = len(pages)

    def tma():
        ring, empty, k = (me.raw_full, me.raw_empty, STAGES_RAW) if widens else (me.kv_full, me.kv_empty, stages)
        for g in range(total):
            if g >= k:
                yield empty[g % k], (g // k - 1) & 1
            ring[g % k].arrive()

    def sender():
        widened = 0
        for g, (it, j, n) in enumerate(pages):
            if j == 0:
                if it > 0:
                    yield me.q_empty, (it - 1) & 1
                me.q_full.arrive()
            while widens and widened < min(g + 2, total):
                yield me.raw_full[widened % STAGES_RAW], (widened // STAGES_RAW) & 1
                if widened >= stages:
                    yield me.kv_empty[widened % stages], (widened // stages - 1) & 1
                me.kv_full[widened % stages].arrive()
                widened += 1
            yield me.s_full, g & 1
            me.s_read.arrive()
            if g >= 1:
                yield me.own_free, (g - 1) & 1
            me.own_full.arrive()

    def qk():
        for g, (it, j, n) in enumerate(pages):
            if j == 0:
                yield me.q_full, it & 1
            yield me.kv_full[g % stages], (g // stages) & 1
            if g > 0:
                yield me.s_read, (g - 1) & 1
            me.s_full.arrive()
            if widens:
                me.raw_empty[g % STAGES_RAW].arrive()
            if j == n - 1:
                me.q_empty.arrive()

    def copy():
        for g in range(total):
            if g >= 1:
                yield me.x_sendok, (g - 1) & 1
            yield me.own_full, g & 1
            peer.peer_tile = g
            peer.x_recv.arrive()
            me.own_free.arrive()

    def softmax():
        for g, (it, j, n) in enumerate(pages):
            if g >= 2:
                yield me.o_full[g & 1], ((g >> 1) - 1) & 1
            yield me.own_full, g & 1
            me.own_free.arrive()
            yield me.x_recv, g & 1
            assert me.peer_tile == g
            peer.x_sendok.arrive()
            if rescales and j > 0:                        # O is rescaled: the product before must be complete
                yield me.o_full[(g - 1) & 1], ((g - 1) >> 1) & 1
            me.p[g & 1] = g
            k = len(me.p_full)
            me.p_full[g % k].arrive()
            if j == n - 1:
                yield me.o_done, it & 1
                me.o_free.arrive()

    def pv():
        k = len(me.p_full)
        for g, (it, j, n) in enumerate(pages):
            yield me.p_full[g % k], (g // k) & 1
            assert me.p[g & 1] == g
            if j == 0 and it > 0:
                yield me.o_free, (it - 1) & 1
            me.kv_empty[g % stages].arrive()
            me.o_full[g & 1].arrive()
            if j == n - 1:
                me.o_done.arrive()

    return [("tma", tma()), ("sender", sender()), ("qk", qk()), ("copy", copy()), ("pv", pv())] + \
           [("softmax", softmax()) for _ in range(SOFT)]


def finishes(stages, widens, p_full, pick, rescales=False):
    """Runs the pair; pick(ready, who) chooses the next role among those that can move.  Whether O is
    rescaled depends on the data."""
    ctas = [Cta(stages, p_full) for _ in range(2)]
    actors = [(c, name, gen) for c in range(2) for name, gen in roles(ctas[c], ctas[1 - c], stages, widens, rescales)]
    waits = {}
    for i, (_, _, gen) in enumerate(actors):
        waits[i] = next(gen, None)
    while any(w is not None for w in waits.values()):
        ready = [i for i, w in waits.items() if w is not None and w[0].done(w[1])]
        if not ready:
            return False
        i = pick(ready, actors)
        waits[i] = next(actors[i][2], None)
    return True


def last(cta, name):
    """The role is held back while any other can move."""
    return lambda ready, actors: min(ready, key=lambda i: ((actors[i][0], actors[i][1]) == (cta, name), i))


KERNELS = [("decode_attn", 5, False), ("decode_attn", 5, True), ("decode_attn_fp4", 4, True)]


@pytest.mark.parametrize("kernel,stages,widens", KERNELS)
def test_no_role_laps_another(kernel, stages, widens):
    assert barriers_named(kernel, "o_full") == 2
    p_full = barriers_named(kernel, "p_full")
    for cta in range(2):
        for name in ("tma", "sender", "qk", "copy", "pv", "softmax"):
            for rescales in (False, True):
                assert finishes(stages, widens, p_full, last(cta, name), rescales), (cta, name)
    for seed in range(200):
        rng = random.Random(seed)
        assert finishes(stages, widens, p_full, lambda ready, _: rng.choice(ready), seed % 4 == 0), seed


def test_the_model_sees_a_lapped_barrier():
    """One barrier for both P buffers: the softmax can complete two phases of it before the
    product's issuer looks, whose wait then never ends."""
    assert not finishes(4, True, 1, last(0, "pv"))
    assert finishes(4, True, 2, last(0, "pv"))


@pytest.mark.parametrize("kernel", ["decode_attn", "decode_attn_fp4"])
def test_the_peer_tile_is_read_before_it_is_refilled(kernel):
    """The arrive that lets the peer copy into this CTA's tile depends on what every lane read there
    (an empty asm statement is no instruction and orders nothing), and the thread that copies
    acquires it at cluster scope."""
    text = " ".join(re.sub(r"//.*", "", source(kernel)).split())
    assert "const uint32_t read = (pr[0].x ^ pr[1].x ^ pr[2].x ^ pr[3].x) & p.zero; " \
           "const uint32_t ok_addr = x_sendok_peer + __ballot_sync(0xffffffffu, read != 0);" in text
    assert text.count("mbar_arrive_relaxed_cluster(") == text.count("mbar_arrive_relaxed_cluster(ok_addr)") == 1
    assert text.count("mbar_wait<true, kWaitHintNs>(&bars->x_sendok") == 1
    assert "mbar_wait<false, kWaitHintNs>(&bars->x_sendok" not in text


@pytest.mark.parametrize("kernel", ["decode_attn", "decode_attn_fp4"])
def test_tensor_memory_is_written_behind_a_fence(kernel):
    """A wait for the products that read a tensor-memory operand orders this thread's next stores into it
    only together with tcgen05.fence::after_thread_sync."""
    text = " ".join(re.sub(r"//.*", "", source(kernel)).split())
    q = text.split("warp_wait(&bars->q_empty, (ii - 1) & 1, wc)) goto sender_fail;")[1]
    assert "tc_fence_after();" in q[:q.index("tmem_st32(")]
    p = text.split("warp_wait(&bars->o_full[gj & 1], ((gj >> 1) - 1) & 1, wc)) goto softmax_fail;")[1]
    p = p[:p.index("tmem + lane_addr + kTmemP")]
    rescale = p[p.index("if (__any_sync(0xffffffffu, move && j > 0)) {"):]
    depth, end = 0, 0
    for end, ch in enumerate(rescale):                       # the block that rescales O has a fence of its own
        depth += (ch == "{") - (ch == "}")
        if ch == "}" and depth == 0:
            break
    assert "tc_fence_after();" in p.replace(rescale[:end + 1], "")
