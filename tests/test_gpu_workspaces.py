"""A plan that needs more than its buffers hold is refused on the device, by every decode kernel and by
the merge, and nothing is written."""
import numpy as np
import pytest
import torch

from head_latent_attention_04_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_04_b200 import mla as m
    return m


class Setup:
    def __init__(self, mla, kind):
        self.w = w = W.make_workload(1, 2, 16, [3000], seed=3, pool="permuted")
        pool = w.kv_pool.to(DEV)
        self.kind = kind
        self.pool = {"fp8": mla.fp8_pool_from, "fp4": mla.fp4_pool_from}.get(kind, lambda p: p)(pool)
        self.dec = mla.Decoder(w.seq_lens, 2, 16, w.max_blocks, w.num_blocks, DEV, causal=kind != "tree",
                               kv_cache=kind if kind in ("fp8", "fp4") else "bf16")
        assert self.dec.num_slots > 2
        self.table = torch.as_tensor(w.block_table, dtype=torch.int32, device=DEV)
        g = torch.Generator().manual_seed(1)
        self.q = torch.randn((2, 16, 512), generator=g).to(torch.bfloat16).to(DEV)
        self.r = torch.randn((2, 16, 64), generator=g).to(torch.bfloat16).to(DEV)
        self.fn = {"bf16": mla.decode_attn, "fp8": mla.decode_attn_fp8cache, "fp4": mla.decode_attn_fp4cache,
                   "tree": mla.decode_attn_tree}[kind]
        self.masks = (torch.tensor([[1, 3]], dtype=torch.int32, device=DEV),) if kind == "tree" else ()

    def run(self, o_part, lse_part, plan=None, out=None):
        d = self.dec
        out = torch.full_like(self.q, 7.0) if out is None else out
        d.status.zero_()
        self.fn(d.dims, self.q, self.r, self.pool, self.table, d.seq_lens_dev, *self.masks,
                d.plan_dev if plan is None else plan, d.num_clusters, o_part, lse_part, out, status=d.status)
        return d.status.item(), out


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4", "tree"])
def test_attention_refuses_a_plan_that_needs_more(mla, kind):
    s = Setup(mla, kind)
    d, n = s.dec, s.dec.num_slots
    room = torch.full((n * 16 * 512 + 4096,), 5.0, device=DEV)
    lse = torch.full((n * 16 + 64,), 5.0, device=DEV)
    full, full_lse = room[:n * 16 * 512], lse[:n * 16]
    for o_part, lse_part in ((None, None), (full, None), (None, full_lse), (full[:-16 * 512], full_lse),
                             (full, full_lse[:-1])):
        status, out = s.run(o_part, lse_part)
        assert status == mla.STATUS_BAD_PLAN and torch.all(out == 7.0)
        assert torch.all(room == 5.0) and torch.all(lse == 5.0)
    words = int(d.plan_host[11])                       # the plan's own length: a buffer of just that will do
    status, _ = s.run(full, full_lse, plan=d.plan_dev[:words - 1].clone())
    assert status == mla.STATUS_BAD_PLAN and torch.all(room == 5.0)
    status, out = s.run(full, full_lse, plan=d.plan_dev[:words].clone())
    assert status == 0 and torch.all(room[full.numel():] == 5.0) and torch.all(lse[full_lse.numel():] == 5.0)
    assert not torch.any(full_lse == 5.0)


def test_merge_refuses_what_the_attention_refuses(mla):
    s = Setup(mla, "bf16")
    d, n = s.dec, s.dec.num_slots
    status, out = s.run(d.o_part, d.lse_part)
    assert status == 0 and torch.all(out == 7.0)      # both rows are split: the merge writes them
    args = d.dims, d.plan_dev
    for o_part, lse_part in ((d.o_part[:-16 * 512], d.lse_part), (d.o_part, d.lse_part[:-1])):
        mla.combine(*args, o_part, lse_part, out, status=d.status)
        assert d.status.item() == mla.STATUS_BAD_PLAN and torch.all(out == 7.0)
        d.status.zero_()
    bad = d.plan_dev.clone()
    for word, value in ((0, 0), (4, 3), (5, 17)):     # no plan, other rows, other heads
        bad.copy_(d.plan_dev)
        bad[word] = value
        mla.combine(d.dims, bad, d.o_part, d.lse_part, out, status=d.status)
        assert d.status.item() == mla.STATUS_BAD_PLAN and torch.all(out == 7.0)
        d.status.zero_()
    mla.combine(*args, d.o_part, d.lse_part, out, status=d.status)
    assert d.status.item() == 0 and not torch.any(out == 7.0)
    with pytest.raises(mla.MlaError):
        mla.combine(*args, None, d.lse_part, out)


def test_plans_of_the_device_with_small_workspaces(mla):
    """The host does not see the slots of a plan made on the device: the check is the kernel's."""
    s = Setup(mla, "fp4")
    d = s.dec
    plan = mla.plan_device(d.dims, d.seq_lens_dev, d.num_clusters)
    np.testing.assert_array_equal(plan.cpu().numpy(), d.plan_host)
    status, out = s.run(d.o_part[:2 * 16 * 512], d.lse_part[:2], plan=plan)
    assert status == mla.STATUS_BAD_PLAN and torch.all(out == 7.0)
    status, out = s.run(d.o_part, d.lse_part, plan=plan)
    assert status == 0
