"""Argument checks of the entry points that take the sizes of plan and workspaces (CPU)."""
import ctypes

import pytest

from head_latent_attention_04_b200 import mla

LIB = mla._lib
A = 0x1000          # aligned, never read: every call here is refused first
D = mla.make_dims(2, 1, 16, 4, 8)
PLAN = mla.plan_size(D, 74)[0]


def refused(code, what, *args):
    assert getattr(LIB, what)(*args) == code, (what, LIB.mla_last_error_string())
    assert LIB.mla_last_error_string()


def test_attention_arguments():
    good = [ctypes.byref(D), 2, A, A, A, A, A, None, A, PLAN, 74, A, 76 * 16 * 2048, A, 76 * 64, A, None, None, None]

    def bad(i, v, code=1):
        args = list(good)
        args[i] = v
        refused(code, "mla_decode_attn_sized", *args)
    for i in (2, 3, 4, 15):
        bad(i, None)
        bad(i, A + 8)
    for i in (5, 6, 8):
        bad(i, None)
        bad(i, A + 2)
    bad(1, 3)
    bad(1, -1)
    bad(7, A, 2)            # masks with a 4-bit cache
    bad(9, 4 * (16 + 75 + 2), 3)
    bad(10, 0)
    bad(10, 4097)
    bad(11, None)
    bad(11, A + 16)
    bad(13, None)
    bad(13, A + 2)
    bad(16, A + 2)
    bad(17, A + 2)
    args = list(good)
    args[1], args[7] = 0, A
    refused(1, "mla_decode_attn_sized", *args)      # masks with a causal plan


def test_combine_arguments():
    good = [ctypes.byref(D), A, PLAN, A, 76 * 16 * 2048, A, 76 * 64, A, None, None, None]

    def bad(i, v, code=1):
        args = list(good)
        args[i] = v
        refused(code, "mla_combine_sized", *args)
    bad(1, None)
    bad(1, A + 2)
    bad(2, 8, 3)
    bad(3, None)
    bad(3, A + 16)
    bad(5, None)
    bad(5, A + 2)
    bad(7, None)
    bad(8, A + 2)
    bad(9, A + 2)


def test_sizes_of_tensors_and_addresses():
    import torch
    plan = torch.zeros(100, dtype=torch.int32)
    assert mla._sizes(D, 74, plan, torch.zeros(3 * 16 * 512), torch.zeros(5, 16)) == (400, 3 * 16 * 2048, 320)
    assert mla._sizes(D, 74, plan, None, torch.zeros(5, 16)) == (400, 0, 320)
    assert mla._sizes(D, 74, A, A, A) == mla.plan_size(D, 74)
    assert mla._sizes(D, 74, plan, A, None) == (400, mla.plan_size(D, 74)[1], 0)


def test_a_tree_needs_its_masks():
    with pytest.raises(mla.MlaError, match="draft_masks"):
        mla.decode_attn_tree(D, A, A, A, A, A, None, A, 74, None, None, A)
