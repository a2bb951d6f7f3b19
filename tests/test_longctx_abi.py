"""Argument checks of the long-context entry points (CPU): nothing invalid reaches a launch."""
import ctypes

import pytest
import torch

from head_latent_attention_04_b200 import mla

LIB = mla._lib
A = 0x1000          # a 16-byte aligned address that is never read: every call here is refused first
OK = dict(B=2, s_q=1, n_heads=16, max_blocks=4, num_blocks=8)


def dims(**kw):
    d = mla.make_dims(**{**OK, **{k: v for k, v in kw.items() if k in OK}})
    for k, v in kw.items():
        if k not in OK:
            setattr(d, k, v)
    return d


def refused(code, what, *args):
    got = getattr(LIB, what)(*args)
    assert got == code, (what, got, LIB.mla_last_error_string())
    assert LIB.mla_last_error_string()


@pytest.mark.parametrize("fn", ["mla_kv_quantize_fp4", "mla_kv_dequantize_fp4"])
def test_fp4_row_arguments(fn):
    refused(1, fn, A, A, -1, A, 8, None, None)
    refused(1, fn, A, A, 4, A, 0, None, None)
    refused(2, fn, A, A, 4, A, 1 << 26, None, None)
    refused(1, fn, None, A, 4, A, 8, None, None)
    refused(1, fn, A + 8, A, 4, A, 8, None, None)
    refused(1, fn, A, None, 4, A, 8, None, None)
    refused(1, fn, A, A + 2, 4, A, 8, None, None)
    refused(1, fn, A, A, 4, A + 4, 8, None, None)
    refused(1, fn, A, A, 4, A, 8, A + 1, None)
    assert getattr(LIB, fn)(None, None, 0, None, 8, None, None) == 0      # no rows: nothing to do


def test_fp4_attention_arguments():
    def call(d=dims(), ptrs=(A,) * 6, clusters=74, o_part=A, lse_part=A, o_lat=A, lse=None, status=None):
        return (ctypes.byref(d), *ptrs, clusters, o_part, lse_part, o_lat, lse, status, None)
    for i in range(6):
        for bad in (None, A + 2):
            refused(1, "mla_decode_attn_fp4cache", *call(ptrs=tuple(bad if j == i else A for j in range(6))))
    refused(1, "mla_decode_attn_fp4cache", *call(clusters=0))
    refused(1, "mla_decode_attn_fp4cache", *call(o_part=A + 16))
    refused(1, "mla_decode_attn_fp4cache", *call(o_lat=None))
    refused(1, "mla_decode_attn_fp4cache", *call(lse=A + 2))
    refused(2, "mla_decode_attn_fp4cache", *call(d=dims(d_c=256)))
    refused(2, "mla_decode_attn_fp4cache", *call(d=dims(n_heads=129)))
    refused(2, "mla_decode_attn_fp4cache", *call(d=dims(s_q=9)))


def test_build_tables_arguments():
    good = [2, A, A, 4, A, A, 8, A, 8, 16, A, A, A, A, A, None, None]
    def bad(i, v, code=1):
        args = list(good)
        args[i] = v
        refused(code, "mla_build_tables", *args)
    for i in (0, 3, 8):
        bad(i, 0)
    for i in (6, 9):
        bad(i, -1)
    bad(0, 65537, 2)
    bad(3, 1 << 25, 2)
    bad(9, (1 << 30) + 1, 2)
    bad(8, 1 << 26, 2)
    for i in (1, 2, 4, 5, 7, 10, 11, 12, 14):
        bad(i, None)
        bad(i, A + 1)
    bad(13, A + 2)      # positions may be NULL, not misaligned


def test_plan_device_arguments():
    d = dims()
    need = mla.plan_size(d, 74)[0]
    refused(1, "mla_plan_device", ctypes.byref(d), None, 74, A, need, None, None)
    refused(1, "mla_plan_device", ctypes.byref(d), A, 74, A + 2, need, None, None)
    refused(1, "mla_plan_device", ctypes.byref(d), A, 0, A, need, None, None)
    refused(1, "mla_plan_device", ctypes.byref(d), A, 4097, A, need, None, None)
    refused(3, "mla_plan_device", ctypes.byref(d), A, 74, A, need - 4, None, None)
    refused(2, "mla_plan_device", ctypes.byref(dims(max_blocks=1 << 25)), A, 74, A, 1 << 20, None, None)


def test_summary_and_selection_arguments():
    refused(1, "mla_summarize_pages", A, 3, A, 2, 8, A, A, None, None)
    refused(1, "mla_summarize_pages", A, 0, A, -1, 8, A, A, None, None)
    refused(1, "mla_summarize_pages", A, 0, A, 2, 8, A + 8, A, None, None)
    refused(1, "mla_summarize_pages", A, 0, A, 2, 8, A, None, None, None)
    d = dims()
    good = [ctypes.byref(d), A, A, A, A, A, A, 3, 1, 1, A, A, A, A, 74, A, 1 << 20, None, None]
    def bad(i, v, code=1):
        args = list(good)
        args[i] = v
        refused(code, "mla_select_pages", *args)
    for i in (1, 2, 3, 4, 5, 6, 10, 11, 12):
        bad(i, None)
        bad(i, A + 2)
    bad(13, A + 2)
    bad(7, 0)
    bad(7, 1)           # fewer than the first and the recent pages
    bad(7, 1 << 26, 2)
    bad(8, -1)
    bad(9, 0)
    bad(14, 0)
    bad(14, 4097)
    bad(15, A + 2)
    bad(16, 64, 3)


def test_python_side_refuses_types_shapes_and_devices():
    cpu = torch.zeros((4, 576), dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros((2, 64, 416), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        mla.kv_quantize_fp4(cpu, slots, pool)
    with pytest.raises(ValueError, match="kv_cache"):
        mla.summarize_pages(pool, slots, None, None, kv_cache="int4")
    with pytest.raises(ValueError, match="n_recent"):
        mla.SparseAttention(1, 1, 16, 4, 8, k=2, n_first=1, n_recent=2)
    with pytest.raises(ValueError, match="kv_cache"):
        mla.Decoder([64], 1, 16, 1, 1, kv_cache="fp6")
    with pytest.raises(ValueError, match="expected torch.int32"):
        mla._arg(slots.long(), "slots", torch.int32, 4)
    with pytest.raises(ValueError, match="shape"):
        mla._arg(slots, "slots", torch.int32, 5)
    with pytest.raises(ValueError, match="shape"):
        mla._arg(slots, "slots", torch.int32, 4, None)
