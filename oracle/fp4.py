"""The 4-bit latent cache row, page summaries and page selection -- TEST INFRASTRUCTURE ONLY.

Written from the definitions in float64; it shares no code with the CUDA path.

A 4-bit row keeps c_KV in groups of 32 columns with one fp16 scale s = fp16(amax / 6)
and E2M1 codes of c / s (values 0, .5, 1, 1.5, 2, 3, 4, 6 and negatives; nearest, ties
to the even code, saturated at 6), column 2i in the low nibble of byte i.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GROUP, ROW, ROW_BYTES, PAGE = 32, 576, 416, 64


def e2m1_codes(x) -> np.ndarray:
    """Codes 0..15 of the nearest grid values, ties to the even code."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    code = np.zeros(a.shape, dtype=np.uint8)
    for i in range(7):
        border = (GRID[i] + GRID[i + 1]) / 2
        code += (a > border) if i % 2 == 0 else (a >= border)    # a tie goes to the even one of i, i + 1
    return code | (np.signbit(x).astype(np.uint8) << 3)


def e2m1_values(codes) -> np.ndarray:
    codes = np.asarray(codes)
    return np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]


def quantize(rows):
    """float rows [n][512] -> (codes uint8 [n][512], scales float16 [n][16])."""
    x = np.asarray(rows, dtype=np.float64).reshape(len(rows), 16, GROUP)
    scales = (np.abs(x).max(-1) / 6.0).astype(np.float16)
    s = scales.astype(np.float64)[..., None]
    q = np.divide(x, s, out=np.zeros_like(x), where=s > 0)
    return e2m1_codes(np.copysign(np.abs(q), x)).reshape(len(rows), 512), scales


def pack(codes, scales, rope_bytes) -> np.ndarray:
    """Codes [n][512], scales float16 [n][16], k_rope as bytes [n][128] -> uint8 [n][416]."""
    out = np.empty((len(codes), ROW_BYTES), dtype=np.uint8)
    out[:, :256] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    out[:, 256:288] = np.ascontiguousarray(scales).view(np.uint8)
    out[:, 288:] = rope_bytes
    return out


def unpack(rows):
    """uint8 [n][416] -> (codes [n][512], scales float16 [n][16])."""
    rows = np.ascontiguousarray(rows)
    codes = np.empty((len(rows), 512), dtype=np.uint8)
    codes[:, 0::2], codes[:, 1::2] = rows[:, :256] & 15, rows[:, :256] >> 4
    return codes, rows[:, 256:288].copy().view(np.float16)


def bf16_from_bytes(b) -> np.ndarray:
    """bf16 as bytes [..., 2k] -> float64 [..., k]."""
    u = np.ascontiguousarray(b).view(np.uint16).astype(np.uint32) << 16
    return u.view(np.float32).astype(np.float64)


def dequantize_rows(rows) -> np.ndarray:
    """uint8 [n][416] -> float64 [n][576]."""
    codes, scales = unpack(rows)
    c = e2m1_values(codes).reshape(len(codes), 16, GROUP) * scales.astype(np.float64)[..., None]
    return np.concatenate([c.reshape(len(codes), 512), bf16_from_bytes(rows[:, 288:])], axis=1)


def code8(x):
    """The 8-bit form of vectors [..., 576]: codes rint(127 x / amax) and scales fp32(amax / 127)."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.abs(x).max(-1, keepdims=True)
    codes = np.rint(np.divide(127.0 * x, amax, out=np.zeros_like(x), where=amax > 0))
    return codes, (amax[..., 0] / 127.0).astype(np.float32)


def select(q, pcodes, pscales, kv_len, k, n_first, n_recent):
    """Pages of one query row: q float [h][576], the summaries of its pages in order."""
    count = -(-kv_len // PAGE)
    if count <= k:
        return list(range(count))
    qc, qs = code8(q)
    dot = qc @ np.asarray(pcodes[:count], dtype=np.float64).T
    score = (dot * qs.astype(np.float64)[:, None]).max(0) * np.asarray(pscales[:count], dtype=np.float64)
    score = score.astype(np.float32)
    middle = sorted(range(n_first, count - n_recent), key=lambda p: (-score[p], p))
    return sorted(list(range(n_first)) + middle[:k - n_first - n_recent] + list(range(count - n_recent, count)))


def build_tables(cached, new, table, free, head, max_new, held_pages=None):
    """Request by request; returns (table, seq_lens, cu_new, slots, positions, head, no_space).
    ``held_pages`` (a list, updated): pages whose blocks the rows hold, at least those of the cached tokens."""
    table = [list(r) for r in table]
    width = len(table[0])
    lens, cu, slots, pos = [], [0], [], []
    no_space = False
    if head < 0 or head > len(free):
        head, no_space = len(free), True
    pages_asked, tokens_asked, start = 0, 0, head
    for b, (c, n) in enumerate(zip(cached, new)):
        in_row = held_pages[b] if held_pages else 0
        valid = c >= 0 and n >= 0 and c + n <= width * PAGE and in_row <= width
        admitted = valid
        if valid:
            held = max(in_row, -(-c // PAGE))
            need = max(-(-(c + n) // PAGE) - held, 0)
            pages_asked += need
            admitted = need == 0 or start + pages_asked <= len(free)
            if admitted:                       # a request refused for its blocks asks for no room in the slot map
                tokens_asked += n
                admitted = n == 0 or tokens_asked <= max_new
        if not admitted:
            no_space = True
            lens.append(max(c, 0))
        else:
            for j in range(need):
                table[b][held + j] = free[head]
                head += 1
            if held_pages:
                held_pages[b] = held + need
            for t in range(c, c + n):
                slots.append(table[b][t // PAGE] * PAGE + t % PAGE)
                pos.append(t)
            lens.append(c + n)
        cu.append(len(slots))
    pad = [-1] * (max_new - len(slots))
    return table, lens, cu, slots + pad, pos + pad, head, no_space
