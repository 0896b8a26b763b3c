"""The query side of a step in float64 numpy: pages, FP8 rows and their product, rotary positions, drafted trees.

Test infrastructure only (see ``oracle/__init__.py``).  These operators are not on the pages; the readings are
R17 to R21 of include/csa2.h.
"""
from __future__ import annotations

import math

import numpy as np

from . import formats

PAGE = 64
BLOCK = 128


# ---- R17: pages ---------------------------------------------------------------------------------

def page_plan(seq_len, n_new, held, table, free, n_free, shift=None, Tq=None, max_new=None):
    """One sequence after the other, pages one by one.  Returns a dict of the arrays after the call and the
    sequences whose state is impossible."""
    B, max_pages = table.shape
    n_pages = len(free)
    seq_len, n_new, held = (np.array(x, dtype=np.int64) for x in (seq_len, n_new, held))
    shift = np.zeros(B, dtype=np.int64) if shift is None else np.array(shift, dtype=np.int64)
    table, free = np.array(table, dtype=np.int64), np.array(free, dtype=np.int64)
    out = {"seq_len": seq_len.copy(), "held": held.copy(), "table": table, "free": free, "n_free": n_free,
           "n_entries": np.zeros(B, dtype=np.int64), "first_entry": np.zeros(B, dtype=np.int64),
           "granted": np.zeros(B, dtype=np.int64), "bad": []}
    if Tq is not None:
        out["q_pos"] = np.full((B, Tq), -1, dtype=np.int64)
    if max_new is not None:
        out["slots"] = np.full((B, max_new), -1, dtype=np.int64)
    e0 = np.array([math.floor(n / 4) for n in seq_len]) - shift
    e1 = np.array([math.floor(n / 4) for n in seq_len + n_new]) - shift
    need = np.array([math.ceil(max(e, 0) / PAGE) for e in e1])
    for b in range(B):
        ok = (0 <= seq_len[b] and 0 <= seq_len[b] + n_new[b] < 2 ** 31 and shift[b] >= 0 and e0[b] >= 0 and e1[b] >= 0
              and 0 <= held[b] <= max_pages and math.ceil(e0[b] / PAGE) <= held[b] and need[b] <= max_pages
              and (Tq is None or n_new[b] <= Tq) and (max_new is None or e1[b] - e0[b] <= max_new))
        if not ok:
            out["bad"].append(b)
    good = [b for b in range(B) if b not in set(out["bad"])]
    out["n_entries"][:] = np.maximum(e0, 0)
    out["first_entry"][:] = np.maximum(e0, 0)
    stack = free[:max(0, min(n_free, n_pages))].tolist()
    back = [(b, p) for b in good for p in range(need[b], held[b])]
    if not 0 <= n_free <= n_pages or n_free + len(back) > n_pages:
        out["bad"] = "pool"
        return out
    stack += [int(table[b, p]) for b, p in back]
    room = len(stack)
    for b in good:
        want = max(0, need[b] - held[b])
        room -= want
        if want and room < 0:
            continue                          # waits, and so does everybody behind that needs pages
        for p in range(held[b], need[b]):
            table[b, p] = stack.pop()
        out["granted"][b], out["held"][b], out["seq_len"][b] = 1, need[b], seq_len[b] + n_new[b]
        out["n_entries"][b], out["first_entry"][b] = e1[b], min(e0[b], e1[b])
        if Tq is not None:
            for i in range(max(0, n_new[b])):
                out["q_pos"][b, i] = seq_len[b] + i
        if max_new is not None:
            for e in range(e0[b], e1[b]):
                page = table[b, e // PAGE]
                out["slots"][b, e - e0[b]] = page * PAGE + e % PAGE if 0 <= page < n_pages else -1
    free[:len(stack)] = stack
    out["n_free"] = len(stack)
    return out


# ---- R18, R19: FP8 rows and their product ---------------------------------------------------------

def pack_fp8_blocks(x):
    """x [n][K] fp32 values -> codes uint8 [n][K], scales fp32 [n][ceil(K/128)]."""
    x = np.asarray(x, dtype=np.float32)
    n, K = x.shape
    kb = -(-K // BLOCK)
    codes, scales = np.zeros((n, K), dtype=np.uint8), np.zeros((n, kb), dtype=np.float32)
    for k in range(kb):
        blk = x[:, BLOCK * k:BLOCK * (k + 1)]
        a = np.maximum(np.abs(blk).max(axis=1), np.float32(2.0 ** -100))
        scales[:, k] = a / np.float32(448)
        q = blk * (np.float32(448) / a)[:, None]
        codes[:, BLOCK * k:BLOCK * (k + 1)] = formats.e4m3_encode_array(q)
    return codes, scales


def unpack_fp8_blocks(codes, scales, rows_per_scale=1):
    """float64 values; a scale serves rows_per_scale rows (128 for weights)."""
    n, K = codes.shape
    s = np.asarray(scales, dtype=np.float64)[np.arange(n) // rows_per_scale][:, np.arange(K) // BLOCK]
    return formats.E4M3_TABLE[codes] * s


def matmul_fp8(a, sa, b, sb):
    """C and the sum of the products' magnitudes."""
    A, W = unpack_fp8_blocks(a, sa), unpack_fp8_blocks(b, sb, BLOCK)
    return A @ W.T, np.abs(A) @ np.abs(W).T


# ---- R20: rotary positions --------------------------------------------------------------------------

def rope_frequencies(r, base=10000.0, scaling="none", factor=1.0, original=4096, beta_fast=32.0, beta_slow=1.0):
    theta = []
    for i in range(r // 2):
        b = base * factor ** (r / (r - 2)) if scaling == "ntk" else base
        t = 1.0 / b ** (2.0 * i / r)
        if scaling == "linear":
            t = t / factor
        if scaling == "yarn":
            turns = lambda n: r * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(0, math.floor(turns(beta_fast))), min(r - 1, math.ceil(turns(beta_slow)))
            g = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            t = t * (1 - g) + t / factor * g
        theta.append(t)
    return np.array(theta)


def rope(x, positions, theta, start=0, layout="half", inverse=False, amplitude=1.0):
    """x [n][heads][d]: the pairs as complex numbers times amplitude e^(+-i p theta)."""
    x = np.array(x, dtype=np.float64)
    half = len(theta)
    turn = amplitude * np.exp((-1j if inverse else 1j) * np.asarray(positions, dtype=np.float64)[:, None] * theta[None, :])
    i1 = start + (np.arange(half) if layout == "half" else 2 * np.arange(half))
    i2 = i1 + (half if layout == "half" else 1)
    z = (x[:, :, i1] + 1j * x[:, :, i2]) * turn[:, None, :]
    x[:, :, i1], x[:, :, i2] = z.real, z.imag
    return x


# ---- R21: drafted trees -----------------------------------------------------------------------------

def tree_plan(parent, ctx_len, max_depth):
    """q_pos, path and whether a place's data is impossible (index, count)."""
    B, T = parent.shape
    q_pos, path = np.full((B, T), -1, dtype=np.int64), np.full((B, T, max_depth), -1, dtype=np.int64)
    bad_index = bad_count = False
    for b in range(B):
        lines = {}
        bad_count |= ctx_len[b] < 0
        for i in range(T):
            p = parent[b, i]
            if p >= i:
                bad_index = True
                continue
            if p < -1:
                continue
            if p >= 0 and p not in lines:
                bad_index = True
                continue
            lines[i] = (lines[p] if p >= 0 else []) + [i]
            if ctx_len[b] < 0:
                continue
            if len(lines[i]) > max_depth or ctx_len[b] + len(lines[i]) - 1 >= 2 ** 31:
                bad_count = True
                continue
            q_pos[b, i] = ctx_len[b] + len(lines[i]) - 1
            path[b, i, :len(lines[i])] = lines[i]
    return q_pos, path, bad_index, bad_count


def tree_window(t, W, ctx, pos0, cap, line):
    """Window rows of the node whose path is `line`: committed rows (places in the buffer) and nodes."""
    old, new = [], []
    for p in range(max(0, t - W + 1), t + 1):
        if p >= ctx:
            new.append(line[p - ctx])
        elif 0 <= p - pos0 < cap:
            old.append(p - pos0)
    return old, new


def attention(Q, keys, tau):
    """Q [H][d], keys [n][d] -> O, lse, sum of p |v|, and the largest sum |q k| tau of each head."""
    H, d = Q.shape
    if len(keys) == 0:
        return np.zeros((H, d)), np.full(H, -np.inf), np.zeros((H, d)), np.zeros(H)
    x = Q @ keys.T * tau
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - m)
    l = e.sum(axis=1, keepdims=True)
    return e @ keys / l, (m + np.log(l))[:, 0], e @ np.abs(keys) / l, (np.abs(Q) @ np.abs(keys).T * abs(tau)).max(axis=1)
