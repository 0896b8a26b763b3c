"""Small caches with known rows, and the error bounds of the whole-cache kernels.

A case holds packed rows in randomly permuted pages of a shared pool in which
everything that no sequence owns is poisoned: spare slots and pages hold the
E4M3 NaN scale, window rows outside the buffer's valid part hold NaN scales,
weights of foreign slots a sentinel.  Expected values come from oracle.bounded on
the dequantised operands, in float64.

Bounds (u16 = 2^-11, one rounding of P to fp16; ub = 2^-8, half a bf16 step):
* a logit's error: the fp32 dot product of exact products, kappa * tau * |q|.|k|
  with kappa = 2^-20 (the bound this suite uses for its other fp32 contractions),
  plus 2^-21 of the logit's own terms (scale, cap, bias and their sum: at most
  eight fp32 roundings, each 2^-24 of the largest term);
* lse: the largest logit error, 2^-20 for exp2, log2 and the sum of positive
  terms, and 2^-23 |lse|;
* O: ub |o| for its rounding, plus for every key p_j |v_j| (u16 + 2 logit errors +
  2^-20), plus 2^-25 * 2^8 |v_j| / l for a P below fp16's normal range (the
  reference maximum may lie up to 2^8 below the largest term, never above it, so
  l >= 1 in its units and the absolute step is at most 2^-25);
* weights: every term's relative error, logit error + 2^-22 (|l| + |lse|) + 2^-20,
  times the term, plus 2^-23 of the result.
"""
import math

import numpy as np
import torch

from compressed_sparse_attention_05_gb300 import abi
from oracle import bounded as OB
from oracle import formats as F

SENTINEL = 12345.0


class Case:
    def __init__(self, seed=0, B=1, Tq=1, Hq=64, d=512, lens=(100,), W=128, cap=0.0, slopes=None, docs=None,
                 prefix=None, shift=None, scrambled=False, q_pos=None, q_scale=1.0, window=True, swa_slack=3,
                 max_entries=None, tau=None, k_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.Tq, self.Hq, self.d, self.W, self.cap = B, Tq, Hq, d, W, cap
        self.lens = [lens[b % len(lens)] for b in range(B)]
        self.tau = 1.0 / math.sqrt(d) if tau is None else tau
        self.shift = None if shift is None else [shift[b % len(shift)] for b in range(B)]
        sh = self.shift or [0] * B
        if q_pos is None:   # the last Tq tokens, the cache complete up to the last of them
            q_pos = [[max(0, 4 * (self.lens[b] + sh[b]) + b % 4 + i - Tq + (1 if self.lens[b] == 0 else 0))
                      for i in range(Tq)] for b in range(B)]
        self.q_pos = np.array(q_pos, dtype=np.int64).reshape(B, Tq)
        self.max_entries = max(self.lens) if max_entries is None else max_entries
        # ---- pages
        per = [(n + 63) // 64 for n in self.lens]
        self.n_pages = sum(per) + 3
        perm = torch.randperm(self.n_pages, generator=g).numpy()
        width = max(max(per), 1) + 1
        self.table = np.full((B, width), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            self.table[b, :per[b]] = perm[at:at + per[b]]
            at += per[b]
        ns = self.n_pages * 64
        self.codes = torch.full((ns, d // 2), 0x77, dtype=torch.uint8)
        self.scales = torch.full((ns, d // 16), 0x7F, dtype=torch.uint8)     # NaN
        self.slots = []
        for b in range(B):
            n = self.lens[b]
            s = self.table[b, np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64
            self.slots.append(s)
            if n:
                x = (k_scale * torch.randn(n, d, generator=g)).numpy().astype(np.float32)
                c, sc = F.mxfp4_pack(x)
                self.codes[s], self.scales[s] = torch.from_numpy(c), torch.from_numpy(sc)
        self.entry_pos = None
        if scrambled:
            self.entry_pos = torch.full((ns,), -(1 << 30), dtype=torch.int32)
            for b in range(B):
                ids = torch.randperm(self.lens[b] + sh[b], generator=g)[:self.lens[b]].numpy()
                self.entry_pos[self.slots[b]] = torch.from_numpy((4 * ids + 3).astype(np.int32))
        # ---- window rows: the positions that the first token's window starts with, to the last token
        self.window = window and W > 0
        self.pos0 = np.maximum(0, self.q_pos.min(axis=1) - W + 1)
        self.cap_rows = int((self.q_pos.max(axis=1) - self.pos0).max()) + 1 + swa_slack if self.window else 0
        rows = max(1, self.cap_rows)
        self.wcodes = torch.full((B, rows, d), 0x7F, dtype=torch.uint8)
        self.wscales = torch.full((B, rows), float("nan"))
        for b in range(B):
            held = int(self.q_pos[b].max() - self.pos0[b]) + 1
            if self.window and held > 0:
                x = torch.randn(held, d, generator=g).numpy().astype(np.float32)
                c, sc = F.fp8_pack(x)
                self.wcodes[b, :held], self.wscales[b, :held] = torch.from_numpy(c), torch.from_numpy(sc)
        self.Q = (q_scale * torch.randn(B, Tq, Hq, d, generator=g)).to(torch.bfloat16)
        self.slopes = None
        if slopes is not None:
            self.slopes = torch.tensor([slopes[h % len(slopes)] for h in range(Hq)], dtype=torch.float32)
        self.docs = None if docs is None else np.array(docs, dtype=np.int64).reshape(B, Tq)
        self.prefix = None if prefix is None else [prefix[b % len(prefix)] for b in range(B)]
        self._device()

    def _device(self):
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
        self.t = {"codes": self.codes.cuda(), "scales": self.scales.cuda(), "table": i32(self.table),
                  "n": i32(self.lens), "q_pos": i32(self.q_pos), "Q": self.Q.cuda(), "wcodes": self.wcodes.cuda(),
                  "wscales": self.wscales.cuda(), "pos0": i32(self.pos0)}
        for k, v in (("shift", self.shift), ("docs", self.docs), ("prefix", self.prefix)):
            self.t[k] = None if v is None else i32(v)
        self.t["pos"] = None if self.entry_pos is None else self.entry_pos.cuda()
        self.t["slopes"] = None if self.slopes is None else self.slopes.cuda()
        self.O = torch.full((self.B, self.Tq, self.Hq, self.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.B, self.Tq, self.Hq), float("nan"), device="cuda")

    # ---- the calls --------------------------------------------------------------------
    def dims(self):
        return abi.Dims(B=self.B, Tq=self.Tq, d=self.d, r=0, Hq=self.Hq, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=1,
                        W=self.W, max_pages=self.table.shape[1], n_pool_blocks=0, pool_block=8, swa_cap=self.cap_rows,
                        kv_format=abi.CSA2_KV_MXFP4)

    def p(self, k):
        return None if self.t[k] is None else self.t[k].data_ptr()

    def structs(self):
        cache = abi.Cache(kv_codes=self.p("codes"), kv_scales=self.p("scales"), idx_k=None, page_table=self.p("table"),
                          n_entries=self.p("n"), n_pages=self.n_pages)
        bounded = abi.Bounded(entry_pos=self.p("pos"), weight=None, shift=self.p("shift"))
        win = abi.Window(codes=self.p("wcodes"), scales=self.p("wscales"), pos0=self.p("pos0"))
        mods = abi.ScoreMods(logit_cap=self.cap, slopes=self.p("slopes"), doc_start=self.p("docs"),
                             prefix_len=self.p("prefix"))
        return cache, bounded, win, mods

    def attend(self, ws=None, stream=None):
        dm = self.dims()
        cache, bounded, win, mods = self.structs()
        need = abi.csa2_dense_attn_workspace_size(dm, self.max_entries)
        if ws is None:
            ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        abi.csa2_dense_attn(dm, cache, win if self.window else None, self.t["Q"], self.t["q_pos"], self.tau,
                            self.max_entries, self.O, self.lse, ws, mods=mods, bounded=bounded, stream=stream)
        return self.O, self.lse

    def weigh(self, lse, weight_in, weight_out, decay=1.0, ws=None, stream=None):
        dm = self.dims()
        cache, bounded, _, mods = self.structs()
        need = abi.csa2_entry_weights_workspace_size(dm, self.max_entries)
        if ws is None:
            ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        abi.csa2_entry_weights(dm, cache, self.t["Q"], self.t["q_pos"], lse, self.tau, decay, weight_in, weight_out,
                               self.max_entries, ws, mods=mods, bounded=bounded, stream=stream)
        return weight_out

    # ---- the oracle's view --------------------------------------------------------------
    def keys(self, b):
        """(rows [n, d], positions [n]) of sequence b's entries."""
        n = min(self.lens[b], self.max_entries)
        s = self.slots[b][:n]
        rows = F.mxfp4_unpack(self.codes[s].numpy(), self.scales[s].numpy()) if n else np.zeros((0, self.d))
        sh = self.shift[b] if self.shift else 0
        pos = self.entry_pos[s].numpy().astype(np.int64) if self.entry_pos is not None else 4 * (np.arange(n) + sh) + 3
        return rows, pos

    def seen(self, b, i, pos):
        """Indices of the entries that token (b, i) sees."""
        t = int(self.q_pos[b, i])
        nv = OB.visible_count(len(pos), self.shift[b] if self.shift else 0, t, self.prefix[b] if self.prefix else 0)
        j = np.arange(nv)
        return j[pos[:nv] - 3 >= self.docs[b, i]] if self.docs is not None else j

    def window_rows(self, b, i):
        t = int(self.q_pos[b, i])
        lo = max(0, t - self.W + 1, int(self.docs[b, i]) if self.docs is not None else 0)
        p = np.arange(lo, t + 1) if self.window else np.zeros(0, np.int64)
        r = p - self.pos0[b]
        if len(p) == 0:
            return np.zeros((0, self.d)), p
        return F.fp8_unpack_bf16(self.wcodes[b, r].numpy(), self.wscales[b, r].numpy()), p

    def logit_error(self, q, k, x, tau):
        mag = (np.abs(q) @ np.abs(k).T) * tau
        return 2.0 ** -20 * mag + 2.0 ** -21 * (np.abs(x) + mag)

    def one(self, b, i, entries=None):
        """Logits, keys and logit errors of token (b, i): entries first, then window rows."""
        K, pos = entries if entries is not None else self.keys(b)
        j = self.seen(b, i, pos)
        Kw, pw = self.window_rows(b, i)
        q = self.Q[b, i].double().numpy()
        sl = None if self.slopes is None else self.slopes.double().numpy()
        t = int(self.q_pos[b, i])
        keys, p = np.concatenate([K[j], Kw]), np.concatenate([pos[j], pw])
        x = OB.logits(q, keys, self.tau, t, p, self.cap, sl)
        e = self.logit_error(q, keys, x, self.tau)
        if sl is not None:
            e = e + 2.0 ** -22 * sl[:, None] * np.abs(t - p.astype(np.float64))[None, :]
        return j, keys, x, e

    def check_attention(self, tokens=None):
        O, lse = self.O.double().cpu().numpy(), self.lse.double().cpu().numpy()
        cached = {}
        for b, i in tokens or [(b, i) for b in range(self.B) for i in range(self.Tq)]:
            if b not in cached:
                cached = {b: self.keys(b)}
            _, keys, x, e = self.one(b, i, cached[b])
            o, z = OB.attention(x, keys)
            where = f"sequence {b} token {i}"
            if x.shape[1] == 0:
                assert not O[b, i].any() and np.all(np.isneginf(lse[b, i])), where
                continue
            assert np.all(np.isfinite(O[b, i])) and np.all(np.isfinite(lse[b, i])), where
            e_max = e.max(axis=1)
            tol_z = e_max + 2.0 ** -20 + 2.0 ** -23 * np.abs(z)
            bad = np.abs(lse[b, i] - z) > tol_z
            assert not bad.any(), (where, "lse", np.argmax(bad), np.max(np.abs(lse[b, i] - z) / tol_z))
            w = np.exp(x - z[:, None])
            top = np.exp(x.max(axis=1) - z)                       # 1 / l in units of the largest term
            spread = (w * (2.0 ** -11 + 2 * e + e_max[:, None] + 2.0 ** -20)) @ np.abs(keys)
            tiny = 2.0 ** -17 * top[:, None] * np.abs(keys).sum(axis=0)[None, :]
            tol = 2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * spread + np.minimum(tiny, spread + tiny)
            bad = np.abs(O[b, i] - o) > tol
            assert not bad.any(), (where, "O", np.argwhere(bad)[:3], np.max(np.abs(O[b, i] - o) / tol))

    def check_weights(self, lse, w_in, w_out, decay=1.0):
        """w_in / w_out: the slot arrays before and after (w_in None: zeros)."""
        z_all, got = lse.double().cpu().numpy(), w_out.double().cpu().numpy()
        owned = np.zeros(self.n_pages * 64, bool)
        for b in range(self.B):
            K, pos = self.keys(b)
            n = len(pos)
            s = self.slots[b][:n]
            owned[s] = True
            ref, tol = np.zeros(n), np.zeros(n)
            for i in range(self.Tq):
                z = z_all[b, i]
                j, keys, x, e = self.one(b, i, (K, pos))
                x, e = x[:, :len(j)], e[:, :len(j)]
                live = np.isfinite(z)
                term = np.exp(x[live] - z[live][:, None])
                ref[j] += term.sum(axis=0)
                tol[j] += (term * (2 * e[live] + 2.0 ** -22 * (np.abs(x[live]) + np.abs(z[live])[:, None]) +
                                   2.0 ** -20)).sum(axis=0)
            if w_in is not None:
                ref += decay * w_in.double().cpu().numpy()[s]
            tol += 2.0 ** -22 * np.abs(ref) + 1e-37
            bad = np.abs(got[s] - ref) > tol
            assert not bad.any(), (b, np.argwhere(bad)[:4].ravel(), np.max(np.abs(got[s] - ref) / tol))
        return owned
