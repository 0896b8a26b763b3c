"""Cases of the bounded-cache operators: attention over the whole 4-bit compressed
cache, the attention weight that each entry receives, and the eviction of entries
by that weight.

  attn     csa2_dense_attn     every visible entry of the MXFP4 cache and the FP8
                               window, with an optional tanh cap, distance bias,
                               document mask and prefix mask; O in bf16, lse in fp32
  weights  csa2_entry_weights  weight_out[j] = decay * weight_in[j] + the softmax
                               weight of entry j summed over query tokens and heads
  evict    csa2_evict          the `keep` entries of highest weight stay (the first
                               entries and the most recent ones always); the others'
                               slots below `keep` are filled with survivors from above

`own` False computes them in elementary torch operations, True calls the library.
A case's lengths and positions follow from the case alone, its values from the seed.
"""
import math

import numpy as np
import torch

own = False

D = 512          # latent width
PAGE = 64        # entries per page
ENTRY_BYTES = D // 2 + D // 16
IDX_W = 128      # indexer key width (moved by the eviction)
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _attn(name, **kw):
    c = {"name": name, "op": "attn", "B": 1, "Tq": 1, "Hq": 64, "n": 1024, "ragged": False, "W": 128, "cap": 0.0,
         "slopes": False, "docs": False, "prefix": False, "bounded": False}
    c.update(kw)
    return c


def _weights(name, **kw):
    c = _attn(name, **kw)
    c["op"] = "weights"
    return c


def _evict(name, **kw):
    c = {"name": name, "op": "evict", "B": 32, "n": 4160, "keep": 4096, "ragged": False, "sinks": 4, "recent": 64}
    c.update(kw)
    return c


def listed():
    return [
        # one token of a short conversation: latency alone
        _attn("attn_one_short", n=99),
        # the decode batch of the benchmark: 32 sequences at 131,072 tokens
        _attn("attn_decode_b32_128k", B=32, n=32768),
        # a serving batch of mixed lengths (16 .. 65,536 entries), capped scores
        _attn("attn_decode_ragged", B=64, n=65536, ragged=True, cap=30.0),
        # one sequence of a million tokens
        _attn("attn_one_1m", n=262144),
        # a few drafted tokens over a cache that entries were evicted from, distance bias, an odd number of heads
        _attn("attn_drafts_bounded", B=8, Tq=5, Hq=40, n=4131, slopes=True, bounded=True),
        # a prefill chunk of packed documents, capped scores
        _attn("attn_prefill_docs", Tq=1024, n=16384, cap=50.0, docs=True),
        # the weights of one decode step over bounded caches
        _weights("weights_decode_bounded", B=32, n=4160, bounded=True),
        # one decode step over the decode batch's whole context
        _weights("weights_decode_b32_128k", B=32, n=32768),
        # the weights of a prompt's last tokens, the usual choice before a first eviction
        _weights("weights_prompt_tail", B=2, Tq=257, n=16384, cap=30.0, slopes=True),
        # steady state: one page's worth of entries leaves each cache
        _evict("evict_step"),
        # a long prompt cut to half
        _evict("evict_prompt_half", B=8, n=65536, keep=32768, recent=256),
        # ragged prompts cut to one budget, the short ones untouched
        _evict("evict_ragged", B=16, n=131072, keep=2048, ragged=True, sinks=16, recent=128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attn", "attn", "weights", "evict"])
    if op == "evict":
        B = log(1, 64)
        n = log(64, max(64, (1 << 20) // B))
        keep = max(8, int(n * rng.uniform(0.05, 0.99)))
        return {"op": "evict", "B": B, "n": n, "keep": keep, "ragged": rng.random() < 0.4,
                "sinks": rng.randint(0, keep // 4), "recent": rng.randint(0, keep // 4)}
    c = {"op": op}
    if rng.random() < 0.65:      # decode: one token, or a few drafted ones
        c["Tq"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["B"] = log(1, 64)
        c["n"] = log(1, max(16, 1000000 // (c["B"] * c["Tq"])))
    else:                        # a chunk of a prompt
        c["Tq"] = log(16, 700)
        c["B"] = rng.choice([1, 1, 2, 3])
        c["n"] = max(-(-c["Tq"] // 4), log(64, max(128, 16000000 // (c["Tq"] * c["B"] * 2))))
        c["n"] = min(c["n"], 40000)
    c["Hq"] = rng.choice([64, 64, 64, 128, 16, 8, 40, 1])
    if c["Hq"] > 64:
        c["n"] = max(-(-c["Tq"] // 4), c["n"] // 2)
    c["ragged"] = rng.random() < 0.3
    c["W"] = rng.choice([128, 128, 128, 16, 0, 1000])
    c["cap"] = rng.choice([0.0, 0.0, 30.0, 12.5])
    c["slopes"] = rng.random() < 0.3
    c["bounded"] = c["Tq"] <= 8 and rng.random() < 0.3
    c["docs"] = not c["bounded"] and rng.random() < 0.3
    c["prefix"] = not c["docs"] and not c["bounded"] and rng.random() < 0.15
    return c


# ---- what a case fixes: lengths and positions ------------------------------------------

def _lengths(case):
    B, n = case["B"], case["n"]
    if not case["ragged"] or B == 1:
        return np.full(B, n, dtype=np.int64)
    lo = min(16, n)
    f = np.arange(B) * 0.61803398875 % 1.0       # log-uniform, in no order
    f[0] = 1.0
    return np.maximum(1, np.round(np.exp(np.log(lo) + f * (np.log(n) - np.log(lo))))).astype(np.int64)


def _layout(case):
    """Host arrays: entries, evicted entries, query positions, document starts, prefix lengths."""
    B, Tq = case["B"], case["Tq"]
    n = np.maximum(_lengths(case), -(-Tq // 4))
    shift = (n // 3 + 7) if case["bounded"] else np.zeros(B, dtype=np.int64)
    end = 4 * (n + shift) + np.arange(B) % 4     # tokens so far; the queries are the last Tq of them
    end = np.maximum(end, Tq)
    q_pos = (end - Tq)[:, None] + np.arange(Tq)[None, :]
    doc = np.zeros((B, Tq), dtype=np.int64)
    if case["docs"]:                             # documents of uneven lengths, the last of them still running
        for b in range(B):
            r = np.random.RandomState(1000 + b)
            starts, at = [], 0
            while at < end[b]:
                starts.append(at)
                at += 1 + int(r.randint(max(2, end[b] // 6)))
            starts = np.array(starts)
            doc[b] = starts[np.searchsorted(starts, q_pos[b], side="right") - 1]
    prefix = (end - Tq // 2).astype(np.int64) if case["prefix"] else np.zeros(B, dtype=np.int64)
    return n, shift, q_pos, doc, prefix


def _visible_counts(case):
    """Keys that each query token attends to: entries [B][Tq], window rows [B][Tq]."""
    n, shift, q_pos, doc, prefix = _layout(case)
    last = np.maximum(q_pos + 1, np.where(q_pos < prefix[:, None], prefix[:, None], 0))
    nv = np.clip(last // 4 - shift[:, None], 0, n[:, None])
    ent = np.maximum(0, nv - (doc + 3) // 4) if case["docs"] else nv
    win = np.minimum(np.minimum(case["W"], q_pos + 1), q_pos - doc + 1)
    return ent, win


def work(case):
    if case["op"] == "evict":
        n, keep = _lengths(case), case["keep"]
        cut = n > keep
        moved = np.where(cut, np.minimum(keep, n - keep) * keep // np.maximum(n, 1), 0).sum()
        row = ENTRY_BYTES + 2 * IDX_W + 8
        return {"bytes": int(8 * n[cut].sum() + 2 * row * moved + 4 * (n // PAGE + 1).sum() + 8 * case["B"]),
                "flops": int(4 * n.sum())}
    ent, win = _visible_counts(case)
    n, _, _, _, _ = _layout(case)
    rows = case["B"] * case["Tq"] * case["Hq"]
    read = np.minimum(n, ent.max(axis=1) + (n - ent.max(axis=1)) * case["docs"])
    nbytes = read.sum() * ENTRY_BYTES + 4 * (n // PAGE + 1).sum() + rows * (2 * D + 4) + 4 * case["B"] * case["Tq"]
    if case["op"] == "attn":
        held = min(case["W"], 1 << 30)
        nbytes += rows * 2 * D + case["B"] * (D + 4) * ((held + case["Tq"] - 1) if held else 0)
        flops = 4 * D * case["Hq"] * (ent.sum() + win.sum())
    else:
        nbytes += 8 * n.sum()
        flops = 2 * D * case["Hq"] * ent.sum()
    return {"bytes": int(nbytes), "flops": int(flops)}


# ---- inputs ------------------------------------------------------------------------------

def _pack_rows(rows, g):
    """MXFP4 rows of normalised N(0,1) latents: E2M1 codes and one E4M3 scale per 16 channels."""
    codes = torch.empty(rows, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, D // 16, dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for s in range(0, rows, 1 << 17):
        m = min(rows, s + (1 << 17)) - s
        x = torch.randn(m, D // 16, 16, device="cuda", generator=g)
        sc = (x.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
        scales[s:s + m] = sc.view(torch.uint8)
        x = x / sc.float().clamp_min(2.0 ** -9).unsqueeze(-1)
        c = torch.bucketize(x.abs(), edges).to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)
        c = c.view(m, D)
        codes[s:s + m] = c[:, 0::2] | (c[:, 1::2] << 4)
    return codes, scales


def _pages(n, g):
    """A page table over one shared pool, its pages in random order, and the pool's size."""
    per = (n + PAGE - 1) // PAGE + 1
    total = int(per.sum())
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(len(n), int(per.max()), dtype=torch.int32, device="cuda")
    at = 0
    for b, p in enumerate(per.tolist()):
        table[b, :p] = perm[at:at + p]
        at += p
    return table, total


def _slots(table, n):
    j = torch.arange(n, device="cuda")
    return table[:, j // PAGE].long() * PAGE + j % PAGE


def _positions(n, shift, table, pages, recent, g):
    """Raw position of every entry's last token: evicted caches hold a scattered subset, then the newest."""
    pos = torch.zeros(pages * PAGE, dtype=torch.int32, device="cuda")
    for b, (m, s) in enumerate(zip(n.tolist(), shift.tolist())):
        old = max(0, m - recent)
        order = torch.randperm(old + s, device="cuda", generator=g)[:old]
        j = torch.cat([order, torch.arange(old + s, m + s, device="cuda")])
        i = torch.arange(m, device="cuda")
        pos[table[b, i // PAGE].long() * PAGE + i % PAGE] = (4 * j + 3).to(torch.int32)
    return pos


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"op": case["op"]}
    if case["op"] == "evict":
        n = _lengths(case)
        table, pages = _pages(n, g)
        codes = torch.randint(0, 256, (pages * PAGE, D // 2), dtype=torch.uint8, device="cuda", generator=g)
        scales = torch.randint(0, 120, (pages * PAGE, D // 16), dtype=torch.uint8, device="cuda", generator=g)
        idx_k = torch.randn(pages * PAGE, IDX_W, device="cuda", generator=g).bfloat16()
        shift = n // 5
        pos = _positions(n, shift, table, pages, case["recent"] + 8, g)
        # accumulated weights have a long tail, and some entries were never attended to
        w = torch.exp(1.7 * torch.randn(pages * PAGE, device="cuda", generator=g) - 3.0)
        w = torch.where(torch.rand(pages * PAGE, device="cuda", generator=g) < 0.03, torch.zeros_like(w), w)
        # weights, positions, counts and shifts in one buffer, so that a pass starts from them with one copy
        first = torch.cat([w.view(torch.int32), pos, torch.tensor(n, **i32), torch.tensor(shift, **i32)])
        now, m, B = first.clone(), pages * PAGE, case["B"]
        pad = -(2 * m + B) % 4
        if pad:                                  # the shifts start on 16 bytes as well
            first = torch.cat([first[:2 * m + B], torch.zeros(pad, **i32), first[2 * m + B:]])
            now = first.clone()
        s.update(codes=codes, scales=scales, idx_k=idx_k, table=table, pages=pages, first=first, now=now,
                 weight=now[:m].view(torch.float32), pos=now[m:2 * m], n_entries=now[2 * m:2 * m + B],
                 shift=now[2 * m + B + pad:], keep=case["keep"], sinks=case["sinks"], recent=case["recent"],
                 max_entries=int(n.max()))
        return s
    n, shift, q_pos, doc, prefix = _layout(case)
    B, Tq, Hq, W = case["B"], case["Tq"], case["Hq"], case["W"]
    table, pages = _pages(n, g)
    codes, scales = _pack_rows(pages * PAGE, g)
    Q = torch.randn(B, Tq, Hq, D, device="cuda", generator=g).bfloat16()
    s.update(codes=codes, scales=scales, table=table, pages=pages, Q=Q, q_pos=torch.tensor(q_pos, **i32),
             n_entries=torch.tensor(n, **i32), max_entries=int(n.max()), scale=1.0 / math.sqrt(D), cap=case["cap"],
             W=W, slopes=None, doc=None, prefix=None, pos=None, shift=None)
    if case["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, dtype=torch.float32, device="cuda") / Hq)
    if case["docs"]:
        s["doc"] = torch.tensor(doc, **i32)
    if case["prefix"]:
        s["prefix"] = torch.tensor(prefix, **i32)
    if case["bounded"]:
        s["shift"] = torch.tensor(shift, **i32)
        s["pos"] = _positions(n, shift, table, pages, 64, g)
    if case["op"] == "attn":
        rows = max(1, W + Tq - 1) if W else 1
        x = torch.randn(B, rows, D, device="cuda", generator=g)
        sc = x.abs().amax(-1) / 448
        s["win_codes"] = (x / sc.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
        s["win_scales"] = sc
        s["win_pos0"] = torch.tensor(np.maximum(0, q_pos[:, 0] - max(0, W - 1)), **i32)
        s["O"] = torch.empty(B, Tq, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(B, Tq, Hq, dtype=torch.float32, device="cuda")
    else:
        # what the attention's lse is for such inputs: the log of the visible keys' number plus half the variance
        ent, win = _visible_counts(case)
        keys = torch.tensor(ent + win, dtype=torch.float32, device="cuda").clamp_min(1).log()
        s["lse"] = keys.unsqueeze(-1) + 0.5 + 0.1 * torch.randn(B, Tq, Hq, device="cuda", generator=g)
        s["weight_in"] = torch.rand(pages * PAGE, device="cuda", generator=g)
        s["weight_out"] = torch.zeros(pages * PAGE, device="cuda")
        s["decay"] = 0.98
    return s


# ---- the library's calls -----------------------------------------------------------------

def _handle(s):
    """The descriptors and the workspace that a program builds once and keeps."""
    h = s.get("handle")
    if h is not None:
        return h
    from compressed_sparse_attention_05_gb300 import abi
    p = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
    h = {"abi": abi}
    cache = abi.Cache(kv_codes=p(s["codes"]), kv_scales=p(s["scales"]), idx_k=p(s.get("idx_k")),
                      page_table=p(s["table"]), n_entries=p(s["n_entries"]), n_pages=s["pages"])
    if s["op"] == "evict":
        dims = abi.Dims(B=s["table"].shape[0], Tq=1, d=D, r=64, Hq=64, Hi=8, Di=IDX_W, idx_dtype=abi.CSA2_BF16,
                        K=512, W=0, max_pages=s["table"].shape[1], kv_format=abi.CSA2_KV_MXFP4)
        need = abi.csa2_evict_workspace_size(dims, s["max_entries"])
    else:
        B, Tq, Hq, _ = s["Q"].shape
        cap = s["win_codes"].shape[1] if "win_codes" in s else 0
        dims = abi.Dims(B=B, Tq=Tq, d=D, r=64, Hq=Hq, Hi=8, Di=IDX_W, idx_dtype=abi.CSA2_BF16, K=512, W=s["W"],
                        max_pages=s["table"].shape[1], swa_cap=cap, kv_format=abi.CSA2_KV_MXFP4)
        h["mods"] = abi.ScoreMods(logit_cap=s["cap"], slopes=p(s["slopes"]), doc_start=p(s["doc"]),
                                  prefix_len=p(s["prefix"]))
        if s["op"] == "attn":
            h["window"] = abi.Window(codes=p(s["win_codes"]), scales=p(s["win_scales"]), pos0=p(s["win_pos0"]))
            need = abi.csa2_dense_attn_workspace_size(dims, s["max_entries"])
        else:
            need = abi.csa2_entry_weights_workspace_size(dims, s["max_entries"])
    h["dims"], h["cache"] = dims, cache
    h["bounded"] = abi.Bounded(entry_pos=p(s["pos"]), weight=p(s.get("weight")), shift=p(s["shift"]))
    h["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    s["handle"] = h
    return h


def run(s):
    if s["op"] == "evict":
        s["now"].copy_(s["first"])       # every pass evicts from the same cache
        if own:
            h = _handle(s)
            h["abi"].csa2_evict(h["dims"], h["cache"], h["bounded"], s["n_entries"], s["keep"], s["sinks"], s["recent"],
                                s["max_entries"], h["ws"])
        else:
            _plain_evict(s)
        return {"codes": s["codes"], "scales": s["scales"], "idx_k": s["idx_k"], "weight": s["weight"], "pos": s["pos"],
                "n": s["n_entries"], "shift": s["shift"]}
    if s["op"] == "attn":
        if own:
            h = _handle(s)
            h["abi"].csa2_dense_attn(h["dims"], h["cache"], h["window"], s["Q"], s["q_pos"], s["scale"],
                                     s["max_entries"], s["O"], s["lse"], h["ws"], mods=h["mods"], bounded=h["bounded"])
            return {"O": s["O"], "lse": s["lse"]}
        return _plain_attn(s)
    if own:
        h = _handle(s)
        h["abi"].csa2_entry_weights(h["dims"], h["cache"], s["Q"], s["q_pos"], s["lse"], s["scale"], s["decay"],
                                    s["weight_in"], s["weight_out"], s["max_entries"], h["ws"], mods=h["mods"],
                                    bounded=h["bounded"])
        return {"weight": s["weight_out"]}
    return _plain_weights(s)


# ---- the plain forms ---------------------------------------------------------------------

def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _entries(s):
    """The sequences' rows, dequantised: fp32 [B][max_entries][D], and their slots."""
    slots = _slots(s["table"], s["max_entries"])
    values = torch.tensor(_E2M1 + [-v for v in _E2M1], device="cuda")
    c = s["codes"][slots]
    x = torch.stack([values[(c & 15).int()], values[(c >> 4).int()]], dim=-1)
    sc = _e4m3(s["scales"][slots])
    return (x.view(*sc.shape, 16) * sc.unsqueeze(-1)).view(*slots.shape, D), slots


def _scores(s, K, pos):
    """fp32 logits [B][Tq][Hq][keys] of keys whose (last) raw positions are pos [B][keys], without masks."""
    B, Tq, Hq, _ = s["Q"].shape
    x = (s["Q"].float().view(B, Tq * Hq, D) @ K.transpose(1, 2)).view(B, Tq, Hq, -1) * s["scale"]
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    if s["slopes"] is not None:
        far = (s["q_pos"].unsqueeze(-1) - pos.unsqueeze(1)).abs().float()
        x = x - s["slopes"].view(1, 1, Hq, 1) * far.unsqueeze(2)
    return x


def _entry_scores(s, K, slots):
    """Logits of the entries, -inf where the query token does not see one."""
    B, n = slots.shape
    t = s["q_pos"].long().unsqueeze(-1)
    j = torch.arange(n, device="cuda").view(1, 1, n)
    pos = s["pos"][slots].long() if s["pos"] is not None else (4 * j.view(1, n) + 3).expand(B, n)
    last = t + 1
    if s["prefix"] is not None:
        pre = s["prefix"].long().view(B, 1, 1)
        last = torch.where(t < pre, pre, last)
    shift = s["shift"].long().view(B, 1, 1) if s["shift"] is not None else 0
    seen = (j < last // 4 - shift) & (j < s["n_entries"].view(B, 1, 1))
    if s["doc"] is not None:
        seen = seen & (pos.unsqueeze(1) - 3 >= s["doc"].unsqueeze(-1))
    return torch.where(seen.unsqueeze(2), _scores(s, K, pos), float("-inf"))


def _plain_attn(s):
    B, Tq, Hq, _ = s["Q"].shape
    K, slots = _entries(s)
    x = _entry_scores(s, K, slots)
    # the window rows: raw positions max(0, t-W+1) .. t, inside the document
    Kw = (_e4m3(s["win_codes"]) * s["win_scales"].unsqueeze(-1)).bfloat16().float()
    t = s["q_pos"].long().unsqueeze(-1)
    p = s["win_pos0"].long().unsqueeze(-1) + torch.arange(Kw.shape[1], device="cuda")
    seen = (p.unsqueeze(1) <= t) & (p.unsqueeze(1) > t - s["W"])
    if s["doc"] is not None:
        seen = seen & (p.unsqueeze(1) >= s["doc"].unsqueeze(-1))
    x = torch.cat([x, torch.where(seen.unsqueeze(2), _scores(s, Kw, p), float("-inf"))], dim=-1)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    del x
    l = e.sum(-1, keepdim=True)
    V = torch.cat([K, Kw], dim=1)
    o = (e.view(B, Tq * Hq, -1) @ V).view(B, Tq, Hq, D) / torch.where(l == 0, torch.ones_like(l), l)
    return {"O": o.bfloat16(), "lse": (m + torch.log(l)).squeeze(-1)}


def _plain_weights(s):
    K, slots = _entries(s)
    x = _entry_scores(s, K, slots)
    w = torch.exp(x - s["lse"].unsqueeze(-1)).sum(dim=(1, 2))
    new = s["decay"] * s["weight_in"][slots] + w
    # rows past a sequence's last entry go to a spare slot behind the pool
    held = torch.arange(slots.shape[1], device="cuda") < s["n_entries"].unsqueeze(-1)
    out = torch.cat([s["weight_out"], s["weight_out"][:1]])
    out[torch.where(held, slots, out.numel() - 1)] = new
    s["weight_out"].copy_(out[:-1])
    return {"weight": s["weight_out"]}


def _plain_evict(s):
    B, n, keep = s["table"].shape[0], s["max_entries"], s["keep"]
    if n <= keep:
        return
    slots = _slots(s["table"], n)
    j = torch.arange(n, device="cuda").unsqueeze(0)
    count, shift = s["n_entries"].long().unsqueeze(-1), s["shift"].long().unsqueeze(-1)
    pos, w = s["pos"][slots].long(), s["weight"][slots]
    always = (pos < 4 * s["sinks"]) | (pos >= 4 * (count + shift - s["recent"]) + 3)
    key = torch.where(always, float("inf"), w)
    key = torch.where(j < count, key, float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(1, order[:, :keep], True) & (j < count)
    cut = count > keep
    hole, mover = ~kept & (j < keep) & cut, kept & (j >= keep) & cut
    spare = torch.full_like(hole, n, dtype=torch.int64)
    nth = torch.zeros(B, n + 1, dtype=torch.int64, device="cuda")
    nth.scatter_(1, torch.where(mover, mover.cumsum(1) - 1, spare), j.expand(B, n).contiguous())
    src = torch.where(hole, nth.gather(1, (hole.cumsum(1) - 1).clamp_min(0)), j)[:, :keep]
    to, frm = slots[:, :keep], slots.gather(1, src)
    # rows of sequences shorter than `keep` stay: their slots past the end are not theirs
    mine = (j[:, :keep] < count) & cut
    safe = s["table"][:, :1].long() * PAGE
    to, frm = torch.where(mine, to, safe), torch.where(mine, frm, safe)
    first = torch.where(cut, src[:, :1], 0)
    frm = torch.where(mine, frm, slots.gather(1, first))
    for k in ("codes", "scales", "idx_k", "weight", "pos"):
        s[k][to] = s[k][frm]
    s["shift"] += torch.where(cut, count - keep, 0).view(-1).int()
    s["n_entries"].copy_(torch.where(cut, keep, count).view(-1))


# ---- from the definitions, in 64 bits ------------------------------------------------------

def _row64(s, slots):
    """Dequantised rows by the formats' formulas: E2M1 and E4M3 sign, exponent, mantissa."""
    c = s["codes"][slots].int()
    c = torch.stack([c & 15, c >> 4], dim=-1).flatten(1)
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, 0.5 * m, torch.pow(2.0, e.double() - 1) * (1 + 0.5 * m))
    f = s["scales"][slots].int()
    fe, fm = (f >> 3) & 15, (f & 7).double()
    sc = torch.where(fe == 0, fm * 2.0 ** -9, torch.pow(2.0, fe.double() - 7) * (1 + fm / 8))
    return torch.where(c >= 8, -mag, mag) * sc.repeat_interleave(16, dim=1)


def _logits64(s, b, i0, i1, K, pos):
    x = torch.einsum("thd,kd->thk", s["Q"][b, i0:i1].double(), K) / math.sqrt(D)
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    if s["slopes"] is not None:
        t = s["q_pos"][b, i0:i1].double()
        x -= s["slopes"].double()[None, :, None] * (t[:, None] - pos.double()[None, :]).abs()[:, None, :]
    return x


def _seen64(s, b, i0, i1, pos):
    j = torch.arange(pos.numel(), device="cuda")
    t = s["q_pos"][b, i0:i1].long()
    last = t
    if s["prefix"] is not None:
        last = torch.where(t < s["prefix"][b], s["prefix"][b].long() - 1, t)
    # entry j (after `shift` evicted ones) is complete at raw position 4 (j + shift) + 3
    done = 4 * (j + (int(s["shift"][b]) if s["shift"] is not None else 0)) + 3
    seen = done[None, :] <= last[:, None]
    if s["doc"] is not None:
        seen &= (pos - 3)[None, :] >= s["doc"][b, i0:i1].long()[:, None]
    return seen


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    B, Tq, Hq, _ = s["Q"].shape
    n = s["n_entries"].tolist()
    O = torch.zeros(B, Tq, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Tq, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    out = s.get("weight_out")
    out = out.double() if out is not None else None
    for b in range(B):
        j = torch.arange(n[b], device="cuda")
        slots = s["table"][b, j // PAGE].long() * PAGE + j % PAGE
        K = _row64(s, slots)
        pos = s["pos"][slots].long() if s["pos"] is not None else 4 * j + 3
        if case["op"] == "weights":
            w = torch.zeros(n[b], dtype=torch.float64, device="cuda")
        else:
            f8 = s["win_codes"][b].int()
            e, m = (f8 >> 3) & 15, (f8 & 7).double()
            v = torch.where(e == 0, m * 2.0 ** -9, torch.pow(2.0, e.double() - 7) * (1 + m / 8))
            v = torch.where(f8 >= 128, -v, v).float() * s["win_scales"][b][:, None]
            Kw = v.bfloat16().double()           # the window operand is a bf16 value by definition
            pw = int(s["win_pos0"][b]) + torch.arange(Kw.shape[0], device="cuda")
        step = max(1, (1 << 28) // max(1, Hq * (n[b] + 1)))
        for i0 in range(0, Tq, step):
            i1 = min(Tq, i0 + step)
            x = _logits64(s, b, i0, i1, K, pos)
            x.masked_fill_(~_seen64(s, b, i0, i1, pos)[:, None, :], float("-inf"))
            if case["op"] == "weights":
                w += torch.exp(x - s["lse"][b, i0:i1].double()[:, :, None]).sum(dim=(0, 1))
                continue
            t = s["q_pos"][b, i0:i1].long()
            back = t[:, None] - pw[None, :]
            ok = (back >= 0) & (back < s["W"])
            if s["doc"] is not None:
                ok &= pw[None, :] >= s["doc"][b, i0:i1].long()[:, None]
            y = _logits64(s, b, i0, i1, Kw, pw).masked_fill_(~ok[:, None, :], float("-inf"))
            z = torch.logsumexp(torch.cat([x, y], dim=-1), dim=-1)
            lse[b, i0:i1] = z
            z = torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, :, None]
            O[b, i0:i1] = torch.einsum("thk,kd->thd", torch.exp(x - z), K) + torch.einsum("thk,kd->thd", torch.exp(y - z), Kw)
        if case["op"] == "weights":
            out[slots] = 0.98 * s["weight_in"][slots].double() + w
    return {"weight": out} if case["op"] == "weights" else {"O": O, "lse": lse}


def _exact_evict(s):
    keep = s["keep"]
    for b, count in enumerate(s["n_entries"].tolist()):
        if count <= keep:
            continue
        j = np.arange(count)
        table = s["table"][b].cpu().numpy().astype(np.int64)
        slots = table[j // PAGE] * PAGE + j % PAGE
        at = torch.from_numpy(slots).cuda()
        pos, w = s["pos"][at].cpu().numpy(), s["weight"][at].cpu().numpy()
        seen = count + int(s["shift"][b])        # entries that the sequence has produced
        always = (pos // 4 < s["sinks"]) | (pos // 4 >= seen - s["recent"])
        rank = np.lexsort((j, -w.astype(np.float64), ~always))
        stays = np.zeros(count, dtype=bool)
        stays[rank[:keep]] = True
        to, frm = j[:keep][~stays[:keep]], j[keep:][stays[keep:]]
        to, frm = torch.from_numpy(slots[to]).cuda(), torch.from_numpy(slots[frm]).cuda()
        for k in ("codes", "scales", "idx_k", "weight", "pos"):
            s[k][to] = s[k][frm].clone()
        s["n_entries"][b] = keep
        s["shift"][b] += count - keep
    return {"codes": s["codes"], "scales": s["scales"], "idx_k": s["idx_k"].double(), "weight": s["weight"].double(),
            "pos": s["pos"], "n": s["n_entries"], "shift": s["shift"]}
