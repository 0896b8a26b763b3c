"""Cases of the operators on the query side of a decoding step with drafted tokens.

  pages   csa2_page_plan        pages taken from and given back to the pool as the
                                sequences' lengths change; positions and cache slots of
                                the step's tokens and entries
  pack    csa2_pack_fp8_blocks  rows to E4M3 codes with one fp32 scale per 128 columns
  matmul  csa2_matmul_fp8       C = A B^T of such rows, B with one scale per 128 x 128
  rope    csa2_rope             rotary positions: half and interleaved pairs, part of the
                                head, frequencies scaled for long contexts, both directions
  tree    csa2_tree_plan,       positions and paths of a tree of drafted tokens, and their
          csa2_tree_attn        attention over selected cache entries, the window and
                                their own ancestors

`own` False computes them in elementary torch operations, True calls the library.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64        # entries per page
BLOCK = 128      # columns (and rows of B) that share a scale
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _case(op, name=None, **kw):
    c = {
        "pages": {"B": 32, "max_len": 131072, "step": 8, "shift": False, "short": False, "ends": 0.1},
        "pack": {"M": 32, "K": 4096, "dtype": "bf16", "extra": 0},
        "matmul": {"M": 32, "N": 32768, "K": 4096, "out": "bf16"},
        "rope": {"rows": 1, "heads": 64, "d": 512, "r": 64, "start": 448, "layout": "half", "scaling": "none", "dtype": "bf16",
                 "out": "bf16", "inverse": False, "extra": 0, "max_pos": 131072},
        "tree": {"B": 1, "Tq": 8, "Hq": 64, "n": 4096, "K": 512, "W": 128, "ragged": False, "fp8": False, "chain": False},
    }[op]
    c = {"op": op, **c, **kw}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a decoding batch: 32 sequences, 8 drafted tokens each, most of them inside their last page
        _case("pages", "pages_step_b32"),
        # 160 sequences of a serving pool: prompts of up to 32,768 tokens come in, others end, the pool runs short
        _case("pages", "pages_prompts_b160", B=160, max_len=131072, step=32768, shift=True, short=True, ends=0.3),
        # the hidden states of a decoding batch
        _case("pack", "pack_b32"),
        # the hidden states of a long prompt, fp32, an odd number of blocks, rows that lie in a wider tensor
        _case("pack", "pack_prompt_f32", M=16411, K=4240, dtype="f32", extra=48),
        # the query projection of 64 heads x 512 channels of a decoding batch of 32 tokens
        _case("matmul", "matmul_decode_b32"),
        # a small ragged product: odd rows and columns, a last block of 16 columns, fp32 out
        _case("matmul", "matmul_odd_f32", M=161, N=1001, K=1552, out="f32"),
        # the query projection of a prefill chunk of 4,096 tokens
        _case("matmul", "matmul_prefill_4k", M=4096),
        # the queries of one token
        _case("rope", "rope_one"),
        # a prefill chunk's queries, a slice of a fused projection, long-context frequencies, into the attention's layout
        _case("rope", "rope_prefill_4k", rows=4096, layout="interleaved", scaling="yarn", extra=1024, max_pos=1000000),
        # one sequence, 8 drafted tokens, a short context
        _case("tree", "tree_one"),
        # the decoding batch of the benchmark with 8 drafted tokens each
        _case("tree", "tree_decode_b32", B=32, n=32768),
        # wide trees of uneven sizes over the FP8 cache, an odd number of heads, the longest selection
        _case("tree", "tree_wide_fp8", B=7, Tq=61, Hq=40, n=8192, K=2048, W=200, ragged=True, fp8=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["pages", "pack", "matmul", "matmul", "rope", "tree", "tree"])
    if op == "pages":
        B = log(1, 600)
        step = log(1, min(32768, max(1, 5000000 // B)))
        return _case(op, B=B, max_len=max(step, log(64, 262144)), step=step, shift=rng.random() < 0.5, short=rng.random() < 0.5,
                     ends=rng.choice([0.0, 0.1, 0.3]))
    if op == "pack":
        K = 16 * log(1, 512)
        M = log(1, max(1, 69000000 // K))
        return _case(op, M=M, K=K, dtype=rng.choice(["bf16", "bf16", "f32"]), extra=rng.choice([0, 0, 16, 1024]))
    if op == "matmul":
        M, K = log(1, 4096), 16 * log(2, 512)
        N = log(16, min(32768, (4096 * 4096 * 32768) // (M * K)))
        return _case(op, M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "rope":
        d = rng.choice([512, 512, 128, 64, 576])
        r = rng.choice([q for q in (64, 64, 32, 128, 16, 62, d) if q <= d])
        heads = rng.choice([64, 64, 128, 40, 8, 1])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        out = rng.choice(["bf16", "f32"]) if dtype == "f32" else "bf16"
        rows = log(1, max(1, (4096 * 64 * 512 * 4 // (8 if out == "f32" else 6 if dtype == "f32" else 4)) // (heads * d)))
        return _case(op, rows=rows, heads=heads, d=d, r=r, start=rng.choice([d - r, d - r, 0]), layout=rng.choice(["half", "interleaved"]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]), dtype=dtype, out=out, inverse=rng.random() < 0.4,
                     extra=rng.choice([0, 0, 1024, 64]), max_pos=rng.choice([4096, 131072, 1000000]))
    Tq = rng.choice([1, 2, 5, 8, 8, 16, 31, 61])
    Hq = rng.choice([64, 64, 64, 128, 40, 16, 1])
    K = rng.choice([512, 512, 64, 17, 2048])
    B = log(1, max(1, min(64, 60000000 // (Tq * max(Hq, 64) * (K + 128)))))
    return _case(op, B=B, Tq=Tq, Hq=Hq, n=log(4, min(131072, max(64, 60000000 // (B * Tq)))), K=K, W=rng.choice([128, 128, 16, 200, 1000]),
                 ragged=rng.random() < 0.4, fp8=rng.random() < 0.3, chain=rng.random() < 0.2)


def _tree_lengths(case):
    """Entries of every sequence, from the case alone."""
    B, n = case["B"], case["n"]
    if not case["ragged"] or B == 1:
        return np.full(B, n, dtype=np.int64)
    f = np.arange(B) * 0.61803398875 % 1.0       # log-uniform, in no order
    f[0] = 1.0
    return np.maximum(1, np.round(np.exp(np.log(min(4, n)) + f * (np.log(n) - np.log(min(4, n)))))).astype(np.int64)


def work(case):
    op = case["op"]
    if op == "pages":
        B, step = case["B"], case["step"]
        # lengths, counts and grants; slots (8 bytes a column) and positions (4 bytes); pages of the new entries
        return {"bytes": int(40 * B + B * (8 * (step // 4 + 1) + 4 * step) + 8 * B * (step // 256 // 2 + 1)), "flops": int(B * step)}
    if op == "pack":
        n = case["M"] * case["K"]
        return {"bytes": int(n * (5 if case["dtype"] == "f32" else 3) + 4 * case["M"] * -(-case["K"] // BLOCK)), "flops": int(3 * n)}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        return {"bytes": int(M * K + N * K + 4 * kb * (M + -(-N // BLOCK)) + M * N * (4 if case["out"] == "f32" else 2)),
                "flops": int(2 * M * N * K)}
    if op == "rope":
        n = case["rows"] * case["heads"] * case["d"]
        size = (4 if case["dtype"] == "f32" else 2) + (4 if case["out"] == "f32" else 2)
        return {"bytes": int(n * size + 4 * case["rows"] + 4 * case["r"]), "flops": int(3 * case["rows"] * case["heads"] * case["r"])}
    B, Tq, Hq, d = case["B"], case["Tq"], case["Hq"], 512
    n = _tree_lengths(case)
    rows = B * Tq
    keys = Tq * (np.minimum(n, case["K"]).sum() + B * case["W"])
    # entries that several nodes select are read once: no more than the sequence has
    entries = np.minimum(n, Tq * np.minimum(n, case["K"])).sum()
    return {"bytes": int(entries * (516 if case["fp8"] else 288) + B * (case["W"] + Tq) * 516 + rows * (Hq * (4 * d + 4) + 4 * case["K"] + 12)),
            "flops": int(4 * d * Hq * keys)}


# ---- inputs ------------------------------------------------------------------------------

def _prepare_pages(case, seed):
    B, step, max_len = case["B"], case["step"], case["max_len"]
    r = np.random.RandomState(seed % (1 << 32))
    length = np.round(np.exp(r.uniform(0, math.log(max_len), B))).astype(np.int64)
    fresh = r.rand(B) < 0.2                                   # sequences that begin with this step
    length[fresh] = 0
    shift = np.where(r.rand(B) < 0.5, length // 4 // 3, 0) if case["shift"] else np.zeros(B, dtype=np.int64)
    n_new = r.randint(0, step + 1, B)
    ended = (r.rand(B) < case["ends"]) & ~fresh
    n_new[ended] = 4 * shift[ended] - length[ended]           # all pages back
    back = (r.rand(B) < 0.2) & ~ended                         # drafts of the last step that were rejected
    n_new[back] = -np.minimum(r.randint(0, 16, B), length - 4 * shift)[back]
    held = -(-(length // 4 - shift) // PAGE)
    max_pages = int((max_len + step) // 4 // PAGE + 2)
    need = -(-((length + n_new) // 4 - shift) // PAGE)
    wanted = int(np.maximum(need - held, 0).sum() - np.maximum(held - need, 0).sum())
    n_free = max(0, wanted * 3 // 4) if case["short"] else max(0, wanted) + 17
    n_pages = B * max_pages + 5                               # (a pool of the same size for every seed)
    n_free = min(n_free, n_pages - int(held.sum()))
    perm = r.permutation(n_pages).astype(np.int32)
    table = r.randint(0, n_pages, (B, max_pages)).astype(np.int32)    # rows hold old pages behind their last one
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(n_pages, -1, dtype=np.int32)
    free[:n_free] = perm[at:at + n_free]
    i32 = dict(dtype=torch.int32, device="cuda")
    first = torch.tensor(np.concatenate([length, held, [n_free]]), **i32)
    now = first.clone()
    return {"first": first, "now": now, "seq_len": now[:B], "held": now[B:2 * B], "n_free": now[2 * B:], "n_new": torch.tensor(n_new, **i32),
            "shift": torch.tensor(shift, **i32) if case["shift"] else None, "table": torch.tensor(table, **i32),
            "free": torch.tensor(free, **i32), "n_pages": n_pages, "step": step, "max_new": step // 4 + 1}


def _fp8(x):
    return x.to(torch.float8_e4m3fn)


def _blocks_of(x):
    """x [M][K] padded to whole blocks of 128 columns: [M][K/128][128]."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    if kb * BLOCK != K:
        x = torch.nn.functional.pad(x, (0, kb * BLOCK - K))
    return x.view(M, kb, BLOCK)


def _prepare_matmul(case, g):
    M, N, K = case["M"], case["N"], case["K"]
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    a = _hidden(M, K, g)
    x = _blocks_of(a)
    sa = x.abs().amax(-1).clamp_min(2.0 ** -100) / 448
    a = _fp8((x / sa.unsqueeze(-1)).reshape(M, -1)[:, :K].contiguous())
    b = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda")
    sb = torch.empty(nb, kb, device="cuda")
    for i in range(0, nb, 64):                   # weights of deviation 0.02, 8,192 rows at a time
        rows = min(N, (i + 64) * BLOCK) - i * BLOCK
        w = 0.02 * torch.randn(rows, K, device="cuda", generator=g)
        w = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, -rows % BLOCK)).view(-1, BLOCK, kb, BLOCK)
        s = w.abs().amax(dim=(1, 3)).clamp_min(2.0 ** -100) / 448
        sb[i:i + 64] = s
        w = (w / s[:, None, :, None]).view(-1, kb * BLOCK)[:rows, :K]
        b[i * BLOCK:i * BLOCK + rows] = _fp8(w)
    return {"a": a, "sa": sa.contiguous(), "b": b, "sb": sb, "out": torch.float32 if case["out"] == "f32" else torch.bfloat16}


def _hidden(M, K, g):
    """Hidden states: N(0, 1), one in a thousand ten times as large."""
    x = torch.randn(M, K, device="cuda", generator=g)
    return torch.where(torch.rand(M, K, device="cuda", generator=g) < 0.001, x * 10, x)


def _prepare_rope(case, g, seed):
    rows, heads, d = case["rows"], case["heads"], case["d"]
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}
    wide = torch.empty(rows, heads * d + case["extra"], dtype=dtype[case["dtype"]], device="cuda")
    for i in range(0, rows, 512):
        wide[i:i + 512] = torch.randn(min(512, rows - i), wide.shape[1], device="cuda", generator=g)
    # chunks of 128 tokens somewhere in their contexts
    r = np.random.RandomState(seed % (1 << 32))
    n = -(-rows // 128)
    pos = (r.randint(0, case["max_pos"] - 127, n)[:, None] + np.arange(128)).reshape(-1)[:rows]
    s = {"x": wide[:, :heads * d].unflatten(1, (heads, d)), "pos": torch.tensor(pos, dtype=torch.int32, device="cuda"), "r": case["r"],
         "start": case["start"], "layout": case["layout"], "scaling": case["scaling"], "inverse": case["inverse"], "base": 10000.0,
         "factor": 1.0, "original": 4096, "amplitude": 1.0, "out": dtype[case["out"]]}
    if case["scaling"] != "none":
        s["factor"] = 40.0 if case["scaling"] == "yarn" else 8.0
    if case["scaling"] == "yarn":
        s["amplitude"] = 0.1 * math.log(s["factor"]) + 1.0
    return s


def _fp8_rows(n, d, g):
    x = torch.randn(n, d, device="cuda", generator=g)
    sc = x.abs().amax(-1) / 448
    return _fp8(x / sc.unsqueeze(-1)).view(torch.uint8), sc


def _prepare_tree(case, g, seed):
    B, Tq, Hq, K, W, d = case["B"], case["Tq"], case["Hq"], case["K"], case["W"], 512
    r = np.random.RandomState(seed % (1 << 32))
    n = _tree_lengths(case)
    i32 = dict(dtype=torch.int32, device="cuda")
    per = (n + PAGE - 1) // PAGE
    pages = int(per.sum()) + 1
    perm = r.permutation(pages).astype(np.int32)
    table = np.zeros((B, int(per.max())), dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :per[b]] = perm[at:at + per[b]]
        at += per[b]
    slots = pages * PAGE
    if case["fp8"]:
        codes, scales = _fp8_rows(slots, d, g)
    else:
        codes = torch.empty(slots, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(slots, d // 16, dtype=torch.uint8, device="cuda")
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        for i in range(0, slots, 1 << 17):
            m = min(slots, i + (1 << 17)) - i
            x = torch.randn(m, d // 16, 16, device="cuda", generator=g)
            sc = _fp8(x.abs().amax(-1) / 6)
            scales[i:i + m] = sc.view(torch.uint8)
            x = x / sc.float().clamp_min(2.0 ** -9).unsqueeze(-1)
            c = (torch.bucketize(x.abs(), edges).to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)).view(m, d)
            codes[i:i + m] = c[:, 0::2] | (c[:, 1::2] << 4)
    ctx = 4 * n + np.arange(B) % 4               # committed tokens
    # node i continues one of the last nodes or of the committed text; ragged trees end before Tq
    parent = np.full((B, Tq), -2, dtype=np.int64)
    for b in range(B):
        count = Tq if not case["ragged"] or b == 0 else int(r.randint(1, Tq + 1))
        for i in range(count):
            parent[b, i] = i - 1 if case["chain"] else max(-1, i - 1 - int(r.geometric(0.4)))
    win_codes, win_scales = _fp8_rows(B * W, d, g)
    new_codes, new_scales = _fp8_rows(B * Tq, d, g)
    # the indexer's selection: K distinct entries of every node, ascending, -1 behind the last
    idx = torch.full((B, Tq, K), -1, **i32)
    for b in range(B):
        k = min(K, int(n[b]))
        pick = torch.rand(Tq, int(n[b]), device="cuda", generator=g).topk(k, dim=-1).indices
        idx[b, :, :k] = pick.sort(dim=-1).values.int()
    cnt = torch.tensor(np.minimum(n, K)[:, None].repeat(Tq, 1), **i32)
    return {"codes": codes, "scales": scales, "fp8": case["fp8"], "table": torch.tensor(table, **i32), "pages": pages,
            "n_entries": torch.tensor(n, **i32), "ctx": torch.tensor(ctx, **i32), "parent": torch.tensor(parent, **i32), "depth": Tq,
            "win_codes": win_codes.view(B, W, d), "win_scales": win_scales.view(B, W), "pos0": torch.tensor(ctx - W, **i32),
            "new_codes": new_codes.view(B, Tq, d), "new_scales": new_scales.view(B, Tq), "idx": idx, "cnt": cnt, "W": W,
            "Q": torch.randn(B, Tq, Hq, d, device="cuda", generator=g).bfloat16(), "scale": 1.0 / math.sqrt(d)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "pages":
        s = _prepare_pages(case, seed)
    elif op == "pack":
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s = {"x": _hidden(case["M"], case["K"] + case["extra"], g).to(dtype)[:, :case["K"]]}
    elif op == "matmul":
        s = _prepare_matmul(case, g)
    elif op == "rope":
        s = _prepare_rope(case, g, seed)
    else:
        s = _prepare_tree(case, g, seed)
    s["op"] = op
    return s


# ---- the library's calls -----------------------------------------------------------------

def _handle(s):
    """The descriptors, outputs and workspaces that a program builds once and keeps."""
    h = s.get("handle")
    if h is not None:
        return h
    from compressed_sparse_attention_05_gb300 import abi
    p = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    h, need = {"abi": abi}, 0
    if s["op"] == "pages":
        B, max_pages = s["table"].shape
        h["dims"] = abi.Dims(B=B, Tq=s["step"], max_pages=max_pages)
        h["pool"] = abi.PagePool(page_table=p(s["table"]), held=p(s["held"]), free_pages=p(s["free"]), n_free=p(s["n_free"]),
                                 n_pages=s["n_pages"])
        h["out"] = {"n_entries": torch.empty(B, **i32), "first_entry": torch.empty(B, **i32), "q_pos": torch.empty(B, s["step"], **i32),
                    "slots": torch.empty(B, s["max_new"], dtype=torch.int64, device="cuda"), "granted": torch.empty(B, **i32)}
        need = abi.csa2_page_plan_workspace_size(h["dims"])
    elif s["op"] == "pack":
        M, K = s["x"].shape
        h["codes"] = torch.empty(M, K, dtype=torch.uint8, device="cuda")
        h["scales"] = torch.empty(M, -(-K // BLOCK), device="cuda")
    elif s["op"] == "matmul":
        M, N = s["a"].shape[0], s["b"].shape[0]
        h["C"] = torch.empty(M, N, dtype=s["out"], device="cuda")
        need = abi.csa2_matmul_fp8_workspace_size(M, N, s["a"].shape[1])
    elif s["op"] == "rope":
        h["y"] = torch.empty(s["x"].shape, dtype=s["out"], device="cuda")
        kind = {"none": abi.ROPE_PLAIN, "linear": abi.ROPE_LINEAR, "ntk": abi.ROPE_NTK, "yarn": abi.ROPE_YARN}[s["scaling"]]
        spec = abi.RopeSpec(scaling=kind, base=s["base"], factor=s["factor"], original_len=s["original"], beta_fast=32.0, beta_slow=1.0)
        h["table"] = torch.empty(s["r"] // 2, dtype=torch.int64, device="cuda")
        abi.csa2_rope_table(spec, s["r"], h["table"])
        h["layout"] = abi.ROPE_HALF if s["layout"] == "half" else abi.ROPE_INTERLEAVED
    else:
        B, Tq, Hq, d = s["Q"].shape
        h["dims"] = abi.Dims(B=B, Tq=Tq, d=d, r=64, Hq=Hq, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=s["idx"].shape[2], W=s["W"],
                             max_pages=s["table"].shape[1], swa_cap=s["win_codes"].shape[1],
                             kv_format=abi.CSA2_KV_FP8 if s["fp8"] else abi.CSA2_KV_MXFP4)
        h["cache"] = abi.Cache(kv_codes=p(s["codes"]), kv_scales=p(s["scales"]), page_table=p(s["table"]), n_entries=p(s["n_entries"]),
                               n_pages=s["pages"])
        h["window"] = abi.Window(codes=p(s["win_codes"]), scales=p(s["win_scales"]), pos0=p(s["pos0"]))
        h["q_pos"], h["path"] = torch.empty(B, Tq, **i32), torch.empty(B, Tq, s["depth"], **i32)
        h["tree"] = abi.Tree(codes=p(s["new_codes"]), scales=p(s["new_scales"]), ctx_len=p(s["ctx"]), path=p(h["path"]), max_depth=s["depth"])
        h["O"] = torch.empty(B, Tq, Hq, d, dtype=torch.bfloat16, device="cuda")
        h["lse"] = torch.empty(B, Tq, Hq, device="cuda")
    h["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    s["handle"] = h
    return h


def run(s):
    op = s["op"]
    if op == "pages":
        s["now"].copy_(s["first"])           # every pass plans from the same state
        if not own:
            return _plain_pages(s)
        h = _handle(s)
        h["abi"].csa2_page_plan(h["dims"], h["pool"], s["seq_len"], s["n_new"], s["seq_len"], h["out"]["n_entries"], h["out"]["first_entry"],
                                h["ws"], shift=s["shift"], q_pos=h["out"]["q_pos"], slots=h["out"]["slots"], granted=h["out"]["granted"])
        return {"table": s["table"], "free": s["free"], "n_free": s["n_free"], "held": s["held"], "seq_len": s["seq_len"], **h["out"]}
    if not own:
        return {"pack": _plain_pack, "matmul": _plain_matmul, "rope": _plain_rope, "tree": _plain_tree}[op](s)
    h = _handle(s)
    if op == "pack":
        h["abi"].csa2_pack_fp8_blocks(s["x"], h["codes"], h["scales"])
        return {"codes": h["codes"].view(torch.float8_e4m3fn), "scales": h["scales"]}
    if op == "matmul":
        h["abi"].csa2_matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], h["C"], h["ws"])
        return {"C": h["C"]}
    if op == "rope":
        h["abi"].csa2_rope(s["x"], h["y"], s["pos"], h["table"], start=s["start"], layout=h["layout"], inverse=s["inverse"],
                           amplitude=s["amplitude"])
        return {"y": h["y"]}
    h["abi"].csa2_tree_plan(h["dims"], s["parent"], s["ctx"], h["q_pos"], h["path"])
    h["abi"].csa2_tree_attn(h["dims"], h["cache"], h["window"], h["tree"], s["Q"], h["q_pos"], s["idx"], s["cnt"], s["scale"], h["O"], h["lse"])
    return {"q_pos": h["q_pos"], "O": h["O"], "lse": h["lse"]}


# ---- the plain forms ---------------------------------------------------------------------

def _plain_pages(s):
    B, max_pages = s["table"].shape
    n_pages, step = s["n_pages"], s["step"]
    length, n_new, held = s["seq_len"].long(), s["n_new"].long(), s["held"].long()
    n_free = s["n_free"].long()
    shift = s["shift"].long() if s["shift"] is not None else torch.zeros_like(length)
    e0, e1 = length // 4 - shift, (length + n_new) // 4 - shift
    need = (e1 + PAGE - 1) // PAGE
    back, want = (held - need).clamp_min(0), (need - held).clamp_min(0)
    R = back.sum()
    granted = (want.cumsum(0) <= n_free + R) | (want == 0)
    take = torch.where(granted, want, 0)
    G = take.sum()
    p = torch.arange(max_pages, device="cuda").unsqueeze(0)
    # the stack with the released pages on top (a spare place behind it for all others)
    stack = torch.cat([s["free"], s["free"][:1]])
    leaves = (p >= need.unsqueeze(-1)) & (p < held.unsqueeze(-1))
    at = n_free + (back.cumsum(0) - back).unsqueeze(-1) + p - need.unsqueeze(-1)
    stack = stack.scatter(0, torch.where(leaves, at, n_pages).view(-1), s["table"].view(-1))
    comes = granted.unsqueeze(-1) & (p >= held.unsqueeze(-1)) & (p < need.unsqueeze(-1))
    at = n_free + R - 1 - (take.cumsum(0) - take).unsqueeze(-1) - (p - held.unsqueeze(-1))
    table = torch.where(comes, stack[at.clamp(0, n_pages - 1)], s["table"])
    left = n_free + R - G
    free = torch.where(torch.arange(n_pages, device="cuda") < left, stack[:n_pages], s["free"])
    first = torch.minimum(e0, e1)
    i = torch.arange(step, device="cuda").unsqueeze(0)
    q_pos = torch.where(granted.unsqueeze(-1) & (i < n_new.unsqueeze(-1)), length.unsqueeze(-1) + i, -1)
    i = torch.arange(s["max_new"], device="cuda").unsqueeze(0)
    e = e0.unsqueeze(-1) + i
    slot = table.gather(1, (e // PAGE).clamp(0, max_pages - 1)).long() * PAGE + e % PAGE
    slots = torch.where(granted.unsqueeze(-1) & (e < e1.unsqueeze(-1)), slot, -1)
    return {"table": table, "free": free, "n_free": left.int(), "held": torch.where(granted, need, held).int(),
            "seq_len": torch.where(granted, length + n_new, length).int(), "n_entries": torch.where(granted, e1, e0).int(),
            "first_entry": torch.where(granted, first, e0).int(), "q_pos": q_pos.int(), "slots": slots, "granted": granted.int()}


def _plain_pack(s):
    M, K = s["x"].shape
    x = _blocks_of(s["x"].float())
    a = x.abs().amax(-1).clamp_min(2.0 ** -100)
    top = torch.full_like(a, 448.0)          # (a scalar in its place would be multiplied by a rounded reciprocal)
    q = x * (top / a).unsqueeze(-1)
    return {"codes": _fp8(q.clamp(-448, 448).view(M, -1)[:, :K]), "scales": a / top}


def _plain_matmul(s):
    M, N, K = s["a"].shape[0], s["b"].shape[0], s["a"].shape[1]
    a = (_blocks_of(s["a"].float()) * s["sa"].unsqueeze(-1)).view(M, -1)[:, :K]
    b = s["b"].float()
    sb = s["sb"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return {"C": (a @ (b * sb).t()).to(s["out"])}


def _frequencies(s):
    """theta_i of the pairs, fp64."""
    r, base, f = s["r"], s["base"], s["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if s["scaling"] == "ntk":
        base = base * f ** (r / (r - 2))
    theta = base ** (-2 * i / r)
    if s["scaling"] == "linear":
        theta = theta / f
    if s["scaling"] == "yarn":
        lo, hi = (r * math.log(s["original"] / (beta * 2 * math.pi)) / (2 * math.log(base)) for beta in (32.0, 1.0))
        lo, hi = max(0, math.floor(lo)), min(r - 1, math.ceil(hi))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        theta = theta / f * ramp + theta * (1 - ramp)
    return theta


def _plain_rope(s):
    r, a = s["r"], s["start"]
    x = s["x"].float()
    angle = s["pos"].double().unsqueeze(-1) * _frequencies(s)
    c = (s["amplitude"] * torch.cos(angle)).float().unsqueeze(1)
    n = (s["amplitude"] * torch.sin(angle)).float().unsqueeze(1)
    if s["inverse"]:
        n = -n
    part = x[..., a:a + r]
    if s["layout"] == "half":
        x1, x2 = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat([x1 * c - x2 * n, x1 * n + x2 * c], dim=-1)
    else:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([x1 * c - x2 * n, x1 * n + x2 * c], dim=-1).flatten(-2)
    return {"y": torch.cat([x[..., :a], turned, x[..., a + r:]], dim=-1).to(s["out"])}


def _window_value(codes, scales):
    return (codes.view(torch.float8_e4m3fn).float() * scales.unsqueeze(-1)).bfloat16().float()


def _plain_tree(s):
    B, Tq, Hq, d = s["Q"].shape
    K, W = s["idx"].shape[2], s["W"]
    # depths and ancestors, one level after the other
    parent, ctx = s["parent"].long(), s["ctx"].long()
    node = torch.arange(Tq, device="cuda").expand(B, Tq)
    live = parent >= -1
    depth = torch.zeros_like(parent)
    up, above = node, []
    for _ in range(Tq):
        above.append(up)                                     # the ancestor so many levels up, -1 behind the root
        step = torch.where(up >= 0, parent.gather(1, up.clamp_min(0)), -1)
        up = torch.where(live, step, -1)
        depth += (up >= 0)
    q_pos = torch.where(live, ctx.unsqueeze(-1) + depth, -1)
    # keys: the selected entries, the committed window rows, then the ancestors by distance
    at = s["idx"].long().clamp_min(0)
    slots = s["table"].long().gather(1, (at // PAGE).view(B, -1)).view(B, Tq, K) * PAGE + at % PAGE
    if s["fp8"]:
        keys = _window_value(s["codes"][slots], s["scales"][slots])
    else:
        values = torch.tensor(_E2M1 + [-v for v in _E2M1], device="cuda")
        c = s["codes"][slots]
        keys = torch.stack([values[(c & 15).int()], values[(c >> 4).int()]], dim=-1).view(B, Tq, K, d // 16, 16)
        keys = (keys * s["scales"][slots].view(torch.float8_e4m3fn).float().unsqueeze(-1)).view(B, Tq, K, d)
    k = torch.arange(K, device="cuda")
    seen = [(k < s["cnt"].unsqueeze(-1)) & (4 * s["idx"].long() + 3 <= q_pos.unsqueeze(-1)) & (s["idx"] >= 0)]
    old = _window_value(s["win_codes"], s["win_scales"])
    p = s["pos0"].long().unsqueeze(-1) + torch.arange(old.shape[1], device="cuda")
    p = p.unsqueeze(1)
    t = q_pos.unsqueeze(-1)
    seen.append((p >= 0) & (p > t - W) & (p <= t) & (p < ctx.view(B, 1, 1)))
    new = _window_value(s["new_codes"], s["new_scales"])
    above = torch.stack(above, dim=-1)                       # [B][Tq][levels]
    seen.append((above >= 0) & (torch.arange(Tq, device="cuda") < W))
    seen = [m & live.unsqueeze(-1) for m in seen]
    Q = s["Q"].float()
    x = torch.cat([Q @ keys.transpose(2, 3), Q @ old.unsqueeze(1).transpose(2, 3),
                   (Q @ new.unsqueeze(1).transpose(2, 3)).gather(3, above.clamp_min(0).unsqueeze(2).expand(B, Tq, Hq, Tq))], dim=-1) * s["scale"]
    x = torch.where(torch.cat(seen, dim=-1).unsqueeze(2), x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    l = e.sum(-1, keepdim=True)
    w = e / torch.where(l == 0, torch.ones_like(l), l)
    nw = old.shape[1]
    by_node = torch.zeros(B, Tq, Hq, Tq, device="cuda").scatter_add_(3, above.clamp_min(0).unsqueeze(2).expand(B, Tq, Hq, Tq), w[..., K + nw:])
    o = w[..., :K] @ keys + w[..., K:K + nw] @ old.unsqueeze(1) + by_node @ new.unsqueeze(1)
    return {"q_pos": q_pos.int(), "O": o.bfloat16(), "lse": (m + torch.log(l)).squeeze(-1)}


# ---- from the definitions, in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "pack": _exact_pack, "matmul": _exact_matmul, "rope": _exact_rope, "tree": _exact_tree}[s["op"]](s)


def _exact_pages(s):
    host = lambda t: t.cpu().numpy().astype(np.int64)  # noqa: E731
    table, free, length, held, n_new = (host(s[k]) for k in ("table", "free", "seq_len", "held", "n_new"))
    B = len(length)
    shift = host(s["shift"]) if s["shift"] is not None else np.zeros(B, dtype=np.int64)
    stack = free[:int(s["n_free"])].tolist()
    old = length.copy()
    after = [(length[b] + n_new[b]) // 4 - shift[b] for b in range(B)]
    need = [(a + PAGE - 1) // PAGE for a in after]
    for b in range(B):                                       # pages come back
        for k in range(need[b], held[b]):
            stack.append(table[b, k])
        held[b] = min(held[b], need[b])
    out = {"n_entries": np.zeros(B, dtype=np.int64), "first_entry": np.zeros(B, dtype=np.int64), "granted": np.zeros(B, dtype=np.int64),
           "q_pos": np.full((B, s["step"]), -1, dtype=np.int64), "slots": np.full((B, s["max_new"]), -1, dtype=np.int64)}
    stuck = False
    for b in range(B):
        e0 = old[b] // 4 - shift[b]
        want = need[b] - held[b]
        stuck = stuck or want > len(stack)                   # who waits is not overtaken
        if stuck and want > 0:
            out["n_entries"][b] = out["first_entry"][b] = e0
            continue
        for k in range(held[b], need[b]):
            table[b, k] = stack.pop()
        held[b] = need[b]
        length[b] = old[b] + n_new[b]
        out["granted"][b], out["n_entries"][b], out["first_entry"][b] = 1, after[b], min(e0, after[b])
        k = max(0, n_new[b])
        out["q_pos"][b, :k] = old[b] + np.arange(k)
        e = np.arange(e0, max(e0, after[b]))
        out["slots"][b, :len(e)] = table[b, e // PAGE] * PAGE + e % PAGE
    free[:len(stack)] = stack
    out.update(table=table, free=free, held=held, seq_len=length, n_free=np.array([len(stack)]))
    kind = {k: torch.int64 if k == "slots" else torch.int32 for k in out}
    order = ("table", "free", "n_free", "held", "seq_len", "n_entries", "first_entry", "q_pos", "slots", "granted")
    return {k: torch.tensor(out[k], dtype=kind[k], device="cuda") for k in order}


def _e4m3_value(code):
    """E4M3 by its formula: sign, exponent of bias 7, 3 bits of mantissa."""
    c = code.view(torch.uint8).int()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.pow(2.0, e.double() - 7) * (1 + m / 8))
    return torch.where(c >= 128, -v, v)


def _exact_pack(s):
    """The nearest E4M3 value (the even one of two) of fp32(x * fp32(448 / amax))."""
    M, K = s["x"].shape
    codes, scales = torch.empty(M, K, dtype=torch.float64, device="cuda"), torch.empty(M, -(-K // BLOCK), dtype=torch.float64, device="cuda")
    for k in range(0, K, BLOCK):
        x = s["x"][:, k:k + BLOCK].double()
        a = x.abs().max(dim=1).values.clamp_min(2.0 ** -100)
        scales[:, k // BLOCK] = a / 448
        q = (x * (448 / a).float().double()[:, None]).float().double()
        # steps of 2^(e-3) in [2^e, 2^(e+1)), of 2^-9 below 2^-6
        e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6)))
        e = torch.where(torch.pow(2.0, e + 1) <= q.abs(), e + 1, e)
        e = torch.where((torch.pow(2.0, e) > q.abs()) & (e > -6), e - 1, e)
        h = torch.pow(2.0, e - 3)
        codes[:, k:k + BLOCK] = (torch.round(q / h) * h).clamp(-448, 448)
    return {"codes": codes, "scales": scales}


def _exact_matmul(s):
    M, K = s["a"].shape
    N = s["b"].shape[0]
    C = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    k = torch.arange(K, device="cuda") // BLOCK
    a = _e4m3_value(s["a"]) * s["sa"].double()[:, k]
    for i in range(0, N, 4096):
        j = torch.arange(i, min(N, i + 4096), device="cuda") // BLOCK
        C[:, i:i + 4096] = a @ (_e4m3_value(s["b"][i:i + 4096]) * s["sb"].double()[j][:, k]).t()
    return {"C": C}


def _exact_rope(s):
    r, a = s["r"], s["start"]
    freq = []
    for i in range(r // 2):
        b = s["base"] * s["factor"] ** (r / (r - 2)) if s["scaling"] == "ntk" else s["base"]
        w = 1.0 / b ** (2 * i / r)
        if s["scaling"] == "linear":
            w /= s["factor"]
        if s["scaling"] == "yarn":
            # pairs that turn more than 32 times in the original context stay, those below one turn are stretched
            at = [r / 2 * math.log(s["original"] / (2 * math.pi * n)) / math.log(s["base"]) for n in (32, 1)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w * (1 - share) + w / s["factor"] * share
        freq.append(w)
    angle = s["pos"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), -angle if s["inverse"] else angle)[:, None, :]
    y = s["x"].double().clone()
    part = y[..., a:a + r]
    z = torch.complex(part[..., :r // 2], part[..., r // 2:]) if s["layout"] == "half" else torch.complex(part[..., 0::2], part[..., 1::2])
    z = z * turn
    if s["layout"] == "half":
        y[..., a:a + r // 2], y[..., a + r // 2:a + r] = z.real, z.imag
    else:
        y[..., a:a + r:2], y[..., a + 1:a + r:2] = z.real, z.imag
    return {"y": y}


def _exact_tree(s):
    B, Tq, Hq, d = s["Q"].shape
    O = torch.zeros(B, Tq, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Tq, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    q_pos = torch.full((B, Tq), -1, dtype=torch.int32)
    parent, ctx, cnt, table, pos0 = s["parent"].tolist(), s["ctx"].tolist(), s["cnt"].tolist(), s["table"].long(), s["pos0"].tolist()

    def row(codes, scales):                      # a window operand is a bf16 value by definition
        return (_e4m3_value(codes).float() * scales[..., None]).bfloat16().double()

    for b in range(B):
        old, new = row(s["win_codes"][b], s["win_scales"][b]), row(s["new_codes"][b], s["new_scales"][b])
        line = {}
        for i in range(Tq):
            if parent[b][i] < -1:
                continue
            line[i] = (line[parent[b][i]] if parent[b][i] >= 0 else []) + [i]
            t = ctx[b] + len(line[i]) - 1
            q_pos[b, i] = t
            j = s["idx"][b, i, :cnt[b][i]].long()
            j = j[4 * j + 3 <= t]
            at = table[b, j // PAGE] * PAGE + j % PAGE
            if s["fp8"]:
                keys = row(s["codes"][at], s["scales"][at])
            else:
                c = s["codes"][at].int()
                c = torch.stack([c & 15, c >> 4], dim=-1).flatten(1)
                e, m = (c >> 1) & 3, (c & 1).double()
                mag = torch.where(e == 0, 0.5 * m, torch.pow(2.0, e.double() - 1) * (1 + 0.5 * m))
                keys = torch.where(c >= 8, -mag, mag) * _e4m3_value(s["scales"][at]).repeat_interleave(16, dim=1)
            lo = max(0, t - s["W"] + 1, pos0[b])
            hi = min(ctx[b], pos0[b] + old.shape[0])
            mine = line[i][max(0, t - s["W"] + 1 - ctx[b]):]
            keys = torch.cat([keys, old[lo - pos0[b]:max(lo, hi) - pos0[b]], new[mine]])
            x = s["Q"][b, i].double() @ keys.t() * s["scale"]
            lse[b, i] = torch.logsumexp(x, dim=-1)
            O[b, i] = torch.softmax(x, dim=-1) @ keys
    return {"q_pos": q_pos.cuda(), "O": O, "lse": lse}
