"""The query side's entry points refuse bad calls on the host, before any launch (no GPU needed)."""
import ctypes as C
import math

import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build

FAKE = 1 << 20   # an aligned non-null address; validation fails before any use


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.lib()


def err():
    return abi.lib().csa2_last_error().decode()


def ref(x):
    return C.byref(x) if x is not None else None


def dims(**kw):
    d = dict(B=2, Tq=3, d=512, r=64, Hq=64, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=512, W=128, max_pages=4, swa_cap=130)
    d.update(kw)
    return abi.Dims(**d)


def pool(**kw):
    d = dict(page_table=FAKE, held=FAKE, free_pages=FAKE, n_free=FAKE, n_pages=9)
    d.update(kw)
    return abi.PagePool(**d)


def plan(lib, dm=None, pl=None, max_new=4, ws=FAKE, nbytes=1 << 30, **kw):
    a = dict(seq_len=FAKE, n_new=FAKE, shift=FAKE, out=FAKE, n_entries=FAKE, first=FAKE, q_pos=FAKE, slots=FAKE, granted=FAKE)
    a.update(kw)
    return lib.csa2_page_plan(ref(dm or dims()), ref(pl or pool()), a["seq_len"], a["n_new"], a["shift"], max_new, a["out"], a["n_entries"],
                              a["first"], a["q_pos"], a["slots"], a["granted"], ws, nbytes, None)


def test_page_plan(lib):
    for bad in (dict(B=-1), dict(Tq=-1), dict(max_pages=0)):
        assert plan(lib, dims(**bad)) == 1, bad
    for bad in (dict(page_table=None), dict(held=None), dict(free_pages=None), dict(n_free=None), dict(page_table=FAKE + 2), dict(n_pages=0),
                dict(n_pages=1 << 31)):
        assert plan(lib, pl=pool(**bad)) == 1, bad
    for k in ("seq_len", "n_new", "out", "n_entries", "first"):
        assert plan(lib, **{k: None}) == 1 and "NULL" in err()
    for k in ("seq_len", "shift", "q_pos", "granted"):
        assert plan(lib, **{k: FAKE + 2}) == 1 and "aligned" in err()
    assert plan(lib, slots=FAKE + 4) == 1 and "slots" in err()
    assert plan(lib, max_new=-1) == 1 and "max_new" in err()
    need = abi.csa2_page_plan_workspace_size(dims())
    assert plan(lib, ws=None) == 4 and plan(lib, nbytes=need - 1) == 4 and plan(lib, ws=FAKE + 8) == 1
    assert plan(lib, dims(B=0)) == 0 and lib.csa2_page_plan_workspace_size(None) == 0
    assert lib.csa2_page_plan(None, ref(pool()), *[FAKE] * 3, 1, *[FAKE] * 6, FAKE, 1 << 30, None) == 1
    assert lib.csa2_page_plan(ref(dims()), None, *[FAKE] * 3, 1, *[FAKE] * 6, FAKE, 1 << 30, None) == 1


def test_pack(lib):
    call = lambda x=FAKE, t=0, stride=128, n=2, K=128, c=FAKE, s=FAKE: lib.csa2_pack_fp8_blocks(x, t, stride, n, K, c, s, None)  # noqa: E731
    assert call(t=2) == 1 and "dtype" in err()
    assert call(n=-1) == 1 and call(n=1 << 31) == 1
    for K in (0, -16, 8, 100):
        assert call(K=K, stride=256) == 1 and "multiple of 16" in err()
    assert call(stride=127) == 1 and call(stride=130) == 1 and call(stride=132, t=abi.CSA2_BF16) == 1 and "row_stride" in err()
    assert call(x=None) == 1 and call(x=FAKE + 8) == 1 and call(c=FAKE + 1) == 1 and call(s=None) == 1
    assert call(n=0, x=None) == 0


def test_matmul(lib):
    call = lambda M=2, N=3, K=32, A=FAKE, sa=FAKE, B=FAKE, sb=FAKE, c=FAKE, t=1, ws=FAKE, n=1 << 40: lib.csa2_matmul_fp8(  # noqa: E731
        A, sa, B, sb, M, N, K, c, t, ws, n, None)
    assert call(M=-1) == 1 and call(N=-1) == 1 and call(M=(1 << 30) + 1) == 1 and call(K=(1 << 30) + 16) == 1
    for K in (0, -16, 24, 1000):
        assert call(K=K) == 1 and "multiple of 16" in err()
    assert call(t=5) == 1 and "c_dtype" in err()
    for k in ("A", "sa", "B", "sb", "c"):
        assert call(**{k: None}) == 1 and call(**{k: FAKE + 4}) == 1, k
    need = abi.csa2_matmul_fp8_workspace_size(8, 256, 4096)
    assert need > 0 and call(M=8, N=256, K=4096, ws=None) == 4 and call(M=8, N=256, K=4096, n=need - 1) == 4
    assert call(M=8, N=256, K=4096, ws=FAKE + 8) == 1
    assert abi.csa2_matmul_fp8_workspace_size(4096, 4096, 4096) == 0 and abi.csa2_matmul_fp8_workspace_size(0, 5, 16) == 0
    assert call(M=0, A=None) == 0 and call(N=0, c=None) == 0


def spec(**kw):
    d = dict(scaling=abi.ROPE_YARN, original_len=4096, base=10000.0, factor=4.0, beta_fast=32.0, beta_slow=1.0)
    d.update(kw)
    return abi.RopeSpec(**d)


def test_rope_table(lib):
    call = lambda r=64, t=FAKE, **kw: lib.csa2_rope_table(ref(spec(**kw)), r, t, None)  # noqa: E731
    assert lib.csa2_rope_table(None, 64, FAKE, None) == 1
    for r in (-2, 3, 2050):
        assert call(r) == 1 and "even" in err()
    for bad in (dict(scaling=4), dict(scaling=-1), dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(factor=0.5),
                dict(factor=math.inf), dict(factor=math.nan), dict(original_len=0), dict(beta_slow=0.0), dict(beta_fast=0.5),
                dict(beta_fast=math.inf), dict(beta_slow=math.nan)):
        assert call(**bad) == 1, bad
    assert call(2, scaling=abi.ROPE_NTK) == 1 and call(4, scaling=abi.ROPE_NTK, base=1e300, factor=1e300) == 1
    assert call(t=None) == 1 and call(t=FAKE + 4) == 1
    assert call(0, t=None) == 0


def test_rope(lib):
    def call(**kw):
        a = dict(x=FAKE, xt=1, xts=128, xhs=64, y=2 * FAKE, yt=1, yts=128, yhs=64, n=4, heads=2, d=64, start=32, r=32, layout=0, inv=0,
                 amp=1.0, pos=FAKE, table=FAKE)
        a.update(kw)
        return lib.csa2_rope(a["x"], a["xt"], a["xts"], a["xhs"], a["y"], a["yt"], a["yts"], a["yhs"], a["n"], a["heads"], a["d"], a["start"],
                             a["r"], a["layout"], a["inv"], a["amp"], a["pos"], a["table"], None)
    for bad in (dict(xt=2), dict(yt=-1), dict(n=-1), dict(n=1 << 31), dict(heads=-1), dict(heads=65536), dict(d=0), dict(d=65537),
                dict(r=31), dict(r=-2), dict(r=2050, d=2200), dict(start=-1), dict(start=33), dict(layout=2), dict(amp=math.nan),
                dict(amp=math.inf), dict(xts=-1), dict(xhs=-64), dict(yts=63), dict(yhs=63), dict(x=None), dict(y=None), dict(x=FAKE + 1),
                dict(yt=0, y=FAKE + 2), dict(pos=None), dict(pos=FAKE + 2), dict(table=None), dict(table=FAKE + 4)):
        assert call(**bad) == 1, bad
    for bad in (dict(yts=64), dict(yts=127), dict(heads=3), dict(yts=64, yhs=255), dict(yts=1 << 62, yhs=1 << 62, n=(1 << 31) - 1, heads=65535)):
        assert call(**bad) == 1 and "overlap" in err(), bad                   # tokens and heads that share rows of y
    for bad in (dict(xts=256), dict(xhs=128, xts=256, yhs=64), dict(yt=0)):   # in place, but not the same layout or type
        assert call(**{**bad, "y": FAKE}) == 1 and "in place" in err()
    assert call(n=0, x=None) == 0 and call(heads=0, y=None) == 0
    assert call(y=FAKE, r=0, table=None) == 0                                 # in place, nothing rotated: no launch


def test_tree_plan(lib):
    call = lambda dm=None, p=FAKE, c=FAKE, depth=3, q=FAKE, path=FAKE: lib.csa2_tree_plan(ref(dm or dims()), p, c, depth, q, path, None)  # noqa: E731
    assert lib.csa2_tree_plan(None, FAKE, FAKE, 3, FAKE, FAKE, None) == 1
    assert call(dims(Tq=1025)) == 2 and "1024" in err()
    assert call(dims(B=-1)) == 1 and call(depth=0) == 1 and "max_depth" in err()
    for k in ("p", "c", "q", "path"):
        assert call(**{k: None}) == 1 and call(**{k: FAKE + 2}) == 1
    assert call(dims(B=0)) == 0 and call(dims(Tq=0), p=None) == 0


def tree(**kw):
    d = dict(codes=FAKE, scales=FAKE, ctx_len=FAKE, path=FAKE, max_depth=3)
    d.update(kw)
    return abi.Tree(**d)


WIN = abi.Window(codes=FAKE, scales=FAKE, pos0=FAKE)


def test_tree_attn(lib):
    def call(dm=None, win=WIN, tr=None, scale=0.1, n_pages=8, **kw):
        a = dict(Q=FAKE, q_pos=FAKE, idx=FAKE, cnt=FAKE, O=FAKE, lse=FAKE, codes=FAKE, table=FAKE)
        a.update(kw)
        c = abi.Cache(kv_codes=a["codes"], kv_scales=FAKE, page_table=a["table"], n_entries=FAKE, n_pages=n_pages)
        return lib.csa2_tree_attn(ref(dm or dims()), ref(c), ref(win), ref(tr or tree()), a["Q"], a["q_pos"], a["idx"], a["cnt"], scale,
                                  a["O"], a["lse"], None)
    assert call(dims(d=256)) == 2 and call(dims(d=64, kv_format=abi.CSA2_KV_FP8)) == 2
    for bad in (dict(Hq=0), dict(Hq=129), dict(K=0), dict(K=2049), dict(W=-1), dict(W=1025), dict(swa_cap=-1), dict(B=-1), dict(Tq=-1),
                dict(max_pages=0), dict(kv_format=3), dict(B=1 << 24, swa_cap=130), dict(B=1 << 20, Tq=256, swa_cap=0),
                dict(d=64, B=256, Tq=256)):
        assert call(dims(**bad)) == 1, bad
    for bad in (dict(codes=None), dict(scales=None), dict(scales=FAKE + 4), dict(ctx_len=None), dict(path=None), dict(path=FAKE + 2),
                dict(max_depth=0)):
        assert call(tr=tree(**bad)) == 1, bad
    for k in ("Q", "q_pos", "idx", "cnt", "O", "codes", "table"):
        assert call(**{k: None}) == 1, k
    assert call(Q=FAKE + 2) == 1 and call(O=FAKE + 8) == 1 and call(lse=FAKE + 4) == 1
    assert call(scale=math.nan) == 1 and call(scale=math.inf) == 1 and "finite" in err()
    assert call(n_pages=0) == 1 and call(n_pages=1 << 31) == 1
    assert call(win=None) == 1 and call(win=abi.Window(codes=FAKE, scales=None, pos0=FAKE)) == 1
    assert lib.csa2_tree_attn(ref(dims()), ref(abi.Cache()), ref(WIN), None, *[FAKE] * 4, 0.1, FAKE, FAKE, None) == 1
    assert call(dims(B=0), win=None) == 0 and call(dims(Tq=0), Q=None) == 0


def test_binding_refuses_tensors_it_cannot_describe():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        abi.csa2_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        abi.csa2_pack_fp8_blocks(torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1))
    assert abi._float_type(x) == abi.CSA2_F32
    with pytest.raises(ValueError, match="same shape"):
        abi.csa2_rope(x, x[:3], torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError, match="same shape"):
        abi.csa2_pack_fp8_blocks(torch.zeros(4, 64), torch.zeros(4, 80, dtype=torch.uint8), torch.zeros(4, 1))
    u8 = lambda *n: torch.zeros(*n, dtype=torch.uint8)  # noqa: E731
    for b, c in ((u8(5, 48), torch.zeros(4, 5)), (u8(5, 32), torch.zeros(5, 4)), (u8(5, 32), torch.zeros(20))):
        with pytest.raises(ValueError, match="fit together"):
            abi.csa2_matmul_fp8(u8(4, 32), torch.zeros(4, 1), b, torch.zeros(1, 1), c)
    with pytest.raises(ValueError, match="bfloat16"):
        abi._float_type(x.half())
