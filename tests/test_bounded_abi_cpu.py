"""The bounded-cache entry points refuse bad calls on the host, before any launch (no GPU needed)."""
import ctypes as C
import math

import pytest

from compressed_sparse_attention_05_gb300 import abi, build

FAKE = 1 << 20   # an aligned non-null address; validation fails before any use


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.lib()


def err():
    return abi.lib().csa2_last_error().decode()


def dims(**kw):
    d = dict(B=2, Tq=3, d=512, r=64, Hq=64, Hi=8, Di=128, idx_dtype=abi.CSA2_BF16, K=512, W=128, max_pages=4,
             n_pool_blocks=0, pool_block=8, swa_cap=130)
    d.update(kw)
    return abi.Dims(**d)


def cache(**kw):
    d = dict(kv_codes=FAKE, kv_scales=FAKE, idx_k=FAKE, page_table=FAKE, n_entries=FAKE, n_pages=8)
    d.update(kw)
    return abi.Cache(**d)


WIN = abi.Window(codes=FAKE, scales=FAKE, pos0=FAKE)
BOUNDED = abi.Bounded(entry_pos=FAKE, weight=FAKE, shift=FAKE)
NO_MODS = abi.ScoreMods()


def attn(lib, dm=None, c=None, bd=None, win=WIN, mods=None, Q=FAKE, q_pos=FAKE, scale=0.1, n=100, O=FAKE, lse=None,
         ws=FAKE, nbytes=1 << 40):
    r = lambda x: C.byref(x) if x is not None else None  # noqa: E731
    return lib.csa2_dense_attn(r(dm or dims()), r(c or cache()), r(bd), r(win), r(mods), Q, q_pos, scale, n, O, lse, ws,
                               nbytes, None)


def weights(lib, dm=None, c=None, bd=None, mods=None, Q=FAKE, q_pos=FAKE, lse=FAKE, scale=0.1, decay=1.0, w_in=FAKE,
            w_out=FAKE, n=100, ws=FAKE, nbytes=1 << 40):
    r = lambda x: C.byref(x) if x is not None else None  # noqa: E731
    return lib.csa2_entry_weights(r(dm or dims()), r(c or cache()), r(bd), r(mods), Q, q_pos, lse, scale, decay, w_in,
                                  w_out, n, ws, nbytes, None)


def evict(lib, dm=None, c=None, bd=BOUNDED, n_entries=FAKE, keep=10, sink=1, recent=2, n=100, ws=FAKE, nbytes=1 << 40):
    r = lambda x: C.byref(x) if x is not None else None  # noqa: E731
    return lib.csa2_evict(r(dm or dims()), r(c or cache()), r(bd), n_entries, keep, sink, recent, n, ws, nbytes, None)


@pytest.mark.parametrize("call", [attn, weights], ids=["attn", "weights"])
def test_shared_refusals(lib, call):
    assert call(lib, dims(d=256)) == 2 and "d must be" in err()
    assert call(lib, dims(kv_format=abi.CSA2_KV_FP8)) == 2 and "MXFP4" in err()
    for bad in (dict(Hq=0), dict(Hq=129), dict(W=-1), dict(W=1025), dict(swa_cap=-1), dict(B=-1), dict(Tq=-1),
                dict(max_pages=0), dict(B=70000), dict(Tq=1 << 30)):
        assert call(lib, dims(**bad)) == 1, bad
    assert call(lib, n=-1) == 1 and "max_entries" in err()
    assert call(lib, scale=math.nan) == 1 and call(lib, scale=math.inf) == 1 and "finite" in err()
    for cap in (-1.0, math.inf, math.nan):
        assert call(lib, mods=abi.ScoreMods(logit_cap=cap)) == 1 and "logit_cap" in err()
    assert call(lib, mods=abi.ScoreMods(slopes=FAKE + 2)) == 1 and "slopes" in err()
    assert call(lib, mods=abi.ScoreMods(doc_start=FAKE + 1)) == 1 and "doc_start" in err()
    assert call(lib, mods=abi.ScoreMods(prefix_len=FAKE + 1)) == 1 and "prefix_len" in err()
    assert call(lib, bd=abi.Bounded(entry_pos=FAKE + 1)) == 1 and "entry_pos" in err()
    assert call(lib, c=cache(kv_codes=None)) == 1 and call(lib, c=cache(kv_scales=FAKE + 8)) == 1
    assert call(lib, c=cache(page_table=None)) == 1 and call(lib, c=cache(n_entries=None)) == 1
    assert call(lib, c=cache(n_pages=0)) == 1 and call(lib, c=cache(n_pages=1 << 40)) == 1
    assert call(lib, Q=None) == 1 and call(lib, Q=FAKE + 2) == 1 and call(lib, q_pos=None) == 1
    assert call(lib, dims(B=0)) == 0 and call(lib, dims(Tq=0)) == 0     # nothing to do: no launch


def test_attn_refusals(lib):
    assert attn(lib, O=None) == 1 and attn(lib, O=FAKE + 2) == 1 and attn(lib, lse=FAKE + 1) == 1
    assert attn(lib, win=None) == 1 and "window" in err()
    assert attn(lib, win=abi.Window(codes=FAKE, scales=None, pos0=FAKE)) == 1
    need = abi.csa2_dense_attn_workspace_size(dims(), 100)
    assert need > 0 and attn(lib, ws=None) == 4 and attn(lib, nbytes=need - 1) == 4 and "workspace" in err()
    assert attn(lib, ws=FAKE + 4) == 1 and "16-byte" in err()
    assert abi.csa2_dense_attn_workspace_size(dims(), -1) == 0


def test_weights_refusals(lib):
    for decay in (-0.1, 1.01, math.nan):
        assert weights(lib, decay=decay) == 1 and "decay" in err()
    assert weights(lib, lse=None) == 1 and weights(lib, w_out=None) == 1 and weights(lib, w_in=FAKE + 2) == 1
    assert weights(lib, n=0) == 0
    need = abi.csa2_entry_weights_workspace_size(dims(Tq=40), 100)
    assert need > 0 and weights(lib, dims(Tq=40), ws=None) == 4 and weights(lib, dims(Tq=40), nbytes=need - 1) == 4
    assert weights(lib, dims(Tq=40), ws=FAKE + 4) == 1 and "16-byte" in err()


def test_evict_refusals(lib):
    assert evict(lib, dims(d=128)) == 2 and evict(lib, dims(d=64, kv_format=abi.CSA2_KV_FP8)) == 2
    assert evict(lib, dims(kv_format=7)) == 1 and evict(lib, dims(B=-1)) == 1 and evict(lib, dims(max_pages=0)) == 1
    assert evict(lib, keep=0) == 1 and "keep" in err()
    assert evict(lib, sink=-1) == 1 and evict(lib, recent=-1) == 1 and evict(lib, sink=6, recent=5) == 1
    assert evict(lib, n=-1) == 1
    assert evict(lib, n_entries=FAKE + 64) == 1 and "n_entries" in err()
    assert evict(lib, bd=None) == 1 and evict(lib, bd=abi.Bounded(entry_pos=FAKE, weight=FAKE)) == 1
    assert evict(lib, bd=abi.Bounded(entry_pos=FAKE, weight=None, shift=FAKE)) == 1
    assert evict(lib, dims(Di=48)) == 1 and evict(lib, dims(Di=48), cache(idx_k=None), ws=None) == 4
    assert evict(lib, c=cache(kv_codes=FAKE + 4)) == 1
    need = abi.csa2_evict_workspace_size(dims(), 100)
    assert need > 0 and evict(lib, ws=None) == 4 and evict(lib, nbytes=need - 1) == 4 and evict(lib, ws=FAKE + 4) == 1
    assert evict(lib, keep=100) == 0 and evict(lib, dims(B=0)) == 0     # nothing can be over its budget


def test_compress_pack_bounded_refusals(lib):
    call = lambda bd, **kw: lib.csa2_compress_pack_bounded(  # noqa: E731
        FAKE, 2, kw.get("T", 64), kw.get("H", 128), FAKE, FAKE, 1e-6, 1e4, FAKE, FAKE, C.byref(dims()),
        C.byref(cache()), C.byref(bd) if bd is not None else None, FAKE, kw.get("nbytes", 1 << 40), None)
    assert call(None) == 1 and "bounded" in err()
    assert call(abi.Bounded(entry_pos=FAKE, weight=FAKE)) == 1 and "shift" in err()
    assert call(BOUNDED, H=100) == 1 and "multiple of 64" in err()
    assert call(BOUNDED, T=3) == 0                                      # no whole group: nothing to do
    assert call(BOUNDED, nbytes=abi.csa2_compress_workspace_size(2, 64, 128, 512, 128) - 1) == 4


def test_pools_past_32_bit_entry_numbers_are_refused(lib):
    big = cache(n_pages=(1 << 31) // 64)
    for rc in (attn(lib, c=big), weights(lib, c=big), evict(lib, c=big)):
        assert rc == 1 and "n_pages" in err()
    assert evict(lib, c=cache(n_pages=(1 << 31) // 64 - 1), keep=100) == 0
