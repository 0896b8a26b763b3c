"""Values that the whole-cache kernels must carry through or keep apart: NaN, infinite lse, scales at the end of
their range, a long tail beside a peak."""
import math

import numpy as np
import pytest
import torch

from bounded_case import Case
from compressed_sparse_attention_05_gb300 import abi, build
from oracle import bounded as OB
from oracle import formats as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def status():
    torch.cuda.synchronize()
    return abi.csa2_get_status()


def two_tokens(**kw):
    """Two tokens of one tile; entries below 295 and window rows below 1180 are hidden from the second."""
    return Case(**{**dict(seed=11, Tq=2, Hq=8, lens=(300,), W=16, q_pos=[[1170, 1199]], docs=[[0, 1180]]), **kw})


def poison_entry(c, j, group=1):
    c.t["scales"][int(c.slots[0][j]), group] = 0x7F


# ---- NaN window rows at d = 64 ---------------------------------------------------------
@pytest.mark.parametrize("bad", ["scale", "code"])
def test_nan_window_rows_of_the_small_kernel(bad):
    c = two_tokens(d=64)
    at = 1165 - int(c.pos0[0])
    if bad == "scale":
        c.t["wscales"][0, at] = float("nan")
    else:
        c.t["wcodes"][0, at, 5] = 0x7F
    c.attend()
    assert status() == 0
    assert c.lse[0, 0].isnan().all() and c.O[0, 0].isnan().all()
    c.check_attention([(0, 1)])


# ---- NaN under a cap ------------------------------------------------------------------
@pytest.mark.parametrize("d", [512, 64])
@pytest.mark.parametrize("bad", ["entry", "window"])
def test_a_cap_lets_nan_keys_through(d, bad):
    """Logits of a few times the cap, so that the cap's branch for large logits is taken."""
    c = two_tokens(d=d, cap=2.0, q_scale=3.0)
    if bad == "entry":
        poison_entry(c, 200)
    else:
        c.t["wscales"][0, 1165 - int(c.pos0[0])] = float("nan")
    c.attend()
    assert status() == 0
    assert c.lse[0, 0].isnan().all() and c.O[0, 0].isnan().all()
    c.check_attention([(0, 1)])


@pytest.mark.parametrize("d", [512, 64])
def test_a_cap_lets_nan_keys_through_to_their_weight(d):
    c = two_tokens(d=d, cap=2.0, q_scale=3.0)
    c.attend()
    lse = c.lse.clone()
    want = c.weigh(lse, None, torch.zeros(c.n_pages * 64, device="cuda")).clone()
    poison_entry(c, 200)
    got = c.weigh(lse, None, torch.zeros(c.n_pages * 64, device="cuda"))
    assert status() == 0
    at = int(c.slots[0][200])
    assert got[at].isnan()
    got[at] = want[at]
    assert torch.equal(got, want)


@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_nan_in_a_query_stays_in_its_head(cap):
    c = two_tokens(cap=cap, q_scale=3.0)
    c.t["Q"][0, 0, 3, 77] = float("nan")
    c.attend()
    assert status() == 0
    assert c.lse[0, 0, 3].isnan() and c.O[0, 0, 3].isnan().all()
    rest = [h for h in range(8) if h != 3]
    assert c.lse[0, 0, rest].isfinite().all() and c.O[0, 0, rest].isfinite().all()
    c.check_attention([(0, 1)])


# ---- NaN where nothing finite came before ----------------------------------------------
@pytest.mark.parametrize("d", [512, 64])
def test_the_only_key_is_nan(d):
    c = Case(seed=12, Hq=8, d=d, lens=(1,), window=False)
    poison_entry(c, 0)
    c.attend()
    assert status() == 0
    assert c.lse.isnan().all() and c.O.isnan().all()


@pytest.mark.parametrize("d", [512, 64])
def test_a_tile_of_nan_keys_before_good_ones(d):
    """The first 32 entries (a whole tile of the d = 64 kernel) are NaN; the token of a later document sees none of
    them."""
    c = Case(seed=13, Tq=2, Hq=8, d=d, lens=(40,), window=False, q_pos=[[159, 159]], docs=[[0, 128]])
    for j in range(32):
        poison_entry(c, j, j % (d // 16))
    c.attend()
    assert status() == 0
    assert c.lse[0, 0].isnan().all() and c.O[0, 0].isnan().all()
    c.check_attention([(0, 1)])


# ---- infinite lse beside a NaN key -------------------------------------------------------
@pytest.mark.parametrize("kw", [dict(), dict(d=64), dict(Hq=128), dict(Tq=4, Hq=64, q_pos=[[1170, 1180, 1190, 1199]],
                                                                       docs=[[0, 1180, 1180, 1180]])],
                         ids=["one_tile", "d64", "hq128", "tiles"])
def test_rows_of_infinite_lse_add_nothing_beside_a_nan_key(kw):
    """The first token sees the NaN entry, but its lse is infinite in every head."""
    c = two_tokens(**kw)
    c.attend()
    lse = c.lse.clone()
    poison_entry(c, 200)
    lse[0, 0, 0::2] = float("inf")
    lse[0, 0, 1::2] = float("-inf")
    out = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(lse, None, out)
    assert status() == 0
    assert out.isfinite().all()
    c.check_weights(lse, None, out)


@pytest.mark.parametrize("d", [512, 64])
def test_one_head_of_infinite_lse_beside_a_nan_key(d):
    c = two_tokens(d=d)
    c.attend()
    lse = c.lse.clone()
    lse[0, 0, 5] = float("inf")
    lse[0, 1, 2] = float("-inf")
    out = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(lse, None, out)
    c.check_weights(lse, None, out)
    poison_entry(c, 200)
    again = torch.zeros(c.n_pages * 64, device="cuda")
    c.weigh(lse, None, again)
    assert status() == 0
    at = int(c.slots[0][200])
    assert again[at].isnan()            # the token's other heads see it
    again[at] = out[at]
    assert torch.equal(again, out)


# ---- window rows of enormous scales --------------------------------------------------------
@pytest.mark.parametrize("scale", [2.0 ** 112, 2.0 ** 125])
def test_rows_past_the_operand_range_stay_with_the_tokens_that_see_them(scale):
    c = two_tokens()
    at = 1165 - int(c.pos0[0])
    c.t["wscales"][0, at] = scale
    c.t["wcodes"][0, at, 0::2] = 0x7E       # 448
    c.t["wcodes"][0, at, 1::2] = 0xFE       # -448
    c.attend()
    assert status() == 0
    c.check_attention([(0, 1)])


# ---- a peak and a long tail ---------------------------------------------------------------
def test_a_long_tail_beside_a_peak():
    """One window row, and 100,000 entries of about 2^-25.5 of its weight each, in tiles that one SM walks alone:
    0.2% of the mass, and all of it in the channels where the window row is zero.

    The error of O in such a channel, of a value of about 2e-3: its rounding, 2^-8 of it, and that of the tail's
    weights.  Those are P = 2^7 w with w in units of the reference, above 2^-19 for a w above 2^-26, and fp16's
    step there is 2^-24: at most 2^-25 / 2^-19 = 2^-6 of each weight, whatever their number.  Logit errors and the
    rest of the kernel's bounds (2^-11 + 2 e + 2^-20) are below 2^-10."""
    n, Tq = 100000, 160
    c = Case(seed=14, Tq=Tq, Hq=64, lens=(64,), W=1, q_pos=[[4 * n - 1] * Tq], tau=25.5 * math.log(2) / 16)
    g = torch.Generator().manual_seed(15)
    x = torch.randn(n, 512, generator=g)
    x[:, :16] = 1.5                                              # scale 1/4, code 6: exact
    x[:, 32:] = x[:, 32:].abs()
    codes, scales = F.mxfp4_pack(x.numpy().astype(np.float32))
    pages = (n + 63) // 64
    c.lens, c.n_pages, c.max_entries = [n], pages, n
    c.table = np.random.RandomState(16).permutation(pages).astype(np.int32)[None, :]
    c.slots = [c.table[0, np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64]
    c.codes, c.scales = torch.zeros(pages * 64, 256, dtype=torch.uint8), torch.zeros(pages * 64, 32, dtype=torch.uint8)
    c.codes[c.slots[0]], c.scales[c.slots[0]] = torch.from_numpy(codes), torch.from_numpy(scales)
    w = np.zeros((1, 512), np.float32)
    w[0, :16] = 2.5
    wc, ws = F.fp8_pack(w)
    c.wcodes[0, 0], c.wscales[0, 0] = torch.from_numpy(wc[0]), float(ws[0])
    c.Q = torch.zeros(1, Tq, 64, 512, dtype=torch.bfloat16)
    c.Q[..., :16] = 1.0
    c.Q[..., 16] = (torch.rand(1, Tq, 64, generator=g) * 0.05).bfloat16()  # the logits differ a little
    c._device()
    c.attend()
    assert status() == 0
    keys, pos = c.keys(0)
    for i, h in ((0, 0), (77, 13), (159, 63)):
        _, rows, xl, e = c.one(0, i, (keys, pos))
        o, z = OB.attention(xl[h:h + 1], rows)
        wt = np.exp(xl[h] - z[0])
        assert wt[:-1].max() < 2.0 ** -25 and wt[:-1].min() > 2.0 ** -26 and wt[-1] > 0.99
        got = c.O[0, i, h].double().cpu().numpy()
        tail = o[0, 32:]                                         # the window row is zero here
        assert tail.min() > 1e-3
        assert np.max(np.abs(got[32:] - tail) / tail) < 2.0 ** -8 + 2.0 ** -6 + 2.0 ** -10
        assert abs(float(c.lse[0, i, h]) - z[0]) < e[h].max() + 2.0 ** -20 + 2.0 ** -23 * abs(z[0])


# ---- the ends of the cap's range -------------------------------------------------------------
@pytest.mark.parametrize("cap", [2.0 ** 127, 1e38, 2.0 ** -126])
@pytest.mark.parametrize("d", [512, 64])
def test_the_largest_and_smallest_caps(d, cap):
    """The largest ones change no logit; under the smallest every logit is 0 to within 2^-125.  (x / cap may be
    subnormal: steps of 2^-149, which cap makes 2^-21.4 of a logit in the log2 domain, well within the bound.)"""
    c = two_tokens(d=d, cap=cap)
    c.t["Q"][0, 1, 2] = 0                    # logits of exactly 0 too
    c.Q[0, 1, 2] = 0
    c.attend()
    assert status() == 0
    c.check_attention()
