"""Rotary positions against oracle.step.

The angle's fraction of a turn is exact to p 2^-53 turns; sine and cosine are within 2 units of 2^-24 of the angle's,
whose rounding (at most pi/4) adds less than one; the amplitude and the two products and their sum round four times:
every rotated value is within 2^-21 a (|x1| + |x2|) before its own rounding."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_05_gb300 import abi, build
from oracle import step as O

pytestmark = pytest.mark.gpu

KIND = {"none": abi.ROPE_PLAIN, "linear": abi.ROPE_LINEAR, "ntk": abi.ROPE_NTK, "yarn": abi.ROPE_YARN}
LAYOUT = {"half": abi.ROPE_HALF, "interleaved": abi.ROPE_INTERLEAVED}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def table_of(r, scaling="none", factor=1.0, base=10000.0, original=4096):
    t = torch.zeros(r // 2, dtype=torch.int64, device="cuda")
    abi.csa2_rope_table(abi.RopeSpec(scaling=KIND[scaling], base=base, factor=factor, original_len=original, beta_fast=32.0,
                                     beta_slow=1.0), r, t)
    return t


@pytest.mark.parametrize("r,base,scaling,factor,original", [
    (2, 10000.0, "none", 1.0, 0), (64, 10000.0, "none", 1.0, 0), (512, 1e6, "none", 1.0, 0), (64, 10000.0, "linear", 8.0, 0),
    (64, 10000.0, "ntk", 8.0, 0), (128, 500000.0, "yarn", 32.0, 8192), (64, 10000.0, "yarn", 40.0, 4096), (64, 10000.0, "yarn", 4.0, 1),
    (6, 100.0, "yarn", 2.0, 100), (64, 1.5, "none", 1.0, 0),
    (514, 10000.0, "ntk", 4.0, 0), (576, 10000.0, "yarn", 40.0, 4096), (2048, 10000.0, "none", 1.0, 0)])
def test_table(r, base, scaling, factor, original):
    """Turns per position to 2^-50 of themselves (the libraries' powers and logarithms) and one unit of 2^-64."""
    t = table_of(r, scaling, factor, base, original).cpu().numpy().astype(np.uint64)
    ref = O.rope_frequencies(r, base, scaling, factor, original) / (2 * np.pi)
    got = t.astype(np.float64) * 2.0 ** -64
    assert np.all(np.abs(got - ref) <= ref * 2.0 ** -50 + 2.0 ** -64)


def check(n, heads, d, start, r, layout="half", x_dtype=torch.bfloat16, y_dtype=None, inverse=False, amplitude=1.0, scaling="none",
          factor=1.0, pos=None, place="apart", seed=0):
    y_dtype = y_dtype or x_dtype
    g = torch.Generator().manual_seed(seed + n + heads + d + r)
    if pos is None:
        pos = torch.randint(-5, 1 << 20, (n,), generator=g)
    table = table_of(r, scaling, factor)
    positions = pos.int().cuda()
    x0 = torch.randn(n, heads, d, generator=g).to(x_dtype)
    if place == "apart" or place == "in_place":
        x = x0.cuda()
        y = x if place == "in_place" else torch.full((n, heads, d), 9.0, dtype=y_dtype, device="cuda")
    else:   # slices of wider tensors; heads outside tokens in y; odd: rows that start on no 16 bytes
        extra = 3 if place == "odd" else 8
        wide = torch.full((n, heads * d + 2 * extra), 5.0, dtype=x_dtype, device="cuda")
        x = wide[:, extra:extra + heads * d].unflatten(1, (heads, d))
        x.copy_(x0)
        y = torch.full((heads, n, d + extra), 9.0, dtype=y_dtype, device="cuda")[:, :, :d].transpose(0, 1)
    abi.csa2_rope(x, y, positions, table, start=start, layout=LAYOUT[layout], inverse=inverse, amplitude=amplitude)
    torch.cuda.synchronize()
    theta = O.rope_frequencies(r, 10000.0, scaling, factor) if r else np.zeros(0)
    xd = x0.double().numpy()
    ref = O.rope(xd, pos.numpy(), theta, start, layout, inverse, amplitude)
    i1 = start + (np.arange(r // 2) if layout == "half" else 2 * np.arange(r // 2))
    i2 = i1 + (r // 2 if layout == "half" else 1)
    tol = np.zeros_like(xd)
    tol[:, :, i1] = tol[:, :, i2] = 2.0 ** -21 * abs(amplitude) * (np.abs(xd[:, :, i1]) + np.abs(xd[:, :, i2]))
    tol += (np.abs(ref) + tol) * torch.finfo(y_dtype).eps / 2
    rest = np.ones(d, dtype=bool)
    rest[start:start + r] = False
    if x_dtype == y_dtype or y_dtype == torch.float32:
        tol[:, :, rest] = 0                                # copied channels are copied
    got = y.double().cpu().numpy()
    err = np.abs(got - ref)
    assert np.all(err <= tol), float((err - tol).max())
    if place in ("slice", "odd"):
        assert bool((wide[:, :extra] == 5).all()) and bool((wide[:, -extra:] == 5).all())
        assert bool((y.transpose(0, 1).as_strided((heads, n, extra), (n * (d + extra), d + extra, 1), d + y.storage_offset()) == 9).all())
    assert abi.csa2_get_status() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("x_dtype,y_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                             (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("n,heads,d,start,r", [(1, 64, 512, 448, 64), (1, 1, 64, 0, 64), (77, 40, 128, 64, 32), (1000, 3, 512, 448, 64),
                                               (5, 128, 576, 512, 64), (9, 2, 512, 0, 512), (301, 1, 16, 0, 16)])
def test_shapes_and_types(n, heads, d, start, r, x_dtype, y_dtype, layout):
    check(n, heads, d, start, r, layout, x_dtype, y_dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,d,start,r", [(3, 2, 7, 1, 6), (10, 5, 62, 0, 62), (4, 3, 64, 2, 8), (2, 1, 2, 0, 2), (33, 2, 65, 1, 64),
                                               (6, 4, 24, 8, 0)])
def test_odd_shapes(n, heads, d, start, r, layout):
    for x_dtype in (torch.bfloat16, torch.float32):
        check(n, heads, d, start, r, layout, x_dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("place", ["in_place", "slice", "odd"])
def test_places(place, layout):
    for dtype in (torch.bfloat16, torch.float32):
        check(50, 6, 128, 64, 64, layout, dtype, place=place)


@pytest.mark.parametrize("place", ["apart", "in_place", "slice"])
@pytest.mark.parametrize("n,heads,d,start,r", [(7, 5, 128, 0, 62), (300, 8, 128, 66, 62), (40, 3, 64, 2, 4), (11, 2, 64, 6, 4), (9, 1, 24, 2, 20),
                                               (2, 4, 16, 4, 8)])
def test_pairs_that_share_a_load_with_copied_channels(n, heads, d, start, r, place):
    """Interleaved pairs from any even channel on, in rows of whole 16 bytes."""
    for x_dtype in (torch.bfloat16, torch.float32):
        check(n, heads, d, start, r, "interleaved", x_dtype, place=place)
        if place != "in_place":
            check(n, heads, d, start, r, "interleaved", x_dtype, torch.float32 if x_dtype == torch.bfloat16 else torch.bfloat16, place=place)


@pytest.mark.parametrize("place", ["apart", "in_place", "slice"])
@pytest.mark.parametrize("n,heads,d,start,r,layout", [(7, 5, 128, 1, 62, "interleaved"), (21, 8, 128, 66, 62, "half"), (5, 40, 512, 450, 62, "half"),
                                                      (9, 1, 24, 3, 20, "interleaved"), (3, 2, 16, 5, 2, "half"), (2, 70, 64, 4, 56, "half")])
def test_any_channels_of_whole_rows(n, heads, d, start, r, layout, place):
    for x_dtype in (torch.bfloat16, torch.float32):
        check(n, heads, d, start, r, layout, x_dtype, place=place)
        if place != "in_place":
            check(n, heads, d, start, r, layout, x_dtype, torch.float32 if x_dtype == torch.bfloat16 else torch.bfloat16, place=place)


@pytest.mark.parametrize("n,heads,d,r", [(4000, 1, 16, 16), (700, 3, 512, 512), (2049, 1, 2, 2), (650, 1, 512, 512), (61, 37, 72, 16), (301, 3, 576, 576), (5, 2, 2048, 2048),
                                         (6, 1, 1990, 1986)])
def test_blocks_that_begin_inside_a_token(n, heads, d, r):
    for place in ("apart", "in_place"):
        for layout in ("half", "interleaved"):
            check(n, heads, d, 0, r, layout, place=place)


def test_tokens_of_more_than_2_31_channels():
    heads, d = 40000, 65535
    x = torch.arange(d, device="cuda").remainder(251).to(torch.bfloat16).expand(heads, d)
    y = torch.full((heads, d), 9.0, dtype=torch.bfloat16, device="cuda")
    abi.csa2_rope(x[None], y[None], torch.zeros(1, dtype=torch.int32, device="cuda"), table_of(2), start=0, layout=abi.ROPE_HALF)
    assert all(bool((part == x[:1]).all()) for part in y.split(1000))


@pytest.mark.parametrize("scaling,factor", [("linear", 8.0), ("ntk", 8.0), ("yarn", 40.0)])
def test_scaled(scaling, factor):
    check(60, 4, 64, 0, 64, "half", torch.float32, scaling=scaling, factor=factor, amplitude=1.3689)


def test_far_positions():
    pos = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 12345678])
    # (the angle p theta itself is known to p 2^-53 turns and to fp64's own 2^-52 p theta here: 2^-19 rad at 2^31)
    for layout in ("half", "interleaved"):
        check(8, 3, 64, 0, 64, layout, torch.bfloat16, pos=pos)


def test_inverse_is_the_transpose():
    """<R x, y> = <x, R' y>: the call with `inverse` is the gradient; and R' R x = a^2 x."""
    g = torch.Generator().manual_seed(0)
    n, h, d, r = 40, 6, 128, 64
    x, y = torch.randn(n, h, d, generator=g).cuda(), torch.randn(n, h, d, generator=g).cuda()
    pos = torch.randint(0, 1 << 18, (n,), generator=g).int().cuda()
    table = table_of(r, "yarn", 8.0)
    for layout in (abi.ROPE_HALF, abi.ROPE_INTERLEAVED):
        rx, ry, back = (torch.empty_like(x) for _ in range(3))
        abi.csa2_rope(x, rx, pos, table, start=32, layout=layout, amplitude=1.25)
        abi.csa2_rope(y, ry, pos, table, start=32, layout=layout, amplitude=1.25, inverse=True)
        a, b = (rx.double() * y.double()).sum(), (x.double() * ry.double()).sum()
        # every rotated value is off by at most 2^-21 a (|x1| + |x2|) + half a step: 2^-20 a (|x1| + |x2|) per product
        bound = 2.0 ** -20 * 1.25 * 4 * (x.double().abs().mean() * y.double().abs().mean()) * x.numel()
        assert abs(float(a - b)) <= float(bound)
        abi.csa2_rope(rx, back, pos, table, start=32, layout=layout, inverse=True)
        want = x.clone()
        want[:, :, 32:96] *= 1.25
        assert float((back - want).abs().max()) <= 2.0 ** -20 * 1.25 * 2 * float(x.abs().max()) * 2


def test_gradient_against_differences():
    """Central differences of f(x) = <w, R x> in fp32 steps of 1/4: f is linear, so they differ by roundings only."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, 2, 16, generator=g).cuda()
    w = torch.randn(3, 2, 16, generator=g).cuda()
    pos = torch.tensor([5, 77, 3000], dtype=torch.int32).cuda()
    table = table_of(8)
    grad = torch.empty_like(x)
    abi.csa2_rope(w, grad, pos, table, start=4, inverse=True)
    y = torch.empty_like(x)
    for i in range(x.numel()):
        f = []
        for h in (0.25, -0.25):
            z = x.clone().view(-1)
            z[i] += h
            abi.csa2_rope(z.view_as(x), y, pos, table, start=4)
            f.append(float((w.double() * y.double()).sum()))
        # two values of a rotation, each within 2^-20 (|x1| + |x2|), over a step of 1/2, and the step's own rounding
        assert abs((f[0] - f[1]) * 2 - float(grad.view(-1)[i])) <= 16 * 2.0 ** -20 * float(w.abs().max()) * float(x.abs().max() + 1)


def test_captured():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(20, 8, 64, generator=g).cuda()
    pos = torch.randint(0, 1000, (20,), generator=g).int().cuda()
    table = table_of(64)
    y, z = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        abi.csa2_rope(x, y, pos, table)
        abi.csa2_rope(y, y, pos, table, inverse=True)
    for _ in range(2):
        x.copy_(torch.randn(20, 8, 64, generator=g))
        pos.copy_(torch.randint(0, 1000, (20,), generator=g).int())
        graph.replay()
        abi.csa2_rope(x, z, pos, table)
        abi.csa2_rope(z, z, pos, table, inverse=True)
        torch.cuda.synchronize()
        assert torch.equal(y, z)


def test_a_head_for_many_tokens():
    """A stride of zero in x: one head's channels rotated for every token."""
    x = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(5)).cuda()
    pos = torch.arange(300, dtype=torch.int32).cuda()
    y = torch.empty(300, 4, 64, device="cuda")
    abi.csa2_rope(x.expand(300, 4, 64), y, pos, table_of(64))
    z = torch.empty_like(y)
    abi.csa2_rope(x.expand(300, 4, 64).contiguous(), z, pos, table_of(64))
    torch.cuda.synchronize()
    assert torch.equal(y, z)


def test_past_4_gb():
    """Rows of x and y whose offsets pass 2^32 bytes."""
    n, h, d = 70000, 64, 512
    x = torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(n, device="cuda") % 251).view(n, 1, 1).expand(n, h, d))
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    y = torch.zeros_like(x)
    abi.csa2_rope(x, y, pos, table_of(64), start=448, layout=abi.ROPE_INTERLEAVED)
    torch.cuda.synchronize()
    for i in (0, 1, 65535, 65536, 69999):
        assert torch.equal(x[i], y[i])


def test_no_tokens():
    x = torch.empty(0, 4, 64, device="cuda")
    abi.csa2_rope(x, x, torch.empty(0, dtype=torch.int32, device="cuda"), table_of(64))
