"""moe_rmsnorm against the plain 64-bit form.

Tolerances, with u = 2^-24 (half an fp32 step). h is one fp32 addition (u
relative). The sum of squares adds at most 32 products per thread, then 32
lanes and 32 warps: every term passes at most 32 + 5 + 31 additions, so its
relative error is below 70 u plus 2u of h's own; the mean, root, reciprocal and
the two products add at most 8 u after the root halves the sum's error. So y
is within 48 u < 2^-18 of |y|.
  bf16      one rounding more: 2^-8 |y|
  int8      scale within 2^-18; a value within half a step, scale / 2
  MXFP8     a value within half an E4M3 step (2^-4 relative, 2^-10 of the
            block's scale below the normal range), clamped at 448 scales; the
            scale is the power of two of max|y|, which may differ only where
            max|y| is within 2^-18 of one
"""

import numpy as np
import pytest
import torch

import _plain
import oracle
import mixture_experts_expert_top_b200 as moe
from mixture_experts_expert_top_b200 import build as moe_build

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
FMT = {"bf16": 0, "mxfp8": 2, "int8": 4}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    moe_build.build()
    moe.lib()
    yield
    assert moe.moe_get_device_error() == 0


def inputs(rows, H, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed + rows * 7 + H)
    x = torch.randn(rows, H, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    r = torch.randn(rows, H, generator=g) * 2 if residual else None
    w = 1 + 0.3 * torch.randn(H, generator=g)
    bf = lambda t: None if t is None else t.to(torch.bfloat16).to(DEV)
    return bf(x), bf(r), bf(w)


def run(x, r, w, fmt, eps=EPS, want_y=True, stream=None, residual_out=None, y=None):
    """Every output has one row more than is written, to see that it stays."""
    rows, H = x.shape
    guard = lambda *s, dtype: torch.full(s, 77, dtype=dtype, device=DEV)
    out = {}
    if r is not None:
        out["residual_out"] = residual_out if residual_out is not None else guard(rows + 1, H, dtype=torch.bfloat16)
    if want_y:
        out["y"] = y if y is not None else guard(rows + 1, H, dtype=torch.bfloat16)
    if fmt == "int8":
        out["q"], out["scales"] = guard(rows + 1, H, dtype=torch.int8), guard(rows + 1, dtype=torch.float32)
    elif fmt == "mxfp8":
        out["q"], out["scales"] = guard(rows + 1, H, dtype=torch.uint8), guard(rows + 1, H // 32, dtype=torch.uint8)
    moe.moe_rmsnorm(x, r, w, eps, rows, H, FMT[fmt], out.get("residual_out"), out.get("y"), out.get("q"),
                    out.get("scales"), stream)
    torch.cuda.synchronize()
    for n, t in out.items():
        if t.shape[0] > rows:
            assert torch.all(t[rows] == 77), n
            out[n] = t[:rows]
    return out


def check(x, r, w, fmt, eps=EPS, out=None, **kw):
    got = out or run(x, r, w, fmt, eps, **kw)
    h, y = _plain.rmsnorm(x, r, w, eps)
    if r is not None:
        assert torch.all((got["residual_out"].double() - h).abs() <= h.abs() * 2.0 ** -8 + 2.0 ** -134)
        assert torch.equal(got["residual_out"], (x.float() + r.float()).to(torch.bfloat16))
    if "y" in got:
        assert torch.all((got["y"].double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -134)
    if fmt == "int8":
        s = got["scales"].double()[:, None]
        ref = y.abs().amax(1, keepdim=True) / 127
        assert torch.all((s - ref).abs() <= ref * 2.0 ** -18)
        v = got["q"].double() * s
        assert torch.all((v - y).abs() <= s * (0.5 + 127 * 2.0 ** -17))
        live = ref[:, 0] > 0
        assert torch.all(got["q"][live].int().abs().amax(1) == 127)
    if fmt == "mxfp8":
        blocks = y.view(y.shape[0], -1, 32)
        amax = blocks.abs().amax(2)
        e = got["scales"].double() - 127
        two_e = torch.exp2(e)
        # 256 <= max|y| / 2^e < 512 up to the norm's error (zero blocks: the smallest exponent)
        live = amax > 2.0 ** -118
        ratio = torch.where(live, amax / two_e, torch.full_like(amax, 300.0))
        assert torch.all((ratio >= 256 * (1 - 2.0 ** -18)) & (ratio < 512 * (1 + 2.0 ** -18)))
        assert torch.all(got["scales"][amax == 0] == 0)
        val = torch.from_numpy(oracle.mx_dequantize(got["q"].cpu().numpy(), got["scales"].cpu().numpy())).to(DEV)
        lim = (448 * two_e).repeat_interleave(32, 1)
        ref = torch.maximum(torch.minimum(y, lim), -lim)
        assert torch.all((val - ref).abs() <= ref.abs() * (2.0 ** -4 + 2.0 ** -17) +
                         two_e.repeat_interleave(32, 1) * 2.0 ** -10)
    return got


SIZES = [(1, 32), (1, 2048), (2, 64), (3, 96), (7, 1024), (64, 2048), (33, 2080), (5, 4096), (4, 7168), (9, 8192),
         (3, 8224), (2, 16384), (1, 32768), (300, 160), (1000, 512)]


@pytest.mark.parametrize("rows,H", SIZES)
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "int8"])
@pytest.mark.parametrize("residual", [True, False], ids=["residual", "alone"])
def test_rmsnorm(rows, H, fmt, residual):
    check(*inputs(rows, H, residual=residual), fmt)


@pytest.mark.parametrize("H,fmt", [(8, "bf16"), (24, "bf16"), (1000, "bf16"), (16, "int8"), (48, "int8"), (2064, "int8")])
def test_row_lengths_of_each_format(H, fmt):
    check(*inputs(5, H), fmt)


@pytest.mark.parametrize("fmt", ["mxfp8", "int8"])
def test_without_the_bf16_rows(fmt):
    x, r, w = inputs(20, 256)
    a, b = run(x, r, w, fmt), run(x, r, w, fmt, want_y=False)
    for n in ("residual_out", "q", "scales"):
        assert torch.equal(a[n], b[n])


@pytest.mark.parametrize("rows,H", [(3, 256), (40, 2048), (2, 9000)])
def test_outputs_in_the_inputs_place(rows, H):
    x, r, w = inputs(rows, H)
    ref = run(x, r, w, "bf16")
    xc, rc = x.clone(), r.clone()
    got = run(xc, rc, w, "bf16", residual_out=rc, y=xc)           # both in place
    assert torch.equal(got["residual_out"], ref["residual_out"]) and torch.equal(got["y"], ref["y"])
    xc, rc = x.clone(), r.clone()
    got = run(xc, rc, w, "bf16", residual_out=xc)
    assert torch.equal(got["residual_out"], ref["residual_out"]) and torch.equal(got["y"], ref["y"])


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "int8"])
def test_extreme_rows(fmt):
    H = 256
    x, r, w = inputs(8, H)
    x[0] = 0; r[0] = 0                                            # zeros: eps keeps y = 0
    x[1] = 3e38; r[1] = 0                                         # squares past the fp32 range
    x[2] = 1e30; r[2] = -5e29
    x[3] = 1e-30; r[3] = 0                                        # far below eps
    x[4] = 0; r[4] = 0; x[4, 17] = 1e25                           # one element carries the norm
    x[5] = 1e-38; r[5] = 1e-39
    got = check(x, r, w, fmt)
    if fmt == "int8":
        assert torch.all(got["q"][0] == 0) and float(got["scales"][0]) == 0.0
    check(x, r, w, fmt, eps=1e-30)
    check(x, r, w, fmt, eps=1.0)


def test_non_finite_rows_stay_in_their_rows():
    H = 512
    x, r, w = inputs(6, H)
    clean = run(x, r, w, "int8")
    x[1, 3] = float("nan")
    x[4, 100] = float("inf")
    got = run(x, r, w, "int8")
    for row in (1, 4):
        assert torch.all(got["q"][row] == 0) and bool(torch.isnan(got["scales"][row]))
    for n in clean:
        assert torch.equal(got[n][[0, 2, 3, 5]], clean[n][[0, 2, 3, 5]]), n
    assert bool(torch.isnan(got["y"][1].float()).all())


def test_int8_rows_equal_moe_i8_quantize_of_exact_rows():
    # rows whose y is exact in bf16 (|h| constant, weight 1): both ways quantise the same values
    H = 256
    x = torch.where(torch.arange(H) % 3 == 0, -2.0, 2.0).to(torch.bfloat16).repeat(4, 1).to(DEV)
    got = run(x, None, torch.ones(H, dtype=torch.bfloat16, device=DEV), "int8", eps=1e-30)
    q, s = _plain.int8_rows(got["y"])
    assert torch.equal(got["q"], q) and torch.allclose(got["scales"], s, rtol=2.0 ** -20)


def test_captured_replayed_and_on_a_side_stream():
    x, r, w = inputs(40, 2048)
    ref = run(x, r, w, "int8")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    side = run(x, r, w, "int8", stream=st)
    for n in ref:
        assert torch.equal(ref[n], side[n]), n
    out = {n: torch.zeros_like(t) for n, t in ref.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_rmsnorm(x, r, w, EPS, 40, 2048, FMT["int8"], out["residual_out"], out["y"], out["q"], out["scales"],
                        torch.cuda.current_stream())
    x.copy_(inputs(40, 2048, seed=5)[0])
    g.replay()
    torch.cuda.synchronize()
    check(x, r, w, "int8", out=out)


def test_many_rows():
    x, r, w = inputs(20000, 128)
    check(x, r, w, "int8")
    check(x, r, w, "mxfp8")


def test_a_lazily_shared_output_leaves_its_twin():
    """An output that shares its storage copy-on-write gets its own before the
    kernel writes: the tensor that it was cloned from keeps its values."""
    x = torch.randn(4, 256, device=DEV).to(torch.bfloat16)
    q0, s0 = torch.full((4, 256), 7, dtype=torch.int8, device=DEV), torch.full((4,), 3.0, device=DEV)
    q, s = torch._lazy_clone(q0), torch._lazy_clone(s0)
    moe.moe_i8_quantize(x, 4, 256, q, s)
    want_q, want_s = torch.empty_like(q0), torch.empty_like(s0)
    moe.moe_i8_quantize(x, 4, 256, want_q, want_s)
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
    assert bool((q0 == 7).all()) and bool((s0 == 3.0).all())


@pytest.mark.parametrize("rows,H", [(256, 7168), (1000, 1024), (37, 2080), (64, 16384), (20, 32768), (500, 96)])
def test_mxfp8_codes_equal_the_formulas(rows, H):
    """x and residual are multiples of 1/8 up to 8: h and its squares' sums over
    a thread (at most 64 of at most 2^14 / 64 each) are exact in fp32, so the
    row's factor is within 2^-45 and each product within 2^-46 of the formula's:
    every code is the 64-bit formula's, rounded to nearest even, unless that
    lies as close to a border, which of these 2 10^6 values one in 10^7 such
    tests would meet."""
    g = torch.Generator().manual_seed(rows + H)
    grid = lambda: (torch.randint(-64, 65, (rows, H), generator=g) / 8).to(torch.bfloat16).to(DEV)
    x, r, w = grid(), grid(), (1 + 0.3 * torch.randn(H, generator=g)).to(torch.bfloat16).to(DEV)
    got = run(x, r, w, "mxfp8")
    h = x.double() + r.double()
    # eps as the entry point takes it
    y = h / (h.square().mean(1, keepdim=True) + float(np.float32(EPS))).sqrt() * w.double()
    blocks = y.view(rows, H // 32, 32)
    amax = blocks.abs().amax(2, keepdim=True)
    e = torch.frexp(amax).exponent - 9
    assert torch.equal(got["scales"].int(), torch.where(amax > 0, e + 127, torch.zeros_like(e))[:, :, 0].int())
    v = torch.ldexp(blocks, -e)
    step = torch.exp2((torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent - 4).double())
    want = ((v / step).round() * step).clamp(-448, 448).view(rows, H)
    code = got["q"].view(torch.float8_e4m3fn).double()
    assert int((code != want).sum()) == 0


@pytest.mark.parametrize("H", [4096, 7168, 8192, 16384, 32768])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "int8"])
def test_long_rows_of_the_largest_values(H, fmt):
    """Squares whose sum is past the fp32 range by up to 2^143: H values of
    nearly 2^128."""
    top = torch.finfo(torch.bfloat16).max
    x, _, w = inputs(7, H, residual=False)
    sign = torch.where(torch.arange(H, device=DEV) % 3 == 0, -1.0, 1.0)
    x[0] = top
    x[1] = (sign * top).to(torch.bfloat16)
    x[2] = 1.6e38
    x[3] = 3e36
    x[4] = x[4] * 2.0 ** 20; x[4, 5] = top                        # ordinary values beside one such: y near 2^-100
    x[5, : H // 2] = 0; x[5, H // 2:] = -top
    got = check(x, None, w, fmt)
    if fmt == "bf16":
        assert torch.equal(got["y"][0], w)                        # (1 + 2^-18) w rounds to w: 8 bits
    # and as h: zeros, then with a residual of the same size and sign that stays below infinity
    half = (sign * 1.6e38).to(torch.bfloat16).expand(7, H).contiguous()
    check(torch.zeros_like(half), half, w, fmt)
    check(half, half, w, fmt)


def mx_codes_differ(x, r, w):
    """How many E4M3 codes of moe_rmsnorm differ from the formula's, of fp32
    h = x + r, in 64 bits from there."""
    rows, H = x.shape
    got = run(x, r, w, "mxfp8")
    h = (x.float() + r.float() if r is not None else x.float()).double()
    # eps as the entry point takes it
    y = h / (h.square().mean(1, keepdim=True) + float(np.float32(EPS))).sqrt() * w.double()
    blocks = y.view(rows, H // 32, 32)
    amax = blocks.abs().amax(2, keepdim=True)
    e = torch.frexp(amax).exponent - 9
    assert torch.equal(got["scales"].int(), torch.where(amax > 0, e + 127, torch.zeros_like(e))[:, :, 0].int())
    v = torch.ldexp(blocks, -e)
    step = torch.exp2((torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent - 4).double())
    want = ((v / step).round() * step).clamp(-448, 448).view(rows, H)
    return int((got["q"].view(torch.float8_e4m3fn).double() != want).sum())


@pytest.mark.parametrize("rows,H", [(4400, 7168), (30000, 1024), (4096, 2048), (1900, 16384), (960, 32768), (8192, 96)])
@pytest.mark.parametrize("residual", [True, False], ids=["residual", "alone"])
def test_mxfp8_codes_equal_the_formulas_on_ordinary_rows(rows, H, residual):
    """Ordinary values, whose squares' sums are not exact in fp32. A row's sum is
    kept to about 2^-45 (2^-37 at worst), and the root, the factor and a product
    to 2^-45. E4M3 has 8 borders per factor of two, 2^-4 to 2^-3 apart: a value
    lies within 2^-44 of one with probability 2^-44 * 2 * 16 = 2^-39, and of 3 10^7
    values one does in 6 10^-5 of such tests."""
    x, r, w = inputs(rows, H, seed=11, residual=residual)
    assert mx_codes_differ(x, r, w) == 0
