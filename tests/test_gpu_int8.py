"""Int8 rows and the int8 grouped products against the plain 64-bit form, and
the layer with int8 weights.

moe_i8_quantize is exact. The products: the int32 sums are exact; the sum's
conversion and the two scales round by 2^-24 each, so v is within 3 * 2^-24 of
|v|, and y = bf16(v) within 2^-8 + 2^-20. silu(g) = g / (1 + exp(-g)) turns a
relative error d of g into at most (1 + |g|) d, an exponential within 2^-22 +
2^-23 |g| (its argument rounded, 2 ulp) adds that, the division and products
2^-22: |act - ref| <= |ref| (2^-8 + 2^-20 (4 + |g|)), and where exp(-g) leaves
the fp32 range (g < -87) act is below 1e-35 |u|.
"""

import numpy as np
import pytest
import torch

import _plain
import moe_synth
import oracle
import mixture_experts_expert_top_b200 as moe
from mixture_experts_expert_top_b200 import build as moe_build
from _util import bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    moe_build.build()
    moe.lib()
    yield
    assert moe.moe_get_device_error() == 0


# ---- moe_i8_quantize ---------------------------------------------------------

def quantize(x, stream=None):
    rows, K = x.shape
    q = torch.full((rows + 1, K), 77, dtype=torch.int8, device=DEV)
    s = torch.full((rows + 1,), 77.0, device=DEV)
    moe.moe_i8_quantize(x, rows, K, q, s, stream)
    torch.cuda.synchronize()
    assert torch.all(q[rows] == 77) and float(s[rows]) == 77.0
    return q[:rows], s[:rows]


def same_rows(x):
    q, s = quantize(x)
    rq, rs = _plain.int8_rows(x)
    assert torch.equal(q, rq)
    assert torch.equal(s.view(torch.int32)[~torch.isnan(rs)], rs.view(torch.int32)[~torch.isnan(rs)])
    assert torch.equal(torch.isnan(s), torch.isnan(rs))


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (17, 768), (512, 768), (64, 2048), (5, 2064), (7, 7168), (2, 8208),
                                    (1, 32768), (4099, 272), (70000, 64)])
def test_quantize_is_bit_exact(rows, K):
    g = torch.Generator().manual_seed(rows + K)
    x = torch.randn(rows, K, generator=g) * torch.exp(6 * torch.randn(rows, 1, generator=g))
    same_rows(x.to(torch.bfloat16).to(DEV))


def test_quantize_every_pair_of_mantissas():
    # 127 x / amax for every 8-bit significand of amax and of x, x from amax down
    # to 2^-9 amax: all ties n + 1/2 and all nearest misses are among them
    m = torch.arange(128, 256, dtype=torch.float64)
    x = torch.cat([m * 2.0 ** -s for s in range(0, 11)])           # 1408 values
    rows = torch.cat([x.expand(128, -1), -x.expand(128, -1)], 1)
    rows = torch.where(rows.abs() <= m[:, None], rows, torch.zeros_like(rows))
    rows[:, 0] = m                                                   # the row's maximum
    for scale in (1.0, 2.0 ** -126, 2.0 ** 100):
        same_rows((rows * scale).to(torch.bfloat16).to(DEV))


def test_quantize_special_rows():
    x = torch.randn(9, 64, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 5] = float("-inf")
    x[3] = torch.finfo(torch.bfloat16).max
    x[4] = 2.0 ** -133                                               # the smallest subnormal
    x[5] = 2.0 ** -130; x[5, 0] = 2.0 ** -126
    x[6] = -0.0
    x[7] = -1.0
    same_rows(x.to(torch.bfloat16).to(DEV))


# ---- grouped products --------------------------------------------------------

def routing(T, E, k, seed, skew=0.0, n_shared=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) - skew * torch.log(torch.arange(1, E + 1, dtype=torch.float32))
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    ids = torch.cat([ids, torch.arange(E, E + n_shared).expand(T, n_shared)], 1)
    flat = ids.reshape(-1)
    perm = torch.argsort(flat, stable=True).to(torch.int32)
    off = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat, minlength=E + n_shared).cumsum(0)])
    return perm.to(DEV), off.to(torch.int32).to(DEV)


def codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8, device=DEV)


def scales(g, *shape):
    return torch.exp(0.5 * torch.randn(*shape, generator=g, device=DEV))


def case(T, H, I, E, k, seed=0, skew=0.0, n_shared=0):
    g = torch.Generator(device=DEV).manual_seed(seed + T + H + I)
    Et, P = E + n_shared, T * (k + n_shared)
    perm, off = routing(T, E, k, seed + 1, skew, n_shared)
    c = {"shape": moe.Shape.of(T, H, I, E, k, "int8", n_shared=n_shared), "perm": perm, "off": off, "P": P,
         "hq": codes(g, T, H), "hs": scales(g, T) * 1e-2, "w_gu": codes(g, Et, 2 * I, H),
         "gs": scales(g, Et, 2 * I) * (2.0 / (H ** 0.5 * 5500 * 1e-2)),      # g and u of the order of 2
         "aq": codes(g, P, I), "as": scales(g, P), "w_d": codes(g, Et, H, I), "ds": scales(g, Et, H)}
    return c


def gate_up(c, a, a_s, perm, stream=None):
    sh = c["shape"]
    act = torch.full((c["P"] + 1, sh.I), 77, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_swiglu_i8(a, a_s, perm, c["off"], c["w_gu"], c["gs"], sh, act, stream)
    torch.cuda.synchronize()
    assert torch.all(act[c["P"]] == 77)
    return act[:c["P"]]


def down(c, stream=None):
    sh = c["shape"]
    y = torch.full((c["P"] + 1, sh.H), 77, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_down_i8(c["aq"], c["as"], c["off"], c["w_d"], c["ds"], sh, y, stream)
    torch.cuda.synchronize()
    assert torch.all(y[c["P"]] == 77)
    return y[:c["P"]]


def close_act(act, v):
    ref, g, u = _plain.swiglu(v)
    tol = ref.abs() * (2.0 ** -8 + 2.0 ** -20 * (4 + g.abs())) + 1e-35 * u.abs()
    bad = (act.double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((act.double() - ref).abs() / tol.clamp_min(1e-300)).max()))


def close_y(y, v):
    assert torch.all((y.double() - v).abs() <= v.abs() * (2.0 ** -8 + 2.0 ** -20))


def check(c, gather_too=True):
    slots = c["shape"].slots
    close_y(down(c), _plain.grouped_int8(c["aq"], c["as"], None, c["off"], c["w_d"], c["ds"], slots))
    v = _plain.grouped_int8(c["hq"], c["hs"], c["perm"], c["off"], c["w_gu"], c["gs"], slots)
    src = c["perm"].long() // slots
    rows = gate_up(c, c["hq"][src].contiguous(), c["hs"][src].contiguous(), None)
    close_act(rows, v)
    if gather_too:
        # the same rows through perm: the sums are exact, so the results agree bit for bit
        assert torch.equal(gate_up(c, c["hq"], c["hs"], c["perm"]).view(torch.int16), rows.view(torch.int16))


PRODUCTS = [
    (1, 128, 64, 1, 1), (1, 16, 16, 1, 1), (1, 2048, 768, 8, 8),       # one token
    (2, 32, 48, 4, 2), (5, 144, 80, 3, 2), (7, 272, 176, 5, 3),        # K and features off every tile
    (15, 256, 128, 1, 1), (16, 256, 128, 1, 1), (17, 256, 128, 1, 1),  # around a 16-row MMA step
    (33, 256, 144, 1, 1), (65, 256, 128, 1, 1), (129, 256, 272, 1, 1), (255, 128, 128, 1, 1),
    (256, 128, 128, 1, 1), (257, 400, 336, 1, 1), (300, 640, 208, 2, 1),
    (64, 1024, 384, 128, 8), (200, 512, 256, 24, 4), (500, 528, 272, 8, 4), (1000, 384, 656, 6, 3),
    (3000, 256, 128, 16, 2),
]


@pytest.mark.parametrize("T,H,I,E,k", PRODUCTS)
def test_grouped_products(T, H, I, E, k):
    check(case(T, H, I, E, k))


@pytest.mark.parametrize("T,H,I,E,k,skew", [(40, 256, 128, 64, 2, 4.0), (900, 256, 160, 32, 2, 4.0),
                                            (2000, 304, 128, 128, 1, 2.0)])
def test_uneven_loads_and_experts_without_rows(T, H, I, E, k, skew):
    c = case(T, H, I, E, k, skew=skew)
    assert int((c["off"][1:] == c["off"][:-1]).sum()) > 0            # experts with no rows
    check(c)


@pytest.mark.parametrize("T", [10, 400])
def test_shared_experts(T):
    check(case(T, 256, 128, 8, 2, n_shared=2))


@pytest.mark.parametrize("K", [16, 112, 128, 144, 1024, 32768])
def test_sums_are_exact_at_their_largest(K):
    # every product 2^14 with one sign: sums up to 2^29 at K = 32768, then one
    # product less; exact before the scales, which are 1
    T, E, H = 3, 2, 32
    perm, off = routing(T, E, 1, 0)
    sh = moe.Shape.of(T, H, K, E, 1, "int8")
    aq = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((E, H, K), -128, dtype=torch.int8, device=DEV)
    w[:, 1::2] = 127
    w[:, 5, 0] = 0
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(E * H, device=DEV)
    moe.moe_grouped_gemm_down_i8(aq, torch.ones(T, device=DEV), off, w, one, sh, y)
    torch.cuda.synchronize()
    v = aq.double() @ w[0].double().T
    assert torch.equal(y, v.float().to(torch.bfloat16))


def test_a_row_with_scale_nan_or_zero_stays_its_own():
    c = case(20, 256, 128, 4, 2)
    ref_y = down(c)
    c["as"][7] = float("nan")
    c["as"][9] = 0.0
    y = down(c)
    assert bool(torch.isnan(y[7].float()).all()) and bool((y[9] == 0).all())
    keep = [i for i in range(c["P"]) if i not in (7, 9)]
    assert torch.equal(y[keep].view(torch.int16), ref_y[keep].view(torch.int16))


def test_large_gates_and_signs():
    # gates far out on both sides: silu saturates to g and to 0 without NaN
    c = case(64, 256, 128, 4, 2)
    c["gs"] *= 200.0
    check(c)


def test_products_are_deterministic_and_run_on_a_side_stream():
    c = case(700, 512, 256, 8, 2)
    y, act = down(c), gate_up(c, c["hq"], c["hs"], c["perm"])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        assert torch.equal(down(c, st).view(torch.int16), y.view(torch.int16))
        assert torch.equal(gate_up(c, c["hq"], c["hs"], c["perm"], st).view(torch.int16), act.view(torch.int16))


def test_prefill_sized_products():
    check(case(4096, 1024, 512, 32, 4), gather_too=False)
    check(case(2048, 2048, 768, 16, 8, skew=1.0), gather_too=False)


def test_arrays_past_32_bit_offsets():
    # more than 2^31 elements in the quantised rows, in gate/up's token rows and in
    # down's output; the last rows are checked
    rows, K = 66000, 32768
    tail = 40
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x[-tail:] = torch.randn(tail, K, generator=g, device=DEV).to(torch.bfloat16)
    q, s = torch.empty(rows, K, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    moe.moe_i8_quantize(x, rows, K, q, s)
    rq, rs = _plain.int8_rows(x[-tail:])
    assert torch.equal(q[-tail:], rq) and torch.equal(s[-tail:], rs) and bool((s[:-tail] == 0).all())
    del x
    off = torch.tensor([0, rows - 10, rows], dtype=torch.int32, device=DEV)
    # gate/up: H = 32768, I = 16; down: H = 32768, I = 16
    sh = moe.Shape.of(rows, K, 16, 2, 1, "int8")
    w_gu, gs = codes(g, 2, 32, K), scales(g, 2, 32) * 1e-6
    act = torch.empty(rows, 16, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_swiglu_i8(q, s, None, off, w_gu, gs, sh, act)
    v = _plain.grouped_int8(q[-tail:], s[-tail:], None, (off - (rows - tail)).clamp_min(0), w_gu, gs, 1)
    close_act(act[-tail:], v)
    del q
    aq, as_ = codes(g, rows, 16), scales(g, rows)
    w_d, ds = codes(g, 2, K, 16), scales(g, 2, K)
    y = torch.empty(rows, K, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_down_i8(aq, as_, off, w_d, ds, sh, y)
    close_y(y[-tail:], _plain.grouped_int8(aq[-tail:], as_[-tail:], None, (off - (rows - tail)).clamp_min(0), w_d, ds, 1))


def test_first_call_of_every_kernel_may_be_captured():
    # a fresh process whose first calls are under capture: set-up calls (function
    # attributes, occupancy, tensor maps) are legal there
    import os
    import subprocess
    import sys
    code = """
import torch, mixture_experts_expert_top_b200 as moe
D = dict(device="cuda")
T, H, I, E, k = 40, 256, 128, 8, 2
x = torch.randn(T, H, **D).to(torch.bfloat16); l = torch.randn(T, E, **D); b = torch.zeros(E, **D)
w = torch.ones(H, dtype=torch.bfloat16, **D)
q, s = torch.empty(T, H, dtype=torch.int8, **D), torch.empty(T, **D)
wg = torch.randint(-9, 9, (E, 2 * I, H), dtype=torch.int8, **D); wd = torch.randint(-9, 9, (E, H, I), dtype=torch.int8, **D)
gs, ds = torch.rand(E, 2 * I, **D), torch.rand(E, H, **D)
outs = []
sh = moe.Shape.of(T, H, I, E, k, "int8")
ws = torch.empty(moe.moe_workspace_size(sh), dtype=torch.uint8, **D)
out, out2 = torch.empty_like(x), torch.empty_like(x)
r = moe.Router.of("sigmoid")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    moe.moe_rmsnorm(x, None, w, 1e-6, T, H, moe.FMT_INT8, None, None, q, s)
    moe.moe_forward_scored(x, l, b, r, wg, gs, wd, ds, sh, out, ws)
g.replay(); torch.cuda.synchronize()
moe.moe_forward_scored(x, l, b, r, wg, gs, wd, ds, sh, out2, ws)
torch.cuda.synchronize()
assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and moe.moe_get_device_error() == 0
print("captured ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stderr[-2000:]


def test_two_calls_at_once_on_two_streams():
    c = case(900, 512, 256, 8, 2)
    d = case(60, 512, 256, 8, 2, seed=3)
    refs = [down(c), gate_up(c, c["hq"], c["hs"], c["perm"]), down(d), gate_up(d, d["hq"], d["hs"], d["perm"])]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(r) for r in refs] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o in zip(streams, outs):
            moe.moe_grouped_gemm_down_i8(c["aq"], c["as"], c["off"], c["w_d"], c["ds"], c["shape"], o[0], st)
            moe.moe_grouped_gemm_swiglu_i8(c["hq"], c["hs"], c["perm"], c["off"], c["w_gu"], c["gs"], c["shape"], o[1], st)
            moe.moe_grouped_gemm_down_i8(d["aq"], d["as"], d["off"], d["w_d"], d["ds"], d["shape"], o[2], st)
            moe.moe_grouped_gemm_swiglu_i8(d["hq"], d["hs"], d["perm"], d["off"], d["w_gu"], d["gs"], d["shape"], o[3], st)
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, refs):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# rows per expert around the sizes where another kernel or tile takes over (16 rows
# on average and 64 tokens, 24, 48; N steps of 16 and 32, blocks of 32, 64, 128, 256)
@pytest.mark.parametrize("T", [8, 9, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 96, 97, 127, 128, 160, 256, 511, 513])
def test_kernel_boundaries(T):
    check(case(T, 272, 144, 4, 2, seed=T))
    check(case(T, 144, 80, 1, 1, seed=T))


@pytest.mark.parametrize("T,H,I,E,k", [(1, 2048, 768, 8, 8), (16, 272, 144, 4, 2), (40, 512, 256, 8, 3), (64, 144, 80, 4, 1)])
def test_the_three_kernels_give_the_same_bits(T, H, I, E, k):
    """The same rows of the same experts in calls of 65 tokens and more, whose other
    rows go to one more expert: at most 64 tokens and 16 rows per expert take the
    warp kernel, more than 48 rows per expert the pair kernel, those between the
    single-CTA one."""
    c = case(T, H, I, E, k, seed=5)
    P, src = c["P"], c["perm"].long() // k
    a, a_s = c["hq"][src].contiguous(), c["hs"][src].contiguous()
    assert P <= 16 * E and (min(E, P) * 2 * I * H) <= 32 << 20
    y, act = down(c), gate_up(c, a, a_s, None)
    g = torch.Generator(device=DEV).manual_seed(6)
    more = lambda t, extra: torch.cat([t, extra])
    for T2, per_expert in ((65, 30), (400, 60)):
        P2 = T2 * k
        X = max(1, P2 // per_expert - E)                              # more experts, all but the last without rows
        assert P2 / (E + X) <= 48 if per_expert == 30 else P2 / (E + X) > 48
        d = {"shape": moe.Shape.of(T2, H, I, E + X, k, "int8"), "P": P2,
             "off": more(c["off"], torch.tensor([P] * (X - 1) + [P2], dtype=torch.int32, device=DEV)),
             "w_gu": more(c["w_gu"], codes(g, X, 2 * I, H)), "gs": more(c["gs"], scales(g, X, 2 * I) * 1e-3),
             "w_d": more(c["w_d"], codes(g, X, H, I)), "ds": more(c["ds"], scales(g, X, H)),
             "aq": more(c["aq"], codes(g, P2 - P, I)), "as": more(c["as"], scales(g, P2 - P))}
        assert torch.equal(down(d)[:P].view(torch.int16), y.view(torch.int16))
        a2, a2_s = more(a, codes(g, P2 - P, H)), more(a_s, scales(g, P2 - P) * 1e-2)
        assert torch.equal(gate_up(d, a2, a2_s, None)[:P].view(torch.int16), act.view(torch.int16))


# ---- the layer ----------------------------------------------------------------

def layer_inputs(T, H, I, E, k, seed=0, n_shared=0):
    g = torch.Generator().manual_seed(seed)
    hidden = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    gd = torch.Generator(device=DEV).manual_seed(seed)
    Et = E + n_shared
    w = lambda *s: (torch.randn(*s, generator=gd, device=DEV) * 0.02).to(torch.bfloat16)
    w_gu, gs = _plain.int8_rows(w(Et * 2 * I, H))
    w_d, ds = _plain.int8_rows(w(Et * H, I))
    return hidden, logits, w_gu.view(Et, 2 * I, H), gs.view(Et, 2 * I), w_d.view(Et, H, I), ds.view(Et, H)


LAYERS = [(1, 256, 128, 8, 2, 0), (64, 2048, 768, 128, 8, 0), (33, 272, 144, 8, 3, 2), (500, 512, 256, 32, 4, 0),
          (1024, 512, 256, 16, 4, 1), (3000, 256, 128, 8, 2, 0)]


@pytest.mark.parametrize("T,H,I,E,k,S", LAYERS)
def test_layer_equals_its_steps_and_is_near_the_exact_layer(T, H, I, E, k, S):
    hidden, logits, w_gu, gs, w_d, ds = layer_inputs(T, H, I, E, k, n_shared=S)
    out = moe.forward(hidden, logits, w_gu, w_d, k, gs, ds)
    out2 = moe.forward(hidden, logits, w_gu, w_d, k, gs, ds)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    # the step entry points
    sh = moe.Shape.of(T, H, I, E, k, "int8", n_shared=S)
    K, Et, P = k + S, E + S, T * (k + S)
    i32 = dict(dtype=torch.int32, device=DEV)
    ids, w = torch.empty(T, K, **i32), torch.empty(T, K, device=DEV)
    counts, off, perm, inv = (torch.empty(n, **i32) for n in (Et, Et + 1, P, P))
    ws = torch.empty(max(1, moe.moe_permute_workspace_size(sh)), dtype=torch.uint8, device=DEV)
    moe.moe_route(logits, sh, ids, w)
    moe.moe_permute(ids, sh, counts, off, perm, inv, ws=ws)
    hq, hs = torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    act = torch.empty(P, I, dtype=torch.bfloat16, device=DEV)
    aq, as_ = torch.empty(P, I, dtype=torch.int8, device=DEV), torch.empty(P, device=DEV)
    y, step = (torch.empty(n, H, dtype=torch.bfloat16, device=DEV) for n in (P, T))
    moe.moe_i8_quantize(hidden, T, H, hq, hs)
    moe.moe_grouped_gemm_swiglu_i8(hq, hs, perm, off, w_gu, gs, sh, act)
    moe.moe_i8_quantize(act, P, I, aq, as_)
    moe.moe_grouped_gemm_down_i8(aq, as_, off, w_d, ds, sh, y)
    moe.moe_finalize(y, w, inv, sh, step)
    torch.cuda.synchronize()
    assert torch.equal(step.view(torch.int16), out.view(torch.int16))
    # the layer in 64 bits from the same int8 operands, nothing rounded in between
    # but the int8 rows: rel-L2 within the layer's 1e-2
    rq, rs = _plain.int8_rows(hidden)
    v = _plain.grouped_int8(rq, rs, perm, off, w_gu, gs, K)
    a64 = _plain.swiglu(v)[0]
    rq, rs = _plain.int8_rows(a64.to(torch.bfloat16))
    y64 = _plain.grouped_int8(rq, rs, None, off, w_d, ds, K)
    ref = (y64[inv.long()].view(T, K, H) * w.double()[:, :, None]).sum(1)
    rel = float((out.double() - ref).norm() / ref.norm())
    assert rel <= 1e-2, rel


def test_norm_scored_route_and_int8_layer_together():
    # one block of a model: residual and norm (bf16 rows for the router, int8 rows
    # for the experts), router logits, scored routing, int8 products, combine
    T, H, I, E, k = 200, 512, 256, 32, 4
    hidden, _, w_gu, gs, w_d, ds = layer_inputs(T, H, I, E, k, seed=4)
    g = torch.Generator(device=DEV).manual_seed(9)
    res = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    nw = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
    w_r = torch.randn(E, H, generator=g, device=DEV) * 0.05
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    router = moe.Router.of("sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)
    sh = moe.Shape.of(T, H, I, E, k, "int8")
    bf = dict(dtype=torch.bfloat16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    res_out, yn = torch.empty(T, H, **bf), torch.empty(T, H, **bf)
    hq, hs = torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    moe.moe_rmsnorm(hidden, res, nw, 1e-6, T, H, moe.FMT_INT8, res_out, yn, hq, hs)
    logits = yn.float() @ w_r.T
    P = T * k
    ids, w = torch.empty(T, k, **i32), torch.empty(T, k, device=DEV)
    counts, off, perm, inv = (torch.empty(n, **i32) for n in (E, E + 1, P, P))
    moe.moe_route_scored(logits, bias, router, sh, ids, w)
    moe.moe_permute(ids, sh, counts, off, perm, inv)
    act, y, out = torch.empty(P, I, **bf), torch.empty(P, H, **bf), torch.empty(T, H, **bf)
    aq, as_ = torch.empty(P, I, dtype=torch.int8, device=DEV), torch.empty(P, device=DEV)
    moe.moe_grouped_gemm_swiglu_i8(hq, hs, perm, off, w_gu, gs, sh, act)
    moe.moe_i8_quantize(act, P, I, aq, as_)
    moe.moe_grouped_gemm_down_i8(aq, as_, off, w_d, ds, sh, y)
    moe.moe_finalize(y, w, inv, sh, out)
    torch.cuda.synchronize()
    rid, rw = _plain.route_scored(logits.cpu(), bias.cpu(), k, "sigmoid", 4, 2, 2, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # 64 bits throughout, dense over the selected experts, weights dequantised: int8
    # rows cost at most half a step of 127 per operand, about 1% of the row in L2
    _, y64 = _plain.rmsnorm(hidden, res, nw, 1e-6)
    ref = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = np.nonzero(rid == e)
        if len(t) == 0:
            continue
        ti = torch.from_numpy(t).to(DEV)
        a = _plain.swiglu(y64[ti] @ (w_gu[e].double() * gs[e].double()[:, None]).T)[0]
        ref.index_add_(0, ti, (a @ (w_d[e].double() * ds[e].double()[:, None]).T) *
                       torch.from_numpy(rw[t, j]).to(DEV)[:, None])
    rel = float((out.double() - ref).norm() / ref.norm())
    assert rel <= 3e-2, rel


def test_layer_replays_from_a_graph_and_shares_a_workspace_in_turn():
    T, H, I, E, k = 48, 512, 256, 16, 4
    hidden, logits, w_gu, gs, w_d, ds = layer_inputs(T, H, I, E, k)
    ref = moe.forward(hidden, logits, w_gu, w_d, k, gs, ds)
    sh = moe.Shape.of(T, H, I, E, k, "int8")
    ws = torch.empty(moe.moe_workspace_size(sh), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(ref) for _ in range(2)]
    ins = [(hidden.clone(), logits.clone()), (hidden.flip(0).contiguous(), logits.flip(0).contiguous())]
    graphs = []
    for (h, l), o in zip(ins, outs):                 # two graphs on one workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_forward(h, l, w_gu, gs, w_d, ds, sh, o, ws, torch.cuda.current_stream())
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0].view(torch.int16), ref.view(torch.int16))
    assert torch.equal(outs[1].view(torch.int16), ref.flip(0).contiguous().view(torch.int16))


@pytest.mark.parametrize("T", [100, 2500])
def test_host_form(T):
    H, I, E, k = 256, 128, 8, 2
    hidden, logits, w_gu, gs, w_d, ds = layer_inputs(T, H, I, E, k)
    ref = moe.forward(hidden, logits, w_gu, w_d, k, gs, ds)
    sh = moe.Shape.of(T, H, I, E, k, "int8")
    ws = torch.empty(moe.moe_forward_host_workspace_size(sh), dtype=torch.uint8, device=DEV)
    out = torch.empty(T, H, dtype=torch.bfloat16).pin_memory()
    moe.moe_forward_host(hidden.cpu().pin_memory(), logits.cpu().pin_memory(), w_gu, gs, w_d, ds, sh, out, ws)
    assert torch.equal(out.view(torch.int16), ref.cpu().view(torch.int16))


def test_debug_bounds_build_agrees():
    c = case(300, 256, 128, 8, 2)
    y = down(c)
    act = gate_up(c, c["hq"], c["hs"], c["perm"])
    moe_build.build(debug_bounds=True)
    with moe.debug_bounds_library():
        assert torch.equal(down(c).view(torch.int16), y.view(torch.int16))
        assert torch.equal(gate_up(c, c["hq"], c["hs"], c["perm"]).view(torch.int16), act.view(torch.int16))
        assert moe.moe_get_device_error() == 0
