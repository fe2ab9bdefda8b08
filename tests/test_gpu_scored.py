"""moe_route_scored and moe_forward_scored against the plain 64-bit form.

Ids: equal. Weights, with u = 2^-24 (half an fp32 step): l - max rounds by
u |l - max|, which the exponential turns into a relative error; expf is within
2 ulp (4u); a sum over n terms adds at most n u and the average of its terms'
errors (|l - max| averages at most ln E < 7 over a softmax); division, scale
and store one u each. Renormalised, numerator and sum both carry the
exponential's error: a slot's own |l - max| = d, and the average over the
selected, below ln 32 < 4. So |w - ref| <= u ref (40 + k + ceil(E/32) + 2 d),
plus 4 steps of the smallest subnormal where the exponential underflows.
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
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    moe_build.build()
    moe.lib()
    yield
    assert moe.moe_get_device_error() == 0


def run(logits, bias, k, n_shared=0, stream=None, **kw):
    T, E = logits.shape
    r = moe.Router.of(logits="bf16" if logits.dtype == torch.bfloat16 else "fp32", **kw)
    sh = moe.Shape.of(T, 128, 64, E, k, n_shared=n_shared)
    K = k + n_shared
    ids = torch.full((T + 1, K), -7, dtype=torch.int32, device=DEV)      # one row more than is written
    w = torch.full((T + 1, K), -7.0, device=DEV)
    moe.moe_route_scored(logits.to(DEV), None if bias is None else bias.to(DEV), r, sh, ids, w, stream)
    torch.cuda.synchronize()
    assert torch.all(ids[T] == -7) and torch.all(w[T] == -7.0)
    return ids[:T].cpu().numpy(), w[:T].cpu().double().numpy()


def check(logits, bias, k, n_shared=0, **kw):
    ids, w = run(logits, bias, k, n_shared, **kw)
    rid, rw = _plain.route_scored(logits, bias, k, n_shared=n_shared, **kw)
    assert np.array_equal(ids, rid), f"{int((ids != rid).any(1).sum())} rows differ, first {np.argwhere((ids != rid).any(1))[0]}"
    E = logits.shape[1]
    l = logits.double().numpy()
    l = np.where(np.isnan(l), -INF, l)
    sel = np.take_along_axis(l, rid[:, :k], 1)
    with np.errstate(invalid="ignore"):
        # non-renormalised softmax is taken relative to the row's maximum, the rest to the selected one's
        top = l.max(1) if kw.get("score", "softmax") == "softmax" else sel.max(1)
        d = np.where(np.isfinite(sel) & np.isfinite(top)[:, None], np.abs(sel - top[:, None]), 0.0)
    d = np.concatenate([d, np.zeros((len(l), n_shared))], 1)
    tol = 2.0 ** -24 * (40 + k + -(-E // 32) + 2 * d) * np.abs(rw) + 4 * 2.0 ** -149
    assert np.all(np.abs(w - rw) <= tol), float((np.abs(w - rw) / np.maximum(tol, 1e-300)).max())


def logits_of(T, E, seed, dtype=torch.float32, sigma=1.5):
    return (torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * sigma).to(dtype)


def bias_of(E, seed, sigma=0.1):
    return torch.randn(E, generator=torch.Generator().manual_seed(1000 + seed)) * sigma


# E: one lane per expert, fewer, odd counts, each register count of a lane (1, 2, 4, 8, 16, 32)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (65, 31, 5), (64, 32, 32), (33, 60, 6), (130, 64, 8),
                                   (77, 100, 7), (256, 128, 8), (301, 256, 8), (50, 257, 16), (40, 512, 10),
                                   (20, 1000, 32), (9, 1024, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_no_groups(T, E, k, score, biased, dtype):
    check(logits_of(T, E, T + E, dtype), bias_of(E, E) if biased else None, k, score=score,
          renormalize=(T + k) % 2 == 0, scale=1.0 if T % 2 else 2.5, n_shared=min(T % 3, 32 - k))


@pytest.mark.parametrize("T,E,k,G,keep", [(301, 256, 8, 8, 4), (64, 64, 6, 8, 3), (33, 32, 4, 4, 1), (40, 96, 5, 32, 9),
                                          (29, 60, 6, 5, 2), (17, 1024, 8, 32, 4), (50, 160, 6, 8, 3), (12, 12, 4, 2, 2),
                                          (23, 250, 3, 2, 1), (31, 40, 2, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
def test_groups(T, E, k, G, keep, score, top, biased):
    check(logits_of(T, E, T + E + G), bias_of(E, G) if biased else None, k, score=score, n_group=G, topk_group=keep,
          group_top=top, renormalize=T % 2 == 0, scale=2.5)
    check(logits_of(T, E, T + E + G, torch.bfloat16), bias_of(E, G) if biased else None, k, score=score, n_group=G,
          topk_group=keep, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [1, 4])
def test_ties_go_to_the_lower_id(score, G):
    # equal logits, with and without equal biases; -0 equals +0
    l = torch.zeros(4, 64)
    l[1, ::2] = -0.0
    l[2, 10:20] = 1.0
    l[3] = torch.arange(64) % 3
    for b in (None, torch.zeros(64), torch.full((64,), 0.25)):
        for top in (1, 2):
            check(l, b, 8, score=score, n_group=G, topk_group=max(1, G // 2), group_top=top)


def test_order_decided_in_the_last_bits():
    # s + b of two experts differ by less than an fp32 step, in either direction:
    # the biases undo most of the difference of the scores
    g = torch.Generator().manual_seed(3)
    T, E = 512, 64
    l = torch.randn(T, E, generator=g)
    for score in ("softmax", "sigmoid"):
        s = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
        b = torch.zeros(E)
        b[1::2] = (s[7, 0::2] - s[7, 1::2]).float()           # in row 7 each pair nearly ties
        check(l, b, 8, score=score)
        rows = l[7:8] + torch.arange(T)[:, None] * 2.0 ** -23
        check(rows, b, 8, score=score)
        check(rows, b, 8, score=score, n_group=8, topk_group=4, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_special_values(score, renorm):
    E = 16
    l = torch.randn(12, E, generator=torch.Generator().manual_seed(5))
    l[0] = -INF                                              # nothing left: weights 0
    l[1] = NAN
    l[2, 3:] = -INF                                          # fewer than k finite
    l[3, 5] = INF
    l[4, 5:8] = INF                                          # +inf shares
    l[5] = -200.0 + torch.arange(E)                          # every sigmoid far below the fp32 range of s
    l[6] = 300.0 - 50 * torch.arange(E)
    l[7] = torch.finfo(torch.float32).min                    # a mask of the type's lowest value
    l[8, ::2] = torch.finfo(torch.float32).min
    l[9] = 1e-30 * torch.arange(E)
    l[10] = torch.finfo(torch.float32).max
    l[11, 0] = NAN
    check(l, None, 6, score=score, renormalize=renorm)
    check(l, None, 6, score=score, renormalize=renorm, n_group=4, topk_group=2, group_top=1)
    finite = l[[2, 3, 8, 9, 11]]
    check(finite, bias_of(E, 1), 6, score=score, renormalize=renorm)
    check(l[[0, 1, 4, 7]], bias_of(E, 2), 6, score=score, renormalize=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_special_biases(score):
    E = 64
    l = logits_of(40, E, 2)
    b = bias_of(E, 3)
    b[::3] = -INF                                            # experts switched off
    check(l, b, 8, score=score)
    check(l, b, 8, score=score, n_group=8, topk_group=4, group_top=2)
    b[5] = INF                                               # an expert that every token takes
    check(l, b, 8, score=score)
    b[7] = NAN
    check(l, b, 8, score=score)
    off = torch.full((E,), -INF)
    off[:3] = 0.0                                            # fewer experts on than slots: the rest have weight 0
    ids, w = run(l, off, 8, score=score)
    assert np.all(w[:, 3:] == 0) and np.all(ids[:, 3:] == np.arange(3, 8))
    check(l, off, 8, score=score)
    check(l, torch.full((E,), 1e30), 8, score=score)         # the scores vanish beside the bias: ties
    check(l, torch.full((E,), 1e4) + bias_of(E, 9), 8, score=score)
    check(l, torch.where(torch.arange(E) < 8, 3e38, -3e38), 8, score=score)


def test_near_biases_decide_rows_without_scores():
    # every logit -inf: all scores are 0 and the order is the biases', which here
    # differ by one fp32 step near 1e-30 and would vanish beside any score
    E = 16
    b = torch.full((E,), -1.0) * 1e-28
    b[3] = 1e-30
    b[7] = torch.nextafter(b[3], torch.tensor(1.0))
    b[11] = torch.nextafter(b[7], torch.tensor(1.0))
    l = torch.full((3, E), -INF)
    l[1] = NAN
    for score in ("softmax", "sigmoid"):
        ids, w = run(l, b, 3, score=score)
        assert np.array_equal(ids, np.tile([11, 7, 3], (3, 1))) and np.all(w == 0)
        check(l, b, 3, score=score)
        check(l, b, 3, score=score, n_group=4, topk_group=3, group_top=2)


def test_equals_moe_route_where_both_apply():
    l = logits_of(300, 128, 8).to(DEV)
    sh = moe.Shape.of(300, 128, 64, 128, 8)
    a, aw = torch.empty(300, 8, dtype=torch.int32, device=DEV), torch.empty(300, 8, device=DEV)
    b, bw = torch.empty_like(a), torch.empty_like(aw)
    moe.moe_route(l, sh, a, aw)
    moe.moe_route_scored(l, None, moe.Router.of(), sh, b, bw)
    assert torch.equal(a, b) and torch.equal(aw, bw)


def test_large_batch_on_a_side_stream():
    T, E = 16384, 256
    l, b = logits_of(T, E, 4), bias_of(E, 4)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)
    st = torch.cuda.Stream()
    ld = l.to(DEV)
    torch.cuda.synchronize()
    ids, w = run(ld, b, 8, stream=st, **kw)
    # the same in torch, in 64 bits
    s = torch.sigmoid(l.double())
    c = s + b.double()
    g = c.view(T, 8, 32).topk(2, dim=2).values.sum(2)
    keep = torch.zeros(T, 8, dtype=torch.bool).scatter_(1, g.topk(4, dim=1).indices, True)
    c = torch.where(keep.repeat_interleave(32, 1), c, torch.full_like(c, -INF))
    rid = c.topk(8, dim=1).indices
    assert np.array_equal(ids, rid.numpy())
    rw = s.gather(1, rid)
    rw = (rw / rw.sum(1, keepdim=True) * 2.5).numpy()
    assert np.all(np.abs(w - rw) <= 2.0 ** -24 * 60 * rw)


def test_logits_past_32_bit_offsets():
    T, E, k = 2_200_000, 1000, 2
    l = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    tail = logits_of(50, E, 6, torch.bfloat16)
    l[-50:] = tail.to(DEV)
    b = bias_of(E, 6).to(DEV)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    moe.moe_route_scored(l, b, moe.Router.of("sigmoid", logits="bf16"), moe.Shape.of(T, 8, 8, E, k), ids, w)
    torch.cuda.synchronize()
    assert np.array_equal(ids[-50:].cpu().numpy(), _plain.route_scored(tail, b.cpu(), k, "sigmoid")[0])
    assert bool((ids[:-50] == torch.sort(b, descending=True, stable=True).indices[:k].to(torch.int32)).all())


def test_captured_and_replayed_on_new_logits():
    T, E, k = 64, 64, 6
    sh, r = moe.Shape.of(T, 128, 64, E, k), moe.Router.of("sigmoid", 8, 3, 2)
    l, b = logits_of(T, E, 1).to(DEV), bias_of(E, 1).to(DEV)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device=DEV), torch.zeros(T, k, device=DEV)
    moe.moe_route_scored(l, b, r, sh, ids, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_route_scored(l, b, r, sh, ids, w, torch.cuda.current_stream())
    for seed in (7, 8):
        l.copy_(logits_of(T, E, seed))
        g.replay()
        torch.cuda.synchronize()
        rid, _ = _plain.route_scored(l.cpu(), b.cpu(), k, "sigmoid", 8, 3, 2)
        assert np.array_equal(ids.cpu().numpy(), rid)


# ---- the layer with the scored router ---------------------------------------

LAYERS = [
    ("bf16", moe_synth.MoeConfig("s1", T=40, H=256, I=128, E=16, k=4), dict(score="sigmoid", n_group=4, topk_group=2,
                                                                            group_top=2, scale=2.5), True),
    ("bf16 shared", moe_synth.MoeConfig("s2", T=17, H=256, I=128, E=16, k=3, n_shared=1), dict(score="softmax",
                                                                                              renormalize=False), True),
    ("int4", moe_synth.MoeConfig("s3", T=40, H=256, I=128, E=16, k=4, fmt="int4_g128"), dict(score="sigmoid"), False),
    ("mxfp8", moe_synth.MoeConfig("s4", T=300, H=256, I=128, E=16, k=4, fmt="mxfp8"), dict(score="sigmoid"), True),
    ("prefill", moe_synth.MoeConfig("s5", T=1500, H=256, I=128, E=8, k=4), dict(score="sigmoid"), True),
]


@pytest.mark.parametrize("what,cfg,kw,biased", LAYERS, ids=[x[0] for x in LAYERS])
def test_forward_scored_equals_its_steps(what, cfg, kw, biased):
    inp = moe_synth.gen_inputs(cfg, seed=3)
    d = {n: t.to(DEV) for n, t in inp.items()}
    bias = bias_of(cfg.E, 5) if biased else None
    S = cfg.n_shared
    sh = moe.Shape.of(cfg.T, cfg.H, cfg.I, cfg.E, cfg.k, cfg.fmt, n_shared=S)
    r = moe.Router.of(**kw)
    out = moe.forward(d["hidden"], d["logits"], d["w_gu"], d["w_d"], cfg.k, d.get("w_gu_scales"), d.get("w_d_scales"),
                      router=r, bias=None if bias is None else bias.to(DEV))
    again = torch.empty_like(out)
    ws = torch.empty(moe.moe_workspace_size(sh), dtype=torch.uint8, device=DEV)
    moe.moe_forward_scored(d["hidden"], d["logits"], None if bias is None else bias.to(DEV), r, d["w_gu"],
                           d.get("w_gu_scales"), d["w_d"], d.get("w_d_scales"), sh, again, ws)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    # routing by the plain form, then the step entry points
    K, Et, P = cfg.k + S, cfg.E + S, cfg.T * (cfg.k + S)
    ids, w = run(inp["logits"], bias, cfg.k, S, **kw)
    rid, _ = _plain.route_scored(inp["logits"], bias, cfg.k, n_shared=S, **kw)
    assert np.array_equal(ids, rid)
    _, offsets, perm, inv = oracle.permute(ids, Et)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    act = torch.empty(P, cfg.I, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(P, cfg.H, dtype=torch.bfloat16, device=DEV)
    step = torch.empty_like(out)
    if cfg.fmt == "mxfp8":
        q, s = (dev(a) for a in oracle.mx_quantize(inp["hidden"]))
        aq = torch.empty(P, cfg.I, dtype=torch.uint8, device=DEV)
        as_ = torch.empty(P, cfg.I // 32, dtype=torch.uint8, device=DEV)
        moe.moe_grouped_gemm_swiglu_mx(q, s, dev(perm), dev(offsets), d["w_gu"], d["w_gu_scales"], sh, aq, as_)
        moe.moe_grouped_gemm_down_mx(aq, as_, dev(offsets), d["w_d"], d["w_d_scales"], sh, y)
    else:
        if moe.moe_forward_gathers_in_gemm(sh):
            rows, pm = d["hidden"], dev(perm)
        else:
            rows, pm = dev(oracle.gather(inp["hidden"], perm, K).view(np.int16)).view(torch.bfloat16), None
        moe.moe_grouped_gemm_swiglu(rows, pm, dev(offsets), d["w_gu"], d.get("w_gu_scales"), sh, act)
        moe.moe_grouped_gemm_down(act, dev(offsets), d["w_d"], d.get("w_d_scales"), sh, y)
    moe.moe_finalize(y, dev(w.astype(np.float32)), dev(inv), sh, step)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_bits(step), bf16_bits(out))


@pytest.mark.parametrize("dtype", [torch.float32, torch.int64, torch.bfloat16])
def test_forward_scored_takes_a_workspace_of_any_type(dtype):
    cfg = moe_synth.MoeConfig("s6", T=24, H=256, I=128, E=16, k=4)
    d = {n: t.to(DEV) for n, t in moe_synth.gen_inputs(cfg, seed=4).items()}
    r, sh = moe.Router.of("sigmoid"), moe.Shape.of(cfg.T, cfg.H, cfg.I, cfg.E, cfg.k)
    ref = moe.forward(d["hidden"], d["logits"], d["w_gu"], d["w_d"], cfg.k, router=r)
    size = moe.moe_workspace_size(sh)
    ws = torch.zeros(-(-size // dtype.itemsize), dtype=dtype, device=DEV)
    out = torch.empty_like(ref)
    moe.moe_forward_scored(d["hidden"], d["logits"], None, r, d["w_gu"], None, d["w_d"], None, sh, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_forward_scored(d["hidden"], d["logits"], None, r, d["w_gu"], None, d["w_d"], None, sh, out, ws[:8])


def test_binding_refuses_another_device_and_host_memory():
    sh, r = moe.Shape.of(4, 128, 64, 8, 2), moe.Router.of()
    ids, w = torch.empty(4, 2, dtype=torch.int32, device=DEV), torch.empty(4, 2, device=DEV)
    with pytest.raises(ValueError):
        moe.moe_route_scored(torch.zeros(4, 8), None, r, sh, ids, w)                    # host logits
    with pytest.raises(ValueError):
        moe.moe_route_scored(torch.zeros(4, 8, device=DEV), torch.zeros(8), r, sh, ids, w)
    with pytest.raises(ValueError):
        moe.moe_route_scored(torch.zeros(3, 8, device=DEV), None, r, sh, ids, w)        # too few rows


# from 2960 rows on, rows of at most 16 slots are weighed several per warp (8 or
# 16 lanes each): T ends a block after each count of rows, slots fill the lanes
# or leave some, experts take each register count of a lane up to 8
@pytest.mark.parametrize("T,E,k,n_shared", [(2960, 256, 8, 0), (2961, 128, 6, 2), (2962, 60, 4, 1), (2963, 31, 1, 0),
                                            (3001, 160, 12, 0), (2967, 256, 15, 1), (2970, 64, 8, 1), (2959, 64, 8, 0),
                                            (2960, 100, 16, 1), (2966, 300, 8, 0)])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
def test_long_calls(T, E, k, n_shared, score, renormalize, biased):
    l = logits_of(T, E, T + E)
    l[5] = -INF
    l[6, : E - 1] = -INF
    l[T - 1, ::2] = NAN
    if T % 2:
        l = l.to(torch.bfloat16)
    b = bias_of(E, E) if biased else None
    G = 4 if E % 4 == 0 and k <= E // 2 and E >= 60 else 1
    kw = dict(score=score, renormalize=renormalize, scale=2.5, n_group=G, topk_group=max(1, G // 2), group_top=1 + biased)
    check(l, b, k, n_shared, **kw)
    # and as the same rows do in short calls, bit by bit
    ids, w = run(l, b, k, n_shared, **kw)
    for lo, hi in ((0, 9), (1000, 1007), (T - 11, T)):
        i, v = run(l[lo:hi], b, k, n_shared, **kw)
        assert np.array_equal(i, ids[lo:hi]) and np.array_equal(v, w[lo:hi])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 8), (60, 5), (256, 8)])
def test_groups_whose_biases_span_more_than_the_fp32_range(score, E, G):
    # a group's two largest choices may cancel (3e38 - 3e38 = 0 in 64 bits) or add past
    # the fp32 range, and the choices' span hi - lo is past it too
    l = logits_of(40, E, 7)
    size = E // G
    b = torch.zeros(E)
    b[0] = 3e38
    b[1:size] = -3e38                                        # group 0: 0, below every s1 + s2 > 0
    for k, keep, top in ((4, 2, 2), (2, 1, 2), (4, 2, 1), (6, G - 1, 2)):
        check(l, b, k, score=score, n_group=G, topk_group=keep, group_top=top)
    b[size] = 2e38                                           # group 1: 2e38, its second one near 0
    check(l, b, 4, score=score, n_group=G, topk_group=1, group_top=2)
    b[2 * size:2 * size + 2] = 3e38                          # group 2: 6e38
    b[3 * size:4 * size] = -3e38                             # group 3: -6e38
    b[3 * size] = -INF
    for keep in (1, 2, G - 1, G):
        check(l, b, 4, score=score, n_group=G, topk_group=keep, group_top=2)
    check(l, b, 8, score=score)                              # without groups


@pytest.mark.parametrize("T", [40, 3000])
def test_sigmoid_weights_of_scores_near_and_below_the_smallest_normal(T):
    # s = exp(l) from 2^-83 down to 2^-150: as they are, and relative to a selected
    # score that is larger by any factor
    E, k = 64, 8
    l = torch.full((T, E), -120.0)
    l[:, :k] = -60.0 - 44.0 * torch.rand(T, k, generator=torch.Generator().manual_seed(1))
    check(l, None, k, score="sigmoid", renormalize=False)
    check(l, None, k, score="sigmoid")
    for top in (-59.0, -50.0, -61.0, -20.0, 3.0):
        l[:, 3] = top
        check(l, None, k, score="sigmoid")
        check(l, None, k, score="sigmoid", renormalize=False)


def test_as_many_rows_as_a_shape_allows():
    T = 2 ** 31 - 1
    l = torch.zeros(T, 1, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((T, 1), -7, dtype=torch.int32, device=DEV)
    w = torch.empty(T, 1, device=DEV)
    moe.moe_route_scored(l, None, moe.Router.of(logits="bf16"), moe.Shape.of(T, 8, 8, 1, 1), ids, w)
    torch.cuda.synchronize()
    for lo in range(0, T, 2 ** 28):
        assert bool((ids[lo:lo + 2 ** 28] == 0).all()) and bool((w[lo:lo + 2 ** 28] == 1).all())
