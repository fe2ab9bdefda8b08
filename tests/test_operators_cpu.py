"""Host side of the scored router, the RMS norm, the int8 rows and products and
moe_forward_scored: what each entry point refuses, before anything is
enqueued (no GPU needed, addresses are never used), and the plain forms that
the GPU tests compare with."""

import ctypes
import os

import numpy as np
import pytest
import torch

import _plain
import moe_synth
import mixture_experts_expert_top_b200 as moe
from mixture_experts_expert_top_b200 import build as moe_build

A = 1 << 20            # an aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    moe_build.build()


def router(**kw):
    return moe.Router.of(**kw)


ROUTE_SHAPE = (16, 128, 64, 64, 8)


@pytest.mark.parametrize("kw,shape,status", [
    (dict(n_group=3), ROUTE_SHAPE, 1),                              # 64 experts do not split into 3 groups
    (dict(n_group=0), ROUTE_SHAPE, 1),
    (dict(n_group=8, topk_group=9), ROUTE_SHAPE, 1),                # more groups kept than there are
    (dict(n_group=8, topk_group=0), ROUTE_SHAPE, 1),
    (dict(n_group=16, topk_group=1), ROUTE_SHAPE, 1),               # 4 experts kept, 8 wanted
    (dict(n_group=8, topk_group=4, group_top=3), ROUTE_SHAPE, 1),
    (dict(n_group=32, topk_group=32, group_top=2), (16, 128, 64, 32, 8), 1),   # groups of one expert
    (dict(scale=float("nan")), ROUTE_SHAPE, 1),
    (dict(scale=float("inf")), ROUTE_SHAPE, 1),
    (dict(n_group=64, topk_group=64), ROUTE_SHAPE, 2),              # more than 32 groups
    (dict(), (16, 128, 64, 8, 9), 1),                               # k > E
    (dict(), (16, 128, 64, 2048, 2), 2),                            # E > 1024
])
def test_scored_router_refuses(kw, shape, status):
    L, sh, r = moe.lib(), moe.Shape.of(*shape), router(**kw)
    assert L.moe_route_scored(A, None, ctypes.byref(r), ctypes.byref(sh), A, A, None) == status
    assert L.moe_forward_scored(A, A, None, ctypes.byref(r), A, None, A, None, ctypes.byref(sh), A, A, 1 << 30,
                                None) == status


def test_scored_router_refuses_arguments():
    L, sh, r = moe.lib(), moe.Shape.of(*ROUTE_SHAPE), router()
    f = L.moe_route_scored
    rr, ss = ctypes.byref(r), ctypes.byref(sh)
    assert f(A, None, None, ss, A, A, None) == 1                    # no router
    assert f(None, None, rr, ss, A, A, None) == 1
    assert f(A, None, rr, ss, None, A, None) == 1
    assert f(A, None, rr, ss, A, None, None) == 1
    assert f(A + 2, None, rr, ss, A, A, None) == 1                  # fp32 logits need 4-byte alignment
    assert f(A, A + 1, rr, ss, A, A, None) == 1
    assert f(A, None, rr, ss, A + 1, A, None) == 1
    for name, value in (("score", 2), ("logits", 2), ("renormalize", 2), ("group_top", 0)):
        bad = router()
        setattr(bad, name, value)
        assert f(A, None, ctypes.byref(bad), ss, A, A, None) == 1
    r16 = router(logits="bf16")
    assert f(A + 1, None, ctypes.byref(r16), ss, A, A, None) == 1   # bf16 logits need 2
    empty = moe.Shape.of(0, 128, 64, 64, 8)
    assert f(None, None, rr, ctypes.byref(empty), None, None, None) == 0


@pytest.mark.parametrize("rows,H,fmt,ptrs,status", [
    (4, 128, 0, dict(y=None), 1),                                   # nothing to write
    (4, 128, 0, dict(q=A, scales=A), 1),                            # bf16 rows have no codes
    (4, 128, 4, dict(), 1),                                         # int8 without codes
    (4, 128, 4, dict(q=A), 1),                                      # codes without scales
    (4, 128, 2, dict(scales=A), 1),
    (4, 128, 0, dict(residual=A), 1),                               # a residual without its output
    (4, 128, 0, dict(residual_out=A), 1),
    (4, 128, 0, dict(x=None), 1),
    (4, 128, 0, dict(weight=None), 1),
    (4, 128, 0, dict(x=A + 8), 1),
    (4, 128, 4, dict(q=A + 8, scales=A), 1),
    (4, 128, 4, dict(q=A, scales=A + 2), 1),
    (4, 128, 0, dict(eps=0.0), 1),
    (4, 128, 0, dict(eps=-1.0), 1),
    (4, 128, 0, dict(eps=float("nan")), 1),
    (4, 128, 0, dict(eps=float("inf")), 1),
    (4, 124, 0, dict(), 1),                                         # H % 8
    (4, 136, 4, dict(q=A, scales=A), 1),                            # H % 16
    (4, 144, 2, dict(q=A, scales=A), 1),                            # H % 32
    (4, 0, 0, dict(), 1),
    (-1, 128, 0, dict(), 1),
    (4, 128, 5, dict(), 1),                                         # unknown format
    (4, 32776, 0, dict(), 2),                                       # longer than a row may be
    (0, 128, 0, dict(x=None, weight=None, y=None), 0),              # no rows: nothing to do
])
def test_rmsnorm_refuses(rows, H, fmt, ptrs, status):
    p = dict(x=A, residual=None, weight=A, eps=1e-6, residual_out=None, y=A, q=None, scales=None)
    p.update(ptrs)
    assert moe.lib().moe_rmsnorm(p["x"], p["residual"], p["weight"], p["eps"], rows, H, fmt, p["residual_out"], p["y"],
                                 p["q"], p["scales"], None) == status


def test_int8_entry_points_refuse():
    L = moe.lib()
    q = L.moe_i8_quantize
    assert q(A, -1, 128, A, A, None) == 1
    assert q(A, 4, 120, A, A, None) == 1                            # K % 16
    assert q(A, 4, 0, A, A, None) == 1
    assert q(A, 4, 32784, A, A, None) == 2
    assert q(None, 4, 128, A, A, None) == 1
    assert q(A, 4, 128, A + 8, A, None) == 1
    assert q(A, 4, 128, A, A + 2, None) == 1
    assert q(None, 0, 128, None, None, None) == 0
    sh = moe.Shape.of(16, 256, 128, 8, 2, "int8")
    b = ctypes.byref
    gu, dn = L.moe_grouped_gemm_swiglu_i8, L.moe_grouped_gemm_down_i8
    other = moe.Shape.of(16, 256, 128, 8, 2, "mxfp8")
    assert gu(A, A, None, A, A, A, b(other), A, None) == 1          # another format's shape
    assert dn(A, A, A, A, A, b(other), A, None) == 1
    for args in ([None, A, None, A, A, A], [A, None, None, A, A, A], [A, A, None, None, A, A], [A, A, None, A, None, A],
                 [A, A, None, A, A, None], [A + 8, A, None, A, A, A], [A, A, A + 2, A, A, A], [A, A, None, A, A + 8, A],
                 [A, A, None, A, A, A + 2]):
        assert gu(*args, b(sh), A, None) == 1, args
        if args[2] is None:
            assert dn(*(args[:2] + args[3:]), b(sh), A, None) == 1, args
    assert gu(A, A, None, A, A, A, b(sh), None, None) == 1
    assert dn(A, A, A, A, A, b(sh), A + 2, None) == 1
    # the bf16 and MX entry points refuse int8 shapes
    assert L.moe_grouped_gemm_swiglu(A, None, A, A, A, b(sh), A, None) == 2
    assert L.moe_grouped_gemm_down(A, A, A, A, b(sh), A, None) == 2
    assert L.moe_grouped_gemm_swiglu_mx(A, A, None, A, A, A, b(sh), A, A, None) == 1
    assert L.moe_grouped_gemm_down_mx(A, A, A, A, A, b(sh), A, None) == 1
    # int8 weights need scales; a short workspace
    assert L.moe_forward(A, A, A, None, A, None, b(sh), A, A, 1 << 30, None) == 1
    assert L.moe_forward(A, A, A, A, A, A, b(sh), A, A, 64, None) == 3
    r = router()
    assert L.moe_forward_scored(A, A, None, b(r), A, A, A, A, b(sh), A, A, 64, None) == 3
    assert L.moe_forward_scored(A, A, None, b(r), A, A, A, A, b(sh), A, A + 16, 1 << 30, None) == 1
    none = moe.Shape.of(0, 256, 128, 8, 2, "int8")
    assert gu(None, None, None, None, None, None, b(none), None, None) == 0
    assert dn(None, None, None, None, None, b(none), None, None) == 0


@pytest.mark.parametrize("shape,ok", [
    ((16, 144, 48, 8, 2, 4), True),
    ((16, 136, 48, 8, 2, 4), False),           # H % 16
    ((16, 144, 40, 8, 2, 4), False),           # I % 16
    ((16, 32768, 64, 8, 2, 4), True),
    ((16, 32784, 64, 8, 2, 4), False),         # longer than a row may be
    ((16, 64, 32784, 8, 2, 4), False),
])
def test_int8_shapes(shape, ok):
    assert (moe.moe_workspace_size(moe.Shape.of(*shape)) > 0) == ok


def test_int8_kernel_count_and_workspace():
    sh = lambda T: moe.Shape.of(T, 2048, 768, 128, 8, "int8")
    # route + permute in one CTA, hidden's rows, gate/up, act's rows, down, finalize
    assert moe.moe_forward_kernel_count(sh(64)) == 6
    assert moe.moe_forward_kernel_count(sh(65)) == 7
    # prefill: two bucketing kernels; the quantisation writes the permuted rows itself
    assert moe.moe_forward_kernel_count(sh(8192)) == 8
    assert not moe.moe_forward_is_fused(sh(64))
    assert moe.moe_forward_gathers_in_gemm(sh(64)) and not moe.moe_forward_gathers_in_gemm(sh(8192))
    # the host form stages its inputs behind the layer's own workspace
    P, gap = 8192 * 8, moe.moe_forward_host_workspace_size(sh(8192)) - moe.moe_workspace_size(sh(8192))
    assert gap >= 8192 * (2048 * 4 + 128 * 4)
    assert moe.moe_workspace_size(sh(8192)) > P * (2048 + 768 + 2 * 768 + 2 * 2048)


def test_binding_refuses_tensors_it_cannot_pass():
    # host tensors, short ones and other types are refused before the library is called
    bf = torch.zeros(4, 128, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        moe.moe_i8_quantize(bf, 4, 128, q, s, stream=0)                             # host memory
    with pytest.raises(TypeError):
        moe.moe_i8_quantize(bf.float(), 4, 128, q, s, stream=0)
    with pytest.raises(ValueError):
        moe.moe_i8_quantize(bf, 5, 128, q, s, stream=0)                             # too short
    with pytest.raises(ValueError):
        moe.moe_i8_quantize(bf.t(), 4, 128, q, s, stream=0)                         # not contiguous
    sh = moe.Shape.of(4, 128, 64, 8, 2)
    with pytest.raises(TypeError):                                                  # fp32 logits for a bf16 router
        moe.moe_route_scored(torch.zeros(4, 8), None, router(logits="bf16"), sh, torch.zeros(4, 2, dtype=torch.int32),
                             torch.zeros(4, 2), stream=0)
    with pytest.raises(TypeError):
        moe.moe_rmsnorm(bf, None, bf[0], 1e-6, 4, 128, moe.FMT_INT8, None, None, q.to(torch.uint8), s, stream=0)
    with pytest.raises(ValueError):
        moe.forward(bf, torch.zeros(4, 8), bf, bf, 2, bias=torch.zeros(8))          # a bias without a router


# ---- the layer's weights: types and sizes by format ---------------------------

LAYER = (4, 256, 128, 8, 2)          # T, H, I, E, top_k


def layer_call(which, fmt, codes, scales):
    """One call of a layer entry point with weights of these types; `scales` may also be a function of the number of
    scales per weight array (an array of another length)."""
    T, H, I, E, k = LAYER
    per = {"bf16": (1, 0), "int4_g128": (2, 128), "mxfp8": (1, 32), "mxfp4": (2, 32), "int8": (1, None)}[fmt]

    def weights(rows, K):
        n = rows * (1 if per[1] is None else K // per[1] if per[1] else 0)
        w = torch.zeros(rows * (K // per[0]), dtype=codes)
        return w, scales(n) if callable(scales) else torch.zeros(n, dtype=scales)

    w_gu, gs = weights(E * 2 * I, H)
    w_d, ds = weights(E * H, I)
    hidden, logits, out = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, E), torch.zeros(T, H, dtype=torch.bfloat16)
    sh = moe.Shape.of(*LAYER, fmt)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    if which == "forward":
        return moe.forward(hidden, logits, w_gu.view(E, 2 * I, -1), w_d.view(E, H, -1), k, gs.view(E, 2 * I, -1),
                           ds.view(E, H, -1), out=out, ws=ws, stream=0)
    f = moe.moe_forward if which == "moe_forward" else moe.moe_forward_host
    return f(hidden, logits, w_gu, gs, w_d, ds, sh, out, ws, stream=0)


@pytest.fixture
def library_not_reached(monkeypatch):
    class Stub:
        def __getattr__(self, name):
            if name == "moe_workspace_size":
                return lambda *a: 1 << 20
            raise AssertionError(f"{name} was called")
    monkeypatch.setattr(moe, "lib", lambda: Stub())


@pytest.mark.parametrize("which", ["moe_forward", "moe_forward_host"])
@pytest.mark.parametrize("fmt,codes,scales", [
    ("int4_g128", torch.int8, torch.float32), ("int4_g128", torch.uint8, torch.float32),
    ("int4_g128", torch.int8, torch.bfloat16), ("mxfp8", torch.int8, torch.uint8), ("mxfp4", torch.uint8, torch.float32),
    ("bf16", torch.int8, torch.bfloat16), ("int8", torch.int8, torch.bfloat16), ("int8", torch.uint8, torch.float32),
    ("int8", torch.bfloat16, torch.float32), ("int8", torch.int8, torch.uint8)])
def test_layer_refuses_another_formats_weights(library_not_reached, which, fmt, codes, scales):
    with pytest.raises(TypeError):
        layer_call(which, fmt, codes, scales)


@pytest.mark.parametrize("which", ["moe_forward", "moe_forward_host", "forward"])
def test_int8_layer_refuses_short_scales_and_bf16_scales(library_not_reached, which):
    # the kernels read one fp32 scale per weight row: fewer, or 16-bit ones, would be read past their end
    with pytest.raises(TypeError):
        layer_call(which, "int8", torch.int8, torch.bfloat16)
    if which != "forward":
        with pytest.raises(ValueError, match="at least"):
            layer_call(which, "int8", torch.int8, lambda n: torch.zeros(4))
    with pytest.raises(ValueError, match="current CUDA device"):
        layer_call(which, "int8", torch.int8, torch.float32)


def test_int8_layer_refuses_short_activations(library_not_reached):
    T, H, I, E, k = LAYER
    w_gu, w_d = torch.zeros(E, 2 * I, H, dtype=torch.int8), torch.zeros(E, H, I, dtype=torch.int8)
    gs, ds = torch.zeros(E, 2 * I), torch.zeros(E, H)
    x, l, ws = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, E), torch.zeros(64, dtype=torch.uint8)
    sh = moe.Shape.of(*LAYER, "int8")
    for hidden, logits, out in ((x[1:], l, x), (x, l[1:], x), (x, l, x[1:])):
        with pytest.raises(ValueError, match="at least"):
            moe.moe_forward(hidden, logits, w_gu, gs, w_d, ds, sh, out, ws, stream=0)


@pytest.mark.parametrize("ws", [torch.zeros(1 << 18), torch.zeros(1 << 17, 2, dtype=torch.int64), torch.tensor(1.0)],
                         ids=["fp32", "int64", "0-d"])
def test_forward_scored_takes_a_workspace_of_any_type(library_not_reached, ws):
    # as moe_forward does: what is refused here is the host memory
    with pytest.raises(ValueError, match="current CUDA device"):
        moe.moe_forward_scored(A, A, None, router(), A, None, A, None, moe.Shape.of(*LAYER), A, ws, stream=0)
    strided = torch.zeros(4, 8)[:, ::2]
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_forward_scored(A, A, None, router(), A, None, A, None, moe.Shape.of(*LAYER), A, strided, stream=0)


def test_router_struct_has_the_c_layout():
    assert [f[0] for f in moe.Router._fields_] == ["logits", "score", "n_group", "topk_group", "group_top",
                                                   "renormalize", "scale"]
    assert ctypes.sizeof(moe.Router) == 28


def test_marshal_module_belongs_to_one_torch_and_python(monkeypatch):
    # it reads at::Tensor's internals: with another torch, the file of this one is not up to date
    moe_build.build_marshal()
    assert moe_build.marshal_up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert not moe_build.marshal_up_to_date()


def test_two_processes_may_build_the_marshal_module_at_once(monkeypatch, tmp_path):
    # each compiles to a file of its own and puts the whole of it in place: the second
    # process here builds while the compiler of the first is running
    target = str(tmp_path / "module.so")
    monkeypatch.setattr(moe_build, "marshal_file", lambda: target)
    written = []

    def compiler(cmd, check):
        assert check
        out = cmd[cmd.index("-o") + 1]
        assert os.path.dirname(out) == str(tmp_path) and not os.path.exists(out)
        with open(out, "w") as f:
            f.write("first half, ")
            f.flush()
            written.append(out)
            if len(written) == 1:
                moe_build.build_marshal(force=True)
                assert open(target).read() == "first half, second half"
            f.write("second half")

    monkeypatch.setattr(moe_build.subprocess, "run", compiler)
    assert moe_build.build_marshal(force=True) == target
    assert open(target).read() == "first half, second half" and len(written) == 2
    assert os.listdir(tmp_path) == ["module.so"]


def test_a_failed_build_of_the_marshal_module_leaves_nothing(monkeypatch, tmp_path):
    monkeypatch.setattr(moe_build, "marshal_file", lambda: str(tmp_path / "module.so"))

    def compiler(cmd, check):
        open(cmd[cmd.index("-o") + 1], "w").close()
        raise RuntimeError("no compiler")

    monkeypatch.setattr(moe_build.subprocess, "run", compiler)
    with pytest.raises(RuntimeError):
        moe_build.build_marshal(force=True)
    assert os.listdir(tmp_path) == []


# ---- the plain forms themselves ---------------------------------------------

def test_plain_router_by_hand():
    l = torch.tensor([[0.0, 1.0, 2.0, 3.0]])
    ids, w = _plain.route_scored(l, None, 2)
    assert ids.tolist() == [[3, 2]] and np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]])
    # the bias picks, the weight ignores it
    ids, w = _plain.route_scored(l, torch.tensor([5.0, 0, 0, 0]), 1, score="sigmoid", renormalize=False, scale=2.0)
    assert ids.tolist() == [[0]] and np.allclose(w, [[1.0]])
    # groups {0,1}, {2,3}: the best pair wins with two summed, the best single with one
    l = torch.tensor([[2.0, 2.0, 3.0, -9.0]])
    assert _plain.route_scored(l, None, 1, "sigmoid", 2, 1, 2)[0].tolist() == [[0]]
    assert _plain.route_scored(l, None, 1, "sigmoid", 2, 1, 1)[0].tolist() == [[2]]


def test_plain_int8_rows_by_hand():
    x = torch.tensor([[127.0, 0.5, -0.5, 1.5], [2.0, 1.0, -1.0, 0.0], [0.0, 0.0, 0.0, 0.0],
                      [1.0, float("inf"), 0.0, 0.0]]).to(torch.bfloat16)
    q, s = _plain.int8_rows(x)
    assert q.tolist() == [[127, 0, 0, 2], [127, 64, -64, 0], [0, 0, 0, 0], [0, 0, 0, 0]]   # ties to even
    assert s[0] == 1.0 and s[2] == 0.0 and bool(torch.isnan(s[3]))
