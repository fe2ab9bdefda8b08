"""Performance cases of the layer's scored router, RMS norm and 8-bit integer products.

Each case is one call of one operator. `run` computes it in its plain form
(elementary torch operations) or, with `own`, through the library's entry
points; `exact` computes it in 64 bits.

  route     moe_route_scored: scores, selection bias, groups, top-k, weights
  norm      moe_rmsnorm: residual addition, RMS norm, bf16 and 8-bit outputs
  quantize  moe_i8_quantize: one int8 row and one scale per token
  gate_up   moe_grouped_gemm_swiglu_i8: int8 gate/up products with SwiGLU
  down      moe_grouped_gemm_down_i8: int8 down products
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one token of a single decoding stream: softmax scores, renormalised
        dict(name="route one token", op="route", T=1, E=128, k=8, S=0, score="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, renorm=True, scale=1.0, logits="fp32"),
        # a mid-size batch whose router ran in bf16: an expert count that is no multiple of the warp, shared experts,
        # weights left as probabilities
        dict(name="route bf16 odd", op="route", T=777, E=60, k=6, S=2, score="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, renorm=False, scale=16.0, logits="bf16"),
        # prefill with the balance bias on sigmoid scores, 4 of 8 groups kept by their two best experts
        dict(name="route groups prefill", op="route", T=16384, E=256, k=8, S=0, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, renorm=True, scale=2.5, logits="fp32"),
        # before the layer of one decoded token: the int8 row goes to the experts
        dict(name="norm one token int8", op="norm", T=1, H=2048, fmt="int8", y=False, residual=True),
        # a decode batch at a wide hidden size: bf16 rows for the router, MXFP8 rows for the experts
        dict(name="norm decode mxfp8", op="norm", T=256, H=7168, fmt="mxfp8", y=True, residual=True),
        # prefill: bf16 rows for the router, int8 rows for the experts
        dict(name="norm prefill int8", op="norm", T=8192, H=2048, fmt="int8", y=True, residual=True),
        # act between the two products of a decode batch of 64 tokens with 8 experts each
        dict(name="quantize decode", op="quantize", rows=512, K=768),
        # the same at prefill: 8192 tokens with 8 experts each
        dict(name="quantize prefill", op="quantize", rows=65536, K=768),
        # gate/up of the decode layer: four rows per expert on average, read through perm
        dict(name="gate_up decode", op="gate_up", T=64, H=2048, I=768, E=128, k=8, skew=0.0, perm=True),
        # gate/up of the prefill layer: uneven loads, rows already gathered
        dict(name="gate_up prefill", op="gate_up", T=8192, H=2048, I=768, E=128, k=8, skew=0.5, perm=False),
        # down of a single token: eight experts with one row each
        dict(name="down one token", op="down", T=1, H=2048, I=768, E=128, k=8, skew=0.0),
        # down with skewed loads: some experts see nearly every token, others a few rows or none
        dict(name="down skewed", op="down", T=4096, H=4096, I=1408, E=64, k=6, skew=3.0),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "norm", "quantize", "gate_up", "gate_up", "down", "down"])
    if op == "route":
        T = _spread(rng, 1, 16384)
        n_group = rng.choice([1, 1, 2, 4, 8])
        size = _spread(rng, 4, 256 // n_group)
        topk_group = rng.randint(1, n_group)
        return dict(op=op, T=T, E=n_group * size, k=rng.randint(1, min(8, topk_group * size)), S=rng.choice([0, 0, 1, 2]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, n_group=n_group,
                    topk_group=topk_group, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), logits=rng.choice(["fp32", "bf16"]))
    if op == "norm":
        H = 32 * _spread(rng, 4, 256)
        return dict(op=op, T=_spread(rng, 1, max(1, 8192 * 2048 // H)), H=H, fmt=rng.choice(["bf16", "mxfp8", "int8"]),
                    y=True, residual=rng.random() < 0.7)
    if op == "quantize":
        K = 16 * _spread(rng, 8, 512)
        return dict(op=op, rows=_spread(rng, 1, max(1, 65536 * 768 // K)), K=K)
    H = 16 * _spread(rng, 16, 256)
    I = 16 * _spread(rng, 8, 88)
    E = _spread(rng, 2, max(2, min(128, 200_000_000 // (H * I))))      # weights of at most 400 MB
    k = rng.randint(1, min(8, E))
    T = _spread(rng, 1, max(1, min(8192, 400_000_000_000 // (4 * H * I * k))))
    c = dict(op=op, T=T, H=H, I=I, E=E, k=k, skew=rng.choice([0.0, 0.5, 3.0]))
    if op == "gate_up":
        # few rows per expert: read through perm by the product; many: gathered before it
        c["perm"] = T * k <= 32 * E
    return c


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _router_logits(g, T, E, skew):
    """Router logits: N(0,1), plus a per-expert offset for uneven loads
    (skew < 1: N(0,skew); above: skew times the log of a Zipf popularity)."""
    logits = _randn(g, T, E)
    if skew >= 1.0:
        p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32).pow(-1.2)
        logits += skew * torch.log(p / p.sum())
    elif skew > 0.0:
        logits += skew * _randn(g, E)
    return logits


def _int8(g, *shape):
    """Codes of rows quantised by their largest value: N(0, 36), clipped."""
    return _randn(g, *shape).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if own:
        import mixture_experts_expert_top_b200 as moe
        s["moe"] = moe
    if op == "route":
        T, E, K = case["T"], case["E"], case["k"] + case["S"]
        s["logits"] = _randn(g, T, E).mul_(1.5).to(torch.float32 if case["logits"] == "fp32" else torch.bfloat16)
        s["bias"] = _randn(g, E).mul_(0.1) if case["bias"] else None
        s["ids"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, K, device="cuda")
        if own:
            s["shape"] = moe.Shape.of(T, 128, 128, E, case["k"], n_shared=case["S"])
            s["router"] = moe.Router.of(case["score"], case["n_group"], case["topk_group"], case["group_top"],
                                        case["renorm"], case["scale"], case["logits"])
        return s
    if op in ("norm", "quantize"):
        rows, H = (case["T"], case["H"]) if op == "norm" else (case["rows"], case["K"])
        # rows of different sizes, and channels that stand out
        x = _randn(g, rows, H) * torch.exp(0.7 * _randn(g, rows, 1)) * torch.exp(0.5 * _randn(g, 1, H))
        s["x"] = x.to(torch.bfloat16)
        if op == "norm":
            s["residual"] = _randn(g, rows, H).mul_(2.0).to(torch.bfloat16) if case["residual"] else None
            s["weight"] = (1.0 + 0.2 * _randn(g, H)).to(torch.bfloat16)
            s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["y"] = torch.empty_like(s["x"]) if case["y"] else None
        fmt = case.get("fmt", "int8")
        s["q"] = s["scales"] = None
        if fmt == "int8":
            s["q"] = torch.empty(rows, H, dtype=torch.int8, device="cuda")
            s["scales"] = torch.empty(rows, dtype=torch.float32, device="cuda")
            s["values"] = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
        elif fmt == "mxfp8":
            s["q"] = torch.empty(rows, H, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(rows, H // 32, dtype=torch.uint8, device="cuda")
        if own:
            s["fmt"] = {"bf16": moe.FMT_BF16, "mxfp8": moe.FMT_MXFP8, "int8": moe.FMT_INT8}[fmt]
        return s
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    P = T * k
    ids = torch.topk(_router_logits(g, T, E, case["skew"]), k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())
    rows, K, N = (H, H, 2 * I) if op == "gate_up" else (I, I, H)
    through = op == "gate_up" and case["perm"]
    s["perm"] = order.to(torch.int32) if through else None
    n_rows = T if through else P
    s["a"] = _int8(g, n_rows, K)
    # rows of N(0,1) hidden states (gate/up) or of act (down); weights N(0, 0.02): the largest value is about 3.5 sigma
    s["a_scales"] = (3.5 / 127.0) * torch.exp(0.3 * _randn(g, n_rows))
    s["w"] = _int8(g, E, N, K)
    s["w_scales"] = (3.5 * 0.02 / 127.0) * torch.exp(0.1 * _randn(g, E, N))
    s["out"] = torch.empty(P, I if op == "gate_up" else H, dtype=torch.bfloat16, device="cuda")
    if own:
        s["shape"] = moe.Shape.of(T, H, I, E, k, moe.FMT_INT8)
    return s


# ---- one pass ---------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    moe, c = s["moe"], s["case"]
    op = c["op"]
    if op == "route":
        moe.moe_route_scored(s["logits"], s["bias"], s["router"], s["shape"], s["ids"], s["w"])
        return {"ids": s["ids"], "w": s["w"]}
    if op == "norm":
        moe.moe_rmsnorm(s["x"], s["residual"], s["weight"], EPS, c["T"], c["H"], s["fmt"], s["residual_out"], s["y"],
                        s["q"], s["scales"])
        out = {}
        if c["residual"]:
            out["residual_out"] = s["residual_out"]
        if c["y"]:
            out["y"] = s["y"]
        if c["fmt"] == "int8":
            out["values"] = torch.mul(s["q"], s["scales"][:, None], out=s["values"])
            out["scales"] = s["scales"]
        elif c["fmt"] == "mxfp8":
            out["values"] = s["q"].view(torch.float8_e4m3fn)
            out["scales"] = s["scales"].view(torch.float8_e8m0fnu)
        return out
    if op == "quantize":
        moe.moe_i8_quantize(s["x"], c["rows"], c["K"], s["q"], s["scales"])
        return {"values": torch.mul(s["q"], s["scales"][:, None], out=s["values"]), "scales": s["scales"]}
    if op == "gate_up":
        moe.moe_grouped_gemm_swiglu_i8(s["a"], s["a_scales"], s["perm"], s["offsets"], s["w"], s["w_scales"], s["shape"],
                                       s["out"])
    else:
        moe.moe_grouped_gemm_down_i8(s["a"], s["a_scales"], s["offsets"], s["w"], s["w_scales"], s["shape"], s["out"])
    return {"out": s["out"]}


def _run_plain(s):
    return {"route": _plain_route, "norm": _plain_norm, "quantize": _plain_quantize, "gate_up": _plain_product,
            "down": _plain_product}[s["case"]["op"]](s)


def _plain_route(s):
    # scores in 64 bits: the order of two experts may hang on their last bits
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    lg = s["logits"].double()
    lg = torch.where(torch.isnan(lg), torch.full_like(lg, -math.inf), lg)
    if c["score"] == "softmax":
        e = torch.exp(lg - lg.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-lg))
    choice = lg if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        groups = (score if s["bias"] is None and c["group_top"] > 1 else choice).view(T, G, E // G)
        best = torch.sort(groups, dim=2, descending=True, stable=True).values[:, :, :c["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=lg.device).scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, torch.full_like(choice, -math.inf))
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    shared = torch.arange(E, E + c["S"], device=ids.device).expand(T, c["S"])
    return {"ids": torch.cat([ids, shared], 1).to(torch.int32),
            "w": torch.cat([w, torch.ones_like(shared, dtype=w.dtype)], 1).float()}


def _int8_rows(y):
    amax = y.abs().amax(1, keepdim=True)
    q = torch.round(y * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)))
    return q, amax / 127.0


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    out = {}
    if c["residual"]:
        h = h + s["residual"].float()
        out["residual_out"] = h.to(torch.bfloat16)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if c["y"]:
        out["y"] = y.to(torch.bfloat16)
    if c["fmt"] == "int8":
        q, scale = _int8_rows(y)
        out["values"] = (q * scale).to(torch.bfloat16)
        out["scales"] = scale[:, 0]
    elif c["fmt"] == "mxfp8":
        b = y.view(c["T"], c["H"] // 32, 32)
        # floor(log2 max|y|) - 8: frexp's exponent is one more than the floor of the logarithm
        e = torch.frexp(b.abs().amax(2, keepdim=True)).exponent - 9
        v = torch.ldexp(b, -e).clamp(-448.0, 448.0)
        out["values"] = v.view(c["T"], c["H"]).to(torch.float8_e4m3fn)
        out["scales"] = (e[:, :, 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_quantize(s):
    # 64 bits decide the rounding: many quotients of bf16 values lie on a border
    q, _ = _int8_rows(s["x"].double())
    scale = s["x"].float().abs().amax(1, keepdim=True) / 127.0
    return {"values": (q.float() * scale).to(torch.bfloat16), "scales": scale[:, 0]}


def _plain_product(s):
    # every expert's rows padded to the longest, one batched product, rows taken back in order
    c = s["case"]
    off = s["offsets"].long()
    P = c["T"] * c["k"]
    if s["perm"] is not None:
        src = s["perm"].long() // c["k"]
        a, a_scales = s["a"][src], s["a_scales"][src]
    else:
        a, a_scales = s["a"], s["a_scales"]
    r = torch.arange(P, device=a.device)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    at = r - off[e]
    rows = (off[:-1, None] + torch.arange(s["most"], device=a.device)).clamp_max(P - 1)
    acc = torch.bmm(a.float()[rows], s["w"].float().transpose(1, 2))
    v = acc[e, at] * s["w_scales"][e] * a_scales[:, None]
    if c["op"] == "gate_up":
        gate, up = v[:, :c["I"]], v[:, c["I"]:]
        v = gate / (1.0 + torch.exp(-gate)) * up
    return {"out": v.to(torch.bfloat16)}


# ---- from the definition, in 64 bits ----------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, s["logits"].double().cpu().numpy(),
                            None if s["bias"] is None else s["bias"].double().cpu().numpy())
    if op in ("norm", "quantize"):
        h = s["x"].double()
        out = {}
        if op == "norm":
            if case["residual"]:
                h = h + s["residual"].double()
                out["residual_out"] = h
            h = h * (h.square().sum(1) / case["H"] + EPS).rsqrt()[:, None] * s["weight"].double()
            if case["y"]:
                out["y"] = h
        if op == "quantize" or case["fmt"] == "int8":
            step = h.abs().max(1).values[:, None] / 127.0
            out["values"] = (h / step).round() * step if op == "norm" else (127.0 * h / h.abs().max(1).values[:, None]).round() * step
            out["scales"] = step[:, 0]
        elif case["fmt"] == "mxfp8":
            blocks = h.reshape(-1, 32)
            scale = torch.exp2(torch.floor(torch.log2(blocks.abs().max(1).values)) - 8.0)[:, None]
            v = blocks / scale
            # E4M3: 3 mantissa bits, the spacing of the smallest normal (2^-6) below it
            grid = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
            out["values"] = ((v / grid).round() * grid).clamp(-448.0, 448.0).reshape(h.shape)
            out["scales"] = scale.reshape(case["T"], -1)
        return out
    off = s["offsets"].tolist()
    pieces = []
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        rows = torch.arange(lo, hi, device="cuda") if s["perm"] is None else s["perm"][lo:hi].long() // case["k"]
        x = s["a"][rows].double() * s["a_scales"][rows].double()[:, None]
        v = x @ (s["w"][e].double() * s["w_scales"][e].double()[:, None]).T
        if op == "gate_up":
            gate, up = v.chunk(2, dim=1)
            v = gate * torch.sigmoid(gate) * up
        pieces.append(v)
    return {"out": torch.cat(pieces)}


def _exact_route(c, lg, bias):
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    if c["score"] == "softmax":
        p = np.exp(lg - lg.max(axis=1)[:, None])
        p /= p.sum(axis=1)[:, None]
    else:
        p = np.exp(-np.logaddexp(0.0, -lg))
    pick = lg if bias is None else p + bias
    if G > 1:
        by = p if bias is None and c["group_top"] == 2 else pick
        value = np.partition(by.reshape(T, G, -1), -c["group_top"], axis=2)[:, :, -c["group_top"]:].sum(axis=2)
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        pick = np.where(np.repeat(rank < c["topk_group"], E // G, axis=1), pick, -np.inf)
    ids = np.argsort(-pick, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, 1)
    w = w / w.sum(axis=1)[:, None] * c["scale"] if c["renorm"] else w * c["scale"]
    shared = np.broadcast_to(np.arange(E, E + c["S"]), (T, c["S"]))
    return {"ids": np.concatenate([ids, shared], 1).astype(np.int32), "w": np.concatenate([w, np.ones((T, c["S"]))], 1)}


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    op = case["op"]
    if op == "route":
        T, E, K = case["T"], case["E"], case["k"] + case["S"]
        return {"bytes": T * E * (4 if case["logits"] == "fp32" else 2) + 8 * T * K + (4 * E if case["bias"] else 0),
                "flops": 4 * T * E}
    if op == "norm":
        T, H = case["T"], case["H"]
        n = 2 + (4 if case["residual"] else 0) + (2 if case["y"] else 0)
        eight = {"bf16": 0, "int8": T * (H + 4), "mxfp8": T * (H + H // 32)}[case["fmt"]]
        return {"bytes": T * H * n + eight + 2 * H, "flops": 6 * T * H}
    if op == "quantize":
        return {"bytes": case["rows"] * (3 * case["K"] + 4), "flops": 3 * case["rows"] * case["K"]}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    P = T * k
    active = E * (1.0 - (1.0 - k / E) ** T)              # experts with a row, at even loads
    K, N, n_out = (H, 2 * I, I) if op == "gate_up" else (I, H, H)
    rows = T if op == "gate_up" and case["perm"] else P
    return {"bytes": int(active * N * (K + 4)) + rows * (K + 4) + 2 * P * n_out, "flops": 2 * P * K * N}
