"""Cases of the operators around the routed experts of one MoE block.

Four operators, in the order in which a block runs them:

* ``norm``   residual addition + root-mean-square norm, the normed rows in
             bf16 / fp32 and, for the FP8 experts, as MXFP8 codes with scales;
* ``linear`` matrix product with bias, activation and residual (the router's
             projection, the shared expert's two products);
* ``route``  top-k routing on softmax or sigmoid scores, with a balance bias,
             expert groups, renormalised and scaled weights;
* ``gather`` the MXFP8 token rows copied to the permuted rows of their experts.

``run`` computes a case in elementary torch operations in 32 bits, or, where
``own`` is true, through the package's entry points.  Sizes are those of the
package's workloads (H 4096 / 7168, I 2048, 384 / 256 experts, top-8, 8 to
16384 tokens) and ragged ones of the same ranges.
"""
import math

import torch

own = False

_BF16, _F32 = torch.bfloat16, torch.float32
_EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 8 sequences: residual stream in fp32, bf16 rows for the router and the 2-bit experts
        dict(name="norm_decode", op="norm", T=8, H=4096, res="f32", pad=0, out="bf16", mx=False),
        # FP8 prefill, the last chunk a few tokens short: bf16 residual stream, bf16 rows for the router and MXFP8
        # rows for the experts
        dict(name="norm_prefill", op="norm", T=16373, H=7168, res="bf16", pad=0, out="bf16", mx=True),
        # router of one decode step (fp32 logits)
        dict(name="linear_router_decode", op="linear", T=8, N=384, K=4096, act="none", bias=False, res="none", out="f32"),
        # shared expert, first product of one decode step: gate and up with SwiGLU
        dict(name="linear_swiglu_decode", op="linear", T=8, N=2048, K=4096, act="swiglu", bias=False, res="none", out="bf16"),
        # a ragged chunk through a biased GELU projection onto an fp32 residual
        dict(name="linear_ragged", op="linear", T=777, N=1900, K=1464, act="gelu", bias=True, res="f32", out="f32"),
        # router of an FP8 prefill
        dict(name="linear_router_prefill", op="linear", T=16384, N=256, K=7168, act="none", bias=True, res="none", out="f32"),
        # shared expert of a prefill: first product, and the second onto the routed experts' output
        dict(name="linear_swiglu_prefill", op="linear", T=8192, N=2048, K=4096, act="swiglu", bias=False, res="none", out="bf16"),
        dict(name="linear_down_prefill", op="linear", T=16384, N=7168, K=2048, act="none", bias=False, res="bf16", out="bf16"),
        # one decode step: sigmoid scores, balance bias, 4 of 8 groups by their two best experts
        dict(name="route_decode", op="route", T=8, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, best=2, renorm=True, scale=2.5),
        # a prefill over 384 experts: softmax scores with a balance bias, no groups
        dict(name="route_prefill", op="route", T=8192, E=384, k=8, score="softmax", bias=True, groups=1, keep=1, best=1, renorm=True, scale=1.0),
        # the MXFP8 rows of one mixed decode step
        dict(name="gather_decode", op="gather", T=64, H=4096, k=8),
        # FP8 prefill: the MXFP8 rows of 16384 tokens to 131072 permuted rows
        dict(name="gather_prefill", op="gather", T=16384, H=7168, k=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    most = [max(work(c)[key] for c in listed()) for key in ("bytes", "flops")]
    while any(work(case)[key] > m for key, m in zip(("bytes", "flops"), most)):
        case["T"] = case["T"] * 3 // 4
    return case


def _draw(rng):
    op = rng.choice(["norm", "linear", "linear", "route", "gather"])
    T = _log_int(rng, 1, 16384)
    if op == "norm":
        mx = rng.random() < 0.5
        H = 32 * _log_int(rng, 4, 224) if mx else _log_int(rng, 65, 7168)
        return dict(op=op, T=T, H=H, res=rng.choice(["none", "bf16", "f32"]), pad=rng.choice([0, 0, 8, 96, 5]),
                    out=rng.choice(["bf16", "f32"]), mx=mx)
    if op == "linear":
        K = 8 * _log_int(rng, 8, 896)
        act = rng.choice(["none", "silu", "gelu", "swiglu"])
        N = 16 * _log_int(rng, 2, 256) if act == "swiglu" else _log_int(rng, 17, 7168)
        return dict(op=op, T=T, N=N, K=K, act=act, bias=rng.random() < 0.5, res=rng.choice(["none", "bf16", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "route":
        groups = rng.choice([1, 1, 4, 8, 16])
        per = _log_int(rng, 4, 1024 // groups if groups > 1 else 512)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * per))
        return dict(op=op, T=T, E=groups * per, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    groups=groups, keep=keep, best=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]))
    return dict(op=op, T=T, H=32 * _log_int(rng, 4, 224), k=rng.randint(1, 8))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=_F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=_F32) * scale).to(dtype)


def _dtype(name):
    return {"bf16": _BF16, "f32": _F32, "none": None}[name]


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _selection64(case, logits, bias):
    """Selection scores, in 64 bits."""
    l = logits.double()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, -1)
    return s if bias is None else s + bias.double()


def _undecided(case, logits, bias):
    """Rows whose choice of groups or experts hangs on the last bits of a
    score: their ids would be a matter of rounding.  Equal scores are decided
    (lowest index first)."""
    c = _selection64(case, logits, bias)
    T, E = c.shape
    G = case["groups"]
    least = 2e-6 * c.abs().amax(-1, keepdim=True)
    bad = torch.zeros(T, dtype=torch.bool, device=c.device)

    def near(v):
        gap = v[:, :-1] - v[:, 1:]
        return ((gap > 0) & (gap < least)).any(-1)

    if G > 1:
        best = c.view(T, G, E // G).topk(case["best"], -1)[0].sum(-1)
        ranked = best.sort(dim=-1, descending=True, stable=True)
        if case["keep"] < G:
            bad |= near(ranked[0][:, case["keep"] - 1:case["keep"] + 1])
        kept = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, ranked[1][:, :case["keep"]], True)
        c = c.masked_fill(~kept.repeat_interleave(E // G, 1), -1e30)
    return bad | near(c.topk(min(E, case["k"] + 1), -1)[0])


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    s = dict(case=case)
    if op == "norm":
        H, pad = case["H"], case["pad"]
        s["x"] = _randn(g, T, H + pad, dtype=_BF16)[:, :H]
        s["gain"] = 1.0 + _randn(g, H, scale=0.1)
        rt = _dtype(case["res"])
        s["res"] = None if rt is None else _randn(g, T, H + pad, dtype=rt, scale=4.0)[:, :H]
        s["sum"] = None if rt is None else _empty(T, H, dtype=rt)
        s["out"] = _empty(T, H, dtype=_dtype(case["out"]))
        s["q"] = _empty(T, H, dtype=torch.uint8) if case["mx"] else None
        s["q_scale"] = _empty(T, H // 32, dtype=torch.uint8) if case["mx"] else None
    elif op == "linear":
        N, K = case["N"], case["K"]
        rows = 2 * N if case["act"] == "swiglu" else N
        s["x"] = _randn(g, T, K, dtype=_BF16)
        s["w"] = _randn(g, rows, K, dtype=_BF16, scale=K ** -0.5)
        s["bias"] = _randn(g, rows, scale=0.5) if case["bias"] else None
        rt = _dtype(case["res"])
        s["res"] = None if rt is None else _randn(g, T, N, dtype=rt)
        s["out"] = _empty(T, N, dtype=_dtype(case["out"]))
        s["dev_err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    elif op == "route":
        E = case["E"]
        s["bias"] = None
        if case["bias"]:
            s["bias"] = _randn(g, E, scale=0.02 if case["score"] == "sigmoid" else 0.2 / E)
        # without a bias the logits are those of a bf16 product, with equal ones among them
        def make():
            l = _randn(g, T, E)
            return l if case["bias"] else l.to(_BF16).float()
        s["logits"] = make()
        for _ in range(12):
            bad = _undecided(case, s["logits"], s["bias"])
            if not bool(bad.any()):
                break
            s["logits"] = torch.where(bad[:, None], make(), s["logits"])
        s["ids"] = _empty(T, case["k"], dtype=torch.int32)
        s["w"] = _empty(T, case["k"], dtype=_F32)
        s["dev_err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        H, k = case["H"], case["k"]
        # E4M3 codes of every finite value, E8M0 scales around 1
        code = torch.randint(0, 254, (T, H), generator=g, device="cuda", dtype=torch.int32)
        s["xq"] = torch.where(code >= 127, code + 1, code).to(torch.uint8)
        s["xs"] = torch.randint(115, 124, (T, H // 32), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
        s["inv"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
        s["out"] = _empty(T * k, H, dtype=torch.uint8)
        s["out_scale"] = _empty(T * k, H // 32, dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ the package's calls
def _run_own(s):
    from bit_moe_expert_top_gb300 import _lib as L

    case = s["case"]
    op = case["op"]
    if op == "norm":
        L.moe_add_rmsnorm(s["x"], s["gain"], _EPS, res=s["res"], sum_out=s["sum"], out=s["out"], q=s["q"],
                          q_scale=s["q_scale"])
        return _norm_outputs(s["sum"], s["out"], s["q"], s["q_scale"])
    if op == "linear":
        act = {"none": L.ACT_NONE, "silu": L.ACT_SILU, "gelu": L.ACT_GELU, "swiglu": L.ACT_SWIGLU}[case["act"]]
        L.moe_linear(s["x"], s["w"], s["out"], bias=s["bias"], act=act, res=s["res"], dev_err=s["dev_err"])
        return {"out": s["out"]}
    if op == "route":
        L.moe_route_scored(s["logits"], case["k"], s["ids"], s["w"], bias=s["bias"],
                           score=L.SCORE_SIGMOID if case["score"] == "sigmoid" else L.SCORE_SOFTMAX,
                           n_group=case["groups"], topk_group=case["keep"], group_top=case["best"],
                           renorm=case["renorm"], scale=case["scale"], dev_err=s["dev_err"])
        return {"ids": s["ids"], "w": s["w"]}
    L.moe_gather_mxfp8(s["xq"], s["xs"], s["inv"], case["k"], s["out"], s["out_scale"])
    return {"q": s["out"].view(torch.float8_e4m3fn), "q_scale": s["out_scale"].view(torch.float8_e8m0fnu)}


def _norm_outputs(total, out, q, q_scale):
    r = {"out": out}
    if total is not None:
        r["sum"] = total
    if q is not None:
        r["q"], r["q_scale"] = q.view(torch.float8_e4m3fn), q_scale.view(torch.float8_e8m0fnu)
    return r


# ------------------------------------------------------------------ the plain forms
def _norm(s):
    case = s["case"]
    y = s["x"].float()
    total = None
    if s["res"] is not None:
        y = y + s["res"].float()
        total = y.to(s["res"].dtype)
    n = y / torch.sqrt((y * y).mean(-1, keepdim=True) + _EPS) * s["gain"]
    q = q_scale = None
    if case["mx"]:  # MXFP8 of the bf16 rows: per 32 elements 2^(floor(log2 amax) - 8), E4M3 codes
        b = n.to(_BF16).float().view(case["T"], -1, 32)
        amax = b.abs().amax(-1, keepdim=True)
        X = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), -127)
        power = ((127 - X).clamp(max=254) << 23).to(torch.int32).view(_F32)
        q = (b * power).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(case["T"], -1)
        q_scale = (X + 127).to(torch.uint8).squeeze(-1)
    return _norm_outputs(total, n.to(s["out"].dtype), q, q_scale)


def _linear(s):
    case = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif case["act"] == "swiglu":
        gate, up = y[:, :case["N"]], y[:, case["N"]:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"out": y.to(s["out"].dtype)}


def _route(s):
    case = s["case"]
    l, T, E, G = s["logits"], case["T"], case["E"], case["groups"]
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        z = torch.exp(l - l.amax(-1, keepdim=True))
        score = z / z.sum(-1, keepdim=True)
    c = score if s["bias"] is None else score + s["bias"]
    if G > 1:
        best = c.view(T, G, E // G).sort(-1, descending=True)[0][:, :, :case["best"]].sum(-1)
        order = best.sort(dim=-1, descending=True, stable=True)[1][:, :case["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        kept[torch.arange(T, device=c.device)[:, None], order] = True
        c = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), c, -math.inf)
    ids = c.sort(dim=-1, descending=True, stable=True)[1][:, :case["k"]]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": w * case["scale"]}


def _gather(s):
    row = torch.empty_like(s["inv"])  # the token of each permuted row
    row[s["inv"].long()] = torch.arange(s["inv"].numel(), device="cuda", dtype=torch.int32) // s["case"]["k"]
    q, q_scale = s["xq"][row.long()], s["xs"][row.long()]
    return {"q": q.view(torch.float8_e4m3fn), "q_scale": q_scale.view(torch.float8_e8m0fnu)}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "linear": _linear, "route": _route, "gather": _gather}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work, and the values in 64 bits
def _size(name):
    return {"bf16": 2, "f32": 4, "none": 0}[name]


def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        per = 2 + 2 * _size(case["res"]) + _size(case["out"]) + (33 / 32 if case["mx"] else 0)
        return {"bytes": T * H * per + 4 * H, "flops": 5 * T * H}
    if op == "linear":
        N, K = case["N"], case["K"]
        rows = 2 * N if case["act"] == "swiglu" else N
        return {"bytes": 2 * T * K + 2 * rows * K + (4 * rows if case["bias"] else 0)
                + T * N * (_size(case["res"]) + _size(case["out"])), "flops": 2 * T * rows * K}
    if op == "route":
        return {"bytes": 4 * T * case["E"] + 8 * T * case["k"] + (4 * case["E"] if case["bias"] else 0),
                "flops": 6 * T * case["E"]}
    return {"bytes": (1 + case["k"]) * case["T"] * case["H"] * 33 / 32 + 4 * T * case["k"], "flops": 0}


def exact(case, seed):
    """From the definitions in 64 bits.  What is rounded to 8 or 16 bits is
    given before its rounding (the codes of a block as multiples of its scale)."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].to(torch.float64)
        r = {}
        if s["res"] is not None:
            v += s["res"]
            r["sum"] = v
        rms = (torch.einsum("th,th->t", v, v) / v.shape[1] + _EPS) ** 0.5
        n = torch.einsum("th,h,t->th", v, s["gain"].to(torch.float64), 1 / rms)
        r["out"] = n
        if case["mx"]:
            blocks = n.unflatten(1, (-1, 32))
            top = blocks.to(_BF16).to(torch.float64).abs().max(-1).values
            scale = 2.0 ** (torch.floor(torch.log2(top)) - 8)
            r["q"] = (blocks / scale[..., None]).clamp(-448, 448).flatten(1)
            r["q_scale"] = scale
        return r
    if op == "linear":
        out = torch.empty(case["T"], case["N"], dtype=torch.float64, device="cuda")
        wt = s["w"].to(torch.float64).T
        for a in range(0, case["T"], 1024):
            v = torch.matmul(s["x"][a:a + 1024].to(torch.float64), wt)
            if s["bias"] is not None:
                v += s["bias"]
            if case["act"] == "silu":
                v = torch.nn.functional.silu(v)
            elif case["act"] == "gelu":
                v = torch.nn.functional.gelu(v)
            elif case["act"] == "swiglu":
                v = torch.nn.functional.silu(v[:, :case["N"]]) * v[:, case["N"]:]
            if s["res"] is not None:
                v = v + s["res"][a:a + 1024]
            out[a:a + 1024] = v
        return {"out": out}
    if op == "route":
        c = _selection64(case, s["logits"], s["bias"])
        score = c if s["bias"] is None else c - s["bias"].double()
        T, E, G = case["T"], case["E"], case["groups"]
        if G > 1:
            best = c.view(T, G, E // G).topk(case["best"], -1)[0].sum(-1)
            rank = (best[:, :, None] < best[:, None, :]).sum(-1)  # groups that are better
            first = (best[:, :, None] == best[:, None, :]).tril(-1).sum(-1)  # equal ones of a lower index
            kept = (rank + first < case["keep"]).repeat_interleave(E // G, 1)
            c = c.masked_fill(~kept, -1e30)
        ids = c.sort(dim=-1, descending=True, stable=True)[1][:, :case["k"]]
        w = score.gather(1, ids)
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        return {"ids": ids.to(torch.int32), "w": w * case["scale"]}
    return None
