"""GPU parity of the block operators against oracle/block.py (float64).

Tolerances, from the arithmetic:
A bf16 output has to lie between the roundings of the two ends of its fp32
interval.

  * norm: the fp32 sum of squares adds at most 64 terms in sequence and 10
    levels of a tree, 74 * 2^-24 relative, half of it after the root, and five
    more roundings: 3e-6 relative per element.
  * sum, q, scales, gathers: bit-exact (q against the quantisation of the bf16
    rows that the same arithmetic gives).
  * routing weights: e^x to 2 ulp of an argument rounded at |l| <= 16 (1e-6), a
    sum of at most 32 + 5 steps (2.2e-6), twice for the renormalisation: 1e-5
    relative.  ids equal (inputs whose order is decided by more than 1e-5).
  * linear: integer operands whose sums are exact in fp32: bit-exact without
    an activation, else 4e-6 relative to the largest intermediate (fp32
    exp / erf / divide, a few ulp).  Random operands, fp32
    output: a chunk of 512 is 32 truncated additions of at most 2^-23, mean
    half, of a partial sum that grows like a random walk: 32 * 2/3 * 2^-24 =
    1.3e-6 of the 2-norm, plus the rounded sums of the chunks: 2e-6.
"""
import numpy as np
import pytest
import torch

from bit_moe_expert_top_gb300 import _lib as L
from oracle import block as B

from tests._gpu import host

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return host(t.contiguous().view(torch.int16)).view(np.uint16)


def within(t, want, err) -> bool:
    """Every value of t is the rounding, to t's type, of a number in want +- err."""
    lo, hi = (torch.from_numpy(want + s * err).to(DEV).float().to(t.dtype).double() for s in (-1, 1))
    return bool(((t.double() >= lo) & (t.double() <= hi)).all())


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


# ------------------------------------------------------------------ norm
NORM = [  # T, H, x, res, out, mx, pad
    (1, 4096, "bf16", "f32", "bf16", False, 0),
    (8, 7168, "bf16", "bf16", "bf16", True, 0),
    (3, 1, "f32", None, "f32", False, 0),
    (5, 31, "bf16", "f32", "f32", False, 0),
    (7, 33, "bf16", "bf16", "bf16", False, 1),
    (4, 32, "bf16", None, "bf16", True, 0),
    (300, 2080, "bf16", "f32", "f32", True, 96),
    (9, 2080, "bf16", "bf16", "bf16", True, 5),
    (2, 16384, "f32", "bf16", "f32", True, 0),
    (2, 16383, "f32", "f32", "bf16", False, 0),
    (2, 8200, "bf16", "bf16", "bf16", False, 8),
    (1201, 1000, "bf16", "bf16", "bf16", False, 0),
    (2000, 160, "bf16", "bf16", "bf16", True, 0),
]


@pytest.mark.parametrize("T,H,xd,rd,od,mx,pad", NORM)
@pytest.mark.parametrize("gain", ["f32", "bf16", None])
def test_add_rmsnorm(T, H, xd, rd, od, mx, pad, gain):
    g = gen(T * 31 + H)
    x = randn(g, T, H + pad, dtype=DT[xd])[:, pad:]
    res = None if rd is None else randn(g, T, H + pad, dtype=DT[rd], scale=5.0)[:, :H]
    gn = None if gain is None else (1 + randn(g, H, scale=0.2)).to(DT[gain])
    s = None if res is None else torch.full((T, H + 3), 7.0, device=DEV, dtype=DT[rd])
    out = torch.empty(T, H, device=DEV, dtype=DT[od])
    q = torch.empty(T, H, device=DEV, dtype=torch.uint8) if mx else None
    qs = torch.empty(T, H // 32, device=DEV, dtype=torch.uint8) if mx else None
    L.moe_add_rmsnorm(x, gn, 1e-5, res=res, sum_out=None if s is None else s[:, :H], out=out, q=q, q_scale=qs)
    y, n = B.add_rmsnorm(f64(x), None if gn is None else f64(gn), 1e-5, None if res is None else f64(res))
    assert within(out, n, 3e-6 * np.abs(n) + 1e-30)
    if s is not None:
        want = (x.float() + res.float()).to(DT[rd])
        assert torch.equal(s[:, :H], want)
        assert bool((s[:, H:] == 7.0).all())  # nothing beyond the row
    if mx:  # the codes of the bf16 rows the same call writes
        ob = torch.empty(T, H, device=DEV, dtype=torch.bfloat16)
        L.moe_add_rmsnorm(x, gn, 1e-5, res=res, out=ob)
        wq, ws = B.mxfp8_rows(bits(ob))
        assert np.array_equal(host(qs), ws) and np.array_equal(host(q), wq)


def test_add_rmsnorm_in_place_and_streams():
    g = gen(3)
    x, res = randn(g, 50, 512, dtype=torch.bfloat16), randn(g, 50, 512)
    want = x.float() + res
    out = torch.empty_like(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    L.moe_add_rmsnorm(x, None, 1e-6, res=res, sum_out=res, out=out, stream=st)
    st.synchronize()
    assert torch.equal(res, want)


def test_add_rmsnorm_special_rows():
    """A row of zeros gives zeros (eps), NaN stays in its row, an infinite element zeroes the
    finite ones of its row; the neighbours are untouched."""
    x = torch.ones(4, 64, device=DEV, dtype=torch.bfloat16)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 6] = float("inf")
    out = torch.empty(4, 64, device=DEV)
    q = torch.empty(4, 64, device=DEV, dtype=torch.uint8)
    qs = torch.empty(4, 2, device=DEV, dtype=torch.uint8)
    L.moe_add_rmsnorm(x, None, 1e-6, out=out, q=q, q_scale=qs)
    o = host(out)
    assert not o[0].any() and not host(q)[0].any() and host(qs)[0].tolist() == [0, 0]
    assert np.isnan(o[1]).all()
    assert np.isnan(o[2, 6]) and not np.delete(o[2], 6).any()
    assert np.allclose(o[3], 1.0, atol=1e-6)


def test_add_rmsnorm_long_rows_apart():
    """Row offsets past 32 bits."""
    ld = (1 << 31) + 64
    base = torch.zeros(ld + 64, device=DEV, dtype=torch.bfloat16)
    x = torch.as_strided(base, (2, 64), (ld, 1))
    x[1] = 2.0
    out = torch.empty(2, 64, device=DEV)
    L.moe_add_rmsnorm(x, None, 0.0 + 1e-6, out=out)
    assert not host(out)[0].any() and np.allclose(host(out)[1], 1.0, atol=1e-6)


def placed(t, off):
    """A copy of t [T, H] `off` elements behind a 16-byte boundary, rows one element further apart
    than they are long, in a buffer of sevens; returns (buffer, view)."""
    T, H = t.shape
    buf = torch.full((off + T * (H + 1) + 32,), 7.0, device=DEV, dtype=t.dtype)
    v = torch.as_strided(buf, (T, H), (H + 1, 1), off)
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 15, 16, 17, 23, 24, 40, 261, 512, 1031, 4608])
@pytest.mark.parametrize("xd,rd,od", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", "f32")])
def test_add_rmsnorm_bits_do_not_depend_on_alignment(H, xd, rd, od):
    """Rows at every offset from a 16-byte boundary give the bits of rows at the boundary, and
    nothing is written beside the rows."""
    T = 9
    g = gen(H)
    x, res, gn = randn(g, T, H, dtype=DT[xd]), randn(g, T, H, dtype=DT[rd], scale=5.0), 1 + randn(g, H, scale=0.2)
    want_s = (x.float() + res.float()).to(DT[rd])
    want = torch.empty(T, H, device=DEV, dtype=DT[od])
    for t in range(T):  # one row a call: at the boundary whatever H is
        row = torch.empty(1, H, device=DEV, dtype=DT[od])
        L.moe_add_rmsnorm(x[t:t + 1].clone(), gn, 1e-5, res=res[t:t + 1].clone(), out=row)
        want[t] = row[0]
    for off in range(8):
        xv, rv = placed(x, off)[1], placed(res, (3 * off + 1) % 8)[1]
        sbuf, sv = placed(torch.zeros_like(res), (5 * off + 2) % 8)
        obuf = torch.full((off + T * H + 32,), 7.0, device=DEV, dtype=DT[od])
        out = torch.as_strided(obuf, (T, H), (H, 1), off)
        gv = torch.empty(off + H, device=DEV)[off:].copy_(gn)
        L.moe_add_rmsnorm(xv, gv, 1e-5, res=rv, sum_out=sv, out=out)
        assert torch.equal(out, want) and torch.equal(sv, want_s), off
        assert bool((obuf[:off] == 7).all()) and bool((obuf[off + T * H:] == 7).all())
        sv.fill_(7)
        assert bool((sbuf == 7).all())
        L.moe_add_rmsnorm(xv, gv, 1e-5, res=rv, sum_out=rv, out=out)  # in place
        assert torch.equal(out, want) and torch.equal(rv, want_s), off


# ------------------------------------------------------------------ route
ROUTE = [  # T, E, k, score, bias, groups, keep, best, renorm, scale
    (1, 1, 1, "softmax", False, 1, 1, 1, True, 1.0),
    (8, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (65, 384, 8, "softmax", True, 1, 1, 1, True, 1.0),
    (33, 384, 8, "softmax", False, 1, 1, 1, False, 16.0),
    (20, 33, 33 - 1, "sigmoid", False, 1, 1, 2, True, 1.0),
    (40, 96, 6, "softmax", False, 32, 3, 1, True, 1.0),
    (40, 160, 6, "softmax", True, 8, 3, 1, False, 16.0),
    (17, 1024, 16, "sigmoid", True, 16, 5, 2, True, 1.0),
    (9, 1024, 32, "sigmoid", False, 1, 1, 1, True, 1.0),
    (31, 62, 2, "sigmoid", True, 2, 1, 2, True, 1.0),
    (300, 8, 2, "softmax", True, 4, 2, 2, True, 1.0),
    (70, 512, 4, "sigmoid", True, 4, 4, 1, True, 3.0),
    (5, 384, 1, "sigmoid", True, 1, 1, 1, True, 1.0),
]


def _decided(c, k, groups, keep, best, eps=1e-5):
    """Rows whose order hangs on no difference below eps of the largest score."""
    T, E = c.shape
    ok = np.ones(T, dtype=bool)
    for t in range(T):
        v = c[t].copy()
        least = eps * np.abs(v).max()
        if groups > 1:
            b = np.sort(v.reshape(groups, -1), axis=1)[:, ::-1][:, :best].sum(1)
            o = np.argsort(-b, kind="stable")
            if keep < groups and 0 < b[o[keep - 1]] - b[o[keep]] < least:
                ok[t] = False
            v[~np.isin(np.arange(E) // (E // groups), o[:keep])] = -1e30
        d = -np.diff(np.sort(v)[::-1][:k + 1])
        ok[t] &= not np.any((d > 0) & (d < least))
    return ok


def _run_route(lg, k, bias=None, **kw):
    T = lg.shape[0]
    ids = torch.full((T, k), -7, device=DEV, dtype=torch.int32)
    w = torch.full((T, k), -7.0, device=DEV)
    err = torch.zeros(1, device=DEV, dtype=torch.int32)
    kw["score"] = L.SCORE_SIGMOID if kw.pop("score", "softmax") == "sigmoid" else L.SCORE_SOFTMAX
    L.moe_route_scored(lg, k, ids, w, bias=bias, dev_err=err, **kw)
    return host(ids), host(w).astype(np.float64), L.moe_get_error(err)


@pytest.mark.parametrize("T,E,k,score,bias,groups,keep,best,renorm,scale", ROUTE)
def test_route_scored(T, E, k, score, bias, groups, keep, best, renorm, scale):
    rng = np.random.default_rng(E * 1000 + k)
    b = (rng.standard_normal(E) * (0.05 if score == "sigmoid" else 0.3 / E)).astype(np.float32) if bias else None
    kw = dict(score=score, n_group=groups, topk_group=keep, group_top=best, renorm=renorm, scale=scale)
    lg = np.empty((0, E), np.float32)
    while lg.shape[0] < T:  # rows whose order is decided
        new = rng.standard_normal((2 * T, E)).astype(np.float32)
        if not bias:
            new = np.round(new * 16) / 16  # equal logits among them
        c = B.scores(new, score) + (0 if b is None else b.astype(np.float64))
        lg = np.concatenate([lg, new[_decided(c, k, groups, keep, best)]])
    lg = lg[:T].copy()
    wide = torch.zeros(T, E + 5, device=DEV)
    wide[:, :E] = torch.from_numpy(lg).to(DEV)
    bt = None if b is None else torch.from_numpy(b).to(DEV)
    want_ids, want_w, _ = B.route_scored(lg, k, b, **kw)
    for t in (wide[:, :E], wide[:, :E].contiguous()):
        ids, w, err = _run_route(t, k, bt, **kw)
        assert err == 0
        assert np.array_equal(ids, want_ids)
        assert np.all(np.abs(w - want_w) <= 1e-5 * np.abs(want_w))


@pytest.mark.parametrize("E,groups,keep", [(128, 1, 1), (129, 1, 1), (513, 1, 1), (640, 4, 2), (641, 1, 1), (768, 16, 16), (769, 1, 1),
                                           (896, 8, 3), (897, 1, 1), (1000, 8, 8), (1024, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored_widths(E, groups, keep, score):
    """Both sides of every number of experts a lane can hold; groups that all stay."""
    test_route_scored(37, E, 8, score, True, groups, keep, 2, True, 2.5)


def test_route_scored_all_groups_kept_is_no_groups():
    """Masked and NaN logits among them."""
    g = gen(11)
    l = randn(g, 64, 256)
    l[randn(g, 64, 256) > 1] = -float("inf")
    l[3, 7] = float("nan")
    l[5] = -float("inf")
    l[6, :32] = float("nan")  # a whole group
    b = randn(g, 256, scale=0.01)
    r = []
    for n in (1, 8):
        ids, w, err = torch.empty(64, 8, device=DEV, dtype=torch.int32), torch.empty(64, 8, device=DEV), torch.zeros(1, device=DEV, dtype=torch.int32)
        L.moe_route_scored(l, 8, ids, w, bias=b, score=L.SCORE_SIGMOID, n_group=n, topk_group=n, group_top=2, dev_err=err)
        r.append((host(ids), host(w), int(err)))
    assert np.array_equal(r[0][0], r[1][0]) and np.array_equal(r[0][1], r[1][1]) and r[0][2] == r[1][2]


def test_route_scored_is_moe_route():
    """Softmax, no bias, one group, renormalised: the ids of moe_route, its weights to rounding."""
    g = gen(5)
    lg = torch.randint(-20, 20, (200, 384), generator=g, device=DEV).float() / 4
    ids, w, _ = _run_route(lg, 8)
    ids0 = torch.empty(200, 8, device=DEV, dtype=torch.int32)
    w0 = torch.empty(200, 8, device=DEV)
    L.moe_route(lg, 8, ids0, w0)
    assert np.array_equal(ids, host(ids0)) and np.allclose(w, host(w0), rtol=2e-5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,best", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_scored_masks(score, groups, keep, best):
    """Masked experts, rows with one and with none left, NaN and infinite logits, the
    type's lowest value, a -inf bias."""
    E, k = 40, 4
    rng = np.random.default_rng(9)
    lg = rng.permuted(np.tile(np.linspace(-3, 3, E), (10, 1)), axis=1).astype(np.float32)
    lg[0, rng.permutation(E)[:30]] = -np.inf
    lg[1] = -np.inf
    lg[2] = -np.inf
    lg[2, 17] = 0.5
    lg[3, 5] = np.nan
    lg[4] = np.nan
    lg[5, 7] = np.inf
    lg[6] = np.finfo(np.float32).min
    lg[7, :20] = np.finfo(np.float32).min
    lg[8, 3] = np.nan
    lg[8, 4:] = -np.inf
    for bias in (None, np.where(np.arange(E) == 12, -np.inf, np.linspace(0, 0.01, E)).astype(np.float32)):
        kw = dict(score=score, n_group=groups, topk_group=keep, group_top=best)
        bt = None if bias is None else torch.from_numpy(bias).to(DEV)
        ids, w, err = _run_route(torch.from_numpy(lg).to(DEV), k, bt, **kw)
        want_ids, want_w, _ = B.route_scored(lg, k, bias, **kw)
        assert err == L.DEVERR_NAN_LOGIT
        assert np.array_equal(ids, want_ids)
        assert np.all(np.isfinite(w)) and np.all(np.abs(w - want_w) <= 1e-5 * np.abs(want_w) + 1e-37)


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("T,k,H", [(1, 1, 32), (3, 2, 96), (64, 8, 4096), (5, 32, 544), (700, 3, 7168), (33, 1, 2080)])
def test_gather_mxfp8(T, k, H):
    g = gen(H + T)
    xq = torch.randint(0, 256, (T, H), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    xs = torch.randint(0, 256, (T, H // 32), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    inv = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
    drop = T * k > 4
    if drop:
        inv[2] = -1  # an assignment without a row
    xp = torch.full((T * k, H), 9, device=DEV, dtype=torch.uint8)
    xps = torch.full((T * k, H // 32), 9, device=DEV, dtype=torch.uint8)
    L.moe_gather_mxfp8(xq, xs, inv, k, xp, xps)
    want, wants = np.full((T * k, H), 9, np.uint8), np.full((T * k, H // 32), 9, np.uint8)
    iv = host(inv)
    for a in range(T * k):
        if iv[a] >= 0:
            want[iv[a]], wants[iv[a]] = host(xq)[a // k], host(xs)[a // k]
    assert np.array_equal(host(xp), want) and np.array_equal(host(xps), wants)


def test_norm_then_gather_is_the_quantising_gather():
    """norm's MXFP8 rows gathered = moe_permute quantising norm's bf16 rows: the same bytes."""
    T, H, k, E = 77, 1024, 4, 16
    g = gen(11)
    x = randn(g, T, H, dtype=torch.bfloat16)
    out = torch.empty_like(x)
    q, qs = (torch.empty(T, n, device=DEV, dtype=torch.uint8) for n in (H, H // 32))
    L.moe_add_rmsnorm(x, None, 1e-6, out=out, q=q, q_scale=qs)
    ids = torch.stack([torch.randperm(E, generator=g, device=DEV)[:k] for _ in range(T)]).to(torch.int32)
    off, perm, inv = (torch.empty(n, device=DEV, dtype=torch.int32) for n in (E + 1, T * k, T * k))
    rows = [[torch.empty(T * k, n, device=DEV, dtype=torch.uint8) for n in (H, H // 32)] for _ in range(2)]
    L.moe_permute(ids, E, off, perm, inv, x=out, act_fmt=L.FMT_MXFP8, x_perm=rows[0][0], x_perm_scale=rows[0][1])
    L.moe_gather_mxfp8(q, qs, inv, k, *rows[1])
    assert torch.equal(rows[0][0], rows[1][0]) and torch.equal(rows[0][1], rows[1][1])


# ------------------------------------------------------------------ linear
def _ints(g, *shape):
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(torch.bfloat16)


ACT = {"none": L.ACT_NONE, "silu": L.ACT_SILU, "gelu": L.ACT_GELU, "swiglu": L.ACT_SWIGLU}
LINEAR = [  # T, N, K
    (1, 1, 1), (1, 384, 4096), (3, 5, 7), (8, 256, 520), (16, 2048, 512), (17, 384, 1032), (33, 130, 64), (64, 300, 264),
    (65, 77, 136), (100, 512, 2048), (128, 128, 72), (200, 1000, 1000), (257, 640, 328), (777, 190, 1464), (1500, 256, 200),
    (2049, 513, 64), (300, 4100, 40), (40, 32, 8192), (1100, 2304, 520),
]


def _strided(g, T, C, pad, make):
    return make(g, T, C + pad)[:, :C]


@pytest.mark.parametrize("T,N,K", LINEAR)
@pytest.mark.parametrize("out,res,bias,pad", [("f32", None, False, 0), ("f32", "f32", True, 8), ("bf16", "bf16", True, 8),
                                              ("bf16", None, False, 3), ("f32", "bf16", True, 0)])
def test_linear_exact_sums(T, N, K, out, res, bias, pad):
    """Integer operands: every sum is exact, so the product, bias and residual are, too."""
    g = gen(T + 7 * N + 13 * K)
    x, w = _strided(g, T, K, pad, _ints), _strided(g, N, K, pad, _ints)
    b = torch.randint(-50, 50, (N,), generator=g, device=DEV).float() if bias else None
    r = None if res is None else torch.randint(-60, 60, (T, N + pad), generator=g, device=DEV).to(DT[res])[:, :N]
    o = torch.full((T, N + pad), 11.0, device=DEV, dtype=DT[out])
    err = torch.zeros(1, device=DEV, dtype=torch.int32)
    L.moe_linear(x, w, o[:, :N], bias=b, res=r, dev_err=err)
    want = x.double() @ w.double().t()
    if b is not None:
        want = want + b.double()
    if r is not None:
        want = want + r.double()
    assert L.moe_get_error(err) == 0
    assert torch.equal(o[:, :N], want.to(DT[out]))
    assert bool((o[:, N:] == 11.0).all())


@pytest.mark.parametrize("T,N,K", [(1, 16, 64), (8, 2048, 512), (5, 7, 33), (50, 304, 136), (130, 256, 1024), (700, 528, 264),
                                   (300, 24, 64), (1030, 1152, 520)])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_activations(T, N, K, act, out):
    g = gen(T + N + K)
    rows = 2 * N if act == "swiglu" else N
    x, w = _ints(g, T, K), (_ints(g, rows, K).float() / 8).to(torch.bfloat16)
    b = torch.randint(-8, 8, (rows,), generator=g, device=DEV).float() / 4
    r = torch.randint(-60, 60, (T, N), generator=g, device=DEV).float() / 16
    o = torch.empty(T, N, device=DEV, dtype=DT[out])
    L.moe_linear(x, w, o, bias=b, act=ACT[act], res=r)
    want = B.linear(f64(x), f64(w), f64(b), act, f64(r))
    v = np.abs(B.linear(f64(x), f64(w), f64(b)))
    size = (v[:, :N] * (1 + v[:, N:]) if act == "swiglu" else v) + np.abs(f64(r))
    assert within(o, want, 4e-6 * size)


@pytest.mark.parametrize("T,N,K", [(8, 384, 7168), (64, 256, 4096), (300, 384, 4096), (2500, 256, 7168), (900, 1152, 1024)])
def test_linear_fp32_sums(T, N, K):
    g = gen(K + T)
    x, w = randn(g, T, K, dtype=torch.bfloat16), randn(g, N, K, dtype=torch.bfloat16)
    o = torch.empty(T, N, device=DEV)
    L.moe_linear(x, w, o)
    want = x.double() @ w.double().t()
    assert float((o.double() - want).norm() / want.norm()) <= 2e-6


def test_linear_in_place_streams_and_repeat():
    g = gen(2)
    x, w = randn(g, 90, 512, dtype=torch.bfloat16), randn(g, 640, 512, dtype=torch.bfloat16)
    base = randn(g, 90, 640, dtype=torch.bfloat16)
    a, b = base.clone(), base.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    L.moe_linear(x, w, a, res=a, stream=st)
    st.synchronize()
    c = torch.empty_like(base)
    L.moe_linear(x, w, c, res=base)
    L.moe_linear(x, w, b, res=b)
    assert torch.equal(a, c) and torch.equal(b, c)  # the same bits, in place or not, every time


def test_linear_non_finite_operands_stay_in_their_row_and_column():
    g = gen(4)
    for T, N, K in ((20, 200, 72), (300, 300, 136)):  # K and tiles end inside a block
        x, w = randn(g, T, K, dtype=torch.bfloat16), randn(g, N, K, dtype=torch.bfloat16)
        x[3, K - 1] = float("nan")
        w[N - 1, 0] = float("inf")
        o = torch.empty(T, N, device=DEV)
        L.moe_linear(x, w, o)
        bad = ~np.isfinite(host(o))
        assert bad[3].all() and bad[:, N - 1].all()
        bad[3] = False
        bad[:, N - 1] = False
        assert not bad.any()


def test_linear_long_rows_apart():
    """Row offsets past 32 bits, in x and in the output."""
    ld = (1 << 31) + 64
    base = torch.zeros(ld + 64, device=DEV, dtype=torch.bfloat16)
    x = torch.as_strided(base, (2, 64), (ld, 1))
    x[0], x[1] = 1.0, 2.0
    w = torch.ones(48, 64, device=DEV, dtype=torch.bfloat16)
    ob = torch.zeros(ld + 48, device=DEV, dtype=torch.bfloat16)
    o = torch.as_strided(ob, (2, 48), (ld, 1))
    L.moe_linear(x, w, o)
    assert bool((o[0] == 64).all()) and bool((o[1] == 128).all())
