"""One MoE block (residual + norm, router, scored routing, experts, shared
expert) on the GPU: every stage against the float64 oracle of the values the
stage before it produced, the MXFP8 rows' way against the quantising gather,
and the captured graph against the eager step (same bits).

Tolerances: norm and products as in test_gpu_block_ops (fp32 sums 2e-6 of the
2-norm at these K; bf16 results half a step); the routed experts at the
layer's own gates (TOL_BF16 / TOL_FP8)."""
import numpy as np
import pytest
import torch

from bit_moe_expert_top_gb300 import _lib as L
from bit_moe_expert_top_gb300 import synth
from bit_moe_expert_top_gb300.block import MoEBlock
from oracle import block as B
from oracle import moe as M

from tests._gpu import TOL_BF16, TOL_FP8, host, make_layer, rel_err

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def _block(base, T, direct=False, score=L.SCORE_SIGMOID, shared=True, res=torch.float32, H=512, I=512):
    w = synth.get_workload(base).replace(E=16, H=H, I=I, k=4, T=T, logits="uniform")
    if w.weights == "mixed":
        w = w.replace(n_hot=4)
    ml, acc, prof = make_layer(w, mode=L.MODE_AUTO, direct=direct)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + 1)
    rnd = lambda *s, scale=1.0: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
    sh = None
    if shared:
        sh = (rnd(2 * 384, H, scale=H ** -0.5).bfloat16(), rnd(H, 384, scale=384 ** -0.5).bfloat16())
    bl = MoEBlock(ml, 1 + rnd(H, scale=0.1), rnd(w.E, H, scale=2 * H ** -0.5).bfloat16(), shared=sh,
                  balance=rnd(w.E, scale=0.02), score=score, n_group=4, topk_group=2, group_top=2, scale=1.5)
    return w, bl, acc, prof, rnd(T, H).bfloat16(), rnd(T, H, scale=3.0).to(res)


def _experts(x, ids, wt, acc, prof):
    """The routed experts for given ids and weights."""
    ffn = M.expert_ffn_fp8 if prof == "fp8" else M.expert_ffn_bf16
    T, k = ids.shape
    y = np.empty((T, k, x.shape[1]))
    for e in np.unique(ids):
        W1, W2 = acc(int(e))
        rows, slots = np.nonzero(ids == e)
        y[rows, slots] = ffn(x[rows], W1, W2)
    return M.combine(y, wt)


PATHS = [("tiny", False, L.SCORE_SIGMOID, True, torch.float32), ("tiny", False, L.SCORE_SOFTMAX, False, torch.bfloat16),
         ("mixed_decode", False, L.SCORE_SIGMOID, True, torch.bfloat16),
         ("prefill_fp8", True, L.SCORE_SIGMOID, True, torch.float32), ("prefill_fp8", False, L.SCORE_SOFTMAX, True, torch.bfloat16)]


@pytest.mark.parametrize("base,direct,score,shared,res", PATHS)
@pytest.mark.parametrize("T", [1, 24])
def test_block_stage_by_stage(base, direct, score, shared, res, T):
    w, bl, acc, prof, x, r = _block(base, T, direct, score, shared, res)
    r0 = r.clone()
    b = bl.buffers(T)
    out = bl.step(x, r, b)
    torch.cuda.synchronize()
    assert L.moe_get_error(b.step.dev_err) == 0
    assert torch.equal(r, (x.float() + r0.float()).to(res))  # the residual, in place
    _, n = B.add_rmsnorm(f64(x), f64(bl.gain), bl.eps, f64(r0))
    assert np.all(np.abs(f64(b.normed) - n) <= (2.0 ** -8 + 3e-6) * np.abs(n))
    lg = B.linear(f64(b.normed), f64(bl.router))
    assert np.linalg.norm(f64(b.logits) - lg) <= 2e-6 * np.linalg.norm(lg)
    ids, wt, _ = B.route_scored(host(b.logits), w.k, host(bl.routing["bias"]),
                                score="sigmoid" if score == L.SCORE_SIGMOID else "softmax", n_group=4, topk_group=2,
                                group_top=2, scale=1.5)
    assert np.array_equal(host(b.step.ids), ids) and np.allclose(host(b.step.w), wt, rtol=1e-5)
    want = _experts(f64(b.normed), ids, host(b.step.w), acc, prof)
    if shared:
        h = B.linear(f64(b.normed), f64(bl.shared[0]), act="swiglu")
        assert np.all(np.abs(f64(b.h) - h) <= 2.0 ** -8 * np.abs(h) + 1e-5 * np.abs(h).max())
        want = want + B.linear(f64(b.h), f64(bl.shared[1]))
    err, rms = rel_err(f64(out), want)
    assert rms > 0 and err <= (TOL_FP8 if prof == "fp8" else TOL_BF16), err


def test_block_mxfp8_rows_are_the_gathers():
    """The experts' outputs do not depend on who quantised the rows: same bits."""
    w, bl, _, _, x, r = _block("prefill_fp8", 40, direct=True, shared=False)
    b = bl.buffers(40)
    out = bl.step(x, r, b).clone()
    s2 = bl.layer.buffers(40)
    s2.ids.copy_(b.step.ids)
    s2.w.copy_(b.step.w)
    assert torch.equal(out, bl.layer.experts(b.normed, s2))
    assert torch.equal(b.step.x_perm, s2.x_perm) and torch.equal(b.step.x_perm_scale, s2.x_perm_scale)


@pytest.mark.parametrize("base", ["tiny", "prefill_fp8"])
def test_block_graph_replays_the_step(base):
    w, bl, _, _, x, r = _block(base, 8, direct=True)
    g = bl.capture(8)
    for i in range(2):
        b = bl.buffers(8)
        r1 = r.clone()
        want = bl.step(x + i, r1, b)
        got = g.run(x + i, r)
        assert torch.equal(got, want) and torch.equal(g.residual, r1)


def test_block_empty_batch():
    w, bl, _, _, x, r = _block("tiny", 0)
    b = bl.buffers(0)
    assert bl.step(x, r, b).shape[0] == 0
    assert L.moe_get_error(b.step.dev_err) == 0


def test_experts_is_the_step_after_routing():
    """MoELayer.step = moe_route + experts, bit for bit."""
    w = synth.get_workload("tiny").replace(E=16, H=512, I=512, k=4, T=40, logits="uniform")
    ml, _, _ = make_layer(w)
    x = torch.from_numpy(synth.make_x(w).view(np.int16)).cuda()
    lg = torch.from_numpy(synth.make_logits(w)).cuda()
    b1, b2 = ml.buffers(40), ml.buffers(40)
    out = ml.step(x, lg, b1)
    L.moe_route(lg, w.k, b2.ids, b2.w)
    assert torch.equal(out, ml.experts(x, b2))
