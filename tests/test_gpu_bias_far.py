"""Bias entries far from 0 on the GPU: mask constants and the types' extremes give the softmax over fp32 scores in every
kernel, whatever the number of rows."""
import pytest
import torch

import bias_far as far
import bias_reference as ref
import ragged_variable_length_b200 as rv

pytestmark = pytest.mark.gpu
F16, BF16 = far.F16, far.BF16


@pytest.mark.parametrize("lens_q,lens_k,H,Hkv", far.LENGTHS, ids=str)
@pytest.mark.parametrize("pattern", far.PATTERNS)
@pytest.mark.parametrize("dtype,value", far.VALUES, ids=str)
@pytest.mark.parametrize("where,D", [("none", 16), ("sorted", 128)])
def test_attention(monkeypatch, dtype, value, pattern, lens_q, lens_k, H, Hkv, where, D):
    s = far.problem(dtype, value, pattern, lens_q, lens_k, H, Hkv, where, D)
    q, k, v, args, at = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args, **at)
    far.check(s, far.definition(monkeypatch, s), {"out": out, "lse": lse})
    assert rv.ragged_get_device_status() == 0


@pytest.mark.parametrize("lens_q,lens_k,H,Hkv", far.LENGTHS, ids=str)
@pytest.mark.parametrize("pattern", far.PATTERNS)
@pytest.mark.parametrize("dtype,value", far.VALUES, ids=str)
@pytest.mark.parametrize("where,D", [("none", 16), ("sorted", 128)])
def test_gradients_and_weights(monkeypatch, dtype, value, pattern, lens_q, lens_k, H, Hkv, where, D):
    s = far.problem(dtype, value, pattern, lens_q, lens_k, H, Hkv, where, D)
    q, k, v, args, at = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args, **at)
    r = {"weight": rv.ragged_attn_weight(q, k, lse, *args, **at)}
    r.update(zip(("dq", "dk", "dv", "dtable"), rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *args, **at)))
    far.check(s, far.definition(monkeypatch, s, s["dout"]), r)
    assert rv.ragged_get_device_status() == 0


@pytest.mark.parametrize("dtype,value", [(F16, None), (BF16, None)] + far.VALUES, ids=str)
@pytest.mark.parametrize("bound", [20, 200])
def test_calls_with_different_bounds(monkeypatch, dtype, value, bound):
    """The statistics of one kernel family serve the other: the bounds of the two calls lie on either side of 32 rows."""
    lens = [20, 3, 11]
    s = far.problem(dtype, 0.5 if value is None else value, "self and later", lens, lens, 1, 1)
    q, k, v, args, at = ref.on_gpu(s)
    forward = (*args[:2], bound, bound, *args[4:])
    other = (*args[:2], 220 - bound, 220 - bound, *args[4:])
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *forward, **at)
    r = {"out": out, "lse": lse, "weight": rv.ragged_attn_weight(q, k, lse, *other, **at)}
    r.update(zip(("dq", "dk", "dv", "dtable"), rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *other, **at)))
    far.check(s, far.definition(monkeypatch, s, s["dout"]), r)


@pytest.mark.parametrize("lens_q,lens_k,H,Hkv", far.LENGTHS, ids=str)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale", [1.0e4, 1.0e9, 1.0e30])
def test_scores_far_from_zero(dtype, scale, lens_q, lens_k, H, Hkv):
    """Large scores from q k: every row is its best key's, except where two keys come within an fp32 step of 64 products."""
    s = ref.problem(lens_q, lens_k, H, Hkv, dtype, 32, 128, seed=H, layout="rows", extra=0)
    q, k, v, args, at = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args, **at, scale=scale)
    w = rv.ragged_attn_weight(q, k, lse, *args, **at, scale=scale)
    # dS is 0 but for the rounding of out, and dq and dk are that times the scale: they say nothing, and may be past f16
    _, _, dv, dt = rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *args, **at, scale=scale)
    for t in (out, lse, w, dv, dt):
        assert torch.isfinite(t).all()
    s["scale"] = scale
    weight, clear = torch.zeros(H, sum(lens_k), dtype=torch.float64), True
    u = torch.finfo(dtype).eps
    for b in range(len(lens_q)):
        for h in range(H):
            x, _, i, j, z = ref.scores(s, b, h)
            if x.numel() == 0:
                continue
            top = torch.topk(x, min(2, x.shape[1]), dim=1)
            err = 2.0 ** -17 * (s["q"][i, h].double().abs() @ s["k"][j, z].double().abs().T).amax(1) * scale
            sure = (top.values[:, 0] - top.values[:, -1] > 2 * err + 40) if x.shape[1] > 1 else torch.ones(x.shape[0], dtype=torch.bool)
            best = s["v"][j, z].double()[top.indices[:, 0]]
            assert ((out[i, h].double().cpu() - best).abs() <= u * best.abs() + 1e-6)[sure].all()
            assert ((lse[h, i].double().cpu() - top.values[:, 0]).abs() <= err + 2.0 ** -22 * top.values[:, 0].abs() + 1.0).all()
            weight[h, j] += torch.zeros(x.shape[1], dtype=torch.float64).index_add(0, top.indices[:, 0], torch.ones(x.shape[0], dtype=torch.float64))
            clear &= bool(sure.all())
    if clear:
        assert ((w.double().cpu() - weight).abs() <= 2.0 ** -10 * (1 + weight)).all()
