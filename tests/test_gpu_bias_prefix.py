"""A prefix array whose last sequence ends past the query rows, or past the rows of the weights: it is skipped and flagged,
nothing of it is written, and the others are not disturbed."""
import pytest
import torch

import bias_reference as ref
import ragged_variable_length_b200 as rv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,extra", [([5, 3, 9], 4), ([100, 70, 130], 90), ([700, 60, 1], 3000)], ids=str)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 2)])
def test_rows_past_the_queries(lens, extra, H, Hkv, dtype):
    s = ref.problem(lens, lens, H, Hkv, dtype, 32, 128, layout="rows", extra=0)
    q, k, v, args, _ = ref.on_gpu(s)
    # the last sequence, one row too long at least; keys as many as there are
    cu_q = args[0].clone()
    cu_q[-1] += extra
    longest = max(lens) + extra
    bad = (cu_q, args[1], longest, args[3], *args[4:])
    n, T = lens[0] + lens[1], sum(lens)
    rv.ragged_get_device_status()
    nan = lambda *shape, dt=dtype: torch.full(shape, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    out, lse = nan(T, H, 64), nan(H, T, dt=torch.float32)
    rv.ragged_attn_bias_fwd(q, k, v, *bad, out=out, lse=lse)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    weight = rv.ragged_attn_weight(q, k, lse, *bad, weight=nan(H, T, dt=torch.float32))
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    grads = dict(dq=nan(T, H, 64), dk=nan(T, Hkv, 64), dv=nan(T, Hkv, 64))
    rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *bad, **grads)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    good = ref.attention(s, s["dout"])
    for name, t in dict(grads, out=out).items():
        ref.check(name, t[:n], good[name][0][:n], good[name][1][:n])
        assert torch.isnan(t[n:]).all(), name
    for name, t in (("lse", lse), ("weight", weight)):
        ref.check(name, t[:, :n], good[name][0][:, :n], good[name][1][:, :n])
        assert torch.isnan(t[:, n:]).all(), name


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens_q,lens_k,extra", [([1, 2], [40, 30], 9), ([100, 70], [50, 90], 300)], ids=str)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 2)])
def test_keys_past_the_weights(lens_q, lens_k, extra, H, Hkv, dtype):
    s = ref.problem(lens_q, lens_k, H, Hkv, dtype, 32, 128, layout="rows", extra=0)
    q, k, v, args, _ = ref.on_gpu(s)
    _, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    cu_k = args[1].clone()
    cu_k[-1] += extra
    weight = torch.full((H, sum(lens_k)), float("nan"), device="cuda")
    rv.ragged_get_device_status()
    rv.ragged_attn_weight(q, k, lse, args[0], cu_k, args[2], args[3] + extra, *args[4:], weight=weight)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    good = ref.attention(s)["weight"]
    n = lens_k[0]
    ref.check("weight", weight[:, :n], good[0][:, :n], good[1][:, :n])
    assert torch.isnan(weight[:, n:]).all()
