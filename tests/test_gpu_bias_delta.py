"""Gradients where the rounding of out, from which the row sums delta = dout . out come, would show: values far from 0 (mean
16) whose differences make the gradients.

out is off by up to 16 u in each of 64 elements, so delta by tens of u against dP - delta of size 8, in every dS of a row with
one sign.  A row's dS add up to 0; what they add up to is what delta is off by.  The kernels take that out of dk, out of
dtable where a tile's distances all lie past one end of the map, and out of everything where a row's keys are one tile.  What
stays in dtable is known: off_i P_ij of the other pairs.

Else dS and the results are rounded, u each.  Errors of one sum are independent, at most u of their terms and on average half of
it, and add in squares to about the sum's own size: 2 u of a gradient's norm is three times what they come to.  dtable adds up
dS unrounded: u, and 2^-12 for fp32 scores and sums.
"""
import pytest
import torch

import bias_reference as ref
import ragged_variable_length_b200 as rv

pytestmark = pytest.mark.gpu


def outside_flat_tiles(n, D):
    """Pairs of a sequence with consecutive positions: those in tiles of 32 rows and 64 columns with a distance inside the map."""
    i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
    first_row, last_row = i // 32 * 32, (i // 32 * 32 + 31).clamp_max(n - 1)
    first_col, last_col = j // 64 * 64, (j // 64 * 64 + 63).clamp_max(n - 1)
    return ~((last_col - first_row <= -D) | (first_col - last_row >= D))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 1)])
@pytest.mark.parametrize("lens,D", [([1500], 16), ([1100, 65, 900], 8), ([300, 129], 200), ([50], 128), ([64, 33, 1, 7], 128)], ids=str)
def test_values_far_from_zero(lens, D, H, Hkv, dtype):
    s = ref.problem(lens, lens, H, Hkv, dtype, 32, D, layout="rows", extra=0, seed=sum(lens))
    s["base"]["kv"][:, 1] += 16.0   # s["v"] is a view of it
    q, k, v, args, where = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args, **where)
    got = dict(zip(("dq", "dk", "dv", "dtable"), rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *args, **where)))
    good = ref.attention(s, s["dout"])
    one_tile = max(lens) <= 64
    left = torch.zeros_like(good["dtable"][0])
    if not one_tile:
        for b, n in enumerate(lens):
            for h in range(H):
                x, bucket, i, j, z = ref.scores(s, b, h)
                off = (s["dout"][i, h].double() * (out[i, h].double().cpu() - good["out"][0][i, h])).sum(1, keepdim=True)
                left[:, h] -= torch.bincount(bucket.reshape(-1), (off * torch.softmax(x, 1) * outside_flat_tiles(n, D)).reshape(-1), 32)
    u = torch.finfo(dtype).eps / 2
    for name in ("dq", "dk", "dtable") if one_tile else ("dk", "dtable"):
        want = good[name][0] + (left if name == "dtable" else 0.0)
        error = ((got[name].double().cpu() - want).norm() / want.norm()).item()
        assert error <= (u + 2.0 ** -12 if name == "dtable" else 2 * u), (name, error / u)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_short_sequences_beside_a_long_one(dtype):
    """Sequences of one tile in a batch whose bound is longer: the same bits every time, and dk as it is without the rounding
    of out."""
    lens = [1 + (29 * i) % 64 for i in range(120)] + [400]
    s = ref.problem(lens, lens, 4, 2, dtype, 32, 128, layout="rows", extra=0)
    s["base"]["kv"][:, 1] += 16.0
    q, k, v, args, where = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args, **where)
    do = s["dout"].cuda()
    first = rv.ragged_attn_bias_bwd(do, q, k, v, out, lse, *args, **where)
    for _ in range(20):
        for a, b in zip(first, rv.ragged_attn_bias_bwd(do, q, k, v, out, lse, *args, **where)):
            assert torch.equal(a, b)
    want = ref.attention(s, s["dout"])["dk"][0]
    assert ((first[1].double().cpu() - want).norm() / want.norm()).item() <= torch.finfo(dtype).eps
