"""Problems whose bias entries are far from 0 (mask constants, a type's extremes), and what they have to give.

Scores are fp32, so where |s| is large what fp32 holds of them counts: q k is lost beside a bias of -1e9 (steps of 64),
and a row whose keys all carry it has equal weights.  `definition` is that of bias_reference over the scores rounded to
fp32, with each row's largest subtracted first (64 bits lose the logarithm of a sum beside 1e38 as 32 do).

A kernel's score and the rounded one here are each within half an fp32 step of the same number, so they differ by at most
one step, 2^-23 |bias|, where q k does not vanish beside it; a probability then by twice that (itself and its row's
sum).  bf16 values here are 5e8 and above: steps of 32 or more, against |q k| scale below 16, so both round to the bias.
"""
import torch

import bias_reference as ref

F16, BF16 = torch.float16, torch.bfloat16
VALUES = [(F16, -3.0e4), (F16, "lowest"), (F16, "highest"), (BF16, -1.0e9), (BF16, -1.0e10), (BF16, 1.0e10), (BF16, -1.0e30), (BF16, -1.0e38),
          (BF16, "lowest"), (BF16, "highest")]
# every key at the value; only a token itself and those behind it; two values, one far below the other
PATTERNS = ["all", "self and later", "two"]
# one to 32 rows per key head (kernels that share a small tile among them), and more
LENGTHS = [([1], [1], 1, 1), ([5, 0, 2], [5, 0, 2], 2, 2), ([20], [20], 1, 1), ([8, 3], [300, 70], 8, 2), ([40, 200], [40, 200], 2, 2),
           ([33, 5], [700, 64], 2, 1), ([700], [700], 1, 1)]


def problem(dtype, value, pattern, lens_q, lens_k, H, Hkv, where="none", D=128):
    s = ref.problem(lens_q, lens_k, H, Hkv, dtype, 32, D, where=where, seed=len(lens_q) + H, layout="rows", extra=2)
    v = {"lowest": torch.finfo(dtype).min, "highest": torch.finfo(dtype).max}.get(value, value)
    if pattern == "all":
        s["table"][:] = v
    elif pattern == "two":
        s["table"][0::2] = v
        s["table"][1::2] = v / 2
    else:
        s["table"][0] = v
        s["table"][16:] = v
    return s


def eps32(dtype):
    """EPS32 of bias_reference and the step of a score of f16's largest size, twice."""
    return 2.0 ** -14 + (2.02 * 65504 * 2.0 ** -23 if dtype == F16 else 0.0)


def definition(monkeypatch, s, dout=None):
    tops, plain = {}, ref.scores

    def rounded(s, b, h):
        x, bucket, i, j, z = plain(s, b, h)
        x = x.float().double()
        if x.numel():
            top = x.amax(1, keepdim=True)
            tops[h, i.start, i.stop] = top = torch.where(torch.isinf(top), 0.0, top)
            x = x - top
        return x, bucket, i, j, z

    with monkeypatch.context() as m:
        m.setattr(ref, "scores", rounded)
        m.setattr(ref, "EPS32", eps32(s["q"].dtype))
        r = ref.attention(s, dout)
    for (h, a, z), top in tops.items():
        r["lse"][0][h, a:z] += top[:, 0]
        # the reference and its sum's logarithm, added and rounded; a step of the reference
        r["lse"][1][h, a:z] += 2.0 ** -22 * top[:, 0].abs()
    return r


def check(s, good, got):
    nq, nk = s["cu_q"][-1], s["cu_k"][-1]
    rows = {"out": slice(0, nq), "dq": slice(0, nq), "dk": slice(0, nk), "dv": slice(0, nk), "lse": (slice(None), slice(0, nq)),
            "weight": (slice(None), slice(0, nk)), "dtable": slice(None)}
    for name, value in got.items():
        ref.check(name, value, *good[name], rows[name])
