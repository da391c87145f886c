"""Refusals of the operators with a position bias and of the eviction, and the bucket map: no GPU needed."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import ragged_variable_length_b200 as rv
from ragged_variable_length_b200 import build as rbuild

A16 = 1 << 20
A2, A4, A8 = A16 + 2, A16 + 4, A16 + 8
BAD, UNSUPPORTED = rv.RAGGED_ERR_INVALID_ARG, rv.RAGGED_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rv.load()


def _problem(**kw):
    a = dict(q=A16, k=A16, v=A16, q_tok_stride=384, q_head_stride=64, kv_tok_stride=384, kv_head_stride=64, cu_seqlens_q=A16,
             cu_seqlens_k=A16, B=2, max_seqlen_q=197, max_seqlen_k=197, H=6, Hkv=6, head_dim=64, table=A16, buckets=A16,
             num_buckets=32, max_distance=128, pos_q=None, pos_k=None, lse=A16, lse_stride=400, scale=0.125, dtype=rv.RAGGED_F16)
    a.update(kw)
    return rv.BiasAttn(**a)


PROBLEMS = [
    (dict(B=-1), BAD, "negative"), (dict(B=70000), UNSUPPORTED, "65535"), (dict(H=0), BAD, "H ="), (dict(H=6, Hkv=4), BAD, "multiple of Hkv"),
    (dict(Hkv=0), BAD, "Hkv"), (dict(H=70000, Hkv=70000), BAD, "H ="), (dict(head_dim=128), UNSUPPORTED, "head_dim"), (dict(dtype=7), BAD, "dtype"),
    (dict(dtype=rv.RAGGED_F32), UNSUPPORTED, "f16 and bf16"), (dict(max_seqlen_q=0), BAD, "max_seqlen"), (dict(max_seqlen_k=0), BAD, "max_seqlen"),
    (dict(max_seqlen_k=rv.RAGGED_MAX_TOKENS + 1), BAD, "max_seqlen"), (dict(scale=0.0), BAD, "scale"), (dict(scale=-1.0), BAD, "scale"),
    (dict(scale=math.nan), BAD, "scale"), (dict(scale=math.inf), BAD, "scale"), (dict(scale=2e38), BAD, "scale"), (dict(num_buckets=0), UNSUPPORTED, "num_buckets"),
    (dict(num_buckets=65), UNSUPPORTED, "num_buckets"), (dict(max_distance=-1), UNSUPPORTED, "max_distance"),
    (dict(max_distance=1025), UNSUPPORTED, "max_distance"), (dict(q=None), BAD, "NULL"), (dict(k=None), BAD, "NULL"),
    (dict(cu_seqlens_q=None), BAD, "NULL"), (dict(cu_seqlens_k=None), BAD, "NULL"), (dict(table=None), BAD, "NULL"), (dict(buckets=None), BAD, "NULL"),
    (dict(lse=None), BAD, "NULL"), (dict(q=A8), BAD, "16-byte"), (dict(k=A8), BAD, "16-byte"), (dict(cu_seqlens_k=A2), BAD, "4-byte"),
    (dict(pos_q=A2), BAD, "4-byte"), (dict(pos_k=A2), BAD, "4-byte"), (dict(buckets=A2), BAD, "4-byte"), (dict(lse=A2), BAD, "4-byte"),
    (dict(table=A16 + 1), BAD, "2-byte"), (dict(q_tok_stride=0), BAD, "q_tok_stride"), (dict(q_tok_stride=388), BAD, "q_tok_stride"),
    (dict(q_head_stride=60), BAD, "q_head_stride"), (dict(kv_tok_stride=-8), BAD, "kv_tok_stride"), (dict(kv_head_stride=0), BAD, "kv_head_stride"),
    (dict(lse_stride=-1), BAD, "lse_stride"),
]


@pytest.mark.parametrize("kw,status,needle", PROBLEMS, ids=[str(p[0]) for p in PROBLEMS])
def test_problem_rejects(lib, kw, status, needle):
    p, n = _problem(**kw), ctypes.c_int64(7)
    calls = [lambda: lib.ragged_attn_bias_fwd(p, A16, 384, A16, 1 << 40, None),
             lambda: lib.ragged_attn_bias_fwd_workspace(p, n),
             lambda: lib.ragged_attn_bias_bwd(p, A16, 384, A16, 384, A16, 384, 64, A16, A16, 384, 64, A16, A16, 1 << 40, None),
             lambda: lib.ragged_attn_bias_bwd_workspace(p, n),
             lambda: lib.ragged_attn_weight(p, None, A16, 400, None)]
    for call in calls:
        assert call() == status
        assert needle in rv.ragged_last_error()


def test_no_problem_and_no_sequences(lib):
    n = ctypes.c_int64(7)
    assert lib.ragged_attn_bias_fwd(None, A16, 384, None, 0, None) == BAD
    assert lib.ragged_attn_weight(None, None, A16, 400, None) == BAD
    assert lib.ragged_attn_bias_fwd_workspace(_problem(), None) == BAD
    empty = _problem(B=0, q=None, k=None, v=None, cu_seqlens_q=None, cu_seqlens_k=None, table=None, buckets=None, lse=None)
    assert lib.ragged_attn_bias_fwd(empty, None, 0, None, 0, None) == rv.RAGGED_OK
    assert lib.ragged_attn_weight(empty, None, None, 0, None) == rv.RAGGED_OK
    assert lib.ragged_attn_bias_bwd_workspace(empty, n) == rv.RAGGED_OK


@pytest.mark.parametrize("kw,needle", [(dict(out=None), "NULL"), (dict(out=A8), "16-byte"), (dict(stride=376), "out_tok_stride"),
                                       (dict(stride=388), "out_tok_stride")], ids=str)
def test_fwd_rejects(lib, kw, needle):
    a = dict(out=A16, stride=384)
    a.update(kw)
    assert lib.ragged_attn_bias_fwd(_problem(), a["out"], a["stride"], A16, 1 << 40, None) == BAD
    assert needle in rv.ragged_last_error()
    assert lib.ragged_attn_bias_fwd(_problem(v=None), A16, 384, A16, 1 << 40, None) == BAD
    assert lib.ragged_attn_bias_fwd(_problem(v=A8), A16, 384, A16, 1 << 40, None) == BAD


@pytest.mark.parametrize("kw,needle", [
    (dict(out=None), "NULL"), (dict(dout=None), "NULL"), (dict(dq=None), "NULL"), (dict(dk=None), "NULL"), (dict(dv=None), "NULL"),
    (dict(dtable=None), "dtable"), (dict(dtable=A16 + 1), "dtable"), (dict(dout=A8), "16-byte"), (dict(dq=A8), "16-byte"), (dict(dv=A8), "16-byte"),
    (dict(out_s=376), "out_tok_stride"), (dict(dout_s=380), "dout_tok_stride"), (dict(dq_s=4), "dq_tok_stride"), (dict(dq_h=4), "dq_head_stride"),
    (dict(dkv_s=0), "dkv_tok_stride"), (dict(dkv_h=-64), "dkv_head_stride"), (dict(ws=None), "workspace"), (dict(ws_bytes=64), "workspace"),
    (dict(ws=A8), "workspace")], ids=str)
def test_bwd_rejects(lib, kw, needle):
    a = dict(out=A16, out_s=384, dout=A16, dout_s=384, dq=A16, dq_s=384, dq_h=64, dk=A16, dv=A16, dkv_s=384, dkv_h=64, dtable=A16, ws=A16,
             ws_bytes=1 << 40)
    a.update(kw)
    assert lib.ragged_attn_bias_bwd(_problem(), a["out"], a["out_s"], a["dout"], a["dout_s"], a["dq"], a["dq_s"], a["dq_h"], a["dk"], a["dv"],
                                    a["dkv_s"], a["dkv_h"], a["dtable"], a["ws"], a["ws_bytes"], None) == BAD
    assert needle in rv.ragged_last_error()


@pytest.mark.parametrize("weight,prev,stride,needle", [(None, None, 400, "NULL"), (A2, None, 400, "4-byte"), (A16, A2, 400, "4-byte"),
                                                       (A16, None, -4, "weight_stride")])
def test_weight_rejects(lib, weight, prev, stride, needle):
    assert lib.ragged_attn_weight(_problem(v=None), prev, weight, stride, None) == BAD
    assert needle in rv.ragged_last_error()


EVICTS = [
    (dict(B=-1), BAD, "negative"), (dict(B=70000), UNSUPPORTED, "65535"), (dict(H=0), BAD, "H ="), (dict(max_seqlen=0), BAD, "max_seqlen"),
    (dict(max_seqlen=16385), BAD, "max_seqlen"), (dict(sinks=-1), BAD, "sinks"), (dict(recents=-1), BAD, "recents"), (dict(capacity=-1), BAD, "capacity"),
    (dict(capacity=1 << 31), BAD, "capacity"), (dict(cu_out=None), BAD, "cu_out"), (dict(weight=None), BAD, "NULL"), (dict(cu=None), BAD, "NULL"),
    (dict(budget=None), BAD, "NULL"), (dict(src=None), BAD, "NULL"), (dict(rows=None), BAD, "rows_out"), (dict(rows_out=None), BAD, "rows_out"),
    (dict(row_bytes=24), BAD, "multiple of 16"), (dict(row_bytes=0), BAD, "multiple of 16"), (dict(rows=A8), BAD, "16-byte"),
    (dict(rows=3 * A16), BAD, "rows_out must not be rows"), (dict(weight=A2), BAD, "4-byte"), (dict(pos=A2), BAD, "4-byte"),
    (dict(weight_out=A16), BAD, "the outputs"), (dict(cu_out=A16), BAD, "the outputs"), (dict(pos=5 * A16), BAD, "the outputs"),
    (dict(weight_out_stride=100), BAD, "stride"), (dict(weight_stride=-1), BAD, "stride"), (dict(tokens=-1), BAD, "tokens"),
    (dict(max_seqlen=1025, ws=None), BAD, "workspace"), (dict(max_seqlen=1025, ws_bytes=1596), BAD, "workspace"),
    (dict(max_seqlen=1025, ws=A8), BAD, "workspace"),
]


@pytest.mark.parametrize("kw,status,needle", EVICTS, ids=[str(p[0]) for p in EVICTS])
def test_evict_rejects(lib, kw, status, needle):
    a = dict(rows=A16, row_bytes=768, weight=A16, weight_stride=400, H=6, tokens=400, ws=A16, ws_bytes=1600, cu=A16, B=2, max_seqlen=197, budget=A16, sinks=1, recents=0, pos=None,
             capacity=400, rows_out=3 * A16, cu_out=2 * A16, src=2 * A16, weight_out=4 * A16, weight_out_stride=400, pos_out=5 * A16)
    a.update(kw)
    assert lib.ragged_evict(a["rows"], a["row_bytes"], a["weight"], a["weight_stride"], a["H"], a["tokens"], a["cu"], a["B"], a["max_seqlen"], a["budget"],
                            a["sinks"], a["recents"], a["pos"], a["capacity"], a["rows_out"], a["cu_out"], a["src"], a["weight_out"],
                            a["weight_out_stride"], a["pos_out"], a["ws"], a["ws_bytes"], None) == status
    assert needle in rv.ragged_last_error()


@pytest.mark.parametrize("nb,D,both", [(32, 128, True), (32, 128, False), (64, 1024, True), (50, 200, True), (7, 20, False), (4, 1000, True)])
def test_bucket_map(nb, D, both):
    """Against the formula in exact fractions: bucket e + k holds the distances with (d / e)^m in [(D / e)^k, (D / e)^(k + 1))."""
    n = nb // 2 if both else nb
    e = n // 2
    m = n - e
    got = rv.ragged_rel_buckets(nb, D, both, device="cpu").tolist()
    for delta in range(-D, D + 1):
        d = abs(delta) if both or delta < 0 else 0
        b = got[delta + D] - (n if both and delta > 0 else 0)
        if d < e:
            assert b == d
        elif b < n - 1:
            assert Fraction(D, e) ** (b - e) <= Fraction(d, e) ** m < Fraction(D, e) ** (b - e + 1)
        else:
            assert b == n - 1 and Fraction(D, e) ** (b - e) <= Fraction(d, e) ** m


def test_small_bucket_maps():
    assert rv.ragged_rel_buckets(1, 3, False, device="cpu").tolist() == [0] * 7
    assert rv.ragged_rel_buckets(2, 2, True, device="cpu").tolist() == [0, 0, 0, 1, 1]
    assert rv.ragged_rel_buckets(32, 4, True, device="cpu").tolist() == [4, 3, 2, 1, 0, 17, 18, 19, 20]
    for nb, D, both in ((0, 4, False), (65, 4, False), (3, 4, True), (4, -1, True), (4, 1025, True)):
        with pytest.raises(rv.RaggedError):
            rv.ragged_rel_buckets(nb, D, both, device="cpu")


def test_struct_matches_the_header(lib):
    """The fields of struct ragged_bias_attn, in the header's order."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ragged.h")).read()
    body = re.search(r"typedef struct ragged_bias_attn \{(.*?)\} ragged_bias_attn;", text, re.S).group(1)
    names = [n.strip(" *\n") for line in body.split(";") for n in re.sub(r"^\s*(const )?\w+ ", "", line.strip()).split(",") if line.strip()]
    assert names == [n for n, _ in rv.BiasAttn._fields_]


def _tensors(**kw):
    """Arguments of ragged_attn_bias_fwd on the CPU: every check before the device's passes."""
    h = torch.float16
    a = dict(q=torch.zeros(8, 4, 64, dtype=h), k=torch.zeros(8, 2, 64, dtype=h), v=torch.zeros(8, 2, 64, dtype=h),
             cu_seqlens_q=torch.zeros(3, dtype=torch.int32), cu_seqlens_k=torch.zeros(3, dtype=torch.int32), max_seqlen_q=8, max_seqlen_k=8,
             table=torch.zeros(4, 4, dtype=h), buckets=torch.zeros(5, dtype=torch.int32))
    a.update(kw)
    return a


I32, F16 = torch.int32, torch.float16
REFUSED = [
    (dict(), "current CUDA device"), (dict(q=torch.zeros(8, 4, 32, dtype=F16)), "head_dim"), (dict(q=torch.zeros(8, 4, dtype=F16)), "Tq, H"),
    (dict(k=torch.zeros(8, 2, 64, dtype=torch.bfloat16)), "one dtype"), (dict(table=torch.zeros(4, 4)), "one dtype"),
    (dict(v=torch.zeros(9, 2, 64, dtype=F16)), "one dtype"), (dict(v=torch.zeros(2, 8, 64, dtype=F16).transpose(0, 1)), "strides"),
    (dict(q=torch.zeros(8, 64, 4, dtype=F16).transpose(1, 2)), "innermost"), (dict(table=torch.zeros(4, 3, dtype=F16)), "num_buckets"),
    (dict(table=torch.zeros(4, 4, dtype=F16).t()), "contiguous"), (dict(cu_seqlens_q=torch.zeros(3)), "int32"),
    (dict(cu_seqlens_k=torch.zeros(4, dtype=I32)), "int32"), (dict(cu_seqlens_q=torch.zeros(0, dtype=I32)), "at least one"),
    (dict(buckets=torch.zeros(6, dtype=I32)), "odd"), (dict(buckets=torch.zeros(5)), "int32"), (dict(pos_q=torch.zeros(7, dtype=I32)), "pos_q"),
    (dict(pos_k=torch.zeros(16, dtype=I32)[::2]), "pos_k"), (dict(lse=torch.zeros(4, 7)), "lse"), (dict(lse=torch.zeros(4, 8, dtype=F16)), "lse"),
    (dict(lse=torch.zeros(1, 8).expand(4, 8)), "overlap"), (dict(out=torch.zeros(8, 4, 32, dtype=F16)), "out"),
    (dict(out=torch.zeros(4, 8, 64, dtype=F16).transpose(0, 1)), "contiguous heads"), (dict(out=torch.zeros(1, 4, 64, dtype=F16).expand(8, 4, 64)), "heads"),
]


@pytest.mark.parametrize("kw,needle", REFUSED, ids=[str(n) + "-" + w for n, (_, w) in enumerate(REFUSED)])
def test_attention_refuses_tensors(lib, kw, needle):
    with pytest.raises(ValueError, match=needle):
        rv.ragged_attn_bias_fwd(**_tensors(**kw))


def test_gradient_weight_and_eviction_refuse_tensors(lib):
    a = _tensors(lse=torch.zeros(4, 8))
    rest = {n: a[n] for n in ("cu_seqlens_q", "cu_seqlens_k", "max_seqlen_q", "max_seqlen_k", "table", "buckets", "lse")}
    bwd = dict(rest, dout=a["q"], q=a["q"], k=a["k"], v=a["v"], out=a["q"])
    for kw, needle in ((dict(dout=a["q"][:7]), "dout"), (dict(out=a["k"]), "out"), (dict(lse=torch.zeros(4, 9)), "lse"), (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=needle):
            rv.ragged_attn_bias_bwd(**dict(bwd, **kw))
    other = dict(bwd, out=torch.zeros_like(a["q"]), dout=torch.zeros_like(a["q"]))
    for kw, needle in ((dict(dq=a["q"]), "dq"), (dict(dk=a["v"]), "dk"), (dict(dv=a["k"]), "dv"), (dict(dtable=a["table"]), "dtable"),
                       (dict(dk=torch.zeros_like(a["k"])), "CUDA device")):
        with pytest.raises(ValueError, match=needle):
            rv.ragged_attn_bias_bwd(**dict(other, **kw))
    both = torch.zeros_like(a["k"])
    with pytest.raises(ValueError, match="dk must not share"):
        rv.ragged_attn_bias_bwd(**dict(other, dk=both, dv=both))
    with pytest.raises(ValueError, match="out must not share"):
        rv.ragged_attn_bias_fwd(**_tensors(out=a["q"], q=a["q"]))
    with pytest.raises(ValueError, match="current CUDA device"):
        rv.ragged_attn_weight(q=a["q"], k=a["k"], **rest)
    w, cu, budget = torch.zeros(2, 9), torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32)
    for args, needle in (((None, w.half(), cu, 9, budget), "weight"), ((None, w.t().contiguous().t(), cu, 9, budget), "weight"),
                         ((torch.zeros(8, 8), w, cu, 9, budget), "rows"), ((torch.zeros(9, 16)[:, ::2], w, cu, 9, budget), "rows"),
                         ((None, w, cu.long(), 9, budget), "int32"), ((None, w, cu, 9, budget[:1]), "budget"),
                         ((None, w, cu, 9, budget, 1, 0, torch.zeros(8, dtype=I32)), "pos"), ((None, w, cu, 9, budget), "current CUDA device")):
        with pytest.raises(ValueError, match=needle):
            rv.ragged_evict(*args)
    with pytest.raises(TypeError, match="tensor"):
        rv.ragged_evict(None, w, cu, 9, None)


def test_struct_layout_of_the_binding():
    """ctypes' copy of the struct, which these tests use, has the size that the header's fields give."""
    assert ctypes.sizeof(rv.BiasAttn) == 3 * 8 + 4 * 8 + 2 * 8 + 6 * 8 + 2 * 8 + 2 * 8 + 3 * 8 + 8 + 8
