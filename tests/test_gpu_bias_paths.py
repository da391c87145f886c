"""Paths that only some shapes take: key rows whose queries are split into parts, several heads per CTA over more rows than
one chunk of column offsets (512), and batches of one long sequence among short ones."""
import ctypes

import pytest
import torch

import bias_far as far
import bias_reference as ref
import ragged_variable_length_b200 as rv
from test_gpu_bias_attention import compare, run_all

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def gradient_workspace(s):
    p = rv.BiasAttn(q=1 << 20, k=1 << 20, v=1 << 20, q_tok_stride=64, q_head_stride=64, kv_tok_stride=64, kv_head_stride=64, cu_seqlens_q=1 << 20,
                    cu_seqlens_k=1 << 20, B=len(s["lens_q"]), max_seqlen_q=max(s["lens_q"]), max_seqlen_k=max(s["lens_k"]), H=s["H"], Hkv=s["Hkv"], head_dim=64,
                    table=1 << 20, buckets=1 << 20, num_buckets=s["table"].shape[0], max_distance=s["D"], lse=1 << 20, lse_stride=s["q"].shape[0], scale=0.125,
                    dtype=rv.DTYPE_CODES[s["q"].dtype])
    n = ctypes.c_int64(0)
    assert rv.load().ragged_attn_bias_bwd_workspace(p, n) == 0
    return n.value


def part_bytes(s):
    """One part's sums of dK and dV."""
    return 4 * len(s["lens_k"]) * -(-max(s["lens_k"]) // 128) * 128 * s["Hkv"] * 128


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("where", ["none", "sorted"])
@pytest.mark.parametrize("lens_q,lens_k,H,Hkv", [([2200, 70], [2200, 70], 8, 2), ([1600, 3], [1600, 700], 16, 1), ([1500], [140], 4, 1)], ids=str)
def test_key_rows_in_parts(lens_q, lens_k, H, Hkv, where, dtype):
    """The short sequences have fewer query tiles than there are parts: some parts are empty."""
    s = ref.problem(lens_q, lens_k, H, Hkv, dtype, 32, 128, where=where, layout="rows", seed=H)
    assert gradient_workspace(s) >= 2 * part_bytes(s)
    compare(s, run_all(s))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("Hkv", [96, 48])
@pytest.mark.parametrize("where", ["none", "sorted"])
def test_several_heads_over_several_chunks(Hkv, where, dtype):
    """About twelve row tiles and 96 heads: more than two waves of CTAs with one head each, so each takes two; and 600
    columns, so that the offsets are loaded again for every head."""
    lens = [600, 20, 577]
    s = ref.problem(lens, lens, 96, Hkv, dtype, 32, 128, where=where, layout="rows", seed=Hkv)
    assert gradient_workspace(s) < part_bytes(s) + (64 << 20)   # one part
    compare(s, run_all(s))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 1)])
def test_one_long_sequence_among_short_ones(H, Hkv, dtype):
    lens = [(5 * i) % 9 for i in range(150)]
    lens[40] = 1700
    s = ref.problem(lens, lens, H, Hkv, dtype, 32, 128, where="sorted", layout="rows", seed=H)
    compare(s, run_all(s))


@pytest.mark.parametrize("dtype,value", [(F16, -3.0e4), (BF16, "lowest"), (BF16, 1.0e10)], ids=str)
@pytest.mark.parametrize("pattern", far.PATTERNS)
@pytest.mark.parametrize("lens_q,lens_k,H,Hkv", [([2200, 70], [2200, 70], 8, 2), ([600, 20, 577], [600, 20, 577], 96, 48)], ids=str)
def test_far_scores(monkeypatch, dtype, value, pattern, lens_q, lens_k, H, Hkv):
    """Bias entries far from 0 on these paths."""
    s = far.problem(dtype, value, pattern, lens_q, lens_k, H, Hkv, where="sorted")
    far.check(s, far.definition(monkeypatch, s, s["dout"]), run_all(s))
