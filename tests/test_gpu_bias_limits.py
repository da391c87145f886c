"""The operators with a position bias and the eviction at their limits on the GPU: the most sequences, calls at the same
time, graphs that replay side by side, bounded waits that expire, row ranges past the buffer."""
import ctypes

import pytest
import torch

import bias_reference as ref
import ragged_variable_length_b200 as rv
from ragged_variable_length_b200 import build as rbuild

pytestmark = pytest.mark.gpu
F16, BF16, I32 = torch.float16, torch.bfloat16, torch.int32


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("longest", [1, 200])
def test_the_most_sequences(longest, dtype):
    """65535 sequences of one token each (one bound says 200, which takes the kernels with 128-row tiles):
    out = v, lse = the score, weight = 1, dv = dout, and no other gradient."""
    n = 65535
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((n, 1, 64), generator=g, device="cuda").to(dtype) for _ in range(4))
    cu = torch.arange(n + 1, dtype=I32, device="cuda")
    table, buckets = torch.tensor([[0.5]], dtype=dtype, device="cuda"), torch.zeros(3, dtype=I32, device="cuda")
    args = (cu, cu, longest, longest, table, buckets)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    assert torch.equal(out, v)
    score = (q.double() * k.double()).sum(2).T * 0.125 + 0.5
    assert ((lse - score).abs() <= 2.0 ** -14 * (1 + score.abs())).all()
    assert ((rv.ragged_attn_weight(q, k, lse, *args) - 1).abs() <= 2.0 ** -14).all()
    dq, dk, dv, dtable = rv.ragged_attn_bias_bwd(do, q, k, v, out, lse, *args)
    # P = 1 + e with |e| <= 2^-14, and dP and delta the same sum in two orders: 64 roundings of 2^-24 each
    size = (do.double() * v.double()).abs().sum(2, keepdim=True)
    u = torch.finfo(dtype).eps / 2
    assert ((dv.double() - do.double()).abs() <= (u + 2.0 ** -14) * (1 + u) * do.double().abs() + u * do.double().abs()).all()
    assert (dq.double().abs() <= 2.0 ** -17 * size * k.double().abs() * 0.125 + 2.0 ** -24).all()
    assert (dk.double().abs() <= 2.0 ** -17 * size * q.double().abs() * 0.125 + 2.0 ** -24).all()
    assert dtable.double().abs().item() <= 2.0 ** -17 * size.sum().item()
    weight = torch.rand((2, n), generator=g, device="cuda")
    budget = (torch.arange(n, device="cuda") % 2).to(I32)
    rows, cu_out, src, _, _ = rv.ragged_evict(v, weight, cu, longest, budget, sinks=0)
    kept = torch.arange(1, n, 2, device="cuda")
    assert cu_out[-1].item() == len(kept) and torch.equal(src[:len(kept)].long(), kept) and torch.equal(rows[:len(kept)], v[kept])
    assert rv.ragged_get_device_status() == 0


def _calls(s):
    q, k, v, args, where = ref.on_gpu(s)
    do = s["dout"].cuda()

    def run():
        out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args, **where)
        weight = rv.ragged_attn_weight(q, k, lse, *args, **where)
        grads = rv.ragged_attn_bias_bwd(do, q, k, v, out, lse, *args, **where)
        kept = rv.ragged_evict(None, weight, args[1], args[3], torch.full((len(s["lens_k"]),), 9, dtype=I32, device="cuda"), total=9 * len(s["lens_k"]))
        return out, lse, weight, *grads, kept[1], kept[2]
    return run


def _same(a, b, rows):
    for x, y in zip(a, b):
        x, y = (t[:, :rows] if t.dim() == 2 and t.dtype == torch.float32 else t[:rows] for t in (x, y))
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_two_calls_and_two_graphs_at_once(dtype):
    """Two problems on two streams, eager and replayed, give the bits that each gives alone."""
    probs = [ref.problem(lens, lens, H, Hkv, dtype, 32, 128, where="sorted", seed=H) for lens, H, Hkv in (([300, 77, 1], 4, 2), ([1500, 640], 2, 2))]
    runs = [_calls(s) for s in probs]
    rows = [s["cu_q"][-1] for s in probs]
    alone = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(runs[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            _same(g, alone[i], rows[i])
    graphs, results = [], []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(r())
        graphs.append(graph)
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        _same(results[i], alone[i], rows[i])
    assert rv.ragged_get_device_status() == 0


def test_eviction_of_rows_past_the_buffer_is_flagged():
    """A sequence whose rows end past the input keeps nothing; the others are not disturbed."""
    for n, last in ((100, 60), (1500, 1200)):   # one launch, and the long form
        w = torch.rand((2, 2 * n + 50), device="cuda")
        rows = torch.randn((2 * n + 50, 8), device="cuda")
        cu = torch.tensor([0, n, 2 * n, 2 * n + last], dtype=I32, device="cuda")
        _, cu_out, src, _, _ = rv.ragged_evict(rows, w, cu, n, torch.full((3,), 7, dtype=I32, device="cuda"))
        assert cu_out.tolist() == [0, 7, 14, 14]
        assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
        want = rv.ragged_evict(rows, w, cu[:3], n, torch.full((2,), 7, dtype=I32, device="cuda"))
        assert torch.equal(src[:14], want[2][:14]) and rv.ragged_get_device_status() == 0


SHORT_SPIN, PRODUCT_SPIN = 1 << 8, 1 << 22


@pytest.fixture(scope="module")
def hooks():
    rbuild.build()
    lib = rv.load(rbuild.build_test_hooks())
    lib.ragged_test_set_hooks.argtypes = [ctypes.c_int32, ctypes.c_uint32]
    lib.ragged_test_set_hooks.restype = ctypes.c_int
    yield lib
    lib.ragged_test_set_hooks(0, PRODUCT_SPIN)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_expired_waits_are_reported_and_the_next_launch_is_exact(hooks, dtype):
    """The load warps issue nothing, so every bounded wait behind them runs out: the launches return, flag it and leave
    the results alone; the next ones take the TMEM that these freed."""
    lens, H = [300, 0, 77, 129], 2
    s = ref.problem(lens, lens, H, H, dtype, 32, 128, extra=0)
    q, k, v, args, _ = ref.on_gpu(s)
    T, do = q.shape[0], s["dout"].cuda()
    want_out, want_lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    want = (want_out, want_lse, rv.ragged_attn_weight(q, k, want_lse, *args), *rv.ragged_attn_bias_bwd(do, q, k, v, want_out, want_lse, *args))
    assert rv.ragged_get_device_status() == 0
    lse = want_lse.clone()
    p = rv.BiasAttn(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), q_tok_stride=q.stride(0), q_head_stride=q.stride(1), kv_tok_stride=k.stride(0),
                    kv_head_stride=k.stride(1), cu_seqlens_q=args[0].data_ptr(), cu_seqlens_k=args[1].data_ptr(), B=len(lens), max_seqlen_q=300,
                    max_seqlen_k=300, H=H, Hkv=H, head_dim=64, table=args[4].data_ptr(), buckets=args[5].data_ptr(), num_buckets=32,
                    max_distance=128, lse=lse.data_ptr(), lse_stride=T, scale=0.125, dtype=rv.DTYPE_CODES[dtype])
    size = ctypes.c_int64(0)
    assert hooks.ragged_attn_bias_bwd_workspace(p, size) == 0
    ws = torch.zeros(size.value, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def status():
        bits = ctypes.c_uint32(0)
        assert hooks.ragged_get_device_status(ctypes.byref(bits), stream) == 0
        return bits.value

    def launches():
        return {"fwd": (lambda o: hooks.ragged_attn_bias_fwd(p, o[0].data_ptr(), H * 64, None, 0, stream), (0,)),
                "weight": (lambda o: hooks.ragged_attn_weight(p, None, o[2].data_ptr(), T, stream), (2,)),
                "bwd": (lambda o: hooks.ragged_attn_bias_bwd(p, want_out.data_ptr(), H * 64, do.data_ptr(), H * 64, o[3].data_ptr(), H * 64, 64,
                                                             o[4].data_ptr(), o[5].data_ptr(), H * 64, 64, o[6].data_ptr(), ws.data_ptr(), size.value,
                                                             stream), (3, 4, 5))}
    status()
    for name, (call, written) in launches().items():
        results = [torch.full_like(t, 3.0, memory_format=torch.contiguous_format) for t in want]
        assert hooks.ragged_test_set_hooks(1, SHORT_SPIN) == 0
        try:
            assert call(results) == 0
            torch.cuda.synchronize()
        finally:
            assert hooks.ragged_test_set_hooks(0, PRODUCT_SPIN) == 0
        assert status() & rv.RAGGED_DEV_TIMEOUT, name
        for i in written:
            assert (results[i] == 3.0).all(), name
        assert torch.equal(lse, want_lse)
        assert call(results) == 0
        torch.cuda.synchronize()
        assert status() == 0
        for i in written + ((6,) if name == "bwd" else ()):
            assert torch.equal(results[i], want[i]), name
