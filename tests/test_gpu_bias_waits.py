"""The bounded waits of the gradient kernels count their own work only: the key-row kernel is launched while the query-row
kernel runs, and may come up long before that one ends."""
import ctypes

import pytest
import torch

import ragged_variable_length_b200 as rv
from ragged_variable_length_b200 import build as rbuild

pytestmark = pytest.mark.gpu
PRODUCT_SPIN = 1 << 22
# 64 sleeps of 4 us.  A wait within one kernel is for a tile (some us) or a set-up (some 10 us); the query-row kernel walks over
# 256 tiles here, at more than 2,000 cycles each: over 250 us, in which the other kernel's CTAs wait on the free SMs.
SPIN = 64


@pytest.fixture(scope="module")
def hooks():
    rbuild.build()
    lib = rv.load(rbuild.build_test_hooks())
    lib.ragged_test_set_hooks.argtypes = [ctypes.c_int32, ctypes.c_uint32]
    lib.ragged_test_set_hooks.restype = ctypes.c_int
    yield lib
    lib.ragged_test_set_hooks(0, PRODUCT_SPIN)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_waiting_for_the_kernel_before_is_no_timeout(hooks, dtype):
    T = rv.RAGGED_MAX_TOKENS
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (torch.randn((T, 1, 64), generator=g, device="cuda").to(dtype) for _ in range(4))
    table = torch.randn((32, 1), generator=g, device="cuda").to(dtype)
    cu, buckets = torch.tensor([0, T], dtype=torch.int32, device="cuda"), rv.ragged_rel_buckets(32, 128)
    args = (cu, cu, T, T, table, buckets)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    want = rv.ragged_attn_bias_bwd(do, q, k, v, out, lse, *args)
    p = rv.BiasAttn(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), q_tok_stride=64, q_head_stride=64, kv_tok_stride=64, kv_head_stride=64,
                    cu_seqlens_q=cu.data_ptr(), cu_seqlens_k=cu.data_ptr(), B=1, max_seqlen_q=T, max_seqlen_k=T, H=1, Hkv=1, head_dim=64,
                    table=table.data_ptr(), buckets=buckets.data_ptr(), num_buckets=32, max_distance=128, lse=lse.data_ptr(), lse_stride=T,
                    scale=0.125, dtype=rv.DTYPE_CODES[dtype])
    size = ctypes.c_int64(0)
    assert hooks.ragged_attn_bias_bwd_workspace(p, size) == 0
    ws = torch.zeros(size.value, dtype=torch.uint8, device="cuda")
    got = [torch.empty_like(t) for t in want]
    stream = torch.cuda.current_stream().cuda_stream
    bits = ctypes.c_uint32(0)
    assert hooks.ragged_get_device_status(ctypes.byref(bits), stream) == 0
    assert hooks.ragged_test_set_hooks(0, SPIN) == 0
    try:
        for _ in range(3):
            assert hooks.ragged_attn_bias_bwd(p, out.data_ptr(), 64, do.data_ptr(), 64, got[0].data_ptr(), 64, 64, got[1].data_ptr(), got[2].data_ptr(),
                                              64, 64, got[3].data_ptr(), ws.data_ptr(), size.value, stream) == 0
        torch.cuda.synchronize()
    finally:
        assert hooks.ragged_test_set_hooks(0, PRODUCT_SPIN) == 0
    assert hooks.ragged_get_device_status(ctypes.byref(bits), stream) == 0
    assert bits.value == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
