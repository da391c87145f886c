"""Inputs that require a gradient are refused while a graph would be recorded: the results would come out without one."""
import pytest
import torch

import ragged_variable_length_b200 as rv
from ragged_variable_length_b200 import build as rbuild
from test_bias_memory_cpu import H, HKV, I32, T, arguments, half

CALLS = {
    "ragged_attn_bias_fwd": (lambda: arguments(), ("q", "k", "v", "table")),
    "ragged_attn_bias_bwd": (lambda: arguments(lse=torch.zeros(H, T), out=half(T, H, 64), dout=half(T, H, 64)), ("dout", "q", "k", "v", "table", "out", "lse")),
    "ragged_attn_weight": (lambda: {n: t for n, t in arguments(lse=torch.zeros(H, T)).items() if n != "v"}, ("q", "k", "table", "lse")),
    "ragged_evict": (lambda: dict(rows=half(T, HKV, 64), weight=torch.zeros(H, T), cu_seqlens=torch.zeros(3, dtype=I32), max_seqlen=T,
                                  budget=torch.zeros(2, dtype=I32)), ("rows", "weight")),
}


@pytest.mark.parametrize("name,given", [(n, a) for n, (_, names) in CALLS.items() for a in names])
def test_refused(name, given):
    rbuild.build()
    call, args = getattr(rv, name), CALLS[name][0]()
    args[given].requires_grad_()
    with pytest.raises(ValueError, match="records no graph"):
        call(**args)
    with torch.no_grad(), pytest.raises(ValueError, match="current CUDA device"):   # the next refusal
        call(**args)
