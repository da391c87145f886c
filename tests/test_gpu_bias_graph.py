"""The two attention calls in a torch.autograd.Function, as the README has it."""
import os
import re

import pytest
import torch

import bias_reference as ref
import ragged_variable_length_b200 as rv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_autograd_function(dtype):
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    source = re.search(r"^class Attend\(torch\.autograd\.Function\):.*?(?=^\S)", text, re.S | re.M).group(0)
    scope = {"torch": torch, "rv": rv}
    exec(source, scope)
    lens = [70, 5, 33]
    s = ref.problem(lens, lens, 4, 2, dtype, 32, 128, where="sorted", layout="rows", extra=0)
    q, k, v, args, where = ref.on_gpu(s)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v, args[4])]
    out = scope["Attend"].apply(*leaves, args[0], args[2], args[5], where["pos_q"])
    out.backward(s["dout"].cuda())
    good = ref.attention(s, s["dout"])
    ref.check("out", out, *good["out"])
    for leaf, name in zip(leaves, ("dq", "dk", "dv", "dtable")):
        ref.check(name, leaf.grad, *good[name])
