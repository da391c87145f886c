"""Results given by the caller that share memory with an input, with one another or with themselves are refused; ones that
only lie between other rows of one buffer are not (they get as far as the refusal of tensors that are not on the GPU)."""
import random

import pytest
import torch

import ragged_variable_length_b200 as rv
from ragged_variable_length_b200 import build as rbuild

F16, I32 = torch.float16, torch.int32
T, H, HKV = 8, 4, 2


@pytest.fixture(scope="module", autouse=True)
def built():
    rbuild.build()


def half(*shape):
    return torch.zeros(shape, dtype=F16)


def arguments(**kw):
    a = dict(q=half(T, H, 64), k=half(T, HKV, 64), v=half(T, HKV, 64), cu_seqlens_q=torch.zeros(3, dtype=I32), cu_seqlens_k=torch.zeros(3, dtype=I32),
             max_seqlen_q=T, max_seqlen_k=T, table=half(4, H), buckets=torch.zeros(5, dtype=I32))
    a.update(kw)
    return a


def refused(call, needle, **kw):
    with pytest.raises(ValueError, match=needle):
        call(**kw)


def forward(**kw):
    return rv.ragged_attn_bias_fwd(**arguments(**kw))


def backward(**kw):
    a = arguments(lse=torch.zeros(H, T), out=half(T, H, 64), dout=half(T, H, 64))
    a.update(kw)
    return rv.ragged_attn_bias_bwd(**a)


def weights(**kw):
    a = arguments(lse=torch.zeros(H, T))
    del a["v"]
    a.update(kw)
    return rv.ragged_attn_weight(**a)


def test_forward():
    shifted = half(T + 1, H, 64)
    refused(forward, "out must not share", q=shifted[:T], out=shifted[1:])
    refused(forward, "out must not share", k=shifted[1:, :HKV], out=shifted[:T], v=shifted[1:, HKV:])
    raw = half(T * H * 64)
    refused(forward, "out must not share", out=raw.view(T, H, 64), lse=raw[64:64 + 2 * H * T].view(torch.float32).view(H, T))
    refused(forward, "lse must not share", q=raw.view(T, H, 64), lse=raw[-2 * H * T:].view(torch.float32).view(H, T))
    refused(forward, "lse must not share", table=raw[100:100 + 4 * H].view(4, H), lse=raw[96:96 + 2 * H * T].view(torch.float32).view(H, T))
    side = half(T, 4, H, 64)
    refused(forward, "current CUDA device", q=side[:, 0], k=side[:, 1, :HKV], v=side[:, 2, HKV:], out=side[:, 3])
    refused(forward, "current CUDA device", q=shifted[:T], out=half(T, H, 64))


def test_gradients():
    both = half(T, 3, 64)
    refused(backward, "dk must not share", dk=both[:, :2], dv=both[:, 1:])
    fused = half(T, H + 2 * HKV, 64)
    apart = dict(dq=fused[:, :H], dk=fused[:, H:H + HKV], dv=fused[:, H + HKV:])
    refused(backward, "current CUDA device", **apart)
    refused(backward, "dq must not share", **dict(apart, dq=fused[:, 1:H + 1]))
    refused(backward, "dq must not share", dq=fused[:, :H], dout=fused[:, 2:2 + H])
    refused(backward, "dq must not overlap itself", dq=half(T * 64 + H * 64).as_strided((T, H, 64), (64, 64, 1)))
    refused(backward, "dk must not overlap itself", dk=half(HKV, 64).expand(T, HKV, 64), dv=half(HKV, 64).expand(T, HKV, 64))
    out = half(T, H, 64)
    refused(backward, "dtable must not share", out=out, dtable=out.view(-1)[64:80].view(4, H))
    dq = half(T, H, 64)
    refused(backward, "dq must not share", dq=dq, dtable=dq.view(-1)[-16:].view(4, H))
    lse = torch.zeros(H, T)
    refused(backward, "dtable must not share", lse=lse, dtable=lse.view(-1).view(F16)[3:19].view(4, H))
    one = torch.zeros((), dtype=F16).expand(T, H, 64)   # an input may repeat itself
    refused(backward, "current CUDA device", dout=one, dq=half(T, H, 64))


def test_weights():
    w = torch.zeros(H, T + 1)
    refused(weights, "weight must not share", prev=w[:, :T], weight=w[:, 1:])
    refused(weights, "current CUDA device", prev=w[:, :T], weight=w[:, :T])
    lse = torch.zeros(H, T)
    refused(weights, "weight must not share", lse=lse, weight=lse)
    wide = torch.zeros(H, 2 * T)
    refused(weights, "current CUDA device", prev=wide[:, :T], weight=wide[:, T:])
    refused(weights, "weight must not share", lse=wide[:, 4:4 + T], weight=wide[:, T:])


@pytest.mark.parametrize("seed", range(8))
def test_against_the_bytes(seed):
    """Random layouts of q and of a gradient in one buffer: refused just where they have an element in common."""
    r = random.Random(seed)
    buffer = half(6000)
    done = {True: 0, False: 0}
    while min(done.values()) < 25:
        n, h = r.randint(1, 4), r.randint(1, 3)
        shapes, views, sets = (n, h, 64), [], []
        for _ in range(2):
            a, b = 64 * r.randint(1, 4) + 8 * r.randint(0, 3), 64 * r.randint(1, 6) + 8 * r.randint(0, 3)
            lo, hi = (a, max(b, (h - 1) * a + 64)) if r.random() < 0.5 else (max(a, (n - 1) * b + 64), b)   # heads within rows, or rows within heads
            t = buffer.as_strided(shapes, (hi, lo, 1), r.randint(0, 2000))
            views.append(t)
            sets.append({t.storage_offset() + i * hi + j * lo + c for i in range(n) for j in range(h) for c in range(64)})
        q, dq = views
        common = bool(sets[0] & sets[1])
        with pytest.raises(ValueError, match="dq must not share" if common else "current CUDA device"):
            rv.ragged_attn_bias_bwd(half(n, h, 64), q, half(n, h, 64), half(n, h, 64), half(n, h, 64), torch.zeros(h, n), torch.zeros(2, dtype=I32),
                                    torch.zeros(2, dtype=I32), n, n, half(4, h), torch.zeros(5, dtype=I32), dq=dq)
        done[common] += 1
