"""Attention with a learned relative position bias on the GPU, against its definition in 64 bits."""
import pytest
import torch

import bias_reference as ref
import ragged_variable_length_b200 as rv

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def run_all(s, want=("out", "lse", "weight", "grad")):
    q, k, v, args, where = ref.on_gpu(s)
    Tq, H, d = q.shape
    nan = lambda *shape, dt=q.dtype: torch.full(shape, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    out, lse = nan(Tq, H, d), nan(H, Tq, dt=torch.float32)
    rv.ragged_attn_bias_fwd(q, k, v, *args, **where, out=out, lse=lse)
    r = {"out": out, "lse": lse}
    if "weight" in want:
        r["weight"] = rv.ragged_attn_weight(q, k, lse, *args, **where, weight=nan(H, k.shape[0], dt=torch.float32))
    if "grad" in want:
        grads = dict(dq=nan(Tq, H, d), dk=nan(*k.shape), dv=nan(*k.shape), dtable=nan(*s["table"].shape))
        rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *args, **where, **grads)
        r.update(grads)
    torch.cuda.synchronize()
    assert rv.ragged_get_device_status() == 0
    return r


def compare(s, r):
    good = ref.attention(s, s["dout"] if "dq" in r else None)
    nq, nk = s["cu_q"][-1], s["cu_k"][-1]
    for name, got in r.items():
        want, bound = good[name]
        rows = {"out": slice(0, nq), "dq": slice(0, nq), "dk": slice(0, nk), "dv": slice(0, nk),
                "lse": (slice(None), slice(0, nq)), "weight": (slice(None), slice(0, nk)), "dtable": slice(None)}[name]
        ref.check(name, got, want, bound, rows)
        if name != "dtable":   # rows past the last sequence stay as they were
            past = got[:, (nq if name == "lse" else nk):] if name in ("lse", "weight") else got[(nq if name in ("out", "dq") else nk):]
            assert torch.isnan(past).all(), f"{name}: a row past the last sequence was written"


LENGTHS = [[1], [2, 1, 3], [0, 5, 0], [15, 16, 17, 33], [63, 64, 65], [127, 128, 129], [1, 300, 0, 17], [577], [191, 257, 40]]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_self_attention(lens, dtype):
    s = ref.problem(lens, lens, 2, 2, dtype, 32, 128, seed=len(lens))
    compare(s, run_all(s))


@pytest.mark.parametrize("where", ["none", "sorted", "shuffled", "far", "equal"])
@pytest.mark.parametrize("nb,D", [(1, 0), (2, 1), (8, 3), (32, 128), (50, 200), (64, 1024), (5, 16)])
def test_buckets_and_positions(where, nb, D):
    s = ref.problem([70, 200, 3], [70, 200, 3], 2, 1, F16 if nb % 4 else BF16, nb, D, where=where, seed=nb)
    compare(s, run_all(s))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (4, 2), (6, 1), (8, 2)])
@pytest.mark.parametrize("layout", ["fused", "rows", "heads"])
def test_head_layouts(H, Hkv, layout):
    lens = [37, 130, 64]
    s = ref.problem(lens, lens, H, Hkv, BF16, 32, 64, where="sorted", layout=layout, seed=H)
    compare(s, run_all(s))


@pytest.mark.parametrize("lens_q,lens_k", [([1], [1]), ([1, 1, 1], [577, 1, 64]), ([1, 2, 3], [5, 200, 1000]), ([1] * 9, [4097] + [33] * 8),
                                           ([0, 1, 4], [7, 0, 9]), ([8, 5], [300, 20]), ([3, 140], [1, 20]), ([20, 1], [129, 700])], ids=str)
@pytest.mark.parametrize("H,Hkv,dtype", [(2, 2, F16), (8, 2, BF16), (16, 1, F16), (5, 5, BF16)])
@pytest.mark.parametrize("where", ["none", "sorted"])
def test_queries_against_a_longer_cache(lens_q, lens_k, H, Hkv, dtype, where):
    s = ref.problem(lens_q, lens_k, H, Hkv, dtype, 32, 128, where=where, layout="rows", seed=7)
    compare(s, run_all(s))


@pytest.mark.parametrize("where", ["none", "sorted", "shuffled", "far", "equal"])
@pytest.mark.parametrize("H,Hkv,D,nb", [(2, 2, 1024, 32), (4, 1, 16, 50), (3, 3, 0, 1), (2, 1, 200, 64)])
@pytest.mark.parametrize("lens_q,lens_k", [([7, 3, 12], [7, 3, 12]), ([2, 8, 1, 0], [128, 16, 3, 5])], ids=str)
def test_short_sequences(lens_q, lens_k, H, Hkv, D, nb, where):
    s = ref.problem(lens_q, lens_k, H, Hkv, F16 if nb % 4 else BF16, nb, D, where=where, layout="rows", seed=D)
    compare(s, run_all(s))


@pytest.mark.parametrize("where", ["none", "sorted", "shuffled", "far"])
@pytest.mark.parametrize("H,Hkv,D,nb,longest", [(2, 2, 128, 32, 8), (8, 2, 1024, 64, 8), (2, 2, 16, 50, 30), (4, 2, 200, 7, 1)])
def test_many_short_sequences(H, Hkv, D, nb, longest, where):
    """More groups than the GPU has room for at a time: a few queries against up to 100 keys each, some without either."""
    lens_q = [(7 * i) % (longest + 1) for i in range(170)]
    lens_k = [(n + 37 * i) % 101 if i % 3 else n for i, n in enumerate(lens_q)]
    s = ref.problem(lens_q, lens_k, H, Hkv, F16 if nb % 4 else BF16, nb, D, where=where, layout="rows", seed=D)
    compare(s, run_all(s, want=("out", "lse", "weight")))


@pytest.mark.parametrize("H,Hkv,dtype", [(300, 300, F16), (300, 100, BF16)])
def test_many_heads(H, Hkv, dtype):
    """More heads than a CTA walks over."""
    lens = [3, 40, 0, 130]
    s = ref.problem(lens, lens, H, Hkv, dtype, 32, 128, where="sorted", layout="rows")
    compare(s, run_all(s))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_long_sequence(dtype):
    s = ref.problem([2049, 100], [2049, 100], 1, 1, dtype, 32, 128)
    compare(s, run_all(s))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("entry", [float("-inf"), "lowest", "highest"])
def test_extreme_bias(dtype, entry):
    """A bucket that masks its pairs; where it is a row's only one, -inf leaves the row empty and the lowest value does not."""
    s = ref.problem([40, 200], [40, 200], 2, 2, dtype, 32, 128, seed=3)
    value = {"lowest": torch.finfo(dtype).min, "highest": torch.finfo(dtype).max}.get(entry, entry)
    if value > 0:
        value = 300.0
    s["table"][0] = value          # the token itself
    s["table"][17:] = value        # keys after the query: the last row keeps only earlier ones
    r = run_all(s)
    good = ref.attention(s)
    # scores this far from 0 carry the fp32 step of their size into the exponent
    step = 2.0 ** -23 * 1.4427 * 600 if value == 300.0 else 0.0
    nq = s["cu_q"][-1]
    first = torch.tensor(s["cu_q"][:-1])   # the first row of a sequence sees only masked keys
    rows = torch.ones(nq, dtype=torch.bool)
    if value == float("-inf"):
        assert (r["out"][first.cuda()] == 0).all() and (r["lse"][:, first.cuda()] == -torch.inf).all()
        assert (r["dq"][first.cuda()] == 0).all()
    elif entry == "lowest":
        rows[first] = False
        assert torch.isfinite(r["out"][:nq]).all()
    out, bound = good["out"]
    ref.check("out", r["out"][:nq], out[:nq], bound[:nq] + step * s["v"][:nq].double().abs().max(), rows)
    for name in ("dq", "dk", "dv"):
        assert torch.isfinite(r[name][:nq]).all(), name


def test_lowest_value_everywhere_is_no_mask():
    """Every score at the type's lowest value: the plain softmax over equal scores."""
    s = ref.problem([50], [50], 1, 1, BF16, 32, 128)
    s["table"][:] = torch.finfo(BF16).min
    r = run_all(s, want=())
    mean = s["v"][:50].double().mean(0)
    ref.check("out", r["out"][:50], mean.expand(50, 1, 64), (2.0 ** -7 * s["v"][:50].double().abs().mean(0)).expand(50, 1, 64))


def test_nan_and_infinity_stay_in_their_sequence():
    """The last tile of a sequence ends where the next one's NaN rows begin."""
    lens = [37, 20, 130]
    s = ref.problem(lens, lens, 2, 2, F16, 32, 128)
    for bad in (float("nan"), float("inf")):
        s["base"]["qkv"][37:57] = bad
        r = run_all(s)
        keep = [0, 2]
        good = ref.attention(s, s["dout"])
        for b in keep:
            rows = slice(s["cu_q"][b], s["cu_q"][b + 1])
            for name in ("out", "dq", "dk", "dv"):
                ref.check(name, r[name][rows], good[name][0][rows], good[name][1][rows])
            for name in ("lse", "weight"):
                ref.check(name, r[name][:, rows], good[name][0][:, rows], good[name][1][:, rows])
        assert torch.isnan(r["out"][37:57]).all()


@pytest.mark.parametrize("size", [2.0 ** -12, 1.0, 2.0 ** 10])
def test_gradient_scale(size):
    """f16 gradients far below and above 1 keep their precision (loss scaling moves them by powers of two)."""
    lens = [700, 129]
    s = ref.problem(lens, lens, 1, 1, F16, 32, 128, where="sorted")
    s["dout"] = (s["dout"].float() * size).half()
    compare(s, run_all(s))


@pytest.mark.parametrize("v_size,do_size", [(2.0 ** 7, 1.0), (2.0 ** 12, 2.0 ** -12), (2.0 ** 12, 2.0 ** -4), (2.0 ** -8, 1.0), (2.0 ** -4, 2.0 ** 8)])
@pytest.mark.parametrize("H,Hkv,lens", [(1, 1, [700, 129]), (4, 2, [33, 1, 300])])
def test_value_scale(v_size, do_size, H, Hkv, lens):
    """f16: large values must not push a product's operand past 65504, nor small ones lose it."""
    s = ref.problem(lens, lens, H, Hkv, F16, 32, 128, where="sorted", layout="rows")
    s["v"].mul_(v_size)
    s["dout"] = (s["dout"].float() * do_size).half()
    compare(s, run_all(s))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens_q,where", [([37, 20, 65], "none"), ([37, 20, 65], "sorted"), ([1, 5, 2], "none"), ([1, 5, 2], "sorted")])
def test_table_entry_that_no_pair_uses(dtype, bad, lens_q, where):
    """A tile's places without a column must not see it."""
    s = ref.problem(lens_q, [37, 20, 65], 2, 1, dtype, 64, 1024, where=where, layout="rows")
    used = torch.cat([ref.scores(s, b, 0)[1].flatten() for b in range(3)]).unique()
    unused = torch.ones(64, dtype=torch.bool)
    unused[used] = False
    assert unused.sum() > 10
    s["table"][unused] = bad
    good = dict(s, table=torch.where(unused[:, None], torch.zeros_like(s["table"]), s["table"]))
    compare(good, run_all(s))


def test_gradients_against_differences():
    """d sum(out dout) / dx by central differences of the definition, at random elements of every input."""
    lens = [9, 21]
    s = ref.problem(lens, lens, 2, 1, BF16, 8, 16, where="sorted", extra=0, layout="rows")
    r = run_all(s, want=("grad",))
    s64 = {n: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t) for n, t in s.items()}

    def loss():
        total = 0.0
        for b in range(2):
            for h in range(2):
                x, _, i, j, z = ref.scores(s64, b, h)
                total += ((torch.softmax(x, 1) @ s64["v"][j, z]) * s64["dout"][i, h]).sum().item()
        return total

    g = torch.Generator().manual_seed(1)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("table", "dtable")):
        scale = r[grad].double().abs().max().item()
        for _ in range(6):
            at = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in s64[name].shape)
            old = s64[name][at].item()
            vals = []
            for sign in (1, -1):
                s64[name][at] = old + sign * 1e-5
                vals.append(loss())
            s64[name][at] = old
            assert abs((vals[0] - vals[1]) / 2e-5 - r[grad][at].item()) <= 2.0 ** -6 * scale, (name, at)


def test_same_bits_every_time():
    s = ref.problem([300, 77, 129], [300, 77, 129], 4, 2, BF16, 32, 128, where="sorted")
    a, b = run_all(s), run_all(s)
    for name in a:
        assert torch.equal(a[name].view(torch.int16 if a[name].element_size() == 2 else torch.int32),
                           b[name].view(torch.int16 if b[name].element_size() == 2 else torch.int32)), name


def test_broadcast_and_strided_gradients():
    """dout as autograd hands it over: one value expanded over everything, and a transposed one."""
    lens = [30, 45]
    s = ref.problem(lens, lens, 2, 2, F16, 32, 128, extra=0)
    q, k, v, args, where = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    one = torch.ones((), dtype=F16, device="cuda").expand(75, 2, 64)
    r = dict(zip(("dq", "dk", "dv", "dtable"), rv.ragged_attn_bias_bwd(one, q, k, v, out, lse, *args)))
    s["dout"] = one.cpu().contiguous()
    good = ref.attention(s, s["dout"])
    for name in r:
        ref.check(name, r[name], *good[name])
    fused = torch.full((75, 3, 2, 64), float("nan"), dtype=F16, device="cuda")
    rv.ragged_attn_bias_bwd(one.contiguous().transpose(0, 1).contiguous().transpose(0, 1), q, k, v, out, lse, *args,
                            dq=fused[:, 0], dk=fused[:, 1], dv=fused[:, 2])
    for n, name in enumerate(("dq", "dk", "dv")):
        assert torch.equal(fused[:, n], r[name])


def test_weights_add_up_in_place_and_apart():
    s = ref.problem([1, 2], [100, 300], 4, 2, F16, 32, 128, layout="rows", extra=0)
    q, k, v, args, where = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    prev = torch.rand(4, 400, device="cuda")
    before = prev.clone()
    w = rv.ragged_attn_weight(q, k, lse, *args)
    apart = rv.ragged_attn_weight(q, k, lse, *args, prev=prev)
    assert torch.equal(prev, before)
    assert torch.equal(apart, before + w)
    rv.ragged_attn_weight(q, k, lse, *args, prev=prev, weight=prev)
    assert torch.equal(prev, apart)


def test_on_another_stream_and_in_a_graph():
    lens = [200, 64, 31]
    s = ref.problem(lens, lens, 4, 4, BF16, 32, 128, where="sorted", extra=0)
    q, k, v, args, where = ref.on_gpu(s)
    dout = s["dout"].cuda()

    def step(stream=None):
        out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args, **where, stream=stream)
        w = rv.ragged_attn_weight(q, k, lse, *args, **where, stream=stream)
        return (out, lse, w, *rv.ragged_attn_bias_bwd(dout, q, k, v, out, lse, *args, **where, stream=stream))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = step(stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    graphs, outputs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outputs.append(step())
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for got in outputs:
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_bad_lengths_and_buckets_are_flagged():
    lens = [40, 50, 60]
    s = ref.problem(lens, lens, 2, 2, F16, 32, 128, extra=0)
    q, k, v, args, where = ref.on_gpu(s)
    rv.ragged_get_device_status()
    short = (args[0], args[1], 50, 60, *args[4:])   # the third sequence is longer than its bound
    out = torch.full(q.shape, float("nan"), dtype=F16, device="cuda")
    _, lse = rv.ragged_attn_bias_fwd(q, k, v, *short, out=out)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    assert torch.isfinite(out[:90]).all() and torch.isnan(out[90:]).all()
    rv.ragged_attn_weight(q, k, lse, *short)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    grads = dict(dq=torch.full(q.shape, float("nan"), dtype=F16, device="cuda"))
    rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *short, **grads)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    assert torch.isfinite(grads["dq"][:90]).all() and torch.isnan(grads["dq"][90:]).all()
    # buckets outside the table: no bias there
    wild = s["buckets"].clone()
    wild[:128], wild[129:] = 32, -1
    s["table"][0] = 0
    want = ref.problem(lens, lens, 2, 2, F16, 1, 0, extra=0)
    want.update(q=s["q"], k=s["k"], v=s["v"], table=torch.zeros(1, 2, dtype=F16), dout=s["dout"])
    args = (*args[:4], s["table"].cuda(), wild.cuda())
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    dq, dk, dv, dt = rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *args)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_BUCKETS
    good = ref.attention(want, want["dout"])
    for name, got in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, got, *good[name])
    assert (dt[1:] == 0).all()


def test_offsets_past_32_bits():
    """A cache whose last rows lie beyond 2^31 elements (strides of a wide row), read at both ends."""
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    wide = 1 << 20   # elements per token row
    T = 2300
    row = torch.empty((T, wide), dtype=F16, device="cuda")
    lens_k = [T - 40, 40]
    s = ref.problem([3, 2], lens_k, 2, 1, F16, 32, 128, layout="rows", extra=0)
    row[:, 128:256] = s["base"]["kv"].view(T, 128).cuda()
    k, v = (row[:, 128 + 64 * n:192 + 64 * n].unsqueeze(1) for n in (0, 1))
    q, _, _, args, _ = ref.on_gpu(s)
    out, lse = rv.ragged_attn_bias_fwd(q, k, v, *args)
    w = rv.ragged_attn_weight(q, k, lse, *args)
    grads = [row[:, 256 + 64 * n:320 + 64 * n].unsqueeze(1) for n in (0, 1)]
    dq, dk, dv, dt = rv.ragged_attn_bias_bwd(s["dout"].cuda(), q, k, v, out, lse, *args, dk=grads[0], dv=grads[1])
    good = ref.attention(s, s["dout"])
    for name, got in (("out", out), ("lse", lse), ("weight", w), ("dq", dq), ("dk", dk), ("dv", dv), ("dtable", dt)):
        ref.check(name, got, *good[name])


def test_prune_attend_score_evict_attend():
    """The operators as they are used together: survivors of a pruned batch attend with the bias of their old places, the
    weights they collect choose who stays, the kept rows attend again, and one new token follows against the kept cache."""
    B, L, H = 3, 197, 2
    g = torch.Generator().manual_seed(5)
    dense = torch.randn((B, L, 3, H, 64), generator=g).half().cuda()
    keep = (torch.rand((B, L), generator=g) < 0.6).to(torch.uint8).cuda()
    src = torch.empty(B * L, dtype=torch.int32, device="cuda")
    packed, cu = rv.ragged_pack(dense, keep, src_idx=src)
    T = int(cu[-1])
    pos = (src[:T] % L).contiguous()
    packed = packed[:T]
    table = torch.randn((32, H), generator=g).half().cuda()
    buckets = rv.ragged_rel_buckets(32, 128)
    seq = (cu, cu, L, L, table, buckets)
    out, lse = rv.ragged_attn_bias_fwd(packed[:, 0], packed[:, 1], packed[:, 2], *seq, pos_q=pos, pos_k=pos)
    weight = rv.ragged_attn_weight(packed[:, 0], packed[:, 1], lse, *seq, pos_q=pos, pos_k=pos)
    budget = torch.tensor([20, 50, 400], dtype=torch.int32, device="cuda")
    rows, cu2, src2, weight2, pos2 = rv.ragged_evict(packed, weight, cu, L, budget, sinks=1, recents=2, pos=pos)
    n = cu2.cpu().tolist()
    lens = [b - a for a, b in zip(n, n[1:])]
    assert lens == [min(b, c) for b, c in zip([20, 50, 400], (cu[1:] - cu[:-1]).tolist())]
    T2 = n[-1]
    assert torch.equal(rows[:T2], packed[src2[:T2].long()]) and torch.equal(pos2[:T2], pos[src2[:T2].long()])
    s = dict(q=rows[:T2, 0].cpu(), k=rows[:T2, 1].cpu(), v=rows[:T2, 2].cpu(), table=table.cpu(), buckets=buckets.cpu(), D=128,
             group=1, scale=0.125, cu_q=n, cu_k=n, lens_q=lens, lens_k=lens, pos_q=pos2[:T2].cpu(), pos_k=pos2[:T2].cpu())
    got, _ = rv.ragged_attn_bias_fwd(rows[:T2, 0], rows[:T2, 1], rows[:T2, 2], cu2, cu2, L, L, table, buckets,
                                     pos_q=pos2[:T2], pos_k=pos2[:T2])
    ref.check("out", got, *ref.attention(s)["out"])
    # one new token per sequence against the kept rows
    q = torch.randn((B, H, 64), generator=g).half().cuda()
    cq = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    at = torch.full((B,), L, dtype=torch.int32, device="cuda")
    seq = (cq, cu2, 1, L, table, buckets)
    got, lse = rv.ragged_attn_bias_fwd(q, rows[:T2, 1], rows[:T2, 2], *seq, pos_q=at, pos_k=pos2[:T2])
    w = rv.ragged_attn_weight(q, rows[:T2, 1], lse, *seq, pos_q=at, pos_k=pos2[:T2], prev=weight2[:, :T2].contiguous())
    s.update(q=q.cpu(), cu_q=[0, 1, 2, 3], lens_q=[1, 1, 1], pos_q=at.cpu())
    good = ref.attention(s)
    ref.check("out", got, *good["out"])
    ref.check("weight", w - weight2[:, :T2], good["weight"][0], good["weight"][1] + 2.0 ** -22 * w.double().cpu())
    assert rv.ragged_get_device_status() == 0
