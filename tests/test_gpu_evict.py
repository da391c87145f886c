"""Eviction by collected attention weight on the GPU, bit for bit against its definition."""
import math

import pytest
import torch

import ragged_variable_length_b200 as rv

pytestmark = pytest.mark.gpu


def definition(weight, lens, budget, sinks, recents):
    src, cu, a = [], [0], 0
    total = weight.double().sum(0).float().tolist()
    for n, m in zip(lens, budget):
        def place(t):
            fixed = t - a < sinks or a + n - t <= recents
            x = total[t]
            return (0 if fixed else 1, 0 if fixed else (1 if math.isnan(x) else 0), 0.0 if fixed or math.isnan(x) else -x, t)
        src += sorted(sorted(range(a, a + n), key=place)[:max(0, min(m, n))])
        cu.append(len(src))
        a += n
    return src, cu


def check(weight, lens, budget, sinks=1, recents=0, pos=None, rows=None, total=None, max_seqlen=None):
    T = weight.shape[1]
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    rows = torch.arange(T * 24).view(T, 3, 8).half().cuda() if rows is None else rows
    got = rv.ragged_evict(rows, weight.cuda(), cu, max_seqlen or max(1, *lens), torch.tensor(budget, dtype=torch.int32).cuda(), sinks=sinks,
                          recents=recents, pos=None if pos is None else pos.cuda(), total=total)
    torch.cuda.synchronize()
    src, cu_out = definition(weight, lens, budget, sinks, recents)
    rows_out, cu2, src2, weight2, pos2 = got
    n = len(src) if total is None else min(total, len(src))
    src = torch.tensor(src[:n], dtype=torch.long)
    assert cu2.tolist() == cu_out
    assert torch.equal(src2[:n].long().cpu(), src)
    assert torch.equal(rows_out[:n], rows[src.cuda()])
    assert torch.equal(weight2[:, :n].cpu().view(torch.int32), weight[:, src].contiguous().view(torch.int32))
    place = torch.cat([torch.arange(n) for n in lens]).int() if pos is None else pos
    assert torch.equal(pos2[:n].cpu(), place[src])


@pytest.mark.parametrize("lens", [[1], [5], [0, 3, 0], [31, 32, 33], [197, 1, 64], [1023, 1024, 1025], [5000], [16384, 7]], ids=str)
@pytest.mark.parametrize("sinks,recents", [(0, 0), (1, 0), (4, 64), (3, 16384)])
@pytest.mark.parametrize("H", [1, 6])
def test_lengths(lens, sinks, recents, H):
    g = torch.Generator().manual_seed(sum(lens))
    weight = torch.randn((H, sum(lens)), generator=g).exp()
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (sum(lens),), generator=g).int()
    for budget in ([n // 2 for n in lens], [1] * len(lens), [0] * len(lens), [n for n in lens], [n - 1 for n in lens], [10 ** 9] * len(lens), [-3] * len(lens)):
        check(weight, lens, budget, sinks, recents, pos if budget[0] != 1 else None)


def test_ties_and_special_values():
    g = torch.Generator().manual_seed(2)
    pick = torch.tensor([0.0, -0.0, 1.0, float("nan"), float("inf"), float("-inf"), 1e-45, -1e-45, 3.0e38, -2.5])
    weight = pick[torch.randint(0, 10, (1, 900), generator=g)]
    for budget in (1, 3, 77, 300, 500, 899):
        check(weight, [400, 500], [budget, budget], sinks=0)
    check(torch.zeros(4, 300), [300], [100], sinks=2, recents=5)     # all equal: the lowest indices
    close = torch.full((1, 4096), 1.0)                               # keys that differ in their last bits only
    close[0] += torch.randint(0, 7, (4096,), generator=g) * 2.0 ** -23
    check(close, [4096], [1234], sinks=0)


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 60, (3000,), generator=g).tolist()
    check(torch.rand((3, sum(lens)), generator=g), lens, torch.randint(-1, 40, (3000,), generator=g).tolist(), sinks=1, recents=1)


@pytest.mark.parametrize("row", [8, 24, 64, 1152])
def test_row_widths(row):
    g = torch.Generator().manual_seed(4)
    rows = torch.randn((333, row), generator=g).half().cuda()
    check(torch.rand((2, 333), generator=g), [100, 233], [17, 99], rows=rows)


def test_outputs_of_the_stated_size():
    g = torch.Generator().manual_seed(5)
    weight = torch.rand((2, 300), generator=g)
    check(weight, [100, 200], [30, 60], total=90)
    assert rv.ragged_get_device_status() == 0
    check(weight, [100, 200], [30, 60], total=70)   # too small: what fits is written, and flagged
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_CAPACITY
    check(weight, [100, 200], [30, 60], total=0)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_CAPACITY


def test_selection_alone_and_strided_weights():
    w = torch.rand(4, 512, device="cuda")[:, 100:400]
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    budget = torch.tensor([50], dtype=torch.int32, device="cuda")
    rows, cu2, src, w2, pos = rv.ragged_evict(None, w, cu, 300, budget)
    want, _ = definition(w.cpu(), [300], [50], 1, 0)
    assert rows is None and src[:50].tolist() == want and pos[:50].tolist() == want


def test_a_sequence_longer_than_its_bound_keeps_nothing():
    w = torch.rand(1, 60, device="cuda")
    cu = torch.tensor([0, 20, 50, 60], dtype=torch.int32, device="cuda")
    budget = torch.tensor([5, 5, 5], dtype=torch.int32, device="cuda")
    rv.ragged_get_device_status()
    _, cu2, src, _, _ = rv.ragged_evict(None, w, cu, 20, budget)
    assert rv.ragged_get_device_status() == rv.RAGGED_DEV_BAD_SEQLENS
    assert cu2.tolist() == [0, 5, 5, 10] and (src[:5] < 20).all() and (src[5:10] >= 50).all()


def test_on_another_stream_and_in_a_graph():
    w = torch.rand(6, 700, device="cuda")
    rows = torch.randn(700, 384, device="cuda").half()
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    budget = torch.tensor([100, 150], dtype=torch.int32, device="cuda")
    call = lambda stream=None: rv.ragged_evict(rows, w, cu, 400, budget, total=250, stream=stream)  # noqa: E731
    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    w[:, 0:700:3] += 2.0
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(call(), got))
