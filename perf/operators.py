"""Cases of the ragged operators with a learned relative position bias: attention and its gradients, the
attention weight that each token collects, and eviction by it.

Every sequence b holds the rows cu[b] .. cu[b + 1] - 1 of flat buffers, head_dim is 64, and query head h
reads key / value head h // (H / Hkv).  With positions p (where None: keys count 0, 1, ...; queries are
the last ones of their sequence's keys) and buckets of clamped relative distances:

    s[i, j]  = scale q_i k_j + table[buckets[clamp(p_j - p_i, -D, D) + D], h]
    attend     out_i = sum_j softmax_j(s)[i, j] v_j, lse_i = log sum_j exp s[i, j]
    train      attend, and from d out the gradients of q, k, v and table
    score      attend, and weight[h, j] = sum_i exp(s[i, j] - lse_i)
    decode     as score for one or a few new tokens per sequence, added to the weights collected so far
    evict      per sequence the `budget` tokens with the largest sum of weights over the heads stay, in
               their order; the first `sinks` and the last `recents` rank above all others
"""
import math
import random

import torch

own = False

DIM = 64
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases ----------------------------------------------------------------------------------

def listed():
    return [
        # one serving batch of a small pruned image encoder: about half the patches are left
        dict(name="attend_serving", op="attend", B=4, L=197, lo=0.4, hi=0.6, pruned=True, H=6, Hkv=6, nq=0, dtype="f16", nb=32, D=128),
        # a high-resolution pruned batch, lengths spread widely
        dict(name="attend_hires", op="attend", B=64, L=577, lo=0.3, hi=0.7, pruned=True, H=12, Hkv=12, nq=0, dtype="bf16", nb=32, D=128),
        # two long documents through an encoder with shared key / value heads
        dict(name="attend_long", op="attend", B=2, L=8191, lo=0.6, hi=1.0, pruned=False, H=12, Hkv=4, nq=0, dtype="bf16", nb=32, D=128),
        # one new token against a short cache: latency
        dict(name="decode_small", op="decode", B=1, L=577, lo=1.0, hi=1.0, pruned=False, H=12, Hkv=12, nq=1, dtype="f16", nb=32, D=128),
        # a serving step of many sequences with long caches
        dict(name="decode_cache", op="decode", B=32, L=8192, lo=0.5, hi=1.0, pruned=False, H=16, Hkv=4, nq=1, dtype="bf16", nb=32, D=128),
        # caches that were thinned out before (positions with holes), three tokens at once
        dict(name="decode_evicted", op="decode", B=13, L=4001, lo=0.2, hi=0.5, pruned=True, H=6, Hkv=6, nq=3, dtype="f16", nb=64, D=512),
        # the scores that thin out a large batch of pruned images
        dict(name="score_sweep", op="score", B=512, L=197, lo=0.4, hi=0.6, pruned=True, H=6, Hkv=6, nq=0, dtype="f16", nb=32, D=128),
        # fine-tuning steps: a small pruned batch, a high-resolution one, and long texts
        dict(name="train_serving", op="train", B=4, L=197, lo=0.4, hi=1.0, pruned=True, H=6, Hkv=6, nq=0, dtype="f16", nb=32, D=128),
        dict(name="train_hires", op="train", B=64, L=577, lo=0.3, hi=0.7, pruned=True, H=12, Hkv=12, nq=0, dtype="bf16", nb=32, D=128),
        dict(name="train_long", op="train", B=2, L=4099, lo=0.8, hi=1.0, pruned=False, H=8, Hkv=2, nq=0, dtype="f16", nb=32, D=128),
        # thinning out the fused q/k/v rows of a serving batch, and the key / value rows of long caches
        dict(name="evict_serving", op="evict", B=4, L=197, lo=0.4, hi=1.0, pruned=True, H=6, Hkv=6, nq=0, dtype="f16", share=0.5, sinks=1, recents=0),
        dict(name="evict_cache", op="evict", B=32, L=8192, lo=0.5, hi=1.0, pruned=False, H=16, Hkv=4, nq=0, dtype="bf16", share=0.5, sinks=4, recents=64),
    ]


def _cost(c):
    """Score elements of a padded batch (decode: of shared heads, a quarter of a query head's rows each; evict: tokens)."""
    if c["op"] == "evict":
        return c["B"] * c["L"]
    if c["op"] == "decode":
        return c["B"] * c["L"] * c["hi"] * max(c["Hkv"], c["H"] * c["nq"] / 4)
    return c["B"] * c["H"] * (c["L"] * c["hi"]) ** 2


def _fits(c):
    """Whether a drawn case costs no more than the largest listed one of its kind."""
    same = [x for x in listed() if x["op"] == c["op"]]
    return (_cost(c) <= max(map(_cost, same)) and work(c)["bytes"] <= max(work(x)["bytes"] for x in same)
            and (c["op"] != "train" or c["B"] * (c["L"] * c["hi"]) ** 2 * c["nb"] <= 1 << 32))


def draw(rng):
    def log_int(a, b):
        return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 1)))))))

    while True:
        op = rng.choice(["attend", "decode", "score", "train", "evict"])
        longest = {"attend": 8191, "decode": 16384, "score": 4099, "train": 4099, "evict": 16384}[op]
        pruned = rng.random() < 0.5
        lo = rng.uniform(0.05, 0.9)
        Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12])
        c = dict(op=op, B=log_int(1, 512), L=log_int(5, longest), lo=round(lo, 3), hi=round(rng.uniform(lo, 1.0), 3), pruned=pruned,
                 H=Hkv * rng.choice([1, 1, 2, 4]), Hkv=Hkv, nq=rng.choice([1, 1, 2, 3, 5]) if op == "decode" else 0,
                 dtype=rng.choice(["f16", "bf16"]))
        if op == "evict":
            c.update(share=round(rng.uniform(0.05, 1.0), 3), sinks=rng.choice([0, 1, 4]), recents=rng.choice([0, 1, 17, 64]))
        else:
            c.update(nb=rng.choice([2, 8, 16, 32, 50, 64]), D=rng.choice([16, 64, 128, 200, 512]))
        if _fits(c):
            return c


def _lengths(c):
    """Rows of every sequence: the case's own, whatever the seed."""
    r = random.Random("%d %d %g %g" % (c["B"], c["L"], c["lo"], c["hi"]))
    return [max(1, min(c["L"], int(round(r.uniform(c["lo"], c["hi"]) * c["L"])))) for _ in range(c["B"])]


def _query_lengths(c, lens):
    return [min(c["nq"], n) for n in lens] if c["nq"] else lens


def _budgets(c, lens):
    r = random.Random("budget %d %g" % (c["B"], c["share"]))
    return [max(1, int(round(r.uniform(0.8, 1.2) * c["share"] * n))) for n in lens]


# ---- inputs -------------------------------------------------------------------------------------

def _bucket_map(nb, D):
    """Bucket of every relative distance -D .. D: half the buckets for each direction, of these half for single
    distances and the others spaced by the logarithm up to D."""
    n = nb // 2
    exact = n // 2
    out = []
    for delta in range(-D, D + 1):
        d = abs(delta)
        if d < exact or n == 1:
            b = min(d, n - 1)
        elif exact == 0:
            b = n - 1
        else:
            m = n - exact
            k = 0  # the largest k with (D / exact)^k <= (d / exact)^m, in whole numbers
            while k < m and D ** (k + 1) * exact ** m <= d ** m * exact ** (k + 1):
                k += 1
            b = min(n - 1, exact + k)
        out.append(b + (n if delta > 0 else 0))
    return torch.tensor(out, dtype=torch.int32)


def _prefix(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES[c["dtype"]]
    lens = _lengths(c)
    cu = _prefix(lens)
    T, B, H, Hkv = cu[-1], c["B"], c["H"], c["Hkv"]
    s = dict(c, T=T, max_k=max(lens), cu_k=torch.tensor(cu, dtype=torch.int32, device=dev), pos_k=None, pos_q=None)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dt)

    if c["pruned"]:  # survivors among L tokens: the first one, and those with the smallest draws
        r = torch.rand((B, c["L"]), generator=g, device=dev)
        r[:, 0] = -1.0
        cut = torch.sort(r, dim=1).values.gather(1, torch.tensor(lens, device=dev)[:, None] - 1)
        s["pos_k"] = torch.nonzero(r <= cut)[:, 1].to(torch.int32)
    if c["op"] == "evict":
        # sums of probabilities over many queries: most tokens get little, a few get much; the newest have none yet
        w = torch.randn((H, T), generator=g, device=dev).mul_(1.5).exp_()
        at = torch.arange(T, device=dev)
        w[:, at % 61 == 7] = 0.0
        budget = _budgets(c, lens)
        kept = sum(min(n, m) for n, m in zip(lens, budget))
        three = 3 if H == Hkv else 2
        s.update(rows=normal(T, three, Hkv, DIM), weight=w, budget=torch.tensor(budget, dtype=torch.int32, device=dev), kept=kept)
        return s
    if c["nq"]:  # new tokens against a cache: rows of keys and values side by side
        ql = _query_lengths(c, lens)
        cq = _prefix(ql)
        kv = normal(T, 2, Hkv, DIM)
        s.update(q=normal(cq[-1], H, DIM), k=kv[:, 0], v=kv[:, 1], max_q=max(ql), cu_q=torch.tensor(cq, dtype=torch.int32, device=dev))
        s["weight"] = torch.randn((H, T), generator=g, device=dev).exp_()
        if c["pruned"]:  # the new tokens follow the whole sequence
            t = torch.arange(cq[-1], device=dev)
            b = torch.searchsorted(s["cu_q"], t, right=True) - 1
            s["pos_q"] = (c["L"] + t - s["cu_q"][b]).to(torch.int32)
    elif H == Hkv:  # one fused row of q, k and v per token
        qkv = normal(T, 3, H, DIM)
        s.update(q=qkv[:, 0], k=qkv[:, 1], v=qkv[:, 2], max_q=s["max_k"], cu_q=s["cu_k"], pos_q=s["pos_k"])
    else:
        s.update(q=normal(T, H, DIM), k=normal(T, Hkv, DIM), v=normal(T, Hkv, DIM), max_q=s["max_k"], cu_q=s["cu_k"], pos_q=s["pos_k"])
    s["table"] = normal(c["nb"], H, std=0.7)
    s["buckets"] = _bucket_map(c["nb"], c["D"]).to(dev)
    if c["op"] == "train":
        s["dout"] = normal(T, H, DIM)
    return s


# ---- the operators' plain forms -------------------------------------------------------------------

def _padded(cu, longest):
    """Flat row of every (sequence, place), and where there is one."""
    at = cu[:-1, None].long() + torch.arange(longest, device=cu.device)
    there = at < cu[1:, None]
    return torch.where(there, at, 0), there


def _flat(x, cu, T):
    """[B, longest, ...] -> [T, ...]"""
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu, t.to(cu.dtype), right=True) - 1
    return x[b, t - cu[b].long()]


def _scores(s):
    """The padded fp32 operands, bucket of every pair and scores, -inf where a sequence has no such key."""
    iq, there_q = _padded(s["cu_q"], s["max_q"])
    ik, there_k = _padded(s["cu_k"], s["max_k"])
    group = s["H"] // s["Hkv"]
    q = s["q"].float()[iq].transpose(1, 2)
    k = s["k"].float()[ik].transpose(1, 2).repeat_interleave(group, 1)
    v = s["v"].float()[ik].transpose(1, 2).repeat_interleave(group, 1)
    if s["pos_k"] is None:
        pk = torch.arange(s["max_k"], device=q.device).expand(ik.shape)
        lq, lk = s["cu_q"].diff(), s["cu_k"].diff()
        pq = torch.arange(s["max_q"], device=q.device) + (lk - lq)[:, None]
    else:
        pk, pq = s["pos_k"].long()[ik], s["pos_q"].long()[iq]
    bucket = s["buckets"][(pk[:, None, :] - pq[:, :, None]).clamp_(-s["D"], s["D"]).add_(s["D"])].long()
    x = torch.matmul(q, k.transpose(2, 3)).mul_(DIM ** -0.5)
    x.add_(s["table"].float().t().contiguous()[:, bucket].transpose(0, 1))
    x.masked_fill_(~there_k[:, None, None, :], -math.inf)
    return q, k, v, bucket, x, iq, there_q, ik, there_k


def _softmax(x):
    m = x.amax(3, keepdim=True)
    p = torch.exp(x.sub_(m))
    total = p.sum(3, keepdim=True)
    return p.div_(total), (m + total.log())[..., 0]


def _plain_attention(s):
    q, k, v, bucket, x, iq, there_q, ik, there_k = _scores(s)
    p, lse = _softmax(x)
    Tq = s["q"].shape[0]
    out = _flat(torch.matmul(p, v).transpose(1, 2), s["cu_q"], Tq).to(s["q"].dtype)
    lse_flat = _flat(lse.transpose(1, 2), s["cu_q"], Tq).t().contiguous()
    if s["op"] == "attend":
        return {"out": out, "lse": lse_flat}
    if s["op"] in ("score", "decode"):
        p.masked_fill_(~there_q[:, None, :, None], 0.0)
        weight = _flat(p.sum(2, dtype=torch.float64).transpose(1, 2), s["cu_k"], s["T"]).t()
        if s["op"] == "decode":
            weight = weight + s["weight"]
        return {"out": out, "lse": lse_flat, "weight": weight.float().contiguous()}
    do = s["dout"].float()[iq].transpose(1, 2) * there_q[:, None, :, None]
    p.mul_(there_q[:, None, :, None])
    dp = torch.matmul(do, v.transpose(2, 3))
    ds = dp.sub_((dp * p).sum(3, keepdim=True)).mul_(p)
    B, H, Hkv, n = s["B"], s["H"], s["Hkv"], s["nb"]
    dq = torch.matmul(ds, k).mul_(DIM ** -0.5)
    dk = torch.matmul(ds.transpose(2, 3), q).mul_(DIM ** -0.5).view(B, Hkv, H // Hkv, -1, DIM).sum(2)
    dv = torch.matmul(p.transpose(2, 3), do).view(B, Hkv, H // Hkv, -1, DIM).sum(2)
    one_hot = (bucket[..., None] == torch.arange(n, device=q.device)).float()
    dtable = torch.matmul(ds.transpose(1, 2), one_hot).sum((0, 1), dtype=torch.float64).t().contiguous()
    dt = s["q"].dtype
    return {"out": out, "lse": lse_flat, "dq": _flat(dq.transpose(1, 2), s["cu_q"], Tq).to(dt),
            "dk": _flat(dk.transpose(1, 2), s["cu_k"], s["T"]).to(dt),
            "dv": _flat(dv.transpose(1, 2), s["cu_k"], s["T"]).to(dt), "dtable": dtable.to(s["table"].dtype)}


def _plain_evict(s):
    cu, T, L = s["cu_k"], s["T"], s["max_k"]
    at, there = _padded(cu, L)
    lens = cu.diff()
    total = s["weight"].sum(0, dtype=torch.float64).float()[at]
    place = torch.arange(L, device=cu.device)
    fixed = (place < s["sinks"]) | (place >= (lens - s["recents"])[:, None])
    total = torch.where(fixed, math.inf, total).masked_fill(~there, -math.inf)
    rank = total.sort(dim=1, descending=True, stable=True).indices.sort(1).indices  # place of each token in that order
    keep = _flat((rank < s["budget"].long()[:, None]) & there, cu, T)
    src = torch.sort((~keep).to(torch.uint8), stable=True).indices[:s["kept"]]
    cu_out = torch.zeros_like(cu)
    cu_out[1:] = torch.minimum(lens, s["budget"]).cumsum(0)
    pos = torch.arange(T, device=cu.device, dtype=torch.int32) - cu[torch.searchsorted(cu, torch.arange(T, device=cu.device, dtype=torch.int32), right=True) - 1] \
        if s["pos_k"] is None else s["pos_k"]
    return {"rows": s["rows"][src], "cu": cu_out, "src": src.to(torch.int32), "weight": s["weight"][:, src], "pos": pos[src]}


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    if not own:
        return _plain_evict(s) if s["op"] == "evict" else _plain_attention(s)
    import ragged_variable_length_b200 as rv

    def places(p, rows):  # two equal draws at a sequence's cut leave a place too many; the calls take one per row
        return p if p is None or p.shape[0] == rows else p[:rows]

    pos_k = places(s["pos_k"], s["T"])
    if s["op"] == "evict":
        rows, cu, src, weight, pos = rv.ragged_evict(s["rows"], s["weight"], s["cu_k"], s["max_k"], s["budget"], sinks=s["sinks"],
                                                     recents=s["recents"], pos=pos_k, total=s["kept"])
        return {"rows": rows, "cu": cu, "src": src, "weight": weight, "pos": pos}
    where = dict(pos_q=places(s["pos_q"], s["q"].shape[0]), pos_k=pos_k)
    seq = (s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], s["table"], s["buckets"])
    out, lse = rv.ragged_attn_bias_fwd(s["q"], s["k"], s["v"], *seq, **where)
    if s["op"] == "attend":
        return {"out": out, "lse": lse}
    if s["op"] in ("score", "decode"):
        weight = rv.ragged_attn_weight(s["q"], s["k"], lse, *seq, **where, prev=s["weight"] if s["op"] == "decode" else None)
        return {"out": out, "lse": lse, "weight": weight}
    dq, dk, dv, dtable = rv.ragged_attn_bias_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, *seq, **where)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}


def work(case):
    c, e = case, 2
    lens = _lengths(c)
    T, H, Hkv = sum(lens), c["H"], c["Hkv"]
    if c["op"] == "evict":
        kept = sum(min(n, m) for n, m in zip(lens, _budgets(c, lens)))
        row = (3 if H == Hkv else 2) * Hkv * DIM * e
        # the weights of all tokens; rows, weights, positions of the kept ones, read and written
        return {"bytes": 4 * H * T + kept * (2 * row + 4 * H + 4 + 4 + (4 if c["pruned"] else 0)) + 12 * c["B"], "flops": H * T}
    ql = _query_lengths(c, lens)
    Tq, pairs = sum(ql), H * sum(a * b for a, b in zip(ql, lens))
    small = 4 * (2 * c["D"] + 1) + e * c["nb"] * H + 8 * (c["B"] + 1) + (4 * (T + Tq) if c["pruned"] else 0)
    b = e * DIM * (2 * Tq * H + 2 * T * Hkv) + 4 * H * Tq + small
    f = 4 * DIM * pairs
    if c["op"] in ("score", "decode"):
        b += 4 * H * T * (2 if c["op"] == "decode" else 1)
        f += 2 * DIM * pairs
    if c["op"] == "train":  # d out in, three gradients out, and the table's
        b += e * DIM * (2 * Tq * H + 2 * T * Hkv) + e * c["nb"] * H
        f += 10 * DIM * pairs
    return {"bytes": b, "flops": f}


# ---- from the definition, in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    cu = s["cu_k"].tolist()
    if s["op"] == "evict":
        total = s["weight"].double().sum(0).float().tolist()
        budget, src, bounds = s["budget"].tolist(), [], [0]
        for b, (a, z) in enumerate(zip(cu, cu[1:])):
            def place(t):
                first = t - a < s["sinks"] or z - t <= s["recents"]
                return (0 if first else 1, 0.0 if first else -total[t], t)
            src += sorted(sorted(range(a, z), key=place)[:budget[b]])
            bounds.append(len(src))
        src = torch.tensor(src, device="cuda")
        return {"rows": s["rows"][src].double(), "cu": None, "src": None, "weight": s["weight"][:, src].double(), "pos": None}
    cq, D, H, group = s["cu_q"].tolist(), s["D"], s["H"], s["H"] // s["Hkv"]
    q, k, v, table = (s[n].double() for n in ("q", "k", "v", "table"))
    out, lse = torch.zeros_like(q), torch.zeros((H, q.shape[0]), dtype=torch.float64, device="cuda")
    weight = torch.zeros((H, s["T"]), dtype=torch.float64, device="cuda")
    if s["op"] == "decode":
        weight += s["weight"].double()
    if s["op"] == "train":
        do, dq, dk, dv = s["dout"].double(), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dtable = torch.zeros_like(table)
    for b in range(s["B"]):
        i, j = slice(cq[b], cq[b + 1]), slice(cu[b], cu[b + 1])
        nq, nk = cq[b + 1] - cq[b], cu[b + 1] - cu[b]
        pk = torch.arange(nk, device="cuda") if s["pos_k"] is None else s["pos_k"][j].long()
        pq = torch.arange(nk - nq, nk, device="cuda") if s["pos_q"] is None else s["pos_q"][i].long()
        far = pk[None, :] - pq[:, None]
        far = torch.where(far > D, D, torch.where(far < -D, -D, far)) + D
        bucket = s["buckets"].long()[far]
        for h in range(H):
            z = h // group
            x = q[i, h] @ k[j, z].T / math.sqrt(DIM) + table[bucket, h]
            lse[h, i] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[h, i][:, None])
            out[i, h] = p @ v[j, z]
            weight[h, j] += p.sum(0)
            if s["op"] == "train":
                dp = do[i, h] @ v[j, z].T
                ds = p * (dp - (do[i, h] * out[i, h]).sum(1, keepdim=True))
                dq[i, h] = ds @ k[j, z] / math.sqrt(DIM)
                dk[j, z] += ds.T @ q[i, h] / math.sqrt(DIM)
                dv[j, z] += p.T @ do[i, h]
                dtable[:, h] += torch.bincount(bucket.reshape(-1), weights=ds.reshape(-1), minlength=s["nb"])
    if s["op"] == "attend":
        return {"out": out, "lse": lse}
    if s["op"] in ("score", "decode"):
        return {"out": out, "lse": lse, "weight": weight}
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}
