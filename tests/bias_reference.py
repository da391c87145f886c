"""Attention with a learned relative position bias, its gradients and collected
weights from the definition, in float64 with torch on the CPU, one sequence and
head at a time; and error bounds of the kernels' results.

The bounds count roundings.  u is half a step of the 16-bit type (eps / 2).
EPS32 covers the fp32 part of a probability: the score's fp32 sum over 64
products (64 * 2^-24 of sum |q k| scale, at most 2^-17 relative to exp for the
|score| <= 16 of these inputs: 64 * 2^-24 * 16 = 2^-14.0 at the very worst,
2^-18 for sums that err at random), ex2.approx (2^-22) and the sums over the
keys.  2^-14 is used.  SUB is the absolute spacing of f16 below 2^-14, where a
rounding is off by 2^-25 instead of u relative; the kernels scale probabilities
to at least 1 at a row's largest before rounding, so it applies to values
relative to that.

  out  : u |out|  (the result)  +  sum_j p_j |v_j| (u + EPS32)  +  n SUB max|v|
  delta: sum_c |do_c| err(out_c) + EPS32 sum_c |do_c out_c|
  dS   : |dS| u + P (err(delta) + EPS32 (|dP| + |delta|)) with |dP| <= sum |do v|
         (f16: dS 2^(14 - e - f) is rounded, 2^e and 2^f at most twice the largest norms of the rows of dO and V,
         so SUB of it is at most SUB 2^-12 max|do| max|v|)
  dq   : u |dq| + scale sum_j err(dS) |k|;  dk, dv alike;  dtable: u |dtable| + sum err(dS) without its rounding
"""
import torch

EPS32 = 2.0 ** -14
SUB = 2.0 ** -25


def prefix(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def positions(s, b):
    nq, nk = s["lens_q"][b], s["lens_k"][b]
    cq, ck = s["cu_q"][b], s["cu_k"][b]
    pk = torch.arange(nk) if s["pos_k"] is None else s["pos_k"][ck:ck + nk].long()
    pq = torch.arange(nk - nq, nk) if s["pos_q"] is None else s["pos_q"][cq:cq + nq].long()
    return pq, pk


def scores(s, b, h):
    """float64 scores of one sequence and head, and the bucket of every pair."""
    i = slice(s["cu_q"][b], s["cu_q"][b + 1])
    j = slice(s["cu_k"][b], s["cu_k"][b + 1])
    pq, pk = positions(s, b)
    D = s["D"]
    bucket = s["buckets"].long()[(pk[None, :] - pq[:, None]).clamp(-D, D) + D]
    z = h // s["group"]
    q, k = s["q"][i, h].double(), s["k"][j, z].double()
    return q @ k.T * s["scale"] + s["table"].double()[bucket, h], bucket, i, j, z


def attention(s, dout=None):
    """Results and their error bounds: {name: (value, bound)}."""
    u = torch.finfo(s["q"].dtype).eps / 2
    sub = SUB if s["q"].dtype == torch.float16 else 0.0
    Tq, H, d = s["q"].shape
    Tk = s["k"].shape[0]
    z64 = lambda *shape: torch.zeros(shape, dtype=torch.float64)  # noqa: E731
    r = {n: (z64(*shape), z64(*shape)) for n, shape in
         dict(out=(Tq, H, d), lse=(H, Tq), weight=(H, Tk), dq=(Tq, H, d), dk=tuple(s["k"].shape),
              dv=tuple(s["k"].shape), dtable=tuple(s["table"].shape)).items()}
    for b in range(len(s["lens_q"])):
        for h in range(H):
            x, bucket, i, j, z = scores(s, b, h)
            n = x.shape[1]
            if x.numel() == 0:   # no keys: an empty row; no queries: nothing
                r["lse"][0][h, i] = -torch.inf
                continue
            lse = torch.logsumexp(x, 1)
            p = torch.where(lse[:, None] == -torch.inf, 0.0, torch.exp(x - lse[:, None]))
            v = s["v"][j, z].double()
            out = p @ v
            eo = u * out.abs() + (u + EPS32) * (p @ v.abs()) + n * sub * v.abs().max()
            r["out"][0][i, h], r["out"][1][i, h] = out, eo
            r["lse"][0][h, i], r["lse"][1][h, i] = lse, EPS32 + 2.0 ** -22 * lse.abs()
            r["weight"][0][h, j], r["weight"][1][h, j] = p.sum(0), EPS32 * p.sum(0)
            if dout is None:
                continue
            q, k, do = s["q"][i, h].double(), s["k"][j, z].double(), dout[i, h].double()
            dp, delta = do @ v.T, (do * out).sum(1, keepdim=True)
            ds = p * (dp - delta)
            ed = (do.abs() * eo).sum(1, keepdim=True) + EPS32 * (do * out).abs().sum(1, keepdim=True)
            es32 = p * (ed + EPS32 * (do.abs() @ v.abs().T + delta.abs()))
            es = es32 + u * ds.abs() + sub * 2.0 ** -12 * do.norm(dim=1).amax() * v.norm(dim=1).amax()
            ep = (u + EPS32) * p + sub * 2.0 ** -14
            r["dq"][0][i, h] = ds @ k * s["scale"]
            r["dq"][1][i, h] = es @ k.abs() * s["scale"]
            r["dk"][0][j, z] += ds.T @ q * s["scale"]
            r["dk"][1][j, z] += es.T @ q.abs() * s["scale"]
            r["dv"][0][j, z] += p.T @ do
            r["dv"][1][j, z] += ep.T @ do.abs()
            ok = bucket.reshape(-1)
            r["dtable"][0][:, h] += torch.bincount(ok, ds.reshape(-1), s["table"].shape[0])
            r["dtable"][1][:, h] += torch.bincount(ok, es32.reshape(-1), s["table"].shape[0])
    for name in ("dq", "dk", "dv", "dtable"):
        value, bound = r[name]
        bound += u * (value.abs() + bound)
        if s["q"].dtype == torch.float16:
            bound += SUB   # a result below f16's normal range
    return r


def problem(lens_q, lens_k, H, Hkv, dtype, nb, D, where="none", layout="fused", seed=0, table_std=1.0, bidirectional=True,
            extra=3):
    """Inputs on the CPU, `extra` rows past the last sequence (NaN, never to be read)."""
    import ragged_variable_length_b200 as rv
    g = torch.Generator().manual_seed(seed)
    cu_q, cu_k = prefix(lens_q), prefix(lens_k)
    Tq, Tk = cu_q[-1] + extra, cu_k[-1] + extra

    def normal(*shape):
        return torch.randn(shape, generator=g).to(dtype)

    if layout == "fused" and H == Hkv and lens_q == lens_k:
        qkv = normal(Tq, 3, H, 64)
        qkv[cu_q[-1]:] = torch.nan
        q, k, v = qkv[:, 0], qkv[:, 1], qkv[:, 2]
        base = {"qkv": qkv}
    elif layout == "heads":   # [heads, tokens, 64] seen as [tokens, heads, 64]
        q, kv = normal(H, Tq, 64).transpose(0, 1), normal(2, Hkv, Tk, 64)
        k, v = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
        q[cu_q[-1]:] = torch.nan
        kv[:, :, cu_k[-1]:] = torch.nan
        base = {"q": q, "kv": kv}
    else:
        q, kv = normal(Tq, H, 64), normal(Tk, 2, Hkv, 64)
        q[cu_q[-1]:] = torch.nan
        kv[cu_k[-1]:] = torch.nan
        k, v = kv[:, 0], kv[:, 1]
        base = {"q": q, "kv": kv}

    def place(lens, cu, T, spread):
        pos = torch.full((T,), -7, dtype=torch.int32)
        for b, n in enumerate(lens):
            p = torch.randperm(max(1, spread * n), generator=g)[:n]
            pos[cu[b]:cu[b] + n] = (p if where == "shuffled" else p.sort().values).int()
        return pos

    if where == "none":
        pos_q = pos_k = None
    elif where == "far":   # differences that only fit an int32
        pos_k = torch.randint(-2 ** 30, 2 ** 30, (Tk,), generator=g).int()
        pos_q = torch.randint(-2 ** 30, 2 ** 30, (Tq,), generator=g).int()
    elif where == "equal":
        pos_k, pos_q = torch.full((Tk,), 11, dtype=torch.int32), torch.full((Tq,), 11, dtype=torch.int32)
    else:
        pos_k = place(lens_k, cu_k, Tk, 2)
        pos_q = pos_k if lens_q == lens_k else place(lens_q, cu_q, Tq, 5)
    return dict(base=base, layout=layout, q=q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, lens_q=lens_q, lens_k=lens_k, pos_q=pos_q,
                pos_k=pos_k, table=(torch.randn((nb, H), generator=g) * table_std).to(dtype),
                buckets=rv.ragged_rel_buckets(nb, D, bidirectional and nb % 2 == 0, device="cpu"), D=D, group=H // Hkv,
                scale=0.125, H=H, Hkv=Hkv, dout=normal(Tq, H, 64))


def on_gpu(s):
    """Device copies with the same strides, and the arguments shared by the entry points."""
    base = {n: t.cuda() for n, t in s["base"].items()}
    if "qkv" in base:
        q, k, v = base["qkv"].unbind(1)
    elif s["layout"] == "heads":
        q = base["q"].transpose(0, 1).contiguous().transpose(0, 1)
        k, v = base["kv"][0].transpose(0, 1), base["kv"][1].transpose(0, 1)
    else:
        q, (k, v) = base["q"], base["kv"].unbind(1)
    ints = [torch.tensor(s[n], dtype=torch.int32).cuda() for n in ("cu_q", "cu_k")]
    args = (*ints, max(1, *s["lens_q"]), max(1, *s["lens_k"]), s["table"].cuda(), s["buckets"].cuda())
    where = {n: None if s[n] is None else s[n].cuda() for n in ("pos_q", "pos_k")}
    return q, k, v, args, where


def check(name, got, want, bound, rows=None):
    """Every element within its bound; -inf where the definition has -inf."""
    got = got.detach().double().cpu()
    if rows is not None:
        got, want, bound = got[rows], want[rows], bound[rows]
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), finite), f"{name}: values that are not finite"
    assert torch.equal(got[~finite], want[~finite]), f"{name}: other infinities"
    over = ((got - want).abs() - bound)[finite]
    worst = ((got - want).abs() / bound.clamp_min(1e-300))[finite].max().item() if over.numel() else 0.0
    assert over.numel() == 0 or over.max() <= 0, f"{name}: an error {worst:.2f} times its bound"
