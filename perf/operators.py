"""The operators that train the gate of the routed layer, as measured cases.

One pass of each: the balance loss with its per-expert counts, the gradient of
the router logits (gates, balance and z terms), the combine's backward, the
router's backward, and the clipping of a list of gradients by their global
norm.  ``run`` computes a case in plain torch operations, or through the
library's calls where ``own`` is set."""

import math
import random

import numpy as np
import torch

own = False

# The largest case of each operator, by the work() bytes (or flops) that a
# drawn case may cost.
_MAX_LOGITS = 1 << 26


def listed():
    return [
        # one decode-sized batch of the tiny layer: latency alone
        {"name": "balance-tiny-t64-e8", "op": "balance", "T": 64, "E": 8, "k": 2, "S": 1, "masked": False},
        # a prefill-sized micro-batch of 128 experts: packed sequences of unequal length, some tokens masked
        {"name": "balance-t8192-e128-seqs", "op": "balance", "T": 8192, "E": 128, "k": 8, "S": 16, "masked": True},
        # a whole training batch of 256 experts, one statistic over all of it
        {"name": "balance-t262144-e256", "op": "balance", "T": 262144, "E": 256, "k": 8, "S": 1, "masked": False},
        # eight experts, an odd number of tokens, gates and both auxiliary terms
        {"name": "gate-t4095-e8", "op": "gate", "T": 4095, "E": 8, "k": 2, "S": 1, "masked": False},
        # a large batch of 256 experts with per-sequence balance terms and padding
        {"name": "gate-t131072-e256-seqs", "op": "gate", "T": 131072, "E": 256, "k": 8, "S": 64, "masked": True},
        # the gates' gradient of a small batch, experts frozen (no gradient of their rows)
        {"name": "combine-t64-d2048-dw", "op": "combine", "T": 64, "d": 2048, "k": 8, "dz": False},
        # a prefill-sized batch whose experts train too: every row of dz is written
        {"name": "combine-t8192-d2048", "op": "combine", "T": 8192, "d": 2048, "k": 8, "dz": True},
        # the router's backward at 64 tokens: the weight gradient's write
        {"name": "router-t64-d2048-e128", "op": "router", "T": 64, "d": 2048, "E": 128, "dx": True},
        # ... of a prefill-sized micro-batch
        {"name": "router-t8192-d2048-e128", "op": "router", "T": 8192, "d": 2048, "E": 128, "dx": True},
        # ... of a large one with 256 experts of a wide model
        {"name": "router-t16384-d7168-e256", "op": "router", "T": 16384, "d": 7168, "E": 256, "dx": True},
        # the gates of 48 layers (weight and bias each), fp32 gradients
        {"name": "clip-gates-96", "op": "clip", "tensors": 96, "elements": 48 * (2048 * 128 + 128), "dtype": "gates"},
        # expert weight gradients in bf16, a few very large tensors
        {"name": "clip-experts-bf16", "op": "clip", "tensors": 8, "elements": 1 << 29, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "gate", "combine", "router", "clip"])
    if op in ("balance", "gate"):
        E = _log_int(rng, 2, 1024)
        T = _log_int(rng, 1, min(262144 if op == "balance" else 131072, _MAX_LOGITS // (2 * E)))
        k = rng.randint(1, min(E, 16))
        S = _log_int(rng, 1, 512) if rng.random() < 0.5 else 1
        return {"op": op, "T": T, "E": E, "k": k, "S": S, "masked": rng.random() < 0.5}
    if op == "combine":
        d = 64 * _log_int(rng, 1, 112)
        k = rng.randint(1, 16)
        T = _log_int(rng, 1, max(1, min(16384, (1 << 27) // (d * k))))
        return {"op": op, "T": T, "d": d, "k": k, "dz": rng.random() < 0.6}
    if op == "router":
        d = 64 * _log_int(rng, 1, 112)
        E = _log_int(rng, 2, 256)
        return {"op": op, "T": _log_int(rng, 1, 16384), "d": d, "E": E, "dx": rng.random() < 0.7}
    n = _log_int(rng, 1, 400)
    return {"op": op, "tensors": n, "elements": _log_int(rng, n, 1 << 28), "dtype": rng.choice(["fp32", "bf16", "mixed"])}


# --------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _logits(T, E, g):
    """Router logits with a popular-expert skew, and their top-k order."""
    rank = torch.randperm(E, generator=g, device="cuda").float()
    return torch.randn(T, E, generator=g, device="cuda") - 0.5 * torch.log(rank + 1.0)


def _offsets(T, S, seed):
    """S ragged sequences, empty ones among them where S is near T; a few rows
    behind the last one."""
    r = np.random.RandomState(seed % (1 << 31))
    end = T if S == 1 else max(1, T - T // 50)
    cuts = np.sort(r.randint(0, end + 1, S - 1))
    return torch.tensor(np.concatenate([[0], cuts, [end]]).astype(np.int32)).cuda()


def _gate_inputs(c, seed):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    g = _gen(seed)
    L = _logits(T, E, g)
    top, idx = torch.topk(L, k, dim=1)
    st = {"logits": L, "idx": idx.int().contiguous(), "w": torch.softmax(top, 1).contiguous(),
          "seq_offsets": _offsets(T, S, seed) if S > 1 else None,
          "token_mask": (torch.rand(T, generator=g, device="cuda") > 0.06).to(torch.uint8) if c["masked"] else None,
          "balance_coef": 1e-2, "z_coef": 1e-3}
    return st, g


def _sizes(c):
    """The tensors' sizes: pairs of a gate's weight and bias, or a ragged
    split of the elements; the same for every seed."""
    n, total = c["tensors"], c["elements"]
    if c["dtype"] == "gates":
        return [2048 * 128, 128] * (n // 2)
    r = random.Random(n * 1000003 + total)
    part = [r.expovariate(1.0) + 1e-3 for _ in range(n)]
    got = [max(1, int(p / sum(part) * total)) for p in part]
    got[got.index(max(got))] += max(0, total - sum(got))
    return got


def _types(c):
    n = c["tensors"]
    return [torch.bfloat16 if c["dtype"] == "bf16" or (c["dtype"] == "mixed" and i % 3 == 0) else torch.float32
            for i in range(n)]


def _views(sizes, types):
    """One flat buffer per type, and each tensor's slice of it in turn."""
    used = {t: sum(s for s, u in zip(sizes, types) if u == t) for t in dict.fromkeys(types)}
    flat = {t: torch.empty(n, dtype=t, device="cuda") for t, n in used.items()}
    at, got = {t: 0 for t in used}, []
    for s, t in zip(sizes, types):
        got.append(flat[t][at[t]:at[t] + s])
        at[t] += s
    return flat, got


def prepare(case, seed):
    c = case
    st = {"case": c}
    if c["op"] in ("balance", "gate"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        inp, g = _gate_inputs(c, seed)
        st.update(inp)
        if c["op"] == "balance":
            st.update(loss=torch.empty(3, device="cuda"), counts=torch.empty(S, E, dtype=torch.int32, device="cuda"),
                      tokens=torch.empty(S + 2, dtype=torch.int32, device="cuda"),
                      prob_mean=torch.empty(S, E, device="cuda"))
        else:
            # what the loss of the same batch left: counts and token numbers
            _, counts, tokens, _ = _plain_balance(st, T, E, k, S)
            st.update(dw=torch.randn(T, k, generator=g, device="cuda"), counts=counts, tokens=tokens,
                      dloss=torch.full((1,), 0.75, device="cuda"), dlogits=torch.empty(T, E, device="cuda"))
    elif c["op"] == "combine":
        T, d, k = c["T"], c["d"], c["k"]
        g = _gen(seed)
        st.update(dy=torch.randn(T, d, generator=g, device="cuda").bfloat16(),
                  z=torch.randn(T * k, d, generator=g, device="cuda").bfloat16(),
                  row_of=torch.randperm(T * k, generator=g, device="cuda").int().view(T, k),
                  w=torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1),
                  dw=torch.empty(T, k, device="cuda"),
                  dz=torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda") if c["dz"] else None)
    elif c["op"] == "router":
        T, d, E = c["T"], c["d"], c["E"]
        g = _gen(seed)
        st.update(x=torch.randn(T, d, generator=g, device="cuda").bfloat16(),
                  w_g=torch.randn(d, E, generator=g, device="cuda") / math.sqrt(d),
                  dlogits=torch.randn(T, E, generator=g, device="cuda") * torch.rand(T, 1, generator=g, device="cuda") / T,
                  dw_g=torch.empty(d, E, device="cuda"), dbias=torch.empty(E, device="cuda"),
                  dx=torch.empty(T, d, dtype=torch.bfloat16, device="cuda") if c["dx"] else None)
    else:
        g = _gen(seed)
        sizes, types = _sizes(c), _types(c)
        grads = [(torch.randn(s, generator=g, device="cuda", dtype=t) * 1e-2) for s, t in zip(sizes, types)]
        flat, out = _views(sizes, types)
        st.update(grads=grads, out=out, flat=list(flat.values()), max_norm=1.0,
                  norm=torch.empty(1, device="cuda"))
    if own:
        _handles(st)
    return st


def _handles(st):
    """The shapes, workspaces and gradient lists that a program keeps."""
    import routing_dispatch_expert_softmax_b200 as moe
    c = st["case"]
    if c["op"] == "clip":
        st["list"] = moe.GradList(st["grads"], st["out"])
        return
    st["shape"] = moe.MoEShape.of(c["T"], c.get("d", 64), c.get("E", c.get("k")), c.get("k", 1), 64)
    if c["op"] != "combine":
        st["ws"] = moe.workspace_bwd(st["shape"], c.get("S", 1))


# ----------------------------------------------------------------------- run
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import routing_dispatch_expert_softmax_b200 as moe
    op = st["case"]["op"]
    if op == "balance":
        moe.moe_balance_loss(st["logits"], st["idx"], st["loss"], st["counts"], st["tokens"], st["shape"], st["ws"],
                             balance_coef=st["balance_coef"], z_coef=st["z_coef"], token_mask=st["token_mask"],
                             seq_offsets=st["seq_offsets"], prob_mean=st["prob_mean"])
        return {"loss": st["loss"], "counts": st["counts"], "tokens": st["tokens"], "prob_mean": st["prob_mean"]}
    if op == "gate":
        moe.moe_gate_bwd(st["logits"], st["idx"], st["dlogits"], st["shape"], st["ws"], w=st["w"], dw=st["dw"],
                         counts=st["counts"], tokens=st["tokens"], balance_coef=st["balance_coef"],
                         z_coef=st["z_coef"], dloss=st["dloss"], token_mask=st["token_mask"],
                         seq_offsets=st["seq_offsets"])
        return {"dlogits": st["dlogits"]}
    if op == "combine":
        moe.moe_combine_bwd(st["dy"], st["z"], st["row_of"], st["w"], st["shape"], dw=st["dw"], dz=st["dz"])
        return {"dw": st["dw"], "dz": st["dz"]}
    if op == "router":
        moe.moe_router_bwd(st["x"], st["w_g"], st["dlogits"], st["shape"], st["ws"], dw_g=st["dw_g"],
                           dbias=st["dbias"], dx=st["dx"])
        return {"dw_g": st["dw_g"], "dbias": st["dbias"], "dx": st["dx"]}
    moe.moe_clip_grads(st["list"], st["max_norm"], st["norm"])
    return {"norm": st["norm"], "out": st["flat"]}


def _segments(st, T, S):
    """The sequence of each token, and whether it lies in one."""
    if st["seq_offsets"] is None:
        return torch.zeros(T, dtype=torch.long, device="cuda"), torch.ones(T, dtype=torch.bool, device="cuda")
    o = st["seq_offsets"].long()
    t = torch.arange(T, device="cuda")
    seg = torch.searchsorted(o, t, right=True) - 1
    inside = (seg >= 0) & (seg < S)
    return seg.clamp(0, S - 1), inside


def _valid(st, T, S):
    seg, ok = _segments(st, T, S)
    ok = ok & (st["logits"] != -math.inf).any(1)
    return seg, ok & (st["token_mask"] != 0) if st["token_mask"] is not None else ok


def _plain_softmax(L):
    """(logsumexp, softmax) of each row."""
    top = L.max(1, keepdim=True).values
    e = torch.exp(L - top)
    total = e.sum(1, keepdim=True)
    return (top + torch.log(total)).squeeze(1), e / total


def _plain_balance(st, T, E, k, S):
    seg, ok = _valid(st, T, S)
    lse, p = _plain_softmax(st["logits"])
    member = ((seg[None, :] == torch.arange(S, device="cuda")[:, None]) & ok[None, :])  # (S, T)
    n = member.sum(1)
    row = (seg[:, None] * E + st["idx"].long())[ok].reshape(-1)
    counts = torch.bincount(row, minlength=S * E).view(S, E)
    # sums over many tokens: 64 bits
    psum = torch.zeros(S, E, dtype=torch.float64, device="cuda").index_add_(0, seg[ok], p[ok].double())
    some = n.clamp(min=1).double()
    live = (n > 0).sum().clamp(min=1).double()
    total = n.sum().clamp(min=1).double()
    mean = psum / some[:, None]
    bal = st["balance_coef"] * ((E / (k * some)) * (counts.double() * mean).sum(1)).sum() / live
    z = st["z_coef"] * (lse[ok].double() ** 2).sum() / total
    tokens = torch.cat([n, n.sum()[None], (n > 0).sum()[None]]).int()
    return torch.stack([bal + z, bal, z]).float(), counts.int(), tokens, mean.float()


def _plain_gate(st, T, E, k, S):
    L, idx, w, dw = st["logits"], st["idx"].long(), st["w"], st["dw"]
    seg, ok = _valid(st, T, S)
    n = st["tokens"][:S].clamp(min=1).double()
    total, live = st["tokens"][S].clamp(min=1).double(), st["tokens"][S + 1].clamp(min=1).double()
    lse, p = _plain_softmax(L)
    f = (st["counts"].double() * (st["balance_coef"] * E / (live * k * n * n))[:, None]).float()[seg]
    aux = p * (f - (f * p).sum(1, keepdim=True) + (2 * st["z_coef"] / total).float() * lse[:, None])
    aux = torch.where(ok[:, None], aux * st["dloss"], torch.zeros_like(aux))
    gate = w * (dw - (w * dw).sum(1, keepdim=True))
    return aux.scatter_add(1, idx, gate)


def _run_plain(st):
    c, op = st["case"], st["case"]["op"]
    if op == "balance":
        loss, counts, tokens, mean = _plain_balance(st, c["T"], c["E"], c["k"], c["S"])
        return {"loss": loss, "counts": counts, "tokens": tokens, "prob_mean": mean}
    if op == "gate":
        return {"dlogits": _plain_gate(st, c["T"], c["E"], c["k"], c["S"])}
    if op == "combine":
        T, k, row = c["T"], c["k"], st["row_of"].long()
        dy = st["dy"].float()
        dw = (st["z"].float()[row.view(-1)].view(T, k, -1) * dy[:, None, :]).sum(2)
        dz = None
        if c["dz"]:
            dz = torch.empty_like(st["z"])
            dz[row.view(-1)] = (st["w"][:, :, None] * dy[:, None, :]).view(T * k, -1).bfloat16()
        return {"dw": dw, "dz": dz}
    if op == "router":
        dl, x = st["dlogits"], st["x"].float()
        return {"dw_g": x.t() @ dl, "dbias": dl.double().sum(0).float(),
                "dx": (dl @ st["w_g"].t()).bfloat16() if c["dx"] else None}
    # every square sum in 64 bits, one rounding at the end
    sq = torch.stack([g.double().square().sum() for g in st["grads"]]).sum()
    norm = sq.sqrt()
    coef = torch.where(norm.isfinite(), (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0), torch.ones_like(norm)).float()
    [o.copy_(g.float() * coef) for g, o in zip(st["grads"], st["out"])]
    return {"norm": norm.float().view(1), "out": st["flat"]}


# ---------------------------------------------------------------------- work
def work(case):
    c, op = case, case["op"]
    if op in ("balance", "gate"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        small = T * c["masked"] + 4 * (S + 1) * (S > 1) + 4 * (S + 2)
        if op == "balance":
            return {"bytes": 4 * T * E + 4 * T * k + 8 * S * E + 12 + small, "flops": 6 * T * E}
        return {"bytes": 8 * T * E + 12 * T * k + 4 * S * E + small, "flops": 10 * T * E}
    if op == "combine":
        T, d, k = c["T"], c["d"], c["k"]
        return {"bytes": 2 * T * d + 2 * T * k * d * (2 if c["dz"] else 1) + 12 * T * k,
                "flops": 2 * T * k * d + (T * k * d if c["dz"] else 0)}
    if op == "router":
        T, d, E = c["T"], c["d"], c["E"]
        two = 2 if c["dx"] else 1
        return {"bytes": 2 * T * d * two + 4 * T * E + 4 * d * E * two + 4 * E, "flops": 2 * T * d * E * two + T * E}
    each = [s * (2 if t == torch.bfloat16 else 4) for s, t in zip(_sizes(c), _types(c))]
    return {"bytes": 2 * sum(each) + 4, "flops": 3 * sum(_sizes(c))}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions, in 64 bits, from the same inputs."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    c, op = case, case["op"]
    if op in ("balance", "gate"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        L = st["logits"].double()
        off = [0, T] if st["seq_offsets"] is None else st["seq_offsets"].tolist()
        keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["token_mask"] is None else st["token_mask"] > 0
        prob = torch.softmax(L, 1)
        lse = L.max(1).values + (L - L.max(1, keepdim=True).values).exp().sum(1).log()
        idx = st["idx"].long()
        rows = [torch.nonzero(keep[a:b]).flatten() + a for a, b in zip(off[:-1], off[1:])]
        n = [int(r.numel()) for r in rows]
        N, live = max(sum(n), 1), max(sum(m > 0 for m in n), 1)
        cnt = torch.stack([torch.bincount(idx[r].flatten(), minlength=E) for r in rows]).double()
        if op == "balance":
            mean = torch.stack([prob[r].sum(0) / max(m, 1) for r, m in zip(rows, n)])
            bal = sum(float((cnt[s] / (max(n[s], 1) * k) * mean[s]).sum()) * E for s in range(S)) / live * st["balance_coef"]
            z = sum(float(lse[r].square().sum()) for r in rows) / N * st["z_coef"]
            return {"loss": torch.tensor([bal + z, bal, z], dtype=torch.float64), "counts": None, "tokens": None,
                    "prob_mean": mean}
        w, dw = st["w"].double(), st["dw"].double()
        out = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        for s, r in enumerate(rows):
            if n[s]:
                pr = prob[r]
                frac = cnt[s] / (n[s] * k)
                # d/dL of E * sum_e frac_e * mean_e, then of the mean squared logsumexp
                out[r] = st["balance_coef"] * E / (live * n[s]) * (pr * frac - pr * (pr @ frac)[:, None])
                out[r] += st["z_coef"] * 2.0 / N * lse[r][:, None] * pr
        out *= 0.75
        out.scatter_add_(1, idx, w * dw - w * (w * dw).sum(1, keepdim=True))
        return {"dlogits": out}
    if op == "combine":
        T, k, d = c["T"], c["k"], c["d"]
        row = st["row_of"].long()
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        dz = torch.empty(T * k, d, dtype=torch.float64, device="cuda") if c["dz"] else None
        dy = st["dy"].double()
        for j in range(k):
            dw[:, j] = torch.einsum("td,td->t", dy, st["z"][row[:, j]].double())
            if c["dz"]:
                dz[row[:, j]] = st["w"][:, j, None].double() * dy
        return {"dw": dw, "dz": dz}
    if op == "router":
        x, dl = st["x"].double(), st["dlogits"].double()
        return {"dw_g": torch.einsum("td,te->de", x, dl), "dbias": torch.einsum("te->e", dl),
                "dx": torch.einsum("te,de->td", dl, st["w_g"].double()) if c["dx"] else None}
    total = math.sqrt(math.fsum(float(torch.dot(g.double(), g.double())) for g in st["grads"]))
    scale = min(1.0, st["max_norm"] / (total + 1e-6))
    out = {t: torch.cat([g.double() * scale for g, u in zip(st["grads"], _types(c)) if u == t])
           for t in dict.fromkeys(_types(c))}
    return {"norm": torch.tensor([total], dtype=torch.float64), "out": list(out.values())}
