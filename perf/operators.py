"""The key-set attention operators on real shapes: plain forms and the library's calls.

  attend  attention of the active rows over a key set per sequence (the first
          key_len cache entries, or a list of kept positions) and a prefix
          shared by the batch; outputs o and lse
  mass    the attention weight each cached key receives from those rows
  evict   the kept list after an eviction by accumulated weight

The plain forms compute in float32 with elementary torch operations and round
once at the end.  `exact` restates the definitions in float64.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attend(name, dtype, batch, n_ctx, rows, heads, kv_heads, head_dim, keys, listed_keys, prefix,
            ragged):
    return {"name": name, "op": "attend", "dtype": dtype, "batch": batch, "n_ctx": n_ctx,
            "rows": rows, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "keys": keys, "listed": listed_keys, "prefix": prefix, "ragged": ragged}


def _mass(name, dtype, batch, n_ctx, rows, heads, kv_heads, head_dim, keys, listed_keys, ragged):
    c = _attend(name, dtype, batch, n_ctx, rows, heads, kv_heads, head_dim, keys, listed_keys, 0,
                ragged)
    c["op"] = "mass"
    return c


def _evict(name, batch, n_ctx, budget, protect, present):
    return {"name": name, "op": "evict", "batch": batch, "n_ctx": n_ctx, "budget": budget,
            "protect": protect, "present": present}


def listed():
    return [
        # one query row per sequence over a prompt of 2048 and a few own keys, four query
        # heads per K/V head: the smallest call, where launches count
        _attend("prefix_one_row", "bf16", 8, 128, 1, 32, 8, 128, 64, False, 2048, False),
        # sixteen samples of one long prompt, a block of 32 masked rows each (block_len 32)
        _attend("prefix_block", "bf16", 16, 256, 32, 32, 32, 128, 256, False, 8192, False),
        # ragged rows and lengths, an empty sequence, one without own keys, seven query heads
        # per K/V head, a prefix that ends one key into a tile
        _attend("prefix_ragged", "bf16", 5, 333, 77, 28, 4, 128, 333, False, 4097, True),
        # many active rows of four sequences over a very long shared prompt: the largest
        _attend("prefix_long", "bf16", 4, 512, 256, 32, 32, 128, 512, False, 16384, False),
        # the decode windows of the batch 4 x 2048 workload with half of the cache evicted
        _attend("kept_window", "bf16", 4, 2048, 384, 32, 32, 128, 1024, True, 0, True),
        # its first steps: every row active, a quarter of the cache evicted
        _attend("kept_all_rows", "bf16", 4, 2048, 2048, 32, 32, 128, 1536, True, 0, False),
        # the fp32 path of a small model, half of the cache evicted
        _attend("kept_f32", "f32", 2, 384, 200, 8, 8, 64, 192, True, 0, True),
        # the weights of the batch 1 x 384 workload's window
        _mass("mass_window", "bf16", 1, 384, 200, 32, 32, 128, 384, False, False),
        # all rows and keys of the batch 4 x 2048 workload
        _mass("mass_all_rows", "bf16", 4, 2048, 2048, 32, 32, 128, 2048, False, False),
        # the fp32 path over kept keys
        _mass("mass_f32", "f32", 2, 384, 200, 8, 4, 64, 301, True, True),
        # the batch 4 x 2048 workload: half of the cache stays
        _evict("evict_window", 4, 2048, 1024, 0.1, 1.0),
        # long caches, an eviction on top of an earlier one
        _evict("evict_long", 4, 131072, 32768, 0.02, 0.6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "mass", "evict"])
    if op == "evict":
        n = _log_int(rng, 64, 131072)
        return {k: v for k, v in _evict("", rng.choice([1, 2, 3, 4]), n, rng.randint(0, n),
                                        rng.uniform(0.0, 0.3), rng.uniform(0.3, 1.0)).items()
                if k != "name"}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 1, 2, 4, 7])
    if dtype == "bf16":
        dh, batch, n = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 8]), _log_int(rng, 16, 2048)
    else:
        dh, batch, n = rng.choice([16, 32, 64]), rng.choice([1, 2, 3]), _log_int(rng, 16, 400)
    rows, keys = _log_int(rng, 1, n), _log_int(rng, 1, n)
    ragged, lst = rng.random() < 0.5, rng.random() < 0.5
    if op == "mass":
        c = _mass("", dtype, batch, n, rows, kv * group, kv, dh, keys, lst, ragged)
    else:
        # a long prefix goes with blocks of rows, none or a short one with any
        prefix = 0
        if rng.random() < 0.6:
            top = 16384 if dtype == "bf16" and rows <= 256 else 512
            prefix = _log_int(rng, 1, top)
        c = _attend("", dtype, batch, n, rows, kv * group, kv, dh, keys, lst, prefix, ragged)
    return {k: v for k, v in c.items() if k != "name"}


def _spread(n, batch, ragged, empty):
    """Per-sequence sizes: n each, or ragged below n with sequence `empty` at zero."""
    if not ragged:
        return [n] * batch
    out = [n - (b * 7919) % (n // 2 + 1) for b in range(batch)]
    if batch > 2:
        out[empty] = 0
    return out


def _rows(case):
    return _spread(case["rows"], case["batch"], case["ragged"], 1)


def _keys(case):
    return _spread(case["keys"], case["batch"], case["ragged"], 2)


def work(case):
    if case["op"] == "evict":
        n = case["batch"] * case["n_ctx"]
        # mass, protected and present flags in; presence flags and at most the budget's list out
        return {"bytes": n * (4 + 1 + 1 + 1) + 4 * case["batch"] * (min(case["budget"], case["n_ctx"]) + 1),
                "flops": n}
    size = 2 if case["dtype"] == "bf16" else 4
    rows, keys = _rows(case), _keys(case)
    H, Hk, dh, P = case["heads"], case["kv_heads"], case["head_dim"], case["prefix"]
    pairs = sum(r * (k + P) for r, k in zip(rows, keys)) * H
    kv_rows = P + sum(k for r, k in zip(rows, keys) if r)
    if case["op"] == "mass":
        return {"bytes": size * dh * (sum(rows) * H + kv_rows * Hk) + 4 * sum(rows) * H
                + 4 * case["batch"] * case["n_ctx"] * 2,
                "flops": 2 * pairs * dh}
    return {"bytes": size * dh * (2 * sum(rows) * H + 2 * kv_rows * Hk) + 4 * sum(rows) * H,
            "flops": 4 * pairs * dh}


class _State:
    pass


def prepare(case, seed):
    s = _State()
    s.case = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, device=dev, generator=g)

    if case["op"] == "evict":
        B, N = case["batch"], case["n_ctx"]
        # accumulated weights: a heavy tail, and many entries that received nothing
        m = torch.exp(2.0 * randn(B, N))
        m[torch.rand((B, N), device=dev, generator=g) < 0.1] = 0.0
        s.mass = m.contiguous()
        s.protect = (torch.rand((B, N), device=dev, generator=g) < case["protect"]).to(torch.uint8)
        s.present = (torch.rand((B, N), device=dev, generator=g) < case["present"]).to(torch.uint8)
        s.keys = torch.full((B, N), -1, dtype=torch.int32, device=dev)
        s.key_len = torch.zeros(B, dtype=torch.int32, device=dev)
        s.present_out = torch.zeros((B, N), dtype=torch.uint8, device=dev)
        return s

    dt = _DT[case["dtype"]]
    B, N, H, Hk, dh = case["batch"], case["n_ctx"], case["heads"], case["kv_heads"], case["head_dim"]
    s.rows, s.lens = _rows(case), _keys(case)
    M = sum(s.rows)
    # a direction shared by the queries and one key in twenty: some keys draw most of the weight
    u = torch.sign(randn(Hk, dh)) * (0.5 * (128.0 / dh) ** 0.25)

    def keys_like(n):
        heavy = (torch.rand((n, 1, 1), device=dev, generator=g) < 0.05).float()
        return (randn(n, Hk, dh) + heavy * u).reshape(n, Hk * dh).to(dt)

    s.q = (randn(M, Hk, H // Hk, dh) + u[:, None, :]).reshape(M, H * dh).to(dt)
    s.k, s.v = keys_like(B * N), randn(B * N, Hk * dh).to(dt)
    off = [0]
    for r in s.rows:
        off.append(off[-1] + r)
    s.seq_off = torch.tensor(off, dtype=torch.int32, device=dev)
    s.key_len = torch.tensor(s.lens, dtype=torch.int32, device=dev)
    s.keys = None
    if case["listed"]:
        s.keys = torch.zeros((B, N), dtype=torch.int32, device=dev)
        for b, n in enumerate(s.lens):
            pick = torch.randperm(N, device=dev, generator=g)[:n]
            s.keys[b, :n] = torch.sort(pick).values.to(torch.int32)
    s.kp = s.vp = None
    if case["prefix"]:
        s.kp, s.vp = keys_like(case["prefix"]), randn(case["prefix"], Hk * dh).to(dt)
    s.scale = 1.0 / math.sqrt(dh)
    s.o = torch.empty((M, H * dh), dtype=dt, device=dev)
    s.lse = torch.empty((M, H), dtype=torch.float32, device=dev)
    if case["op"] == "mass":
        # the log partition an attention call left, and the weights of earlier steps
        s.lse = _attend_plain(s)[1]
        s.prev = torch.rand((B, N), device=dev, generator=g) * 4.0
        s.mass = torch.empty((B, N), dtype=torch.float32, device=dev)
    if own:
        from token_locking_b200 import runtime as rt
        s.op = rt.KeyAttention(batch=B, n_ctx=N, max_rows=max(M, 1), n_heads=H, n_kv_heads=Hk,
                               head_dim=dh, dtype=case["dtype"], prefix=bool(case["prefix"]))
    return s


def _key_set(s, b):
    """Cache rows of sequence b's key set."""
    N, n = s.case["n_ctx"], s.lens[b]
    if s.keys is None:
        return slice(b * N, b * N + n)
    return s.keys[b, :n].long() + b * N


def _scores(s, b, r0, r1, idx, dt, prefix):
    """[Hk, rows * group, keys] scaled scores of sequence b's rows."""
    c = s.case
    H, Hk, dh = c["heads"], c["kv_heads"], c["head_dim"]
    q = s.q[r0:r1].to(dt).reshape(r1 - r0, Hk, H // Hk, dh).permute(1, 0, 2, 3)
    k = s.k[idx].to(dt)
    if prefix and s.kp is not None:
        k = torch.cat([s.kp.to(dt), k])
    k = k.reshape(-1, Hk, dh).permute(1, 2, 0)
    return torch.matmul(q.reshape(Hk, -1, dh), k) * s.scale


def _attend_plain(s):
    c = s.case
    H, Hk, dh = c["heads"], c["kv_heads"], c["head_dim"]
    M = s.q.shape[0]
    o = torch.zeros((M, H * dh), dtype=torch.float32, device=s.q.device)
    lse = torch.full((M, H), -math.inf, dtype=torch.float32, device=s.q.device)
    r0 = 0
    for b in range(c["batch"]):
        r1 = r0 + s.rows[b]
        if r1 > r0 and s.lens[b] + c["prefix"] > 0:
            idx = _key_set(s, b)
            z = _scores(s, b, r0, r1, idx, torch.float32, True)
            top = z.amax(dim=-1, keepdim=True)
            p = torch.exp(z - top)
            tot = p.sum(dim=-1, keepdim=True)
            v = s.v[idx].float()
            if s.vp is not None:
                v = torch.cat([s.vp.float(), v])
            x = torch.matmul(p, v.reshape(-1, Hk, dh).permute(1, 0, 2)) / tot
            n = r1 - r0
            o[r0:r1] = x.reshape(Hk, n, H // Hk, dh).permute(1, 0, 2, 3).reshape(n, H * dh)
            lse[r0:r1] = (top + torch.log(tot)).reshape(Hk, n, H // Hk).permute(1, 0, 2).reshape(n, H)
        r0 = r1
    return o.to(s.q.dtype), lse


def _mass_plain(s):
    c = s.case
    H, Hk = c["heads"], c["kv_heads"]
    out = s.prev.clone()
    r0 = 0
    for b in range(c["batch"]):
        r1 = r0 + s.rows[b]
        if r1 > r0 and s.lens[b] > 0:
            idx = _key_set(s, b)
            z = _scores(s, b, r0, r1, idx, torch.float32, False)
            n = r1 - r0
            ls = s.lse[r0:r1].reshape(n, Hk, H // Hk).permute(1, 0, 2).reshape(Hk, -1, 1)
            w = torch.exp(z - ls).sum(dim=(0, 1))
            local = slice(0, s.lens[b]) if s.keys is None else s.keys[b, :s.lens[b]].long()
            out[b, local] += w
        r0 = r1
    return out


def _evict_plain(s):
    c = s.case
    B, N = c["batch"], c["n_ctx"]
    keys = torch.full((B, N), -1, dtype=torch.int32, device=s.mass.device)
    here = s.present != 0
    fixed = here & (s.protect != 0)
    cand = here & (s.protect == 0)
    # heaviest first, ties to the lower position; entries that are no candidates last
    order = torch.sort(torch.where(cand, s.mass, torch.full_like(s.mass, -math.inf)), dim=1,
                       descending=True, stable=True).indices
    room = (c["budget"] - fixed.sum(dim=1, keepdim=True)).clamp(min=0)
    keep = torch.zeros_like(here)
    keep.scatter_(1, order, torch.arange(N, device=s.mass.device)[None, :] < room)
    keep = (keep & cand) | fixed
    lens = keep.sum(dim=1)
    slot = torch.cumsum(keep, dim=1) - 1
    b, n = torch.nonzero(keep, as_tuple=True)
    keys[b, slot[b, n]] = n.to(torch.int32)
    return {"keys": keys, "key_len": lens.to(torch.int32), "present": keep.to(torch.uint8)}


def run(s):
    op = s.case["op"]
    if not own:
        if op == "attend":
            return _attend_plain(s)
        return _mass_plain(s) if op == "mass" else _evict_plain(s)
    from token_locking_b200 import runtime as rt
    if op == "attend":
        s.op.attend(s.q, s.k, s.v, s.o, s.seq_off, key_len=s.key_len, keys=s.keys,
                    k_prefix=s.kp, v_prefix=s.vp, lse=s.lse)
        return s.o, s.lse
    if op == "mass":
        s.op.mass(s.q, s.k, s.lse, s.mass, s.seq_off, key_len=s.key_len, keys=s.keys,
                  mass_prev=s.prev, decay=1.0)
        return s.mass
    rt.kv_evict(s.mass, s.case["budget"], s.keys, s.key_len, protect=s.protect,
                present=s.present, present_out=s.present_out)
    return {"keys": s.keys, "key_len": s.key_len, "present": s.present_out}


def exact(case, seed):
    """The definitions in float64, one (sequence, head) at a time."""
    global own
    if case["op"] == "evict":
        return None
    if work(case)["flops"] > 3e11:
        return None
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    H, Hk, dh, N, B = (case[x] for x in ("heads", "kv_heads", "head_dim", "n_ctx", "batch"))
    M = s.q.shape[0]
    dev = s.q.device
    f8 = torch.float64
    o = torch.zeros((M, H, dh), dtype=f8, device=dev)
    lse = torch.full((M, H), -math.inf, dtype=f8, device=dev)
    if case["op"] == "mass":
        mass = s.prev.to(f8).clone()
    r0 = 0
    for b in range(B):
        r1 = r0 + s.rows[b]
        if s.keys is None:
            pos = torch.arange(s.lens[b], device=dev)
        else:
            pos = s.keys[b, :s.lens[b]].long()
        if r1 > r0:
            for h in range(H):
                col = slice((h * Hk // H) * dh, (h * Hk // H) * dh + dh)
                qh = s.q[r0:r1, h * dh:(h + 1) * dh].to(f8)
                kh = s.k[pos + b * N, col].to(f8)
                if case["op"] == "mass":
                    w = torch.exp(qh @ kh.T / math.sqrt(dh) - s.lse[r0:r1, h:h + 1].to(f8))
                    mass[b].index_add_(0, pos, w.sum(dim=0))
                    continue
                vh = s.v[pos + b * N, col].to(f8)
                if case["prefix"]:
                    kh = torch.cat([s.kp[:, col].to(f8), kh])
                    vh = torch.cat([s.vp[:, col].to(f8), vh])
                if kh.shape[0] == 0:
                    continue
                z = qh @ kh.T / math.sqrt(dh)
                ls = torch.logsumexp(z, dim=1)
                lse[r0:r1, h] = ls
                o[r0:r1, h] = torch.exp(z - ls[:, None]) @ vh
        r0 = r1
    if case["op"] == "mass":
        return mass
    return o.reshape(M, H * dh), lse
