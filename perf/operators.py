"""Cases of the rotary positions and of the paged, bounded cache: what each call computes, in elementary torch operations, and
the calls a user's program makes for it.

Kinds: "rotate" and "rotate_backward" (rotary positions of q and k and their gradients), "append" (rotate new tokens and put them
into the cache's pages), "attend" (one new token's attention over the pages, the memory's read, and the accumulated weights),
"evict" (append a chunk of tokens, then evict down to the budget into the memory A), "step" (one serving step: append, evict,
attend).

In every cache case row b holds `lens(case)[b]` pairs; -1 marks an empty row, which every call leaves alone.
"""
import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF16, "f32": F32}
NO_SCALING = dict(base=10000.0, inter=False, factor=1.0, low=0.0, high=0.0, train=0, gain=1.0)


# ---- cases ------------------------------------------------------------------

def _rot(d, **kw):
    return {**NO_SCALING, "rot": d, **kw}


def listed():
    # frequencies extended eightfold over a 4096-token training length, with a ramp between 1 and 4 turns
    long = dict(base=500000.0, factor=8.0, low=1.0, high=4.0, train=4096, gain=1.2)
    return [
        # q and k of the LM-shaped prefill before it runs
        dict(name="rotate_lm", kind="rotate", B=8, Hq=12, H=12, T=4096, d=64, dtype="bf16", t0=0, packed=False, **_rot(64)),
        # slices of a fused projection, [B,T,heads,d] in memory, half of each head rotated, far into a long document
        dict(name="rotate_fused_qkv", kind="rotate", B=3, Hq=32, H=8, T=1001, d=128, dtype="bf16", t0=1000003, packed=True,
             **_rot(64, inter=True, **long)),
        # gradients of q and k (float32) of the long-context prefill, an odd length
        dict(name="rotate_backward_long", kind="rotate_backward", B=1, Hq=16, H=16, T=32767, d=64, dtype="f32", t0=0, packed=False,
             **_rot(64, inter=True)),
        # gradients of a small bf16 batch, whose time is the launch
        dict(name="rotate_backward_small", kind="rotate_backward", B=2, Hq=4, H=2, T=129, d=64, dtype="bf16", t0=7, packed=False,
             **_rot(32)),
        # a decode batch's new tokens enter the pages (slices of a fused projection), a few rows empty; each pass takes the last
        # pass's tokens back first, as a server does whose drafted tokens were refused
        dict(name="append_decode", kind="append", B=256, Hq=32, H=8, T=1, d=128, dtype="bf16", lo=100, hi=2048, page=64, ragged=True,
             **_rot(128, **long)),
        # right-padded prompts of different lengths fill the pages of rows that are started anew each pass
        dict(name="append_prompts", kind="append", B=4, Hq=12, H=12, T=2500, d=64, dtype="f32", lo=0, hi=0, page=32, ragged=True,
             **_rot(64)),
        # one sequence of the LM shape: latency
        dict(name="attend_one", kind="attend", B=1, Hq=12, H=12, d=64, dtype="bf16", lo=203, hi=203, page=16, memory=True, mass=True),
        # a serving batch whose rows differ by two orders of magnitude in length
        dict(name="attend_ragged", kind="attend", B=32, Hq=32, H=8, d=128, dtype="bf16", lo=90, hi=16000, page=64, memory=True, mass=True),
        # one long document: the length has to be split
        dict(name="attend_long", kind="attend", B=1, Hq=32, H=4, d=128, dtype="bf16", lo=131001, hi=131001, page=128, memory=False, mass=False),
        # the float32 recall shape
        dict(name="attend_recall_f32", kind="attend", B=8, Hq=4, H=4, d=64, dtype="f32", lo=700, hi=2048, page=16, memory=True, mass=True),
        # a chunk of a prompt joins a cache that is full: the lightest pairs leave into the memory
        # (its keys were rotated for the prefill, so they enter as they are)
        dict(name="evict_chunk", kind="evict", B=8, H=12, T=2047, d=64, dtype="bf16", budget=512, recent=128, page=64),
        # steady serving of a full cache: one token in, one pair out, attention over the rest
        dict(name="step_serving", kind="step", B=64, Hq=32, H=8, T=1, d=128, dtype="bf16", budget=2048, recent=64, page=64, memory=True,
             mass=True, **_rot(128)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotate", "rotate_backward", "append", "attend", "evict", "step"])
    d, dtype = rng.choice([64, 64, 128, 128, 32]), rng.choice(["bf16", "bf16", "f32"])
    H = rng.choice([1, 2, 4, 8, 12])
    G = rng.choice([1, 1, 2, 4, 8])
    c = dict(kind=kind, Hq=H * G, H=H, d=d, dtype=dtype)
    rot = _rot(rng.choice([d, d, d // 2]), inter=rng.random() < 0.5)
    if rng.random() < 0.4:
        rot.update(base=500000.0, factor=float(rng.choice([2, 4, 8])), low=1.0, high=float(rng.choice([4, 32])), train=4096, gain=1.1)
    es = 2 if dtype == "bf16" else 4
    if kind in ("rotate", "rotate_backward"):
        tokens = _log(rng, 1, max(2, (1 << 26) // (H * (G + 1) * d * es)) * 4)
        c["B"] = rng.choice([1, 2, 3, 8])
        c.update(T=max(1, tokens // c["B"]), t0=rng.choice([0, rng.randrange(1 << 20)]), packed=rng.random() < 0.5, **rot)
        return c
    page = rng.choice([16, 32, 64, 128])
    if kind == "append":
        T = rng.choice([1, 1, _log(rng, 2, 2500)])
        B = _log(rng, 1, 256) if T == 1 else rng.choice([1, 2, 4])
        c.update(B=B, T=T, lo=0, hi=rng.choice([0, 777, 2048]), page=page, ragged=rng.random() < 0.7, **rot)
        return c
    if kind == "attend":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, max(2, min(131072, (1 << 29) // (B * H * d * 2 * es))))
        c.update(B=B, lo=max(1, hi // rng.choice([1, 3, 50])), hi=hi, page=page, memory=rng.random() < 0.6, mass=rng.random() < 0.6)
        return c
    budget = _log(rng, 16, 2048)
    c.update(budget=budget, recent=rng.randrange(1, max(2, budget // 2)), page=page)
    if kind == "evict":
        c.pop("Hq")
        c.update(B=rng.choice([1, 2, 8, 8]), T=rng.choice([1, 2, _log(rng, 3, 2047)]))
    else:
        c.update(B=_log(rng, 1, 64), T=1, memory=True, mass=True, **rot)
    return c


def work(c):
    es, d, H = (2 if c["dtype"] == "bf16" else 4), c["d"], c["H"]
    if c["kind"] in ("rotate", "rotate_backward"):
        n = c["B"] * c["T"] * (c["Hq"] + H) * d
        return {"bytes": 2 * n * es, "flops": 3 * n * c["rot"] / d}
    B, held = c["B"], lens(c)
    live = [n for n in held if n >= 0]
    if c["kind"] == "append":
        tok = sum(counts(c))
        return {"bytes": tok * ((2 * c["Hq"] + 4 * H) * d * es + H * 12) + 32 * B, "flops": 3 * tok * (c["Hq"] + H) * c["rot"]}
    A = len(live) * H * d * d * 4
    bytes_, flops = 0, 0
    if c["kind"] in ("evict", "step"):
        T = c["T"]
        out = sum(max(0, n + T - c["budget"]) for n in live)
        moved = sum(min(max(0, n + T - c["budget"]), c["budget"]) for n in live)  # at most: survivors that fill freed slots
        tok = len(live) * T
        # tokens in, weights and positions read, pairs that leave read, A read and written, moved pairs read and written
        bytes_ += tok * H * (4 * d * es + 12) + sum(n + T for n in live) * H * 8 + out * H * 2 * d * es + 2 * A
        bytes_ += 0 if T == 1 else moved * H * (4 * d * es + 16)
        flops += 2 * out * H * d * d + 2 * A // 4
        live = [min(n + T, c["budget"]) for n in live]
    if c["kind"] in ("attend", "step"):
        tot = sum(live)
        bytes_ += tot * H * (2 * d * es + (8 if c["mass"] else 0)) + 2 * len(live) * c["Hq"] * d * es
        flops += 4 * tot * c["Hq"] * d
        if c["memory"]:
            bytes_ += A if c["kind"] == "attend" else 0  # the step's A was just written
            flops += 2 * len(live) * c["Hq"] * d * d
    return {"bytes": bytes_, "flops": flops}


def lens(c):
    """Pairs held by each row before the call; -1: an empty row."""
    B = c["B"]
    if c["kind"] in ("evict", "step"):
        return [c["budget"] if b % 8 != 5 else c["budget"] // 2 for b in range(B)]
    lo, hi = max(1, c["lo"]), max(1, c["hi"])
    n = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * (b / max(1, B - 1))))) for b in range(B)]
    n = [0] * B if c["hi"] == 0 else n
    random.Random(B).shuffle(n)
    if c.get("ragged") or c["kind"] == "attend":
        n = [-1 if b % 16 == 9 else 0 if b % 16 == 3 else x for b, x in enumerate(n)]
    return n


def counts(c):
    """Tokens each row appends."""
    full = [c["T"]] * c["B"]
    if c["T"] > 1 and c.get("ragged"):
        full = [max(1, c["T"] * (b + 1) // c["B"] - b) for b in range(c["B"])]
    return [0 if n < 0 else x for n, x in zip(lens(c), full)]


# ---- inputs -----------------------------------------------------------------

def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt, d, B, H = torch.device("cuda"), DT[c["dtype"]], c["d"], c["B"], c["H"]

    def rnd(*shape, dtype=F32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    def heads(Hn, T, packed):  # [B,Hn,T,d]; packed: a view of token-major rows
        x = rnd(B, T, Hn, d, dtype=dt).transpose(1, 2)
        return x if packed else x.contiguous()

    s = dict(c=c, kind=c["kind"])
    if c["kind"] in ("rotate", "rotate_backward"):
        if c["packed"]:  # one projection's output, q's heads, then k's
            row = rnd(B, c["T"], c["Hq"] + H, d, dtype=dt)
            s["q"], s["k"] = row[:, :, :c["Hq"]].transpose(1, 2), row[:, :, c["Hq"]:].transpose(1, 2)
        else:
            s["q"], s["k"] = heads(c["Hq"], c["T"], False), heads(H, c["T"], False)
        s["q_out"], s["k_out"] = (torch.empty(B, h, c["T"], d, dtype=dt, device=dev) for h in (c["Hq"], H))
        s["positions"] = None
        if c["packed"]:  # rows at positions of their own
            s["positions"] = torch.randint(0, c["t0"] + 1, (B, 1), generator=gen, device=dev) + torch.arange(c["T"], device=dev)
        if own:
            import sliding_window_attention_tc_b200 as tc
            s["tc"], s["rotary"] = tc, _rotary(tc, c)
        return s

    held, page = lens(c), c["page"]
    T = c.get("T", 0)
    # a bounded row grows to its budget over the passes, whatever it holds before the first
    most = [c["budget"] if c["kind"] in ("evict", "step") else max(0, n) for n in held]
    per = [(n + T + page - 1) // page for n in most]
    width, pool = max(1, max(per)), sum(per) + 3
    order = torch.randperm(pool, generator=gen, device=dev).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, p in enumerate(per):
        table[b, :p] = torch.tensor(order[:p], dtype=torch.int32)
        order = order[p:]
    s["table"] = table.to(dev)
    rows = torch.tensor([held, [n + 1000 if n > 0 else n for n in held]], dtype=torch.int64, device=dev)
    s["rows"], s["rows_before"] = rows, rows.clone()
    s["lens"], s["clocks"] = rows[0], rows[1]
    s["k_pages"] = rnd(pool, H, page, d, dtype=dt)
    s["v_pages"] = rnd(pool, H, page, d, dtype=dt)
    # weights as attention leaves them: a few heavy pairs, many light ones, some that nothing has attended to
    w = torch.exp(2.0 * rnd(pool, H, page))
    s["mass"] = torch.where(torch.rand(pool, H, page, generator=gen, device=dev) < 0.01, torch.zeros_like(w), w)
    # positions of the held pairs, in an order of their own within each row
    pos = torch.zeros(pool, H, page, dtype=torch.int32, device=dev)
    idx, ok = _places(s, width * page, torch.zeros(B, dtype=torch.int64, device=dev), s["lens"].clamp(min=0))
    perm = torch.where(ok, torch.rand(B, H, width * page, generator=gen, device=dev), 2.0).argsort(dim=-1, stable=True).argsort(dim=-1)
    pos.view(-1)[idx[ok]] = (perm[ok] + 3).to(torch.int32)
    s["pos"] = pos
    s["lam"] = torch.sigmoid(3 + 4 * torch.rand(H, generator=gen, device=dev))
    s["eta"] = 0.1 + 0.9 * torch.rand(H, generator=gen, device=dev)
    s["A"] = rnd(B, H, d, d)
    if c["kind"] in ("append", "evict", "step"):
        Hq = c.get("Hq", 0)
        row = rnd(B, T, Hq + 2 * H, d, dtype=dt).transpose(1, 2)  # slices of a fused projection
        s["q"] = row[:, :Hq] if Hq else None
        s["k"], s["v"] = row[:, Hq:Hq + H], row[:, Hq + H:]
        s["counts"] = torch.tensor(counts(c), dtype=torch.int64, device=dev) if c.get("ragged") and T > 1 else None
        s["mass_in"] = torch.exp(2.0 * rnd(B, H, T)) if T > 1 else None
        s["q_out"] = torch.zeros(B, Hq, T, d, dtype=dt, device=dev) if c["kind"] == "append" else None
    if c["kind"] in ("attend", "step"):
        Hq = c["Hq"]
        s["gate"] = rnd(Hq) if c["memory"] else None
        s["q1"] = rnd(B, Hq, d, dtype=dt) if c["kind"] == "attend" else s["q"].reshape(B, Hq, d)
        s["y"] = torch.zeros(B, Hq, d, dtype=dt, device=dev)
    if own:
        import sliding_window_attention_tc_b200 as tc
        s["tc"] = tc
        memory = c["kind"] in ("evict", "step") or c.get("memory")
        s["cache"] = tc.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["clocks"], mass=s["mass"], pos=s["pos"],
                                   A=s["A"] if memory else None, lam=s["lam"], eta=s["eta"])
        s["rotary"] = _rotary(tc, c) if "rot" in c else None
        if c["kind"] == "attend":
            s["ws"] = tc.cache_attend_workspace(s["cache"], c["Hq"], accumulate=c["mass"])
        elif c["kind"] == "evict":
            s["ws"] = tc.cache_evict_workspace(s["cache"])
        elif c["kind"] == "step":
            s["k1"], s["v1"] = s["k"].reshape(B, H, d), s["v"].reshape(B, H, d)
            s["ws"] = tc.cache_step_workspace(s["cache"], c["Hq"], accumulate=c["mass"])
    return s


def _rotary(tc, c):
    return tc.Rotary(rot=c["rot"], base=c["base"], interleaved=c["inter"], factor=c["factor"], low=c["low"], high=c["high"],
                     train_len=c["train"], gain=c["gain"])


# ---- one pass ---------------------------------------------------------------

def run(s):
    c, kind = s["c"], s["kind"]
    if own:
        tc = s["tc"]
        if kind == "rotate":
            return tc.rotate(s["q"], s["k"], s["rotary"], positions=s["positions"], t0=c["t0"], q_out=s["q_out"], k_out=s["k_out"])
        if kind == "rotate_backward":
            return tc.rotate_backward(s["q"], s["k"], s["rotary"], positions=s["positions"], t0=c["t0"], dq_out=s["q_out"],
                                      dk_out=s["k_out"])
        if kind == "attend":
            tc.cache_attend(s["cache"], s["q1"], g=s["gate"], accumulate=c["mass"], y=s["y"], workspace=s["ws"])
        elif kind == "step":
            tc.cache_step(s["cache"], s["q1"], s["k1"], s["v1"], c["budget"], rotary=s["rotary"], recent=c["recent"], g=s["gate"],
                          accumulate=c["mass"], y=s["y"], workspace=s["ws"])
        else:
            if kind == "append":
                s["rows"].copy_(s["rows_before"])
            tc.cache_append(s["cache"], s["k"], s["v"], rotary=s["rotary"], q=s["q"], counts=s["counts"], mass=s["mass_in"],
                            q_out=s["q_out"])
            if kind == "evict":
                tc.cache_evict(s["cache"], c["budget"], recent=c["recent"], workspace=s["ws"])
        return _outputs(s)
    if kind in ("rotate", "rotate_backward"):
        sign = 1.0 if kind == "rotate" else -1.0
        p = s["positions"]
        p = c["t0"] + torch.arange(c["T"], device=s["q"].device).expand(c["B"], -1) if p is None else p
        cos, sin = _angles(c, p)
        return _turn(s["q"], cos, sign * sin, c), _turn(s["k"], cos, sign * sin, c)
    if kind == "append":
        s["rows"].copy_(s["rows_before"])
    q = s.get("q1")
    if kind in ("append", "evict", "step"):
        turned = _append(s)
        q = turned.reshape(q.shape) if kind == "step" else q
    if kind in ("evict", "step"):
        _evict(s)
    if kind in ("attend", "step"):
        _attend(s, q)
    return _outputs(s)


def _outputs(s):
    """What the call wrote: the cache's state, and y or the rotated queries."""
    kind = s["kind"]
    if kind == "attend":
        return {"y": s["y"], "mass": s["mass"]}
    out = {n: s[n] for n in ("k_pages", "v_pages", "mass", "pos", "lens", "clocks")}
    if kind in ("evict", "step"):
        out["A"] = s["A"]
    if kind == "step":
        out["y"] = s["y"]
    elif kind == "append":
        out["q"] = s["q_out"]
    return out


def _angles(c, p):
    """cos and sin [B,T,rot/2] at the positions p [B,T]: the angles in 64 bits (float32 has no far positions)."""
    half = c["rot"] // 2
    f = c["base"] ** (-torch.arange(half, device=p.device, dtype=torch.float64) / half) if half else p.new_zeros(0, dtype=torch.float64)
    turns = c["train"] * f / (2 * math.pi)
    keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1) if c["high"] > c["low"] else torch.zeros_like(f)
    a = p.to(torch.float64)[..., None] * (f * (keep + (1 - keep) / c["factor"]))
    return (c["gain"] * torch.cos(a)).float(), (c["gain"] * torch.sin(a)).float()


def _turn(x, cos, sin, c):
    """x [B,H,T,d] turned by the angles [B,T,rot/2]."""
    rot, half, f = c["rot"], c["rot"] // 2, x.float()
    cos, sin = cos[:, None], sin[:, None]
    a, b = (f[..., 0:rot:2], f[..., 1:rot:2]) if c["inter"] else (f[..., :half], f[..., half:rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    head = torch.stack((u, w), -1).flatten(-2) if c["inter"] else torch.cat((u, w), -1)
    return torch.cat((head, f[..., rot:]), -1).to(x.dtype).contiguous()


def _places(s, n, start, count):
    """Flat places [B,H,n] in [pool,H,page] of the slots start .. start+n-1 of each row, and which of them are below start + count."""
    H, page, table = s["c"]["H"], s["c"]["page"], s["table"]
    slot = start[:, None] + torch.arange(n, device=table.device)
    slot_in = slot.clamp(max=table.shape[1] * page - 1)
    pg = table.gather(1, slot_in // page).clamp(min=0).long()
    h = torch.arange(H, device=table.device)[None, :, None]
    idx = (pg[:, None] * H + h) * page + (slot_in % page)[:, None]
    return idx, (torch.arange(n, device=table.device) < count[:, None])[:, None].expand_as(idx)


def _append(s):
    c, B, H, T, d = s["c"], s["c"]["B"], s["c"]["H"], s["c"]["T"], s["c"]["d"]
    live = s["lens"] >= 0
    cnt = s["counts"] if s["counts"] is not None else torch.full_like(s["lens"], T)
    cnt = torch.where(live, cnt, 0)
    p = s["clocks"][:, None] + torch.arange(T, device=cnt.device)
    cos, sin = _angles(c, p) if "rot" in c else (None, None)
    k = _turn(s["k"], cos, sin, c) if "rot" in c else s["k"]
    idx, ok = _places(s, T, s["lens"].clamp(min=0), cnt)
    for pages, new in ((s["k_pages"], k), (s["v_pages"], s["v"])):
        pages.view(-1, d)[idx[ok]] = new[ok]
    s["mass"].view(-1)[idx[ok]] = (torch.zeros(B, H, T, device=p.device) if s["mass_in"] is None else s["mass_in"])[ok]
    s["pos"].view(-1)[idx[ok]] = p[:, None].expand(B, H, T)[ok].to(torch.int32)
    q = None
    if s["q"] is not None:
        q = _turn(s["q"], cos, sin, c)
        if s["q_out"] is not None:
            some = (torch.arange(T, device=cnt.device) < cnt[:, None])[:, None, :, None]
            s["q_out"].copy_(torch.where(some, q, s["q_out"]))
    s["lens"] += cnt
    s["clocks"] += cnt
    return q


def _evict(s):
    c = s["c"]
    H, T, d, budget = c["H"], c["T"], c["d"], c["budget"]
    N = s["table"].shape[1] * c["page"]
    n = s["lens"].clamp(min=0)
    m = (n - budget).clamp(min=0)  # at most T: no row held more than the budget before
    idx, ok = _places(s, N, torch.zeros_like(n), n)
    mass, pos = s["mass"].view(-1)[idx], s["pos"].view(-1)[idx]
    # the pairs in the order in which they would leave: unprotected first, then by weight, then by position
    rank = torch.where(ok, (pos >= (s["clocks"] - c["recent"])[:, None, None]).int(), 2)
    order = pos.argsort(dim=-1, stable=True)
    order = order.gather(-1, mass.gather(-1, order).argsort(dim=-1, stable=True))
    order = order.gather(-1, rank.gather(-1, order).argsort(dim=-1, stable=True))
    i = torch.arange(min(T, N), device=n.device)
    gone = order[..., :T]
    leaves = (i < m[:, None])[:, None].expand_as(gone)
    at = idx.gather(-1, gone)
    k, v = (s[x].view(-1, d)[at].float() for x in ("k_pages", "v_pages"))
    l2 = torch.log2(s["lam"].double())[None, :, None]
    w = torch.where(leaves, torch.exp2((m[:, None] - 1 - i).clamp(min=0)[:, None] * l2).float(), 0.0) * s["eta"][None, :, None]
    keep = torch.exp2(m[:, None] * l2[..., 0]).float()[..., None, None]
    k, v = (torch.where(leaves[..., None], x, 0.0) for x in (k, v))
    s["A"].copy_(keep * s["A"] + (k * w[..., None]).transpose(-1, -2) @ v)
    # the survivors behind the budget fill the freed slots before it, both in ascending order
    out = torch.zeros_like(ok).scatter_(-1, gone, leaves)
    slot = torch.arange(N, device=n.device)
    hole = torch.where(out & (slot < budget), slot, N).sort(dim=-1).values[..., :T]
    fill = torch.where(ok & ~out & (slot >= budget), slot, N).sort(dim=-1).values[..., :T]
    b, h, r = torch.nonzero(fill < N, as_tuple=True)
    src, dst = idx[b, h, fill[b, h, r]], idx[b, h, hole[b, h, r]]
    for x in ("k_pages", "v_pages"):
        s[x].view(-1, d)[dst] = s[x].view(-1, d)[src]
    for x in ("mass", "pos"):
        s[x].view(-1)[dst] = s[x].view(-1)[src]
    s["lens"] -= m


def _attend(s, q):
    c = s["c"]
    B, H, d = c["B"], c["H"], c["d"]
    N = s["table"].shape[1] * c["page"]
    n = s["lens"].clamp(min=0)
    idx, ok = _places(s, N, torch.zeros_like(n), n)
    k, v = (torch.where(ok[..., None], s[x].view(-1, d)[idx].float(), 0.0) for x in ("k_pages", "v_pages"))
    qf = q.float().view(B, H, -1, d)
    z = torch.where(ok[:, :, None], (qf @ k.transpose(-1, -2)) / math.sqrt(d), -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    e = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    y = e @ v
    if c["memory"]:
        y = y + torch.sigmoid(s["gate"]).view(1, H, -1, 1) * (qf @ s["A"])
    if c["mass"]:
        s["mass"].view(-1).index_add_(0, idx.reshape(-1), torch.where(ok, e.sum(2), 0.0).reshape(-1))
    s["y"].copy_(torch.where((s["lens"] >= 0)[:, None, None], y.reshape(B, -1, d).to(s["y"].dtype), s["y"]))


# ---- the definition, in 64 bits, one row and head after another ---------------

def exact(c, seed):
    if own:
        raise RuntimeError("exact() goes by the definition alone")
    s = prepare(c, seed)
    D, d = torch.float64, c["d"]

    def freq(i):
        f = c["base"] ** (-2.0 * i / c["rot"])
        t = c["train"] * f / (2.0 * math.pi)
        r = min(1.0, max(0.0, (t - c["low"]) / (c["high"] - c["low"]))) if c["high"] > c["low"] else 0.0
        return f * (r + (1.0 - r) / c["factor"])

    def turned(x, p, sign=1.0):  # x [..., T, d] at positions p [T]
        y = x.to(D).clone()
        for i in range(c["rot"] // 2):
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + c["rot"] // 2)
            ang = p.to(D) * freq(i)
            co, si = c["gain"] * ang.cos(), sign * c["gain"] * ang.sin()
            u, w = x[..., a].to(D), x[..., b].to(D)
            y[..., a], y[..., b] = u * co - w * si, u * si + w * co
        return y

    if c["kind"] in ("rotate", "rotate_backward"):
        sign = 1.0 if c["kind"] == "rotate" else -1.0
        rows = [s["positions"][b] if s["positions"] is not None else c["t0"] + torch.arange(c["T"], device="cuda") for b in range(c["B"])]
        return tuple(torch.stack([turned(s[x][b], rows[b], sign) for b in range(c["B"])]) for x in ("q", "k"))

    held, cl, table, page, H = s["lens"].tolist(), s["clocks"].tolist(), s["table"].cpu(), c["page"], c["H"]
    kp, vp, mass, pos, A = s["k_pages"].to(D), s["v_pages"].to(D), s["mass"].to(D), s["pos"], s["A"].to(D)
    qn = s["q_out"].to(D) if s.get("q_out") is not None else None
    y = s["y"].to(D) if "y" in s else None
    cnt = counts(c) if c["kind"] == "append" else [c.get("T", 0)] * c["B"]
    lam, eta = s["lam"].to(D), s["eta"].to(D)
    for b, n in enumerate(held):
        if n < 0:
            continue
        at = lambda j: (table[b][j // page].long().cuda(), (j % page).cuda())  # noqa: E731
        q1 = s["q1"][b].to(D) if "q1" in s else None
        if c["kind"] in ("append", "evict", "step"):
            t = cnt[b]
            p = cl[b] + torch.arange(t, device="cuda")
            pg, sl = at(n + torch.arange(t))
            new = turned(s["k"][b][:, :t], p) if "rot" in c else s["k"][b][:, :t].to(D)
            # where later parts of the call read the stored key or the rotated query, they read it in the cache's type
            held_in = (lambda x: x.to(DT[c["dtype"]]).to(D)) if c["kind"] == "step" else (lambda x: x)
            kp[pg, :, sl] = held_in(new).transpose(0, 1)
            vp[pg, :, sl] = s["v"][b][:, :t].transpose(0, 1).to(D)
            mass[pg, :, sl] = s["mass_in"][b][:, :t].transpose(0, 1).to(D) if s["mass_in"] is not None else 0.0
            pos[pg, :, sl] = p[:, None].expand(-1, H).to(torch.int32)
            if s["q"] is not None:
                new = held_in(turned(s["q"][b][:, :t], p))
                if c["kind"] == "append":
                    qn[b, :, :t] = new
                q1 = new[:, 0]
            n, cl[b] = n + t, cl[b] + t
        if c["kind"] in ("evict", "step") and n > c["budget"]:
            m, keep = n - c["budget"], c["budget"]
            pg, sl = at(torch.arange(n))
            ms, ps = mass[pg, :, sl].cpu(), pos[pg, :, sl].cpu()
            for h in range(H):
                w, z = ms[:, h].tolist(), ps[:, h].tolist()
                first = sorted(range(n), key=lambda j: (z[j] >= cl[b] - c["recent"], w[j], z[j]))[:m]
                f = torch.tensor(first)
                lw = eta[h] * lam[h] ** torch.arange(m - 1, -1, -1, device="cuda", dtype=D)
                kk, vv = kp[pg[f], h, sl[f]], vp[pg[f], h, sl[f]]
                A[b, h] = lam[h] ** m * A[b, h] + (kk * lw[:, None]).T @ vv
                gone = set(first)
                free, tail = sorted(j for j in gone if j < keep), [j for j in range(keep, n) if j not in gone]
                if free:
                    g, u = torch.tensor(free), torch.tensor(tail)
                    for x in (kp, vp, mass, pos):
                        x[pg[g], h, sl[g]] = x[pg[u], h, sl[u]]
            n = keep
        held[b] = n
        if c["kind"] in ("attend", "step"):
            pg, sl = at(torch.arange(n))
            for h in range(H):
                G = c["Hq"] // H
                qq, out = q1[h * G:(h + 1) * G], torch.zeros(G, d, dtype=D, device="cuda")
                if n:
                    pr = torch.softmax(qq @ kp[pg, h, sl].T / d ** 0.5, -1)
                    out = pr @ vp[pg, h, sl]
                    if c["mass"]:
                        mass[pg, h, sl] += pr.sum(0)
                if c["memory"]:
                    out = out + torch.sigmoid(s["gate"][h * G:(h + 1) * G].to(D))[:, None] * (qq @ A[b, h])
                y[b, h * G:(h + 1) * G] = out
    new = dict(s, k_pages=kp, v_pages=vp, mass=mass, pos=pos, A=A, y=y, q_out=qn, lens=torch.tensor(held), clocks=torch.tensor(cl))
    return _outputs(new)
