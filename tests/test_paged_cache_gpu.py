"""The paged cache's calls against their definitions in float64.

Bounds.  Stored keys: the rotation's (2^-21 of the pair's magnitudes), one
rounding to the cache's type.  Outputs: paged_reference.Cache.attend's bound,
and half a step of a bf16 result.  Weights: a softmax weight off by the factor
of its score's error, twice (its own and the sum's), float32 additions.  A: m
products and sums, each off by 2^-23 at most of the sum of magnitudes, and the
decay factors by 2^-21.  What is moved or copied, positions and lengths are exact.
"""
import math
import random

import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(held, d=64, H=2, page=16, room=40, dtype="bf16", seed=0, memory=True, spare=3, nan_behind=True, width=None):
    """A device cache whose rows hold `held` pairs (scattered pages, positions in
    a random order, some equal weights), NaN behind the rows, and its CPU twin."""
    import sliding_window_attention_tc_b200 as tc
    gen = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    per = [(max(0, n) + room + page - 1) // page for n in held]
    B, width, pool = len(held), width or max(max(per), 1), sum(per) + spare
    order = list(range(pool))
    rng.shuffle(order)
    table = torch.full((B, width), -1, dtype=torch.int32)
    k, v = (torch.randn(pool, H, page, d, generator=gen).to(DT[dtype]) for _ in range(2))
    mass = torch.exp(2 * torch.randn(pool, H, page, generator=gen))
    mass[torch.rand(pool, H, page, generator=gen) < 0.2] = 0.5
    pos = torch.zeros(pool, H, page, dtype=torch.int32)
    if nan_behind:
        k0, v0 = torch.full_like(k, math.nan), torch.full_like(v, math.nan)
        k0[::2], v0[::2] = math.inf, -math.inf
    else:
        k0, v0 = k.clone(), v.clone()
    for b, n in enumerate(held):
        for i in range(per[b]):
            table[b, i] = order.pop()
        if n > 0:
            s = torch.arange(n)
            pg, sl = table[b][s // page].long(), s % page
            for h in range(H):
                pos[pg, h, sl] = torch.randperm(n, generator=gen).to(torch.int32)
            k0[pg, :, sl], v0[pg, :, sl] = k[pg, :, sl], v[pg, :, sl]
    lens = torch.tensor(held, dtype=torch.int64)
    clocks = torch.where(lens > 0, lens + 5, lens)
    lam, eta = 0.9 + 0.1 * torch.rand(H, generator=gen), 0.1 + torch.rand(H, generator=gen)
    A = torch.randn(B, H, d, d, generator=gen)
    kw = dict(A=A, lam=lam, eta=eta) if memory else {}
    cpu = ref.Cache(k0, v0, table, lens, clocks, mass, pos, **kw)
    dev = torch.device("cuda")
    c = tc.PagedCache(*(t.to(dev) for t in (k0, v0, table, lens, clocks)), mass=mass.to(dev), pos=pos.to(dev),
                      **{n: t.to(dev) for n, t in kw.items()})
    return c, cpu


def same_state(c, cpu, A_terms=0, exact_keys=True, mass_tol=None):
    """The device cache against its twin."""
    assert c.lens.tolist() == cpu.lens and c.clocks.tolist() == cpu.clocks
    assert torch.equal(c.pos.cpu().long(), cpu.pos)
    bits = lambda t: torch.nan_to_num(t.double(), nan=1e30, posinf=2e30, neginf=-2e30)  # noqa: E731
    assert torch.equal(bits(c.v_pages.cpu()), bits(cpu.v))
    got, want = bits(c.k_pages.cpu()), bits(cpu.k)
    if exact_keys:
        assert torch.equal(got, want)
    else:  # rotated: rounded from values 2^-21 of the pair's magnitudes apart
        step = torch.finfo(c.k_pages.dtype).eps if c.k_pages.dtype == torch.bfloat16 else 0.0
        assert torch.all((got - want).abs() <= step * want.abs() + 2.0 ** -20 * 8)
    m = c.mass.double().cpu()
    tol = 0.0 if mass_tol is None else mass_tol
    assert torch.all((m - cpu.mass).abs() <= tol), float((m - cpu.mass).abs().max())
    if cpu.A is not None:
        err = (c.A.double().cpu() - cpu.A).abs()
        assert torch.all(err <= (A_terms + 32) * 2.0 ** -23 * cpu.A_abs), float((err / cpu.A_abs).max())


def check_y(y, want, tol):
    if y.dtype == torch.bfloat16:
        tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (want.abs() + tol)
    else:
        tol = tol + 2.0 ** -24 * want.abs()
    g = y.double().cpu()
    assert torch.all((g - want).abs() <= tol), float(((g - want).abs() - tol).max())


# scores of unit-variance rows stay below about 6 sqrt(d)/... : (d + 4) 2^-23 sum|qk|/sqrt(d) < 2^-12
# for d <= 128, doubled for the sum; per pair weights are at most 1 a head
MASS_TOL = 2.0 ** -11


# ---- insertion --------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,spec", [(64, dict(rot=64)), (128, dict(rot=64, interleaved=True, factor=4.0)), (16, dict(rot=6)), (32, None)])
@pytest.mark.parametrize("T", [1, 3, 29])
@pytest.mark.parametrize("fused", [False, True])
def test_append(cuda_device, dtype, d, spec, T, fused):
    import sliding_window_attention_tc_b200 as tc
    held, H, Hq = [0, 15, 16, -1, 7], 2, 4
    c, cpu = make(held, d=d, H=H, dtype=dtype, seed=T + d)
    gen = torch.Generator().manual_seed(77)
    B = len(held)
    if fused:
        row = torch.randn(B, T, Hq + 2 * H, d, generator=gen).to(DT[dtype]).transpose(1, 2)
        q, k, v = row[:, :Hq], row[:, Hq:Hq + H], row[:, Hq + H:]
        dev = row.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        qd, kd, vd = dev[:, :Hq], dev[:, Hq:Hq + H], dev[:, Hq + H:]
    else:
        q, k, v = (torch.randn(B, h, T, d, generator=gen).to(DT[dtype]) for h in (Hq, H, H))
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    counts = torch.tensor([T, max(0, T - 1), 0, T, T], dtype=torch.int64) if T > 1 else None
    mass = torch.rand(B, H, T, generator=gen) if T > 1 else None
    r = tc.Rotary(**spec) if spec else None
    q_out = torch.full((B, Hq, T, d), 9.0, dtype=DT[dtype], device=cuda_device)
    got = tc.cache_append(c, kd, vd, rotary=r, q=qd, counts=None if counts is None else counts.cuda(),
                          mass=None if mass is None else mass.cuda(), q_out=q_out)
    assert got is q_out
    want_q = cpu.append(k, v, spec, q, counts, mass)
    same_state(c, cpu, exact_keys=spec is None)
    assert tc.device_status() == 0
    for b, n in enumerate(held):
        t = 0 if n < 0 else T if counts is None else int(counts[b])
        assert torch.all(q_out[b, :, t:] == 9.0)
        if t:
            x, w = q_out[b, :, :t].double().cpu(), want_q[b, :, :t]
            eps = torch.finfo(DT[dtype]).eps / 2
            assert torch.all((x - w).abs() <= eps * w.abs() + 2.0 ** -20 * 10)


def test_append_continues_and_skips_bad_rows(cuda_device):
    """Rows that do not fit, bad counts and bad pages are skipped whole and
    reported; the others go on; the clock keeps counting past the held pairs."""
    import sliding_window_attention_tc_b200 as tc
    held, H, d, T = [10, 50, 4, 8, 3], 2, 64, 4
    c, cpu = make(held, H=H, d=d, room=8, seed=4, width=4)  # 64 slots a row at most
    cap = c.table.shape[1] * 16
    c.lens[1] = cap - 2
    cpu.lens[1] = cap - 2  # does not fit
    c.table[2, 0] = 10 ** 6  # a bad page
    c.clocks[3] = 2 ** 31 - 2  # positions would pass 2^31 - 1
    cpu.clocks[3] = 2 ** 31 - 2
    counts = torch.tensor([4, 4, 4, 4, 5]).cuda()  # the last one above T
    k, v = (torch.randn(5, H, T, d).bfloat16().cuda() for _ in range(2))
    before = [t.clone() for t in (c.k_pages, c.v_pages, c.mass, c.pos)]
    tc.cache_append(c, k, v, counts=counts)
    assert tc.device_status() == 5
    assert c.lens.tolist() == [14, cap - 2, 4, 8, 3]
    pg = c.table[0, :1].long()
    changed = (c.pos != before[3]).any(-1).any(-1).nonzero().flatten()
    assert changed.tolist() == pg.tolist()
    assert torch.equal(c.k_pages[pg[0], :, 10:14], k[0])


# ---- attention ----------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("H,G", [(2, 1), (3, 2), (1, 5), (2, 8), (1, 12), (1, 19)])
def test_attend(cuda_device, dtype, d, H, G):
    import sliding_window_attention_tc_b200 as tc
    held = [1, 0, 63, -1, 64, 65, 200, 16, 17]
    c, cpu = make(held, d=d, H=H, page=16 if d < 64 else 48, dtype=dtype, seed=d + G)
    gen = torch.Generator().manual_seed(G)
    q = torch.randn(len(held), H * G, d, generator=gen).to(DT[dtype])
    g = torch.randn(H * G, generator=gen)
    for gate, acc in ((g, True), (None, False), (g, False), (None, True)):
        y = torch.full(q.shape, 7.0, dtype=DT[dtype], device=cuda_device)
        tc.cache_attend(c, q.cuda(), g=None if gate is None else gate.cuda(), accumulate=acc, y=y)
        want, tol = cpu.attend(q, gate, acc)
        assert torch.all(y[3] == 7.0)
        y[3] = 0
        check_y(y, want, tol)
        same_state(c, cpu, mass_tol=2 * G * MASS_TOL)
    assert tc.device_status() == 0


@pytest.mark.parametrize("dtype,d,H,G,held,page", [
    ("bf16", 128, 2, 4, [5000, 3], 64), ("bf16", 64, 1, 1, [9001], 16), ("bf16", 128, 1, 16, [4097], 128),
    ("f32", 64, 2, 3, [3001, 800], 32), ("f32", 128, 1, 8, [2500], 4096), ("bf16", 64, 4, 2, [130] * 40 + [-1, 0, 2000], 32)])
def test_attend_long_and_many(cuda_device, dtype, d, H, G, held, page):
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make(held, d=d, H=H, page=page, dtype=dtype, seed=page, room=0)
    gen = torch.Generator().manual_seed(1)
    q = torch.randn(len(held), H * G, d, generator=gen).to(DT[dtype])
    g = torch.randn(H * G, generator=gen)
    y = torch.zeros(q.shape, dtype=DT[dtype], device=cuda_device)
    tc.cache_attend(c, q.cuda(), g=g.cuda(), accumulate=True, y=y)
    check_y(y, *cpu.attend(q, g, True))
    same_state(c, cpu, mass_tol=2 * G * MASS_TOL)
    again = torch.zeros_like(y)
    tc.cache_attend(c, q.cuda(), g=g.cuda(), y=again)
    assert torch.equal(again, y)  # a fixed order of every sum
    assert tc.device_status() == 0


def test_attend_large_scores_and_sparse_rows(cuda_device):
    """Scores far apart (one pair takes all), all equal, and a maximum that
    rises tile after tile."""
    import sliding_window_attention_tc_b200 as tc
    for dtype in ("f32", "bf16"):
        c, cpu = make([300, 300, 300], d=64, H=1, dtype=dtype, seed=2)
        for x in (c.k_pages, cpu.k):
            for b in range(3):
                s = torch.arange(300)
                pg, sl = c.table[b].cpu()[s // 16].long(), s % 16
                ramp = (s[:, None, None].float() / 8).expand(-1, 1, 64) / 8
                val = ramp if b == 0 else torch.zeros(300, 1, 64) if b == 1 else ramp.flip(0)
                x[pg.to(x.device), :, sl.to(x.device)] = val.to(x.dtype).to(x.device)
        q = torch.full((3, 2, 64), 2.0).to(DT[dtype])
        y = tc.cache_attend(c, q.cuda(), accumulate=True)
        check_y(y, *cpu.attend(q, None, True))
        same_state(c, cpu, mass_tol=2 * 2.0 ** -8)  # scores up to 600: the bound above scales with them


def test_attend_leaves_bad_pages_out(cuda_device):
    import sliding_window_attention_tc_b200 as tc
    for dtype in ("f32", "bf16"):
        c, cpu = make([40, 16, 5], d=64, H=2, dtype=dtype, seed=6)
        bad = [-7, 2 ** 30]
        c.table[0, 1], cpu.table[0, 1] = bad[0], bad[0]
        c.table[1, 0], cpu.table[1, 0] = bad[1], bad[1]
        q = torch.randn(3, 2, 64).to(DT[dtype])
        mass = c.mass.clone()
        y = tc.cache_attend(c, q.cuda(), g=torch.zeros(2).cuda(), accumulate=True)
        assert tc.device_status() == 5
        check_y(y, *cpu.attend(q, torch.zeros(2), True, bad_pages=bad))
        assert torch.all((c.mass - mass).cpu().double() >= 0)
        # a length past the table: the row is skipped
        c.lens[2] = 10 ** 7
        y2 = torch.full_like(y, 3.0)
        tc.cache_attend(c, q.cuda(), y=y2)
        assert tc.device_status() == 5 and torch.all(y2[2] == 3.0)


# ---- eviction -------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,H", [(64, 2), (128, 1), (16, 3), (32, 2)])
@pytest.mark.parametrize("held,budget,recent", [([33, 32, 31, -1, 0, 33], 32, 4), ([40, 200, 33, 64], 32, 7), ([50, 3], 1, 0),
                                                ([300, 299, 150], 100, 100)])
def test_evict(cuda_device, dtype, d, H, held, budget, recent):
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make(held, d=d, H=H, dtype=dtype, seed=budget + d)
    tc.cache_evict(c, budget, recent=recent)
    cpu.evict(budget, recent)
    same_state(c, cpu, A_terms=max(held))
    assert tc.device_status() == 0
    tc.cache_evict(c, budget, recent=recent)  # nothing left to do: nothing changes
    same_state(c, cpu, A_terms=max(held))


@pytest.mark.parametrize("m", [2, 3, 9, 10, 11, 12, 33, 64])
def test_evict_few_and_more(cuda_device, m):
    """Numbers around the one up to which pairs are picked one after the other, in
    rows longer than a block has threads, many heads to a cluster."""
    import sliding_window_attention_tc_b200 as tc
    held = [600 + m, 600, 1300, 600 + m] + [40 + m] * 40
    c, cpu = make(held, d=16, H=9, dtype="f32", seed=m, room=0)
    for budget in (600, 40):
        tc.cache_evict(c, budget, recent=16)
        cpu.evict(budget, 16)
        same_state(c, cpu, A_terms=1300)
    assert tc.device_status() == 0


def test_evict_odd_weights(cuda_device):
    """Zeros of both signs, infinities, NaN, negative weights, equal positions,
    a recent window wider than the budget; no memory; decays 0, 1 and negative."""
    import sliding_window_attention_tc_b200 as tc
    odd = [0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, -1.0, 3.4e38]
    for memory in (True, False):
        for m in (1, 20):
            c, cpu = make([40 + m, 40 + m], d=64, H=3, seed=m, memory=memory)
            for b in range(2):
                for i in range(40 + m):
                    pg, sl = cpu.at(b, [i])
                    val = odd[(i * 7 + b) % len(odd)]
                    c.mass[pg.cuda(), :, sl.cuda()] = val
                    cpu.mass[pg, :, sl] = torch.tensor(val, dtype=torch.float32).double()
            if memory:
                for x in (c.lam, cpu.lam):
                    x[0], x[1], x[2] = 0.0, 1.0, -0.5
            tc.cache_evict(c, 40, recent=1000 if m == 1 else 12)
            cpu.evict(40, 1000 if m == 1 else 12)
            cpu.mass = torch.nan_to_num(cpu.mass, nan=1e38, posinf=2e38, neginf=-2e38)
            c.mass.copy_(torch.nan_to_num(c.mass, nan=1e38, posinf=2e38, neginf=-2e38))
            cpu.mass = cpu.mass.float().double()
            same_state(c, cpu, A_terms=40)


@pytest.mark.parametrize("kind", ["zeros", "zeros and one value", "two groups", "ten groups", "close", "equal positions", "behind"])
def test_evict_crowded_weights(cuda_device, kind):
    """Weights that crowd: many zeros, groups of equal ones (more of them than are
    taken apart one by one, too), neighbours far from the rest, equal positions."""
    import sliding_window_attention_tc_b200 as tc
    n = 1500
    c, cpu = make([n, 700, n], d=16, H=2, dtype="f32", seed=len(kind), room=0)
    gen = torch.Generator().manual_seed(len(kind))
    for b in range(3):
        held = cpu.lens[b]
        pg, sl = cpu.at(b, range(held))
        i = torch.arange(held)
        rare = torch.exp(4 * torch.randn(held, generator=gen))
        w = {"zeros": torch.where(i % 10 == 3, rare, 0.0), "zeros and one value": (i % 4 == 1) * 2.5,
             "two groups": torch.where(i % 3 == 0, 0.25, torch.where(i % 3 == 1, 3.0, rare)),
             "ten groups": 2.0 ** (i % 10), "close": torch.where(i % 7 == 0, rare * 1e20, 1.0 + (i * 977 % held) * 2.0 ** -23),
             "equal positions": torch.where(i % 5 == 0, rare, 7.0), "behind": torch.where(i % 2 == 0, 1e-3 * rare, 1e30)}[kind].float()
        for x in (c.mass, cpu.mass):
            x[pg.to(x.device), :, sl.to(x.device)] = w[:, None].to(x)
        if kind == "equal positions":
            for x in (c.pos, cpu.pos):
                x[pg.to(x.device), :, sl.to(x.device)] = (i // 200)[:, None].to(x)
    for budget in (1100, 640, 300):
        tc.cache_evict(c, budget, recent=40)
        cpu.evict(budget, 40)
        same_state(c, cpu, A_terms=n)
    assert tc.device_status() == 0


def test_evict_many_pairs_at_once(cuda_device):
    """More pairs than are sorted in shared memory, and the same just below."""
    import sliding_window_attention_tc_b200 as tc
    for held, budget in (([8000, 100], 5000), ([9000, 8300], 8100)):
        c, cpu = make(held, d=16, H=1, page=64, seed=budget, dtype="f32")
        tc.cache_evict(c, budget, recent=32)
        cpu.evict(budget, 32)
        same_state(c, cpu, A_terms=4000)


def test_evict_skips_bad_rows(cuda_device):
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make([60, 60, 60], d=64, H=2, seed=9)
    c.table[1, 2] = -3
    A1 = c.A[1].clone()
    c.lens[2] = 10 ** 6
    tc.cache_evict(c, 30, recent=2)
    assert tc.device_status() == 5
    assert c.lens.tolist() == [30, 60, 10 ** 6] and torch.equal(c.A[1], A1)
    cpu.lens = [60, 0, 0]
    cpu.evict(30, 2)
    assert torch.equal(c.pos.cpu().long(), cpu.pos)


def test_equal_weights_are_the_sliding_window(cuda_device):
    """With every weight equal the oldest pair leaves, as in the layer: a prompt
    appended and evicted to W pairs leaves the window and the A of tc_prefill,
    and its steps give tc_decode_step's outputs."""
    import oracle
    import sliding_window_attention_tc_b200 as tc
    import workloads as wl
    B, H, d, W, T, steps = 2, 2, 64, 32, 150, 40
    x = wl.random_prefill(B, H, T + steps, d, d, W, 16, dtype="f32", seed=21)
    dev = cuda_device
    c = tc.PagedCache.empty(B, H, d, 16, 64, 20, lam=x.lam.to(dev), eta=x.eta.to(dev), dtype=torch.float32)
    c.table.copy_(torch.randperm(40).view(2, 20).to(torch.int32))
    tc.cache_append(c, x.k[:, :, :T].to(dev), x.v[:, :, :T].to(dev))
    tc.cache_evict(c, W)
    yo, Ao = oracle.prefill(x.q[:, :, :T], x.k[:, :, :T], x.v[:, :, :T], x.lam, x.eta, x.g, W)
    Ao = torch.from_numpy(Ao)
    assert (c.A.double().cpu() - Ao).abs().max() <= 1e-5 * Ao.abs().max()
    assert c.lens.tolist() == [W, W] and c.clocks.tolist() == [T, T]
    yo, Ao = oracle.prefill(x.q, x.k, x.v, x.lam, x.eta, x.g, W)
    for t in range(T, T + steps):
        y = tc.cache_step(c, *(z[:, :, t].to(dev).contiguous() for z in (x.q, x.k, x.v)), W, g=x.g.to(dev), accumulate=False)
        want = torch.from_numpy(yo[:, :, t])
        assert (y.double().cpu() - want).abs().max() <= 1e-5 * want.abs().max()
    Ao = torch.from_numpy(Ao)
    assert (c.A.double().cpu() - Ao).abs().max() <= 1e-5 * Ao.abs().max()
    assert tc.device_status() == 0


# ---- the calls together -----------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,H,G,spec,memory", [("bf16", 64, 2, 4, dict(rot=64), True), ("f32", 128, 1, 3, dict(rot=32, interleaved=True), True),
                                                     ("bf16", 128, 3, 1, None, True), ("f32", 16, 2, 2, dict(rot=16), False)])
def test_step_is_append_evict_attend(cuda_device, dtype, d, H, G, spec, memory):
    """cache_step against the three calls (the same bits in the state) and against
    the definition, over steps that cross the budget and a page's end."""
    import sliding_window_attention_tc_b200 as tc
    held, budget, recent, steps = [20, 31, 32, 17, -1, 0, 29], 32, 3, 5
    a, cpu = make(held, d=d, H=H, dtype=dtype, seed=d, memory=memory)
    b, _ = make(held, d=d, H=H, dtype=dtype, seed=d, memory=memory)
    gen = torch.Generator().manual_seed(31)
    B, Hq = len(held), H * G
    g = torch.randn(Hq, generator=gen) if memory else None
    gd = None if g is None else g.cuda()
    r = tc.Rotary(**spec) if spec else None
    for i in range(steps):
        row = torch.randn(B, Hq + 2 * H, d, generator=gen).to(DT[dtype])
        q, k, v = row[:, :Hq], row[:, Hq:Hq + H], row[:, Hq + H:]
        dev = row.cuda()
        y = torch.full((B, Hq, d), 7.0, dtype=DT[dtype], device=cuda_device)
        y3 = y.clone()
        # slices of one projection, and on odd steps contiguous tensors
        qkv = (dev[:, :Hq], dev[:, Hq:Hq + H], dev[:, Hq + H:]) if i % 2 == 0 else (q.cuda(), k.cuda(), v.cuda())
        tc.cache_step(a, *qkv, budget, rotary=r, recent=recent, g=gd, y=y)
        q_rot = torch.zeros(B, Hq, 1, d, dtype=DT[dtype], device=cuda_device)
        tc.cache_append(b, k.cuda()[:, :, None], v.cuda()[:, :, None], rotary=r, q=q.cuda()[:, :, None], q_out=q_rot)
        tc.cache_evict(b, budget, recent=recent)
        tc.cache_attend(b, q_rot[:, :, 0].contiguous(), g=gd, accumulate=True, y=y3)
        bits = lambda t: torch.nan_to_num(t.double(), nan=1e30, posinf=2e30, neginf=-2e30)  # noqa: E731
        for n in ("k_pages", "v_pages", "pos", "lens", "clocks"):
            assert torch.equal(bits(getattr(a, n)), bits(getattr(b, n))), n
        assert (a.mass - b.mass).abs().max() <= 1e-5 * a.mass.abs().max()
        if memory:
            assert (a.A - b.A).abs().max() <= 1e-5 * a.A.abs().max()
        cpu.append(k[:, :, None], v[:, :, None], spec)
        cpu.evict(budget, recent)
        # the device's own rotated queries and keys: one rounding apart from the twin's at most
        cpu.k, keep = a.k_pages.cpu().clone(), cpu.k
        want, tol = cpu.attend(q_rot[:, :, 0].cpu(), g, True)
        assert torch.all(y[4] == 7.0) and torch.all(y3[4] == 7.0)
        y[4], y3[4] = 0, 0
        check_y(y, want, tol)
        check_y(y3, want, tol)
    same_state(a, cpu, A_terms=64, mass_tol=2 * steps * G * MASS_TOL)
    assert tc.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_many_rows(cuda_device, dtype):
    """Enough rows that a head's A is no longer cut finer to fill the device."""
    import sliding_window_attention_tc_b200 as tc
    held, H, G, d, budget = [31, 20, 32, 0] * 45, 2, 2, 128, 32
    c, cpu = make(held, d=d, H=H, dtype=dtype, seed=15, room=16)
    gen = torch.Generator().manual_seed(16)
    q, k, v = (torch.randn(len(held), h, d, generator=gen).to(DT[dtype]) for h in (H * G, H, H))
    g = torch.randn(H * G, generator=gen)
    for _ in range(2):
        y = tc.cache_step(c, q.cuda(), k.cuda(), v.cuda(), budget, g=g.cuda())
        cpu.append(k[:, :, None], v[:, :, None])
        cpu.evict(budget, 1)
        check_y(y, *cpu.attend(q, g, True))
    same_state(c, cpu, A_terms=4, mass_tol=4 * G * MASS_TOL)
    assert tc.device_status() == 0


def test_step_above_the_budget_keeps_its_distance(cuda_device):
    """A row above its budget lets one pair leave a step, the least attended one."""
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make([50, 20], H=2, seed=12, width=6)
    q, k, v = (torch.randn(2, h, 64).bfloat16() for h in (4, 2, 2))
    for i in range(3):
        tc.cache_step(c, q.cuda(), k.cuda(), v.cuda(), 32, accumulate=False)
        cpu.append(k[:, :, None], v[:, :, None])
        n1 = cpu.lens[1]
        cpu.lens[1] = 0
        cpu.evict(50, 1)
        cpu.lens[1] = n1
        same_state(c, cpu, A_terms=8)
    assert c.lens.tolist() == [50, 23]


def test_captured_step_replays(cuda_device):
    """A captured step, replayed, against eager steps; two graphs with workspaces
    of their own on two streams."""
    import sliding_window_attention_tc_b200 as tc
    held, H, G, d, budget = [32, 10, 32], 2, 2, 64, 32
    gen = torch.Generator().manual_seed(41)
    q, k, v = (torch.randn(3, h, d, generator=gen).bfloat16().cuda() for h in (H * G, H, H))
    g = torch.randn(H * G, generator=gen).cuda()
    caches = [make(held, d=d, H=H, seed=s)[0] for s in (1, 2)]
    eager = [make(held, d=d, H=H, seed=s)[0] for s in (1, 2)]
    r = tc.Rotary(64)
    graphs, ys, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for c, s in zip(caches, streams):
        ws, y = tc.cache_step_workspace(c, H * G), torch.empty_like(q)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            tc.cache_step(c, q, k, v, budget, rotary=r, g=g, y=y, workspace=ws)
        graphs.append((gr, ws))
        ys.append(y)
    torch.cuda.synchronize()
    for _ in range(4):
        for (gr, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for c, e, y in zip(caches, eager, ys):
        for _ in range(4):
            want = tc.cache_step(e, q, k, v, budget, rotary=r, g=g)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(c.pos, e.pos) and torch.equal(c.mass, e.mass) and torch.equal(c.A, e.A)
    assert tc.device_status() == 0


def test_attend_wait_limit(cuda_device):
    """The loads' bounded waits, made to run out: the call reports it and the
    next one is right."""
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make([5000, 700], d=128, H=2, seed=3, page=64)
    q = torch.randn(2, 2, 128).bfloat16()
    try:
        tc.set_wait_limit_ns(1)
        tc.cache_attend(c, q.cuda())
        assert tc.device_status() == 6
    finally:
        tc.set_wait_limit_ns(0)
    check_y(tc.cache_attend(c, q.cuda()), *cpu.attend(q))
    assert tc.device_status() == 0


def test_given_stream_keeps_the_calls_memory(cuda_device):
    """What a call allocates for itself and hands to a stream it was given is not
    dealt again while that stream still has the call before it."""
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make([300, 40], d=64, H=2, seed=5)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(5)).bfloat16()
    qd, side = q.cuda(), torch.cuda.Stream()
    size = tc.cache_attend_workspace(c, 4).nbytes
    torch.cuda.synchronize()
    # the blocks the allocator would deal for a workspace, found by asking for one
    x = torch.empty(size, dtype=torch.uint8, device="cuda")
    at = x.data_ptr()
    del x
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    y = tc.cache_attend(c, qd, stream=side)
    again = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(t.data_ptr() != at for t in again)
    torch.cuda.synchronize()
    check_y(y, *cpu.attend(q))
    assert tc.device_status() == 0


@pytest.mark.parametrize("clock", [2 ** 31 - 4, 2 ** 62, 2 ** 63 - 1, -1])
def test_clocks_past_the_last_position(cuda_device, clock):
    """Tokens whose positions would pass 2^31 - 1 do not enter, however far the
    clock is; a step refuses a clock that is there."""
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make([20, 20], d=64, H=2, seed=6)
    c.clocks[1] = clock
    k, v = torch.randn(2, 2, 2, 5, 64, generator=torch.Generator().manual_seed(6)).bfloat16()
    tc.cache_append(c, k.cuda(), v.cuda())
    assert tc.device_status() == 5
    assert c.lens.tolist() == [25, 20] and c.clocks.tolist() == [30, clock]
    pg, sl = cpu.at(1, range(20, 25))
    assert torch.equal(torch.isnan(c.k_pages.cpu()[pg, :, sl]), torch.isnan(cpu.k[pg, :, sl]))
    if clock == 2 ** 31 - 4:
        return
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    tc.cache_step(c, q, q, q, 64)
    assert tc.device_status() == 5 and c.lens.tolist() == [26, 20]


def test_step_needs_room_for_one_more(cuda_device):
    """The pair enters before one leaves: a row whose table is full is left as it
    is, the others go on."""
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make([64, 63], d=64, H=2, seed=7, room=0)
    assert c.table.shape[1] * 16 == 64
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(q, 3.0)
    tc.cache_step(c, q, q, q, 64, y=y)
    assert tc.device_status() == 5
    assert c.lens.tolist() == [64, 64] and c.clocks.tolist() == [cpu.clocks[0], cpu.clocks[1] + 1]
    assert torch.all(y[0] == 3.0) and not torch.any(y[1] == 3.0)
    pg, sl = cpu.at(0, range(64))
    assert torch.equal(c.v_pages.cpu()[pg, :, sl], cpu.v[pg, :, sl])


def test_padded_prompts(cuda_device):
    """A padded batch whose rows have no, one, some or all of the tokens, in more
    than one block a row; NaN in the padding."""
    import sliding_window_attention_tc_b200 as tc
    T, counts = 150, [0, 1, 77, 150, 8, 9, 5]
    for dtype, d, spec in (("f32", 64, dict(rot=64)), ("bf16", 128, dict(rot=64)), ("bf16", 16, dict(rot=16))):
        c, cpu = make([0, 3, 16, 5, 0, 7, -1], d=d, H=3, dtype=dtype, seed=d, room=160)
        gen = torch.Generator().manual_seed(d)
        k, v = torch.randn(2, 7, 3, T, d, generator=gen).to(DT[dtype])
        q = torch.randn(7, 6, T, d, generator=gen).to(DT[dtype])
        for b, n in enumerate(counts):
            for x in (k, v, q):
                x[b, :, n:] = math.nan
        q_out = torch.full_like(q, 3.0).cuda()
        tc.cache_append(c, k.cuda(), v.cuda(), rotary=tc.Rotary(**spec), q=q.cuda(), counts=torch.tensor(counts).cuda(), q_out=q_out)
        want = cpu.append(k, v, spec, q=q, counts=counts)
        same_state(c, cpu, exact_keys=False)
        eps = torch.finfo(DT[dtype]).eps / 2
        for b, n in enumerate(counts):
            n = n if b < 6 else 0
            got = q_out[b].cpu().double()
            assert torch.all(got[:, n:] == 3.0)  # rows past a row's tokens are not written
            assert torch.all((got[:, :n] - want[b, :, :n]).abs() <= eps * want[b, :, :n].abs() + 2.0 ** -20 * 10)
    assert tc.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_offsets_past_32_bits(cuda_device, dtype):
    """The same calls on a small pool and on the last pages of one of more than
    2^31 elements: the same bits."""
    import sliding_window_attention_tc_b200 as tc
    H, G, d, page, B, width = 2, 2, 128, 64, 3, 4
    far = 2 ** 31 // (H * page * d) + 7  # pages whose elements pass 2^31
    perm = torch.randperm(B * width, generator=torch.Generator().manual_seed(1)).view(B, width).int()
    lam, eta = torch.tensor([0.9, 0.97]).cuda(), torch.tensor([0.5, 0.7]).cuda()
    caches = []
    for base in (0, far):
        n = base + B * width
        pool = [torch.empty(n, H, page, d, dtype=DT[dtype], device="cuda") for _ in range(2)]
        c = tc.PagedCache(*pool, (perm + base).cuda(), torch.zeros(B, dtype=torch.int64).cuda(), torch.zeros(B, dtype=torch.int64).cuda(),
                          mass=torch.zeros(n, H, page).cuda(), pos=torch.zeros(n, H, page, dtype=torch.int32).cuda(),
                          A=torch.zeros(B, H, d, d).cuda(), lam=lam, eta=eta)
        for t in (*pool, c.mass, c.pos):
            t[base:].zero_()
        caches.append((c, base))
    gen = torch.Generator().manual_seed(2)
    r = tc.Rotary(d)
    k, v = torch.randn(2, B, H, 150, d, generator=gen).to(DT[dtype]).cuda()
    w = torch.rand(B, H, 150, generator=gen).cuda()
    q = torch.randn(B, H * G, d, generator=gen).to(DT[dtype]).cuda()
    g = torch.randn(H * G, generator=gen).cuda()
    out = []
    for c, base in caches:
        ys = []
        tc.cache_append(c, k, v, rotary=r, mass=w)
        ys.append(tc.cache_attend(c, q, g=g, accumulate=True))
        tc.cache_evict(c, 100, recent=8)
        ys.append(tc.cache_attend(c, q, g=g))
        tc.cache_append(c, k[:, :, :1], v[:, :, :1], rotary=r)
        tc.cache_evict(c, 100, recent=8)
        for i in range(3):
            ys.append(tc.cache_step(c, q, k[:, :, i], v[:, :, i], 100, rotary=r, g=g))
        out.append(ys + [c.A, c.lens, c.clocks] + [t[base:] for t in (c.k_pages, c.v_pages, c.mass, c.pos)])
    for a, b in zip(*out):
        assert torch.equal(a, b) and not torch.any(torch.isnan(a.double()))
    assert tc.device_status() == 0
