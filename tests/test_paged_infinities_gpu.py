"""Infinite keys and values of pairs that count: what the definition makes
infinite is infinite, what it makes NaN is NaN, the rest is as it would be."""
import math

import pytest
import torch

from test_paged_cache_gpu import DT, make

pytestmark = pytest.mark.gpu


def same(got, want, tol):
    got, want, tol = got.double().cpu(), want.double(), tol.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    far = torch.isinf(want)
    assert torch.equal(got[far], want[far])
    at = torch.isfinite(want)
    assert torch.all((got - want).abs()[at] <= tol[at]), float(((got - want).abs() - tol)[at].max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,H,G,page", [(64, 2, 1, 16), (128, 1, 12, 64), (16, 2, 3, 16), (32, 1, 8, 48)])
def test_attend(cuda_device, dtype, d, H, G, page):
    """A row of one pair, a few and many (split over blocks); columns with one
    infinity, two of a sign, two of both (NaN), a NaN; weights that fit bf16."""
    import sliding_window_attention_tc_b200 as tc
    held = [1, 2, 40, 3000, 16]
    c, cpu = make(held, d=d, H=H, page=page, dtype=dtype, seed=d, room=0)
    for b, n in enumerate(held):
        for col, slots, vals in ((0, [0], [math.inf]), (1, [0, n - 1], [-math.inf, -math.inf]), (2, [0, n - 1], [math.inf, -math.inf]),
                                 (3, [n // 2], [math.nan]), (5, [n // 3], [-math.inf])):
            for slot, val in zip(slots, vals):
                pg, sl = cpu.at(b, [slot])
                for x in (c.v_pages, cpu.v):
                    x[pg.to(x.device), :, sl.to(x.device), col] = val
    q = torch.randn(len(held), H * G, d, generator=torch.Generator().manual_seed(G)).to(DT[dtype])
    q[4] = 0  # sixteen pairs of equal weight
    g = torch.randn(H * G, generator=torch.Generator().manual_seed(1))
    for gate in (None, g):
        want, tol = cpu.attend(q, gate)
        # half a step of a bf16 result (2^-8), of a float32 one 2^-24
        tol = tol + torch.finfo(DT[dtype]).eps / 2 * (want.abs() + tol)
        same(tc.cache_attend(c, q.cuda(), g=None if gate is None else gate.cuda()), want, tol)
    assert tc.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,H,rows", [(64, 2, 3), (128, 1, 3), (16, 2, 3), (64, 8, 40), (128, 4, 30)])
@pytest.mark.parametrize("m", [1, 2, 12, 300])
def test_evict(cuda_device, dtype, d, H, rows, m):
    """Pairs that leave with infinite keys, values or both; of both signs (NaN),
    against a zero (NaN), a NaN; ones that fit bf16."""
    import sliding_window_attention_tc_b200 as tc
    budget = 30
    c, cpu = make([budget + m] * rows, d=d, H=H, dtype=dtype, seed=m + d, room=0)
    for b in range(rows):
        slots = range(budget + m)
        pg, sl = cpu.at(b, slots)
        put = lambda x, y, i, col, val: [t.__setitem__((pg[i].to(t.device), slice(None), sl[i].to(t.device), col), val) for t in (x, y)]  # noqa: E731
        for x in (c.mass, cpu.mass):  # the first m slots leave, in their order
            x[pg.to(x.device), :, sl.to(x.device)] = torch.arange(budget + m)[:, None].to(x)
        kk, vv = (c.k_pages, cpu.k), (c.v_pages, cpu.v)
        for i in range(0, m, 5):  # values that fit bf16's first part, so that a float32's other parts are 0
            put(*vv, i, slice(8, 12), 0.5)
        put(*vv, 0, 0, math.inf)
        put(*vv, m - 1, 1, -math.inf)
        if b % 3 == 1:
            put(*kk, m // 2, 2, math.inf)
            put(*vv, m // 2, 4, -math.inf)
            put(*vv, m // 2, 5, 0.0)  # inf * 0
        if b % 3 == 2 and m > 1:
            put(*vv, m - 1, 0, -math.inf)
            put(*vv, m // 2, 3, math.nan)
    tc.cache_evict(c, budget, recent=1)
    cpu.evict(budget, 1)
    assert c.lens.tolist() == cpu.lens and torch.equal(c.pos.cpu().long(), cpu.pos)
    assert torch.isinf(cpu.A).any() and torch.isfinite(cpu.A).any()
    same(c.A, cpu.A, (m + 32) * 2.0 ** -23 * cpu.A_abs)
    assert tc.device_status() == 0
