"""Bounded waits of the paged attention that run out: the call reports it, copies
that are under way have landed before their block's memory is given back, rows
that were not read to the end keep their weights, and the next call is right."""
import pytest
import torch

from paged_bounds import weights
from test_paged_cache_gpu import check_y, make

pytestmark = pytest.mark.gpu


# one tile a block, a few (fewer and more than a ring holds), boxes of 16 to 128 rows
@pytest.mark.parametrize("held,d,H,G,page", [([5000, 700], 128, 2, 1, 64), ([300, 0, -1, 40], 64, 2, 4, 16),
                                             ([9000] * 6, 128, 8, 4, 128), ([6000] * 8, 64, 8, 12, 16)])
@pytest.mark.parametrize("limit", [1, 2000, 8000])
def test_a_wait_that_runs_out_leaves_the_weights(cuda_device, held, d, H, G, page, limit):
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make(held, d=d, H=H, seed=3, page=page, room=0, memory=False)
    q = torch.randn(len(held), H * G, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    grow, tol, at = weights(cpu, q)
    before, qd = c.mass.clone(), q.cuda()
    for _ in range(3):
        try:
            tc.set_wait_limit_ns(limit)
            tc.cache_attend(c, qd, accumulate=True)
            status = tc.device_status()
        finally:
            tc.set_wait_limit_ns(0)
        assert status in ((6,) if limit == 1 else (0, 6))
        got, old = c.mass.double().cpu(), before.double().cpu()
        assert torch.equal(got[~at], old[~at])
        kept = 0
        for b, n in enumerate(cpu.lens):
            pg, sl = cpu.at(b, range(max(n, 0)))
            for h in range(H):
                was, now = old[pg, h, sl], got[pg, h, sl]
                if not torch.equal(was, now):
                    assert torch.all((now - was - grow[pg, h, sl]).abs() <= tol[pg, h, sl])
                    kept += 1
        if status == 0:
            assert kept == H * sum(n > 0 for n in held)
        c.mass.copy_(before)
    want = cpu.attend(q)
    # (rows that are empty are not written)
    check_y(tc.cache_attend(c, qd, accumulate=True, y=torch.zeros_like(qd)), *want)
    assert torch.all((c.mass.double().cpu() - before.double().cpu() - grow).abs()[at] <= tol[at])
    assert tc.device_status() == 0


def test_a_step_whose_wait_runs_out_has_moved_its_pairs(cuda_device):
    """The state of a step that was cut short is the state after the step, its
    weights aside."""
    import sliding_window_attention_tc_b200 as tc
    held, H, G, d, budget = [32, 10, 33 * 16, 32], 2, 2, 128, 32
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(4, h, d, generator=gen).bfloat16().cuda() for h in (H * G, H, H))
    (a, _), (b, _) = (make(held, d=d, H=H, seed=4) for _ in range(2))
    try:
        tc.set_wait_limit_ns(1)
        tc.cache_step(a, q, k, v, budget)
        assert tc.device_status() == 6
    finally:
        tc.set_wait_limit_ns(0)
    tc.cache_step(b, q, k, v, budget, accumulate=False)
    for n in ("pos", "lens", "clocks", "A"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    for n in ("k_pages", "v_pages"):
        assert torch.equal(getattr(a, n).view(torch.int16), getattr(b, n).view(torch.int16)), n
    assert torch.all(a.mass >= b.mass)
    assert tc.device_status() == 0
