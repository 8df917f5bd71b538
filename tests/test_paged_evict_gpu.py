"""Eviction where it can go wrong: pairs that compare as the last of all."""
import math

import pytest
import torch

from test_paged_cache_gpu import make, same_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,H", [(64, 3), (128, 1)])
@pytest.mark.parametrize("pos", [-1, 2 ** 31 - 1])
@pytest.mark.parametrize("m", [1, 2, 9, 10, 11, 40])
@pytest.mark.parametrize("whole", [True, False])
def test_pairs_that_are_the_last_of_all(cuda_device, d, H, pos, m, whole):
    """Weights NaN, the last position (or one that was never set), all protected:
    the earliest slots leave.  Or some such pairs among ordinary ones, which then
    leave first."""
    import sliding_window_attention_tc_b200 as tc
    n, budget = 40 + m, 40
    c, cpu = make([n, n, 30], d=d, H=H, seed=m, room=0)
    for b in range(3):
        slots = range(cpu.lens[b]) if whole else range(0, cpu.lens[b], 3)
        pg, sl = cpu.at(b, slots)
        for x, val in ((c.mass, math.nan), (cpu.mass, math.nan), (c.pos, pos), (cpu.pos, pos)):
            x[pg.to(x.device), :, sl.to(x.device)] = val
    recent = 2 ** 40  # every pair is protected
    tc.cache_evict(c, budget, recent=recent)
    # positions are not negative: -1 sorts by its low 31 bits, as the last one
    cpu.pos = torch.where(cpu.pos < 0, 2 ** 31 - 1, cpu.pos)
    cpu.evict(budget, recent)
    c.pos.copy_(torch.where(c.pos < 0, 2 ** 31 - 1, c.pos))
    for x in (c.mass, cpu.mass):
        x.copy_(torch.nan_to_num(x, nan=1e30))
    cpu.mass = cpu.mass.float().double()
    same_state(c, cpu, A_terms=n)
    assert tc.device_status() == 0


def test_two_threads_whose_tables_differ(cuda_device):
    """Evictions of two host threads at once, from caches whose tables are of
    different sizes (and so ask for different shared memory): neither takes the
    other's leave away."""
    import threading

    import sliding_window_attention_tc_b200 as tc
    made = [make([90, 80], d=64, H=2, seed=1, room=0, width=128 * w) for w in (1, 8)]  # 2048 and 16384 slots a row
    made.append(make([90, 80], d=64, H=2, seed=1, room=0, width=6))
    errors, start = [], threading.Barrier(len(made))

    def work(c, lens):
        try:
            s, ws = torch.cuda.Stream(), tc.cache_evict_workspace(c)
            s.wait_stream(torch.cuda.default_stream())
            start.wait()
            with torch.cuda.stream(s):
                for _ in range(3000):
                    c.lens.copy_(lens)
                    tc.cache_evict(c, 60, workspace=ws)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    lens = [c.lens.clone() for c, _ in made]
    for c, cpu in made:  # the first eviction, checked by itself
        tc.cache_evict(c, 60)
        cpu.evict(60, 1)
        same_state(c, cpu, A_terms=40)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c, n)) for (c, _), n in zip(made, lens)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert all(c.lens.tolist() == [60, 60] for c, _ in made) and tc.device_status() == 0


# (row, head) pairs that take one, two and four blocks each, and bf16 rows of more
# tiles than a block's ring holds
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,H,rows", [(64, 4, 1), (64, 12, 8), (64, 16, 16), (128, 2, 1), (128, 8, 8), (128, 16, 10), (32, 16, 20), (32, 3, 2)])
def test_many_pairs_of_many_heads(cuda_device, dtype, d, H, rows):
    import sliding_window_attention_tc_b200 as tc
    held = [700 + 13 * (b % 5) for b in range(rows)]
    c, cpu = make(held, d=d, H=H, page=64, dtype=dtype, seed=d + rows, room=0)
    tc.cache_evict(c, 64, recent=8)
    evict_fast(cpu, 64, 8)
    same_state(c, cpu, A_terms=max(held))
    assert tc.device_status() == 0


def evict_fast(cpu, budget, recent):
    """paged_reference.Cache.evict with A's sum in one product (float64): the same
    up to float64's rounding, for cases of many heads."""
    for b, n in enumerate(cpu.lens):
        if n <= budget:
            continue
        m = n - budget
        pg, sl = cpu.at(b, range(n))
        for h in range(cpu.H):
            w, z = cpu.mass[pg, h, sl], cpu.pos[pg, h, sl]
            order = sorted(range(n), key=lambda j: (bool(z[j] >= cpu.clocks[b] - recent), float(w[j]), int(z[j]), j))  # noqa: B023
            gone = torch.tensor(order[:m])
            f = cpu.eta[h] * cpu.lam[h] ** torch.arange(m - 1, -1, -1, dtype=torch.float64)
            kk, vv = cpu.k[pg[gone], h, sl[gone]].double(), cpu.v[pg[gone], h, sl[gone]].double()
            cpu.A[b, h] = cpu.lam[h] ** m * cpu.A[b, h] + (kk * f[:, None]).T @ vv
            cpu.A_abs[b, h] = cpu.lam[h] ** m * cpu.A_abs[b, h] + (kk.abs() * f[:, None]).T @ vv.abs()
            left = set(order[:m])
            free = torch.tensor(sorted(j for j in left if j < budget), dtype=torch.int64)
            tail = torch.tensor([j for j in range(budget, n) if j not in left], dtype=torch.int64)
            for x in (cpu.k, cpu.v, cpu.mass, cpu.pos):
                x[pg[free], h, sl[free]] = x[pg[tail], h, sl[tail]]
        cpu.lens[b] = budget


def test_the_fast_twin_is_the_twin():
    """The two forms of the definition agree (on the CPU)."""
    import paged_reference as ref
    gen = torch.Generator().manual_seed(3)
    n, H, d, page = 60, 2, 16, 16
    k, v = torch.randn(2, 4, H, page, d, generator=gen)
    mass = torch.rand(4, H, page, generator=gen)
    pos = torch.stack([torch.randperm(64, generator=gen) for _ in range(H)]).view(H, 4, page).transpose(0, 1).contiguous()
    args = (k, v, torch.tensor([[2, 0, 3, 1]]), torch.tensor([n]), torch.tensor([70]), mass, pos)
    kw = dict(A=torch.randn(1, H, d, d, generator=gen), lam=torch.tensor([0.9, 0.99]), eta=torch.tensor([0.5, 1.0]))
    a, b = ref.Cache(*args, **kw), ref.Cache(*args, **kw)
    a.evict(20, 5)
    evict_fast(b, 20, 5)
    for x in ("k", "v", "mass", "pos"):
        assert torch.equal(getattr(a, x), getattr(b, x))
    assert a.lens == b.lens and torch.allclose(a.A, b.A, rtol=0, atol=1e-12) and torch.allclose(a.A_abs, b.A_abs, rtol=0, atol=1e-12)
