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
