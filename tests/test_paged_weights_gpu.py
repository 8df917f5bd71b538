"""The accumulated weights against bounds in the weights themselves, and their
sums: what a (row, key/value head)'s pairs gain is one for each query head."""
import pytest
import torch

from paged_bounds import weights
from test_paged_cache_gpu import DT, check_y, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,H,G,held,page", [
    # rows over many blocks, where the join has to find every partial
    ("bf16", 128, 2, 4, [5000, 3], 64), ("bf16", 64, 1, 1, [9001], 16), ("bf16", 128, 1, 16, [4097], 128),
    ("f32", 64, 2, 3, [3001, 800], 32), ("f32", 128, 1, 8, [2500], 4096), ("bf16", 64, 4, 2, [130] * 40 + [-1, 0, 2000], 32),
    ("bf16", 128, 1, 19, [20000, 1], 16), ("bf16", 64, 1, 128, [1500, 129], 16), ("f32", 32, 1, 12, [7000], 16), ("f32", 16, 3, 5, [257, 1, 1024], 48),
    # many rows of about a tile, several to a block
    ("bf16", 64, 8, 1, [127, 128, 129, 1] * 40, 16), ("f32", 64, 8, 2, [127, 128, 129, 1] * 20, 16)])
def test_weights(cuda_device, dtype, d, H, G, held, page):
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make(held, d=d, H=H, page=page, dtype=dtype, seed=page + G, room=0, memory=False)
    q = torch.randn(len(held), H * G, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    grow, tol, at = weights(cpu, q)
    before = c.mass.double().cpu()
    y = torch.zeros(q.shape, dtype=DT[dtype], device=cuda_device)
    tc.cache_attend(c, q.cuda(), accumulate=True, y=y)
    got = c.mass.double().cpu() - before
    assert torch.all((got - grow).abs()[at] <= tol[at]), float(((got - grow).abs() / tol)[at].max())
    assert torch.equal(got[~at], torch.zeros_like(got[~at]))
    for b, n in enumerate(held):
        if n > 0:
            pg, sl = cpu.at(b, range(n))
            total, off = got[pg, :, sl].sum(0), tol[pg, :, sl].sum(0)
            assert torch.all((total - G).abs() <= off)
    # from nothing, where the old weights' rounding hides none of it
    c.mass.zero_()
    cpu.mass.zero_()
    _, tol, _ = weights(cpu, q)
    tc.cache_attend(c, q.cuda(), accumulate=True, y=y)
    got = c.mass.double().cpu()
    assert torch.all((got - grow).abs()[at] <= tol[at]), float(((got - grow).abs() / tol)[at].max())
    check_y(y, *cpu.attend(q))
    assert tc.device_status() == 0
