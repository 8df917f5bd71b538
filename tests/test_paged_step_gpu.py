"""Serving steps of many query heads to a key head (more than one pass over A
reads), with and without the memory's read."""
import pytest
import torch

from paged_bounds import weights
from test_paged_cache_gpu import DT, check_y, make, same_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,H,G,rows", [(64, 2, 5, 1), (128, 1, 8, 1), (128, 2, 12, 40), (16, 1, 9, 1), (32, 3, 4, 12), (128, 1, 17, 1)])
@pytest.mark.parametrize("spec", [dict(rot=16), dict(rot=8, interleaved=True, gain=1.5), None])
@pytest.mark.parametrize("gate", [True, False])
def test_step_of_grouped_heads(cuda_device, dtype, d, H, G, rows, spec, gate):
    import sliding_window_attention_tc_b200 as tc
    held, budget, recent = [20, 31, 32, 17, -1, 0, 32] * rows, 32, 3
    c, cpu = make(held, d=d, H=H, dtype=dtype, seed=d + G, room=8)
    gen = torch.Generator().manual_seed(31)
    B, Hq = len(held), H * G
    g = torch.randn(Hq, generator=gen) if gate else None
    r = tc.Rotary(**spec) if spec else None
    for i in range(3):
        q, k, v = (torch.randn(B, h, d, generator=gen).to(DT[dtype]) for h in (Hq, H, H))
        y = torch.full((B, Hq, d), 7.0, dtype=DT[dtype], device=cuda_device)
        # the rotated queries, as an insertion into a cache of nothing gives them (the same bits)
        spare = tc.PagedCache.empty(B, H, d, 16, B, 1, dtype=DT[dtype])
        spare.table.copy_(torch.arange(B)[:, None])
        spare.clocks.copy_(c.clocks.clamp(min=0))
        q_rot = tc.cache_append(spare, k.cuda()[:, :, None], v.cuda()[:, :, None], rotary=r, q=q.cuda()[:, :, None])[:, :, 0].cpu()
        tc.cache_step(c, q.cuda(), k.cuda(), v.cuda(), budget, rotary=r, recent=recent, g=None if g is None else g.cuda(), y=y)
        cpu.append(k[:, :, None], v[:, :, None], spec)
        cpu.evict(budget, recent)
        # rotated keys may be one rounding (bf16: 2^-8 of themselves) apart from the
        # twin's, and with them the pairs written into A: 2^-6 of the magnitudes is
        # 4 such roundings.  What follows goes by the device's own keys and A.
        same_state(c, cpu, exact_keys=spec is None, mass_tol=float("inf"), A_terms=64 if spec is None else 1 << 17)
        cpu.k, cpu.A = c.k_pages.cpu().clone(), c.A.double().cpu()
        grow, tol, at = weights(cpu, q_rot)
        m = c.mass.double().cpu()
        assert torch.all((m - cpu.mass - grow).abs()[at] <= tol[at])
        live = torch.tensor([n >= 0 for n in cpu.lens])
        want, wide = cpu.attend(q_rot, g)
        cpu.mass = torch.where(at, m, cpu.mass)
        assert torch.all(y[~live.cuda()] == 7.0)
        check_y(y[live.cuda()], want[live], wide[live])
    assert tc.device_status() == 0
