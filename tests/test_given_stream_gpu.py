"""Calls that are given a stream and allocate for themselves: the memory may be a
block that the current stream's queued work still writes, and the call comes
after that work."""
import pytest
import torch

from test_paged_cache_gpu import check_y, make, same_state

pytestmark = pytest.mark.gpu


def leave_dirty(hold, *sizes):
    """Blocks of these sizes (bytes), given back to the allocator while a write to
    them is still queued on the current stream; every other one is kept, so that
    they stay blocks of these sizes.  Returns where they are."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(64)]
    torch.cuda._sleep(40_000_000)
    for b in blocks:
        b.fill_(0x7f)  # 3.4e38 in bf16 and float32
    hold += blocks[1::2]
    return {b.data_ptr() for b in blocks[::2]}


def side_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    return s


def test_rotate(cuda_device):
    import sliding_window_attention_tc_b200 as tc
    q, k = (torch.randn(2, h, 33, 64, generator=torch.Generator().manual_seed(h)).cuda() for h in (4, 2))
    r, side, hold = tc.Rotary(64), side_stream(), []
    for fn in (tc.rotate, tc.rotate_backward):
        want = [t.clone() for t in fn(q, k, r)]
        at = leave_dirty(hold, q.nbytes, k.nbytes)
        got = fn(q, k, r, stream=side)
        assert all(t.data_ptr() in at for t in got)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        at = leave_dirty(hold, k.nbytes)
        out = {"q_out" if fn is tc.rotate else "dq_out": torch.empty_like(q)}
        got = fn(q, k, r, stream=side, **out)  # one of the two allocated
        torch.cuda.synchronize()
        assert got[1].data_ptr() in at and torch.equal(got[1], want[1])


def test_the_caches_calls(cuda_device):
    import sliding_window_attention_tc_b200 as tc
    held, d, H, G = [300, 40], 64, 2, 2
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(2, h, d, generator=gen).bfloat16() for h in (H * G, H, H))
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    side, hold = side_stream(), []
    warm, _ = make(held, d=d, H=H, seed=5)  # the first launch of a kernel may wait for the device
    tc.cache_append(warm, kd[:, :, None], vd[:, :, None], q=qd[:, :, None])
    tc.cache_attend(warm, qd)
    tc.cache_evict(warm, 100)
    tc.cache_step(warm, qd, kd, vd, 100, accumulate=False)
    c, cpu = make(held, d=d, H=H, seed=5)
    room = [tc.cache_attend_workspace(c, H * G, accumulate=True).nbytes, tc.cache_evict_workspace(c).nbytes,
            tc.cache_step_workspace(c, H * G).nbytes, q.nbytes]
    at = leave_dirty(hold, *room)
    q_out = tc.cache_append(c, kd[:, :, None], vd[:, :, None], q=qd[:, :, None], stream=side)
    assert q_out.data_ptr() in at
    torch.cuda.synchronize()
    cpu.append(k[:, :, None], v[:, :, None])
    assert torch.equal(q_out[:, :, 0], qd)
    at = leave_dirty(hold, *room)
    y = tc.cache_attend(c, qd, stream=side)
    assert y.data_ptr() in at
    torch.cuda.synchronize()
    check_y(y, *cpu.attend(q))
    at = leave_dirty(hold, *room)
    tc.cache_evict(c, 100, stream=side)
    torch.cuda.synchronize()
    cpu.evict(100, 1)
    same_state(c, cpu, A_terms=300)
    at = leave_dirty(hold, *room)
    y = tc.cache_step(c, qd, kd, vd, 100, accumulate=False, stream=side)
    assert y.data_ptr() in at
    torch.cuda.synchronize()
    cpu.append(k[:, :, None], v[:, :, None])
    cpu.evict(100, 1)
    same_state(c, cpu, A_terms=300)
    check_y(y, *cpu.attend(q))
    assert tc.device_status() == 0


def test_a_captured_call_on_a_stream_of_its_own(cuda_device):
    """The stream given is the captured one, or one that was forked from it."""
    import sliding_window_attention_tc_b200 as tc
    c, cpu = make([70, 40], d=64, H=2, seed=6)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(6)).bfloat16()
    qd, main, side = q.cuda(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        a = tc.cache_attend(c, qd, stream=main)
        side.wait_stream(main)
        b = tc.cache_attend(c, qd, stream=side)
        main.wait_stream(side)
    for y in (a, b):
        y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check_y(a, *cpu.attend(q))
    check_y(b, *cpu.attend(q))
