"""tc_rotate against the rotation's formula in float64.

Bound: cos and sin come from sincospif (two units in the last place, 2^-23) at
an angle exact to 2^-32 of a turn and rounded once more (2^-24 of at most an
eighth of a turn), are scaled by gain (2^-24), and enter two products and a sum
(2^-24 each): less than 2^-21 of gain (|x| + |z|).  bf16 results are rounded
once more, by half a step (2^-8) of the result at most.
"""
import math

import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LONG = dict(base=500000.0, factor=8.0, low=1.0, high=4.0, train_len=4096, gain=1.25)


def check(got, x, pos, spec, backward=False):
    """x [B,H,T,d], pos [B,T] on the CPU."""
    want = torch.stack([ref.turn(x[b], pos[b], spec, backward) for b in range(x.shape[0])])
    half, rot = spec["rot"] // 2, spec["rot"]
    mag = x.to(torch.float64).abs()
    a = mag.clone()
    if spec.get("interleaved"):
        a[..., :rot] = (mag[..., 0:rot:2] + mag[..., 1:rot:2]).repeat_interleave(2, -1)
    else:
        a[..., :rot] = (mag[..., :half] + mag[..., half:rot]).repeat(1, 1, 1, 2)
    tol = 2.0 ** -21 * abs(spec.get("gain", 1.0)) * a
    if got.dtype == torch.bfloat16:
        tol = tol + torch.finfo(torch.bfloat16).eps / 2 * (want.abs() + tol)
    g = got.to(torch.float64).cpu()
    assert torch.all((g - want).abs() <= tol), float(((g - want).abs() - tol).max())
    assert torch.equal(g[..., rot:], x.to(torch.float64)[..., rot:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 32, True), (128, 64, False), (128, 128, True), (32, 32, False),
                                         (80, 48, True), (66, 10, False), (5, 4, False), (7, 2, True), (16, 0, False)])
@pytest.mark.parametrize("B,Hq,H,T", [(2, 4, 2, 37), (1, 1, 1, 1), (3, 5, 0, 8)])
def test_forward_and_backward(cuda_device, dtype, d, rot, inter, B, Hq, H, T):
    import sliding_window_attention_tc_b200 as tc
    gen = torch.Generator().manual_seed(d * 100 + rot + T)
    q, k = (torch.randn(B, h, T, d, generator=gen).to(DT[dtype]) for h in (Hq, H))
    spec = dict(rot=rot, interleaved=inter, **(LONG if d == 128 else {}))
    r = tc.Rotary(**spec)
    t0 = 1000
    pos = (t0 + torch.arange(T)).expand(B, T)
    kd = k.to(cuda_device) if H else None
    for fn, back in ((tc.rotate, False), (tc.rotate_backward, True)):
        qo, ko = fn(q.to(cuda_device), kd, r, t0=t0)
        check(qo, q, pos, spec, back)
        if H:
            check(ko, k, pos, spec, back)
        else:
            assert ko is None
    assert tc.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_and_negative_positions(cuda_device, dtype):
    import sliding_window_attention_tc_b200 as tc
    B, T, d = 2, 6, 64
    gen = torch.Generator().manual_seed(3)
    q = torch.randn(B, 2, T, d, generator=gen).to(DT[dtype])
    pos = torch.tensor([[0, 1, 1 << 20, (1 << 31) - 1, -5, 16777217], [7, 7, 7, 99999999, 123456789, 3]])
    for spec in (dict(rot=64), dict(rot=64, interleaved=True, **LONG)):
        # 64-bit angles of positions near 2^31 are off by 2^31 2^-52 themselves
        qo, _ = tc.rotate(q.to(cuda_device), None, tc.Rotary(**spec), positions=pos.to(cuda_device))
        check(qo, q, pos, spec)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_broadcast_in_place(cuda_device, dtype):
    import sliding_window_attention_tc_b200 as tc
    B, T, Hq, H, d = 2, 19, 4, 2, 64
    gen = torch.Generator().manual_seed(5)
    spec = dict(rot=64)
    r = tc.Rotary(**spec)
    pos = torch.arange(T).expand(B, T)
    for pad in (0, 8, 3):  # 3: rows off 16-byte boundaries
        row = torch.randn(B, T, (Hq + H) * d + pad, generator=gen).to(DT[dtype])
        dev = row.to(cuda_device)
        view = lambda x, a, h: x[..., a * d:(a + h) * d].unflatten(-1, (h, d)).transpose(1, 2)  # noqa: E731
        qo, ko = tc.rotate(view(dev, 0, Hq), view(dev, Hq, H), r)
        check(qo, view(row, 0, Hq), pos, spec)
        check(ko, view(row, Hq, H), pos, spec)
        tc.rotate(view(dev, 0, Hq), view(dev, Hq, H), r, q_out=view(dev, 0, Hq), k_out=view(dev, Hq, H))
        assert torch.equal(view(dev, 0, Hq), qo) and torch.equal(view(dev, Hq, H), ko)
        assert torch.equal(dev[..., (Hq + H) * d:].cpu(), row[..., (Hq + H) * d:])  # the padding is as it was
    one = torch.randn(1, 1, T, d, generator=gen).to(DT[dtype])
    wide = one.to(cuda_device).expand(B, Hq, T, d)
    qo, _ = tc.rotate(wide, None, r)
    check(qo, one.expand(B, Hq, T, d), pos, spec)


def test_backward_is_the_gradient(cuda_device):
    """<rotate(x + e) - rotate(x - e), dy> / 2e = <e, rotate_backward(dy)>: the
    rotation is linear, so differences are exact up to rounding."""
    import sliding_window_attention_tc_b200 as tc
    B, H, T, d = 2, 3, 33, 64
    gen = torch.Generator().manual_seed(8)
    x, e, dy = (torch.randn(B, H, T, d, generator=gen).to(cuda_device) for _ in range(3))
    for spec in (dict(rot=64), dict(rot=32, interleaved=True, gain=1.5)):
        r = tc.Rotary(**spec)
        hi, lo = tc.rotate(x + e, None, r, t0=5)[0], tc.rotate(x - e, None, r, t0=5)[0]
        left = ((hi.double() - lo.double()) / 2 * dy.double()).sum()
        right = (e.double() * tc.rotate_backward(dy, None, r, t0=5)[0].double()).sum()
        # three float32 results within 2^-21 of their rows' magnitudes, inputs x +- e rounded (2^-24)
        mag = float(((x.abs() + e.abs()).double() * dy.double().abs()).sum()) * 2 * spec.get("gain", 1.0)
        assert abs(float(left - right)) <= 4 * 2.0 ** -21 * mag


def test_gradients_through_rotation_and_layer(cuda_device):
    """Rotation, the layer, and back: dq, dk of the unrotated inputs against
    autograd of the same function in float64."""
    import sliding_window_attention_tc_b200 as tc
    B, H, T, d, W = 1, 2, 40, 32, 8
    gen = torch.Generator().manual_seed(11)
    q, k, v, dy = (torch.randn(B, H, T, d, generator=gen) * 0.5 for _ in range(4))
    lam, eta, g = torch.tensor([0.95, 0.9]), torch.tensor([0.5, 0.3]), torch.tensor([0.2, -0.4])
    spec = dict(rot=32)
    r = tc.Rotary(**spec)
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    qr, kr = tc.rotate(dev(q), dev(k), r)
    dq, dk, *_ = tc.backward(qr, kr, dev(v), dev(lam), dev(eta), dev(g), W, dev(dy))
    dq, dk = tc.rotate_backward(dq, dk, r)
    q6, k6 = (t.double().requires_grad_() for t in (q, k))
    ang = torch.arange(T).double()[:, None] * torch.tensor(ref.frequencies(32)).double()
    rot = lambda x: torch.cat((x[..., :16] * ang.cos() - x[..., 16:] * ang.sin(),  # noqa: E731
                               x[..., :16] * ang.sin() + x[..., 16:] * ang.cos()), -1)
    qq, kk, vv = rot(q6), rot(k6), v.double()
    i, j = torch.arange(T)[:, None], torch.arange(T)[None]
    band = (j <= i) & (j > i - W)
    s = (qq @ kk.transpose(-1, -2) / math.sqrt(d)).masked_fill(~band, -math.inf)
    y = torch.softmax(s, -1) @ vv
    w = torch.where(j <= i - W, lam.double()[:, None, None] ** (i - W - j).clamp(min=0), 0.0) * eta.double()[:, None, None]
    y = y + torch.sigmoid(g.double())[:, None, None] * ((qq @ kk.transpose(-1, -2) * w) @ vv)
    (y * dy.double()).sum().backward()
    for a, b in ((dq, q6.grad), (dk, k6.grad)):
        assert (a.double().cpu() - b).norm() <= 1e-5 * b.norm()  # the float32 backward's own tolerance


def test_two_streams_and_a_captured_graph(cuda_device):
    import sliding_window_attention_tc_b200 as tc
    B, H, T, d = 2, 4, 65, 64
    gen = torch.Generator().manual_seed(13)
    x = torch.randn(B, H, T, d, generator=gen).to(cuda_device)
    r = tc.Rotary(64)
    want = tc.rotate(x, None, r)[0].clone()
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tc.rotate(x, None, r, q_out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
