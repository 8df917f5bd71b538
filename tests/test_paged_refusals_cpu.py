"""Refusals of the rotary and paged-cache calls (CPU only): the C-ABI's codes for
invalid arguments before any device work, the no-device answer for valid ones,
and the binding's own errors."""
import ctypes

import pytest
import torch

import sliding_window_attention_tc_b200 as tc

HAS_GPU = torch.cuda.is_available()
OK, INVALID, UNSUPPORTED, NO_DEVICE = 0, 1, 2, 3
F = 0x100000  # a fake device address, never dereferenced
no_device_only = pytest.mark.skipif(HAS_GPU, reason="checks the no-device answer")
lib = tc.lib_handle()


# ---- tc_rotate ------------------------------------------------------------------
def rotate(spec=None, q=F, k=F + (1 << 24), qo=F + (2 << 24), ko=F + (3 << 24), pos=None, **kw):
    d = dict(B=2, Hq=4, H=2, T=8, d=64, dtype=tc.TC_BF16, flags=0)
    strides = {n: kw.pop(n) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride") if n in kw}
    d.update(kw)
    full = lambda h: (h * d["T"] * d["d"], d["T"] * d["d"], d["d"])  # noqa: E731
    for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride"):
        strides.setdefault(n, full(d["Hq"] if n[0] == "q" else d["H"]))
    desc = tc.RotateDesc(*d.values(), *((ctypes.c_int64 * 3)(*strides[n]) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")))
    r = tc.RotaryC(64, 0, 10000.0, 1.0, 0.0, 0.0, 0.0, 1.0) if spec is None else spec
    return lib.tc_rotate(ctypes.byref(desc), ctypes.byref(r) if r else None, pos, 0, q, k, qo, ko, None)


def spec(**kw):
    d = dict(rot=64, interleaved=0, base=10000.0, factor=1.0, low=0.0, high=0.0, train_len=0.0, gain=1.0)
    d.update(kw)
    return tc.RotaryC(*d.values())


@pytest.mark.parametrize("bad", [dict(rot=3), dict(rot=-2), dict(rot=66), dict(interleaved=2), dict(base=1.0), dict(base=float("nan")),
                                 dict(factor=0.5), dict(factor=float("inf")), dict(gain=float("nan")), dict(train_len=-1.0),
                                 dict(low=float("nan")), dict(high=float("inf"))])
def test_rotary_parameters(bad):
    assert rotate(spec(**bad)) == INVALID


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(H=-1), INVALID), (dict(d=0), INVALID),
    (dict(d=130), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(flags=2), INVALID), (dict(T=1 << 39), UNSUPPORTED),
    (dict(B=1 << 20, T=1 << 20), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(ko=None), INVALID), (dict(q=F + 1), INVALID), (dict(pos=F + 4), INVALID),
    (dict(q_stride=(-1, 512, 64)), INVALID),
    (dict(q_out_stride=(0, 512, 64)), INVALID),       # outputs that overlap themselves
    (dict(k_out_stride=(1024, 512, 32)), INVALID),
    (dict(qo=F + 128), INVALID),                      # an output that meets its input
    (dict(qo=F, q_out_stride=(2048, 64, 256)), INVALID),  # in place with other strides
])
def test_rotate_refuses(bad, code):
    assert rotate(**bad) == code


@no_device_only
def test_rotate_valid_calls_need_a_device():
    assert rotate() == NO_DEVICE
    assert rotate(qo=F, ko=F + (1 << 24)) == NO_DEVICE            # in place
    assert rotate(q_stride=(0, 0, 64)) == NO_DEVICE               # a broadcast input
    assert rotate(H=0, k=None, ko=None) == NO_DEVICE
    assert rotate(T=0, q=None, k=None, qo=None, ko=None) == NO_DEVICE
    assert rotate(q=F + 2, qo=F + (2 << 24) + 2) == NO_DEVICE     # the type's own alignment is enough


# ---- the cache -------------------------------------------------------------------
def cache(**kw):
    d = dict(B=2, H=2, d=64, page=16, n_pages=10, max_pages=4, dtype=tc.TC_BF16, k_pages=F, v_pages=F, mass=F, pos=F, table=F, len=F,
             clock=F, A=F, lam=F, eta=F)
    d.update(kw)
    return tc.PagedCacheC(*d.values())


def append(c, r=None, **kw):
    a = dict(T=3, Hq=4, q=F + (1 << 24), k=F, v=F, q_stride=(768, 192, 64), k_stride=(384, 192, 64), v_stride=(384, 192, 64), counts=None,
             mass_in=None, q_out=F + (2 << 24))
    a.update(kw)
    for n in ("q_stride", "k_stride", "v_stride"):
        a[n] = (ctypes.c_int64 * 3)(*a[n])
    args = tc.AppendArgs(*a.values())
    return lib.tc_cache_append(ctypes.byref(c), ctypes.byref(r) if r else None, ctypes.byref(args), None)


def attend(c, Hq=4, q=F, g=F, y=F, flags=1, ws=F, room=1 << 40):
    return lib.tc_cache_attend(ctypes.byref(c), Hq, q, g, y, flags, ws, room, None)


def evict(c, budget=8, recent=1, ws=F, room=1 << 40):
    return lib.tc_cache_evict(ctypes.byref(c), budget, recent, ws, room, None)


def step(c, r=None, Hq=4, q=F, k=F, v=F, g=F, budget=8, recent=1, y=F, flags=1, ws=F, room=1 << 40, q_stride=(256, 64)):
    I2 = ctypes.c_int64 * 2
    a = tc.StepArgs(Hq, q, k, v, I2(*q_stride), I2(128, 64), I2(128, 64), g, y, budget, recent, flags)
    return lib.tc_cache_step(ctypes.byref(c), ctypes.byref(r) if r else None, ctypes.byref(a), ws, room, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID), (dict(page=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(dtype=3), INVALID), (dict(k_pages=None), INVALID), (dict(table=None), INVALID),
    (dict(len=None), INVALID), (dict(clock=None), INVALID), (dict(mass=None), INVALID), (dict(pos=None), INVALID),
    (dict(lam=None), INVALID), (dict(k_pages=F + 8), INVALID), (dict(len=F + 4), INVALID), (dict(table=F + 2), INVALID),
    (dict(A=F + 8), INVALID),
    (dict(d=48), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=8192), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(B=2048, H=1024), UNSUPPORTED),
    (dict(n_pages=1 << 27), UNSUPPORTED), (dict(max_pages=1 << 21), UNSUPPORTED), (dict(B=65535, max_pages=1 << 20), UNSUPPORTED),
])
def test_every_call_refuses_a_bad_cache(bad, code):
    c = cache(**bad)
    assert append(c) == code and attend(c) == code and evict(c) == code and step(c) == code
    assert lib.tc_cache_attend_workspace_size(ctypes.byref(c), 4, 0) == tc.SIZE_ERROR
    assert lib.tc_cache_evict_workspace_size(ctypes.byref(c)) == tc.SIZE_ERROR
    assert lib.tc_cache_step_workspace_size(ctypes.byref(c), 4, 0) == tc.SIZE_ERROR


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID),
    (dict(Hq=0), INVALID), (dict(k=F + 1), INVALID), (dict(q_out=F + (2 << 24) + 8), INVALID), (dict(counts=F + 4), INVALID),
    (dict(mass_in=F + 2), INVALID), (dict(k_stride=(-1, 192, 64)), INVALID), (dict(q=F, q_out=F), INVALID),
    (dict(r=spec(rot=66)), INVALID)])
def test_append_refuses(bad, code):
    assert append(cache(), **bad) == code


def test_append_mass_needs_a_cache_with_mass():
    assert append(cache(mass=None, pos=None), mass_in=F) == INVALID


@pytest.mark.parametrize("bad,code", [
    (dict(Hq=0), INVALID), (dict(Hq=3), INVALID), (dict(Hq=512), UNSUPPORTED), (dict(q=None), INVALID), (dict(y=None), INVALID),
    (dict(q=F + 8), INVALID), (dict(y=F + 8), INVALID), (dict(ws=F + 8), INVALID), (dict(flags=2), INVALID)])
def test_attend_refuses(bad, code):
    assert attend(cache(), **bad) == code


def test_calls_refuse_what_the_cache_lacks():
    bare = cache(mass=None, pos=None, A=None, lam=None, eta=None)
    assert attend(bare, flags=0) == INVALID            # g without a memory
    assert attend(bare, g=None, flags=1) == INVALID    # accumulation without mass
    assert evict(bare) == INVALID and step(bare, g=None, flags=0) == INVALID


@pytest.mark.parametrize("bad", [dict(budget=0), dict(recent=-1), dict(ws=F + 4)])
def test_evict_and_step_refuse(bad):
    assert evict(cache(), **bad) == INVALID and step(cache(), **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(q=None), dict(k=None), dict(v=F + 1), dict(y=F + 8), dict(q_stride=(256, -64)), dict(Hq=5), dict(r=spec(rot=5))])
def test_step_refuses(bad):
    assert step(cache(), **bad) == INVALID


@no_device_only
def test_valid_calls_need_a_device():
    c = cache()
    assert append(c) == NO_DEVICE and append(c, spec()) == NO_DEVICE and append(c, T=0, q=None, k=None, v=None) == NO_DEVICE
    assert attend(c) == NO_DEVICE and evict(c) == NO_DEVICE and step(c, spec()) == NO_DEVICE
    bare = cache(mass=None, pos=None, A=None, lam=None, eta=None)
    assert append(bare) == NO_DEVICE and attend(bare, g=None, flags=0) == NO_DEVICE


def test_workspace_sizes():
    c = ctypes.byref(cache())
    plain, acc = (lib.tc_cache_attend_workspace_size(c, 4, f) for f in (0, 1))
    assert 0 < plain and acc - plain == 10 * 16 * 4 * 4  # one score a pair and query head
    assert lib.tc_cache_step_workspace_size(c, 4, 1) > acc + lib.tc_cache_evict_workspace_size(c)
    long = ctypes.byref(cache(max_pages=4096, n_pages=8192))  # rows that sort outside shared memory
    assert lib.tc_cache_evict_workspace_size(long) > lib.tc_cache_evict_workspace_size(c) + 4 * 65536 * 12


# ---- the binding --------------------------------------------------------------------
def py_cache(**kw):
    a = dict(B=2, H=2, d=64, page=16, n_pages=6, max_pages=3, lam=torch.ones(2), eta=torch.ones(2), device="cpu")
    a.update(kw)
    return tc.PagedCache.empty(**a)


@pytest.mark.parametrize("name,bad,err", [
    ("v_pages", torch.zeros(6, 2, 16, 32).bfloat16(), ValueError), ("v_pages", torch.zeros(6, 2, 16, 64), TypeError),
    ("table", torch.zeros(2, 3, dtype=torch.int64), TypeError), ("lens", torch.zeros(3, dtype=torch.int64), ValueError),
    ("clocks", torch.zeros(2, dtype=torch.int32), TypeError), ("mass", torch.zeros(6, 2, 8), ValueError), ("pos", torch.zeros(6, 2, 16), TypeError),
    ("pos", None, ValueError), ("A", torch.zeros(2, 2, 64, 32), ValueError), ("lam", None, ValueError), ("eta", torch.ones(3), ValueError)])
def test_cache_construction(name, bad, err):
    c = py_cache()
    kw = {n: getattr(c, n) for n in ("k_pages", "v_pages", "table", "lens", "clocks", "mass", "pos", "A", "lam", "eta")}
    kw[name] = bad
    with pytest.raises(err):
        tc.PagedCache(**kw)


def test_cache_is_fixed():
    c = py_cache()
    with pytest.raises(AttributeError):
        c.lens = c.lens.clone()
    with pytest.raises(AttributeError):
        tc.Rotary(64).base = 3.0
    with pytest.raises(ValueError):
        tc.Rotary(63)


def test_binding_checks():
    c = py_cache()
    q, k = torch.zeros(2, 4, 64).bfloat16(), torch.zeros(2, 2, 64).bfloat16()
    k4 = k[:, :, None]
    for err, call in [
        (ValueError, lambda: tc.cache_append(c, k, k)), (TypeError, lambda: tc.cache_append(c, k4.float(), k4)),
        (ValueError, lambda: tc.cache_append(c, k4, k4[:, :1])), (TypeError, lambda: tc.cache_append(c, k4, k4, counts=torch.zeros(2))),
        (ValueError, lambda: tc.cache_append(c, k4, k4, mass=torch.zeros(2, 2, 2))),
        (ValueError, lambda: tc.cache_append(c, k4, k4, q_out=q)), (ValueError, lambda: tc.cache_append(c, k4, k4, q=q[:, :, None], q_out=q)),
        (ValueError, lambda: tc.cache_append(c, k4.expand(2, 2, 1, 64).transpose(2, 3)[..., :1].expand(2, 2, 64, 64), k4)),
        (ValueError, lambda: tc.cache_attend(c, q[:, :3])), (TypeError, lambda: tc.cache_attend(c, q.float())),
        (ValueError, lambda: tc.cache_attend(c, q, g=torch.zeros(3))), (ValueError, lambda: tc.cache_attend(c, q, y=q[:, :2])),
        (ValueError, lambda: tc.cache_step(c, q, k[:, :1], k, 8)), (TypeError, lambda: tc.cache_step(c, q, k, k.float(), 8)),
        (ValueError, lambda: tc.rotate(q, None, tc.Rotary(64))), (ValueError, lambda: tc.rotate(q[:, :, None], k4[:1], tc.Rotary(64))),
        (TypeError, lambda: tc.rotate(q[:, :, None], k4.float(), tc.Rotary(64))),
        (TypeError, lambda: tc.rotate(q[:, :, None], None, tc.Rotary(64), positions=torch.zeros(2, 1))),
        (ValueError, lambda: tc.rotate(q[:, :, None], None, tc.Rotary(64), k_out=k4)),
    ]:
        with pytest.raises(err):
            call()
    bare = tc.PagedCache(c.k_pages, c.v_pages, c.table, c.lens, c.clocks)
    for call in (lambda: tc.cache_attend(bare, q, g=torch.zeros(4)), lambda: tc.cache_attend(bare, q, accumulate=True),
                 lambda: tc.cache_evict(bare, 8), lambda: tc.cache_step(bare, q, k, k, 8)):
        with pytest.raises(ValueError):
            call()
