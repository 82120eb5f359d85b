"""dspark_rotate against the 64-bit formula: both layouts, part of the head, bf16 and fp32, the
inverse, far and negative positions, strided and unaligned rows, in place; the inverse as a
gradient; and the host function that makes the frequencies, with the refusals of both."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from speculative_decoding_ragged_gb300 import _binding as bd

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_ragged_gb300 import build
    build.build()
    return bd.lib()


def test_frequencies(lib):
    # a few roundings of pow and a division (2^-53 each), and the fixed point's quantum, 2^-64 of
    # a turn, by which a value is cut off
    quantum = 2 * np.pi * 2.0 ** -64
    for rot, base in ((128, 10000.0), (64, 500000.0), (2, 10000.0), (96, 1e6)):
        f = base ** (-2.0 * np.arange(rot // 2) / rot)
        got = bd.rope_turns(rot, base).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
        np.testing.assert_allclose(got, f, rtol=1e-14, atol=quantum)
        got = bd.rope_turns(rot, base, "linear", factor=4.0).astype(np.float64) / 2.0 ** 64
        np.testing.assert_allclose(got * 2 * np.pi, f / 4, rtol=1e-14, atol=quantum)
        r = 8192 * f / (2 * np.pi)
        keep = np.clip((r - 1.0) / 31.0, 0, 1)
        got = bd.rope_turns(rot, base, "by_parts", factor=16.0, trained=8192.0)
        np.testing.assert_allclose(got.astype(np.float64) / 2.0 ** 64 * 2 * np.pi,
                                   (1 - keep) * f / 16 + keep * f, rtol=1e-13,
                                   atol=quantum)
    assert bd.rope_turns(0).size == 0


@pytest.mark.parametrize("args", [
    dict(rot=3), dict(rot=-2), dict(rot=2048), dict(rot=8, base=1.0), dict(rot=8, base=np.inf),
    dict(rot=8, scaling=7), dict(rot=8, scaling="linear", factor=0.5),
    dict(rot=8, scaling="by_parts", factor=2.0, trained=0.0),
    dict(rot=8, scaling="by_parts", factor=2.0, trained=10.0, slow=4.0, fast=4.0)])
def test_frequencies_refuse(lib, args):
    with pytest.raises(bd.DSparkError) as err:
        bd.rope_turns(**args)
    assert err.value.code == -1


def test_rotate_refuses_on_the_host(lib):
    import ctypes
    P = ctypes.c_void_p
    ok = bd._Rope(4096, 64, 0, 1.0)

    def call(x=4096, xs=256, y=8192, ys=256, dt=0, rows=3, heads=2, dim=128, pos=4096, rope=ok):
        rc = lib.dspark_rotate(P(x), xs, P(y), ys, dt, rows, heads, dim, P(pos),
                               ctypes.byref(rope) if rope is not None else None, 0, None)
        return rc, bd.last_error()

    for kw, word in [(dict(dt=5), "dtype"), (dict(rows=-1), "rows=-1"), (dict(heads=0), "heads=0"),
                     (dict(dim=0), "dim=0"), (dict(dim=1025, xs=4000, ys=4000), "dim=1025"),
                     (dict(xs=255), "row strides"), (dict(ys=255), "row strides"),
                     (dict(rope=None), "rope"), (dict(rope=bd._Rope(4096, 130, 0, 1.0)), "rot"),
                     (dict(rope=bd._Rope(4096, 63, 0, 1.0)), "rot"),
                     (dict(rope=bd._Rope(None, 64, 0, 1.0)), "turns"),
                     (dict(rope=bd._Rope(4100, 64, 0, 1.0)), "turns"),
                     (dict(rope=bd._Rope(4096, 64, 2, 1.0)), "interleaved"),
                     (dict(rope=bd._Rope(4096, 64, 0, float("nan"))), "mscale"),
                     (dict(x=0), "required"), (dict(y=0), "required"), (dict(pos=0), "required"),
                     (dict(x=4097), "aligned")]:
        rc, msg = call(**kw)
        assert rc == -1 and msg.startswith("dspark_rotate") and word in msg, (kw, rc, msg)
    assert call(rows=0, x=0, y=0, pos=0)[0] == 0


CASES = [
    # rows, heads, dim, rot, interleaved, dtype, inverse, extra columns in a row of x, of y
    (1, 1, 64, 64, False, "bf16", False, 0, 0),
    (16, 40, 128, 128, False, "bf16", False, 256, 0),
    (17, 5, 128, 64, True, "bf16", True, 0, 128),
    (1300, 3, 96, 64, True, "f32", True, 96, 96),
    (5, 3, 80, 16, False, "f32", False, 8, 4),
    (7, 2, 34, 20, False, "bf16", False, 1, 3),      # nothing a multiple of 16: scalar accesses
    (7, 2, 33, 32, True, "f32", False, 0, 0),        # odd head
    (3, 2, 256, 256, True, "bf16", False, 0, 0),
    (2, 1, 1024, 1024, False, "f32", False, 0, 0),
    (9, 4, 64, 0, False, "bf16", False, 0, 0),       # nothing rotated: a copy
    (1500, 2, 512, 512, False, "bf16", False, 0, 0),
]


@gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_rotate(lib, case, in_place):
    rows, heads, dim, rot, inter, dt, inverse, xc, yc = case
    dev = torch.device("cuda:0")
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator().manual_seed(rows + dim + rot)
    full = torch.randn(rows, heads * dim + xc, generator=g).to(dtype)
    x = full[:, :heads * dim].view(rows, heads, dim) if xc == 0 else \
        full.as_strided((rows, heads, dim), (heads * dim + xc, dim, 1))
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows,), generator=g).to(torch.int32)
    pos[: min(rows, 3)] = torch.tensor([0, 1, 2 ** 31 - 1], dtype=torch.int32)[: min(rows, 3)]
    turns = bd.rope_turns(rot, 10000.0)
    mscale = 1.25
    xd = full.to(dev).as_strided(x.shape, x.stride())
    yd = xd if in_place else torch.full((rows, heads * dim + yc), 7.0, dtype=dtype, device=dev) \
        .as_strided((rows, heads, dim), (heads * dim + yc, dim, 1))
    rope = bd.Rope(torch.as_tensor(turns.view(np.int64)).to(dev), mscale, inter)
    bd.dspark_rotate(xd, yd, pos.to(dev), rope, inverse=inverse)
    torch.cuda.synchronize()
    xh = x.double().numpy()
    want = ref.rotate(xh, pos.numpy(), turns, mscale, inter, inverse)
    got = yd.double().cpu().numpy()
    tol = ref.rotate_bound(xh, rot // 2, mscale, inter)
    tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(want) + tol)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())
    np.testing.assert_array_equal(got[..., rot:], xh[..., rot:])     # copied, not rounded
    if not in_place and yc:                                           # nothing past a row's heads
        base = yd.as_strided((rows, yc), (heads * dim + yc, 1), heads * dim)
        assert (base[:-1] == 7.0).all()


@gpu
def test_inverse_is_the_gradient(lib):
    """<R x, g> = <x, R^T g>, and the inverse call's result against central differences."""
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, 2, 64, generator=g).to(dev)
    grad = torch.randn(4, 2, 64, generator=g).to(dev)
    pos = torch.tensor([3, 70, 1000, 123456], dtype=torch.int32, device=dev)
    rope = bd.Rope.make(48, 10000.0, scaling="by_parts", factor=8.0, trained=4096.0,
                        interleaved=True, device=dev)
    y, back = torch.empty_like(x), torch.empty_like(x)

    def loss(z):
        bd.dspark_rotate(z, y, pos, rope)
        return float((y.double() * grad.double()).sum())

    bd.dspark_rotate(grad, back, pos, rope, inverse=True)
    # the loss is linear, so a central difference has no truncation error: only y's fp32
    # rounding, ROTATE_TOL of a pair's |a| + |b| per element, over the step
    step = 4.0
    for at in [(0, 0, 0), (1, 1, 47), (2, 0, 13), (3, 1, 63), (3, 0, 22)]:
        z = x.clone()
        z[at] += step
        up = loss(z)
        z[at] -= 2 * step
        down = loss(z)
        assert abs((up - down) / (2 * step) - float(back[at])) <= \
            2 * ref.ROTATE_TOL * rope.mscale * 2 * (step + 8) * 8 / step


@gpu
def test_rotate_python_refusals(lib):
    dev = torch.device("cuda:0")
    x = torch.zeros(4, 2, 64, device=dev)
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    rope = bd.Rope.make(64, device=dev)
    bd.dspark_rotate(x, x, pos, rope)
    for bad in (lambda: bd.dspark_rotate(x, torch.zeros(4, 2, 32, device=dev), pos, rope),
                lambda: bd.dspark_rotate(x, x.to(torch.bfloat16), pos, rope),
                lambda: bd.dspark_rotate(x.half(), x.half(), pos, rope),
                lambda: bd.dspark_rotate(x, x, pos[:3], rope),
                lambda: bd.dspark_rotate(x, x, pos.long(), rope),
                lambda: bd.dspark_rotate(x.transpose(1, 2), x.transpose(1, 2), pos, rope),
                lambda: bd.dspark_rotate(x.cpu(), x, pos, rope),
                lambda: bd.Rope(torch.zeros(3, device=dev))):
        with pytest.raises(ValueError):
            bad()
    # rows == 0 does nothing
    bd.dspark_rotate(x[:0], x[:0], pos[:0], rope)
