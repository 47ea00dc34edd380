"""Roundings of the rotary positions (needs a B200).

fp32 results are the real numbers mscale (a cos - b sin) and mscale (a sin + b cos), formed in 64 bits and rounded once:
half an fp32 step (2^-24 of the result), plus what 64-bit sines, products and sums of either side are off by, at most
2^-48 of mscale (|a| + |b|), plus half the smallest fp32 number."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import long_context_sparse_11_b200 as dsa  # noqa: E402
from test_gpu_kernels import i32_dev  # noqa: E402
from test_gpu_latent4 import f64, lib  # noqa: E402,F401


def turned(x, pos, plan, offset, backward):
    """x [T, H, D] fp64 turned by the plan's frequencies, and mscale (|a| + |b|) of each value."""
    rot, m = plan.rot_dim, plan.mscale
    angle = pos.astype(np.float64)[:, None] * np.array(plan.inv_freq[:rot // 2])
    c, s = (m * np.cos(angle))[:, None], (m * np.sin(-angle if backward else angle))[:, None]
    at = np.arange(rot // 2)
    ia, ib = (at, at + rot // 2) if plan.layout == 1 else (2 * at, 2 * at + 1)
    a, b = x[..., offset + ia], x[..., offset + ib]
    out, size = x.copy(), np.zeros_like(x)
    out[..., offset + ia], out[..., offset + ib] = a * c - b * s, a * s + b * c
    size[..., offset + ia] = size[..., offset + ib] = m * (np.abs(a) + np.abs(b))
    return out, size


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T,H,D,rot,offset", [(1, 1, 64, 64, 0), (700, 8, 128, 64, 64), (2500, 1, 256, 256, 0),
                                              (33, 64, 80, 16, 32), (90, 3, 132, 128, 4)])
def test_fp32_values_are_rounded_once(layout, backward, T, H, D, rot, offset):
    rng = np.random.default_rng(T + rot)
    plan = dsa.RopePlan(rot, layout=layout, scaling="yarn", factor=8.0, original_len=65536)
    x = rng.normal(size=(T, H, D)) * np.exp(3 * rng.normal(size=(T, H, D)))
    pos = rng.integers(0, 1 << 20, size=T).astype(np.int32)
    xt = torch.from_numpy(x).float().cuda()
    ref, size = turned(f64(xt), pos, plan, offset, backward)
    got = dsa.rope(xt, i32_dev(pos), plan, offset=offset, backward=backward)
    dsa.sync_status()
    assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -48 * size + 2.0 ** -150)
    dsa.rope(xt, i32_dev(pos), plan, offset=offset, backward=backward, out=xt)
    assert torch.equal(xt, got)


def test_fp32_values_next_to_the_ends_of_the_range():
    """Sums that cancel and products past fp32 whose result is within it."""
    plan = dsa.RopePlan(16, theta=1e4, layout="half", mscale=1.5)
    big = np.float32(3.0e38)
    x = np.zeros((3, 1, 16))
    x[0, 0, 0], x[0, 0, 8] = big, big          # 1.5 * 3e38 * (cos 1 - sin 1): each product is within, their sum is
    x[1, 0, 0] = 2.0 ** -140
    x[2, 0, :8] = x[2, 0, 8:] = np.float32(1 / 3)
    pos = np.array([1, 0, 25], dtype=np.int32)
    xt = torch.from_numpy(x).float().cuda()
    ref, size = turned(f64(xt), pos, plan, 0, False)
    got = f64(dsa.rope(xt, i32_dev(pos), plan))
    fine = np.abs(ref) < 3.4e38
    assert np.isinf(got[~fine]).all() and not fine.all()
    assert np.all(np.abs(got - ref)[fine] <= (2.0 ** -24 * np.abs(ref) + 2.0 ** -48 * size + 2.0 ** -150)[fine])
