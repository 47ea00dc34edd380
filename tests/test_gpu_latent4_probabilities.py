"""What the 4-bit attention keeps of a probability (needs a B200).

Key j's row is 1 at dim j and zero in the other latent dims, and its RoPE dims set its logit, so out[j] is the
probability of key j itself.  Roundings:
* of the exponential, to f16: 2^-11 of it, or half the f16's smallest step;
* to an e4m3 number and the e5m2 rest: less than 2^-8 of it, or, where the e4m3 number is subnormal, 2^-14 at the scale
  that puts the row's largest probability at 2^4 or more: the rest is at most 2^-10 there, and an e5m2 number's half step
  below 2^-10 is 2^-14.  The f16's smallest step comes to 2^-17 at that scale: 9/8 * 2^-18 of the largest in all;
* of the output: 2^-8 of it.
The exponential's own error, the sums and the logit (dz, natural) are fp32; q's values below 2^-13 of their head's
largest are off by up to 2^-21 of it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import long_context_sparse_11_b200 as dsa  # noqa: E402
import oracle.latent4 as L4  # noqa: E402
from test_gpu_kernels import i32_dev, u8_dev  # noqa: E402
from test_gpu_latent4 import f64, lib  # noqa: E402,F401

SCALE = 1.0 / 24.0


@pytest.mark.parametrize("n,width", [(1, 0.0), (2, 1.0), (90, 3.0), (128, 0.5), (300, 6.0), (512, 12.0)])
def test_what_is_kept_of_a_probability(n, width):
    rng = np.random.default_rng(n)
    rows = np.zeros((n, 576))
    rows[np.arange(n), np.arange(n)] = 1.0
    rows[:, 512:] = rng.choice([-2.0, -1.5, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 2.0], size=(n, 64))
    coded = L4.encode_rows(rows.astype(np.float32))
    assert np.array_equal(L4.decode_rows(coded), rows)
    pages = (n + 63) // 64
    pool = np.zeros((pages * 64, 320), dtype=np.uint8)
    pool[:n] = coded
    q = np.zeros((1, 64, 576))
    q[0, :, 512:] = rng.normal(size=(64, 64)) * width * 24 / (8 * 1.29)  # logits of about that width
    qd = torch.from_numpy(q).bfloat16().cuda()
    idx = rng.permutation(n)[None].astype(np.int32)
    view = dsa.paged_view(u8_dev(pool.reshape(pages, 64, 320)), None, i32_dev(np.arange(pages)[None]), i32_dev([n]))
    out, lse = dsa.sparse_mla_attn(qd, view, i32_dev(idx), n, SCALE)
    dsa.sync_status()
    z = f64(qd)[0] @ rows.T * SCALE
    top = z.max(-1, keepdims=True)
    p = np.exp(z - top)
    l = p.sum(-1, keepdims=True)
    size = np.abs(f64(qd)[0]) @ np.abs(rows).T * SCALE
    dz = (600 * 2.0 ** -24) * size.max(-1, keepdims=True) + 2.0 ** -21 * np.abs(f64(qd)[0]).max(-1, keepdims=True) \
        * np.abs(rows).sum(-1) * SCALE + 2.0 ** -21
    share = 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11 + 2 * dz.max() + n * 2.0 ** -23
    got = f64(out)[0][:, :n]
    assert np.all(np.abs(got - p / l) <= share * p / l + 1.125 * 2.0 ** -18 / l + 2.0 ** -30)
    assert not f64(out)[0][:, n:].any()
    assert np.all(np.abs(f64(lse)[0] - (top + np.log(l))[:, 0]) <= dz.max() + n * 2.0 ** -23 + 1e-5)
