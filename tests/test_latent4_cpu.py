"""The 4-bit latent cache and rotary positions on the CPU: the oracle pinned to hand values, the rotation plans of
the library against it, and every refusal that needs no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_sparse_11_b200 as dsa
from long_context_sparse_11_b200 import binding as B
import oracle.latent4 as L4


@pytest.fixture(scope="module")
def lib():
    from long_context_sparse_11_b200.build import build
    build()
    return dsa.load()


def test_row_format_hand_values():
    row = np.zeros((1, 320), dtype=np.uint8)
    row[0, 288:306] = 127
    # word 0: value 0 = +6 (code 7), value 1 = -0.5 (code 1, sign bit 15), value 7 = -4 (code 6, sign bit 27)
    w = 7 | (1 << 4) | (1 << 15) | (6 << 28) | (1 << 27)
    row[0, 0:4] = [w & 255, (w >> 8) & 255, (w >> 16) & 255, w >> 24]
    row[0, 288] = 129
    v = L4.decode_rows(row)[0]
    assert v[0] == 24.0 and v[1] == -2.0 and v[7] == -16.0 and np.all(v[2:7] == 0) and np.all(v[8:] == 0)
    row[0, 288], row[0, 0:16] = 141, 0x77
    assert np.isnan(L4.decode_rows(row)[0, :32]).all()


def test_encoder_rounds_to_the_nearest_value_and_decodes_back():
    rng = np.random.default_rng(0)
    y = (rng.normal(size=(6, 576)) * np.exp(rng.normal(size=(6, 1)) * 3)).astype(np.float32)
    y[1, :32] = 0.0
    y[2, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]
    y[2, 16:32] = 0
    y[3, 32] = 1e6      # saturates at 6 * 2^13
    y[3, 64] = np.inf
    y[4, 70] = np.nan
    v = L4.decode_rows(L4.encode_rows(y))
    assert list(v[2, :16]) == [0, 1, 1, 2, 2, 4, 4, 6, 0, -1, -1, -2, -2, -4, -4, -6]
    assert v[3, 32] == 49152 and v[3, 64] == 49152 and np.all(v[1, :32] == 0)
    assert np.isnan(v[4, 64:96]).all() and np.isnan(v).sum() == 32
    for b in range(18):
        blk, got = y[0, 32 * b:32 * b + 32].astype(np.float64), v[0, 32 * b:32 * b + 32]
        step = 2.0 ** L4.block_exponent(blk)
        # the grid's spacing at a value is at most a third of it, or half a step near zero
        assert np.all(np.abs(blk - got) <= np.maximum(np.abs(blk) / 5 + 1e-12, step / 4))


def test_encoding_decoded_rows_changes_no_value():
    """The bytes may differ: a block whose largest value rounded down to 3 * 2^e is also 6 * 2^(e - 1)."""
    rng = np.random.default_rng(1)
    v = L4.decode_rows(L4.encode_rows(rng.normal(size=(4, 576)).astype(np.float32) * 0.3))
    assert np.array_equal(L4.decode_rows(L4.encode_rows(v.astype(np.float32))), v)


def test_rotation_closed_forms():
    f, m = L4.inv_freq(64, 8.0e6)
    assert m == 1.0 and f[0] == 1.0
    x = np.zeros((1, 1, 64))
    x[0, 0, 0] = 1.0
    y = L4.rotate(x, [1], f, 1.0, "half")
    assert abs(y[0, 0, 0] - math.cos(1)) < 1e-15 and abs(y[0, 0, 32] - math.sin(1)) < 1e-15
    y = L4.rotate(x, [1], f, 1.0, "interleaved")
    assert abs(y[0, 0, 1] - math.sin(1)) < 1e-15
    assert np.allclose(L4.rotate(y, [1], f, 1.0, "interleaved", backward=True), x, atol=1e-15)
    assert np.allclose(L4.inv_freq(64, 1e4, "linear", 4.0)[0], L4.inv_freq(64, 1e4)[0] / 4)
    ntk = L4.inv_freq(64, 1e4, "ntk", 4.0)[0]
    assert ntk[0] == 1.0 and abs(ntk[31] * 4.0 / L4.inv_freq(64, 1e4)[0][31] - 1) < 1e-12  # the slowest pair: / factor
    y, m = L4.inv_freq(64, 1e4, "yarn", 4.0, 4096)
    p = L4.inv_freq(64, 1e4)[0]
    assert y[0] == p[0] and abs(y[31] * 4 / p[31] - 1) < 1e-15 and abs(m - (0.1 * math.log(4) + 1)) < 1e-15


@pytest.mark.parametrize("rot", [16, 64, 256])
@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=8.0), dict(scaling="ntk", factor=1.0),
    dict(scaling="yarn", factor=40.0, original_len=4096), dict(scaling="yarn", factor=4.0, original_len=131072,
                                                               beta_fast=16.0, beta_slow=2.0),
    dict(scaling="yarn", factor=4.0, original_len=16)])
def test_plans_hold_the_oracles_frequencies(lib, rot, kw):
    for theta in (1e4, 8.0e6):
        plan = dsa.RopePlan(rot, theta=theta, layout="half", **kw)
        f, m = L4.inv_freq(rot, theta, **kw)
        got = np.array(plan.inv_freq[:rot // 2])
        assert np.all(np.abs(got / f - 1) <= 1e-14) and abs(plan.mscale / m - 1) <= 1e-15
        assert plan.rot_dim == rot and plan.layout == 1 and not any(plan.inv_freq[rot // 2:])
    assert dsa.RopePlan(rot, mscale=0.5).mscale == 0.5


def _refused(fn, status=B.DSA_ERR_INVALID_ARG):
    with pytest.raises(dsa.DsaError) as e:
        fn()
    assert e.value.status == status, e.value
    return str(e.value)


def test_plan_refusals(lib):
    for rot in (0, -16, 8, 24, 272):
        _refused(lambda: dsa.RopePlan(rot), B.DSA_ERR_UNSUPPORTED)
    _refused(lambda: dsa.RopePlan(64, layout="diagonal"))
    _refused(lambda: dsa.RopePlan(64, scaling="log"))
    for theta in (1.0, 0.0, -3.0, math.inf, math.nan):
        _refused(lambda: dsa.RopePlan(64, theta=theta))
    for kw in (dict(factor=0.5), dict(factor=math.nan), dict(factor=math.inf)):
        _refused(lambda: dsa.RopePlan(64, scaling="linear", **kw))
    _refused(lambda: dsa.RopePlan(64, scaling="yarn", factor=2.0))
    _refused(lambda: dsa.RopePlan(64, scaling="yarn", factor=2.0, original_len=64, beta_fast=0.5))
    _refused(lambda: dsa.RopePlan(64, mscale=0.0))
    _refused(lambda: dsa.RopePlan(64, mscale=math.inf))
    assert lib.dsa_rope_plan_init(None, 64, 0, 1e4, 0, 1.0, 0.0, 0.0, 0.0, 0.0) == B.DSA_ERR_INVALID_ARG
    assert lib.dsa_abi_sizeof(3) == ctypes.sizeof(dsa.RopePlan)


def test_rope_argument_checks(lib):
    plan = dsa.RopePlan(64)

    def call(x=64, out=4096, dt=B.DSA_BF16, pos=16, T=2, H=4, D=128, off=64, xs=(512, 128), os_=(512, 128), plan=plan):
        return lib.dsa_rope(plan if plan is None else ctypes.byref(plan), x, out, dt, pos, T, H, D, off, xs[0], xs[1],
                            os_[0], os_[1], 0, None)

    assert call(plan=None) == B.DSA_ERR_INVALID_ARG
    blank = dsa.RopePlan.__new__(dsa.RopePlan)
    assert call(plan=blank) == B.DSA_ERR_INVALID_ARG
    assert call(dt=B.DSA_E4M3) == B.DSA_ERR_UNSUPPORTED
    for kw in (dict(T=-1), dict(H=-1), dict(off=72), dict(off=-8), dict(off=4), dict(D=127), dict(x=65), dict(out=0),
               dict(pos=None), dict(xs=(513, 128)), dict(os_=(512, 132)), dict(out=64, os_=(1024, 128)),
               dict(os_=(512, 64)), dict(os_=(384, 128)), dict(os_=(0, 128))):
        assert call(**kw) == B.DSA_ERR_INVALID_ARG, kw
    assert call(T=0) == B.DSA_OK and call(H=0) == B.DSA_OK


def test_rope_tensor_checks(lib):
    plan, x, pos = dsa.RopePlan(64), torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    _refused(lambda: dsa.rope(x.double(), pos, plan))
    _refused(lambda: dsa.rope(x[None], pos, plan))
    _refused(lambda: dsa.rope(x, pos.long(), plan))
    _refused(lambda: dsa.rope(x, pos[:2], plan))
    _refused(lambda: dsa.rope(x, torch.zeros(6, dtype=torch.int32)[::2], plan))
    _refused(lambda: dsa.rope(x, pos, plan, out=x.bfloat16()))
    _refused(lambda: dsa.rope(x.transpose(1, 2).contiguous().transpose(1, 2), pos, plan))
    assert "autograd" in _refused(lambda: dsa.rope(x.requires_grad_(), pos, plan))
    assert "CUDA" in _refused(lambda: dsa.rope(x.detach(), pos, plan))


def _view4(n_pages=4, batch=2, max_pages=3, **kw):
    a = dict(data=64, scale=None, bt=128, lens=256, stride=320, tokens=n_pages * 64, dim=576, dt=B.DSA_MXFP4)
    a.update(kw)
    return B.CacheView(a["data"], a["scale"], a["bt"], a["lens"], a["stride"], a["tokens"], a["dim"], a["dt"], max_pages,
                       batch)


def test_four_bit_views_are_checked_everywhere(lib):
    def attn(v, k=8, n=2, rows=1, ws=None):
        return lib.dsa_sparse_mla_attn(16, ctypes.byref(v), 16, n, rows, k, 0.04, 16, None, ws, 0, None)

    for kw in (dict(scale=16), dict(stride=576), dict(stride=288), dict(tokens=100), dict(tokens=-64), dict(lens=None),
               dict(batch=0), dict(max_pages=0), dict(data=None), dict(data=8), dict(tokens=1 << 31)):
        assert attn(_view4(**kw)) == B.DSA_ERR_INVALID_ARG, kw
    assert attn(_view4(bt=None)) == B.DSA_ERR_UNSUPPORTED          # dense
    assert attn(_view4(dim=128)) == B.DSA_ERR_UNSUPPORTED
    assert attn(_view4(), n=3) == B.DSA_ERR_INVALID_ARG            # batch != n_q
    for dt in (B.DSA_F16, B.DSA_F32, 7):
        assert attn(_view4(dt=dt, stride=576)) == B.DSA_ERR_INVALID_ARG
    # indexer keys are never 4-bit
    v = _view4(dim=128)
    assert lib.dsa_indexer_score(16, B.DSA_MXFP4, None, 16, 2, 0, ctypes.byref(v), 16, 192, None) == B.DSA_ERR_UNSUPPORTED


def test_append_and_read_argument_checks(lib):
    plan, wide = dsa.RopePlan(64), dsa.RopePlan(128)

    def append(v=None, x=64, dt=B.DSA_BF16, stride=576, n=2, gamma=16, eps=1e-6, rope=plan, pos=16):
        v = _view4() if v is None else v
        return lib.dsa_latent_append(x, dt, stride, n, gamma, eps, None if rope is None else ctypes.byref(rope), None, pos,
                                     ctypes.byref(v), None)

    def read(v=None, n=2, pos=16, out=64, stride=576):
        v = _view4() if v is None else v
        return lib.dsa_latent_read(ctypes.byref(v), None, pos, n, out, stride, None)

    assert append(rope=wide) == B.DSA_ERR_UNSUPPORTED and append(dt=B.DSA_F16) == B.DSA_ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(x=None), dict(x=68), dict(stride=512), dict(stride=580), dict(pos=None), dict(eps=-1.0),
               dict(eps=math.nan), dict(gamma=20)):
        assert append(**kw) == B.DSA_ERR_INVALID_ARG, kw
    for kw in (dict(n=-1), dict(pos=None), dict(out=None), dict(out=68), dict(stride=512), dict(stride=580)):
        assert read(**kw) == B.DSA_ERR_INVALID_ARG, kw
    for fn in (append, read):
        assert fn(_view4(bt=None)) == B.DSA_ERR_UNSUPPORTED
        assert fn(_view4(stride=576)) == B.DSA_ERR_INVALID_ARG
        assert fn(B.CacheView(64, None, 128, 256, 576, 256, 576, B.DSA_BF16, 3, 2)) == B.DSA_ERR_UNSUPPORTED
        assert fn(B.CacheView(64, 64, 128, 256, 128, 256, 128, B.DSA_E4M3, 3, 2)) == B.DSA_ERR_UNSUPPORTED
        assert fn(n=0) == B.DSA_OK
    assert read(_view4(lens=None)) == B.DSA_ERR_INVALID_ARG
    assert lib.dsa_latent_append(None, B.DSA_BF16, 576, 0, None, 0.0, None, None, None, ctypes.byref(_view4(lens=None)),
                                 None) == B.DSA_OK  # an append does not read the lengths


def test_four_bit_tensor_checks(lib):
    pool, bt = dsa.latent_pool4(4, "cpu"), torch.zeros(2, 2, dtype=torch.int32)
    lens = torch.ones(2, dtype=torch.int32)
    _refused(lambda: dsa.paged_view(pool[:, :, :306], None, bt, lens))
    _refused(lambda: dsa.paged_view(pool.int(), None, bt, lens))
    _refused(lambda: dsa.paged_view(pool, None, bt.long(), lens))
    _refused(lambda: dsa.paged_view(pool, None, bt.t(), lens[:1]))
    _refused(lambda: dsa.paged_view(pool, None, bt, lens[:1]))
    v = dsa.paged_view(pool, None, bt, lens, rows_per_seq=3)
    assert (v.dtype, v.row_stride, v.dim, v.n_tokens, v.batch, v.scale) == (B.DSA_MXFP4, 320, 576, 256, 6, None)
    v = dsa.paged_view(pool, None, bt, lens)
    x, pos = torch.zeros(2, 576), torch.zeros(2, dtype=torch.int32)
    _refused(lambda: dsa.latent_append(x.half(), pos, v))
    _refused(lambda: dsa.latent_append(x[:, :512], pos, v))
    _refused(lambda: dsa.latent_append(x, pos[:1], v))
    _refused(lambda: dsa.latent_append(x, pos, v, gamma=torch.ones(576)))
    _refused(lambda: dsa.latent_append(x, pos, v, seq=pos.long()))
    assert "CUDA" in _refused(lambda: dsa.latent_append(x, pos, v))
    _refused(lambda: dsa.latent_read(v, pos, out=torch.zeros(2, 576)))
    _refused(lambda: dsa.latent_read(v, pos.float()))
    assert "CUDA" in _refused(lambda: dsa.latent_read(v, pos))
    q, idx = torch.zeros(2, 64, 576, dtype=torch.bfloat16), torch.zeros(2, 8, dtype=torch.int32)
    _refused(lambda: dsa.sparse_mla_attn(q.float(), v, idx, 8, 0.04))
    _refused(lambda: dsa.sparse_mla_attn(q, v, idx.long(), 8, 0.04))
    _refused(lambda: dsa.sparse_mla_attn(q, v, idx, 7, 0.04))
    _refused(lambda: dsa.sparse_mla_attn(q, v, idx, 8, 0.04, q_rows_per_idx_row=0))
    _refused(lambda: dsa.sparse_mla_attn(q, v, idx, 8, 0.04, out=torch.zeros(2, 64, 512)))
    assert "CUDA" in _refused(lambda: dsa.sparse_mla_attn(q, v, idx, 8, 0.04))


def test_rope_refuses_outputs_that_overlap_the_input(lib):
    """Only overlaps are called here: what is accepted would be launched."""
    plan = dsa.RopePlan(64)

    def call(out, T=2, H=4, D=128, xs=(512, 128), os_=(512, 128), x=64, dt=B.DSA_BF16):
        rc = lib.dsa_rope(ctypes.byref(plan), x, out, dt, 16, T, H, D, 0, xs[0], xs[1], os_[0], os_[1], 0, None)
        return rc, lib.dsa_last_error()

    for out, kw in ((64 + 16, {}), (64 + 256, {}), (64 + 2048 - 16, {}), (64 + 1024, dict(os_=(1024, 256))),
                    (64 + 16, dict(T=1, H=1)), (64 + 256, dict(T=1)),
                    (64 + 512 - 16, dict(D=256, H=1, xs=(256, 0), os_=(256, 0))),
                    (64 + 64, dict(D=64)), (64 + 256 - 16, dict(D=64)), (64 + 256, dict(dt=B.DSA_F32)),
                    (64 + 128, dict(H=2, T=4, D=64, xs=(64, 512), os_=(64, 512)))):
        rc, msg = call(out, **kw)
        assert rc == B.DSA_ERR_INVALID_ARG and b"overlaps x" in msg, (out, kw, rc, msg)
        rc, msg = call(64, x=out, **{**kw, "xs": kw.get("os_", (512, 128)), "os_": kw.get("xs", (512, 128))})
        assert rc == B.DSA_ERR_INVALID_ARG and b"overlap" in msg, (out, kw, rc, msg)


def test_four_bit_views_lie_on_one_device(lib):
    pool, bt, lens = dsa.latent_pool4(4, "cpu"), torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    assert "meta" in _refused(lambda: dsa.paged_view(pool, None, bt, lens.to("meta")))
    assert "meta" in _refused(lambda: dsa.paged_view(pool, None, bt.to("meta"), lens))
