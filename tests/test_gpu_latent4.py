"""The 4-bit latent cache and rotary positions on the GPU, against the fp64 oracle (needs a B200).

Tolerances, from the roundings each path makes:
* appended rows: the oracle's bytes (4 bits) and codes and scales (e4m3).  Both sides round the same real numbers to
  fp32, formed in double, so a difference needs a value within about 1e-15 of a border.
* read rows: exact (4 bits); one bf16 rounding of an fp32 product (e4m3).
* rope: the sine, the cosine and the products each carry an fp32 rounding, the result one rounding to its type:
  |err| <= 6 * 2^-24 * (|a| + |b|) m + half a step of the result's type.
* attention: see `attention_bound`.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import long_context_sparse_11_b200 as dsa  # noqa: E402
import oracle.dsa_oracle as O  # noqa: E402
import oracle.latent4 as L4  # noqa: E402
from test_gpu_kernels import bf16_dev, bf16_host, f32_dev, i32_dev, u8_dev  # noqa: E402

SCALE = 1.0 / 24.0


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from long_context_sparse_11_b200.build import build
    build()
    return dsa.load()


def f64(t):
    return t.detach().double().cpu().numpy()


def paged(rng, lens, extra=2):
    """A block table over a permuted pool with spare pages: (n_pages, table [B, max_pages] with -1 behind the end)."""
    need = [(n + 63) // 64 for n in lens]
    n_pages = sum(need) + extra
    perm = rng.permutation(n_pages).astype(np.int32)
    bt = np.full((len(lens), max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return n_pages, bt


def garbage_pool(n_pages):
    """A pool whose every row is NaN until it is written: a row read without being selected shows."""
    pool = np.full((n_pages, 64, 320), 141, dtype=np.uint8)
    pool[:, :, :288] = 0x77
    return pool


def make_rows(rng, n, spread=1.0):
    return (rng.normal(size=(n, 576)) * np.exp(spread * rng.normal(size=(1, 576)) * 0.3)).astype(np.float32)


def cache4(rng, lens, spread=1.0):
    """A 4-bit cache of sequences of these lengths: (pool, block table, per-sequence values [n, 576] fp64)."""
    n_pages, bt = paged(rng, lens)
    pool = garbage_pool(n_pages)
    distinct = L4.encode_rows(make_rows(rng, 96, spread))
    vals = L4.decode_rows(distinct)
    kv = []
    for b, n in enumerate(lens):
        pick = rng.integers(0, 96, size=n)
        t = np.arange(n)
        pool[bt[b][t // 64], t % 64] = distinct[pick]
        kv.append(vals[pick])
    return pool, bt, kv


# ------------------------------------------------------------------------------------------------ rope


TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp16": (torch.float16, 2.0 ** -11), "fp32": (torch.float32, 2.0 ** -24)}


def check_rope(x, pos, rot, offset, layout, backward, out, kw):
    plan = dsa.RopePlan(rot, layout=layout, **kw)
    got = dsa.rope(x, i32_dev(pos), plan, offset=offset, backward=backward, out=out)
    dsa.sync_status()
    return got, plan


def rope_reference(x, pos, rot, offset, layout, backward, kw):
    kw = dict(kw)
    f, m = L4.inv_freq(rot, kw.pop("theta", 8.0e6), **kw)
    x3 = x if x.ndim == 3 else x[:, None]
    ref = x3.copy()
    seg = x3[..., offset:offset + rot]
    ref[..., offset:offset + rot] = L4.rotate(seg, pos, f, m, layout, backward)
    size = np.zeros_like(ref)
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        size[..., offset + a] = size[..., offset + b] = m * (np.abs(seg[..., a]) + np.abs(seg[..., b]))
    return ref.reshape(x.shape), size.reshape(x.shape)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,D,rot,offset", [(1, 1, 64, 64, 0), (7, 64, 64, 64, 0), (33, 3, 128, 64, 64),
                                              (300, 1, 80, 16, 32), (5, 2, 256, 256, 0), (1030, 5, 192, 128, 32)])
def test_rope_matches_the_oracle(dtype, layout, T, H, D, rot, offset):
    rng = np.random.default_rng(T + D + rot)
    dt, half = TYPES[dtype]
    kw = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
          dict(scaling="yarn", factor=16.0, original_len=65536)][(T + H) % 4]
    backward = H == 3
    x = torch.from_numpy(rng.normal(size=(T, H, D))).to(dt).cuda()
    pos = rng.integers(-(1 << 20), 1 << 23, size=T).astype(np.int32)
    pos[0] = 0 if T == 1 else (1 << 31) - 1
    got, _ = check_rope(x, pos, rot, offset, layout, backward, None, kw)
    ref, size = rope_reference(f64(x), pos, rot, offset, layout, backward, kw)
    assert np.all(np.abs(f64(got) - ref) <= 6 * 2.0 ** -24 * size + half * np.abs(ref) + 2.0 ** -26)
    keep = [d for d in range(D) if not offset <= d < offset + rot]
    assert np.array_equal(f64(got)[..., keep], f64(x)[..., keep])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_in_place_strided_and_two_dimensional(layout):
    rng = np.random.default_rng(5)
    wide = torch.from_numpy(rng.normal(size=(9, 4, 576))).bfloat16().cuda()
    before = wide.clone()
    pos = rng.integers(0, 1 << 20, size=9).astype(np.int32)
    part = wide[:, 1:, 512:]                                    # a strided slice, turned where it stands
    ref, size = rope_reference(f64(part), pos, 64, 0, layout, False, {})
    got, plan = check_rope(part, pos, 64, 0, layout, False, part, {})
    assert got.data_ptr() == part.data_ptr()
    assert np.all(np.abs(f64(part) - ref) <= 6 * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(ref) + 2.0 ** -26)
    same = wide == before
    assert bool(same[:, 0].all()) and bool(same[:, :, :512].all())
    # heads outside tokens in memory, a 2-D tensor, and an output with strides of its own
    xt = torch.from_numpy(rng.normal(size=(4, 9, 64))).float().cuda().transpose(0, 1)
    out = torch.full((9, 4, 128), 7.0, device="cuda")
    r3 = dsa.rope(xt, i32_dev(pos), plan, out=out[..., 32:96])
    assert torch.equal(r3, dsa.rope(xt.contiguous(), i32_dev(pos), plan))
    assert bool((out[..., :32] == 7).all()) and bool((out[..., 96:] == 7).all())
    r2 = dsa.rope(xt[:, 2], i32_dev(pos), plan)
    assert torch.equal(r2, r3[:, 2])


def test_rope_agrees_with_the_query_rotation_of_the_path():
    rng = np.random.default_rng(6)
    q = torch.from_numpy(rng.normal(size=(11, 64, 576))).bfloat16().cuda()
    pos = i32_dev(rng.integers(0, 1 << 20, size=11))
    a = dsa.rope(q, pos, dsa.RopePlan(64), offset=512)
    b = dsa.rope_query(q.clone(), pos)
    dsa.sync_status()
    # the same real numbers, each rounded to bf16 from fp32: at most one bf16 step apart
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
    assert float((a != b).float().mean()) < 1e-3


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_gradient(layout):
    """The gradient is the transposed map: <rope(x), g> = <x, rope(g, backward)>, and differences of a linear map."""
    rng = np.random.default_rng(8)
    plan = dsa.RopePlan(64, layout=layout, scaling="yarn", factor=4.0, original_len=4096)
    pos = i32_dev(rng.integers(0, 1 << 20, size=50))
    x, g = (torch.from_numpy(rng.normal(size=(50, 3, 96))).float().cuda() for _ in range(2))
    y, gx = dsa.rope(x, pos, plan, offset=32), dsa.rope(g, pos, plan, offset=32, backward=True)
    lhs, rhs = float((y.double() * g.double()).sum()), float((x.double() * gx.double()).sum())
    n = float((y.double().abs() * g.double().abs()).sum())
    assert abs(lhs - rhs) <= 16 * 2.0 ** -24 * n
    for d in (0, 32, 33, 64, 95):
        e = torch.zeros_like(x)
        e[:, :, d] = 1.0
        diff = dsa.rope(x + e, pos, plan, offset=32) - y
        got = (diff.double() * g.double()).sum(-1)
        # differences of fp32 values of size <= |x| + 1 summed over 96 dims
        assert float((got - gx[:, :, d].double()).abs().max()) <= 96 * 2.0 ** -22 * 6 * float(g.abs().max())


# ------------------------------------------------------------------------------------------------ append, read


def unwritten(pool_before, pool_after, slots):
    """All rows of the pool outside `slots` (flat) are as they were."""
    keep = np.ones(pool_before.shape[0] * 64, dtype=bool)
    keep[slots] = False
    a, b = (p.reshape(len(keep), -1)[keep] for p in (pool_before, pool_after))
    return np.array_equal(a, b)


def append_case(seed, n, n_seqs):
    rng = np.random.default_rng(seed)
    lens = [int(v) for v in rng.integers(1, 400, size=n_seqs)]
    lens[0] = max(lens[0], n)
    n_pages, bt = paged(rng, lens)
    pairs = [(b, t) for b in range(n_seqs) for t in range(lens[b])]
    pick = rng.permutation(len(pairs))[:n]
    seq = np.array([pairs[i][0] for i in pick], dtype=np.int32)
    pos = np.array([pairs[i][1] for i in pick], dtype=np.int32)
    x = rng.normal(size=(n, 576)) * np.exp(rng.normal(size=(n, 1)))
    gamma = (1 + 0.2 * rng.normal(size=512)).astype(np.float32)
    return rng, lens, n_pages, bt, seq, pos, x, gamma


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("n,norm,turn", [(1, True, True), (7, False, True), (33, True, False), (9, False, False),
                                         (130, True, True)])
def test_append4_and_read_match_the_oracle(dtype, layout, n, norm, turn):
    rng, lens, n_pages, bt, seq, pos, x, gamma = append_case(n, n, 3)
    x[0, 64:96] = 0.0                       # a block of zeros
    x[n // 2, 5] = 3e5                      # saturates without the norm
    x[n - 1, 100] = 2e-6                    # below the grid
    xt = torch.from_numpy(x).to(TYPES[dtype][0]).cuda()
    kw = dict(scaling="yarn", factor=8.0, original_len=131072) if layout == "half" else {}
    f, m = L4.inv_freq(64, 8.0e6, **kw)
    y = L4.latent_rows(f64(xt), gamma if norm else None, 1e-6, pos, f if turn else None, m, layout)
    pool = garbage_pool(n_pages)
    ref = L4.append(pool, y, bt, seq, pos)
    pd, btd = u8_dev(pool), i32_dev(bt)
    view = dsa.paged_view(pd, None, btd, i32_dev(lens))
    dsa.latent_append(xt, i32_dev(pos), view, gamma=f32_dev(gamma) if norm else None,
                      rope=dsa.RopePlan(64, layout=layout, **kw) if turn else None, seq=i32_dev(seq))
    dsa.sync_status()
    got = pd.cpu().numpy()
    slots = bt[seq, pos // 64].astype(np.int64) * 64 + pos % 64
    assert np.array_equal(got, ref) and unwritten(pool, got, slots)
    back = dsa.latent_read(view, i32_dev(pos), seq=i32_dev(seq))
    dsa.sync_status()
    want = L4.decode_rows(ref.reshape(-1, 320)[slots])
    assert np.array_equal(f64(back), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("n,norm,turn", [(1, True, True), (40, False, True), (65, True, True)])
def test_append8_and_read_match_the_oracle(dtype, layout, n, norm, turn):
    rng, lens, n_pages, bt, seq, pos, x, gamma = append_case(100 + n, n, 2)
    xt = torch.from_numpy(x).to(TYPES[dtype][0]).cuda()
    f, m = L4.inv_freq(64, 8.0e6)
    y = L4.latent_rows(f64(xt), gamma if norm else None, 1e-6, pos, f if turn else None, m, layout)
    amax = np.abs(y).max(-1)
    s = np.where(amax > 0, amax / np.float32(448.0), np.float32(1)).astype(np.float32)
    codes = torch.from_numpy(y / s[:, None]).to(torch.float8_e4m3fn)
    pool = np.full((n_pages, 64, 576), 0x3C, dtype=np.uint8)
    scale = np.full((n_pages, 64), 0.5, dtype=np.float32)
    pd, sd = u8_dev(pool), f32_dev(scale)
    view = dsa.paged_view(pd, sd, i32_dev(bt), i32_dev(lens))
    dsa.latent_append(xt, i32_dev(pos), view, gamma=f32_dev(gamma) if norm else None,
                      rope=dsa.RopePlan(64, layout=layout) if turn else None, seq=i32_dev(seq))
    dsa.sync_status()
    slots = bt[seq, pos // 64].astype(np.int64) * 64 + pos % 64
    got, gs = pd.cpu().numpy(), sd.cpu().numpy().reshape(-1)
    assert np.array_equal(got.reshape(-1, 576)[slots], codes.view(torch.uint8).numpy())
    assert np.array_equal(gs[slots], s) and unwritten(pool, got, slots)
    back = dsa.latent_read(view, i32_dev(pos), seq=i32_dev(seq))
    want = (codes.float() * torch.from_numpy(s)[:, None]).bfloat16()
    assert torch.equal(back.cpu(), want)


def test_append_of_plain_rows_is_the_cache_write():
    """Without norm and rotation an e4m3 append stores what dsa_cache_write_e4m3 stores."""
    rng, lens, n_pages, bt, seq, pos, x, _ = append_case(31, 50, 4)
    xt = torch.from_numpy(x).bfloat16().cuda()
    pools = [torch.zeros(n_pages, 64, 576, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(n_pages, 64, device="cuda") for _ in range(2)]
    view = dsa.paged_view(pools[0], scales[0], i32_dev(bt), i32_dev(lens))
    dsa.latent_append(xt, i32_dev(pos), view, seq=i32_dev(seq))
    dsa.cache_write_e4m3(xt, i32_dev(pos), i32_dev(bt), pools[1], scales[1], seq=i32_dev(seq))
    dsa.sync_status()
    assert torch.equal(pools[0], pools[1]) and torch.equal(scales[0], scales[1])


def test_append_takes_strided_rows_and_keeps_nan_in_its_block():
    rng, lens, n_pages, bt, seq, pos, x, gamma = append_case(77, 6, 1)
    wide = torch.zeros(6, 640, dtype=torch.bfloat16, device="cuda")
    xt = wide[:, 32:608]
    xt.copy_(torch.from_numpy(x))
    xt[2, 70] = math.nan
    xt[3, 70] = math.inf
    xt[4, 570] = -math.nan
    view = dsa.paged_view(u8_dev(garbage_pool(n_pages)), None, i32_dev(bt), i32_dev(lens))
    dsa.latent_append(xt, i32_dev(pos), view, seq=i32_dev(seq))
    back = f64(dsa.latent_read(view, i32_dev(pos), seq=i32_dev(seq)))
    dsa.sync_status()
    bad = np.isnan(back)
    want = np.zeros_like(bad)
    want[2, 64:96] = want[4, 544:576] = True
    assert np.array_equal(bad, want) and back[3, 70] == 49152.0
    assert np.array_equal(back[5], L4.decode_rows(L4.encode_rows(f64(xt)[5:6].astype(np.float32)))[0])


def test_rows_out_of_range_are_skipped_and_reported():
    rng = np.random.default_rng(3)
    n_pages, bt = paged(rng, [100, 64])
    bt[1, 0] = n_pages + 3                                          # a page that does not exist
    x = torch.from_numpy(rng.normal(size=(6, 576))).bfloat16().cuda()
    seq, pos = i32_dev([0, 2, -1, 0, 1, 0]), i32_dev([5, 5, 5, 128, 5, -1])
    pool = garbage_pool(n_pages)
    pd = u8_dev(pool)
    view = dsa.paged_view(pd, None, i32_dev(bt), i32_dev([100, 64]))
    dsa.latent_append(x, pos, view, seq=seq)
    with pytest.raises(dsa.DsaError) as e:
        dsa.sync_status()
    assert e.value.status == dsa.binding.DSA_ERR_BOUNDS
    assert unwritten(pool, pd.cpu().numpy(), [int(bt[0, 0]) * 64 + 5])
    out = torch.full((6, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.latent_read(view, i32_dev([5, 5, 5, 100, 5, -1]), seq=seq, out=out)  # 100 is the length: not yet a token
    with pytest.raises(dsa.DsaError):
        dsa.sync_status()
    assert bool((out[1:] == 7.0).all()) and not bool((out[0] == 7.0).any())  # 7 is no 4-bit value
    dsa.latent_append(x[:0], pos[:0], view)
    assert dsa.latent_read(view, pos[:0]).shape == (0, 576)
    dsa.sync_status()


# ------------------------------------------------------------------------------------------------ attention


def reference(q, kv, idx):
    """out [R, 64, 512], lse [R, 64] fp64 for rows q [R, 64, 576] over kv[idx >= 0], and the bounds below."""
    sel = idx[idx >= 0]
    R = q.shape[0]
    if len(sel) == 0:
        z = np.zeros((R, 64, 512))
        return z, np.full((R, 64), -np.inf), z, np.zeros((R, 64))
    k = kv[sel]
    z = np.einsum("rhd,jd->rhj", q, k) * SCALE
    mx = z.max(-1, keepdims=True)
    p = np.exp(z - mx)
    l = p.sum(-1, keepdims=True)
    out = np.einsum("rhj,jd->rhd", p / l, k[:, :512])
    return (out, (mx + np.log(l))[..., 0]) + attention_bound(q, k, p, l, out)


def attention_bound(q, k, p, l, out):
    """Bounds of |out - ref| and |lse - ref|.
    Logits: exact products of q (8 significant bits, in two parts of at most 2^-20 of the head's largest) and the
    cache, summed in fp32: dz <= (600 * 2^-24 + 2^-20) * scale * sum_d |q||k|, at its largest key.
    Probabilities: exp2 to 2^-21; split in a nearest e4m3 and a nearest e5m2 part of the rest: 2^-4 * 2^-3 = 2^-7 of
    the probability, and never worse than 2^-19 of the largest one; the sums in fp32.
    Output: one bf16 rounding (2^-8)."""
    dz = (600 * 2.0 ** -24 + 2.0 ** -20) * SCALE * np.einsum("rhd,jd->rhj", np.abs(q), np.abs(k)).max(-1)
    n = k.shape[0]
    mean_abs = np.einsum("rhj,jd->rhd", p / l, np.abs(k[:, :512]))
    rel = 2.0 ** -7 + 2 * dz + 2.0 ** -21 + n * 2.0 ** -23
    tiny = 2.0 ** -19 * np.abs(k[:, :512]).sum(0) / l
    b_out = 2.0 ** -8 * np.abs(out) + rel[..., None] * mean_abs + tiny + 2.0 ** -30
    return b_out, dz + 2.0 ** -20 + n * 2.0 ** -24 + 1e-5


def run_attention(rng, lens, rows, k, idx, spread=1.0, qscale=1.0, q=None):
    pool, bt, kv = cache4(rng, lens, spread)
    nq = len(lens) * rows
    q = rng.normal(size=(nq, 64, 576)) * qscale if q is None else q
    qd = torch.from_numpy(q).bfloat16().cuda()
    view = dsa.paged_view(u8_dev(pool), None, i32_dev(bt), i32_dev(lens))
    out, lse = dsa.sparse_mla_attn(qd, view, i32_dev(idx), k, SCALE, rows)
    return qd, view, kv, out, lse


def check_attention(qd, kv, idx, rows, out, lse):
    q, o, e = f64(qd), f64(out), f64(lse)
    for b in range(len(kv)):
        s = slice(b * rows, (b + 1) * rows)
        ro, rl, bo, bl = reference(q[s], kv[b], idx[b])
        assert np.all(np.abs(o[s] - ro) <= bo), (b, float(np.max(np.abs(o[s] - ro) - bo)))
        dead = np.isinf(rl)
        assert np.array_equal(e[s][dead], rl[dead])
        assert np.all(np.abs(e[s][~dead] - rl[~dead]) <= bl[~dead]), (b, float(np.max(np.abs(e[s] - rl))))


def selection(rng, lens, k, kind="spread"):
    idx = np.full((len(lens), k), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        pick = rng.permutation(n)[:k]
        if kind == "holes":                       # padding in between, not only behind
            at = np.sort(rng.permutation(k)[:min(len(pick), k // 2)])
            idx[b, at] = pick[:len(at)]
        elif kind == "repeat":                    # the same token several times counts several times
            idx[b] = pick[rng.integers(0, len(pick), size=k)]
        else:
            idx[b, :len(pick)] = pick
    return idx


@pytest.mark.parametrize("lens,rows,k,kind", [
    ([1], 1, 1, "spread"), ([1], 1, 64, "spread"), ([200], 1, 128, "spread"), ([200], 2, 129, "spread"),
    ([64, 65, 127, 128], 3, 127, "spread"), ([700, 5, 3000], 5, 2048, "spread"), ([2500], 6, 2048, "spread"),
    ([300] * 7, 1, 256, "holes"), ([90] * 3, 2, 300, "repeat"), ([3000] * 33, 1, 2048, "spread"),
    ([400] * 160, 1, 257, "spread"), ([1000] * 75, 4, 384, "holes")])
def test_attention_over_the_4bit_cache(lens, rows, k, kind):
    rng = np.random.default_rng(k + rows + len(lens))
    idx = selection(rng, lens, k, kind)
    qd, _, kv, out, lse = run_attention(rng, lens, rows, k, idx)
    dsa.sync_status()
    check_attention(qd, kv, idx, rows, out, lse)


def test_attention_rows_without_a_token_are_zero():
    rng = np.random.default_rng(2)
    lens = [200, 200, 0, 300]
    idx = selection(rng, lens, 300)
    idx[1] = -1
    qd, _, kv, out, lse = run_attention(rng, lens, 2, 300, idx)
    dsa.sync_status()
    check_attention(qd, kv, idx, 2, out, lse)
    assert bool((out[2:6] == 0).all()) and bool((lse[2:6] == -math.inf).all())


@pytest.mark.parametrize("qscale,spread", [(1e-3, 1.0), (20.0, 1.0), (1.0, 8.0), (1e30, 0.0), (1e-35, 0.0)])
def test_attention_over_wide_ranges(qscale, spread):
    """Queries of any finite size (a nearly one-hot softmax, a flat one), channels of very different sizes."""
    rng = np.random.default_rng(4)
    lens = [900, 333]
    idx = selection(rng, lens, 700)
    qd, _, kv, out, lse = run_attention(rng, lens, 2, 700, idx, spread, qscale)
    dsa.sync_status()
    check_attention(qd, kv, idx, 2, out, lse)


def test_attention_with_a_growing_maximum():
    """Logits that grow along the selection move the running maximum at every tile."""
    rng = np.random.default_rng(14)
    lens = [1500]
    pool, bt, kv = cache4(rng, lens)
    q = rng.normal(size=(1, 64, 576))
    z = q[0].mean(0) @ kv[0].T
    idx = np.argsort(z)[None].astype(np.int32)[:, -1400:].copy()
    q[:] = q.mean(1, keepdims=True) * 40 + 0.05 * q
    qd = torch.from_numpy(q).bfloat16().cuda()
    view = dsa.paged_view(u8_dev(pool), None, i32_dev(bt), i32_dev(lens))
    for order in (idx, idx[:, ::-1].copy()):
        out, lse = dsa.sparse_mla_attn(qd, view, i32_dev(order), 1400, SCALE)
        dsa.sync_status()
        check_attention(qd, kv, order, 1, out, lse)


def test_attention_passes_nan_on_to_its_heads_only():
    rng = np.random.default_rng(9)
    lens, rows = [300], 2
    idx = selection(rng, lens, 200)
    q = rng.normal(size=(2, 64, 576))
    q[0, 3, 7], q[1, 5, 570] = np.nan, np.inf
    qd, view, kv, out, lse = run_attention(rng, lens, rows, 200, idx, q=q)
    dsa.sync_status()
    bad = torch.isnan(out).all(-1)
    assert bool(bad[0, 3]) and bool(bad[1, 5]) and int(bad.sum()) == 2
    assert int(torch.isnan(out).any(-1).sum()) == 2 and int(torch.isnan(lse).sum()) == 2
    # a NaN block of a selected row reaches every head; of a row not selected, none
    t_in, t_out = int(idx[0, 11]), int(np.setdiff1d(np.arange(300), idx[0])[0])
    pool, _, bt, _ = view._keep
    for t, spoiled in ((t_out, False), (t_in, True)):
        row = pool.view(-1, 320)[int(bt[0, t // 64]) * 64 + t % 64]
        row[:288], row[288:306] = 0x77, 141
        out, _ = dsa.sparse_mla_attn(torch.nan_to_num(qd, 0, 0, 0), view, i32_dev(idx), 200, SCALE, rows)
        assert bool(torch.isnan(out).all()) == spoiled and bool(torch.isnan(out).any()) == spoiled


def test_bad_indices_and_pages_are_skipped_and_reported():
    rng = np.random.default_rng(10)
    lens = [150, 150]
    idx = selection(rng, lens, 140)
    qd, view, kv, _, _ = run_attention(rng, lens, 1, 140, idx)
    dsa.sync_status()
    bad = idx.copy()
    bad[0, 5] = 150                    # past the sequence
    bad[1, 7] = (1 << 31) - 1
    dropped = bad.copy()
    dropped[0, 5] = dropped[1, 7] = -1
    out, lse = dsa.sparse_mla_attn(qd, view, i32_dev(bad), 140, SCALE)
    with pytest.raises(dsa.DsaError) as e:
        dsa.sync_status()
    assert e.value.status == dsa.binding.DSA_ERR_BOUNDS
    check_attention(qd, kv, dropped, 1, out, lse)
    view._keep[2][1, 1] = 1 << 20      # positions 64..127 of sequence 1 lose their page
    gone = idx.copy()
    gone[1][(gone[1] >= 64) & (gone[1] < 128)] = -1
    out, lse = dsa.sparse_mla_attn(qd, view, i32_dev(idx), 140, SCALE)
    with pytest.raises(dsa.DsaError):
        dsa.sync_status()
    check_attention(qd, kv, gone, 1, out, lse)


def test_attention_is_repeatable_captured_and_on_other_streams():
    """Two calls give the same bits; so does a captured call, replayed on new contents, on a side stream."""
    rng = np.random.default_rng(12)
    lens, rows, k = [2600] * 5, 3, 2048
    idx = selection(rng, lens, k)
    qd, view, kv, out, lse = run_attention(rng, lens, rows, k, idx)
    idxd = i32_dev(idx)
    out2, lse2 = dsa.sparse_mla_attn(qd, view, idxd, k, SCALE, rows)
    dsa.sync_status()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    ws = torch.empty(max(16, dsa.sparse_mla_workspace_bytes(len(lens) * rows, k, view)), dtype=torch.uint8, device="cuda")
    o, e = torch.empty_like(out), torch.empty_like(lse)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        dsa.sparse_mla_attn(qd, view, idxd, k, SCALE, rows, out=o, lse=e, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(lse, e)
    q2 = torch.from_numpy(rng.normal(size=tuple(qd.shape))).bfloat16().cuda()
    qd.copy_(q2)
    ws.fill_(255)
    graph.replay()
    dsa.sync_status()
    check_attention(q2, kv, idx, rows, o, e)


def test_rope_between_slices_of_one_tensor_and_far_apart_rows():
    rng = np.random.default_rng(15)
    buf = torch.from_numpy(rng.normal(size=(9, 4, 128))).bfloat16().cuda()
    pos, plan = i32_dev(rng.integers(0, 1 << 20, size=9)), dsa.RopePlan(64)
    want = dsa.rope(buf[..., :64].contiguous(), pos, plan)
    dsa.rope(buf[..., :64], pos, plan, out=buf[..., 64:])       # interleaved in memory, no shared byte
    assert torch.equal(buf[..., 64:], want)
    big = torch.zeros((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((3, 2, 64), (1 << 30, 64, 1))          # token 2 starts at element 2^31
    far.copy_(buf[:3, :2, :64])
    got = dsa.rope(far, pos[:3], plan)
    assert torch.equal(got, want[:3, :2])
    dsa.rope(far, pos[:3], plan, out=far)
    assert torch.equal(far, got)
    dsa.sync_status()


@pytest.mark.parametrize("mx", [True, False])
def test_append_of_rows_at_the_ends_of_the_fp32_range(mx):
    """Sums of squares, reciprocals and products beyond fp32 where the result is not, or saturates."""
    rng = np.random.default_rng(16)
    n = 7
    x = rng.normal(size=(n, 576)).astype(np.float32)
    gamma = (1 + 0.2 * rng.normal(size=512)).astype(np.float32)
    x[0] *= np.float32(1e37)
    x[1, :512] *= np.float32(2.0 ** -130)                        # subnormal, normalised with eps = 0
    x[2, :512] *= np.float32(2.0 ** -147)
    if mx:
        x[3, 7] = np.inf
        x[4, :512] = 0.0                                         # 0 / 0
        gamma[40:48] = 3e38                                      # results past fp32 saturate
    x[5, :500] = 0.0
    x[6, :512] *= np.float32(2.0 ** 100)
    n_pages, bt = paged(rng, [n])
    seq, pos = np.zeros(n, dtype=np.int32), np.arange(n, dtype=np.int32)
    f, m = L4.inv_freq(64, 8.0e6)
    with np.errstate(all="ignore"):
        y = L4.latent_rows(x, gamma, 0.0, pos, f)
    xt, slots = torch.from_numpy(x).cuda(), bt[0, 0].astype(np.int64) * 64 + pos
    kw = dict(gamma=f32_dev(gamma), eps=0.0, rope=dsa.RopePlan(64), seq=i32_dev(seq))
    if mx:
        pool = garbage_pool(n_pages)
        pd = u8_dev(pool)
        dsa.latent_append(xt, i32_dev(pos), dsa.paged_view(pd, None, i32_dev(bt), i32_dev([n])), **kw)
        dsa.sync_status()
        assert np.array_equal(pd.cpu().numpy(), L4.append(pool, y, bt, seq, pos))
    else:
        s = (np.abs(y).max(-1) / np.float32(448.0)).astype(np.float32)
        codes = torch.from_numpy(y / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        pd = torch.zeros(n_pages, 64, 576, dtype=torch.uint8, device="cuda")
        sd = torch.zeros(n_pages, 64, device="cuda")
        dsa.latent_append(xt, i32_dev(pos), dsa.paged_view(pd, sd, i32_dev(bt), i32_dev([n])), **kw)
        dsa.sync_status()
        assert np.array_equal(pd.cpu().numpy().reshape(-1, 576)[slots], codes)
        assert np.array_equal(sd.cpu().numpy().reshape(-1)[slots], s)


def test_a_pool_beyond_32_bit_offsets():
    """Pages whose bytes lie past 2^32: appended to, read back and attended to like any other."""
    rng = np.random.default_rng(17)
    n_pages, n, k = 215000, 130, 130                             # 4.4 GB
    pool = dsa.latent_pool4(n_pages)
    bt = np.array([[n_pages - 1, 3, n_pages - 2]], dtype=np.int32)
    view = dsa.paged_view(pool, None, i32_dev(bt), i32_dev([n]))
    x = torch.from_numpy(rng.normal(size=(n, 576))).bfloat16().cuda()
    pos, seq = i32_dev(np.arange(n)), torch.zeros(n, dtype=torch.int32, device="cuda")
    dsa.latent_append(x, pos, view, seq=seq)
    kv = L4.decode_rows(L4.encode_rows(f64(x).astype(np.float32)))
    assert np.array_equal(f64(dsa.latent_read(view, pos, seq=seq)), kv)
    idx = rng.permutation(n)[None].astype(np.int32)
    qd = torch.from_numpy(rng.normal(size=(2, 64, 576))).bfloat16().cuda()
    out, lse = dsa.sparse_mla_attn(qd, view, i32_dev(idx), k, SCALE, 2)
    dsa.sync_status()
    check_attention(qd, [kv], idx, 2, out, lse)
    assert int(pool[:3].max()) == 0 and int(pool[4:1000].max()) == 0 and int(pool[-1000:-2].max()) == 0


def test_attention_over_many_short_rows():
    """More rows than SMs by far, one tile and two tiles each."""
    rng = np.random.default_rng(18)
    for lens, rows, k in (([40] * 700, 3, 33), ([200] * 331, 2, 131)):
        idx = selection(rng, lens, k)
        idx[5] = -1
        qd, _, kv, out, lse = run_attention(rng, lens, rows, k, idx)
        dsa.sync_status()
        check_attention(qd, kv, idx, rows, out, lse)


@pytest.mark.parametrize("n_seqs,rows,k", [(148, 1, 260), (149, 1, 1300), (40, 4, 1100), (19, 8, 2048), (296, 1, 130)])
def test_attention_over_all_shares_of_the_work(n_seqs, rows, k):
    """Whole rows per SM, parts of a row, and ranges that cut rows anywhere: a sample of the rows of each."""
    rng = np.random.default_rng(23)
    lens = [int(n) for n in rng.integers(max(k - 40, 1), k + 300, size=n_seqs)]
    idx = selection(rng, lens, k)
    qd, _, kv, out, lse = run_attention(rng, lens, rows, k, idx)
    dsa.sync_status()
    q, o, e = f64(qd), f64(out), f64(lse)
    for r in sorted(set([0, 1, n_seqs * rows // 2, n_seqs * rows - 1] + [int(v) for v in rng.integers(0, n_seqs * rows, 10)])):
        ro, rl, bo, bl = reference(q[r:r + 1], kv[r // rows], idx[r // rows])
        assert np.all(np.abs(o[r] - ro[0]) <= bo[0]) and np.all(np.abs(e[r] - rl[0]) <= bl[0]), r


def test_two_attentions_at_once_on_streams_of_their_own():
    rng = np.random.default_rng(19)
    calls = []
    for lens, rows, k in (([2600] * 9, 3, 2048), ([900] * 40, 1, 700)):
        idx = selection(rng, lens, k)
        qd, view, kv, out, lse = run_attention(rng, lens, rows, k, idx)
        calls.append((qd, view, i32_dev(idx), k, rows, out, lse, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for qd, view, idx, k, rows, out, lse, st in calls:
            with torch.cuda.stream(st):
                got.append(dsa.sparse_mla_attn(qd, view, idx, k, SCALE, rows) + (out, lse))
    torch.cuda.synchronize()
    dsa.sync_status()
    for o, e, out, lse in got:
        assert torch.equal(o, out) and torch.equal(e, lse)


def test_attention_refuses_a_workspace_that_is_too_small_or_misaligned():
    rng = np.random.default_rng(20)
    lens, k = [600] * 2, 512
    qd, view, kv, out, lse = run_attention(rng, lens, 1, k, selection(rng, lens, k))
    idx = i32_dev(selection(rng, lens, k))
    need = dsa.sparse_mla_workspace_bytes(2, k, view)
    assert need > 0
    for ws in (torch.empty(need - 16, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 16, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(dsa.DsaError) as e:
            dsa.sparse_mla_attn(qd, view, idx, k, SCALE, workspace=ws)
        assert e.value.status == 6
    dsa.sync_status()


def test_parts_of_a_selection_merge_to_the_whole():
    """Split over ranks: each part's bf16 output and its lse, joined by dsa_combine_partials.  The joined output is a mean of
    the parts' with weights that carry the parts' lse errors, rounded to bf16 once more."""
    rng = np.random.default_rng(21)
    lens, k = [1500] * 3, 1024
    idx = selection(rng, lens, k)
    halves = [np.where(np.arange(k) % 2 == g, idx, -1).astype(np.int32) for g in range(2)]
    halves[0][2], halves[1][2] = idx[2], -1                      # a part without a key
    qd, view, kv, _, _ = run_attention(rng, lens, 1, k, idx)
    parts = [dsa.sparse_mla_attn(qd, view, i32_dev(h), k, SCALE) for h in halves]
    out, lse = dsa.combine_partials(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    dsa.sync_status()
    o, e = f64(out), f64(lse)
    for b in range(3):
        ro, rl, _, _ = reference(f64(qd[b:b + 1]), kv[b], idx[b])
        bound, lse_bound = np.zeros_like(ro), np.zeros_like(rl)
        for h in halves:
            po, pl, bo, bl = reference(f64(qd[b:b + 1]), kv[b], h[b])
            w = np.exp(pl - rl)[..., None]
            lse_bound = np.maximum(lse_bound, bl)
            bound += w * ((1 + 3 * bl[..., None]) * bo + 3 * bl[..., None] * np.abs(po - ro))
        assert np.all(np.abs(o[b] - ro[0]) <= bound[0] + 2.0 ** -8 * (np.abs(ro[0]) + bound[0]) + 2.0 ** -20)
        assert np.all(np.abs(e[b] - rl[0]) <= lse_bound[0] + 2.0 ** -18)


def test_rope_append_read_and_attention_in_one_graph():
    """Captured together and replayed on other rows, positions and lengths."""
    rng = np.random.default_rng(22)
    n_seqs, k = 3, 192
    n_pages, bt = paged(rng, [400] * n_seqs)
    plan = dsa.RopePlan(64, layout="half")
    gamma = f32_dev((1 + 0.2 * rng.normal(size=512)).astype(np.float32))
    lens, pos = i32_dev([1] * n_seqs), i32_dev([0] * n_seqs)
    x = torch.zeros(n_seqs, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(n_seqs, 64, 576, dtype=torch.bfloat16, device="cuda")
    idx = i32_dev(np.full((n_seqs, k), -1))

    def step(view, x, q, pos, idx, out):
        dsa.latent_append(x, pos, view, gamma=gamma, rope=plan)
        dsa.rope(q, pos, plan, offset=512, out=out["q"])
        dsa.sparse_mla_attn(out["q"], view, idx, k, SCALE, out=out["o"], lse=out["lse"], workspace=out["ws"])
        dsa.latent_read(view, pos, out=out["rows"])

    def buffers(view):
        return dict(q=torch.empty_like(q), o=torch.empty(n_seqs, 64, 512, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty(n_seqs, 64, device="cuda"), rows=torch.empty_like(x),
                    ws=torch.empty(max(16, dsa.sparse_mla_workspace_bytes(n_seqs, k, view)), dtype=torch.uint8,
                                   device="cuda"))

    views = [dsa.paged_view(dsa.latent_pool4(n_pages), None, i32_dev(bt), lens) for _ in range(2)]
    eager, graphed = buffers(views[0]), buffers(views[1])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(views[1], x, q, pos, idx, graphed)
    for t in range(4):
        x.copy_(torch.from_numpy(rng.normal(size=(n_seqs, 576))))
        q.copy_(torch.from_numpy(rng.normal(size=(n_seqs, 64, 576))))
        at = t * np.arange(1, n_seqs + 1)
        pos.copy_(torch.from_numpy(at.astype(np.int32)))
        lens.copy_(torch.from_numpy((at + 1).astype(np.int32)))
        sel = np.full((n_seqs, k), -1, dtype=np.int32)
        for b in range(n_seqs):
            sel[b, :at[b] + 1] = rng.permutation(int(at[b]) + 1)
        idx.copy_(torch.from_numpy(sel))
        step(views[0], x, q, pos, idx, eager)
        graph.replay()
        dsa.sync_status()
        for name in ("q", "o", "lse", "rows"):
            assert torch.equal(eager[name], graphed[name]), (t, name)
        assert torch.equal(views[0]._keep[0], views[1]._keep[0])
        assert bool(torch.isfinite(eager["o"]).all())


# ------------------------------------------------------------------------------------------------ together


def test_a_decode_step_over_the_4bit_cache():
    """One decode step as a server makes it: new latent rows appended (norm and rotation on the way), the queries'
    RoPE dims turned, one IndexShare group over an e4m3 key cache and 4-bit, e4m3 and again 4-bit latent caches, the
    appended rows read back."""
    from synth import make_decode, DecodeSpec
    rows, k = 2, 128
    inp = make_decode(DecodeSpec("g4", batch=3, ctx_lo=200, ctx_hi=700, rows_per_seq=rows, k=k, n_layers=3, seed=5))
    bt, ctx = inp["block_table"], inp["ctx"]
    n_pages = inp["idx_keys"].shape[0]
    rng = np.random.default_rng(1)
    btd, lens = i32_dev(bt), i32_dev(ctx)
    f, _ = L4.inv_freq(64, 8.0e6)
    plan = dsa.RopePlan(64)
    gamma = (1 + 0.1 * rng.normal(size=512)).astype(np.float32)
    pos = (ctx - 1).astype(np.int32)
    pools, views, kvs = [], [], []
    for layer in range(3):
        x = torch.from_numpy(rng.normal(size=(3, 576))).bfloat16().cuda()
        if layer == 1:
            pd, sd = u8_dev(inp["KV"][1]), f32_dev(inp["KV_scale"][1])
            view = dsa.paged_view(pd, sd, btd, lens)
            dsa.latent_append(x, i32_dev(pos), view, gamma=f32_dev(gamma), rope=plan)
            codes, scale = pd.cpu().numpy(), sd.cpu().numpy()
            kv = []
            for b in range(3):
                t = np.arange(ctx[b])
                pg = bt[b][t // 64]
                kv.append(O.e4m3_to_f64(codes[pg, t % 64]) * scale[pg, t % 64][:, None])
        else:
            pool = garbage_pool(n_pages)
            for b in range(3):
                t = np.arange(ctx[b] - 1)
                base = L4.encode_rows(make_rows(rng, 32))
                pool[bt[b][t // 64], t % 64] = base[rng.integers(0, 32, size=len(t))]
            y = L4.latent_rows(f64(x), gamma, 1e-6, pos, f)
            ref = L4.append(pool, y, bt, np.arange(3), pos)
            pd = u8_dev(pool)
            view = dsa.paged_view(pd, None, btd, lens)
            dsa.latent_append(x, i32_dev(pos), view, gamma=f32_dev(gamma), rope=plan)
            dsa.sync_status()
            assert np.array_equal(pd.cpu().numpy(), ref)
            kv = [L4.paged_rows(ref, bt, b, int(ctx[b])) for b in range(3)]
            back = dsa.latent_read(view, i32_dev(pos))
            assert np.array_equal(f64(back), np.stack([kv[b][-1] for b in range(3)]))
        pools.append(pd)
        views.append(view)
        kvs.append(kv)
    qs = []
    for layer in range(3):
        q = bf16_dev(inp["Q"][layer])
        qs.append(dsa.rope(q, i32_dev(np.repeat(pos, rows)), plan, offset=512, out=q))
    keys = dsa.paged_view(u8_dev(inp["idx_keys"]), f32_dev(inp["idx_key_scale"]), btd, lens)
    g = dsa.IndexShareGroup(bf16_dev(inp["q_idx"]), f32_dev(inp["w"]), keys, k, qs, views, SCALE,
                            indexer_dtype=dsa.DSA_E4M3, q_rows_per_idx_row=rows)
    for reuse in (False, True):
        outs, lses = g.forward(reuse_only=reuse)
        dsa.sync_status()
        idx = g.idx.cpu().numpy()
        assert all(len(set(r[r >= 0])) == min(k, n) for r, n in zip(idx, ctx))
        for layer in (0, 2):
            check_attention(qs[layer], kvs[layer], idx, rows, outs[layer], lses[layer])
        for b in range(3):                                 # the e4m3 layer, at the tolerance of its own tests
            for r in range(rows):
                ref, _ = O.sparse_mla_row(f64(qs[1][b * rows + r]), kvs[1][b], idx[b], SCALE)
                got = f64(outs[1][b * rows + r])
                assert np.abs(got - ref).max() <= 2e-2 and np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)
