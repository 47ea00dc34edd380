"""The 4-bit latent cache at shapes of their own: many rows of one tile, rows that share one sequence's pages, appends
and reads over many blocks (needs a B200).  Tolerances: those of test_gpu_latent4.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import long_context_sparse_11_b200 as dsa  # noqa: E402
import oracle.latent4 as L4  # noqa: E402
from test_gpu_kernels import f32_dev, i32_dev, u8_dev  # noqa: E402
from test_gpu_latent4 import SCALE, cache4, check_attention, f64, garbage_pool, lib, make_rows, paged  # noqa: E402,F401
from test_gpu_latent4 import reference, run_attention, selection, unwritten  # noqa: E402


@pytest.mark.parametrize("lens,rows,k", [([200] * 1000, 2, 96), ([130] * 1500, 1, 128), ([9] * 900, 3, 1)])
def test_rows_of_one_tile_over_and_over(lens, rows, k):
    """13 rows of one tile and more per SM, every row with data of its own: the same bits each time."""
    rng = np.random.default_rng(k)
    idx = selection(rng, lens, k)
    idx[7] = -1
    qd, view, kv, out, lse = run_attention(rng, lens, rows, k, idx)
    idxd = i32_dev(idx)
    for _ in range(30):
        o, e = dsa.sparse_mla_attn(qd, view, idxd, k, SCALE, rows)
        assert torch.equal(o, out) and torch.equal(e, lse)
    dsa.sync_status()
    some = sorted({0, 7, len(lens) - 1} | {int(b) for b in rng.integers(0, len(lens), 12)})
    take = [r for b in some for r in range(b * rows, (b + 1) * rows)]
    check_attention(qd[take], [kv[b] for b in some], idx[some], rows, out[take], lse[take])


# ------------------------------------------------------------------------------------------------ a prompt's rows


def prompt_view(rng, length, n):
    """One sequence of `length` tokens, its last n query rows as entries of one view: the same pages, lengths of their own."""
    pool, bt, (kv,) = cache4(rng, [length])
    lens = np.arange(length - n + 1, length + 1).astype(np.int32)
    view = dsa.paged_view(u8_dev(pool), None, i32_dev(np.repeat(bt, n, 0)), i32_dev(lens))
    return view, kv, lens


def check_rows(qd, kv, idx, rows, out, lse):
    """Rows `rows` of a call whose rows all read kv (the bounds of `reference`)."""
    q, o, e = f64(qd[rows]), f64(out[rows]), f64(lse[rows])
    for i, r in enumerate(rows):
        ro, rl, bo, bl = reference(q[i:i + 1], kv, idx[r])
        assert np.all(np.abs(o[i] - ro[0]) <= bo[0]), r
        assert np.array_equal(np.isinf(e[i]), np.isinf(rl[0])) and np.all(np.abs(e[i] - rl[0])[np.isfinite(rl[0])] <= bl[0].max()), r


@pytest.mark.parametrize("length,n,k", [(300, 300, 64), (900, 260, 200), (5000, 500, 2048), (150, 150, 2048)])
def test_a_prompts_rows_over_one_sequences_pages(length, n, k):
    """A selection per row, rows earlier in the prompt than k padded; a position at or past a row's length is none of its."""
    rng = np.random.default_rng(n + k)
    view, kv, lens = prompt_view(rng, length, n)
    idx = selection(rng, lens, k)
    qd = torch.from_numpy(rng.normal(size=(n, 64, 576))).bfloat16().cuda()
    out, lse = dsa.sparse_mla_attn(qd, view, i32_dev(idx), k, SCALE)
    dsa.sync_status()
    check_rows(qd, kv, idx, sorted({0, 1, n // 2, n - 1} | {int(r) for r in rng.integers(0, n, 12)}), out, lse)
    first = idx.copy()
    first[0, -1] = lens[0]                    # the second row's newest token is ahead of the first
    got, _ = dsa.sparse_mla_attn(qd, view, i32_dev(first), k, SCALE)
    with pytest.raises(dsa.DsaError) as e:
        dsa.sync_status()
    assert e.value.status == dsa.binding.DSA_ERR_BOUNDS
    first[0, -1] = -1
    check_rows(qd, kv, first, [0], got, _)
    assert torch.equal(got[1:], out[1:])


@pytest.mark.parametrize("pos0,n,k", [(0, 200, 64), (700, 96, 512)])
def test_a_prefill_group_with_dense_keys_over_4bit_pages(pos0, n, k):
    """Dense bf16 indexer keys, causal; the layers' latent caches in 4-bit pages that all rows share."""
    rng = np.random.default_rng(n)
    length = pos0 + n
    keys = torch.from_numpy(rng.normal(size=(length, 128)) / 11).bfloat16().cuda()
    q_idx = torch.from_numpy(rng.normal(size=(n, 32, 128))).bfloat16().cuda()
    w = f32_dev(rng.uniform(0.1, 1.0, size=(n, 32)).astype(np.float32))
    layers = [prompt_view(rng, length, n) for _ in range(3)]
    qs = [torch.from_numpy(rng.normal(size=(n, 64, 576))).bfloat16().cuda() for _ in layers]
    g = dsa.IndexShareGroup(q_idx, w, dsa.dense_view(keys), k, qs, [v for v, _, _ in layers], SCALE, q_pos0=pos0)
    for reuse in (False, True):
        outs, lses = g.forward(reuse_only=reuse)
        dsa.sync_status()
        idx = g.idx.cpu().numpy()
        for r in range(n):
            sel = idx[r][idx[r] >= 0]
            assert len(set(sel)) == len(sel) == min(k, pos0 + r + 1) and sel.max() <= pos0 + r
        for (_, kv, _), q, o, e in zip(layers, qs, outs, lses):
            check_rows(q, kv, idx, sorted({0, n - 1} | {int(r) for r in rng.integers(0, n, 5)}), o, e)


@pytest.mark.parametrize("n_seqs,rows,k", [(1, 1, 2048), (3, 2, 1000), (160, 1, 520), (400, 1, 300)])
def test_selections_whose_first_tiles_are_empty(n_seqs, rows, k):
    """Padding ahead of the entries, over whole tiles; one entry alone, at the very end; parts of a row without a key."""
    rng = np.random.default_rng(k)
    lens = [600] * n_seqs
    idx = np.full((n_seqs, k), -1, dtype=np.int32)
    for b in range(n_seqs):
        m = 1 if b % 3 == 0 else int(rng.integers(1, k - 257))
        idx[b, k - m:] = rng.integers(0, 600, size=m)
    qd, _, kv, out, lse = run_attention(rng, lens, rows, k, idx)
    dsa.sync_status()
    some = sorted({0, n_seqs - 1} | {int(b) for b in rng.integers(0, n_seqs, 8)})
    take = [r for b in some for r in range(b * rows, (b + 1) * rows)]
    check_attention(qd[take], [kv[b] for b in some], idx[some], rows, out[take], lse[take])


# ------------------------------------------------------------------------------------------------ many rows


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mx,layout", [(True, "interleaved"), (True, "half"), (False, "half")])
def test_appends_and_reads_of_many_rows(dtype, mx, layout):
    """More rows than are resident at once: the bytes of calls of 500 rows, a sample of them the oracle's, and read back."""
    rng = np.random.default_rng(31)
    n = 11003
    lens = [5003, 6000]
    n_pages, bt = paged(rng, lens)
    order = rng.permutation(n)
    seq = (order >= lens[0]).astype(np.int32)
    pos = np.where(seq == 1, order - lens[0], order).astype(np.int32)
    x = torch.from_numpy(rng.normal(size=(n, 576)) * np.exp(rng.normal(size=(n, 1)))).to(dtype).cuda()
    gamma = (1 + 0.2 * rng.normal(size=512)).astype(np.float32)
    seqd, posd, btd, lensd, gd = i32_dev(seq), i32_dev(pos), i32_dev(bt), i32_dev(lens), f32_dev(gamma)
    plan = dsa.RopePlan(64, layout=layout)
    blank = garbage_pool(n_pages) if mx else np.full((n_pages, 64, 576), 0x3C, dtype=np.uint8)
    pools = [u8_dev(blank) for _ in range(2)]
    scales = [None if mx else torch.full((n_pages, 64), 0.5, device="cuda") for _ in range(2)]
    views = [dsa.paged_view(p, s, btd, lensd) for p, s in zip(pools, scales)]
    dsa.latent_append(x, posd, views[0], gamma=gd, rope=plan, seq=seqd)
    for a in range(0, n, 500):
        s = slice(a, a + 500)
        dsa.latent_append(x[s], posd[s], views[1], gamma=gd, rope=plan, seq=seqd[s])
    dsa.sync_status()
    assert torch.equal(pools[0], pools[1]) and (mx or torch.equal(scales[0], scales[1]))
    slots = bt[seq, pos // 64].astype(np.int64) * 64 + pos % 64
    got = pools[0].cpu().numpy()
    assert unwritten(blank, got, slots)
    rows = got.reshape(-1, got.shape[-1])[slots]
    some = rng.integers(0, n, 200)
    y = L4.latent_rows(f64(x)[some], gamma, 1e-6, pos[some], L4.inv_freq(64, 8.0e6)[0], 1.0, layout)
    back = dsa.latent_read(views[0], posd, seq=seqd)
    dsa.sync_status()
    if mx:
        assert np.array_equal(rows[some], L4.encode_rows(y))
        assert np.array_equal(f64(back), L4.decode_rows(rows))
    else:
        s = (np.abs(y).max(-1) / np.float32(448.0)).astype(np.float32)
        codes = torch.from_numpy(y / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(rows[some], codes)
        all_s = scales[0].view(-1)[torch.from_numpy(slots).cuda()]
        want = (torch.from_numpy(rows).view(torch.float8_e4m3fn).float().cuda() * all_s[:, None]).bfloat16()
        assert torch.equal(back, want)


def test_reads_over_many_blocks():
    """One prefix, read in an order of its own and more than once."""
    rng = np.random.default_rng(32)
    length, n = 9000, 40000
    n_pages, bt = paged(rng, [length])
    distinct = L4.encode_rows(make_rows(rng, 64))
    pick = rng.integers(0, 64, size=length)
    pool = garbage_pool(n_pages)
    t = np.arange(length)
    pool[bt[0][t // 64], t % 64] = distinct[pick]
    pos = rng.integers(0, length, size=n).astype(np.int32)
    view = dsa.paged_view(u8_dev(pool), None, i32_dev(bt), i32_dev([length]))
    out = torch.full((n + 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    got = dsa.latent_read(view, i32_dev(pos), seq=torch.zeros(n, dtype=torch.int32, device="cuda"), out=out[:n])
    dsa.sync_status()
    vals = torch.from_numpy(L4.decode_rows(distinct)).bfloat16().cuda()
    assert torch.equal(got, vals[torch.from_numpy(pick[pos]).cuda()]) and bool((out[n] == 7.0).all())
