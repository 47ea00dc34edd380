"""The operators of the 4-bit latent cache, as cases to be measured: rotary positions, appending latent rows to a
paged cache, reading them back, and sparse MLA attention over the 4-bit cache.

Each case is one call as a serving program makes it.  ``own`` selects the framework's kernels; otherwise ``run``
computes the same from elementary torch operations.  Sizes are those of this repository's decode and prefill
workloads (64 heads, 576-wide latent rows of 512 + 64 RoPE dims, Top-2,048, 64-token pages, contexts to 2^20) and
ragged ones around them.

The 4-bit row (320 bytes a token): 18 blocks of 32 values, each value an e2m1 code, each block one power-of-two
exponent.  Bytes 0..287: 72 little-endian 32-bit words of 8 values; bits 4i..4i+2 of a word are the magnitude code
of value i; its sign is bit 8i + 7 for i < 4 and bit 8(i - 4) + 3 for i >= 4.  Bytes 288..305: the block exponents
plus 127; the rest is zero.
"""
import math

import torch

own = False

DEV = "cuda"
HEADS, DQK, DV, NOPE, ROT, PAGE = 64, 576, 512, 512, 64, 64
ROW4 = 320
THETA = 8.0e6
EPS = 1e-6
SCALE = 1.0 / math.sqrt(DQK)


def listed():
    return [
        # one sequence of 2^20 tokens: the query token and 5 draft rows that share its selection
        dict(name="attn_1m_mtp5", op="attn", seqs=1, rows=6, k=2048, ctx_lo=1048576, ctx_hi=1048576, chunk=False),
        # decode of sequences of very different lengths, some shorter than the selection (padded rows)
        dict(name="attn_b31_ragged", op="attn", seqs=31, rows=1, k=2048, ctx_lo=700, ctx_hi=262144, chunk=False),
        # decode of 32 long sequences with 4 draft rows each
        dict(name="attn_b32_mtp4", op="attn", seqs=32, rows=5, k=2048, ctx_lo=65536, ctx_hi=262144, chunk=False),
        # a prefill chunk of 512 rows over one sequence's cache, each row with its own selection
        dict(name="attn_chunk_512", op="attn", seqs=512, rows=1, k=2048, ctx_lo=32257, ctx_hi=32768, chunk=True),
        # the RoPE part of one decode step's queries
        dict(name="rope_decode_b32", op="rope", tokens=32, heads=64, dim=64, rot=64, offset=0, dtype="bf16",
             layout="interleaved", scaling="yarn", backward=False, far=1048576),
        # the RoPE part of a prefill chunk's queries
        dict(name="rope_prefill_8k", op="rope", tokens=8192, heads=64, dim=64, rot=64, offset=0, dtype="bf16",
             layout="half", scaling="none", backward=False, far=131072),
        # the gradient of a partly rotated fp32 tensor (training)
        dict(name="rope_grad_fp32", op="rope", tokens=4097, heads=8, dim=128, rot=64, offset=64, dtype="fp32",
             layout="interleaved", scaling="linear", backward=True, far=524288),
        # a decode step's new latent rows into the 4-bit cache, normalised and rotated on the way
        dict(name="append4_decode_b32", op="append", seqs=32, tokens=32, fmt="mxfp4", dtype="bf16", norm=True,
             layout="interleaved", scaling="none", far=65536),
        # a prefill chunk's rows into the 4-bit cache
        dict(name="append4_prefill_8k", op="append", seqs=1, tokens=8192, fmt="mxfp4", dtype="bf16", norm=True,
             layout="interleaved", scaling="none", far=131072),
        # fp32 projection rows of several ragged sequences into the e4m3 cache
        dict(name="append8_ragged", op="append", seqs=7, tokens=4095, fmt="e4m3", dtype="fp32", norm=True,
             layout="half", scaling="yarn", far=65536),
        # a cached prefix read back, for a chunk that attends to it densely
        dict(name="read4_prefix_32k", op="read", seqs=1, tokens=32768, fmt="mxfp4"),
        # e4m3 rows of a few sequences read back
        dict(name="read8_ragged", op="read", seqs=5, tokens=6001, fmt="e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "append", "read"])
    if op == "attn":
        rows = rng.choice([1, 1, 2, 3, 5, 6])
        k = _log(rng, 16, 2048) if rng.random() < 0.5 else rng.choice([512, 1024, 2048, 2047])
        seqs = _log(rng, 1, max(1, min(512, 1048576 // (k * rows))))
        hi = _log(rng, 64, max(64, min(1048576, 6000000 // seqs)))
        lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
        if rows == 1 and rng.random() < 0.3:
            return dict(op=op, seqs=seqs, rows=1, k=k, ctx_lo=lo, ctx_hi=lo + seqs - 1, chunk=True)
        return dict(op=op, seqs=seqs, rows=rows, k=k, ctx_lo=lo, ctx_hi=hi, chunk=False)
    layout, scaling = rng.choice(["interleaved", "half"]), rng.choice(["none", "linear", "ntk", "yarn"])
    far = _log(rng, 256, 1048576)
    if op == "rope":
        dtype, rot = rng.choice(["bf16", "fp16", "fp32"]), rng.choice([16, 32, 64, 128])
        dim, offset = rng.choice([(rot, 0), (rot + 64, 64), (rot + 64, 0)])
        heads = rng.choice([1, 2, 8, 32, 64])
        tokens = _log(rng, 1, max(1, 33554432 // (heads * dim)))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, rot=rot, offset=offset, dtype=dtype, layout=layout,
                    scaling=scaling, backward=rng.random() < 0.3, far=far)
    tokens = _log(rng, 1, 8192 if op == "append" else 32768)
    seqs, fmt = _log(rng, 1, min(tokens, 64)), rng.choice(["mxfp4", "mxfp4", "e4m3"])
    if op == "read":
        return dict(op=op, seqs=seqs, tokens=tokens, fmt=fmt)
    return dict(op=op, seqs=seqs, tokens=tokens, fmt=fmt, dtype=rng.choice(["bf16", "fp32"]), norm=rng.random() < 0.7,
                layout=layout, scaling=scaling, far=min(far, 2000000 // seqs))


# ------------------------------------------------------------------------------------------------ inputs

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV)


def _row_amax_code(y):
    """Block exponents (0 .. 26, standing for -13 .. 13) of rows y [n, 576] fp32: the least one at which no value of
    the block exceeds 6 steps."""
    amax = y.abs().view(-1, 18, 32).amax(-1)
    mant, ex = torch.frexp(amax)                       # amax = mant * 2^ex, mant in [0.5, 1)
    e = ex - 3 + (mant > 0.75).int()                   # amax <= 6 * 2^e = 0.75 * 2^(e + 3)
    return torch.where(amax > 0, e, torch.full_like(e, -13)).clamp(-13, 13) + 13


def _pow2(e):
    """2^e of an int32 tensor, fp32, exactly."""
    return ((e + 127) << 23).view(torch.float32)


def _e2m1(v):
    """Magnitude codes of |v| <= 6 (ties to the even code), above 6: 6."""
    return ((v > 0.25).int() + (v >= 0.75).int() + (v > 1.25).int() + (v >= 1.75).int() + (v > 2.5).int()
            + (v >= 3.5).int() + (v > 5.0).int())


def _pack4(y):
    """4-bit rows [n, 320] uint8 of rows y [n, 576] fp32 (inputs of the attention and read cases)."""
    e = _row_amax_code(y)
    v = y.view(-1, 18, 32) * _pow2(13 - e).unsqueeze(-1)
    mag, sign = _e2m1(v.abs()).view(-1, 72, 8).long(), (v < 0).view(-1, 72, 8).long()
    i = torch.arange(8, device=y.device)
    w = ((mag << (4 * i)) | (sign << torch.where(i < 4, 8 * i + 7, 8 * (i - 4) + 3))).sum(-1)
    by = (w.unsqueeze(-1) >> (8 * torch.arange(4, device=y.device))) & 255
    out = torch.zeros(y.shape[0], ROW4, dtype=torch.uint8, device=y.device)
    out[:, :288] = by.view(-1, 288).to(torch.uint8)
    out[:, 288:306] = (e + 114).to(torch.uint8)
    return out


def _latent_rows(g, n):
    """Rows as a cache holds them: normalised latents with a spread of channel weights, a larger RoPE part."""
    y = _normal(g, n, DQK) * torch.exp(0.3 * _normal(g, DQK))
    y[:, NOPE:] *= 2.0
    return y


def _tables(g, lens):
    """Block table of sequences of the given lengths over a permuted page pool: (n_pages, table [B, max_pages])."""
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    total, width = sum(pages), max(pages)
    perm = torch.randperm(total, generator=g, device=DEV).int()
    first = torch.tensor([0] + pages[:-1], device=DEV).cumsum(0)
    count = torch.tensor(pages, device=DEV)
    col = torch.arange(width, device=DEV)
    at = (first[:, None] + col).clamp(max=total - 1)
    return total, torch.where(col < count[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()


def _lengths(case, seed):
    g = torch.Generator().manual_seed(seed)
    return [int(v) for v in torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (case["seqs"],), generator=g)]


def _spread(case, seed):
    """Tokens of the case over its sequences, ragged: sequence and position of each row, and the sequences' lengths."""
    g = torch.Generator().manual_seed(seed)
    n, s = case["tokens"], case["seqs"]
    cuts = sorted(int(v) for v in torch.randperm(n - 1, generator=g)[: s - 1] + 1) if n > 1 else []
    counts = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    far = case.get("far", 4 * n)
    start = [int(torch.randint(0, max(1, far - c), (1,), generator=g)) if c < far else 0 for c in counts]
    lens = [a + c for a, c in zip(start, counts)]
    seq = torch.arange(s).repeat_interleave(torch.tensor(counts)).int().to(DEV)
    pos = torch.cat([torch.arange(a, a + c) for a, c in zip(start, counts)]).int().to(DEV)
    return seq, pos, lens


def _rope_args(case, rot):
    """Keyword arguments of a rotation plan."""
    kind = case["scaling"]
    a = dict(rot_dim=rot, theta=THETA, layout=case["layout"], scaling=None if kind == "none" else kind)
    if kind != "none":
        a["factor"] = 8.0
    if kind == "yarn":
        a["original_len"] = 131072
    return a


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if own:
        import long_context_sparse_11_b200 as dsa
        s["dsa"] = dsa
    if op == "attn":
        lens = _lengths(case, seed)
        if case["chunk"]:
            # every row of the chunk reads the one sequence's cache up to itself
            lens = list(range(case["ctx_lo"], case["ctx_lo"] + case["seqs"]))
            n_pages, table = _tables(g, [lens[-1]])
            table = table.expand(case["seqs"], -1).contiguous()
        else:
            n_pages, table = _tables(g, lens)
        base = _pack4(_latent_rows(g, 8192))
        pool = base[_ints(g, 0, 8192, n_pages * PAGE)].view(n_pages, PAGE, ROW4)
        n, k = torch.tensor(lens, device=DEV).double()[:, None], case["k"]
        # the selection of a row: k distinct positions spread over its context, in no order, padded with -1
        j = torch.arange(k, device=DEV).double()
        u = torch.rand(len(lens), k, generator=g, device=DEV, dtype=torch.float64)
        far = torch.floor((j + u) * n / k).clamp(max=n - 1)
        idx = torch.where(n > k, far, torch.where(j < n, j, -torch.ones_like(j))).int()
        if max(lens) > k:
            idx = idx[:, torch.randperm(k, generator=g, device=DEV)]
        s["idx"], s["k"], s["rows"] = idx.contiguous(), k, case["rows"]
        nq = len(lens) * case["rows"]
        s["q"] = _normal(g, nq, HEADS, DQK).bfloat16()
        s["pool"], s["table"] = pool, table
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        if own:
            s["view"] = dsa.paged_view(pool, None, table, s["lens"])
            s["out"] = torch.empty(nq, HEADS, DV, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(nq, HEADS, dtype=torch.float32, device=DEV)
            need = dsa.sparse_mla_workspace_bytes(nq, k, s["view"])
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        return s
    if op == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        # the rotated tensor is a slice of wider rows, as the RoPE part of the queries is
        s["x"] = _normal(g, t, h, d + 64).to(DTYPES[case["dtype"]])[:, :, 64:]
        s["pos"] = _ints(g, 0, case["far"], t).int()
        s["out"] = torch.empty(t, h, d, dtype=DTYPES[case["dtype"]], device=DEV)
        s["args"] = _rope_args(case, case["rot"])
        s["freq"] = _inv_freq(**s["args"])
        if own:
            s["plan"] = dsa.RopePlan(**s["args"])
        return s
    if op == "append":
        s["seq"], s["pos"], lens = _spread(case, seed)
        x = _normal(g, case["tokens"], DQK) * torch.exp(0.5 * _normal(g, case["tokens"], 1))
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["gamma"] = 1.0 + 0.1 * _normal(g, NOPE) if case["norm"] else None
        s["args"] = _rope_args(case, ROT)
        s["freq"] = _inv_freq(**s["args"])
    else:
        s["seq"], s["pos"], lens = _spread(case, seed)
    n_pages, s["table"] = _tables(g, lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    scale = None
    if case["fmt"] == "mxfp4":
        base = _pack4(_latent_rows(g, 4096))
        pool = base[_ints(g, 0, 4096, n_pages * PAGE)].view(n_pages, PAGE, ROW4)
    else:
        base = (2.0 * _normal(g, 4096, DQK)).clamp(-7, 7) * 64.0
        base = base.to(torch.float8_e4m3fn).view(torch.uint8)
        pool = base[_ints(g, 0, 4096, n_pages * PAGE)].view(n_pages, PAGE, DQK)
        scale = torch.rand(n_pages, PAGE, generator=g, device=DEV) / 96 + 1.0 / 128
    s["pool"], s["scale"] = pool, scale
    s["out"] = torch.empty(case["tokens"], DQK, dtype=torch.bfloat16, device=DEV)
    if own:
        s["view"] = dsa.paged_view(pool, scale, s["table"], s["lens"])
        if op == "append":
            s["plan"] = dsa.RopePlan(**s["args"])
    return s


# ------------------------------------------------------------------------------------------------ plain forms


def _inv_freq(rot_dim, theta, layout, scaling, factor=1.0, original_len=0):
    """Angle per position of each pair (fp64) and the factor on the rotated values."""
    d = rot_dim
    i = torch.arange(d // 2, dtype=torch.float64, device=DEV)
    if scaling == "ntk":
        theta = theta * factor ** (d / (d - 2))
    f = torch.exp(-2.0 * i / d * math.log(theta))
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0

    def at(turns):
        return d * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))

    low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _turned(x, pos, freq, layout, backward=False):
    """x [n, ..., rot] fp64 turned by its positions, unrounded."""
    f, m = freq
    a = pos.double()[:, None] * f
    c, t = torch.cos(a) * m, torch.sin(a) * (-m if backward else m)
    if x.dim() == 3:
        c, t = c[:, None], t[:, None]
    half = layout == "half"
    d = x.shape[-1]
    a, b = (x[..., : d // 2], x[..., d // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * c - b * t, a * t + b * c
    return torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)


def _value(mag):
    """Values of e2m1 magnitude codes, fp32."""
    return torch.where(mag < 2, mag * 0.5, (2.0 + (mag & 1)) * _pow2((mag >> 1) - 2))


def _unpack4(rows):
    """Values [..., 576] fp32 of 4-bit rows [..., 320]."""
    lead = rows.shape[:-1]
    by = rows[..., :288].reshape(*lead, 72, 4).int()
    # the magnitudes of values 2j and 2j + 1 are in byte j, the signs of values i and 4 + i in byte i
    mag = torch.stack([by & 7, (by >> 4) & 7], -1).flatten(-2)
    sign = torch.cat([by >> 7, (by >> 3) & 1], -1)
    v = (_value(mag) * (1 - 2 * sign)).view(*lead, 18, 32)
    e = rows[..., 288:306].int().clamp(114, 140) - 127
    return (v * _pow2(e).unsqueeze(-1)).view(*lead, DQK)


def _slots(table, seq, pos):
    return table[seq.long(), (pos // PAGE).long()].long() * PAGE + (pos % PAGE).long()


def _read(s):
    at = _slots(s["table"], s["seq"], s["pos"])
    if s["scale"] is None:
        return _unpack4(s["pool"].view(-1, ROW4)[at]).bfloat16()
    codes = s["pool"].view(-1, DQK)[at].view(torch.float8_e4m3fn).float()
    return (codes * s["scale"].view(-1)[at][:, None]).bfloat16()


def _append_rows(s):
    """The rows that an append stores, before quantisation (fp32, from 64-bit arithmetic: a value next to a border
    of its 4-bit grid must not go to the other side)."""
    x = s["x"].double()
    lat, rope = x[:, :NOPE], x[:, NOPE:]
    if s["gamma"] is not None:
        lat = lat / torch.sqrt((lat * lat).mean(-1, keepdim=True) + EPS) * s["gamma"].double()
    return torch.cat([lat, _turned(rope, s["pos"], s["freq"], s["case"]["layout"])], -1).float()


def _quantised(y, fmt):
    """The values that the cache holds for rows y, bf16."""
    if fmt == "mxfp4":
        e = (_row_amax_code(y) - 13).unsqueeze(-1)
        v = y.view(-1, 18, 32) * _pow2(-e)
        return (_value(_e2m1(v.abs())) * torch.where(v < 0, -1.0, 1.0) * _pow2(e)).view(-1, DQK).bfloat16()
    amax = y.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return ((y / scale).to(torch.float8_e4m3fn).float() * scale).bfloat16()


def _attention(s):
    idx, rows = s["idx"].long(), s["rows"]
    valid = idx >= 0
    at = _slots(s["table"], torch.arange(idx.shape[0], device=DEV)[:, None], idx.clamp(min=0))
    kv = _unpack4(s["pool"].view(-1, ROW4)[at])                                   # [B, k, 576]
    q = s["q"].float().view(idx.shape[0], rows * HEADS, DQK)
    z = torch.bmm(q, kv.transpose(1, 2)) * SCALE
    z = torch.where(valid[:, None], z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    out = torch.bmm(p, kv[:, :, :DV]) / l
    lse = m + torch.log(l)
    return out.view(-1, HEADS, DV).bfloat16(), lse.view(-1, HEADS)


def run(state):
    s = state
    op, case = s["op"], s["case"]
    if own:
        dsa = s["dsa"]
        if op == "attn":
            return dsa.sparse_mla_attn(s["q"], s["view"], s["idx"], s["k"], SCALE, s["rows"], out=s["out"],
                                       lse=s["lse"], workspace=s["ws"])
        if op == "rope":
            return dsa.rope(s["x"], s["pos"], s["plan"], offset=case["offset"], backward=case["backward"],
                            out=s["out"])
        if op == "append":
            dsa.latent_append(s["x"], s["pos"], s["view"], gamma=s["gamma"], eps=EPS, rope=s["plan"], seq=s["seq"])
        return dsa.latent_read(s["view"], s["pos"], seq=s["seq"], out=s["out"])
    if op == "attn":
        return _attention(s)
    if op == "rope":
        x, o, r = s["x"], case["offset"], case["rot"]
        y = _turned(x[..., o:o + r].double(), s["pos"], s["freq"], case["layout"], case["backward"]).to(x.dtype)
        return torch.cat([x[..., :o], y, x[..., o + r:]], -1)
    return _quantised(_append_rows(s), case["fmt"]) if op == "append" else _read(s)


# ------------------------------------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op == "attn":
        nq = case["seqs"] * case["rows"]
        mean = (case["ctx_lo"] + case["ctx_hi"]) / 2
        # expected selected keys of a row: min(k, length), the length uniform between the ends
        lo, hi, k = case["ctx_lo"], case["ctx_hi"], case["k"]
        keys = float(k) if lo >= k else mean if hi <= k else ((lo + k) / 2 * (k - lo) + k * (hi - k)) / (hi - lo)
        # a latent row that several selections hold is read from memory once
        table = min(case["seqs"] * keys, hi) if case["chunk"] else case["seqs"] * keys
        byt = table * 306 + case["seqs"] * k * 4 + nq * HEADS * (DQK * 2 + DV * 2 + 4)
        return {"bytes": byt, "flops": nq * keys * HEADS * 2 * (DQK + DV)}
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * size + case["tokens"] * 4,
                "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    row = 306 if case["fmt"] == "mxfp4" else 580
    if op == "read":
        return {"bytes": case["tokens"] * (row + DQK * 2 + 8), "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    # the rows in, the cache's rows out, and once more back as values
    return {"bytes": case["tokens"] * (DQK * size + 2 * row + DQK * 2 + 8), "flops": 10 * case["tokens"] * DQK}


# ------------------------------------------------------------------------------------------------ 64 bits


def exact(case, seed):
    def power(e):
        """2^e of an int64 tensor, fp64, exactly."""
        return ((e + 1023) << 52).view(torch.float64)

    def decode(rows):
        """Values of 4-bit rows by the definition, value by value of a word."""
        b = rows.long()
        word = b[..., 0:288:4] + 256 * b[..., 1:288:4] + 65536 * b[..., 2:288:4] + 16777216 * b[..., 3:288:4]
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        vals = []
        for i in range(8):
            bit = 8 * i + 7 if i < 4 else 8 * (i - 4) + 3
            vals.append(grid[(word // 16 ** i) % 8] * (1 - 2 * ((word // 2 ** bit) % 2)).double())
        v = torch.stack(vals, -1).reshape(*rows.shape[:-1], 18, 32)
        return (v * power(b[..., 288:306] - 127).unsqueeze(-1)).reshape(*rows.shape[:-1], DQK)

    def turn(x, pos, args, backward):
        """x [n, h, rot] turned pair by pair, as complex numbers."""
        d, kind, base = args["rot_dim"], args["scaling"], args["theta"]
        s, length = args.get("factor", 1.0), args.get("original_len", 0)
        if kind == "ntk":
            base *= s ** (d / (d - 2))
        mult = 0.1 * math.log(s) + 1 if kind == "yarn" else 1.0
        out = torch.empty_like(x)
        for i in range(d // 2):
            f = base ** (-2.0 * i / d)
            if kind == "linear":
                f /= s
            if kind == "yarn":
                lo = max(math.floor(d * math.log(length / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
                hi = min(math.ceil(d * math.log(length / (2 * math.pi)) / (2 * math.log(base))), d - 1)
                r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                f = f * (1 - r) + f / s * r
            a, b = (i, i + d // 2) if args["layout"] == "half" else (2 * i, 2 * i + 1)
            angle = torch.remainder(pos.double() * f, 2 * math.pi)
            unit = torch.polar(torch.full_like(angle, mult), -angle if backward else angle)
            z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * unit[:, None]
            out[..., a], out[..., b] = z.real, z.imag
        return out

    def nearest(v, grid):
        """Each value of v moved to the nearest of the sorted grid's values, ties to the even place."""
        hi = torch.searchsorted(grid, v.contiguous()).clamp(1, len(grid) - 1)
        lo = hi - 1
        a, b = v - grid[lo], grid[hi] - v
        return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), grid[lo], grid[hi])

    s, op = prepare(case, seed), case["op"]
    if op == "attn":
        outs, lses = [], []
        rows = s["rows"]
        for b in range(s["idx"].shape[0]):
            sel = s["idx"][b][s["idx"][b] >= 0].long()
            page = s["table"][b][sel // PAGE].long()
            kv = decode(s["pool"][page, sel % PAGE])
            z = s["q"][b * rows:(b + 1) * rows].double() @ kv.T * SCALE
            lses.append(torch.logsumexp(z, -1))
            outs.append(torch.softmax(z, -1) @ kv[:, :DV])
        return torch.cat(outs), torch.cat(lses)
    if op == "rope":
        x, o, r = s["x"].double().clone(), case["offset"], case["rot"]
        x[..., o:o + r] = turn(x[..., o:o + r].clone(), s["pos"], s["args"], case["backward"])
        return x
    if op == "read":
        page, slot = s["table"][s["seq"].long(), s["pos"].long() // PAGE].long(), s["pos"].long() % PAGE
        rows = s["pool"][page, slot]
        if case["fmt"] == "mxfp4":
            return decode(rows)
        return rows.view(torch.float8_e4m3fn).double() * s["scale"][page, slot].double()[:, None]
    x = s["x"].double()
    if s["gamma"] is not None:
        rms = torch.linalg.vector_norm(x[:, :NOPE], dim=-1, keepdim=True) / math.sqrt(NOPE)
        x[:, :NOPE] = x[:, :NOPE] / torch.sqrt(rms ** 2 + EPS) * s["gamma"].double()
    x[:, NOPE:] = turn(x[:, None, NOPE:].clone(), s["pos"], s["args"], False)[:, 0]
    y = x.float().double()                             # the cache's quantisation starts from fp32 values
    if case["fmt"] == "mxfp4":
        blocks = y.view(-1, 18, 32)
        amax = blocks.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2((amax / 6).clamp(min=2.0 ** -20))).long()
        e = torch.where(amax > 6 * power(e), e + 1, torch.where(amax <= 3 * power(e), e - 1, e))  # log2's own rounding
        step = power(e.clamp(-13, 13))
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        return (nearest((blocks / step).abs().clamp(max=6), grid) * torch.sign(blocks) * step).view(-1, DQK)
    amax = y.abs().amax(-1, keepdim=True)
    scale = (amax / torch.full_like(amax, 448.0)).float().double()
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    quotient = (y / scale).float().double()
    grid = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    return nearest(quotient.abs().clamp(max=448), grid) * torch.sign(quotient) * scale
