"""The 8-bit KV cache on the GPU against its fp64 oracle (oracle/kv8.py): codes
and magnitudes exactly, values and attention within bounds that count the
roundings."""
import numpy as np
import pytest
import torch

import greedy_speculative_verify_b200 as vgv
import oracle
import synth_inputs as si
from oracle import kv8

from gpu_common import ACT_TOL, D as DIMS, Guarded, dev, ensure_lib, row_rel_err

pytestmark = pytest.mark.gpu
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
FORMATS = ["int8", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()
    vgv.vg_get_device_status()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    """A cache on the device (inside guard regions) beside its oracle state."""

    def __init__(self, fmt, B, n_kv, L, dim, block, seed=0, fill=True, never=0x7F):
        g = np.random.default_rng(seed)
        self.fmt, self.B, self.n_kv, self.L, self.dim, self.block, self.g = fmt, B, n_kv, L, dim, block, g
        self.codes, self.amax = {}, {}
        self.gd = Guarded()
        t = {}
        for x in "kv":
            amax = np.zeros((B, n_kv, L // block))
            raw = np.full((B, n_kv, L, dim), never, np.uint8)  # bytes that were never written: NaN in e4m3
            if fill:
                amax = oracle.widen(oracle.round_bf16_bits(np.abs(g.normal(0, 1, amax.shape)) + 0.5))
                codes = kv8.to_grid(g.uniform(-1, 1, raw.shape) * kv8.Q_OF[fmt], fmt)
                raw = kv8.pack(codes, fmt, x == "v")
            self.codes[x], self.amax[x] = kv8.unpack(raw, fmt, x == "v"), amax
            t[x] = self.gd.empty((B, n_kv, L, dim), torch.uint8)
            t[x].copy_(torch.from_numpy(raw))
            t[x + "a"] = self.gd.empty((B, n_kv, L // block), torch.float32)
            t[x + "a"].copy_(torch.from_numpy(amax.astype(np.float32)))
        self.t = t
        self.h = vgv.make_kv8(t["k"].view(CODE[fmt]), t["v"].view(CODE[fmt]), t["ka"], t["va"])

    def append(self, rows, pos, n_new, x=None, stride_pad=0):
        """The same rows into both; x: {"k", "v"} fp64 [B, rows, n_kv, dim], bf16 values."""
        w = self.n_kv * self.dim
        x = x or {y: oracle.widen(oracle.round_bf16_bits(self.g.normal(0, 1, (self.B, rows, self.n_kv, self.dim)))) for y in "kv"}
        d = {}
        for y in "kv":
            m = torch.full((self.B * rows, w + stride_pad), float("nan"), dtype=torch.bfloat16, device="cuda")
            m[:, :w] = torch.from_numpy(x[y].reshape(-1, w).astype(np.float32)).to("cuda")
            d[y] = m[:, :w]
        vgv.vg_kv8_append(self.h, rows, d["k"], d["v"], i32(pos), n_new=None if n_new is None else i32(n_new))
        for y in "kv":
            kv8.append(self.codes[y], self.amax[y], x[y], pos, [rows] * self.B if n_new is None else n_new, self.block, self.fmt)
        return x

    def check(self, written=None):
        """Every byte and magnitude as the oracle has them (written [B]: only positions below it)."""
        self.gd.check()
        for y in "kv":
            got = kv8.unpack(self.t[y].cpu().numpy(), self.fmt, y == "v")
            assert np.array_equal(self.t[y + "a"].cpu().numpy().astype(np.float64), self.amax[y]), y
            for b in range(self.B):
                n = self.L if written is None else written[b]
                assert np.array_equal(got[b, :, :n], self.codes[y][b, :, :n], equal_nan=True), (y, b)

    def values(self):
        return [kv8.values(np.nan_to_num(self.codes[y]), self.amax[y], self.block, self.fmt) for y in "kv"]


def ok():
    torch.cuda.synchronize()
    st, info = vgv.vg_get_device_status()
    assert st == 0, (st, info)


# ------------------------------------------------------------------ writing
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,block,n_kv", [(64, 16, 3), (128, 32, 1), (128, 64, 10), (64, 128, 2), (128, 128, 2), (128, 16, 2)])
def test_append(fmt, dim, block, n_kv):
    """Writes inside a block, over its end, from its start, none at all, over
    many blocks; then again over the same positions (rejected drafts) with rows
    a hundred times larger, and smaller."""
    L = 4 * block
    c = Cache(fmt, 6, n_kv, L, dim, block, seed=dim + block)
    rows = 2 * block + 3
    pos, n = [0, 1, block - 1, block, 5, L - rows], [4, block, rows, 0, 1, rows]
    c.append(rows, pos, n, stride_pad=8)
    ok()
    c.check()
    for size in (100.0, 0.01):
        x = {y: oracle.widen(oracle.round_bf16_bits(c.g.normal(0, size, (6, 4, n_kv, dim)))) for y in "kv"}
        c.append(4, [3, block - 2, block - 1, block, 2 * block + 9, L - 4], None, x=x)
        ok()
        c.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
def test_append_few_rows(fmt, dim):
    """One to nine rows (a verify step takes a path of its own) from every
    position of a group of 16, over block ends, magnitudes growing and not."""
    c = Cache(fmt, 16, 2, 128, dim, 32, seed=31)
    for rows in range(1, 10):
        for at in (0, 16, 48, 128 - 15 - rows):
            size = float(c.g.choice([0.1, 3.0]))
            x = {y: oracle.widen(oracle.round_bf16_bits(c.g.normal(0, size, (16, rows, 2, dim)))) for y in "kv"}
            c.append(rows, [at + b for b in range(16)], [min(rows, 1 + (b + at) % 9) for b in range(16)], x=x)
    ok()
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_rounds_ties_to_even(fmt):
    """Rows whose quotients by the magnitude are exact ties (x Q / a = k + 1/2, in
    e4m3 halfway between neighbours), for several magnitudes, and earlier codes
    rounded again at exact ties."""
    c = Cache(fmt, 1, 1, 64, 64, 16, fill=False)
    Q = kv8.Q_OF[fmt]
    x = {}
    for y, a in (("k", 2.0 * Q if fmt == "int8" else 448.0), ("v", 7.0 if fmt == "e4m3" else 127.0 / 64)):
        r = np.zeros((1, 16, 1, 64))
        grid = (np.arange(16 * 64).reshape(16, 64) % 254 - 127 + 0.5) if fmt == "int8" else \
            np.sign(np.arange(16 * 64).reshape(16, 64) % 2 - 0.5) * 2.0 ** (np.arange(64) % 14 - 7)[None] * (17 + 2 * (np.arange(16) % 8)[:, None]) / 16
        r[0, :, 0] = oracle.widen(oracle.round_bf16_bits(np.clip(grid, -Q, Q) * a / Q))
        r[0, 0, 0, 0] = a
        x[y] = r
    c.append(16, [0], None, x=x)
    ok()
    c.check(written=[16])
    for grow in (4.0 / 3, 2.0, 1.25):  # earlier codes times 3/4, 1/2, 4/5
        # the written magnitude of both halves of the cache grows by the factor
        x = {y: oracle.widen(oracle.round_bf16_bits(np.full((1, 1, 1, 64), c.amax[y][0, 0, 0] * grow))) for y in "kv"}
        c.append(1, [15], None, x=x)
        ok()
        c.check(written=[16])


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_extremes(fmt):
    """Zeros, the smallest and largest bf16 magnitudes, a block of zeros that
    grows, and infinities and NaN (recorded; stored as the largest code and 0)."""
    c = Cache(fmt, 5, 2, 64, 64, 32, fill=False)
    x = {y: np.zeros((5, 8, 2, 64)) for y in "kv"}
    for y in "kv":
        x[y][1] = oracle.widen(oracle.round_bf16_bits(c.g.normal(0, 1, (8, 2, 64)) * 2.0 ** -125))
        x[y][2] = 2.0 ** -133 * c.g.integers(-3, 4, (8, 2, 64))
        x[y][3] = oracle.widen(oracle.round_bf16_bits(c.g.uniform(-1, 1, (8, 2, 64)) * 3.3e38))
        x[y][4] = oracle.widen(oracle.round_bf16_bits(c.g.normal(0, 1, (8, 2, 64))))
    c.append(8, [0] * 5, None, x=x)
    ok()
    c.check(written=[8] * 5)
    x = {y: v[:, ::-1].copy() * 1.0 for y, v in x.items()}
    for y in "kv":
        x[y][0] = 1.5
        x[y][4, 0, 0, :3] = [np.inf, -np.inf, np.nan]
        x[y][4, 1, 1, 5] = np.nan
    c.append(8, [8] * 5, None, x=x)
    torch.cuda.synchronize()
    assert vgv.vg_get_device_status() == (6, 341)
    c.check(written=[16] * 5)


def test_append_bad_positions_leave_the_sequence():
    c = Cache("int8", 6, 1, 32, 64, 16, seed=3)
    x = {y: np.ones((6, 4, 1, 64)) for y in "kv"}
    before = {y: (c.codes[y].copy(), c.amax[y].copy()) for y in "kv"}
    c.append(4, [0] * 6, [4, 0, 0, 0, 0, 0], x=x)
    good = {y: (c.codes[y].copy(), c.amax[y].copy()) for y in "kv"}
    ok()
    d = torch.ones(24, 64, dtype=torch.bfloat16, device="cuda")
    vgv.vg_kv8_append(c.h, 4, d, d.clone(), i32([0, -1, 29, 5, 7, 2 ** 31 - 1]), n_new=i32([4, 4, 4, 5, -1, 4]))
    torch.cuda.synchronize()
    assert vgv.vg_get_device_status() == (6, 340)
    for y in "kv":
        assert np.array_equal(good[y][0][1:], before[y][0][1:])
    c.check()


# ------------------------------------------------------------------ reading
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 64)])
def test_read(fmt, dtype, dim, block):
    B, n_kv, L, rows = 5, 3, 192, 70
    c = Cache(fmt, B, n_kv, L, dim, block, seed=7)
    pos, n = [0, 15, 122, 191, 33], [70, 1, 70, 1, 0]
    w = n_kv * dim
    wide = torch.full((B * rows, 2 * w + 8), -3.0, dtype=dtype, device="cuda")
    k_out, v_out = wide[:, :w], wide[:, w + 8:]
    vgv.vg_kv8_read(c.h, rows, i32(pos), k_out, v_out, n_rows=i32(n))
    ok()
    # two fp32 roundings, and one to bf16
    tol = 2 * 2.0 ** -24 * 1.001 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    got = wide.double().cpu().numpy().reshape(B, rows, -1)
    assert (got[:, :, w:w + 8] == -3.0).all()
    for y, ref, part in (("k", c.values()[0], got[:, :, :w]), ("v", c.values()[1], got[:, :, w + 8:])):
        for b in range(B):
            r = ref[b, :, pos[b]:pos[b] + n[b]].transpose(1, 0, 2).reshape(n[b], w)
            assert (np.abs(part[b, :n[b]] - r) <= tol * np.abs(r)).all(), (y, b)
            assert (part[b, n[b]:] == -3.0).all(), (y, b)
    only = torch.full((B * rows, w), -3.0, dtype=dtype, device="cuda")
    vgv.vg_kv8_read(c.h, rows, i32(pos), None, only, n_rows=i32(n))
    ok()
    assert torch.equal(only, v_out)
    vgv.vg_kv8_read(c.h, rows, i32([0, -1, 193, 0, 0]), only, None, n_rows=i32([1, 1, 0, 71, -1]))
    torch.cuda.synchronize()
    assert vgv.vg_get_device_status() == (6, 342)
    assert (only.view(B, rows, w)[1:] == v_out.reshape(B, rows, w)[1:]).all()


# ------------------------------------------------------------------ attention
def check_attention(c, rows, n_heads, lens, seed=0, first=None, n_new=None, pad=0, q_size=1.0, scale=None):
    g = np.random.default_rng(seed)
    scale = scale or c.dim ** -0.5
    w = n_heads * c.dim
    q = oracle.widen(oracle.round_bf16_bits(g.normal(0, q_size, (c.B, rows, n_heads, c.dim))))
    qd = torch.full((c.B * rows, w + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    qd[:, :w] = torch.from_numpy(q.reshape(-1, w).astype(np.float32)).to("cuda")
    if n_new is not None:  # padded rows are not read
        for b in range(c.B):
            qd[b * rows + int(n_new[b]):(b + 1) * rows] = float("nan")
    gd = Guarded()
    od = gd.empty((c.B * rows, w + pad), torch.bfloat16, fill=-3.0)
    ws = gd.empty((max(16, vgv.vg_kv8_attn_workspace_bytes(c.h, rows, n_heads)),), torch.uint8, fill=0)
    args = dict(first=None if first is None else i32(first), n_new=None if n_new is None else i32(n_new))
    vgv.vg_kv8_attn(c.h, rows, n_heads, qd[:, :w], i32(lens), scale, od[:, :w], ws, **args)
    ok()
    gd.check()
    once = od.clone()
    vgv.vg_kv8_attn(c.h, rows, n_heads, qd[:, :w], i32(lens), scale, od[:, :w], ws, **args)
    ok()
    assert torch.equal(once, od)  # the same bits again
    assert int(ws[:4096].count_nonzero()) == 0  # its counters are zero again
    k, v = c.values()
    ref, mag, size = kv8.attention(q, k, v, lens, scale, first, n_new)
    got = od[:, :w].double().cpu().numpy().reshape(ref.shape)
    assert (od[:, w:] == -3.0).all()
    # scores: fp32 sums of dim exact products and three more roundings, each within 2^-23 of the sum of
    # magnitudes (tensor-core sums may truncate), and the exponent's argument rounded (log2 units);
    # weights: two of them enter (numerator and sum), 2^-21 for the exponential; f16 rounding 2^-11 of the
    # numerator's; sums over up to L positions; the result's rounding to bf16, 2^-8. A weight times its block's
    # share of the largest value magnitude, lifted by 2^9, that falls below f16's normal range is off by at most
    # half its subnormal step, 2^-25, so by 2^-34 of the largest value before the lift, for each position; the
    # largest weight is at least 1 (the running maximum is one of the scores), and so is their sum.
    # int8 keys enter the sums as code + 128, and 128 times the row's sum comes off again: magnitudes up to
    # (|c| + 128) |q|.
    L = max(lens) + rows
    seen = [(lens[b] + rows + c.block - 1) // c.block for b in range(c.B)]
    top_k, top_v = (np.array([c.amax[y][b, :, :seen[b]].max() for b in range(c.B)]) for y in "kv")
    if c.fmt == "int8":
        size = size + np.abs(q).sum(axis=3) * scale * top_k[:, None, None] * 128 / 127
    eps_s = (c.dim + 8) * 2.0 ** -23 * size[..., None]
    tol = mag * (2.0 ** -11 + 2 * (eps_s + 2.0 ** -21) + (L + 64) * 2.0 ** -23) + 2.0 ** -8 * np.abs(ref) + 1e-38
    tol = tol + (L * 2.0 ** -34 * top_v)[:, None, None, None]
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= tol).all(), float((err / tol).max())
    return od, got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,block,n_kv,group,rows", [
    (128, 64, 10, 1, 4), (128, 16, 1, 1, 1), (64, 16, 2, 4, 3), (128, 32, 2, 8, 8), (64, 128, 3, 2, 8), (128, 128, 1, 16, 7),
    (128, 64, 2, 3, 5), (64, 32, 1, 8, 1), (128, 64, 2, 4, 8), (64, 16, 1, 3, 8), (128, 32, 1, 5, 7)])
def test_attention(fmt, dim, block, n_kv, group, rows):
    """Ragged lengths from no cached position to several hundred, ends inside
    groups, blocks and chunks."""
    L = 5 * 128
    c = Cache(fmt, 7, n_kv, L, dim, block, seed=dim + rows)
    lens = [0, 1, 15, 16, 127, 300, L - rows]
    check_attention(c, rows, n_kv * group, lens, seed=rows, pad=8)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_masks(fmt):
    """Dropped oldest positions, up to rows that see nothing; padded rows; a
    sequence without real rows."""
    c = Cache(fmt, 8, 2, 512, 128, 32, seed=5)
    lens = [400, 400, 400, 100, 100, 30, 0, 0]
    first = [0, 17, 400, 103, 104, 500, 0, 2]
    n_new = [4, 4, 4, 4, 4, 4, 0, 3]
    _, got = check_attention(c, 4, 4, lens, first=first, n_new=n_new, seed=2)
    assert (got[3, :3] == 0).all() and (got[3, 3] != 0).any()  # row 3 alone sees position 103
    assert (got[4] == 0).all() and (got[5] == 0).all() and (got[6] == 0).all() and (got[7, :2] == 0).all() and (got[7, 3] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_never_reads_unwritten_positions(fmt):
    """Positions behind the last one hold bytes that are NaN in e4m3, and their
    blocks' magnitudes are NaN: nothing of them reaches the result."""
    c = Cache(fmt, 4, 2, 256, 128, 16, seed=9, fill=False)
    lens, rows = [0, 5, 16, 120], 3
    for y in "kv":
        c.t[y + "a"].fill_(float("nan"))
    total = [n + rows for n in lens]
    c.append(max(total), [0] * 4, total)
    ok()
    check_attention(c, rows, 2, lens)
    for y in "kv":  # and the magnitudes of untouched blocks are left as they were
        assert torch.isnan(c.t[y + "a"][0, :, 1:]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,group,never", [(128, 1, 0x7F), (128, 4, 0xFF), (64, 4, 0x7F), (64, 1, 0xFF)])
def test_attention_never_reads_positions_before_the_first(fmt, dim, group, never):
    """Sequences that start inside a group of 16 (padded on the left): the bytes
    before their first position were never written either, and are NaN in e4m3."""
    pos, rows, more = [0, 1, 3, 5, 15, 17, 30, 100, 131, 200], 3, 90
    c = Cache(fmt, len(pos), 2, 320, dim, 64, seed=23, fill=False, never=never)
    for y in "kv":  # magnitudes that the rows do not outgrow: earlier codes stay as they are
        c.amax[y][:] = 8.0
        c.t[y + "a"].fill_(8.0)
    n = [1 + rows if b % 2 else more + rows for b in range(len(pos))]
    c.append(more + rows, pos, n)
    ok()
    assert all((c.t[y].view(torch.uint8) == never).any() for y in "kv")
    check_attention(c, rows, 2 * group, [p + m - rows for p, m in zip(pos, n)], first=pos)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_extreme_scores(fmt):
    """Scores of several hundred (one position takes all), and queries and
    magnitudes near both ends of the bf16 range."""
    c = Cache(fmt, 2, 2, 256, 128, 64, seed=11)
    check_attention(c, 2, 2, [200, 77], q_size=30.0)
    check_attention(c, 2, 2, [200, 77], q_size=1e-36)
    # keys 2^-100 and values 2^100 times as large, with a scale that brings the scores back; then the reverse.
    # (Both in one call would need scores of 2^190 in one of the sequences, which fp32 does not hold.)
    for f, scale in ((2.0 ** 100, 2.0 ** 97), (2.0 ** -100, 2.0 ** -103)):
        d = Cache(fmt, 2, 2, 256, 128, 64, seed=11)
        for y in "kv":
            d.amax[y] *= f if y == "v" else 1 / f
            d.t[y + "a"] *= f if y == "v" else 1 / f
        check_attention(d, 2, 2, [200, 77], scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group", [1, 4])
def test_attention_nan_query(fmt, group):
    """A query row with a NaN gives NaN there, whether one CTA holds its unit or
    several, and changes no bit of the other rows; a row that sees nothing
    stays 0."""
    c = Cache(fmt, 3, 2, 2048, 128, 64, seed=17)
    rows, w = 4, 2 * group * 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(12, w, generator=g, device="cuda").bfloat16()
    bad = q.clone()
    bad[1, 130] = bad[6, 5] = bad[8, 7] = float("nan")  # the last of a row that sees nothing
    lens, first = i32([2000, 30, 9]), i32([0, 0, 10])
    ws = torch.zeros(vgv.vg_kv8_attn_workspace_bytes(c.h, rows, 2 * group), dtype=torch.uint8, device="cuda")
    o = [torch.zeros_like(q) for _ in "ab"]
    for x, y in zip((q, bad), o):
        vgv.vg_kv8_attn(c.h, rows, 2 * group, x, lens, 0.1, y, ws, first=first)
    ok()
    hit = torch.zeros(12, 2 * group, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[6, 0] = True
    nan = o[1].view(12, 2 * group, 128).isnan()
    assert torch.equal(nan, hit[:, :, None].expand_as(nan))
    assert torch.equal(o[0].view_as(nan)[~nan], o[1].view_as(nan)[~nan])
    assert not o[1][8].any()


def test_attention_value_scales_far_apart():
    """Neighbouring blocks whose value magnitudes differ by 2^40, rising and falling."""
    c = Cache("int8", 2, 1, 256, 128, 16, seed=12)
    f = 2.0 ** np.linspace(-20, 20, 16)
    c.amax["v"][0, 0] *= f
    c.amax["v"][1, 0] *= f[::-1]
    c.amax["v"][:] = oracle.widen(oracle.round_bf16_bits(c.amax["v"]))
    c.t["va"].copy_(torch.from_numpy(c.amax["v"].astype(np.float32)))
    check_attention(c, 3, 1, [250, 250])


def test_attention_bad_lengths_are_reported():
    c = Cache("int8", 5, 1, 64, 64, 16, seed=13)
    q = torch.ones(20, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, -3.0)
    ws = torch.zeros(max(16, vgv.vg_kv8_attn_workspace_bytes(c.h, 4, 1)), dtype=torch.uint8, device="cuda")
    vgv.vg_kv8_attn(c.h, 4, 1, q, i32([10, -1, 61, 10, 10]), 1.0, o, ws, first=i32([0, 0, 0, -1, 0]), n_new=i32([4, 4, 4, 4, 5]))
    torch.cuda.synchronize()
    assert vgv.vg_get_device_status() == (6, 343)
    assert (o[4:] == 0).all() and (o[:4] != 0).any()


def test_attention_many_sequences():
    """More sequences than one launch takes, short and empty ones."""
    g = np.random.default_rng(15)
    B = 1030
    c = Cache("int8", B, 1, 32, 64, 16, seed=15)
    lens = g.integers(0, 30, B)
    n_new = g.integers(0, 3, B)
    check_attention(c, 2, 1, lens.tolist(), n_new=n_new.tolist(), first=g.integers(0, 12, B).tolist())


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_longest_cache(fmt):
    """32,768 positions: a few heads, one sequence full, one nearly empty."""
    c = Cache(fmt, 2, 1, 32768, 128, 128, seed=14)
    check_attention(c, 8, 2, [32760, 3])


def test_a_single_row_of_an_odd_matrix():
    """One sequence, one row: columns of a matrix whose rows are no multiple of 8 apart."""
    c = Cache("int8", 1, 2, 64, 64, 16, seed=18)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(1, 4 * 128 + 3, generator=g, device="cuda").bfloat16()
    q, k, v, o = (x[:, i * 128:(i + 1) * 128] for i in range(4))
    plain = [t.contiguous() for t in (q, k, v)]
    d = Cache("int8", 1, 2, 64, 64, 16, seed=18)
    ws = torch.zeros(vgv.vg_kv8_attn_workspace_bytes(c.h, 1, 2), dtype=torch.uint8, device="cuda")
    vgv.vg_kv8_append(c.h, 1, k, v, i32([20]))
    vgv.vg_kv8_attn(c.h, 1, 2, q, i32([20]), 0.1, o, ws)
    vgv.vg_kv8_append(d.h, 1, plain[1], plain[2], i32([20]))
    want, back = torch.zeros_like(plain[0]), torch.zeros(2, 1, 132, device="cuda")
    vgv.vg_kv8_attn(d.h, 1, 2, plain[0], i32([20]), 0.1, want, ws)
    vgv.vg_kv8_read(d.h, 1, i32([20]), back[0][:, :128], None)
    vgv.vg_kv8_read(c.h, 1, i32([20]), back[1][:, :128], None)
    ok()
    assert all(torch.equal(c.t[y], d.t[y]) for y in c.t) and torch.equal(o, want) and bool(want.any())
    assert torch.equal(back[0], back[1]) and bool(back.any()) and not back[:, :, 128:].any()


def test_offsets_past_32_bits():
    """A cache of more than 2^31 codes: the last sequence is written, read and
    attended to."""
    B, n_kv, L, dim, block = 65, 8, 32768, 128, 128
    t = {y: torch.zeros(B, n_kv, L, dim, dtype=torch.int8, device="cuda") for y in "kv"}
    a = {y: torch.zeros(B, n_kv, L // block, device="cuda") for y in "kv"}
    h = vgv.make_kv8(t["k"], t["v"], a["k"], a["v"])
    g = torch.Generator(device="cuda").manual_seed(1)
    x = {y: torch.randn(B * 130, n_kv * dim, generator=g, device="cuda").bfloat16() for y in "kv"}
    p = L - 130
    vgv.vg_kv8_append(h, 130, x["k"], x["v"], i32([0] * (B - 1) + [p]), n_new=i32([1] * (B - 1) + [130]))
    out = torch.zeros(B * 130, n_kv * dim, device="cuda")
    vgv.vg_kv8_read(h, 130, i32([0] * (B - 1) + [p]), out, None, n_rows=i32([1] * (B - 1) + [130]))
    ok()
    last = x["k"][-130:].float()
    assert (out[-130:] - last).abs().max() <= last.abs().max() / 127 * 0.5 * 1.001
    assert int(t["k"][B - 2, :, 16:].count_nonzero()) == 0
    q = torch.randn(B, n_kv * dim, generator=g, device="cuda").bfloat16()
    o = torch.zeros_like(q)
    ws = torch.zeros(vgv.vg_kv8_attn_workspace_bytes(h, 1, n_kv), dtype=torch.uint8, device="cuda")
    vgv.vg_kv8_attn(h, 1, n_kv, q, i32([0] * (B - 1) + [L - 1]), 128 ** -0.5, o, ws, first=i32([0] * (B - 1) + [p]))
    ok()
    k, v = out[-130:].view(130, n_kv, dim).double(), torch.zeros(130, n_kv * dim, device="cuda")
    vv = torch.zeros(B * 130, n_kv * dim, device="cuda")
    vgv.vg_kv8_read(h, 130, i32([0] * (B - 1) + [p]), None, vv, n_rows=i32([1] * (B - 1) + [130]))
    v = vv[-130:].view(130, n_kv, dim).double()
    s = torch.einsum("hd,phd->hp", q[-1].view(n_kv, dim).double(), k) * 128 ** -0.5
    ref = torch.einsum("hp,phd->hd", torch.softmax(s, 1), v)
    assert (o[-1].view(n_kv, dim).double() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 2.0 ** -10 * v.abs().max()


# ------------------------------------------------------------------ the layer
@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_on_an_8_bit_cache(fmt):
    """vg_attn_verify_kv8 against the bf16 layer's oracle: the prompt quantised
    in one call, then steps whose rows overwrite rejected drafts."""
    H, B, K, L, block = DIMS.H, 3, 3, 384, 64
    g = np.random.default_rng(21)
    wqkv = oracle.round_bf16_bits(g.normal(0, 0.02, (3 * H, H)))
    wo = oracle.round_bf16_bits(g.normal(0, 0.05, (H, H)))
    c = Cache(fmt, B, 10, L, 128, block, fill=False)
    lens = np.array([0, 63, 300])
    c.append(300, [0] * B, lens.tolist())
    ok()
    ws = torch.zeros(vgv.vg_attn_verify_kv8_workspace_bytes(c.h, K), dtype=torch.uint8, device="cuda")
    wq_d, wo_d = dev(wqkv), dev(wo)
    for step in range(3):
        x = oracle.round_bf16_bits(g.normal(0, 1, (B * (K + 1), H)))
        # the bf16 oracle on the cache's values before the step
        cache = np.zeros((B, 2, L, H), np.uint16)
        for i, val in enumerate(c.values()):
            for b in range(B):
                cache[b, i, :lens[b]] = oracle.round_bf16_bits(val[b].transpose(1, 0, 2).reshape(L, H)[:lens[b]])
        out = torch.empty(B * (K + 1), H, dtype=torch.bfloat16, device="cuda")
        o = torch.empty_like(out)
        vgv.vg_attn_verify_kv8(c.h, K, dev(x), wq_d, wo_d, i32(lens.tolist()), out, ws, o_out=o)
        ok()
        ref_out, _, mid = oracle.attn_verify(x, wqkv, wo, cache, lens.tolist(), K)
        # the new rows pass one more rounding, to codes: half a step (int8 2^-8 of the block's magnitude, e4m3 2^-4
        # of the value), in keys and values of at most K + 1 of the positions a row sees; at L = 0 they are all of them
        quant = 0.02 if fmt == "int8" else 0.12
        for got, ref in ((o, mid["o"]), (out, ref_out)):
            assert row_rel_err(oracle.widen(si.torch_to_bits(got)), oracle.widen(ref)) <= ACT_TOL + quant
        # the cache after the step, as the library holds it
        for y in "kv":
            c.codes[y] = kv8.unpack(c.t[y].cpu().numpy(), fmt, y == "v")
            c.amax[y] = c.t[y + "a"].cpu().numpy().astype(np.float64)
        lens = lens + np.array([1, 2, 4])  # accepted 0, 1 and 3 drafts


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_against_the_codes_it_wrote(fmt):
    """vg_attn_verify_kv8 in its three parts: the codes and magnitudes of the new
    rows against the rotated rows of the bf16 layer's oracle, the heads' output
    against exact attention over those codes, the result against the projection of
    that output."""
    H, B, K, L, block = DIMS.H, 4, 3, 384, 64
    g = np.random.default_rng(22)
    wqkv = oracle.round_bf16_bits(g.normal(0, 0.02, (3 * H, H)))
    wo = oracle.round_bf16_bits(g.normal(0, 0.05, (H, H)))
    c = Cache(fmt, B, 10, L, 128, block, fill=False)
    lens = [0, 61, 64, 300]
    c.append(300, [0] * B, lens)
    ok()
    before = {y: c.amax[y].copy() for y in "kv"}
    x = oracle.round_bf16_bits(g.normal(0, 1, (B * (K + 1), H)))
    ws = torch.zeros(vgv.vg_attn_verify_kv8_workspace_bytes(c.h, K), dtype=torch.uint8, device="cuda")
    out = torch.empty(B * (K + 1), H, dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(out)
    vgv.vg_attn_verify_kv8(c.h, K, dev(x), dev(wqkv), dev(wo), i32(lens), out, ws, o_out=o)
    ok()
    c.gd.check()
    _, rows, mid = oracle.attn_verify(x, wqkv, wo, np.zeros((B, 2, L, H), np.uint16), lens, K)
    ez = 6 * np.sqrt(H) * 2.0 ** -23 * (np.abs(oracle.widen(x)) @ np.abs(oracle.widen(wqkv)).T).max()
    rows = oracle.widen(rows).reshape(B, 2, L, 10, 128).transpose(1, 0, 3, 2, 4)  # [k, v][B, head, position, dim]
    for y, ref in zip("kv", rows):
        c.codes[y] = kv8.unpack(c.t[y].cpu().numpy(), fmt, y == "v")
        c.amax[y] = c.t[y + "a"].cpu().numpy().astype(np.float64)
        val = kv8.values(np.nan_to_num(c.codes[y]), c.amax[y], block, fmt)
        for b, n in enumerate(lens):
            new, a = ref[b, :, n:n + K + 1], np.repeat(c.amax[y][b], block, 1)[:, n:n + K + 1, None]
            # rows: the projection is an fp32 sum (off by ez at most) rounded to bf16, so both may be a step apart
            # (2^-7 of the element); rotated, that is up to sqrt(2) steps of the larger element of a pair, and the
            # second rounding adds one more
            pair = np.abs(new).reshape(10, K + 1, 64, 2).max(3).repeat(2, 2)
            off = 2.5 * 2.0 ** -7 * pair + 1.5 * ez
            # codes: half a step
            half = a / 254 if fmt == "int8" else np.maximum((np.abs(new) + off) * 2.0 ** -4, a / 448 * 2.0 ** -10)
            assert (np.abs(val[b, :, n:n + K + 1] - new) <= half * 1.001 + off).all(), (y, b)
            # magnitudes: the larger one of the block's and the new rows'
            for k in range(n // block, (n + K) // block + 1):
                lo, hi = max(n, k * block) - n, min(n + K + 1, (k + 1) * block) - n
                top = np.abs(new[:, lo:hi]).max((1, 2))
                top = np.maximum(top, before[y][b, :, k]) if n > k * block else top
                assert (np.abs(c.amax[y][b, :, k] - top) <= 2.5 * 2.0 ** -7 * top + 1.5 * ez).all(), (y, b, k)
    k, v = c.values()
    ref, _, _ = kv8.attention(oracle.widen(mid["q"]).reshape(B, K + 1, 10, 128), k, v, lens, 128 ** -0.5)
    got = oracle.widen(si.torch_to_bits(o))
    assert row_rel_err(got, ref.reshape(-1, H)) <= ACT_TOL
    proj = oracle.round_bf16_bits(got @ oracle.widen(wo).T)
    assert row_rel_err(oracle.widen(si.torch_to_bits(out)), oracle.widen(x) + oracle.widen(proj)) <= ACT_TOL


def test_layer_overflow_leaves_x():
    H, B, K = DIMS.H, 2, 3
    c = Cache("int8", B, 10, 16, 128, 16, seed=22)
    before = {y: c.codes[y][1].copy() for y in "kv"}
    x = torch.randn(B * (K + 1), H, device="cuda").bfloat16()
    w = torch.randn(3 * H, H, device="cuda").bfloat16() * 0.02
    out = torch.empty_like(x)
    ws = torch.zeros(vgv.vg_attn_verify_kv8_workspace_bytes(c.h, K), dtype=torch.uint8, device="cuda")
    vgv.vg_attn_verify_kv8(c.h, K, x, w, w[:H].contiguous(), i32([3, 13]), out, ws)
    torch.cuda.synchronize()
    assert vgv.vg_get_device_status()[0] == 6
    assert torch.equal(out[4:], x[4:])
    for y in "kv":
        assert np.array_equal(kv8.unpack(c.t[y].cpu().numpy(), "int8", y == "v")[1], before[y])


# ------------------------------------------------------------------ as a program runs them
def test_captured_steps_equal_eager_ones():
    """A step (append, read back, attention) captured into a graph and replayed
    with other inputs in the same buffers gives what eager calls give, on a
    stream of its own while another graph works on its own cache."""
    B, n_kv, dim, rows = 4, 2, 128, 4

    def program(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = [torch.zeros(B, n_kv, 256, dim, dtype=torch.int8, device="cuda") for _ in "kv"]
        a = [torch.zeros(B, n_kv, 4, device="cuda") for _ in "kv"]
        h = vgv.make_kv8(*t, *a)
        s = {"x": torch.randn(B * rows, 3 * n_kv * dim, generator=g, device="cuda").bfloat16(), "pos": i32([0, 3, 60, 200]),
             "out": torch.zeros(B * rows, n_kv * dim, device="cuda"), "t": t, "a": a, "h": h,
             "o": torch.zeros(B * rows, n_kv * dim, dtype=torch.bfloat16, device="cuda"),
             "ws": torch.zeros(vgv.vg_kv8_attn_workspace_bytes(h, rows, n_kv), dtype=torch.uint8, device="cuda"), "g": g}
        return s

    def step(s):
        w = n_kv * dim
        vgv.vg_kv8_append(s["h"], rows, s["x"][:, w:2 * w], s["x"][:, 2 * w:], s["pos"])
        vgv.vg_kv8_read(s["h"], rows, s["pos"], s["out"], None)
        vgv.vg_kv8_attn(s["h"], rows, n_kv, s["x"][:, :w], s["pos"], dim ** -0.5, s["o"], s["ws"])

    eager, graphed, other = program(1), program(1), program(2)
    graphs = []
    for s in (graphed, other):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            step(s)
        torch.cuda.synchronize()
        for y in s["t"] + s["a"]:
            y.zero_()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=stream):
            step(s)
        graphs.append((gr, stream))
    for i in range(4):
        for s in (eager, graphed, other):
            s["x"].copy_(torch.randn(s["x"].shape, generator=s["g"], device="cuda").bfloat16() * (i + 1))
            s["pos"].copy_(i32([4 * i, 3 + i, 60 + 2 * i, 200 + i]))
        step(eager)
        torch.cuda.synchronize()
        for gr, stream in graphs:
            with torch.cuda.stream(stream):
                gr.replay()
        torch.cuda.synchronize()
        ok()
        for y in ("out", "o"):
            assert torch.equal(eager[y], graphed[y]), (i, y)
        for y in ("t", "a"):
            assert all(torch.equal(p, q) for p, q in zip(eager[y], graphed[y])), (i, y)
        assert not torch.equal(eager["o"], other["o"])
