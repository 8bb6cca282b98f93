"""Log probabilities from the LM head on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

import greedy_speculative_verify_b200 as vgv
import oracle
import synth_inputs as si
from oracle import kv8

from gpu_common import D as DIMS, Guarded, dev, ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()
    vgv.vg_get_device_status()


def call(h, lm, tokens, n_top, status=0):
    R, H = h.shape
    V = lm.shape[0]
    gd = Guarded()
    lp, en = gd.empty((R,), torch.float32, fill=7.0), gd.empty((R,), torch.float32, fill=7.0)
    ids = gd.empty((R, n_top), torch.int32, fill=-9) if n_top else None
    tl = gd.empty((R, n_top), torch.float32, fill=7.0) if n_top else None
    ws = gd.empty((vgv.vg_token_logprobs_workspace_bytes(R, H, V, n_top),), torch.uint8, fill=0)
    vgv.vg_token_logprobs(h, lm, tokens, lp if tokens is not None else None, en, ids, tl, ws)
    torch.cuda.synchronize()
    assert vgv.vg_get_device_status()[0] == status
    gd.check()
    assert int(ws[:24 * 768 * 4].count_nonzero()) == 0  # what a later call relies on
    n = lambda t: None if t is None else t.cpu().numpy()
    return n(lp), n(en), n(ids), n(tl)


def tolerances(lp, mag, H):
    """What lse and the entropy may be off by: a logit is an fp32 sum of H exact
    products, off by up to 6 sqrt(H) 2^-23 of the sum of their magnitudes (sums
    whose roundings do not conspire stay within 6 standard deviations); lse moves
    by at most the largest error, p-weighted; its sums of exponentials carry
    fewer than 128 roundings in a row and 2^-21 each for the exponential. The
    entropy is a p-weighted mean of log p, whose terms shift with p too."""
    ez = 6 * np.sqrt(H) * 2.0 ** -23 * mag.max(axis=1)
    p = np.exp(lp)
    spread = (p * np.abs(lp)).sum(axis=1)
    rel = 128 * 2.0 ** -24 + 2.0 ** -21
    return ez + rel + 2.0 ** -23 * np.abs(lp).max(axis=1), (2 * ez + 2 * rel) * (1 + spread) + 2.0 ** -22 * spread


def check(h, lm, tokens, n_top):
    """h, lm: bf16 bits."""
    R, H = h.shape
    lp, ent, mag = kv8.logprobs(h, lm)
    t_lse, t_ent = tolerances(lp, mag, H)
    got_lp, got_en, ids, tl = call(dev(h), dev(lm), torch.from_numpy(tokens).cuda(), n_top)
    want = np.where(tokens >= 0, lp[np.arange(R), np.maximum(tokens, 0)], -np.inf)
    real = tokens >= 0
    assert (np.abs(got_lp[real] - want[real]) <= t_lse[real] + 2.0 ** -24 * np.abs(want[real])).all()
    assert (got_lp[~real] == -np.inf).all()
    assert (np.abs(got_en - ent) <= t_ent).all(), float((np.abs(got_en - ent) / t_ent).max())
    if n_top:
        order = np.lexsort((np.broadcast_to(np.arange(lm.shape[0]), lp.shape), -lp), axis=1)[:, :n_top]
        # logits of equal rows are equal, and fp64 sums in another order may differ in the last place
        z = np.take_along_axis(lp, order, 1)
        same = np.take_along_axis(lp, ids.astype(np.int64), 1)
        assert (np.abs(same - z) <= 1e-12 * np.abs(mag).max()).all()
        gap = np.diff(lp[np.arange(R)[:, None], order], axis=1)
        clear = np.ones_like(order, bool)
        clear[:, 1:] &= np.abs(gap) > 1e-11
        clear[:, :-1] &= np.abs(gap) > 1e-11
        clear[:, -1] = False  # its follower is not in the list
        assert np.array_equal(ids[clear], order[clear])
        assert (np.abs(tl - z) <= t_lse[:, None] + 2.0 ** -24 * np.abs(z)).all()


def inputs(R, H, V, seed, sure=0.0):
    g = np.random.default_rng(seed)
    lm = oracle.round_bf16_bits(g.normal(0, 1.2 / np.sqrt(H), (V, H)))
    tok = g.integers(0, V, R).astype(np.int32)
    x = g.normal(0, 1, (R, H)) + sure * g.uniform(0, 1, (R, 1)) * oracle.widen(lm[tok])
    return oracle.round_bf16_bits(x), lm, tok


@pytest.mark.parametrize("R,H,V,n_top", [
    (1, 64, 1, 1), (1, 64, 20, 20), (3, 128, 7, 0), (5, 256, 175, 5), (127, 64, 177, 3), (128, 128, 1000, 20),
    (129, 320, 881, 7), (300, 64, 1761, 1), (257, 1280, 4099, 20), (4, 2048, 999, 12), (2, 8192, 333, 2)])
def test_logprobs(R, H, V, n_top):
    h, lm, tok = inputs(R, H, V, seed=R + V, sure=8.0)
    tok[::4] = -1
    check(h, lm, tok, n_top)


@pytest.mark.parametrize("R,V,n_top", [(300, 20, 20), (129, 1, 1), (512, 130, 4), (257, 256, 8)])
def test_many_rows_few_tokens(R, V, n_top):
    """Vocabularies of one tile, down to one that leaves a pair's second half empty."""
    h, lm, tok = inputs(R, 64, V, seed=R + V, sure=4.0)
    check(h, lm, tok, n_top)


@pytest.mark.parametrize("R,V", [(3, 9000), (260, 9000)])
def test_tokens_with_nearly_all_the_mass(R, V):
    """Their log probability is what the others add to a sum of 1. The 1 is rounded
    with at most four times inside a chunk of 16 logits and once more into the sum,
    which keeps that rounding, and once where S is rescaled: 6 times 2^-24. What the
    others add is off as in tolerances(), in proportion to their mass."""
    H = 64
    g = np.random.default_rng(31)
    lm = g.normal(0, 1.2 / np.sqrt(H), (V, H))
    tok = g.choice(V, R, replace=False).astype(np.int32)
    lm[tok] *= 2.5
    lm = oracle.round_bf16_bits(lm)
    w = oracle.widen(lm)[tok]
    h = oracle.round_bf16_bits(g.uniform(14, 19, (R, 1)) * w / (w * w).sum(1, keepdims=True))
    lp, ent, mag = kv8.logprobs(h, lm)
    want = lp[np.arange(R), tok]
    assert (want > -0.2).mean() > 0.9  # the test's point: rows of the kind it is about
    got, _, _, _ = call(dev(h), dev(lm), torch.from_numpy(tok).cuda(), 5)
    ez = 6 * np.sqrt(H) * 2.0 ** -23 * mag.max(axis=1)
    tol = 6 * 2.0 ** -24 + (ez + 128 * 2.0 ** -24 + 2.0 ** -21) * (1 - np.exp(want)) + 2.0 ** -24 * np.abs(want)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


def test_full_vocabulary():
    h, lm, tok = inputs(8, DIMS.H, DIMS.V, seed=5, sure=14.0)
    check(h, lm, tok, 20)


def test_one_workspace_for_calls_of_several_shapes():
    """The words that have to be zero lie at one place in every cut, whatever ran
    before: full rows, one token, several row blocks, a vocabulary of few tiles."""
    shapes = [(128, 64, 9001, 20), (1, 64, 9001, 3), (300, 64, 2000, 8), (77, 64, 40, 20), (128, 64, 20000, 12), (700, 64, 20000, 12), (1500, 64, 9001, 3), (128, 64, 9001, 20)]
    ws = torch.zeros(max(vgv.vg_token_logprobs_workspace_bytes(*s) for s in shapes), dtype=torch.uint8, device="cuda")
    for R, H, V, n_top in shapes:
        h, lm, tok = inputs(R, H, V, seed=V, sure=6.0)
        out = []
        for w in (ws, torch.zeros_like(ws)):
            t = [torch.zeros(R, device="cuda") for _ in "ab"] + [torch.zeros(R, n_top, dtype=d, device="cuda") for d in (torch.int32, torch.float32)]
            vgv.vg_token_logprobs(dev(h), dev(lm), torch.from_numpy(tok).cuda(), *t, w)
            out.append(t)
        torch.cuda.synchronize()
        assert vgv.vg_get_device_status()[0] == 0
        assert all(torch.equal(x, y) for x, y in zip(*out)), (R, V)


@pytest.mark.parametrize("R", [128, 300])
def test_alternatives_in_one_part_of_the_vocabulary(R):
    """The best tokens all in one tile, and none elsewhere near them: the bound
    from the other parts lets them all in."""
    g = np.random.default_rng(21)
    h, lm, tok = inputs(R, 64, 30000, seed=21)
    big = oracle.widen(h).sum(0)
    for at in (0, 17000, 29970):
        l2 = lm.copy()
        l2[at:at + 30] = oracle.round_bf16_bits(g.normal(0, 1, (30, 64)) + 3 * big / np.abs(big).max())
        check(h, l2, tok, 20)


def test_many_row_blocks():
    """4,096 rows in 32 row blocks over a vocabulary of many groups: the rows
    repeat eight, so every block has to give the same answers."""
    h, lm, tok = inputs(8, 256, 20011, seed=6, sure=10.0)
    rep = lambda a: np.tile(a, (512,) + (1,) * (a.ndim - 1))
    few = call(dev(h), dev(lm), torch.from_numpy(tok).cuda(), 5)
    many = call(dev(rep(h)), dev(lm), torch.from_numpy(rep(tok)).cuda(), 5)
    check(h, lm, tok, 5)
    for a, b in zip(few[2:3], many[2:3]):
        assert np.array_equal(rep(a), b)
    for a, b in zip((few[0], few[1], few[3]), (many[0], many[1], many[3])):
        # only the grouping of the sums differs with the number of rows
        assert np.allclose(rep(a), b, rtol=1e-5, atol=1e-5)
        assert np.array_equal(np.tile(b[:8], (512,) + (1,) * (b.ndim - 1)), b)


def test_ties_over_many_row_blocks():
    """Rows whose logits are all equal (zero, positive, negative, and a mix of
    zeros and others), in several row blocks and vocabulary groups: the lowest
    indices, whatever order the groups finish in."""
    V, H, R = 9001, 64, 520
    lm = np.zeros((V, H))
    lm[:, 0] = 1.0
    lm[:, 1] = np.where(np.arange(V) % 100 == 50, 1.0, 0.0)
    lm[:, 2] = -(np.arange(V) % 2).astype(float)
    h = np.zeros((R, H))
    h[1::5, 0], h[2::5, 0], h[3::5, 1], h[4::5, 2] = 1.5, -1.5, 2.0, 3.0
    ids = call(dev(oracle.round_bf16_bits(h)), dev(oracle.round_bf16_bits(lm)), None, 20)[2]
    low = np.arange(20)
    for k, want in enumerate((low, low, low, low * 100 + 50, low * 2)):
        assert (ids[k::5] == want).all(), k


def test_rising_logits():
    """Logits that rise with the vocabulary index: every column enters the list
    of alternatives, the worst order for it; and falling, and all equal."""
    V, H = 3001, 64
    base = np.zeros((V, H))
    base[:, 0] = np.arange(V) // 8 * 8.0  # exact in bf16 up to 2^11 in steps of 8
    lm = oracle.round_bf16_bits(base)
    h = np.zeros((3, H))
    h[:, 0] = [2.0 ** -7, -(2.0 ** -7), 0.0]
    tok = np.array([3000, 0, 17], np.int32)
    lp, _, _ = kv8.logprobs(oracle.round_bf16_bits(h), lm)
    _, _, ids, _ = call(dev(oracle.round_bf16_bits(h)), dev(lm), torch.from_numpy(tok).cuda(), 20)
    order = np.lexsort((np.broadcast_to(np.arange(V), lp.shape), -lp), axis=1)[:, :20]
    assert np.array_equal(ids, order)  # ties to the lower index


@pytest.mark.parametrize("n_top", [8, 20])
def test_alternatives_beside_each_other(n_top):
    """All the largest logits in neighbouring columns (one group of a bound), at
    the start of a vocabulary, over a tile's end and at its end; with ties."""
    V, H, R = 2100, 64, 9
    at = [0, 1, 170, 250, 255, 700, 1750, V - n_top, V - n_top - 3]
    h, lm = np.zeros((R, H)), np.full((V, H), -1.0)
    for r in range(R):
        h[r, r] = 1.0
        lm[at[r]:at[r] + n_top, r] = 8.0 + np.arange(n_top) // 2  # pairs of equal logits
    lm[:, 10:] = 0
    hb, lb = oracle.round_bf16_bits(h), oracle.round_bf16_bits(lm)
    lp, _, _ = kv8.logprobs(hb, lb)
    ids = call(dev(hb), dev(lb), None, n_top)[2]
    order = np.lexsort((np.broadcast_to(np.arange(V), lp.shape), -np.round(lp, 9)), axis=1)[:, :n_top]
    assert np.array_equal(ids, order)


def test_order_of_alternatives_closer_than_fp32():
    """Two tokens whose logits differ by less than an fp32 sum resolves, in both
    index orders: the larger exact logit comes first."""
    H, V = 64, 400
    lm = np.zeros((V, H))
    lm[:, 0] = -1.0
    lm[[50, 300], 0] = 256.0
    lm[300, 1] = 2.0 ** -12
    lm[[120, 121], 0] = 128.0
    lm[120, 1] = 2.0 ** -12
    h = np.zeros((1, H))
    h[0, :2] = [256.0, 2.0 ** -4]  # 65,536 against 65,536 + 2^-16, below half an ulp
    _, _, ids, _ = call(dev(oracle.round_bf16_bits(h)), dev(oracle.round_bf16_bits(lm)), torch.tensor([5], dtype=torch.int32).cuda(), 4)
    assert ids[0].tolist() == [300, 50, 120, 121]


def test_nan_and_infinite_logits_and_bad_tokens():
    g = np.random.default_rng(8)
    h, lm, tok = inputs(6, 128, 500, seed=8)
    hb, lb = h.copy(), lm.copy()
    hb[1, 3] = 0x7FC0  # a NaN row
    hb[2, 0] = 0x7F7F  # with 3e38: overflows against the row below
    lb[40, :] = 0
    lb[40, 0] = 0xFF7F  # -3.4e38: logit -inf in row 2, hugely negative elsewhere
    tok[3], tok[4], tok[5] = 500, -1, 499
    lp, en, ids, tl = call(dev(hb), dev(lb), torch.from_numpy(tok).cuda(), 3, status=6)
    assert np.isnan(lp[1]) and np.isnan(en[1]) and (ids[1] == -1).all()
    assert lp[3] == -np.inf and lp[4] == -np.inf and np.isfinite(lp[5])
    ref, ent, _ = kv8.logprobs(hb[[0, 5]], lb)
    assert np.allclose(lp[[0, 5]], ref[[0, 1], tok[[0, 5]]], atol=1e-3) and np.allclose(en[[0, 5]], ent, atol=1e-3)


def test_only_what_is_asked_for():
    h, lm, tok = inputs(9, 128, 640, seed=10)
    hd, ld, td = dev(h), dev(lm), torch.from_numpy(tok).cuda()
    full = call(hd, ld, td, 4)
    ws = torch.zeros(vgv.vg_token_logprobs_workspace_bytes(9, 128, 640, 4), dtype=torch.uint8, device="cuda")
    en = torch.zeros(9, device="cuda")
    vgv.vg_token_logprobs(hd, ld, None, None, en, None, None, ws)
    lp = torch.zeros(9, device="cuda")
    vgv.vg_token_logprobs(hd, ld, td, lp, None, None, None, ws)
    torch.cuda.synchronize()
    assert np.array_equal(en.cpu().numpy(), full[1]) and np.array_equal(lp.cpu().numpy(), full[0])
    assert vgv.vg_get_device_status()[0] == 0


def test_verify_step_with_logprobs():
    """A run as a server makes it: attention on the 8-bit cache, the LM head's
    verification, the log probabilities of what was committed; the committed
    tokens are the first alternatives of their rows."""
    H, V, B, K, L = DIMS.H, 8191, 4, 3, 256
    g = np.random.default_rng(12)
    wqkv, wo = (dev(oracle.round_bf16_bits(g.normal(0, s, (n, H)))) for s, n in ((0.02, 3 * H), (0.05, H)))
    lm = dev(oracle.round_bf16_bits(g.normal(0, 1.2 / np.sqrt(H), (V, H))))
    t = [torch.zeros(B, 10, L, 128, dtype=torch.int8, device="cuda") for _ in "kv"]
    a = [torch.zeros(B, 10, L // 64, device="cuda") for _ in "kv"]
    cache = vgv.make_kv8(*t, *a)
    lens = torch.tensor([0, 5, 63, 200], dtype=torch.int32, device="cuda")
    prompt = dev(oracle.round_bf16_bits(g.normal(0, 1, (B * 200, 2 * H))))
    vgv.vg_kv8_append(cache, 200, prompt[:, :H], prompt[:, H:], torch.zeros_like(lens), n_new=lens)
    z8 = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
    ws_a = z8(vgv.vg_attn_verify_kv8_workspace_bytes(cache, K))
    ws_v = z8(vgv.vg_verify_workspace_bytes(B, K, H, V))
    R = B * (K + 1)
    ws_l = z8(vgv.vg_token_logprobs_workspace_bytes(R, H, V, 2))
    out = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
    am, acc = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    tok = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
    lp, en = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    ids, tl = torch.empty(R, 2, dtype=torch.int32, device="cuda"), torch.empty(R, 2, device="cuda")
    for step in range(3):
        x = dev(oracle.round_bf16_bits(g.normal(0, 1, (R, H))))
        drafts = torch.from_numpy(g.integers(0, V, (B, K)).astype(np.int32)).cuda()
        if step:
            drafts[:, 0] = am.view(B, K + 1)[:, 0]
        vgv.vg_attn_verify_kv8(cache, K, x, wqkv, wo, lens, out, ws_a)
        vgv.vg_verify_greedy(B, K, H, V, out, lm, drafts, am, acc, tok, ws_v)
        vgv.vg_token_logprobs(out, lm, tok.view(-1), lp, en, ids, tl, ws_l)
        lens += acc + 1
        torch.cuda.synchronize()
        assert vgv.vg_get_device_status()[0] == 0
        committed = tok.view(-1) >= 0
        assert torch.equal(ids[committed, 0], tok.view(-1)[committed])
        assert torch.equal(lp[committed], tl[committed, 0])
        assert bool((lp[~committed] == -torch.inf).all()) and bool((tl[:, 0] >= tl[:, 1]).all()) and bool((en > 0).all())


def test_pairs_of_ctas_call_after_call():
    """Several row blocks over vocabularies of one to a few tiles, one call right
    behind the other: pairs whose even CTA has work left to signal when the odd
    one has stored its rows. Every call gives the first one's bits."""
    runs = []
    for R, V, n_top in ((129, 40, 3), (300, 256, 20), (257, 700, 8)):
        h, lm, tok = inputs(R, 64, V, seed=R, sure=4.0)
        t = [torch.zeros(R, device="cuda") for _ in "ab"] + [torch.zeros(R, n_top, dtype=d, device="cuda") for d in (torch.int32, torch.float32)]
        ws = torch.zeros(vgv.vg_token_logprobs_workspace_bytes(R, 64, V, n_top), dtype=torch.uint8, device="cuda")
        runs.append((dev(h), dev(lm), torch.from_numpy(tok).cuda(), t, ws))
    first = None
    for _ in range(50):
        for h, lm, tok, t, ws in runs:
            vgv.vg_token_logprobs(h, lm, tok, *t, ws)
        torch.cuda.synchronize()
        assert vgv.vg_get_device_status()[0] == 0
        got = [x.clone() for r in runs for x in r[3]]
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))


def test_two_tokens_with_all_the_mass():
    """Nothing is left of the sums beside the candidates, down to one unit in the
    last place of fp64, and no quotient of such rest enters the entropy. Rows along
    one direction, tokens at multiples of it: two near the top, 16 a factor of 1e-15
    below, the others far off, at H = 8192, where the tensor cores fall short most.
    The candidates' logits are exact, so what is off is the exponential's argument
    d log2(e) (two roundings: |d| 2^-23), the exponential (2^-22), and in S and T at
    most three roundings of 2^-24 each for the two tokens that count, weighted with
    p (1 + |d|); the result's rounding comes on top."""
    H, V, R = 8192, 32, 128
    for seed, tail in ((1, -15.5), (2, -16.5), (3, -17.5)):
        g = np.random.default_rng(seed)
        a = np.full(V, -80.0)
        a[:2], a[16:] = (20.0, 19.0), tail + g.uniform(-0.3, 0.3, 16)
        u = g.normal(0, 1, H)
        lm = oracle.round_bf16_bits(a[:, None] * u / np.sqrt(H))
        h = oracle.round_bf16_bits(g.uniform(0.9, 1.1, (R, 1)) * u / np.sqrt((u * u).mean()) / np.sqrt(H))
        lp, ent, _ = kv8.logprobs(h, lm)
        assert (np.sort(lp, 1)[:, -3] < -30).all() and (ent > 0.4).all()
        lpt, en, _, _ = call(dev(h), dev(lm), torch.zeros(R, dtype=torch.int32).cuda(), 5)
        p, d = np.exp(lp), np.abs(lp - lp.max(1, keepdims=True))
        tol = (p * (1 + d) * (2.0 ** -22 + d * 2.0 ** -23 + 3 * 2.0 ** -24)).sum(1)
        assert (np.abs(en - ent) <= tol + 2.0 ** -24 * ent).all(), float((np.abs(en - ent) / tol).max())
        assert (np.abs(lpt - lp[:, 0]) <= tol + 2.0 ** -24 * np.abs(lp[:, 0])).all()


@pytest.mark.parametrize("V,H", [(2, 8192), (3, 1280), (7, 8192), (12, 1280), (12, 8192), (13, 8192)])
def test_hardly_more_tokens_than_candidates(V, H):
    """All tokens, or all but one, are among the candidates with exact logits: what
    is off is as in the test above, with the roundings of V terms (a chain of them in
    T, of 16 at most; log2 of 16 and one more in S)."""
    h, lm, tok = inputs(64, H, V, seed=V + H, sure=4.0)
    lp, ent, mag = kv8.logprobs(h, lm)
    got, en, _, _ = call(dev(h), dev(lm), torch.from_numpy(tok).cuda(), 2 if V < 5 else 5)
    p, d = np.exp(lp), np.abs(lp - lp.max(1, keepdims=True))
    tol = (p * (1 + d) * (2.0 ** -22 + d * 2.0 ** -23 + min(V, 16) * 2.0 ** -24)).sum(1)
    if V > 12:  # the last token's logit stays the tensor cores'
        tol = tol + (np.sort(p, 1)[:, 0] * (1 + d.max(1)) * 2) * 6 * np.sqrt(H) * 2.0 ** -23 * mag.max(1)
    want = lp[np.arange(64), tok]
    assert (np.abs(en - ent) <= tol + 2.0 ** -24 * ent).all(), float((np.abs(en - ent) / tol).max())
    assert (np.abs(got - want) <= tol + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("H,V,R", [(1280, 5000, 130), (8192, 3000, 64), (64, 1, 5), (1280, 40, 64)])
def test_no_probability_above_1(H, V, R):
    """Rows whose token has all the mass but for 1e-10 and less: no log probability
    above 0, no entropy below it, and none of them negative zero or NaN."""
    g = np.random.default_rng(H + V)
    lm = oracle.round_bf16_bits(g.normal(0, 1.2 / np.sqrt(H), (V, H)))
    tok = g.integers(0, V, R).astype(np.int32)
    w = oracle.widen(lm)[tok]
    h = oracle.round_bf16_bits(g.uniform(20, 60, (R, 1)) * w / (w * w).sum(1, keepdims=True))
    lp, en, _, tl = call(dev(h), dev(lm), torch.from_numpy(tok).cuda(), min(V, 5))
    assert (lp <= 0).all() and (tl <= 0).all() and (en >= 0).all() and not np.signbit(en).any()
    assert (lp > -1e-3).mean() > 0.9  # the test's point
    assert np.array_equal(lp, tl[:, 0])


@pytest.mark.parametrize("R,V,n_top", [(4, 30000, 5), (128, 30000, 20), (300, 9001, 8)])
def test_captured_calls_equal_eager_ones(R, V, n_top):
    """Two graphs with workspaces of their own, replayed side by side on two
    streams with new inputs in the same buffers: the bits of eager calls, one CTA
    and pairs of CTAs a row block."""
    H = 128
    def program():
        h, lm = (torch.zeros(n, H, dtype=torch.bfloat16, device="cuda") for n in (R, V))
        t = [torch.zeros(R, device="cuda") for _ in "ab"] + [torch.zeros(R, n_top, dtype=d, device="cuda") for d in (torch.int32, torch.float32)]
        ws = torch.zeros(vgv.vg_token_logprobs_workspace_bytes(R, H, V, n_top), dtype=torch.uint8, device="cuda")
        return h, lm, torch.zeros(R, dtype=torch.int32, device="cuda"), t, ws

    def step(p):
        vgv.vg_token_logprobs(p[0], p[1], p[2], *p[3], p[4])

    eager, graphs = program(), []
    for _ in range(2):
        p, stream, gr = program(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            step(p)
        torch.cuda.synchronize()
        with torch.cuda.graph(gr, stream=stream):
            step(p)
            step(p)  # one call behind the other in the graph, in one workspace
        graphs.append((p, stream, gr))
    for seed in range(3):
        want = []
        for i, (p, _, _) in enumerate(graphs):
            h, lm, tok = inputs(R, H, V, seed=10 * seed + i, sure=6.0)
            for q in (p, eager):
                q[0].copy_(dev(h)), q[1].copy_(dev(lm)), q[2].copy_(torch.from_numpy(tok))
            step(eager)
            want.append([x.clone() for x in eager[3]])
        torch.cuda.synchronize()
        for _, stream, gr in graphs:
            with torch.cuda.stream(stream):
                gr.replay()
        torch.cuda.synchronize()
        assert vgv.vg_get_device_status()[0] == 0
        for (p, _, _), w in zip(graphs, want):
            assert all(torch.equal(x, y) for x, y in zip(p[3], w)), seed
    assert not torch.equal(want[0][0], want[1][0])


def test_logits_that_the_tensor_cores_sum_exactly():
    """Products and partial sums are whole numbers below 2^24 (times a power of
    two): no logit falls short, nothing is put back, and the sums' own roundings
    are all that is off. A unit has at most 256 columns here, 16 chunks of 16: chains
    of 16 terms in a chunk and of 16 chunks, and a new maximum in each of them at
    worst, which multiplies by an exponential (2^-22) and rounds three times, as the
    units' joining does once."""
    H, V, R = 8192, 3000, 130
    g = np.random.default_rng(41)
    lm = g.integers(-3, 4, (V, H)).astype(np.float64)
    h = g.integers(-3, 4, (R, H)) * 2.0 ** -6
    h[::2, :] = np.abs(h[::2, :])  # rows that lean to one side
    lm[:, :600] += g.integers(-1, 3, (V, 1))
    tok = g.integers(0, V, R).astype(np.int32)
    hb, lb = oracle.round_bf16_bits(h), oracle.round_bf16_bits(lm)
    lp, ent, mag = kv8.logprobs(hb, lb)
    assert mag.max() * 2 ** 6 < 2 ** 24
    for rows in (slice(0, 100), slice(0, R)):  # one row block, and two
        got, en, _, _ = call(dev(hb[rows]), dev(lb), torch.from_numpy(tok[rows]).cuda(), 5)
        l, e = lp[rows], ent[rows]
        p, d = np.exp(l), np.abs(l - l.max(1, keepdims=True))
        tol = (p * (1 + d) * (18 * 2.0 ** -22 + d * 2.0 ** -23 + 83 * 2.0 ** -24)).sum(1)
        want = l[np.arange(len(l)), tok[rows]]
        assert (np.abs(en - e) <= tol + 2.0 ** -24 * e).all(), float((np.abs(en - e) / tol).max())
        assert (np.abs(got - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
