"""Pins of the 8-bit cache oracle (oracle/kv8.py): code grids, byte order,
magnitudes over several writes, attention against the bf16 layer's oracle."""
import numpy as np
import pytest

import oracle
from oracle import kv8


def test_grids():
    import torch

    x = np.concatenate([np.linspace(-127, 127, 4001), np.arange(-127, 127) + 0.5])
    assert np.array_equal(kv8.to_grid(x, "int8"), torch.round(torch.from_numpy(x)).numpy())
    x = np.concatenate([np.linspace(-448, 448, 4001), np.linspace(-0.1, 0.1, 999)]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv8.to_grid(x, "e4m3"), want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("is_v", [False, True])
def test_byte_order(fmt, is_v):
    rng = np.random.default_rng(1)
    c = kv8.to_grid(rng.uniform(-127, 127, (2, 3, 32, 128)), fmt)
    raw = kv8.pack(c, fmt, is_v)
    assert np.array_equal(kv8.unpack(raw, fmt, is_v), c)
    one = kv8.pack(np.full_like(c, 1.0), fmt, is_v).reshape(-1)[0]
    flat = np.zeros_like(c)
    flat[0, 0, 21, 70] = 1.0  # position 21 = group 1, 5th; dimension 70
    at = np.flatnonzero(kv8.pack(flat, fmt, is_v).reshape(-1) == one)
    assert at.tolist() == [16 * 128 + (17 * 64 + 1 * 16 + 2 * 4 + 1 if is_v else 1024 + 5 * 64 + 6)]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_in_pieces_stays_within_half_steps(fmt):
    """Positions written one to five at a time: each value is off by at most half
    a step of its code for every rounding it went through."""
    rng = np.random.default_rng(2)
    B, h, L, D, block = 1, 2, 64, 64, 16
    codes, amax = np.zeros((B, h, L, D)), np.zeros((B, h, L // block))
    x = rng.normal(0, 1, (B, L, h, D)) * np.exp(rng.normal(0, 1, (1, L, 1, 1)))
    p = 0
    while p < L:
        n = min(int(rng.integers(1, 6)), L - p)
        kv8.append(codes, amax, x[:, p:p + n], [p], [n], block, fmt)
        p += n
    assert np.allclose(amax, np.abs(x.transpose(0, 2, 1, 3)).reshape(B, h, L // block, -1).max(3))
    err = np.abs(kv8.values(codes, amax, block, fmt) - x.transpose(0, 2, 1, 3))
    a = np.repeat(amax, block, 2)[..., None]
    ref = np.abs(x.transpose(0, 2, 1, 3))
    # at most `block` roundings, most of them none; the step is a / 127, or 2^-3 of the value (half: 2^-4)
    step = a / 127 / 2 if fmt == "int8" else np.maximum(ref * 2.0 ** -4, a / 448 * 2.0 ** -10)
    assert (err <= 3 * step * (1 + 1e-9)).mean() > 0.999 and (err <= block * step).all()


def test_attention_agrees_with_the_layer_oracle():
    """On values that the codes hold exactly, the attention is the bf16 layer's."""
    rng = np.random.default_rng(3)
    H, B, K, L = 1280, 2, 2, 40
    w = oracle.round_bf16_bits(np.concatenate([np.eye(H) * 0.4, np.eye(H), np.eye(H)]))
    x = oracle.round_bf16_bits(rng.normal(0, 1, (B * (K + 1), H)))
    cache = np.zeros((B, 2, 64, H), np.uint16)
    cache[:, :, :L] = oracle.round_bf16_bits(rng.normal(0, 1, (B, 2, L, H)))
    lens = [L, 7]
    _, new, mid = oracle.attn_verify(x, w, oracle.round_bf16_bits(np.eye(H)), cache, lens, K)
    kv = oracle.widen(new).reshape(B, 2, 64, 10, 128).transpose(1, 0, 3, 2, 4)
    o, _, _ = kv8.attention(oracle.widen(mid["q"]).reshape(B, K + 1, 10, 128), kv[0], kv[1], lens, 128 ** -0.5)
    assert np.array_equal(oracle.round_bf16_bits(o).reshape(-1, H), mid["o"])


def test_logprobs_of_uniform_and_certain_rows():
    h = oracle.round_bf16_bits(np.zeros((1, 64)))
    lm = oracle.round_bf16_bits(np.random.default_rng(4).normal(0, 1, (50, 64)))
    lp, ent, _ = kv8.logprobs(h, lm)
    assert np.allclose(lp, -np.log(50)) and np.allclose(ent, np.log(50))
    lp, ent, _ = kv8.logprobs(oracle.round_bf16_bits(100 * oracle.widen(lm[3:4])), lm)
    assert lp[0].argmax() == 3 and abs(lp[0, 3]) < 1e-9 and ent[0] < 1e-9
