"""Pins of the 8-bit KV cache oracle (CPU): the E4M3 table and rounding
against torch's float8 cast, the exponent rule, the rotation against complex
multiplication, the attention against torch's softmax, and the eviction's
bookkeeping."""
import numpy as np
import pytest
import torch

from oracle import kv8


def test_e4m3_table_and_rounding_match_torch_cast():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv8.e4m3_table(), ref, equal_nan=True)
    g = torch.Generator().manual_seed(0)
    mid = np.sort(kv8.e4m3_table()[:127])
    y = np.concatenate([torch.randn(20000, generator=g).numpy() * 60, (mid[1:] + mid[:-1]) / 2,
                        -(mid[1:] + mid[:-1]) / 2, [0.0, 448.0, -448.0, 2.0 ** -10, 2.0 ** -11]])
    y = np.clip(y, -448, 448).astype(np.float32)
    got = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv8.e4m3_encode(y), got)
    assert list(kv8.e4m3_encode([np.nan, np.inf, -np.inf, 1e9])) == [0, 0x7e, 0xfe, 0x7e]


@pytest.mark.parametrize("amax, e", [(448.0, 0), (np.nextafter(np.float32(448), np.float32(500)), 1),
                                     (1.75, -8), (1.0, -8), (2.0, -7), (0.0, -110), (1e-40, -110),
                                     (3e38, 119)])
def test_block_exponent(amax, e):
    assert kv8.exponent(float(amax)) == e
    if -110 < e < 119:
        assert float(amax) <= 448 * 2.0 ** e and float(amax) > 448 * 2.0 ** (e - 1)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotation_is_complex_multiplication(layout):
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((5, 2, 12)), np.array([0, 1, 7, 1 << 20, -3])
    t = kv8.turns(8, base=500.0)
    y, _ = kv8.norm_rope(x, pos, t, 3, layout, norm=False)
    r = x[..., 3:11].reshape(5, 2, 4, 2) if layout == "interleaved" else \
        x[..., 3:11].reshape(5, 2, 2, 4).swapaxes(-1, -2)
    z = (r[..., 0] + 1j * r[..., 1]) * np.exp(2j * np.pi * pos[:, None, None] * t)
    back = np.stack([z.real, z.imag], -1)
    back = back.reshape(5, 2, 8) if layout == "interleaved" else back.swapaxes(-1, -2).reshape(5, 2, 8)
    assert np.abs(y[..., 3:11] - back).max() < 1e-8
    assert np.array_equal(y[..., :3], x[..., :3]) and np.array_equal(y[..., 11:], x[..., 11:])


def test_scaled_angles_between_trained_and_interpolated():
    t0, t = kv8.turns(64), kv8.turns(64, scaling="parts", factor=8.0, orig_len=4096.0)
    assert np.allclose(kv8.turns(64, scaling="linear", factor=8.0), t0 / 8)
    fast, slow = 4096 * t0 >= 32, 4096 * t0 <= 1
    assert fast.any() and slow.any()
    assert np.allclose(t[fast], t0[fast]) and np.allclose(t[slow], t0[slow] / 8)
    assert np.all(t <= t0 * (1 + 1e-15)) and np.all(t >= t0 / 8 * (1 - 1e-15))


def test_append_token_by_token_equals_one_call_but_for_subnormals():
    rng = np.random.default_rng(2)
    B, T, H, d, block, N = 2, 50, 2, 8, 16, 64
    x = rng.standard_normal((B, T, H, d)) * np.exp(rng.standard_normal((B, T, 1, 1)))
    one = np.zeros((B, H, N, d), np.uint8), np.zeros((B, H, N // block), np.uint8)
    step = one[0].copy(), one[1].copy()
    kv8.append(x, [3, 0], [T, T], *one, block)
    for t in range(T):
        kv8.append(x[:, t:t + 1], [3 + t, t], [1, 1], *step, block)
    assert np.array_equal(one[1][0, :, 1:], step[1][0, :, 1:]) and np.array_equal(one[1][1], step[1][1])
    a, b = kv8.values(*one, block), kv8.values(*step, block)
    # differences only where the larger exponent leaves a subnormal: one step of 2^(e-9)
    e = np.repeat(one[1].astype(float) - 127, block, -1)[..., None]
    diff = np.abs(a - b)
    assert np.all(diff[1] <= 2.0 ** (e[1] - 9)) and np.all(diff[1][np.abs(b[1]) >= 2.0 ** (e[1] - 5)] == 0)


def test_attention_matches_softmax_and_weights_sum_to_rows():
    rng = np.random.default_rng(3)
    q, K, V = rng.standard_normal((4, 6, 8)), rng.standard_normal((2, 3, 32, 8)), rng.standard_normal((2, 3, 32, 8))
    n_vis = np.array([0, 5, 32, 17])
    out, w, _, _ = kv8.attend(q, n_vis, K, V, 16, 0.3)
    for r in range(4):
        for h in range(6):
            n = n_vis[r]
            s = torch.softmax(torch.from_numpy(0.3 * K[r // 2, h // 2, :n] @ q[r, h]), 0).numpy()
            assert np.allclose(out[r, h], s @ V[r // 2, h // 2, :n] if n else 0.0)
    assert np.allclose(w.sum(-1), [[2.0] * 3, [4.0] * 3])   # two heads a KV head, rows that see anything
    low, w2, _, _ = kv8.attend(q, n_vis, K, V, 16, 0.3, sink=np.full(6, 60.0))
    assert np.abs(low).max() < 1e-20 and w2.max() < 1e-20
    assert np.allclose(kv8.attend(q, n_vis, K, V, 16, 0.3, sink=np.full(6, -800.0))[0], out)


def test_eviction_bookkeeping():
    acc = np.array([[[5, 1, 4, 4, 0, 9, 2, 0.5]]])
    kept, out, n = kv8.evict(acc, [125], 4, 1, 16)     # 8 blocks, the last one open
    # the last block stays; of the others 9, 5 and the first of the two 4s
    assert kept[0, 0].tolist() == [0, 5, 2, 7] and out[0, 0].tolist() == [5, 9, 4, 0.5, 0, 0, 0, 0]
    assert n[0] == 125 - 4 * 16
    kept, _, n = kv8.evict(acc, [60], 4, 1, 16)
    assert kept[0, 0].tolist() == [0, 1, 2, 3] and n[0] == 60
    acc[0, 0, 3] = np.nan
    assert kv8.evict(acc, [128], 7, 1, 16)[0][0, 0].tolist() == [0, 1, 2, 6, 4, 5, 7]
