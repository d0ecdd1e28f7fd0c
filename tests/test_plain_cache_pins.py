"""The plain statements of the cache and attention against torch's own arithmetic, on the CPU."""
import numpy as np
import torch

import plain_cache as plain


def test_codes():
    every = np.arange(256).astype(np.uint8)
    want = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(plain.decode(every), want, equal_nan=True)
    x = np.concatenate([np.linspace(-500, 500, 20001), np.ldexp(np.linspace(-2, 2, 4001), -7), plain.MID, -plain.MID])
    x = x[np.abs(x) <= 448]
    x = x.astype(np.float32).astype(np.float64)
    got = plain.decode(plain.encode(x))
    assert np.array_equal(got, torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())
    assert plain.decode(plain.encode(np.array([1e9, -449.0]))).tolist() == [448.0, -448.0]


def test_rotation_is_orthogonal_and_turns_by_the_difference_of_positions():
    x, y = np.random.default_rng(0).standard_normal((2, 40, 3, 16))
    tab = plain.table(64, plain.frequencies(16))
    for interleaved in (False, True):
        a, b = (plain.rope(z, tab, np.arange(40), interleaved) for z in (x, y))
        assert np.allclose((a * b).sum(-1), (x * y).sum(-1), atol=1e-5)
        assert np.allclose(plain.rope(a, tab, np.arange(40), interleaved, back=True), x, atol=1e-5)
        c = plain.rope(x, tab, np.arange(40) + 9, interleaved)
        d = plain.rope(y, tab, np.arange(40) + 9, interleaved)
        assert np.allclose((c * d).sum(-1), (a * b).sum(-1), atol=1e-5)


def test_attention_over_pages():
    g = np.random.default_rng(1)
    H, G, D, page = 2, 3, 64, 16
    k, v = g.integers(0, 127, (2, 5, H, page, D)).astype(np.uint8)
    ks, vs = g.integers(118, 121, (2, 5, H)).astype(np.uint8)
    table = np.array([[3, 0, 4], [1, 2, -1]])
    lengths, offsets = np.array([40, 20]), np.array([0, 5, 25])
    q = g.standard_normal((25, H * G, D))
    for window in (0, 9):
        out, lse, _, _ = plain.attention(q, (k, v, ks, vs), table, lengths, offsets, 0.125, window)
        for b in range(2):
            rows, total = q[offsets[b]:offsets[b + 1]], lengths[b]
            for h in range(H * G):
                kk, vv = (np.concatenate([plain.decode(c[p, h // G]) * 2.0 ** (int(s[p, h // G]) - 127) for p in table[b][:-(-total // page)]])[:total]
                          for c, s in ((k, ks), (v, vs)))
                z = torch.from_numpy(rows[:, h] @ kk.T * 0.125)
                i, j = torch.arange(total - len(rows), total)[:, None], torch.arange(total)[None]
                z[(j > i) | ((j <= i - window) if window else torch.zeros_like(j <= i))] = float("-inf")
                assert np.allclose(out[offsets[b]:offsets[b + 1], h], torch.softmax(z, 1).numpy() @ vv, atol=1e-12)
                assert np.allclose(lse[offsets[b]:offsets[b + 1], h], torch.logsumexp(z, 1).numpy(), atol=1e-12)


def test_appended_blocks():
    H, D, page = 1, 64, 16
    x = np.random.default_rng(2).standard_normal((20, H, D))
    codes, byte = np.zeros((3, H, page, D), np.uint8), np.zeros((3, H), np.uint8)
    whole = plain.append((codes, byte), x, np.array([[2, 0]]), np.array([20]), np.array([0, 20]))
    e = int(np.floor(np.log2(np.abs(x[:16]).max()))) - 8
    assert whole[1][2, 0] == e + 127
    assert np.array_equal(plain.decode(whole[0][2, 0]), torch.from_numpy(x[:16, 0] * 2.0 ** -e).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy())
    c, s = codes, byte
    for n in range(1, 21):
        c, s = plain.append((c, s), x[n - 1:n], np.array([[2, 0]]), np.array([n]), np.array([0, 1]))
    assert np.array_equal(s, whole[1])
