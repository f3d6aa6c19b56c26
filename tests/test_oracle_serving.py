"""The serving operators' oracle against closed forms, torch's E4M3 cast and brute force."""

import numpy as np
import pytest
import torch

import oracle


def test_rotation_is_a_complex_product_and_keeps_the_norm():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 2, 32)), rng.standard_normal((3, 1, 32)), rng.standard_normal((3, 1, 32))
    ang = rng.uniform(0, 6, (5, 8))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = [4, 0, 2]
    for inter in (False, True):
        a, b, c = oracle.qk_norm_rope(q, k, v, None, None, 0.0, table, pos, inter)
        assert np.array_equal(c, v)
        one, two = (np.arange(0, 16, 2), np.arange(1, 16, 2)) if inter else (np.arange(8), np.arange(8, 16))
        z = (q[..., one] + 1j * q[..., two]) * np.exp(1j * ang[pos])[:, None]
        assert np.allclose(a[..., one], z.real) and np.allclose(a[..., two], z.imag)
        assert np.array_equal(a[..., 16:], q[..., 16:])
        assert np.allclose((b ** 2).sum(-1), (k ** 2).sum(-1))


def test_norm_has_unit_mean_square():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((2, 3, 64)) * 100
    a, _, _ = oracle.qk_norm_rope(q, q, q, np.ones(64), None, 0.0, None, [0, 0], False)
    assert np.allclose((a ** 2).mean(-1), 1.0)


def test_commit_scale_is_the_smallest_power_of_two():
    for top, want in ((448.0, 1.0), (450.0, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7),
                      (0.0, 2.0 ** -50), (np.inf, 2.0 ** -50)):
        kt = np.zeros((1, 1, 16), np.float32)
        kt[0, 0, 3] = top
        _, _, s, n = oracle.kv8p_commit(np.zeros((1, 1, 16, 16), np.uint8), np.zeros((1, 1, 16, 16), np.uint8),
                                        np.ones((1, 1, 2), np.float32), [[0]], [0], kt, kt, [[0]], [0], [0, 1])
        assert s[0, 0, 0] == want and n[0] == 1


def test_commit_codes_are_torchs_cast_and_growth_keeps_values():
    rng = np.random.default_rng(2)
    kt = rng.standard_normal((20, 2, 32)).astype(np.float32)
    kt[10:] *= 300.0
    z = lambda: np.zeros((3, 2, 16, 32), np.uint8)
    k1, _, s1, n1 = oracle.kv8p_commit(z(), z(), np.full((3, 2, 2), np.nan, np.float32), [[2, 0]], [0], kt, kt,
                                       [list(range(10))], [9], [0, 20])
    want = torch.from_numpy((kt[:10] / s1[2, :, 0][None, :, None])).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(k1[2, :, :10].transpose(1, 0, 2), want)
    k2, _, s2, n2 = oracle.kv8p_commit(k1, k1, s1, [[2, 0]], n1, kt, kt, [list(range(10, 20))], [9], [0, 20])
    assert (s2[2, :, 0] > s1[2, :, 0]).all() and n2[0] == 20
    before, after = oracle.kv8p_values(k1, s1, 0)[2, :, :10], oracle.kv8p_values(k2, s2, 0)[2, :, :10]
    step = s2[2, :, 0][:, None, None] * 2.0 ** -9      # E4M3's smallest step at the new scale
    assert (np.abs(after - before) <= np.maximum(step / 2, np.abs(before) * 2.0 ** -4)).all()
    big = np.abs(before) >= s2[2, :, 0][:, None, None] * 2.0 ** -6
    assert np.array_equal(after[big], before[big])     # normal numbers only shift their exponent
    assert (k2[0, :, 4:] == 0).all() and (k2[1] == 0).all()


@pytest.mark.parametrize("seed", range(6))
def test_resize_conserves_pages(seed):
    rng = np.random.default_rng(seed)
    B, most, ps, total = 7, 9, 4, 60
    ids = rng.permutation(total)
    held = rng.integers(0, 6, B)
    table = np.full((B, most), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(total, -1, np.int64)
    free[:total - at] = ids[at:]
    qo = np.concatenate([[0], np.cumsum(rng.integers(0, 9, B))])
    lens = rng.integers(0, 20, B)
    t, h, f, n, slots, err = oracle.page_table_resize(lens, qo, held, table, free, total - at, ps, seed % 2)
    have = [x for b in range(B) for x in t[b, :h[b]]] + list(f[:n])
    assert sorted(have) == list(range(total)) and not err
    need = -(-(lens + np.diff(qo)) // ps)
    assert (h >= need).all() and (h == (need if seed % 2 else np.maximum(need, held))).all()
    assert len(set(slots)) == len(slots) and (slots >= 0).all()


def test_resize_grants_in_order_while_the_stack_lasts():
    t, h, f, n, slots, err = oracle.page_table_resize([0, 0, 0], [0, 2, 5, 6], [0, 0, 0], np.full((3, 4), -1),
                                                      [7, 8, 9], 3, 1, False)
    assert list(h) == [2, 0, 0] and list(t[0, :2]) == [9, 8] and n == 1 and f[0] == 7 and err == {"capacity"}
    assert list(slots) == [9, 8, -1, -1, -1, -1]
