"""CPU pins of the oracle's norm, rotation and paged-cache definitions:
closed forms, finite differences, PyTorch's float64 autograd, and the dense
oracle on a contiguous cache."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache


def angles(T, rope_dim, start=0, theta=10000.0):
    inv = theta ** (-np.arange(0, rope_dim, 2) / rope_dim)
    a = (start + np.arange(T))[:, None] * inv
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rope_dim", [(32, 32), (64, 32), (64, 0)])
def test_rotation_is_complex_multiplication_and_turns_back(D, rope_dim, interleaved):
    rng = np.random.default_rng(D + rope_dim)
    x = rng.standard_normal((5, 3, D))
    if rope_dim == 0:
        assert np.array_equal(cache.rotate(x, None, None, interleaved), x)
        return
    c, s = angles(5, rope_dim, start=11)
    y = cache.rotate(x, c, s, interleaved)
    a, b = ((x[..., 0:rope_dim:2], x[..., 1:rope_dim:2]) if interleaved
            else (x[..., :rope_dim // 2], x[..., rope_dim // 2:rope_dim]))
    z = (a + 1j * b) * (c + 1j * s)[:, None]
    ya, yb = ((y[..., 0:rope_dim:2], y[..., 1:rope_dim:2]) if interleaved
              else (y[..., :rope_dim // 2], y[..., rope_dim // 2:rope_dim]))
    assert np.allclose(ya, z.real) and np.allclose(yb, z.imag)
    assert np.array_equal(y[..., rope_dim:], x[..., rope_dim:])
    assert np.allclose(cache.rotate(y, c, -s, interleaved), x)


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    dots = []
    for p in (0, 17, 400):
        cq, sq = angles(1, 64, start=p + 9)
        ck, sk = angles(1, 64, start=p)
        dots.append(float((cache.rotate(q, cq, sq) * cache.rotate(k, ck, sk)).sum()))
    assert np.allclose(dots, dots[0])


def test_normed_rows_have_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((4, 2, 32)) * 37.0
    y = cache.norm_rope(x, np.ones(32), *angles(4, 32), eps=1e-12)
    assert np.allclose((y * y).mean(-1), 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [True, False])
def test_gradients_equal_autograd_and_differences(interleaved, weighted):
    rng = np.random.default_rng(3)
    T, H, D, R = 3, 2, 32, 16
    x, dy, w = rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D)), 1 + 0.3 * rng.standard_normal(D)
    c, s = angles(T, R, start=5)
    weight = w if weighted else None
    dx, dw = cache.norm_rope_backward(x, weight, dy, c, s, interleaved, eps=1e-2)

    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    n = tx * torch.rsqrt(tx.square().mean(-1, keepdim=True) + 1e-2) * tw if weighted else tx
    tc, ts = torch.tensor(c)[:, None], torch.tensor(s)[:, None]
    a, b = (n[..., 0:R:2], n[..., 1:R:2]) if interleaved else (n[..., :R // 2], n[..., R // 2:R])
    ra, rb = a * tc - b * ts, b * tc + a * ts
    y = torch.cat((torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1), n[..., R:]), -1)
    assert np.allclose(y.detach().numpy(), cache.norm_rope(x, weight, c, s, interleaved, eps=1e-2))
    (y * torch.tensor(dy)).sum().backward()
    assert np.allclose(dx, tx.grad.numpy())
    if weighted:
        assert np.allclose(dw, tw.grad.numpy())
    else:
        assert dw is None

    def loss(x_, w_):
        return float((cache.norm_rope(x_, w_, c, s, interleaved, eps=1e-2) * dy).sum())

    h = 1e-6
    for i in rng.integers(0, x.size, 12):
        e = np.zeros(x.size)
        e[i] = h
        e = e.reshape(x.shape)
        assert abs((loss(x + e, weight) - loss(x - e, weight)) / (2 * h) - dx.reshape(-1)[i]) < 1e-7
    if weighted:
        for i in range(0, D, 5):
            e = np.zeros(D)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_append_then_gather_returns_the_rows():
    rng = np.random.default_rng(4)
    pages = rng.standard_normal((9, 2, 8, 32))
    table = np.array([[3, 1, 7], [0, 8, 2], [5, 6, 4]])
    lens, cu = [20, 3, 0], [0, 11, 13, 14]  # the third sequence's token has no place
    rows = rng.standard_normal((14, 2, 32))
    after = cache.paged_append(pages, rows, table, lens, cu)
    assert np.array_equal(cache.gather(after, table[0], 20)[:, 9:], rows[0:11].transpose(1, 0, 2))
    assert np.array_equal(cache.gather(after, table[1], 3)[:, 1:], rows[11:13].transpose(1, 0, 2))
    assert np.array_equal(cache.gather(after, table[0], 9), cache.gather(pages, table[0], 9))
    assert int((after != pages).any(axis=(1, 3)).sum()) == 13
    assert cache.new_tokens([0], [0, 1]) == []


@pytest.mark.parametrize("window", [(-1, -1), (5, -1), (3, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_paged_attention_is_dense_attention_on_gathered_keys(causal, window):
    rng = np.random.default_rng(5)
    lens, cu = [21, 8, 0], [0, 3, 4, 6]
    table = np.array([[2, 0, 5], [4, -1, -1], [-1, -1, -1]])
    k_pages, v_pages = rng.standard_normal((2, 6, 2, 8, 32))
    q = rng.standard_normal((6, 4, 32))
    kw = dict(causal=causal, scale=0.2, window_left=window[0], window_right=window[1])
    o, lse = cache.attention_paged(q, k_pages, v_pages, table, lens, cu, **kw)
    k = np.concatenate([k_pages[p] for p in (2, 0, 5)], axis=1)[:, :21]
    v = np.concatenate([v_pages[p] for p in (2, 0, 5)], axis=1)[:, :21]
    ro, rl = oracle.attention_dense(q[None, 0:3].transpose(0, 2, 1, 3), k[None], v[None], **kw)
    assert np.array_equal(o[:3], ro[0].transpose(1, 0, 2)) and np.array_equal(lse[:, :3], rl[0])
    assert np.all(o[4:] == 0) and np.all(lse[:, 4:] == -np.inf)  # no keys
