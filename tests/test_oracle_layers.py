"""The FP64 oracle of the layers around RMA attention, against what the mathematics fixes."""
import numpy as np
import pytest

import oracle
import synth_inputs as si


def _np(t):
    return t.double().numpy()


def test_rotation_keeps_the_norm_and_depends_on_distances_only():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 3, 2, 256))
    w = np.ones(256)
    f = 1e4 ** (-np.arange(32) / 32)
    for inter in (False, True):
        y = oracle.norm_rope(x, w, np.array([[5, 70, 1000]]), f, 1e-6, inter)
        np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1) / ((x * x).mean(-1) + 1e-6), rtol=1e-12)
        z = oracle.norm_rope(x, w, np.array([[5, 70, 1000]]) + 12345, f, 1e-6, inter)
        a = np.einsum("bihd,bjhd->bhij", y, y)
        b = np.einsum("bihd,bjhd->bhij", z, z)
        np.testing.assert_allclose(a, b, atol=1e-8)
    still = oracle.norm_rope(x, w, np.zeros((1, 3)), f, 0.0)
    np.testing.assert_allclose(still, x / np.sqrt((x * x).mean(-1, keepdims=True)), rtol=1e-14)


def test_convolution_in_pieces_is_the_convolution_at_once():
    rng = np.random.default_rng(2)
    x, st, w = rng.standard_normal((2, 11, 5)), rng.standard_normal((2, 3, 5)), rng.standard_normal((5, 4))
    whole, end = oracle.conv_silu(x, st, w)
    parts, s = [], st
    for lo, hi in ((0, 1), (1, 3), (3, 3), (3, 11)):
        y, s = oracle.conv_silu(x[:, lo:hi], s, w)
        parts.append(y)
    np.testing.assert_array_equal(np.concatenate(parts, 1), whole)
    np.testing.assert_array_equal(s, end)
    np.testing.assert_array_equal(end, x[:, -3:])


def test_delta_rule_stores_and_replaces_what_a_key_holds():
    """beta 1 and no decay: after k -> v, reading with q = k gives v, whatever was there; with beta 0 and
    decay 1 nothing changes; with decay 0 everything is forgotten."""
    D = 128
    rng = np.random.default_rng(3)
    k, v1, v2 = rng.standard_normal(D), rng.standard_normal(D), rng.standard_normal(D)
    qkv = np.stack([np.concatenate([k, k, v1]), np.concatenate([k, k, v2])])[None]
    S0 = rng.standard_normal((1, 1, D, D))
    big = np.full((1, 2, 1), np.inf)
    o, S, _, _ = oracle.delta_rule(qkv, -big, big, [0.0], [0.0], S0, 1, l2_eps=0.0, scale=1.0)
    np.testing.assert_allclose(o[0, 0, 0], v1, atol=1e-12)
    np.testing.assert_allclose(o[0, 1, 0], v2, atol=1e-12)
    _, same, _, _ = oracle.delta_rule(qkv, -big, -big, [0.0], [0.0], S0, 1)
    np.testing.assert_array_equal(same, S0)
    o, S, _, _ = oracle.delta_rule(qkv[:, :1], big[:, :1], big[:, :1], [0.0], [0.0], S0, 1, l2_eps=0.0, scale=1.0)
    np.testing.assert_allclose(S[0, 0], np.outer(k / np.linalg.norm(k), v1), atol=1e-12)


@pytest.mark.parametrize("l2norm", [True, False])
def test_delta_rule_is_the_product_of_its_transitions(l2norm):
    """S_n = (prod e^g (1 - beta k k^T)) S_0 + ... : one head against explicit matrices, and lengths."""
    x = si.gdn_inputs(2, 6, 1, 2, seed=5)
    args = [_np(x[n]) for n in ("qkv", "a", "b", "a_log", "dt_bias", "state")]
    args[0] = args[0] * 0.2
    o, S, osize, size = oracle.delta_rule(*args, 1, l2norm=l2norm, lens=[6, 2])
    g, beta = oracle.delta_gates(*args[1:5])
    for b, n in ((0, 6), (1, 2)):
        for h in range(2):
            M = args[5][b, h]
            for t in range(n):
                q, k = args[0][b, t, :128], args[0][b, t, 128:256]
                v = args[0][b, t, 256 + 128 * h:384 + 128 * h]
                if l2norm:
                    q, k = q / np.sqrt(q @ q + 1e-6), k / np.sqrt(k @ k + 1e-6)
                M = np.exp(g[b, t, h]) * (np.eye(128) - beta[b, t, h] * np.outer(k, k)) @ M + beta[b, t, h] * np.outer(k, v)
                np.testing.assert_allclose(o[b, t, h], M.T @ q * 128 ** -0.5, rtol=1e-9, atol=1e-12)
            np.testing.assert_allclose(S[b, h], M, rtol=1e-9, atol=1e-12)
    assert np.isnan(o[1, 2:]).all() and np.isfinite(o[1, :2]).all()
    assert (size >= np.abs(S) - 1e-12).all() and (osize[0] >= np.abs(o[0]) - 1e-12).all()
