"""Pins of the gated-delta-rule and group-norm oracles (CPU): closed forms, a brute-force
product of the state maps, and the relations to the gated state scan."""
import numpy as np
import pytest
import torch


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_matches_products_of_the_state_maps(orc):
    """S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T, multiplied out."""
    b, s, hk, hv, dk, dv = 2, 9, 2, 4, 5, 3
    q, k = _rand(1, b, s, hk, dk), 0.5 * _rand(2, b, s, hk, dk)
    v, g, beta = _rand(3, b, s, hv, dv), -np.abs(_rand(4, b, s, hv)), _rand(5, b, s, hv)
    h0 = _rand(6, b, hv, dk, dv)
    reset = np.zeros((b, s), np.uint8)
    reset[1, 4] = 1
    out = orc.delta_scan(q, k, v, g, beta, reset=reset, h0=h0, scale=0.7)
    for i in range(b):
        for h in range(hv):
            S = h0[i, h]
            for t in range(s):
                kt = k[i, t, h // 2][:, None]
                a = 0.0 if reset[i, t] else np.exp(g[i, t, h])
                S = a * (np.eye(dk) - beta[i, t, h] * kt @ kt.T) @ S + beta[i, t, h] * kt @ v[i, t, h][None]
                np.testing.assert_allclose(out["outputs"][i, t, h], 0.7 * q[i, t, h // 2] @ S, rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(out["final_state"][i, h], S, rtol=1e-12, atol=1e-12)


def test_unit_key_with_full_strength_stores_its_value(orc):
    """beta = 1 and |k| = 1: afterwards the key reads exactly the value just written, and a
    second write under the same key replaces the first."""
    k = np.zeros((1, 2, 1, 4))
    k[..., 2] = 1.0
    v = _rand(7, 1, 2, 1, 3)
    out = orc.delta_scan(k, k, v, scale=1.0)
    np.testing.assert_allclose(out["outputs"], v, atol=1e-15)
    np.testing.assert_allclose(out["final_state"][0, 0, 2], v[0, 1, 0], atol=1e-15)
    assert not out["final_state"][0, 0, [0, 1, 3]].any()


def test_orthonormal_keys_equal_the_gated_scan(orc):
    """Keys that never meet leave nothing to take away: the gated state scan."""
    s, d = 6, 6
    k = np.eye(d)[None, :, None, :]
    q, v, g = _rand(8, 1, s, 1, d), _rand(9, 1, s, 1, 2), -np.abs(_rand(10, 1, s, 1))
    out = orc.delta_scan(q, k, v, g, scale=1.0)
    ref = orc.gated_scan(q[:, :, 0], k[:, :, 0], v[:, :, 0], np.exp(g[..., 0]))
    np.testing.assert_allclose(out["outputs"][:, :, 0], ref["outputs"], atol=1e-14)
    np.testing.assert_allclose(out["final_state"][:, 0], ref["final_state"], atol=1e-14)


def test_zero_strength_only_decays(orc):
    h0 = _rand(11, 1, 1, 4, 2)
    z = np.zeros((1, 3, 1))
    out = orc.delta_scan(_rand(12, 1, 3, 1, 4), _rand(13, 1, 3, 1, 4), _rand(14, 1, 3, 1, 2), z - 0.5, z, h0=h0)
    np.testing.assert_allclose(out["final_state"], np.exp(-1.5) * h0, rtol=1e-14)


def test_l2norm_ignores_the_length_and_chaining(orc):
    q, k, v = _rand(15, 1, 8, 1, 4), 10 * _rand(16, 1, 8, 1, 4), _rand(17, 1, 8, 1, 3)
    a = orc.delta_scan(q, k, v, qk_l2norm=True)
    b = orc.delta_scan(3 * q, 5 * k, v, qk_l2norm=True)
    np.testing.assert_allclose(a["outputs"], b["outputs"], rtol=1e-5, atol=1e-6)  # the eps in the root
    x = orc.delta_scan(q[:, :5], k[:, :5], v[:, :5], qk_l2norm=True)
    y = orc.delta_scan(q[:, 5:], k[:, 5:], v[:, 5:], qk_l2norm=True, h0=x["final_state"])
    np.testing.assert_allclose(y["final_state"], a["final_state"], rtol=1e-12)


@pytest.mark.parametrize("groups", [1, 3])
def test_group_norm_equals_torch(orc, groups):
    x, w, b = _rand(20, 4, 12), _rand(21, 12), _rand(22, 12)
    t = torch.nn.functional.group_norm(torch.from_numpy(x), groups, torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    np.testing.assert_allclose(orc.group_norm(x, groups, w, b), t.numpy(), rtol=1e-12, atol=1e-12)


def test_group_norm_forms(orc):
    x, z = _rand(23, 3, 8), _rand(24, 3, 8)
    silu = z / (1 + np.exp(-z))
    n = x / np.sqrt((x.reshape(3, 2, 4) ** 2).mean(-1, keepdims=True).repeat(4, -1).reshape(3, 8))
    np.testing.assert_allclose(orc.group_norm(x, 2, center=False, eps=0.0), n, rtol=1e-13)
    np.testing.assert_allclose(orc.group_norm(x, 2, center=False, eps=0.0, gate=z), n * silu, rtol=1e-13)
    np.testing.assert_allclose(orc.group_norm(x, 2, gate=z, gate_first=True), orc.group_norm(x * silu, 2), rtol=1e-13)
    w = _rand(25, 4)
    np.testing.assert_allclose(orc.group_norm(x, 2, w), orc.group_norm(x, 2, np.tile(w, 2)), rtol=1e-15)
