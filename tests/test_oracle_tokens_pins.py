"""Pins for the oracle of the token operators: against torch's library
routines in float64, closed forms and invariances."""
import numpy as np
import pytest
import torch

from oracle import tokens as ot

rng = np.random.default_rng(4)


@pytest.mark.parametrize("act,fn", [
    ("none", lambda z: z), ("relu", torch.relu), ("gelu", torch.nn.functional.gelu),
    ("quick_gelu", lambda z: z * torch.sigmoid(1.702 * z)), ("silu", torch.nn.functional.silu)])
def test_linear_equals_torch(act, fn):
    x, w, b, r = (rng.standard_normal(s) for s in ((5, 7), (3, 7), (3,), (5, 3)))
    want = fn(torch.nn.functional.linear(torch.from_numpy(x), torch.from_numpy(w), torch.from_numpy(b)))
    got, size = ot.linear(x, w, b, r, act)
    np.testing.assert_allclose(got, want.numpy() + r, rtol=0, atol=1e-13)
    assert np.all(size >= np.abs(x @ w.T))


def test_rope_is_a_rotation_of_each_pair_by_its_angle():
    x = rng.standard_normal((2, 3, 4, 10))
    pos = rng.integers(0, 50, (2, 3, 2)).astype(np.float32)
    freqs = np.array([[0.5, 0, 0.25, 0], [0, 1, 0, 0.125]], np.float32)
    for inter in (False, True):
        y, _ = ot.rope(x, pos, freqs, interleaved=inter)
        a = x[..., 0:8:2] + 1j * x[..., 1:8:2] if inter else x[..., :4] + 1j * x[..., 4:8]
        z = a * np.exp(1j * (pos @ freqs))[:, :, None]
        got = y[..., 0:8:2] + 1j * y[..., 1:8:2] if inter else y[..., :4] + 1j * y[..., 4:8]
        np.testing.assert_allclose(got, z, atol=1e-12)
        np.testing.assert_array_equal(y[..., 8:], x[..., 8:])


def test_rope_scores_depend_on_the_distance_alone():
    q, k = rng.standard_normal((1, 1, 1, 16)), rng.standard_normal((1, 1, 1, 16))
    freqs = np.abs(rng.standard_normal((2, 8))).astype(np.float32)
    dots = []
    for shift in (0, 7, 1000):
        a, _ = ot.rope(q, np.array([[[3 + shift, 5 + shift]]], np.float32), freqs)
        b, _ = ot.rope(k, np.array([[[9 + shift, 1 + shift]]], np.float32), freqs)
        dots.append((a * b).sum())
    np.testing.assert_allclose(dots, dots[0], atol=1e-10)


def test_norm_equals_torch_and_scales_away():
    x, w = rng.standard_normal((2, 2, 3, 12)), rng.standard_normal(12)
    pos, freqs = np.zeros((2, 2, 1), np.float32), np.ones((1, 6), np.float32)
    y, _ = ot.rope(x, pos, freqs, weight=w, eps=1e-6)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (12,), torch.from_numpy(w), 1e-6)
    np.testing.assert_allclose(y, want.numpy(), atol=1e-12)
    np.testing.assert_allclose(ot.rope(1e3 * x, pos, freqs, weight=w, eps=0.0)[0],
                               ot.rope(x, pos, freqs, weight=w, eps=0.0)[0], atol=1e-12)


def attend_inputs(B=3, Tq=4, Hq=4, Hk=2, D=8, P=5, S=6):
    return [rng.standard_normal(s) for s in
            ((B, Tq, Hq, D), (P, Hk, D), (P, Hk, D), (B, S, Hk, D), (B, S, Hk, D))]


@pytest.mark.parametrize("causal", [False, True])
def test_attention_equals_torch(causal):
    q, kp, vp, ko, vo = attend_inputs()
    own_len, mask = np.array([6, 4, 5]), rng.random((3, 6)) < 0.7
    got, mean_abs, _ = ot.prefix_attention(q, kp, vp, ko, vo, own_len, None, mask, causal)
    for b in range(3):
        n = own_len[b]
        k, v = (np.concatenate([p, o[b, :n]]) for p, o in ((kp, ko), (vp, vo)))
        allow = np.ones((4, 5 + n), bool)
        allow[:, 5:] &= mask[b, :n]
        if causal:
            allow[:, 5:] &= np.tril(np.ones((4, n), bool), n - 4)
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[b]).transpose(0, 1),
            torch.from_numpy(k).transpose(0, 1).repeat_interleave(2, 0),
            torch.from_numpy(v).transpose(0, 1).repeat_interleave(2, 0), torch.from_numpy(allow))
        np.testing.assert_allclose(got[b], want.transpose(0, 1).numpy(), atol=1e-12)
    assert np.all(mean_abs >= np.abs(got) - 1e-12)


def test_attention_without_keys_is_zero_and_hidden_places_do_not_matter():
    q, kp, vp, ko, vo = attend_inputs(P=0)
    own_len, q_len = np.array([6, 0, 2]), np.array([4, 4, 3])
    mask = np.ones((3, 6), bool)
    mask[0] = False
    got, _, _ = ot.prefix_attention(q, kp, vp, ko, vo, own_len, q_len, mask)
    assert not got[0].any() and not got[1].any() and not got[2, 3].any() and got[2, :3].all()
    ko[2, 2:], vo[2, 2:] = np.nan, np.nan
    np.testing.assert_array_equal(ot.prefix_attention(q, kp, vp, ko, vo, own_len, q_len, mask)[0], got)
