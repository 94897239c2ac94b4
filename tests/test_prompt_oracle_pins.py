"""Pins of the prompt-side oracle (CPU): closed forms, second routes, and the
absorbed attention on the same latents."""
import math

import numpy as np
import pytest

from oracle import mla_oracle as O
from oracle import prompt_oracle as P


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_is_a_complex_product_and_keeps_relative_positions(interleaved):
    rng = np.random.default_rng(1)
    f = P.rope_inv_freq()
    x, y = rng.standard_normal((5, 64)), rng.standard_normal((5, 64))
    pos = np.array([0, 1, 7, 4000, 163839])
    z = (x[:, 0::2] + 1j * x[:, 1::2]) if interleaved else (x[:, :32] + 1j * x[:, 32:])
    w = z * np.exp(1j * pos[:, None] * f) * 1.5
    got = P.rope_rotate(x, pos, f, interleaved, 1.5)
    gz = (got[:, 0::2] + 1j * got[:, 1::2]) if interleaved else (got[:, :32] + 1j * got[:, 32:])
    assert np.allclose(gz, w, atol=1e-12)
    assert np.array_equal(P.rope_rotate(x[:1], pos[:1], f, interleaved), x[:1])          # position 0
    # the product of two rotated vectors depends on the distance alone
    a = (P.rope_rotate(x, pos + 11, f, interleaved) * P.rope_rotate(y, pos, f, interleaved)).sum(1)
    b = (P.rope_rotate(x, np.full(5, 11), f, interleaved) * y).sum(1)
    assert np.allclose(a, b, atol=1e-9)


def test_scalings_meet_their_limits():
    f = P.rope_inv_freq()
    assert f[0] == 1.0 and math.isclose(f[16], 0.01)
    assert np.allclose(P.rope_inv_freq(scaling="linear", factor=8.0) * 8.0, f)
    y = P.rope_inv_freq(scaling="yarn", factor=40.0)
    assert np.allclose(P.rope_inv_freq(scaling="yarn", factor=1.0), f)
    # a pair that turns more than beta_fast times over the original context is left alone, one that turns
    # less than beta_slow times is interpolated, the rest lie between
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(y[turns > 40], f[turns > 40]) and np.allclose(y[turns < 0.8], f[turns < 0.8] / 40)
    assert (y <= f + 1e-15).all() and (y >= f / 40 - 1e-15).all()


def test_norm_and_row():
    rng = np.random.default_rng(2)
    rows, w = rng.standard_normal((3, 576)) * 3, rng.standard_normal(512)
    got = P.append_values(rows, [0, 5, 9], P.rope_inv_freq(), weight=w, eps=0.0)
    unit = got[:, :512] / w
    assert np.allclose((unit ** 2).mean(1), 1.0)
    assert np.allclose(unit / rows[:, :512], (unit / rows[:, :512])[:, :1])
    plain = P.append_values(rows, [0, 5, 9], P.rope_inv_freq())
    assert np.array_equal(plain[:, :512], rows[:, :512]) and np.array_equal(plain[0, 512:], rows[0, 512:])
    assert np.allclose((plain[:, 512:] ** 2).sum(1), (rows[:, 512:] ** 2).sum(1))


def test_expanded_attention_is_the_absorbed_one():
    rng = np.random.default_rng(3)
    H, L = 3, 17
    lat, kr = rng.standard_normal((L, 512)), rng.standard_normal((L, 64))
    w_kc, w_vc = rng.standard_normal((H, 128, 512)) / 22, rng.standard_normal((H, 512, 128)) / 22
    q = rng.standard_normal((L, H, 192))
    k, v = P.expand_rows(lat, w_kc, w_vc)
    out, lse, _ = P.prefill_attention(q, k, kr, v, [0, L], [0, L], 0.07)
    for i in (0, 5, L - 1):
        q_lat = O.absorb_query(q[i:i + 1, :, :128], w_kc)[0]
        o, l = O.partial_state(q_lat, q[i, :, 128:], np.concatenate([lat, kr], 1)[:i + 1], 0.07)
        assert np.allclose(O.project_output(o[None], w_vc)[0], out[i], atol=1e-10)
        assert np.allclose(l, lse[i], atol=1e-10)


def test_attention_closed_forms():
    rng = np.random.default_rng(4)
    q, v = rng.standard_normal((6, 2, 192)), rng.standard_normal((5, 2, 128))
    same = np.broadcast_to(rng.standard_normal((1, 2, 128)), (5, 2, 128))
    kr = np.zeros((5, 64))
    # equal keys: every row averages the values that it sees; the first request's second row is its last
    out, lse, mag = P.prefill_attention(q, same, kr, v, [0, 2, 6], [0, 3, 5], 0.1)
    assert np.allclose(out[1], v[:3].mean(0)) and np.allclose(out[0], v[:2].mean(0))
    assert np.allclose(mag[1], np.abs(v[:3]).mean(0))
    assert np.allclose(lse[1], 0.1 * (q[1, :, :128] * same[0]).sum(1) + math.log(3))
    # four queries over two keys: the first two see nothing
    assert (out[2:4] == 0).all() and np.isneginf(lse[2:4]).all()
    assert np.allclose(out[4], v[3]) and np.allclose(out[5], v[3:5].mean(0))
    full, _, _ = P.prefill_attention(q, same, kr, v, [0, 2, 6], [0, 3, 5], 0.1, causal=False)
    assert np.allclose(full[2], v[3:5].mean(0)) and np.allclose(full[0], v[:3].mean(0))
