"""GPU tests of the draft verification where it is decided by a number's last
bits: products below fp32's range, what rejected siblings left, numbers of one and
more, rows at the limits."""
import numpy as np
import pytest

from oracle import serving_oracle as S
from tests.test_gpu_between_steps import _dev, _same, _verify

pytestmark = pytest.mark.gpu

F = float.fromhex


@pytest.mark.parametrize("side", [-1, 0, 1])
@pytest.mark.parametrize("exponent", [-126, -100, -60, -3])
def test_a_sampled_drafts_product_is_exact(side, exponent):
    # u q is 2^-25 of itself below the nearest fp32 number, which is t, the one below it or the one above
    e = exponent // 2
    u1 = np.float32((1 + 2.0 ** -23) * 2.0 ** e)
    q1 = np.float32(1.75 * 2.0 ** (exponent - e))
    near = np.float32(np.float64(u1) * np.float64(q1))
    assert near > np.float64(u1) * np.float64(q1)
    t1 = near if side == 0 else np.nextafter(near, np.float32(side))
    target, draft = np.zeros((1, 2, 3), dtype=np.float32), np.zeros((1, 2, 3), dtype=np.float32)
    target[0, 0] = [1, t1, 0]
    draft[0, 1] = [0, q1, 1]
    u, tokens = np.array([[0.5, u1]], dtype=np.float32), np.array([[0, 1]])
    ref = S.verify(target, tokens, u, draft)
    assert ref[1][0] == (2 if side >= 0 else 1)
    _same(_verify(_dev(target, np.float32), tokens, u, _dev(draft, np.float32)), ref)


# masses of three rejected siblings, a number and a fourth one's mass: 64 bits decide between u (1 - sum) and it
CLOSE = [
    (("0x1.38dd6ap-2", "0x1.640386p-27", "0x1.638248p-1"), "0x1.7f0566p-1", "0x1.67548ep-14", False),
    (("0x1.370812p-2", "0x1.44e5dep-26", "0x1.646e1ep-1"), "0x1.578770p-2", "0x1.294388p-15", False),
    (("0x1.35a76ap-2", "0x1.2020eep-26", "0x1.651bb6p-1"), "0x1.c11a2cp-6", "0x1.d160a4p-19", False),
    (("0x1.3b6062p-2", "0x1.ee1424p-27", "0x1.623af2p-1"), "0x1.a01d06p-1", "0x1.0f45a6p-13", True),
    (("0x1.3436b2p-2", "0x1.5f70b4p-27", "0x1.65d6b6p-1"), "0x1.baaa5cp-1", "0x1.81ac92p-14", True),
    (("0x1.39a63ap-2", "0x1.811aaap-27", "0x1.631ef2p-1"), "0x1.a58f96p-1", "0x1.6f4884p-14", True),
]


@pytest.mark.parametrize("masses,u1,t1,taken", CLOSE)
def test_what_siblings_left_is_that_of_64_bits(masses, u1, t1, taken):
    target = np.zeros((1, 6, 6), dtype=np.float32)
    target[0, 0, :4] = [F(m) for m in masses] + [F(t1)]
    target[0, 4:] = 1 / 6
    tokens = np.array([[0, 0, 1, 2, 3, 1]])
    parents = np.array([[-1, 0, 0, 0, 0, 4]])
    u = np.array([[0.25, 1.0, 1.0, 1.0, F(u1), 0.99]], dtype=np.float32)     # 1.0: the first three are rejected
    ref = S.verify(target, tokens, u, parents=parents)
    assert (ref[0][0, 1] == 4) == taken
    _same(_verify(_dev(target, np.float32), tokens, u, parents=parents), ref)


def test_what_siblings_left_where_it_is_nearly_nothing():
    # masses that add up to one but for the last bits, and past it
    rng = np.random.default_rng(7)
    B, V = 400, 12
    target = np.zeros((B, 9, V), dtype=np.float32)
    m = np.sort(rng.random((B, 7)) ** 3, axis=1)[:, ::-1]
    target[:, 0, :7] = m / m.sum(1, keepdims=True) * (1 + rng.integers(-3, 4, (B, 1)) * 2.0 ** -24)
    target[:, 0, 7] = 2.0 ** -rng.integers(20, 60, B).astype(np.float64)
    target[:, 1:] = 1 / V
    tokens = np.tile([0, 0, 1, 2, 3, 4, 5, 6, 7], (B, 1))
    parents = np.tile([-1] + [0] * 8, (B, 1))
    u = np.ones((B, 9), dtype=np.float32)
    u[:, 0] = rng.random(B)
    u[:, 8] = rng.random(B)
    _same(_verify(_dev(target, np.float32), tokens, u, parents=parents), S.verify(target, tokens, u, parents=parents))


@pytest.mark.parametrize("V", [37, 4099, 32001, 129280])
@pytest.mark.parametrize("u0", [1.0, 1.5, float("inf"), float("nan")])
def test_a_number_of_one_draws_the_last_token(V, u0):
    # however little mass the last tokens have beside the sums' last bits
    rng = np.random.default_rng(V)
    B = 48
    target = rng.random((B, 1, V)).astype(np.float32)
    target /= target.sum(-1, keepdims=True)
    last = V - 1 - rng.integers(0, 30, B)
    for b in range(B):
        target[b, 0, last[b] - 5:] = 0
        target[b, 0, last[b]] = np.float32(2.0 ** -rng.integers(30, 120))
    u = np.full((B, 1), u0, dtype=np.float32)
    got = _verify(_dev(target, np.float32), np.zeros((B, 1), int), u)
    assert got[2].tolist() == last.tolist()
    _same(got, S.verify(target, np.zeros((B, 1), int), u))
