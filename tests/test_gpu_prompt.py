"""GPU tests of the prompt side (rotary query and append, latent expansion,
expanded attention) against the fp64 oracle, operator by operator and as they
run together, beside the absorbed decode on the same cache.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of E4M3
2^-4 (2^-10 below its smallest normal 2^-6); fp32 intermediates add what each
test states."""
import math

import numpy as np
import pytest

from oracle import mla_oracle as O
from oracle import prompt_oracle as P

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


def _t():
    import torch
    from mla_latent_kv_absorbed_gb300 import binding
    return torch, binding


def _normal(seed, *shape, scale=1.0):
    """bf16 N(0, scale^2) on the GPU and its exact float64 values."""
    torch, _ = _t()
    x = np.random.default_rng(seed).standard_normal(shape, dtype=np.float32) * np.float32(scale)
    d = torch.from_numpy(x).to(torch.bfloat16).cuda()
    return d, d.double().cpu().numpy()


def _f64(t):
    return t.double().cpu().numpy()


def _within(got, ref, bound, what):
    assert got.shape == ref.shape
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"{what}: {int((err > bound).sum())} of {err.size} off, worst by {(err - bound).max():.3e}"


YARN = dict(scaling="yarn", factor=40.0)


def _inv(kw):
    return P.rope_inv_freq(**kw)


def _rope_bound(ref, x, amplitude=1.0):
    """One bf16 rounding; in fp32: the phase's conversion to 24 bits (2^-24 of half a turn: pi 2^-24 rad), sincospi
    and three roundings, under 2^-20 of |x0| + |x1|; the float64 angle itself, pos * f, is good to 2^-52 of at most
    2^31 rad."""
    both = np.abs(x).max(axis=-1, keepdims=True) * 2 * abs(amplitude)
    return BF * np.abs(ref) + (2.0 ** -20 + 2.0 ** -21) * both


# ------------------------------------------------------------------- rotary query

@pytest.mark.parametrize("T,H,nope,interleaved,kw,amplitude,split", [
    (1, 1, 128, True, {}, 1.0, True),
    (3, 16, 128, False, YARN, 1.25, True),
    (64, 128, 128, True, YARN, 1.0, True),
    (5, 5, 0, False, {}, 1.0, False),
    (37, 33, 64, True, dict(scaling="linear", factor=8.0), 0.5, True),
    (200, 48, 192, False, YARN, 1.0, False),
    (1000, 32, 8, True, {}, 1.0, True),
])
def test_rope_query(T, H, nope, interleaved, kw, amplitude, split):
    torch, B = _t()
    q, x = _normal(T + H, T, H, nope + 64)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 163840, T).astype(np.int32)
    out = torch.full((T, H, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    rest = torch.full((T, H, nope), float("nan"), dtype=torch.bfloat16, device="cuda") if split else None
    before = q.clone()
    B.rope_query(q, torch.from_numpy(pos).cuda(), B.rope_frequencies(**kw), out, q_nope=rest, amplitude=amplitude,
                 interleaved=interleaved)
    ref = P.rope_rotate(x[..., nope:], pos, _inv(kw), interleaved, amplitude)
    _within(_f64(out), ref, _rope_bound(ref, x[..., nope:], amplitude), "rope")
    if split:
        assert torch.equal(rest, q[..., :nope])
    assert torch.equal(q, before)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,nope", [(100, 160, 128), (90, 130, 64), (5, 3, 2064), (3, 2, 65536), (700, 33, 200),
                                      (80, 300, 8)])
def test_rope_query_of_many_heads_and_wide_ones(T, H, nope, interleaved):
    # units of 128 heads with a rest, blocks that take several, heads whose other part is wider than a block moves at once
    torch, B = _t()
    q, x = _normal(T + nope, T, H, nope + 64)
    pos = np.random.default_rng(T).integers(0, 163840, T).astype(np.int32)
    out = torch.full((T, H, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    rest = torch.full((T, H, nope), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.rope_query(q, torch.from_numpy(pos).cuda(), B.rope_frequencies(**YARN), out, q_nope=rest, interleaved=interleaved)
    ref = P.rope_rotate(x[..., nope:], pos, _inv(YARN), interleaved)
    _within(_f64(out), ref, _rope_bound(ref, x[..., nope:]), "rope")
    assert torch.equal(rest, q[..., :nope])


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_query_at_the_ends_of_the_positions(interleaved):
    torch, B = _t()
    pos = np.array([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], dtype=np.int32)
    q, x = _normal(5, len(pos), 4, 64)
    out = torch.empty_like(q)
    B.rope_query(q, torch.from_numpy(pos).cuda(), B.rope_frequencies(), out, interleaved=interleaved)
    ref = P.rope_rotate(x, pos.astype(np.int64), _inv({}), interleaved)
    _within(_f64(out), ref, _rope_bound(ref, x), "far positions")
    assert torch.equal(out[0], q[0])                            # position 0 turns nothing


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("kw", [dict(theta=1e6, scaling="linear", factor=40.0), dict(scaling="yarn", factor=40.0),
                                dict(theta=1e7, scaling="yarn", factor=160.0)])
def test_small_angles_keep_their_relative_precision(kw, interleaved):
    # the slowest pairs turn by 1e-9 of a turn and less a position: with x1 = 0 the second value is x0 times a sine of
    # that size, one rounding and 2^-20 of it (the angle's conversion to 24 bits, sincospi, the product) off
    torch, B = _t()
    pos = np.array([1, 2, 3, 7, -1, -5, 100, 4095], dtype=np.int32)
    T = len(pos)
    first = np.zeros(64, dtype=bool)
    first[0::2 if interleaved else 1] = True
    if not interleaved:
        first[32:] = False
    q = torch.zeros((T, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[..., torch.from_numpy(first).cuda()] = 1.5
    out = torch.empty_like(q)
    p, fr = torch.from_numpy(pos).cuda(), B.rope_frequencies(**kw)
    B.rope_query(q, p, fr, out, interleaved=interleaved)
    ref = P.rope_rotate(_f64(q), pos, _inv(kw), interleaved)
    bound = (BF + 2.0 ** -20) * np.abs(ref)
    sines = np.abs(ref[..., ~first]) < 1.0                      # (near a zero of a cosine the angle's own error counts)
    err = np.abs(_f64(out) - ref)
    assert (err[..., ~first][sines] <= bound[..., ~first][sines]).all(), (err / np.abs(ref))[..., ~first].max()
    cache = torch.zeros((T, 576), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros((T, 576), dtype=torch.bfloat16, device="cuda")
    rows[:, 512:] = q[:, 0]
    B.rope_append_kv(cache, torch.arange(T, dtype=torch.int32, device="cuda"), rows, p, fr, interleaved=interleaved)
    assert torch.equal(cache[:, 512:], out[:, 0])


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_query_in_place_and_strided(interleaved):
    # a query cut out of a wider projection, rotated where it lies; and heads outermost
    torch, B = _t()
    T, H = 29, 6
    wide, x = _normal(6, T, H * 192 + 40)
    q = wide[:, 24:24 + H * 192].view(T, H, 192)
    xq = x[:, 24:24 + H * 192].reshape(T, H, 192)
    pos = np.arange(T, dtype=np.int32) + 4000
    before = wide.clone()
    fr = B.rope_frequencies(**YARN)
    p = torch.from_numpy(pos).cuda()
    heads_first = torch.full((H, T, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.rope_query(q, p, fr, heads_first[:, :, :64].transpose(0, 1), interleaved=interleaved)
    ref = P.rope_rotate(xq[..., 128:], pos, _inv(YARN), interleaved)
    bound = _rope_bound(ref, xq[..., 128:])
    _within(_f64(heads_first[:, :, :64].transpose(0, 1)), ref, bound, "heads outermost")
    assert torch.isnan(heads_first[:, :, 64:]).all()
    assert torch.equal(wide, before)
    B.rope_query(q, p, fr, q[..., 128:], interleaved=interleaved)
    _within(_f64(q[..., 128:]), ref, bound, "in place")
    wide.view(T, -1)[:, 24:24 + H * 192].view(T, H, 192)[..., 128:] = before[:, 24:24 + H * 192].view(T, H, 192)[..., 128:]
    assert torch.equal(wide, before)                            # nothing else was written


def test_rope_query_of_no_tokens_writes_nothing():
    torch, B = _t()
    z = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    B.rope_query(z(0, 4, 192), z(0, dt=torch.int32), B.rope_frequencies(), z(0, 4, 64), q_nope=z(0, 4, 128))


# ------------------------------------------------------------------------ append

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,norm,interleaved,kw,stride,amplitude", [
    (1, True, True, YARN, 576, 1.0), (4, False, False, {}, 576, 1.0), (37, True, False, YARN, 584, 1.5),
    (300, True, True, dict(scaling="linear", factor=8.0), 2112, 1.0), (9, False, True, YARN, 1344, 1.0),
])
def test_rope_append(fp8, T, norm, interleaved, kw, stride, amplitude):
    torch, B = _t()
    N, scale = T + 50, 2.0 ** -5
    wide, x = _normal(T, T, stride, scale=2.0)
    rows, xr = wide[:, stride - 576:], x[:, stride - 576:]
    w, xw = _normal(T + 1, 512)
    rng = np.random.default_rng(T + 2)
    slots, pos = rng.permutation(N)[:T].astype(np.int32), rng.integers(0, 163840, T).astype(np.int32)
    cache = torch.from_numpy(rng.integers(0, 120, (N, 576)).astype(np.uint8)).cuda() if fp8 else _normal(T + 3, N, 576)[0]
    before = cache.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (cache, torch.from_numpy(slots).cuda(), rows, torch.from_numpy(pos).cuda(), B.rope_frequencies(**kw))
    more = dict(norm_weight=w if norm else None, eps=1e-5, amplitude=amplitude, interleaved=interleaved, workspace=ws)
    if fp8:
        B.rope_append_kv_fp8(*args, scale, **more)
    else:
        B.rope_append_kv(*args, **more)
    assert B.check_errors(ws) == 0
    ref = P.append_values(xr, pos, _inv(kw), xw if norm else None, 1e-5, interleaved, amplitude)
    # fp32: the sum of squares (32 roundings), rsqrt and the products, or the rotation: under 2^-18 of the value or
    # 2^-19 of the pair
    slack = 2.0 ** -18 * np.abs(ref)
    slack[:, 512:] += 2.0 ** -19 * np.abs(xr[:, 512:]).max(axis=1, keepdims=True) * 2 * amplitude
    got = cache[torch.from_numpy(slots).long().cuda()]
    if fp8:
        want = np.clip(ref / scale, -448, 448)
        bound = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + slack / scale
        _within(_f64(got.view(torch.float8_e4m3fn)), want, bound, "append fp8")
        if not norm:                                            # latents as mla_append_kv_fp8 quantises them
            codes = O.quantize_rows_e4m3(rows.contiguous().cpu().view(torch.int16).numpy().view(np.uint16), scale)
            assert np.array_equal(got[:, :512].cpu().numpy(), codes[:, :512])
    else:
        _within(_f64(got), ref, BF * np.abs(ref) + slack, "append")
        if not norm:
            assert torch.equal(got[:, :512], rows[:, :512])     # bits pass unchanged
    rest = np.setdiff1d(np.arange(N), slots)
    assert torch.equal(cache[rest], before[rest])


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("scale", [0.0371, 3.0, 1e-3])
def test_rope_append_of_any_fp8_scale(scale, norm):
    # scales that are no power of two divide; values past 448 scales saturate, infinities with them, NaN stays NaN
    torch, B = _t()
    T = 70
    s32 = float(np.float32(scale))
    rows, x = _normal(T, T, 576, scale=2.0)
    rows[1] *= 4096.0
    rows[2, 512:] *= 2048.0
    x = _f64(rows)
    w, xw = _normal(T + 1, 512)
    pos = np.random.default_rng(3).integers(0, 163840, T).astype(np.int32)
    cache = torch.zeros((T, 576), dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    B.rope_append_kv_fp8(cache, slots, rows, torch.from_numpy(pos).cuda(), B.rope_frequencies(**YARN), scale,
                         norm_weight=w if norm else None)
    ref = P.append_values(x, pos, _inv(YARN), xw if norm else None)
    slack = 2.0 ** -18 * np.abs(ref)                            # as in test_rope_append; the division adds 2^-24
    slack[:, 512:] += 2.0 ** -19 * np.abs(x[:, 512:]).max(axis=1, keepdims=True) * 2
    want = np.clip(ref / s32, -448, 448)
    bound = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + slack / s32
    got = _f64(cache.view(torch.float8_e4m3fn))
    _within(got, want, bound, "append fp8")
    assert (np.abs(ref / s32) > 500).any() and (np.abs(got)[np.abs(ref / s32) > 500] == 448).all()
    if not norm:
        # latents that are not finite, as mla_append_kv_fp8 quantises them
        rows[3, 5], rows[3, 6], rows[3, 7], rows[3, 8] = float("inf"), float("-inf"), float("nan"), 1e30
        B.rope_append_kv_fp8(cache, slots, rows, torch.from_numpy(pos).cuda(), B.rope_frequencies(**YARN), scale)
        codes = O.quantize_rows_e4m3(rows.contiguous().cpu().view(torch.int16).numpy().view(np.uint16), s32)
        assert np.array_equal(cache[:, :512].cpu().numpy(), codes[:, :512])
        assert cache[3, 5:9].tolist() == [0x7E, 0xFE, 0x7F, 0x7E]


@pytest.mark.parametrize("T,H", [(37, 3), (700, 33)])
@pytest.mark.parametrize("scale", [0.0371, 3.0])
def test_expand_of_any_fp8_scale(T, H, scale):
    torch, B = _t()
    s32 = float(np.float32(scale))
    cache, x = _codes(T, T)
    x = x * s32
    wk, xk = _normal(T + 2, H, 128, 512, scale=512 ** -0.5)
    wv, xv = _normal(T + 3, H, 512, 128, scale=512 ** -0.5)
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    k, kr, v = bf(T, H, 128), bf(T, 64), bf(T, H, 128)
    B.expand_kv_fp8(cache, scale, torch.arange(T, dtype=torch.int32, device="cuda"), wk, wv, k, kr, v)
    lat = x[:, :512]
    rk, rv = P.expand_rows(lat, xk, xv)
    _within(_f64(k), rk, _expand_bound(rk, lat, xk, "tr,hnr->thn"), "k")
    _within(_f64(v), rv, _expand_bound(rv, lat, xv, "tr,hrn->thn"), "v")
    # code times scale in fp32 (2^-24), then to bf16
    _within(_f64(kr), x[:, 512:], (BF + 2.0 ** -22) * np.abs(x[:, 512:]), "k_rope")


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_append_skips_and_reports_bad_slots(fp8):
    torch, B = _t()
    N, T = 20, 5
    rows, _ = _normal(8, T, 576)
    cache = torch.zeros((N, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    slots = torch.tensor([3, -1, N, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fr = B.rope_frequencies()
    call = (lambda w: B.rope_append_kv_fp8(cache, slots, rows, pos, fr, 1.0, workspace=w)) if fp8 else \
        (lambda w: B.rope_append_kv(cache, slots, rows, pos, fr, workspace=w))
    call(ws)
    assert B.check_errors(ws) == 6 and B.check_errors(ws) == 0
    written = cache.float().abs().sum(1).nonzero().flatten().tolist()
    assert written == [3, 7]
    if not fp8:
        assert torch.equal(cache[7], rows[4])                   # position 0, no norm: the row itself
    call(None)                                                  # without a status word


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_append_of_more_rows_than_warps(fp8, interleaved):
    # a warp takes several rows, the next one's loads ahead, with slots outside the cache among them
    torch, B = _t()
    T, N, scale = 9001, 9500, 2.0 ** -5
    rows, x = _normal(7, T, 576)
    w, xw = _normal(8, 512)
    rng = np.random.default_rng(9)
    slots, pos = rng.permutation(N)[:T].astype(np.int32), rng.integers(0, 163840, T).astype(np.int32)
    lost = rng.permutation(T)[:300]
    slots[lost[:100]], slots[lost[100:200]], slots[lost[200:]] = -1, N, 2 ** 31 - 1
    cache = torch.zeros((N, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (cache, torch.from_numpy(slots).cuda(), rows, torch.from_numpy(pos).cuda(), B.rope_frequencies(**YARN))
    if fp8:
        B.rope_append_kv_fp8(*args, scale, norm_weight=w, interleaved=interleaved, workspace=ws)
    else:
        B.rope_append_kv(*args, norm_weight=w, interleaved=interleaved, workspace=ws)
    assert B.check_errors(ws) == 6
    there = np.setdiff1d(np.arange(T), lost)
    ref = P.append_values(x[there], pos[there], _inv(YARN), xw, 1e-6, interleaved)
    slack = 2.0 ** -18 * np.abs(ref)                            # as in test_rope_append
    slack[:, 512:] += 2.0 ** -19 * np.abs(x[there, 512:]).max(axis=1, keepdims=True) * 2
    got = cache[torch.from_numpy(slots[there]).long().cuda()]
    if fp8:
        want = np.clip(ref / scale, -448, 448)
        _within(_f64(got.view(torch.float8_e4m3fn)), want, np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + slack / scale, "rows")
    else:
        _within(_f64(got), ref, BF * np.abs(ref) + slack, "rows")
    rest = np.setdiff1d(np.arange(N), slots[there])
    assert not cache[torch.from_numpy(rest).cuda()].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_append_past_4_gib_of_the_cache(fp8):
    torch, B = _t()
    row = 576 * (1 if fp8 else 2)
    slot = (2 ** 32) // row + 5
    cache = torch.empty((slot + 1, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    cache[5] = 0
    rows, _ = _normal(9, 1, 576)
    s, pos = torch.tensor([slot], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    if fp8:
        B.rope_append_kv_fp8(cache, s, rows, pos, B.rope_frequencies(), 1.0)
        assert torch.equal(cache[slot].view(torch.float8_e4m3fn).float(), rows[0].to(torch.float8_e4m3fn).float())
    else:
        B.rope_append_kv(cache, s, rows, pos, B.rope_frequencies())
        assert torch.equal(cache[slot], rows[0])
    assert (cache[5].float() == 0).all()


# --------------------------------------------------------------------- expansion

def _codes(seed, n):
    torch, _ = _t()
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((n, 576), dtype=np.float32) * 32)
    c = x.to(torch.float8_e4m3fn)
    return c.view(torch.uint8).cuda(), c.double().numpy()


def _expand_bound(ref, lat, w, eq, scale=1.0):
    """One bf16 rounding, and 512 fp32 additions that may each lose 2^-22 of the sum of magnitudes' running
    value (an accumulator that truncates, with a guard bit): at most 512 * 2^-22 of it."""
    return BF * np.abs(ref) + 2.0 ** -13 * scale * np.einsum(eq, np.abs(lat), np.abs(w), optimize=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (2, 5), (127, 16), (128, 1), (129, 3), (300, 16), (64, 33), (515, 2),
                                 (100, 160), (1290, 33), (2560, 17), (4700, 17), (1290, 61)])
def test_expand(fp8, T, H):
    torch, B = _t()
    N, scale = T + 77, 2.0 ** -5
    cache, x = _codes(T, N) if fp8 else _normal(T, N, 576)
    x = x * scale if fp8 else x
    idx = np.random.default_rng(T + 1).integers(0, N, T).astype(np.int32)           # repeats among them
    wk, xk = _normal(T + 2, H, 128, 512, scale=512 ** -0.5)
    wv, xv = _normal(T + 3, H, 512, 128, scale=512 ** -0.5)
    full = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    # one row more than the call is given: it has to stay as it is
    k, kr, v = full(T + 1, H, 128), full(T + 1, 64), full(T + 1, H, 128)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ind = torch.from_numpy(idx).cuda()
    if fp8:
        B.expand_kv_fp8(cache, scale, ind, wk, wv, k[:T], kr[:T], v[:T], workspace=ws)
    else:
        B.expand_kv(cache, ind, wk, wv, k[:T], kr[:T], v[:T], workspace=ws)
    assert B.check_errors(ws) == 0
    lat = x[idx][:, :512]
    rk, rv = P.expand_rows(lat, xk, xv)
    _within(_f64(k[:T]), rk, _expand_bound(rk, lat, xk, "tr,hnr->thn"), "k")
    _within(_f64(v[:T]), rv, _expand_bound(rv, lat, xv, "tr,hrn->thn"), "v")
    assert np.array_equal(_f64(kr[:T]), x[idx][:, 512:])        # a power-of-two scale: exact in bf16
    for y in (k, kr, v):
        assert torch.isnan(y[T]).all()


def test_expand_reports_bad_indices_and_reads_row_0():
    torch, B = _t()
    N, H = 9, 2
    cache, _ = _normal(1, N, 576)
    wk, wv = _normal(2, H, 128, 512)[0], _normal(3, H, 512, 128)[0]
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    got = [bf(4, H, 128), bf(4, 64), bf(4, H, 128)]
    ref = [bf(4, H, 128), bf(4, 64), bf(4, H, 128)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.expand_kv(cache, torch.tensor([3, -1, N, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), wk, wv, *got, workspace=ws)
    assert B.check_errors(ws) == 6
    B.expand_kv(cache, torch.tensor([3, 0, 0, 0], dtype=torch.int32, device="cuda"), wk, wv, *ref, workspace=ws)
    assert B.check_errors(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("fp8", [False, True])
def test_expand_a_row_that_is_not_finite_stays_alone(fp8):
    torch, B = _t()
    N, H = 200, 3
    cache, x = _codes(1, N) if fp8 else _normal(1, N, 576)
    if fp8:
        cache[7, 5] = 0x7F                                      # the NaN code
    else:
        cache[7, 5] = float("nan")
        cache[8, 600 - 576] = float("inf")
    wk, wv = _normal(2, H, 128, 512)[0], _normal(3, H, 512, 128)[0]
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    k, kr, v = bf(N, H, 128), bf(N, 64), bf(N, H, 128)
    idx = torch.arange(N, dtype=torch.int32, device="cuda")
    B.expand_kv_fp8(cache, 0.5, idx, wk, wv, k, kr, v) if fp8 else B.expand_kv(cache, idx, wk, wv, k, kr, v)
    assert torch.isnan(k[7]).all() and torch.isnan(v[7]).all()
    fine = [i for i in range(N) if i not in (7, 8)]
    assert torch.isfinite(k[fine]).all() and torch.isfinite(v[fine]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_expand_past_4_gib_of_the_cache(fp8):
    torch, B = _t()
    row = 576 * (1 if fp8 else 2)
    slot = (2 ** 32) // row + 3
    small, _ = _codes(4, 2) if fp8 else _normal(4, 2, 576)
    cache = torch.empty((slot + 1, 576), dtype=small.dtype, device="cuda")
    cache[3] = small[1]
    cache[slot] = small[0]
    wk, wv = _normal(2, 4, 128, 512)[0], _normal(3, 4, 512, 128)[0]
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    got, ref = [bf(1, 4, 128), bf(1, 64), bf(1, 4, 128)], [bf(1, 4, 128), bf(1, 64), bf(1, 4, 128)]
    call = (lambda c, i, o: B.expand_kv_fp8(c, 0.5, i, wk, wv, *o)) if fp8 else (lambda c, i, o: B.expand_kv(c, i, wk, wv, *o))
    call(cache, torch.tensor([slot], dtype=torch.int32, device="cuda"), got)
    call(small, torch.tensor([0], dtype=torch.int32, device="cuda"), ref)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


# --------------------------------------------------------------------- attention

SM = 1.0 / math.sqrt(192.0)


def _attention_bound(ref, mag):
    """The output's rounding to bf16, the weights' (2^-8 of sum p |v|), and in fp32 the scores (192 products,
    under 2^-12 absolute at these inputs, so 2 * 2^-12 of a normalised weight) and the exponential (2^-20)."""
    return BF * np.abs(ref) + (BF + 2.0 ** -10) * mag


LSE_ATOL = 2.0 ** -11      # a score's 2^-12, and the fp32 sum of at most 4096 weights (2^-12)


MANY = [
    # more (tile, head) items than SMs, so that blocks take several in turn: with and without a second row tile,
    # whole and partly seen key tiles, rows without keys
    ([1, 7, 33, 100, 140, 260, 300, 0, 129], [1, 7, 33, 100, 140, 260, 300, 9, 129], 64, True),
    ([130, 64, 5, 280], [700, 64, 0, 100], 80, True),
    ([300, 1, 1, 1, 200], [300, 400, 128, 129, 513], 48, False),
]


def _attention_inputs(seed, nq, nk, H):
    return [_normal(seed, nq, H, 192), _normal(seed + 1, nk, H, 128), _normal(seed + 2, nk, 64), _normal(seed + 3, nk, H, 128)]


def _indptr(lengths):
    return np.cumsum(np.r_[0, lengths]).astype(np.int32)


def _attend(plan, q, k, kr, v, lse=True, sm=SM):
    torch, B = _t()
    out = torch.full((q.shape[0], q.shape[1], 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    l = torch.full((q.shape[0], q.shape[1]), float("nan"), device="cuda") if lse else None
    plan.run(q, k, kr, v, sm, out, l)
    assert plan.check() == 0
    return out, l


def _check_attention(out, lse, ref, ref_lse, mag, what=""):
    _within(_f64(out), ref, _attention_bound(ref, mag), "out " + what)
    if lse is not None:
        l = lse.cpu().numpy()
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(l), empty), "rows without keys " + what
        assert (_f64(out)[empty] == 0).all()
        assert np.abs(l[~empty] - ref_lse[~empty]).max(initial=0) <= LSE_ATOL, "lse " + what


ATTENTION = [
    ([1], [1], 1, True), ([1], [1], 16, False), ([2], [1], 3, True), ([5], [0], 2, True), ([0, 3], [7, 0], 2, False),
    ([1, 7, 33, 100], [1, 7, 33, 100], 16, True),
    ([127, 128, 129], [127, 128, 129], 2, True), ([255, 256, 257], [255, 256, 257], 2, True),
    ([64], [64 + 127], 5, True), ([130], [600], 3, True), ([300], [100], 2, True), ([0, 200, 0, 1], [50, 77, 0, 300], 3, True),
    ([513], [513], 2, True), ([100, 300], [260, 31], 4, False), ([1, 1, 1], [128, 129, 127], 7, True),
    ([385], [1000], 2, True), ([17], [900], 1, False),
]


@pytest.mark.parametrize("ql,kl,H,causal", ATTENTION)
def test_prefill(ql, kl, H, causal):
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(sum(ql) + H, int(qp[-1]), int(kp[-1]), H)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    out, lse = _attend(B.Prefiller(qp, kp, H, causal), q, k, kr, v)
    _check_attention(out, lse, ref, ref_lse, mag)
    again, none = _attend(B.Prefiller(qp, kp, H, causal), q, k, kr, v, lse=False)
    assert none is None and torch.equal(again, out)             # no order of atomics, and lse is optional


@pytest.mark.parametrize("ql,kl,H,causal", MANY)
def test_prefill_of_more_items_than_sms(ql, kl, H, causal):
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(11 + H, int(qp[-1]), int(kp[-1]), H)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    plan = B.Prefiller(qp, kp, H, causal)
    out, lse = _attend(plan, q, k, kr, v)
    _check_attention(out, lse, ref, ref_lse, mag)
    # one call behind the other, without a wait between them
    outs = [torch.empty_like(out) for _ in range(6)]
    for o in outs:
        plan.run(q, k, kr, v, SM, o)
    assert plan.check() == 0
    assert all(torch.equal(o, out) for o in outs)


@pytest.mark.parametrize("group,tail", [(64, 0), (7, 0), (1, 3), (7, 5), (64, 2), (20, -1)])
def test_prefill_in_any_order_of_items(group, tail):
    # groups of heads (the last one smaller) and items kept for the end change the order alone
    torch, B = _t()
    qp = _indptr([1, 7, 33, 100, 140, 260, 300, 0, 129, 600])
    H = 64
    (q, _), (k, _), (kr, _), (v, _) = _attention_inputs(77, int(qp[-1]), int(qp[-1]), H)
    plan = B.Prefiller(qp, qp, H)
    want, want_lse = _attend(plan, q, k, kr, v)
    plan.plan_host[10], plan.plan_host[15] = group, int(plan.plan_host[7]) if tail < 0 else tail
    plan.plan_dev = torch.from_numpy(plan.plan_host).cuda()
    out, lse = _attend(plan, q, k, kr, v)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def _on_pairs(plan, qp, kp, H, causal):
    """The same batch in items of 512 rows, which pairs of CTAs work on (a plan takes them where it expects that
    schedule to end first)."""
    torch, _ = _t()
    items = []
    for b in range(len(qp) - 1):
        lq, lk = int(qp[b + 1] - qp[b]), int(kp[b + 1] - kp[b])
        for r in range(0, lq, 512):
            nq, off = min(512, lq - r), r + lk - lq if causal else 0x3FFFFFFF
            items.append([b, int(qp[b]) + r, nq, int(kp[b]), min(lk, max(0, off + nq)), off, -1, 0])
    items.sort(key=lambda i: -i[4])
    words = plan.plan_host[:16].tolist()
    words[7:12] = [len(items), 0, 0, H, 16 + 8 * len(items)]
    words[13], words[15] = 512, 0
    plan.plan_host = np.array(words + sum(items, []), dtype=np.int32)
    plan.plan_dev = torch.from_numpy(plan.plan_host).cuda()
    return plan


PAIRS = [
    ([512], [512], 2, True), ([513], [513], 2, True), ([1030], [1100], 3, True), ([700, 300], [900, 300], 2, True),
    ([600], [50], 1, True), ([520, 5, 0, 511], [520, 700, 9, 1000], 3, False),
    ([300, 600, 1000, 40], [300, 900, 1000, 40], 24, True), ([1], [4000], 1, True), ([260], [129], 2, True),
    ([1, 7, 33, 100, 140, 260, 300, 0, 129], [1, 7, 33, 100, 140, 260, 300, 9, 129], 33, True),
]


@pytest.mark.parametrize("ql,kl,H,causal", PAIRS)
def test_prefill_on_cta_pairs(ql, kl, H, causal):
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    plan = _on_pairs(B.Prefiller(qp, kp, H, causal), qp, kp, H, causal)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(31 + H, int(qp[-1]), int(kp[-1]), H)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    out, lse = _attend(plan, q, k, kr, v)
    _check_attention(out, lse, ref, ref_lse, mag)
    outs = [torch.empty_like(out) for _ in range(6)]
    for o in outs:
        plan.run(q, k, kr, v, SM, o)
    assert plan.check() == 0
    assert all(torch.equal(o, out) for o in outs)


@pytest.mark.parametrize("ql,kl,H,causal", [([3], [4000], 1, True), ([64, 1], [3500, 700], 2, True),
                                            ([300], [4000], 1, False), ([200], [3300], 2, True)])
def test_prefill_cut_along_the_keys(ql, kl, H, causal):
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(77 + H, int(qp[-1]), int(kp[-1]), H)
    plan = B.Prefiller(qp, kp, H, causal)
    assert plan.plan_host[8] > 1                                # partial outputs
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    out, lse = _attend(plan, q, k, kr, v)
    _check_attention(out, lse, ref, ref_lse, mag, "cut")
    whole, _ = _attend(B.Prefiller(qp, kp, H, causal, num_sms=1), q, k, kr, v)
    _check_attention(whole, None, ref, ref_lse, mag, "whole")


def _cut(plan, qp, kp, H, causal, rows, parts):
    """The same batch in items of `rows` rows whose keys are cut into up to `parts` pieces of whole tiles."""
    torch, _ = _t()
    items, joins, slot = [], [], 0
    for b in range(len(qp) - 1):
        lq, lk = int(qp[b + 1] - qp[b]), int(kp[b + 1] - kp[b])
        for r in range(0, lq, rows):
            nq, off = min(rows, lq - r), r + lk - lq if causal else 0x3FFFFFFF
            seen = min(lk, max(0, off + nq))
            tiles = (seen + 127) // 128
            n = max(1, min(parts, tiles))
            for k in range(n):
                a, e = 128 * (tiles * k // n), 128 * (tiles * (k + 1) // n)
                items.append([b, int(qp[b]) + r, nq, int(kp[b]) + a, min(seen, e) - a, off - a if causal else off,
                              slot + k if n > 1 else -1, 0])
            if n > 1:
                joins.append([int(qp[b]) + r, nq, slot, slot + n])
                slot += n
    words = plan.plan_host[:16].tolist()
    words[7:12] = [len(items), slot, len(joins), H, 16 + 8 * len(items) + 4 * len(joins)]
    words[13:16] = [rows, int(all(i[2] <= 128 for i in items) and rows == 256), 0]
    plan.plan_host = np.array(words + sum(items, []) + sum(joins, []), dtype=np.int32)
    plan.plan_dev = torch.from_numpy(plan.plan_host).cuda()
    plan.workspace = torch.zeros(256 + slot * H * rows * 129 * 4, dtype=torch.uint8, device="cuda")
    return plan


CUT = [
    # rows of an item, pieces: one row tile, two, and pairs, whose items have up to 512 rows
    ([100, 128, 1, 17], [700, 1290, 900, 60], 2, 256, 4), ([256, 129, 300], [900, 1500, 130], 2, 256, 3),
    ([512], [1700], 1, 512, 5), ([1100, 300], [1500, 2000], 2, 512, 4), ([513, 290], [513, 100], 2, 512, 9),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,H,rows,parts", CUT)
def test_prefill_cut_along_the_keys_in_every_form(ql, kl, H, rows, parts, causal):
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    plan = _cut(B.Prefiller(qp, kp, H, causal), qp, kp, H, causal, rows, parts)
    assert plan.plan_host[8] > 1 and plan.plan_host[13] == rows
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(61 + H, int(qp[-1]), int(kp[-1]), H)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    out, lse = _attend(plan, q, k, kr, v)
    _check_attention(out, lse, ref, ref_lse, mag)
    outs = [torch.empty_like(out) for _ in range(3)]
    for o in outs:
        plan.run(q, k, kr, v, SM, o)
    assert plan.check() == 0
    assert all(torch.equal(o, out) for o in outs)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,H,rows,parts", CUT)
def test_prefill_cut_items_keep_what_is_masked_out(ql, kl, H, rows, parts, causal, bad):
    # values that are not finite in partly seen tiles of a cut item reach the rows that see them, through the join
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    plan = _cut(B.Prefiller(qp, kp, H, causal), qp, kp, H, causal, rows, parts)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(71 + H, int(qp[-1]), int(kp[-1]), H)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    sees = np.zeros(ref.shape, dtype=bool)
    for b, back in zip(range(len(ql)), (5, 60, 1, 33)):
        key = kl[b] - min(back, kl[b])
        v[int(kp[b]) + key, H - 1, 17 + b] = bad
        last = np.arange(ql[b]) + (kl[b] - ql[b] if causal else kl[b])
        sees[int(qp[b]):int(qp[b + 1]), H - 1, 17 + b] = last >= key
    out, lse = _attend(plan, q, k, kr, v)
    o = _f64(out)
    assert sees.any() and np.array_equal(o[sees], np.full(int(sees.sum()), bad), equal_nan=True)
    assert np.isfinite(o[~sees]).all()
    assert (np.abs(o - ref)[~sees] <= _attention_bound(ref, mag)[~sees]).all()
    l = lse.cpu().numpy()
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(l), empty) and np.abs(l[~empty] - ref_lse[~empty]).max() <= LSE_ATOL


@pytest.mark.parametrize("n,keys,H", [(400, 4096, 16), (1024, 4096, 8), (300, 2048, 32), (512, 16384, 32)])
def test_prefill_of_a_chunk_that_continues_a_long_context(n, keys, H):
    # items of 512 rows on CTA pairs whose keys the plan cuts; some rows of each row tile against the oracle
    torch, B = _t()
    qp, kp = _indptr([n]), _indptr([keys])
    plan = B.Prefiller(qp, kp, H, num_sms=152)
    assert plan.plan_host[13] == 512 and plan.plan_host[8] > 1
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(81, n, keys, H)
    out, lse = _attend(plan, q, k, kr, v)
    o, l = _f64(out), lse.cpu().numpy()
    for i in sorted({0, 1, 127, 128, 200, 255, 256, 260, n - 130, n - 2, n - 1}):
        seen = keys - n + i + 1
        ref, ref_lse, mag = P.prefill_attention(xq[i:i + 1], xk[:seen], xr[:seen], xv[:seen], [0, 1], [0, seen], SM)
        _within(o[i:i + 1], ref, _attention_bound(ref, mag), f"row {i}")
        # the sum of so many weights in fp32: four partial sums a tile and pieces of at most 2^14 keys
        assert np.abs(l[i:i + 1] - ref_lse).max() <= LSE_ATOL + keys * 2.0 ** -24
    assert np.isfinite(o).all()


@pytest.mark.parametrize("scale", [8.0, 60.0])
def test_prefill_of_peaked_scores(scale):
    # large scores: the running maximum moves a lot, and most weights vanish; a key that grows along the
    # sequence makes every tile raise the maximum
    torch, B = _t()
    n, H = 700, 2
    (q, xq), (k, _), (kr, xr), (v, xv) = _attention_inputs(5, n, n, H)
    k = (k.float() * torch.linspace(0.1, scale, n, device="cuda")[:, None, None]).to(torch.bfloat16)
    qp = _indptr([n])
    ref, ref_lse, mag = P.prefill_attention(xq, _f64(k), xr, xv, qp, qp, SM, True)
    out, lse = _attend(B.Prefiller(qp, qp, H), q, k, kr, v)
    # a score's fp32 error grows with the scores: 192 products of |q||k| up to 4 * 4 * scale, 2^-22 each,
    # times sm_scale, under 2^-12 * scale / 2; a weight's relative error is twice that
    off = 2.0 ** -13 * scale
    _within(_f64(out), ref, _attention_bound(ref, mag) + 2 * off * mag, "out")
    assert np.abs(lse.cpu().numpy() - ref_lse).max() <= LSE_ATOL + off


@pytest.mark.parametrize("sm", [-SM, 0.0, -0.5, 1e-20])
def test_prefill_of_any_scale(sm):
    # a negative scale turns the order of the scores around; zero weighs every key alike
    torch, B = _t()
    qp, kp = _indptr([150]), _indptr([200])
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(6, 150, 200, 2)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, sm)
    out, lse = _attend(B.Prefiller(qp, kp, 2), q, k, kr, v, sm=sm)
    # 192 products at |sm| up to 0.5: at most 7 times the score error of SM's
    _within(_f64(out), ref, _attention_bound(ref, mag) + 2.0 ** -8 * mag, "out")
    assert np.abs(lse.cpu().numpy() - ref_lse).max() <= 4 * LSE_ATOL


@pytest.mark.parametrize("sm", [0.0, -0.0, 1e-38, 3e-36, -3e-36])
def test_prefill_of_scales_near_zero(sm):
    # scores of up to 1e37 before the scale: zero weighs every key alike, and a tiny scale is not another one
    torch, B = _t()
    qp, kp = _indptr([150]), _indptr([200])
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(6, 150, 200, 2)
    q, k, kr = q * 2.0 ** 59, k * 2.0 ** 59, kr * 2.0 ** 59      # exact: 2^118 is 3e35
    f = 2.0 ** 59
    ref, ref_lse, mag = P.prefill_attention(xq * f, xk * f, xr * f, xv, qp, kp, float(np.float32(sm)))
    out, lse = _attend(B.Prefiller(qp, kp, 2), q, k, kr, v, sm=sm)
    # scaled scores of at most 60: 192 products to 2^-22 of the sum of their magnitudes (under 200 * sm * 2^118), the
    # scale itself to 2^-24 (a subnormal one: its last bit, 2^-149, times 2^118 * 60)
    off = 200 * abs(sm) * 2.0 ** 118 * 2.0 ** -21 + 2.0 ** -24
    _within(_f64(out), ref, _attention_bound(ref, mag) + 2 * off * mag, "out")
    assert np.abs(lse.cpu().numpy() - ref_lse).max() <= LSE_ATOL + off


def test_prefill_strides():
    # q out of a wider projection; keys and values as the halves of one [T, H, 256] projection; heads outermost
    torch, B = _t()
    ql, kl, H = [70, 140], [200, 140], 3
    qp, kp = _indptr(ql), _indptr(kl)
    nq, nk = int(qp[-1]), int(kp[-1])
    wide, xw = _normal(1, nq, H * 192 + 16)
    q, xq = wide[:, 16:].view(nq, H, 192), xw[:, 16:].reshape(nq, H, 192)
    kv, xkv = _normal(2, nk, H, 256)
    row, xrow = _normal(3, nk, 576)
    ref, ref_lse, mag = P.prefill_attention(xq, xkv[..., :128], xrow[:, 512:], xkv[..., 128:], qp, kp, SM, True)
    plan = B.Prefiller(qp, kp, H)
    out, lse = _attend(plan, q, kv[..., :128], row[:, 512:], kv[..., 128:])
    _check_attention(out, lse, ref, ref_lse, mag, "projection")
    heads_first = kv.transpose(0, 1).contiguous().transpose(0, 1)
    out2, _ = _attend(plan, q.transpose(0, 1).contiguous().transpose(0, 1), heads_first[..., :128], row[:, 512:],
                      heads_first[..., 128:])
    assert torch.equal(out2, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("pairs", [False, True])
def test_prefill_keeps_what_is_masked_out(bad, causal, pairs):
    # keys and values that are not finite reach the rows that see them, and no other: neither the rows before
    # them (causal) nor another request's
    torch, B = _t()
    ql, kl, H = [40, 200, 30], [40, 330, 30], 2
    qp, kp = _indptr(ql), _indptr(kl)
    plan = B.Prefiller(qp, kp, H, causal)
    if pairs:
        plan = _on_pairs(plan, qp, kp, H, causal)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(9, int(qp[-1]), int(kp[-1]), H)
    at = int(kp[1]) + 330 - 60                                   # a key of the second request, and a value before it
    v[at - 9, 1, 17] = bad
    k[at, 0, 3] = bad
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    out, lse = _attend(plan, q, k, kr, v)
    o, l = _f64(out), lse.double().cpu().numpy()
    sees_v = np.zeros(o.shape, dtype=bool)
    sees_k = np.zeros(o.shape[:2], dtype=bool)
    last = np.arange(200) + 330 - 200                            # the last key of each row of the second request
    rows = np.arange(40, 240)
    sees_v[rows[(last >= 270 - 9) if causal else slice(None)], 1, 17] = True
    sees_k[rows[(last >= 270) if causal else slice(None)], 0] = True
    free = ~sees_v & ~sees_k[..., None]
    assert np.isfinite(o[free]).all()
    err = np.abs(o - ref) - _attention_bound(ref, mag)
    assert (err[free] <= 0).all()
    assert np.abs(l - ref_lse)[~sees_k].max() <= LSE_ATOL
    # the value itself passes on (a weight is never zero at these scores)
    want = np.full(int(sees_v.sum()), bad)
    assert np.array_equal(o[sees_v], want, equal_nan=True)
    # the score is bad (NaN) or +-inf with the query's sign; +inf takes all the weight or makes a NaN, -inf none
    if math.isnan(bad):
        assert np.isnan(o[sees_k]).all() and np.isnan(l[sees_k]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("ql,kl,pairs", [([40], [200], False), ([200], [330], False), ([600], [800], True)])
def test_prefill_rows_without_a_score_above_minus_infinity(ql, kl, pairs, bad):
    # such a row has no weights: whatever the values are, in tiles that all rows see whole and in partly seen ones,
    # its output is zero
    torch, B = _t()
    qp, kp, H = _indptr(ql), _indptr(kl), 2
    plan = B.Prefiller(qp, kp, H)
    if pairs:
        plan = _on_pairs(plan, qp, kp, H, True)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(15, ql[0], kl[0], H)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM)
    none = [ql[0] // 2, ql[0] - 3, ql[0] - 1]
    k[:, 0, 5] = -k[:, 0, 5].abs() - 0.5
    q[none, 0, 5] = float("inf")
    v[[3, kl[0] - 2, kl[0] - 30], 0, 9] = bad
    out, lse = _attend(plan, q, k, kr, v)
    assert (out[none, 0] == 0).all()
    assert torch.isneginf(lse[none, 0]).all()
    _check_attention(out[:, 1:], lse[:, 1:], ref[:, 1:], ref_lse[:, 1:], mag[:, 1:])


@pytest.mark.parametrize("at", [10, 330 - 4])
@pytest.mark.parametrize("pairs", [False, True])
def test_prefill_values_that_are_not_finite_under_a_vanished_weight(pairs, at):
    # a score some 400 below the others: its weight is zero in fp32, but the value it weighs is not finite, and so is
    # the sum, in a tile that every row sees whole and in a partly seen one
    torch, B = _t()
    qp, kp = _indptr([200]), _indptr([330])
    plan = B.Prefiller(qp, kp, 1)
    if pairs:
        plan = _on_pairs(plan, qp, kp, 1, True)
    q = torch.full((200, 1, 192), 4.0, dtype=torch.bfloat16, device="cuda")
    k = torch.full((330, 1, 128), 4.0, dtype=torch.bfloat16, device="cuda")
    kr = torch.zeros((330, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.ones((330, 1, 128), dtype=torch.bfloat16, device="cuda")
    k[at] = -8.0
    v[at, 0, 7] = float("inf")
    out, lse = _attend(plan, q, k, kr, v)
    sees = torch.arange(200, device="cuda") + 130 >= at
    assert not torch.isfinite(out[sees, 0, 7]).any()
    assert torch.isfinite(out[~sees]).all()
    rest = [c for c in range(128) if c != 7]
    assert (out[:, 0, rest] == 1).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("ql,kl,H,causal", [
    ([64] * 4, [4000, 3000, 3500, 4096], 48, True),              # several items a block, of many key tiles
    ([128, 1, 17, 100] * 9, [700, 1290, 5, 2000] * 9, 12, True),
    ([128] * 5 + [3] * 60, [128] * 5 + [400] * 60, 8, False),
    ([100] * 3, [0, 30, 3100], 70, True),
])
def test_prefill_of_one_row_tile(ql, kl, H, causal):
    # at most 128 rows a request
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(41 + H, int(qp[-1]), int(kp[-1]), H)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, causal)
    plan = B.Prefiller(qp, kp, H, causal)
    out, lse = _attend(plan, q, k, kr, v)
    _check_attention(out, lse, ref, ref_lse, mag)
    outs = [torch.empty_like(out) for _ in range(6)]
    for o in outs:
        plan.run(q, k, kr, v, SM, o)
    assert plan.check() == 0
    assert all(torch.equal(o, out) for o in outs)


@pytest.mark.parametrize("pairs", [False, True])
def test_prefill_keeps_its_notes_until_they_are_read(pairs):
    # values that are not finite in partly seen tiles, of items with two row tiles, and behind each of those items
    # several with one row tile, which the block goes on to while the second row tile's output is still written
    torch, B = _t()
    L = 512 if pairs else 256
    big, small = 152 if not pairs else 76, 900
    ql = [L] * big + [64] * small
    qp = kp = _indptr(ql)
    plan = B.Prefiller(qp, kp, 1)
    if pairs:
        plan = _on_pairs(plan, qp, kp, 1, True)
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(21, int(qp[-1]), int(kp[-1]), 1)
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM, True)
    first = L - 126                                              # the first of the keys with a bad value
    sees = np.zeros(ref.shape, dtype=bool)
    for b in range(big):
        v[int(kp[b]) + first:int(kp[b]) + L, 0, 5] = float("inf")
        sees[int(qp[b]) + first:int(qp[b]) + L, 0, 5] = True
    out, lse = _attend(plan, q, k, kr, v)
    o = _f64(out)
    assert (o[sees] == np.inf).all()
    assert np.isfinite(o[~sees]).all()
    assert (np.abs(o - ref)[~sees] <= _attention_bound(ref, mag)[~sees]).all()
    assert np.abs(lse.double().cpu().numpy() - ref_lse).max() <= LSE_ATOL


def test_prefill_leaves_rows_behind_the_last_sequence():
    torch, B = _t()
    qp = kp = _indptr([100, 60])
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(3, 160, 160, 2)
    out = torch.full((200, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((200, 2), float("nan"), device="cuda")
    # the arrays go on behind the batch, with anything in them
    tail = lambda t: torch.cat([t, torch.full((40,) + t.shape[1:], float("nan"), dtype=t.dtype, device="cuda")])  # noqa: E731
    plan = B.Prefiller(qp, kp, 2)
    plan.run(tail(q)[:160], tail(k)[:160], tail(kr)[:160], tail(v)[:160], SM, out[:160], lse[:160])
    assert plan.check() == 0
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, kp, SM)
    _check_attention(out[:160], lse[:160], ref, ref_lse, mag)
    assert torch.isnan(out[160:]).all() and torch.isnan(lse[160:]).all()


def test_prefill_keys_past_2_gib_elements():
    # a head's values more than 2^31 elements into the array, by the head stride
    torch, B = _t()
    n, H = 130, 2
    (q, xq), (k, xk), (kr, xr), (v, xv) = _attention_inputs(4, n, n, H)
    far = torch.empty(2 ** 31 + n * 128 + 8, dtype=torch.bfloat16, device="cuda")
    kf = far.as_strided((n, H, 128), (128, 2 ** 31 + 8, 1))
    kf.copy_(k)
    qp = _indptr([n])
    ref, ref_lse, mag = P.prefill_attention(xq, xk, xr, xv, qp, qp, SM)
    out, lse = _attend(B.Prefiller(qp, qp, H), q, kf, kr, v)
    _check_attention(out, lse, ref, ref_lse, mag)


def test_prefill_bad_device_plan_is_reported_not_followed():
    torch, B = _t()
    qp = _indptr([100])
    (q, _), (k, _), (kr, _), (v, _) = _attention_inputs(4, 100, 100, 2)
    for word, value in ((1, 60), (1, -5), (2, 0), (2, 257), (3, -1), (3, 50), (4, 101), (4, -1), (6, 0), (6, -2), (5, 2 ** 31 - 1)):
        plan = B.Prefiller(qp, qp, 2)
        plan.plan_dev[16 + word] = value
        out = torch.full((100, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        plan.run(q, k, kr, v, SM, out)
        assert plan.check() == 7, (word, value)
        assert (out == 7).all(), (word, value)


def test_prefill_bad_device_join_is_reported_not_followed():
    # the entry of a cut tile's join: first row, rows, first piece, one past the last
    torch, B = _t()
    qp, kp = _indptr([100]), _indptr([1500])
    (q, _), (k, _), (kr, _), (v, _) = _attention_inputs(4, 100, 1500, 2)
    for word, value in ((0, -1), (0, 1), (1, 0), (1, 257), (2, -1), (2, 4), (3, 5), (3, 0)):
        plan = _cut(B.Prefiller(qp, kp, 2), qp, kp, 2, True, 256, 4)
        plan.plan_dev[16 + 8 * 4 + word] = value
        out = torch.full((100, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        plan.run(q, k, kr, v, SM, out)
        assert plan.check() == 7, (word, value)
        assert (out == 7).all(), (word, value)


@pytest.mark.parametrize("ql,kl,H,pairs", [([3, 100, 200], [3, 100, 200], 80, False), ([5], [40], 2, False),
                                           ([600, 100], [600, 100], 60, True), ([64] * 4, [300] * 4, 60, False)])
@pytest.mark.parametrize("word,value", [(16, 5), (16, 1 << 20), (16, -3), (16, 2 ** 31 - 1), (17, -1), (17, 1 << 30),
                                        (17, 3), (18, 9)])
def test_prefill_reports_a_workspace_whose_counters_are_not_zero(ql, kl, H, pairs, word, value):
    # items handed out, blocks that have finished, items worked on: wrong output is never without a status
    torch, B = _t()
    qp, kp = _indptr(ql), _indptr(kl)
    plan = B.Prefiller(qp, kp, H)
    if pairs:
        plan = _on_pairs(plan, qp, kp, H, True)
    (q, _), (k, _), (kr, _), (v, _) = _attention_inputs(19, int(qp[-1]), int(kp[-1]), H)
    want, want_lse = _attend(plan, q, k, kr, v)
    words = plan.workspace[:256].view(torch.int32)
    assert not words.any()
    words[word] = value
    out = torch.zeros_like(want)
    plan.run(q, k, kr, v, SM, out)
    status = plan.check()
    # every item is some block's first where there are so few, and a few blocks too many leave none out
    harmless = word == 16 and H == 2 or word == 17 and value == 3
    assert status in ((0, 3) if harmless else (3,))
    if harmless:
        assert torch.equal(out, want)
    words.zero_()
    again, lse = _attend(plan, q, k, kr, v)                     # (its status is checked there)
    assert torch.equal(again, want) and torch.equal(lse, want_lse)
    assert not words.any()


def test_prefill_on_another_stream_and_replayed():
    torch, B = _t()
    ql, kl, H = [3, 150], [4000, 300], 2
    qp, kp = _indptr(ql), _indptr(kl)
    plan = B.Prefiller(qp, kp, H)
    bufs = [x.clone() for x, _ in _attention_inputs(1, 153, 4300, H)]
    out = torch.empty((153, H, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((153, H), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.run(*bufs, SM, out, lse, stream=side)                  # named, without being current
    torch.cuda.current_stream().wait_stream(side)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(*bufs, SM, out, lse)
    for seed in (1, 2):
        new = _attention_inputs(seed, 153, 4300, H)
        for dst, (src, _) in zip(bufs, new):
            dst.copy_(src)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, ref_lse, mag = P.prefill_attention(*[x for _, x in new], qp, kp, SM)
        _check_attention(out, lse, ref, ref_lse, mag, f"replay {seed}")
        if seed == 1:
            assert torch.equal(out, first)
    assert plan.check() == 0


def test_prefiller_is_ready_on_every_stream():
    # made while its own stream is busy, in memory that held something else, and run on another stream at once
    torch, B = _t()
    qp, kp = _indptr([300] * 4), _indptr([300] * 4)
    H = 60
    (q, _), (k, _), (kr, _), (v, _) = _attention_inputs(23, 1200, 1200, H)
    want, _ = _attend(B.Prefiller(qp, kp, H), q, k, kr, v)
    out, side = torch.zeros_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.full((256,), 77, dtype=torch.uint8, device="cuda")    # (the allocator gives this block out again)
    torch.cuda._sleep(100_000_000)
    plan = B.Prefiller(qp, kp, H)
    plan.run(q, k, kr, v, SM, out, stream=side)
    side.synchronize()
    assert plan.check() == 0 and torch.equal(out, want)


def test_prefiller_dropped_before_its_work_is_done():
    # its plan and workspace stay its own until the stream that runs it has finished
    torch, B = _t()
    qp, kp = _indptr([3]), _indptr([4000])
    (q, _), (k, _), (kr, _), (v, _) = _attention_inputs(24, 3, 4000, 2)
    want, _ = _attend(B.Prefiller(qp, kp, 2), q, k, kr, v)
    out, side = torch.zeros_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = B.Prefiller(qp, kp, 2)
    held = {t.data_ptr(): t.numel() * t.element_size() for t in (plan.plan_dev, plan.workspace)}
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    plan.run(q, k, kr, v, SM, out, stream=side)
    del plan
    new = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in held.values()]
    assert not held.keys() & {t.data_ptr() for t in new}
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("how", ["handle", "given", "current"])
def test_prefiller_outlives_a_stream_made_elsewhere(how):
    # such a stream may be destroyed once its work is done: nothing is recorded on it when the memory is given back
    import ctypes
    torch, B = _t()
    qp, kp = _indptr([3]), _indptr([4000])
    (q, _), (k, _), (kr, _), (v, _) = _attention_inputs(24, 3, 4000, 2)
    want, _ = _attend(B.Prefiller(qp, kp, 2), q, k, kr, v)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    raw = ctypes.c_void_p()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(raw))) == 0
    plan = B.Prefiller(qp, kp, 2)
    other = torch.cuda.ExternalStream(raw.value)
    if how == "current":
        with torch.cuda.stream(other):
            plan.run(q, k, kr, v, SM, out)
    else:
        plan.run(q, k, kr, v, SM, out, stream=raw.value if how == "handle" else other)
    other.synchronize()
    assert torch.equal(out, want)
    assert int(torch.cuda.cudart().cudaStreamDestroy(raw.value)) == 0
    del plan
    assert B.Prefiller(qp, kp, 2).check() == 0
    torch.cuda.synchronize()


def test_two_prefills_at_once_with_their_own_workspaces():
    torch, B = _t()
    qp, kp = _indptr([5]), _indptr([4000])
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for i in range(2):
        ins = _attention_inputs(20 + i, 5, 4000, 2)
        runs.append((B.Prefiller(qp, kp, 2), ins, torch.empty((5, 2, 128), dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (plan, ins, out) in zip(streams, runs):
            plan.run(*[x for x, _ in ins], SM, out, stream=s)
    torch.cuda.synchronize()
    for plan, ins, out in runs:
        ref, ref_lse, mag = P.prefill_attention(*[x for _, x in ins], qp, kp, SM)
        assert plan.check() == 0
        _check_attention(out, None, ref, ref_lse, mag)


def test_strides_of_a_dimension_of_one_are_not_looked_at():
    # one token cut out of an array whose rows are no multiple of 8 apart, one head likewise
    torch, B = _t()
    fr, pos = B.rope_frequencies(), torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    rows = _normal(1, 1, 579)[0][:, :576]
    assert rows.stride(0) == 579
    cache = torch.zeros((4, 576), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((4, 576), dtype=torch.uint8, device="cuda")
    B.rope_append_kv(cache, slot, rows, pos, fr)
    B.rope_append_kv_fp8(codes, slot, rows, pos, fr, 1.0)
    assert torch.equal(cache[2], rows[0])
    assert torch.equal(codes[2].view(torch.float8_e4m3fn).float(), rows[0].to(torch.float8_e4m3fn).float())
    # a token stride, then a head stride, that nothing steps by
    x = _normal(2, 1, 3 * 192)[0]
    q = x.as_strided((1, 3, 192), (577, 192, 1))
    one = x.as_strided((3, 1, 192), (192, 193, 1))
    for t in (q, one):
        out = torch.empty(192, dtype=torch.bfloat16, device="cuda")
        out = out.as_strided(t[..., 128:].shape, tuple(67 if n == 1 else 64 for n in t.shape[:2]) + (1,))
        B.rope_query(t, torch.zeros(t.shape[0], dtype=torch.int32, device="cuda"), fr, out)
        assert torch.equal(out.contiguous(), t[..., 128:].contiguous())
    qp = _indptr([1])
    (a, xa), (k, xk), (kr, xr), (v, xv) = _attention_inputs(4, 1, 1, 1)
    ref, ref_lse, mag = P.prefill_attention(xa, xk, xr, xv, qp, qp, SM)
    off = lambda t: t.as_strided(t.shape, tuple(s + 1 if n == 1 else s for n, s in zip(t.shape, t.stride())))  # noqa: E731
    out, lse = _attend(B.Prefiller(qp, qp, 1), off(a), off(k), off(kr), off(v))
    _check_attention(out, lse, ref, ref_lse, mag)


# ---------------------------------------------------------------- as they run together

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,interleaved", [(16, True), (64, False)])
def test_prompt_then_decode_step(fp8, H, interleaved):
    # a prompt's rows go into the cache (norm, rotation), come back expanded, and its queries attend to them;
    # then the next token is decoded in the absorbed form over the same cache.  Every stage against the oracle
    # on what the stage before left; the prompt's last row, attended in both forms, closes the circle.
    torch, B = _t()
    lengths = [1, 90, 260]
    nb, T, N = len(lengths), sum(lengths), 600
    ptr = _indptr(lengths)
    rng = np.random.default_rng(H)
    fr, inv = B.rope_frequencies(**YARN), _inv(YARN)
    rows, xrows = _normal(1, T, 576)
    q, xq = _normal(2, T, H, 192)
    w, xw = _normal(3, 512)
    wk, xk = _normal(4, H, 128, 512, scale=512 ** -0.5)
    wv, xv = _normal(5, H, 512, 128, scale=512 ** -0.5)
    slots = torch.from_numpy(rng.permutation(N)[:T].astype(np.int32)).cuda()
    pos = np.concatenate([np.arange(n) for n in lengths]).astype(np.int32)
    dpos = torch.from_numpy(pos).cuda()
    cache = torch.zeros((N, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    k, kr, v, out, lse = bf(T, H, 128), bf(T, 64), bf(T, H, 128), bf(T, H, 128), torch.empty((T, H), device="cuda")
    scale = 2.0 ** -5
    plan = B.Prefiller(ptr, ptr, H)
    turned = q.clone()

    def prompt():
        if fp8:
            B.rope_append_kv_fp8(cache, slots, rows, dpos, fr, scale, norm_weight=w, interleaved=interleaved, workspace=ws)
            B.expand_kv_fp8(cache, scale, slots, wk, wv, k, kr, v, workspace=ws)
        else:
            B.rope_append_kv(cache, slots, rows, dpos, fr, norm_weight=w, interleaved=interleaved, workspace=ws)
            B.expand_kv(cache, slots, wk, wv, k, kr, v, workspace=ws)
        B.rope_query(q, dpos, fr, turned[..., 128:], interleaved=interleaved)
        plan.run(turned, k, kr, v, SM, out, lse)

    prompt()
    assert B.check_errors(ws) == 0 and plan.check() == 0
    stored = cache[slots.long()]
    x = _f64(stored.view(torch.float8_e4m3fn)) * scale if fp8 else _f64(stored)
    val = P.append_values(xrows, pos, inv, xw, 1e-6, interleaved)
    step = np.maximum(2.0 ** -4 * np.abs(val), 2.0 ** -10 * scale) if fp8 else BF * np.abs(val)
    _within(x, val, step + 2.0 ** -17 * (np.abs(val) + np.abs(xrows).max()), "cache")
    rk, rv = P.expand_rows(x[:, :512], xk, xv)
    _within(_f64(k), rk, _expand_bound(rk, x[:, :512], xk, "tr,hnr->thn"), "k")
    _within(_f64(v), rv, _expand_bound(rv, x[:, :512], xv, "tr,hrn->thn"), "v")
    rq = P.rope_rotate(xq[..., 128:], pos, inv, interleaved)
    _within(_f64(turned[..., 128:]), rq, _rope_bound(rq, xq[..., 128:]), "query")
    ref, ref_lse, mag = P.prefill_attention(_f64(turned), _f64(k), _f64(kr), _f64(v), ptr, ptr, SM)
    _check_attention(out, lse, ref, ref_lse, mag, "prompt")

    # the last token of each request once more, in the absorbed form, from the cache alone
    last = ptr[1:] - 1
    lt = torch.from_numpy(last).long().cuda()
    q_rope, q_pre, q_lat = bf(nb, H, 64), bf(nb, H, 128), bf(nb, H, 512)
    B.rope_query(q[lt], dpos[lt], fr, q_rope, q_nope=q_pre, interleaved=interleaved)
    assert torch.equal(q_rope, turned[lt][..., 128:]) and torch.equal(q_pre, q[lt][..., :128])
    B.absorb_query(q_pre, wk, q_lat)
    o_lat, dlse, dout = bf(nb, H, 512), torch.empty((nb, H), device="cuda"), torch.empty((nb, H, 128), device="cuda")
    dec = B.Decoder(ptr, H)
    dptr = torch.from_numpy(ptr).cuda()
    if fp8:
        dws = torch.zeros(B.decode_fp8_workspace_bytes(dec.plan_host), dtype=torch.uint8, device="cuda")
        B.decode_run_fp8(dec.plan_host, dec.plan_dev, q_lat, q_rope, cache, scale, dptr, slots, SM, o_lat, dlse, dws)
        assert B.check_errors(dws) == 0
    else:
        dec.run(q_lat, q_rope, cache, dptr, slots, SM, o_lat, dlse)
        assert dec.check() == 0
    B.project_output(o_lat, wv, dout)
    # the two forms round at different places (keys and values, or query and latent output): the decode's own
    # bar on each side
    a, b = _f64(out[lt]), _f64(dout)
    assert (np.abs(a - b) <= 2e-2 + 2e-2 * np.abs(b)).all(), np.abs(a - b).max()
    assert (lse[lt] - dlse).abs().max() <= 1e-2

    # the whole prompt captured once and replayed on new rows gives what the calls give
    eager = [t.clone() for t in (cache, k, v, turned, out)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prompt()
    for t in (k, v, turned[..., 128:], out):
        t.zero_()
    cache.zero_()
    turned[..., :128] = q[..., :128]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache[slots.long()], eager[0][slots.long()])
    assert all(torch.equal(a, b) for a, b in zip((k, v, turned, out), eager[1:]))
