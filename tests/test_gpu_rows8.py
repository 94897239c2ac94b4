"""GPU tests of the FP8 cache with a scale for every row: append, expansion and
decode against 64-bit formulas, and as they run together.

Tolerances count roundings: half a step of bf16 is 2^-8 of the value, of E4M3
2^-4 (2^-10 below its smallest normal 2^-6); fp32 intermediates add what each
test states."""
import math

import numpy as np
import pytest

from oracle import prompt_oracle as P

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8
SM = 1.0 / math.sqrt(192.0)
LOW, HIGH = 2.0 ** -64, 2.0 ** 64


def _t():
    import torch
    from mla_latent_kv_absorbed_gb300 import binding
    return torch, binding


def _gen(seed):
    torch, _ = _t()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    torch, _ = _t()
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _cache(seed, slots, spread):
    """Codes of rows about N(0, 1) at a scale of 2^(+-spread) each."""
    torch, _ = _t()
    g = _gen(seed)
    x = _randn(g, slots, 576)
    top = x.abs().amax(1)
    codes = (x * (448 / top)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    u = torch.rand(slots, generator=g, device="cuda") * 2 - 1
    return codes, top / 448 * torch.exp2(u * spread)


def _rows64(codes, scales, at):
    torch, _ = _t()
    return codes[at].view(torch.float8_e4m3fn).double() * scales[at].double().clamp(LOW, HIGH)[:, None]


# ------------------------------------------------------------------------ append

@pytest.mark.parametrize("T,stride,norm,interleaved,kw", [
    (1, 576, True, True, {}), (4, 576, False, False, dict(scaling="yarn", factor=40.0)),
    (33, 584, True, False, dict(scaling="linear", factor=8.0)), (700, 2112, True, True, dict(scaling="yarn", factor=40.0)),
    (5000, 1344, False, True, {}),
])
def test_append(T, stride, norm, interleaved, kw):
    torch, B = _t()
    g = _gen(T)
    loud = torch.exp2(16 * torch.rand(T, generator=g, device="cuda") - 8)
    wide = (_randn(g, T, stride) * loud[:, None]).bfloat16()
    rows = wide[:, stride - 576:]
    w = (1 + 0.1 * _randn(g, 512)).bfloat16() if norm else None
    pos = torch.randint(0, 163840, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(T + 50, generator=g, device="cuda")[:T].to(torch.int32)
    codes, scales = _cache(T + 1, T + 50, 2.0)
    was_c, was_s = codes.clone(), scales.clone()
    B.rope_append_kv_fp8_rows(codes, scales, slots, rows, pos, B.rope_frequencies(**kw), norm_weight=w,
                              interleaved=interleaved)
    x = rows.double()
    lat = x[:, :512]
    if norm:
        lat = lat / ((lat * lat).mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    rope = P.rope_rotate(x[:, None, 512:].cpu().numpy(), pos.cpu().numpy(), P.rope_inv_freq(**kw), interleaved)[:, 0]
    ref = torch.cat((lat, torch.from_numpy(rope).cuda()), 1)
    at = slots.long()
    top = ref.abs().amax(1)
    # the scale: fp32 values off by 2^-20 of the pair's size (phase and rotation) or 2^-21 (norm), one rounding each
    # of the quotient
    assert ((scales[at].double() - top / 448).abs() <= top / 448 * 2.0 ** -19).all()
    got = _rows64(codes, scales, at)
    # a code is off by 2^-4 of itself, 2^-10 of a scale below 2^-6 of it; the values' own error is far below that,
    # but may turn a code at the border of two: 2^-18 of the row's largest beside them
    bound = ref.abs() * (2.0 ** -4 + 2.0 ** -18) + (top / 448 * (2.0 ** -10) + top * 2.0 ** -18)[:, None]
    assert ((got - ref).abs() <= bound).all()
    assert (codes[at].view(torch.float8_e4m3fn).float().abs().amax(1) == 448).all()       # the range is used
    rest = torch.ones(T + 50, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(codes[rest], was_c[rest]) and torch.equal(scales[rest], was_s[rest])


def test_append_of_extreme_rows():
    torch, B = _t()
    rows = torch.zeros((6, 576), dtype=torch.bfloat16, device="cuda")
    rows[1, 3] = 2.0 ** -100                    # below the smallest scale's smallest code: zero
    rows[2, 5] = 3e38                           # past the largest scale: saturates
    rows[3, 7], rows[3, 8] = float("inf"), 2.0
    rows[4, 9], rows[4, 10] = float("nan"), 448.0
    rows[5, 511] = -1.0
    codes = torch.full((8, 576), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((8,), 7.0, device="cuda")
    slots = torch.tensor([0, 1, 2, 3, 4, 6], dtype=torch.int32, device="cuda")
    B.rope_append_kv_fp8_rows(codes, scales, slots, rows, torch.zeros(6, dtype=torch.int32, device="cuda"),
                              B.rope_frequencies())
    v = codes.view(torch.float8_e4m3fn).float()
    assert scales.tolist()[:5] == [LOW, LOW, HIGH, HIGH, 1.0] and scales[5] == 7.0 and scales[7] == 7.0
    assert (v[0] == 0).all() and (v[1] == 0).all()
    assert v[2, 5] == 448 and v[3, 7] == 448 and v[3, 8] == 0
    assert torch.isnan(v[4, 9]) and v[4, 10] == 448
    assert v[6, 511] == -448 and scales[6] == np.float32(1 / 448)


def test_append_skips_and_records_a_bad_slot():
    torch, B = _t()
    g = _gen(3)
    rows = _randn(g, 3, 576).bfloat16()
    codes, scales = _cache(4, 5, 1.0)
    was_c, was_s = codes.clone(), scales.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.rope_append_kv_fp8_rows(codes, scales, torch.tensor([5, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), rows,
                              torch.arange(3, dtype=torch.int32, device="cuda"), B.rope_frequencies(), workspace=ws)
    assert B.check_errors(ws) == 6
    assert torch.equal(codes, was_c) and torch.equal(scales, was_s)


# --------------------------------------------------------------------- expansion

@pytest.mark.parametrize("T,H", [(1, 1), (127, 5), (129, 16), (257, 3), (1000, 32), (1300, 128)])
def test_expand(T, H):
    torch, B = _t()
    g = _gen(T + H)
    codes, scales = _cache(T, T + 20, 10.0)
    at = torch.randint(0, T + 20, (T,), generator=g, device="cuda", dtype=torch.int32)     # repeats
    wk, wv = (_randn(g, H, 128, 512) / 22.6).bfloat16(), (_randn(g, H, 512, 128) / 22.6).bfloat16()
    k, v = (torch.full((T, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kr = torch.full((T, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.expand_kv_fp8_rows(codes, scales, at, wk, wv, k, kr, v)
    x = _rows64(codes, scales, at.long())
    c = x[:, :512]
    for got, w, eq in ((k, wk, "tr,hnr->thn"), (v, wv, "tr,hrn->thn")):
        ref = torch.einsum(eq, c, w.double())
        size = torch.einsum(eq, c.abs(), w.double().abs())
        # one bf16 rounding of the result; the fp32 sum of 512 products and the scale's product
        assert ((got.double() - ref).abs() <= BF * ref.abs() + 2.0 ** -14 * size).all()
    assert ((kr.double() - x[:, 512:]).abs() <= BF * x[:, 512:].abs()).all()


def test_expand_reads_row_zero_for_a_bad_index():
    torch, B = _t()
    g = _gen(1)
    codes, scales = _cache(2, 40, 4.0)
    wk, wv = (_randn(g, 2, 128, 512) / 22.6).bfloat16(), (_randn(g, 2, 512, 128) / 22.6).bfloat16()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(at, ws=None):
        k, v = (torch.empty((len(at), 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kr = torch.empty((len(at), 64), dtype=torch.bfloat16, device="cuda")
        B.expand_kv_fp8_rows(codes, scales, torch.tensor(at, dtype=torch.int32, device="cuda"), wk, wv, k, kr, v,
                             workspace=ws)
        return k, kr, v

    bad, good = run([3, -7, 40, 2], ws), run([3, 0, 0, 2])
    assert B.check_errors(ws) == 6
    assert all(torch.equal(a, b) for a, b in zip(bad, good))


# ------------------------------------------------------------------------ decode

def _decode(codes, scales, lens, H, seed, dtype=None, sm=SM, stream=None, indices=None):
    torch, B = _t()
    g = _gen(seed)
    n, b = sum(lens), len(lens)
    indptr = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    if indices is None:
        indices = torch.randperm(len(codes), generator=g, device="cuda")[:n].to(torch.int32)
    qn, qr = _randn(g, b, H, 512).bfloat16(), _randn(g, b, H, 64).bfloat16()
    plan = B.decode_plan(indptr, H)[0]
    ws = torch.zeros(B.decode_fp8_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    out = torch.full((b, H, 512), float("nan"), dtype=dtype or torch.float32, device="cuda")
    lse = torch.full((b, H), float("nan"), device="cuda")
    args = (plan, torch.from_numpy(plan).cuda(), qn, qr, codes, scales, torch.from_numpy(indptr).cuda(), indices, sm,
            out, lse, ws)
    torch.cuda.synchronize()
    B.decode_run_fp8_rows(*args, stream=stream)
    return args, indptr


def _check(args, indptr, status=0):
    torch, B = _t()
    plan, _, qn, qr, codes, scales, _, indices, sm, out, lse, ws = args
    assert B.check_errors(ws) == status
    q = torch.cat((qn, qr), -1).double()
    for i in range(len(indptr) - 1):
        at = indices[indptr[i]:indptr[i + 1]].long()
        if not len(at):
            assert (out[i] == 0).all() and (lse[i] == -math.inf).all()
            continue
        at = torch.where((at < 0) | (at >= len(codes)), torch.zeros_like(at), at)
        x = _rows64(codes, scales, at)
        s = q[i] @ x.t() * sm
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[:, None])
        ref = p @ x[:, :512]
        # weights: 2^-8 of themselves, or 2^-15 of the head's largest weight of codes; for an fp32 output 2^-15 of
        # themselves, or 2^-19 (two or four 8-bit parts; the head's largest weight is 32 or more).  Their sum is taken
        # before they are rounded; scores: fp32 sums of 576 products, of which 2^-18 of the largest possible score is
        # ample
        own, least = (BF, 2.0 ** -15) if out.dtype is torch.bfloat16 else (2.0 ** -15, 2.0 ** -19)
        code = codes[at].view(torch.float8_e4m3fn).double()[:, :512].abs()
        r = scales[at].double().clamp(LOW, HIGH)
        top = (p * r).amax(1, keepdim=True)
        off = 2.0 ** -18 * (q[i].abs() @ x.abs().t()).amax(1, keepdim=True) * abs(sm)
        bound = (own + off) * (p @ x[:, :512].abs()) + least * top * code.sum(0)
        if out.dtype is torch.bfloat16:
            bound = bound + BF * (ref.abs() + bound)
        err = (out[i].double() - ref).abs()
        assert (err <= bound).all(), (i, float((err - bound).max()))
        assert ((lse[i].double() - z).abs() <= off[:, 0] + 2.0 ** -20 * z.abs() + 2.0 ** -16).all(), i


LENS = [1, 2, 63, 64, 65, 0, 300, 129, 7, 1500, 0, 64]


@pytest.mark.parametrize("H", [16, 32, 48, 80, 112, 128])
@pytest.mark.parametrize("spread", [0.0, 3.0, 12.0])
@pytest.mark.parametrize("half", [False, True])
def test_decode(H, spread, half):
    torch, _ = _t()
    codes, scales = _cache(H, 4000, spread)
    _check(*_decode(codes, scales, LENS, H, 5, dtype=torch.bfloat16 if half else torch.float32))


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("lens", [[1], [33] * 200, [20000], [9000, 17, 30000]])
@pytest.mark.parametrize("half", [False, True])
def test_decode_few_long_and_many_short(H, lens, half):
    torch, _ = _t()
    codes, scales = _cache(H + len(lens), sum(lens) + 9, 2.0)
    _check(*_decode(codes, scales, lens, H, 6, dtype=torch.bfloat16 if half else torch.float32))


@pytest.mark.parametrize("H,half", [(16, True), (64, False), (128, True), (128, False)])
def test_decode_more_items_than_a_worker_keeps_at_hand(H, half):
    torch, _ = _t()
    lens = [3, 0, 130, 1, 64, 65, 2, 5] * 260
    codes, scales = _cache(H, 90000, 6.0)
    _check(*_decode(codes, scales, lens, H, 12, dtype=torch.bfloat16 if half else torch.float32))


@pytest.mark.parametrize("H", [16, 128])
def test_decodes_on_two_streams_at_once(H):
    torch, B = _t()
    codes, scales = _cache(H, 30000, 3.0)
    calls = [_decode(codes, scales, lens, H, 20 + i) for i, lens in enumerate(([700, 9, 4000], [2500, 64], [33] * 90))]
    first = [(a[9].clone(), a[10].clone()) for a, _ in calls]
    torch.cuda.synchronize()
    for _ in range(3):
        for a, _ in calls:
            a[9].fill_(float("nan"))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in calls]
        for st, (a, _) in zip(streams, calls):
            B.decode_run_fp8_rows(*a, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(a[9], o) and torch.equal(a[10], z) for (a, _), (o, z) in zip(calls, first))
    for a, ip in calls:
        _check(a, ip)


@pytest.mark.parametrize("H", [32, 64])
def test_decode_scales_outside_the_range(H):
    # zero, negative, NaN, infinite and subnormal scales are read as the nearest end; the rest of the batch is exact
    torch, _ = _t()
    codes, scales = _cache(9, 600, 1.0)
    scales[::97] = 0.0
    scales[1::97] = -3.0
    scales[2::97] = float("nan")
    scales[3::97] = 1e-42
    args, indptr = _decode(codes, scales, [500, 64, 1], H, 7)
    args = list(args)
    args[5] = torch.nan_to_num(scales, nan=0.0)
    _check(args, indptr)
    # an infinite scale takes its own request with it, not its neighbours
    scales[:] = _cache(9, 600, 1.0)[1]
    at = torch.arange(565, dtype=torch.int32, device="cuda")
    scales[510] = float("inf")
    args, indptr = _decode(codes, scales, [500, 64, 1], H, 7, indices=at)
    out, lse = args[9], args[10]
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()       # 2^64: large, and finite


@pytest.mark.parametrize("H", [16, 96])
def test_decode_of_equal_scales_is_that_of_one_scale(H):
    torch, B = _t()
    codes, scales = _cache(2, 3000, 0.0)
    scales.fill_(0.0078125)
    args, indptr = _decode(codes, scales, [700, 1, 2000], H, 8)
    _check(args, indptr)
    plan, plan_dev, qn, qr, _, _, ip, ix, sm, out, lse, ws = args
    other, other_lse = torch.empty_like(out), torch.empty_like(lse)
    B.decode_run_fp8(plan, plan_dev, qn, qr, codes, 0.0078125, ip, ix, sm, other, other_lse, ws)
    # both weigh the same codes by the same weights, up to their roundings
    assert torch.allclose(out, other, rtol=2 * BF, atol=2 * BF * 0.0078125 * 16)
    assert torch.allclose(lse, other_lse, atol=2 * BF)


@pytest.mark.parametrize("H", [16, 128])
def test_decode_records_a_bad_slot_and_reads_row_zero(H):
    torch, _ = _t()
    codes, scales = _cache(3, 500, 6.0)
    at = torch.randperm(500, device="cuda").to(torch.int32)[:400]
    at[7], at[100], at[399] = -1, 500, 2 ** 31 - 1
    _check(*_decode(codes, scales, [100, 300], H, 9, indices=at), status=6)


@pytest.mark.parametrize("sm", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("H", [32, 112])
def test_decode_at_other_softmax_scales(H, sm):
    codes, scales = _cache(4, 900, 1.0)
    _check(*_decode(codes, scales, [65, 800], H, 10, sm=sm))


@pytest.mark.parametrize("H", [16, 128])
def test_decode_on_a_stream_and_replayed(H):
    torch, B = _t()
    codes, scales = _cache(5, 1500, 2.0)
    side = torch.cuda.Stream()
    args, indptr = _decode(codes, scales, [1000, 3, 400], H, 11, stream=side)
    side.synchronize()
    _check(args, indptr)
    first, first_lse = args[9].clone(), args[10].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.decode_run_fp8_rows(*args)
    args[9].fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    _check(args, indptr)
    assert torch.equal(args[9], first) and torch.equal(args[10], first_lse)
    scales.mul_(0.5)                              # the replay reads what the buffers hold now
    graph.replay()
    torch.cuda.synchronize()
    _check(args, indptr)


# ---------------------------------------------------------------- as they are used

def test_rows_past_four_gigabytes():
    """The same rows in a small cache and at the end of one of 4.4 GB: appended, expanded, attended to, copied and
    compacted, bit for bit."""
    torch, B = _t()
    g = _gen(31)
    T, N, H = 500, 7_600_000, 16
    rows, pos = _randn(g, T, 576).bfloat16(), torch.arange(T, dtype=torch.int32, device="cuda")
    fr = B.rope_frequencies()
    wk, wv = _randn(g, H, 128, 512).bfloat16(), _randn(g, H, 512, 128).bfloat16()
    qn, qr = _randn(g, 2, H, 512).bfloat16(), _randn(g, 2, H, 64).bfloat16()
    indptr = np.array([0, 470, T], dtype=np.int32)
    plan = B.decode_plan(indptr, H)[0]
    results = []
    for n in (T, N):
        slots = n - 1 - (n // T) * torch.arange(T, dtype=torch.int32, device="cuda")
        codes = torch.zeros((n, 576), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(n, device="cuda")
        B.rope_append_kv_fp8_rows(codes, scales, slots, rows, pos, fr)
        k, v = (torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kr = torch.empty((T, 64), dtype=torch.bfloat16, device="cuda")
        B.expand_kv_fp8_rows(codes, scales, slots, wk, wv, k, kr, v)
        ws = torch.zeros(B.decode_fp8_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty((2, H, 512), device="cuda"), torch.empty((2, H), device="cuda")
        B.decode_run_fp8_rows(plan, torch.from_numpy(plan).cuda(), qn, qr, codes, scales,
                              torch.from_numpy(indptr).cuda(), slots, SM, out, lse, ws)
        assert B.check_errors(ws) == 0
        at = slots.long()
        results.append((codes[at], scales[at], k, kr, v, out, lse))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    want, want_s = results[0][:2]
    other = slots - 1                                # free slots among them
    B.copy_rows(codes, slots, codes, other, src_scales=scales, dst_scales=scales)
    assert torch.equal(codes[other.long()], want) and torch.equal(scales[other.long()], want_s)
    ws = torch.zeros(B.slots_workspace_bytes(N), dtype=torch.uint8, device="cuda")
    new, live = torch.empty_like(other), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.compact_cache(codes, torch.tensor([0, T], dtype=torch.int32, device="cuda"), other, new, live, ws, kv_scales=scales)
    assert B.check_errors(ws) == 0 and int(live) == T and int(new.max()) < T
    assert torch.equal(codes[new.long()], want) and torch.equal(scales[new.long()], want_s)


@pytest.mark.parametrize("H", [16, 128])
def test_a_prompt_and_its_next_step(H):
    """Rows appended, expanded and attended to in both forms: the absorbed decode of the last token and the expanded
    attention of the same query agree."""
    torch, B = _t()
    g = _gen(12)
    T = 333
    rows = _randn(g, T, 576).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    codes = torch.zeros((T + 7, 576), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(T + 7, device="cuda")
    slots = torch.randperm(T + 7, generator=g, device="cuda")[:T].to(torch.int32)
    fr = B.rope_frequencies()
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    B.rope_append_kv_fp8_rows(codes, scales, slots, rows, pos, fr, norm_weight=w)
    wk, wv = (_randn(g, H, 128, 512) / 22.6).bfloat16(), (_randn(g, H, 512, 128) / 22.6).bfloat16()
    k, v = (torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kr = torch.empty((T, 64), dtype=torch.bfloat16, device="cuda")
    B.expand_kv_fp8_rows(codes, scales, slots, wk, wv, k, kr, v)
    q = _randn(g, 1, H, 192).bfloat16()
    out = torch.empty((1, H, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((1, H), device="cuda")
    B.Prefiller([0, 1], [0, T], H).run(q, k, kr, v, SM, out, lse)
    q_nope = torch.empty((1, H, 512), dtype=torch.bfloat16, device="cuda")
    B.absorb_query(q[..., :128].contiguous(), wk, q_nope)
    plan = B.decode_plan([0, T], H)[0]
    ws = torch.zeros(B.decode_fp8_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    lat = torch.empty((1, H, 512), dtype=torch.bfloat16, device="cuda")
    lse2 = torch.empty((1, H), device="cuda")
    B.decode_run_fp8_rows(plan, torch.from_numpy(plan).cuda(), q_nope, q[..., 128:].contiguous(), codes, scales,
                          torch.tensor([0, T], dtype=torch.int32, device="cuda"), slots, SM, lat, lse2, ws)
    out2 = torch.empty((1, H, 128), dtype=torch.bfloat16, device="cuda")
    B.project_output(lat, wv, out2)
    x = _rows64(codes, scales, slots.long())
    kk = torch.einsum("tr,hnr->htn", x[:, :512], wk.double())
    vv = torch.einsum("tr,hrn->htn", x[:, :512], wv.double())
    s = (torch.einsum("hn,htn->ht", q[0, :, :128].double(), kk) + q[0, :, 128:].double() @ x[:, 512:].t()) * SM
    ref = torch.einsum("ht,htn->hn", torch.softmax(s, -1), vv)
    # expanded keys are rounded to bf16 (scores off by 2^-8 |q||k| sm a key at most, 2^-9 of it typically), absorbed
    # queries likewise; probabilities and values then by as much: 6 % of the values' size covers the worst of both
    size = torch.einsum("ht,htn->hn", torch.softmax(s, -1), vv.abs())
    for got in (out, out2):
        assert ((got[0].double() - ref).abs() <= 0.06 * size).all()
    for got in (lse, lse2):
        assert ((got[0].double() - torch.logsumexp(s, -1)).abs() <= 0.03).all()
