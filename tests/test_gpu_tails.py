"""GPU tests of the 8-bit decodes where one row outweighs each of very many
others and they still make up a visible part of the result (an attention sink
before a long flat tail), against 64-bit formulas.  The scores are set through
one rope dimension, so that they are exact; the latents share a mean.  A plan for
one worker makes a request one item, however long."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SM = 1.0 / math.sqrt(192.0)
SCALE = 1.0 / 64.0


def _t():
    import torch
    from mla_latent_kv_absorbed_gb300 import binding
    return torch, binding


def _e4m3(x):
    torch, _ = _t()
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _case(n, H, kind, seed):
    """codes uint8 [n, 576], a scale for each row, queries [1, H, ..]: in head h the row that stands out has about
    exp(gap[h]) times the weight of an ordinary one, 0.05 to 0.99 of the whole."""
    torch, _ = _t()
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    scales = torch.full((n,), SCALE, device="cuda")
    if kind == "loud":
        scales = SCALE * torch.exp2(torch.randint(-3, 4, (n,), generator=g, device="cuda").float())
    x = 100.0 * (rand(n, 512) + torch.where(rand(512) > 0, 1.0, -1.0))
    values = torch.zeros(n, device="cuda")                      # what a unit of the query's gives to the score
    if kind in ("spread", "loud"):
        values = 0.4 * rand(n)
    elif kind == "stairs":                                       # ever lower, 0.9 of the way to the top a step
        values = -6.3 * torch.div(torch.arange(n, device="cuda"), max(n // 8, 64), rounding_mode="floor")
    elif kind == "wide":                                         # scores N(0, 4)
        values = 2.5 * rand(n)
    if kind == "often":
        values[::997] = 448 * SCALE
    elif kind == "last":
        values[n - 1] = 448 * SCALE
    elif kind != "wide":
        values[0] = 448 * SCALE
    codes = torch.zeros((n, 576), device="cuda")
    codes[:, :512] = x
    scales[values >= 448 * SCALE] = SCALE
    codes[:, 512] = values / scales
    codes = _e4m3(codes).view(torch.uint8)
    share = torch.tensor([0.05, 0.2, 0.5, 0.8, 0.95, 0.99], device="cuda", dtype=torch.float64)
    gap = (math.log(n) + torch.log(share / (1 - share)))[torch.arange(H, device="cuda") % len(share)]
    qn = torch.zeros((1, H, 512), device="cuda", dtype=torch.bfloat16)
    qr = torch.zeros((1, H, 64), device="cuda", dtype=torch.bfloat16)
    qr[0, :, 0] = (gap / (448 * SCALE * SM)).bfloat16()
    return codes, scales, qn, qr


def _reference(codes, scales, qr):
    torch, _ = _t()
    x = codes.view(torch.float8_e4m3fn).double() * scales.double()[:, None]
    p = torch.softmax(qr[0].double() @ x[:, 512:].t() * SM, -1)
    return p @ x[:, :512], (p @ x[:, :512].norm(dim=1))[:, None]


def _run(codes, scales, qn, qr, half, sms):
    """One request of all rows over `sms` SMs: the row-scaled decode, or for a number in the place of scales the other."""
    torch, B = _t()
    n, H = len(codes), qn.shape[1]
    indptr = np.array([0, n], dtype=np.int32)
    plan = B.decode_plan(indptr, H, num_sms=sms)[0]
    ws = torch.zeros(B.decode_fp8_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    out = torch.full((1, H, 512), float("nan"), dtype=torch.bfloat16 if half else torch.float32, device="cuda")
    lse = torch.full((1, H), float("nan"), device="cuda")
    run = B.decode_run_fp8 if isinstance(scales, float) else B.decode_run_fp8_rows
    run(plan, torch.from_numpy(plan).cuda(), qn, qr, codes, scales, torch.from_numpy(indptr).cuda(),
        torch.arange(n, dtype=torch.int32, device="cuda"), SM, out, lse, ws)
    assert B.check_errors(ws) == 0
    return out[0], lse[0]


def _sums(n, products=0):
    """Sums in 32 bits.  l: a thread adds a tile's sum (of up to 16 rows, then with its neighbours': 2^-20) at every
    second tile of 64 rows, each addition off by 2^-24 of the sum, all with one sign where the weights are equal.  O: the
    tensor core cuts what it has added up to 24 bits after every `products` of 32 rows, towards zero: 2^-23 of the sum
    each, all of one sign where one row has most of it."""
    return n / 128 * 2.0 ** -24 + 2.0 ** -20 + products * n / 32 * 2.0 ** -23


def _bound(half, n):
    """Weights off by 2^-8 of themselves (fp32 out: 2^-16) and, whatever their number, twice 2^-9 (2^-16) of their sum
    in all; rows' norms, which that is relative to, are alike but for a factor below 1.5; the output's own rounding, or
    for fp32 exponents of up to 2^5 (2^-18); sums in 32 bits of two (four) parts."""
    return 2.5 * 2.0 ** -8 + 2.0 ** -8 + _sums(n, 2) if half else 4 * 2.0 ** -16 + 2.0 ** -18 + _sums(n, 4)


KINDS = ["equal", "spread", "loud", "last", "often", "stairs", "wide"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [4096, 16384, 131072])
@pytest.mark.parametrize("H", [16, 48, 128])
def test_rows_tail(n, H, kind):
    torch, _ = _t()
    codes, scales, qn, qr = _case(n, H, kind, n + H)
    ref, size = _reference(codes, scales, qr)
    x = codes.view(torch.float8_e4m3fn).double()[:, 512:] * scales.double()[:, None]
    z = torch.logsumexp(qr[0].double() @ x.t() * SM, -1)
    for half in (False, True):
        out, lse = _run(codes, scales, qn, qr, half, 1 if H <= 32 else 2)
        err = (out.double() - ref).norm(dim=1, keepdim=True) / size
        assert err.max() <= _bound(half, n), (half, float(err.max()))
        # (exponents of up to 2^5, in fp32, and the sum)
        assert ((lse.double() - z).abs() <= 2.0 ** -18 + _sums(n)).all()


@pytest.mark.parametrize("kind", ["equal", "spread", "often", "stairs"])
@pytest.mark.parametrize("H", [16, 128])
def test_rows_tail_over_all_sms(H, kind):
    codes, scales, qn, qr = _case(200000, H, kind, H)
    ref, size = _reference(codes, scales, qr)
    for half in (False, True):
        out, _ = _run(codes, scales, qn, qr, half, 0)
        assert ((out.double() - ref).norm(dim=1, keepdim=True) <= _bound(half, 200000) * size).all()


@pytest.mark.parametrize("kind", [k for k in KINDS if k != "loud"])
@pytest.mark.parametrize("n", [4096, 16384, 131072])
@pytest.mark.parametrize("H", [16, 32, 48, 128])
def test_one_scale_tail(n, H, kind):
    torch, _ = _t()
    codes, scales, qn, qr = _case(n, H, kind, n + H)
    ref, size = _reference(codes, scales, qr)
    x = codes.view(torch.float8_e4m3fn).double()[:, 512:] * SCALE
    z = torch.logsumexp(qr[0].double() @ x.t() * SM, -1)
    for half in (False, True):
        out, lse = _run(codes, SCALE, qn, qr, half, 1 if H <= 32 else 2)
        err = (out.double() - ref).norm(dim=1, keepdim=True) / size
        # two parts of the weights whatever the output, off by 2^-8 of themselves at most, and 2^-7 of what a window of
        # 1024 rows adds up to where all of its weights are small
        assert err.max() <= _bound(True, n), (half, float(err.max()))
        # (16 and 32 heads: the sum is that of the rounded weights)
        assert ((lse.double() - z).abs() <= 2.5 * 2.0 ** -8 + _sums(n)).all()


@pytest.mark.parametrize("H", [16, 128])
def test_one_scale_tail_over_all_sms(H):
    for kind in ("equal", "spread", "often", "stairs"):
        codes, _, qn, qr = _case(200000, H, kind, H)
        torch, _ = _t()
        ref, size = _reference(codes, torch.full((200000,), SCALE, device="cuda"), qr)
        out, _ = _run(codes, SCALE, qn, qr, False, 0)
        assert ((out.double() - ref).norm(dim=1, keepdim=True) <= _bound(True, 200000) * size).all(), kind
