"""Host-side tests of the prompt side (no GPU needed): frequencies, the prefill
plan, and arguments refused before any launch."""
import ctypes

import numpy as np
import pytest

from oracle import prompt_oracle as P
from tests.test_abi import B, _fake_ptr  # noqa: F401  (the fixture)

F = ctypes.c_float


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=8.0), dict(scaling="yarn", factor=40.0),
                                dict(theta=500000.0, scaling="yarn", factor=4.0, original_positions=8192),
                                dict(theta=1000000.0, scaling="yarn", factor=16.0, beta_fast=16.0, beta_slow=2.0)])
def test_frequencies_match_the_oracle(B, kw):
    got = B.rope_frequencies(**kw).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    ref = P.rope_inv_freq(**{k.replace("original_positions", "original"): v for k, v in kw.items()})
    # both sides in float64: a few roundings of pow and the division by 2 pi, and half a unit of 2^-64 turns
    assert np.allclose(got, ref, rtol=1e-14, atol=np.pi * 2.0 ** -64)


def test_frequencies_refuse_bad_arguments(B):
    lib = B.library()
    out = np.zeros(32, dtype=np.uint64)

    def f(theta=1e4, scaling=0, factor=2.0, orig=4096, fast=32.0, slow=1.0, p=out.ctypes.data):
        return lib.mla_rope_frequencies(theta, scaling, factor, orig, fast, slow, p)

    assert f() == 0
    assert f(p=None) == 1
    assert f(theta=1.0) == 1 and f(theta=float("nan")) == 1 and f(theta=float("inf")) == 1
    assert f(scaling=3) == 2 and f(scaling=-1) == 2
    assert f(scaling=1, factor=0.5) == 1 and f(scaling=1, factor=float("inf")) == 1
    assert f(scaling=0, factor=float("nan"), orig=0) == 0          # unused values are not looked at
    assert f(scaling=2, orig=0) == 1 and f(scaling=2, slow=0.0) == 1 and f(scaling=2, fast=0.5) == 1
    assert f(scaling=2, fast=float("inf")) == 1
    with pytest.raises(B.MLAError):
        B.rope_frequencies(scaling="other")


def test_rope_query_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()
    fr = B.rope_frequencies()

    def f(q=fake, qts=16 * 192, qhs=192, pos=fake, T=4, H=16, nope=128, freqs=fr.ctypes.data, amp=1.0, il=1, r=fake,
          rts=16 * 64, rhs=64, n=None):
        return lib.mla_rope_query(q, qts, qhs, pos, T, H, nope, freqs, F(amp), il, r, rts, rhs, n, None)

    assert f(T=0) == 0 and f(T=0, q=None, pos=None, r=None) == 0
    assert f(q=None) == 1 and f(q=fake + 8) == 1 and f(pos=None) == 1 and f(pos=fake + 2) == 1
    assert f(r=None) == 1 and f(r=fake + 8) == 1 and f(n=fake + 8) == 1
    assert f(T=-1) == 1 and f(H=0) == 1 and f(H=65536) == 1 and f(nope=-8) == 1
    assert f(nope=4) == 2
    assert f(freqs=None) == 1 and f(amp=float("nan")) == 1 and f(il=2) == 1
    assert f(qts=-8) == 1 and f(qts=12) == 1 and f(qhs=100) == 1 and f(qts=1 << 38) == 1
    # output rows that overlap, in either order of tokens and heads
    assert f(rhs=56) == 1 and f(rts=64, rhs=64) == 1 and f(rts=64, rhs=192) == 1


def test_rope_query_refuses_rows_that_overlap_far_apart(B):
    # heads as far apart as tokens, over more tokens than 64 bits of elements hold
    lib, fake = B.library(), _fake_ptr()
    fr = B.rope_frequencies()
    for T, stride in (((1 << 29) + 1, 1 << 34), ((1 << 30) - 1, (1 << 38) - 8), ((1 << 27) + 3, 1 << 37)):
        assert lib.mla_rope_query(fake, 384, 192, fake, T, 2, 128, fr.ctypes.data, F(1.0), 1, fake, stride, stride,
                                  None, None) == 1, (T, stride)


def test_rope_append_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()
    fr = B.rope_frequencies()

    def f(kv=fake, n=100, slots=fake, rows=fake, rs=576, pos=fake, T=4, w=None, eps=1e-6, freqs=fr.ctypes.data,
          amp=1.0, il=1, ws=None, scale=None):
        if scale is None:
            return lib.mla_rope_append_kv(kv, n, slots, rows, rs, pos, T, w, F(eps), freqs, F(amp), il, ws, None)
        return lib.mla_rope_append_kv_fp8(kv, n, slots, rows, rs, pos, T, w, F(eps), freqs, F(amp), il, F(scale), ws,
                                          None)

    for s in (None, 0.5):
        assert f(T=0, scale=s) == 0 and f(T=0, kv=None, slots=None, rows=None, pos=None, scale=s) == 0
        for bad in (dict(kv=None), dict(kv=fake + 8), dict(slots=None), dict(slots=fake + 2), dict(rows=None),
                    dict(rows=fake + 2), dict(pos=None), dict(pos=fake + 1), dict(w=fake + 2), dict(ws=fake + 4),
                    dict(n=0), dict(n=1 << 31), dict(T=-1), dict(rs=-8), dict(rs=580), dict(rs=568),
                    dict(eps=-1.0), dict(eps=float("inf")), dict(freqs=None), dict(amp=float("inf")), dict(il=-1)):
            assert f(scale=s, **bad) == 1, bad
    assert f(scale=0.0) == 1 and f(scale=-1.0) == 1 and f(scale=float("nan")) == 1


def test_expand_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()

    def f(kv=fake, n=100, idx=fake, T=4, wk=fake, wv=fake, H=16, k=fake, kr=fake, v=fake, ws=None, scale=None):
        if scale is None:
            return lib.mla_expand_kv(kv, n, idx, T, wk, wv, H, k, kr, v, ws, None)
        return lib.mla_expand_kv_fp8(kv, n, F(scale), idx, T, wk, wv, H, k, kr, v, ws, None)

    for s in (None, 0.5):
        assert f(T=0, scale=s) == 0 and f(T=0, kv=None, idx=None, wk=None, k=None, scale=s) == 0
        for bad in (dict(kv=None), dict(kv=fake + 8), dict(idx=None), dict(idx=fake + 2), dict(wk=fake + 8),
                    dict(wv=None), dict(k=None), dict(kr=fake + 8), dict(v=fake + 2), dict(ws=fake + 8), dict(n=0),
                    dict(T=-1), dict(H=0), dict(H=65536)):
            assert f(scale=s, **bad) == 1, bad
    assert f(scale=0.0) == 1 and f(scale=float("inf")) == 1


def _plan_cases():
    rng = np.random.default_rng(7)
    yield [0], [0], 4
    yield [0, 0, 0], [0, 5, 9], 4
    yield [0, 1], [0, 0], 1
    yield [0, 300], [0, 20], 3
    yield [0, 64, 128], [0, 65536, 97600], 16
    yield [0, 1], [0, 131072], 1
    for _ in range(40):
        n = int(rng.integers(1, 12))
        ql = rng.integers(0, 900, n) * (rng.random(n) < 0.8)
        kl = np.maximum(0, ql + rng.integers(-100, 4000, n))
        yield np.cumsum(np.r_[0, ql]).tolist(), np.cumsum(np.r_[0, kl]).tolist(), int(rng.choice([1, 5, 16, 128]))


@pytest.mark.parametrize("sms", [152, 7, 1])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_plan_covers_every_row_and_key_once(B, sms, causal):
    for qp, kp, H in _plan_cases():
        plan, ws = B.prefill_plan(qp, kp, H, causal, num_sms=sms)
        n, partials, merges, group, R = (int(plan[i]) for i in (7, 8, 9, 10, 13))
        assert R in (256, 512)
        assert plan.size == 16 + 8 * n + 4 * merges and 1 <= group <= H
        assert ws == 256 + partials * H * R * 129 * 4
        seen, used = {}, set()
        for b, q0, nq, k0, nk, off, part, _ in plan[16:16 + 8 * n].reshape(-1, 8).tolist():
            lq, lk = qp[b + 1] - qp[b], kp[b + 1] - kp[b]
            assert qp[b] <= q0 and q0 + nq <= qp[b + 1] and 1 <= nq <= R and (q0 - qp[b]) % R == 0
            assert nq == min(R, qp[b + 1] - q0)
            assert nk >= 0 and kp[b] <= k0 and k0 + nk <= kp[b + 1]
            if causal:       # row r of the item sees the piece's keys j <= r + off
                assert off == (q0 - qp[b]) + lk - lq - (k0 - kp[b])
            assert part == -1 or (0 <= part < partials and part not in used)
            used.add(part) if part >= 0 else None
            seen.setdefault(q0, []).append((k0 - kp[b], nk, part, b, nq))
        for b in range(len(qp) - 1):
            for q0 in range(qp[b], qp[b + 1], R):
                pieces = sorted(seen.pop(q0))
                lq, lk = qp[b + 1] - qp[b], kp[b + 1] - kp[b]
                nq = min(R, qp[b + 1] - q0)
                last = lk if not causal else min(lk, max(0, q0 - qp[b] + nq + lk - lq))
                at = 0
                for k, nk, part, bb, _ in pieces:
                    assert bb == b and k == at and (part >= 0) == (len(pieces) > 1)
                    at += nk
                assert at == last
        assert not seen
        entries = plan[16 + 8 * n:].reshape(-1, 4).tolist()
        assert sum(e[3] - e[2] for e in entries) == partials == len(used)
        again, _ = B.prefill_plan(qp, kp, H, causal, num_sms=sms)
        assert np.array_equal(plan, again)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_plan_bounds_the_keys_of_an_item(B, causal):
    # 1000 rows over 2^28 keys on one SM: nothing to gain from a cut, but no item may keep its warps waiting long
    plan, ws = B.prefill_plan([0, 1000], [0, 1 << 28], 1, causal, num_sms=1)
    n = int(plan[7])
    items = plan[16:16 + 8 * n].reshape(-1, 8)
    assert (items[:, 4] <= 1 << 24).all() and (items[:, 6] >= 0).all()
    for q0 in sorted(set(items[:, 1].tolist())):
        mine = items[items[:, 1] == q0]
        mine = mine[np.argsort(mine[:, 3])]
        assert mine[0, 3] == 0 and (mine[1:, 3] == mine[:-1, 3] + mine[:-1, 4]).all()
        last = (1 << 28) if not causal else min(1 << 28, q0 + int(mine[0, 2]) + (1 << 28) - 1000)
        assert mine[-1, 3] + mine[-1, 4] == last
    assert ws == 256 + int(plan[8]) * int(plan[13]) * 129 * 4


def test_prefill_plan_keeps_short_items_for_the_end(B):
    # many heads whose keys do not fit L2 together, rows of very different lengths
    ql = [1500, 1, 640, 2047, 333, 16, 1024, 129, 800, 257, 64]
    qp = np.cumsum([0] + ql)
    plan, _ = B.prefill_plan(qp, qp, 64, True, num_sms=152)
    n, tail = int(plan[7]), int(plan[15])
    assert plan[10] < 64 and 0 < tail < n
    cost = plan[16:16 + 8 * n].reshape(-1, 8)[:, 4]
    assert cost[n - tail:].sum() * 3 <= cost.sum()
    one, _ = B.prefill_plan(qp, qp, 1, True, num_sms=152)
    assert one[15] == 0


def test_prefill_plan_cuts_long_keys_of_few_rows_only(B):
    few, _ = B.prefill_plan([0, 64], [0, 65536], 16, True, num_sms=152)
    assert few[8] > 1 and few[9] == 1
    many, _ = B.prefill_plan([0, 8192], [0, 8192], 128, True, num_sms=152)
    assert many[8] == 0 and many[7] == 8192 // many[13]
    # heaviest first
    nk = many[16:].reshape(-1, 8)[:, 4]
    assert (np.diff(nk) <= 0).all()


def test_prefill_plan_refuses_bad_arguments(B):
    lib = B.library()
    n, ws = ctypes.c_size_t(0), ctypes.c_size_t(0)

    def f(qp=(0, 5), kp=(0, 9), b=1, H=16, causal=1, sms=152, plan=None, words=0):
        qa, ka = np.array(qp, dtype=np.int32), np.array(kp, dtype=np.int32)
        return lib.mla_prefill_plan(qa.ctypes.data, ka.ctypes.data, b, H, causal, sms, plan, words, ctypes.byref(n),
                                    ctypes.byref(ws))

    assert f() == 0 and n.value == 24
    assert f(qp=(1, 5)) == 1 and f(kp=(1, 9)) == 1 and f(qp=(0, -1)) == 1 and f(b=2, qp=(0, 5, 4), kp=(0, 1, 2)) == 1
    assert f(b=-1) == 1 and f(H=0) == 1 and f(H=65536) == 1 and f(causal=2) == 1 and f(sms=-1) == 1
    assert f(kp=(0, (1 << 30) - 1)) == 2 and f(qp=(0, (1 << 30) - 1)) == 2
    assert f(qp=(0, 1 << 24), kp=(0, 0), H=65535) == 2         # more tiles than a launch counts
    assert f(sms=2 ** 31 - 1) == 0
    buf = np.zeros(24, dtype=np.int32)
    assert f(plan=buf.ctypes.data, words=23) == 3 and f(plan=buf.ctypes.data, words=24) == 0
    assert lib.mla_prefill_plan(None, buf.ctypes.data, 0, 1, 1, 152, None, 0, None, None) == 1
    with pytest.raises(ValueError):
        B.prefill_plan([0, 4], [0, 4, 8], 16)


def test_prefill_run_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()
    plan, need = B.prefill_plan([0, 64], [0, 65536], 16, True, num_sms=152)

    def f(ph=plan, pd=fake, q=fake, qts=16 * 192, qhs=192, k=fake, kts=2048, khs=128, kr=fake, krs=64, v=fake,
          vts=2048, vhs=128, scale=0.1, out=fake, lse=fake, ws=fake, wsb=need):
        return lib.mla_prefill_run(None if ph is None else ph.ctypes.data, pd, q, qts, qhs, k, kts, khs, kr, krs, v,
                                   vts, vhs, F(scale), out, lse, ws, wsb, None)

    assert f(ph=None) == 1 and f(pd=None) == 1 and f(pd=fake + 4) == 1
    for i in (0, 1, 11):                                   # magic, version, word count
        bad = plan.copy()
        bad[i] += 1
        assert f(ph=bad) == 1
    for i, x in ((13, 300), (14, 2), (15, -1), (15, int(plan[7]) + 1)):   # rows of an item, one row tile, items kept for the end
        bad = plan.copy()
        bad[i] = x
        assert f(ph=bad) == 1
    assert f(wsb=need - 1) == 3 and f(ws=None) == 1 and f(ws=fake + 8) == 1
    assert f(scale=float("inf")) == 1
    for name in ("q", "k", "kr", "v", "out"):
        assert f(**{name: None}) == 1 and f(**{name: fake + 8}) == 1
    assert f(lse=fake + 2) == 1
    for name, least in (("qts", 192), ("qhs", 192), ("kts", 128), ("khs", 128), ("krs", 64), ("vts", 128),
                        ("vhs", 128)):
        assert f(**{name: least - 8}) == 1 and f(**{name: least + 4}) == 1 and f(**{name: -least}) == 1
        assert f(**{name: 1 << 38}) == 1
    # no query row: nothing is launched, and only plan, scale and workspace are looked at
    empty, _ = B.prefill_plan([0, 0], [0, 50], 16, num_sms=152)
    assert f(ph=empty, q=None, k=None, kr=None, v=None, out=None, lse=None) == 0


def test_wrappers_refuse_tensors_that_do_not_fit(B):
    # raised before the library is called (CPU tensors stand in; a CPU tensor itself is the last refusal)
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    fr = B.rope_frequencies()

    def no(match, call):
        with pytest.raises(ValueError, match=match):
            call()

    q, pos, r = z(3, 4, 192), z(3, dt=i32), z(3, 4, 64)
    no("not on a CUDA device", lambda: B.rope_query(q, pos, fr, r))
    no("q is torch.float32", lambda: B.rope_query(q.float(), pos, fr, r))
    no("q has shape", lambda: B.rope_query(q[0], pos, fr, r))
    no("its last dimension together", lambda: B.rope_query(z(3, 192, 4).transpose(1, 2), pos, fr, r))
    rows, slots = z(3, 576), z(3, dt=i32)
    no("kv_cache is torch.uint8", lambda: B.rope_append_kv(z(9, 576, dt=torch.uint8), slots, rows, pos, fr))
    no("kv_cache is torch.bfloat16", lambda: B.rope_append_kv_fp8(z(9, 576), slots, rows, pos, fr, 1.0))
    no("kv_cache has shape", lambda: B.rope_append_kv(z(9, 512), slots, rows, pos, fr))
    no("not on a CUDA device", lambda: B.rope_append_kv(z(9, 576), slots, rows, pos, fr))
    idx, wk, wv = z(5, dt=i32), z(2, 128, 512), z(2, 512, 128)
    k, kr, v = z(5, 2, 128), z(5, 64), z(5, 2, 128)
    no("kv_cache is torch.uint8", lambda: B.expand_kv(z(9, 576, dt=torch.uint8), idx, wk, wv, k, kr, v))
    no("kv_cache is torch.bfloat16", lambda: B.expand_kv_fp8(z(9, 576), 1.0, idx, wk, wv, k, kr, v))
    no("kv_cache has shape", lambda: B.expand_kv(z(9, 64), idx, wk, wv, k, kr, v))
    no("not on a CUDA device", lambda: B.expand_kv(z(9, 576), idx, wk, wv, k, kr, v))
    plan, ws = B.prefill_plan([0, 3], [0, 5], 2, num_sms=152)
    pd = torch.from_numpy(plan)
    out = z(3, 2, 128)
    no("plan_dev has shape", lambda: B.prefill_run(plan, pd[1:], z(3, 2, 192), k, kr, v, 0.1, out, None, z(1)))
    no("plan_host is the int32", lambda: B.prefill_run(plan.astype(np.int64), pd, z(3, 2, 192), k, kr, v, 0.1, out,
                                                       None, z(1)))
    no("not on a CUDA device", lambda: B.prefill_run(plan, pd, z(3, 2, 192), k, kr, v, 0.1, out, None, z(1)))


def test_prefill_run_refuses_a_plan_that_is_cut_short(B):
    # the library reads the plan's items on the device as the header counts them: an array that ends before them is
    # refused, on both sides, and one that goes on behind them too
    import torch
    plan, need = B.prefill_plan([0, 3, 300], [0, 5, 400], 2, num_sms=152)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    for ph in (plan[:16], plan[:-1], np.r_[plan, plan[-1:]], plan[:15], plan[:0]):
        with pytest.raises(ValueError, match="plan_host"):
            B.prefill_run(ph, torch.from_numpy(ph.copy()), z(300, 2, 192), z(400, 2, 128), z(400, 64), z(400, 2, 128), 0.1,
                          z(300, 2, 128), None, z(need, dt=torch.uint8))


def test_wrappers_refuse_a_workspace_without_a_status_word(B):
    # the kernels write four bytes there
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i32, u8, fr = torch.int32, torch.uint8, B.rope_frequencies()
    rows, pos = z(3, 576), z(3, dt=i32)
    heads = (z(2, 128, 512), z(2, 512, 128), z(3, 2, 128), z(3, 64), z(3, 2, 128))
    for ws in (z(0, dt=u8), z(3, dt=u8)):
        for call in (lambda: B.rope_append_kv(z(9, 576), pos, rows, pos, fr, workspace=ws),
                     lambda: B.rope_append_kv_fp8(z(9, 576, dt=u8), pos, rows, pos, fr, 1.0, workspace=ws),
                     lambda: B.expand_kv(z(9, 576), pos, *heads, workspace=ws),
                     lambda: B.expand_kv_fp8(z(9, 576, dt=u8), 1.0, pos, *heads, workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
