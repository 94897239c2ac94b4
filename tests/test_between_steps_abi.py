"""Host-side tests of the row-scaled FP8 cache and of what happens between two
decode steps (no GPU needed): arguments refused before any launch, and hand-made
cases of the oracle."""
import ctypes

import numpy as np
import pytest

from oracle import serving_oracle as S
from tests.test_abi import B, _fake_ptr  # noqa: F401  (the fixture)

F = ctypes.c_float
FAR = 1 << 40


# ------------------------------------------------------------------ row-scaled FP8

def test_decode_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()
    for H in (16, 32, 48, 128):
        plan, _ = B.decode_plan(np.array([0, 100, 300], dtype=np.int32), H, num_sms=152)
        need = B.decode_fp8_workspace_bytes(plan)

        def run(plan_host=plan, q=fake, qr=fake, kv=fake, n=1000, sc=fake, ip=fake, idx=fake, scale=0.1, out=fake,
                out_dtype=0, lse=fake, ws=fake, wsb=need):
            return lib.mla_decode_run_fp8_rows(plan_host.ctypes.data, fake, q, qr, kv, n, sc, ip, idx, F(scale), out,
                                               out_dtype, lse, ws, wsb, None)

        for bad in (dict(sc=None), dict(sc=fake + 2), dict(q=fake + 2), dict(qr=None), dict(kv=fake + 8), dict(n=0),
                    dict(ip=None), dict(out=None), dict(ws=fake + 8), dict(scale=float("nan")),
                    dict(scale=float("inf"))):
            assert run(**bad) == 1, (H, bad)
        assert run(out_dtype=2) == 2 and run(wsb=need - 1) == 3
        other = plan.copy()
        other[0] ^= 1
        assert run(plan_host=other) == 1


def test_row_scaled_append_and_expansion_refuse_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()
    fr = B.rope_frequencies()

    def append(kv=fake, sc=fake, n=100, slots=fake, rows=fake, rs=576, pos=fake, T=4, w=None, eps=1e-6,
               freqs=fr.ctypes.data, amp=1.0, il=1, ws=None):
        return lib.mla_rope_append_kv_fp8_rows(kv, sc, n, slots, rows, rs, pos, T, w, F(eps), freqs, F(amp), il, ws,
                                               None)

    assert append(T=0) == 0 and append(T=0, kv=None, sc=None, slots=None, rows=None, pos=None) == 0
    for bad in (dict(kv=None), dict(kv=fake + 8), dict(sc=None), dict(sc=fake + 2), dict(slots=None),
                dict(rows=fake + 2), dict(pos=None), dict(n=0), dict(n=1 << 31), dict(T=-1), dict(rs=568),
                dict(eps=-1.0), dict(freqs=None), dict(amp=float("nan")), dict(il=2), dict(ws=fake + 4)):
        assert append(**bad) == 1, bad

    def expand(kv=fake, sc=fake, n=100, idx=fake, T=4, wk=fake, wv=fake, H=16, k=fake, kr=fake, v=fake, ws=None):
        return lib.mla_expand_kv_fp8_rows(kv, sc, n, idx, T, wk, wv, H, k, kr, v, ws, None)

    assert expand(T=0) == 0 and expand(T=0, sc=None, kv=None) == 0
    for bad in (dict(sc=None), dict(sc=fake + 1), dict(kv=fake + 4), dict(idx=None), dict(wk=None), dict(wv=fake + 8),
                dict(k=None), dict(kr=fake + 8), dict(v=None), dict(T=-1), dict(H=0), dict(H=65536), dict(n=0),
                dict(ws=fake + 8)):
        assert expand(**bad) == 1, bad


# ------------------------------------------------------------------ between two steps

def test_verify_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()

    def f(t=fake, tb=40, tr=10, d=None, db=40, dr=10, tok=fake, par=None, u=fake, b=2, w=4, v=10, path=fake, acc=fake,
          nxt=fake, ws=None):
        return lib.mla_verify_drafts(t, tb, tr, d, db, dr, tok, par, u, b, w, v, path, acc, nxt, ws, None)

    assert f(b=0) == 0 and f(b=0, t=None, tok=None, u=None, path=None, acc=None, nxt=None) == 0
    for bad in (dict(b=-1), dict(w=0), dict(w=-1), dict(v=0), dict(t=None), dict(t=fake + 2), dict(tok=None),
                dict(tok=fake + 1), dict(u=None), dict(u=fake + 2), dict(path=None), dict(acc=fake + 2),
                dict(nxt=None), dict(ws=fake + 8), dict(par=fake + 2), dict(d=fake + 2), dict(tb=-1), dict(tr=-1),
                dict(tb=FAR), dict(tr=FAR), dict(d=fake, db=-1), dict(d=fake, dr=FAR)):
        assert f(**bad) == 1, bad
    assert f(w=65) == 2 and f(d=fake, par=fake) == 2


def test_slots_workspace(B):
    for n in (1, 31, 32, 33, 1000, 1 << 20, (1 << 31) - 1):
        words = (n + 31) // 32
        got = B.slots_workspace_bytes(n)
        assert got >= 12 * words + 8 * (n // 2) and got % 256 == 0 and got < 12 * words + 4 * n + 4096
    for n in (0, -1, 1 << 31):
        assert B.library().mla_slots_workspace_bytes(n) == 0
        with pytest.raises(B.MLAError):
            B.slots_workspace_bytes(n)


def test_repack_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()
    need = B.slots_workspace_bytes(1000)

    def f(ip=fake, idx=fake, n=50, b=3, src=fake, nb=2, path=None, acc=None, w=0, nip=fake, nidx=fake, cap=60,
          slots=1000, freed=None, fcap=0, fcount=None, ws=fake, wsb=need):
        return lib.mla_repack_requests(ip, idx, n, b, src, nb, path, acc, w, nip, nidx, cap, slots, freed, fcap, fcount,
                                       ws, wsb, None)

    for bad in (dict(ip=None), dict(ip=fake + 2), dict(idx=None), dict(n=-1), dict(n=1 << 31), dict(b=-1), dict(nb=-1),
                dict(src=None), dict(src=fake + 1), dict(path=fake, w=4), dict(acc=fake, w=4),
                dict(path=fake, acc=fake, w=0), dict(path=fake + 2, acc=fake, w=4), dict(nip=None), dict(nidx=None),
                dict(nidx=fake + 2), dict(cap=-1), dict(cap=1 << 31), dict(slots=0), dict(slots=1 << 31),
                dict(freed=fake), dict(fcount=fake), dict(freed=fake + 2, fcount=fake), dict(freed=fake, fcount=fake + 2),
                dict(fcap=-1), dict(ws=None), dict(ws=fake + 8)):
        assert f(**bad) == 1, bad
    assert f(path=fake, acc=fake, w=65) == 2 and f(freed=fake, fcount=fake, b=65537) == 2
    assert f(wsb=need - 1) == 3 and f(slots=1001 + 256 * 32) == 3


def test_copy_rows_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()

    def f(src=fake, ss=None, sn=100, sr=100, sl=fake, dst=fake, ds=None, dn=100, dr=100, dl=fake, n=5, layers=2,
          nbytes=1152, ws=None):
        return lib.mla_copy_rows(src, ss, sn, sr, sl, dst, ds, dn, dr, dl, n, layers, nbytes, ws, None)

    assert f(n=0) == 0 and f(layers=0) == 0 and f(n=0, src=None, dst=None, sl=None, dl=None) == 0
    for bad in (dict(src=None), dict(src=fake + 8), dict(dst=None), dict(dst=fake + 4), dict(sl=None),
                dict(dl=fake + 2), dict(n=-1), dict(layers=-1), dict(sn=0), dict(dn=1 << 31), dict(sr=99), dict(dr=0),
                dict(sr=FAR + 1), dict(ss=fake), dict(ds=fake, nbytes=576), dict(ss=fake, ds=fake),
                dict(ss=fake + 2, ds=fake, nbytes=576), dict(ws=fake + 8)):
        assert f(**bad) == 1, bad
    assert f(nbytes=1024) == 2 and f(nbytes=0) == 2


def test_compact_refuses_bad_arguments(B):
    lib, fake = B.library(), _fake_ptr()
    need = B.slots_workspace_bytes(100)

    def f(kv=fake, sc=None, n=100, rows=100, layers=2, nbytes=576, ip=fake, b=3, idx=fake, m=50, new=fake, live=fake,
          ws=fake, wsb=need):
        return lib.mla_compact_cache(kv, sc, n, rows, layers, nbytes, ip, b, idx, m, new, live, ws, wsb, None)

    for bad in (dict(kv=None), dict(kv=fake + 8), dict(sc=fake + 2), dict(sc=fake, nbytes=1152), dict(n=0),
                dict(n=1 << 31), dict(rows=99), dict(layers=0), dict(ip=None), dict(b=-1), dict(idx=None), dict(m=-1),
                dict(m=1 << 31), dict(new=None), dict(new=fake + 2), dict(live=None), dict(ws=None), dict(ws=fake + 8)):
        assert f(**bad) == 1, bad
    assert f(nbytes=1000) == 2 and f(wsb=need - 1) == 3


def test_binding_checks_types_and_shapes(B):
    torch = pytest.importorskip("torch")
    i32, f32 = torch.int32, torch.float32
    z = lambda *shape, dtype=i32: torch.zeros(shape, dtype=dtype)    # noqa: E731  (host tensors: refused at the latest)
    t, ws = z(2, 3, 7, dtype=f32), z(4096, dtype=torch.uint8)
    calls = [
        lambda: B.verify_drafts(t.double(), z(2, 3), z(2, 3, dtype=f32), z(2, 3), z(2), z(2)),
        lambda: B.verify_drafts(t, z(2, 4), z(2, 3, dtype=f32), z(2, 3), z(2), z(2)),
        lambda: B.verify_drafts(t.transpose(1, 2), z(2, 7), z(2, 7, dtype=f32), z(2, 7), z(2), z(2)),
        lambda: B.verify_drafts(t, z(2, 3), z(2, 3, dtype=f32), z(2, 3), z(2), z(2), draft_probs=t[:1]),
        lambda: B.verify_drafts(t, z(2, 3), z(2, 3, dtype=f32), z(2, 3), z(2), z(2)),
        lambda: B.repack_requests(z(0), z(5), z(1), z(2), z(5), 10, ws),
        lambda: B.repack_requests(z(2), z(5), z(1), z(1), z(5), 10, ws),
        lambda: B.repack_requests(z(2), z(5), z(1), z(2), z(5), 10, ws, path=z(1, 2)),
        lambda: B.repack_requests(z(2), z(5), z(1), z(2), z(5), 10, ws, freed=z(5)),
        lambda: B.copy_rows(z(4, 576, dtype=f32), z(1), z(4, 576, dtype=f32), z(1)),
        lambda: B.copy_rows(z(4, 576, dtype=torch.uint8), z(1), z(2, 4, 576, dtype=torch.uint8), z(1)),
        lambda: B.copy_rows(z(4, 576, dtype=torch.uint8), z(1), z(4, 576, dtype=torch.bfloat16), z(1)),
        lambda: B.copy_rows(z(4, 576, dtype=torch.bfloat16), z(1), z(4, 576, dtype=torch.bfloat16), z(1),
                            src_scales=z(4, dtype=f32), dst_scales=z(4, dtype=f32)),
        lambda: B.copy_rows(z(4, 576, dtype=torch.uint8), z(2), z(4, 576, dtype=torch.uint8), z(1)),
        lambda: B.compact_cache(z(4, 1152, dtype=torch.uint8), z(2), z(3), z(3), z(1), ws),
        lambda: B.compact_cache(z(4, 576, dtype=torch.uint8), z(2), z(3), z(2), z(1), ws),
        lambda: B.compact_cache(z(4, 576, dtype=torch.uint8)[:, ::2], z(2), z(3), z(3), z(1), ws),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")


# ------------------------------------------------------------------ the oracle, by hand

def test_oracle_walks_a_sampled_chain():
    t = np.zeros((1, 3, 4), dtype=np.float32)
    q = np.zeros_like(t)
    t[0] = [[.1, .2, .3, .4], [.25, .25, .25, .25], [0, 0, 1, 0]]
    q[0, 1:] = [[.5, .5, 0, 0], [.4, .3, .2, .1]]
    # u_1 q_1(1) = .39 * .5 < t_0(1) = .2: taken; u_2 q_2(0) = .7 * .4 > t_1(0) = .25: rejected, and what is left of
    # t_1 is max(t_1 - q_2, 0) = [0, 0, .05, .15]
    args = t, np.array([[9, 1, 0]]), np.array([[.3, .39, .7]]), q
    path, n, nxt, bad = S.verify(*args)
    assert path.tolist() == [[0, 1, -1]] and n.tolist() == [2] and nxt.tolist() == [3] and not bad
    args[2][0] = [.2, .39, .7]
    assert S.verify(*args)[2].tolist() == [2]
    args[2][0] = [.5, .41, .0]                      # .41 * .5 > .2: left of t_0 is [0, 0, .3, .4]
    path, n, nxt, _ = S.verify(*args)
    assert path.tolist() == [[0, -1, -1]] and n.tolist() == [1] and nxt.tolist() == [3]


def test_oracle_walks_a_tree():
    t = np.zeros((1, 4, 4), dtype=np.float32)
    t[0] = [[.5, .25, .25, 0], [1, 0, 0, 0], [0, .5, .5, 0], [0, 0, 0, 1]]
    tok, par = np.array([[0, 0, 1, 2]]), np.array([[-1, 0, 0, 2]])
    # child 1: u = .6 > .5; child 2: .4 * (1 - .5) < .25: taken; its child 3: .5 of token 2, u = .9 > .5: rejected, and
    # t_2 without token 2 is token 1
    path, n, nxt, _ = S.verify(t, tok, np.array([[.9, .6, .4, .9]]), parents=par)
    assert path.tolist() == [[0, 2, -1, -1]] and n.tolist() == [2] and nxt.tolist() == [1]
    # both children rejected: t_0 without tokens 0 and 1
    path, n, nxt, _ = S.verify(t, tok, np.array([[.0, .6, .6, .9]]), parents=par)
    assert path.tolist() == [[0, -1, -1, -1]] and nxt.tolist() == [2]
    # a bad parent is reached by nobody, a bad token is not taken
    path, n, nxt, bad = S.verify(t, np.array([[0, 9, 1, 2]]), np.zeros((1, 4)), parents=np.array([[-1, 0, 5, 0]]))
    assert path.tolist() == [[0, 3, -1, -1]] and bad == {"tree", "token"}


def test_oracle_lists_and_compaction():
    ip, idx = [0, 4, 6, 9], [5, 6, 7, 8, 1, 2, 5, 6, 3]
    rows, freed = S.repack(ip, idx, [2, 0, 0, -1])
    assert rows == [[5, 6, 3], [5, 6, 7, 8], [5, 6, 7, 8], []] and freed == [1, 2]
    rows, freed = S.repack(ip, idx, [0, 2], np.array([[0, 2, -1], [0, -1, -1], [0, 1, 2]]), [2, 1, 3])
    assert rows == [[5, 6, 8], [5, 6, 3]] and freed == [1, 2, 7]
    assert S.compact([7, 1, 9, 1, 0, 3]) == (5, {7: 2, 9: 4})
