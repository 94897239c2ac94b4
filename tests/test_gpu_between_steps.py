"""GPU tests of what happens between two decode steps: draft verification,
request lists, row moves - each against the 64-bit oracle, and as they run
together around the decode.  All results are whole numbers or copied bytes."""
import math

import numpy as np
import pytest

from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu


def _t():
    import torch
    from mla_latent_kv_absorbed_gb300 import binding
    return torch, binding


def _dev(a, dtype=np.int32):
    torch, _ = _t()
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


# ------------------------------------------------------------------ verification

def _rows(rng, *shape):
    x = np.exp(rng.standard_normal(shape) * 3)
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def _tree(rng, B, W, wide):
    return np.array([[-1] + [int(rng.integers(max(0, i - wide), i)) for i in range(1, W)] for _ in range(B)])


def _verify(target, tokens, u, draft=None, parents=None, ws=None, stream=None):
    torch, B = _t()
    b, w, _ = target.shape
    path = torch.full((b, w), -7, dtype=torch.int32, device="cuda")
    acc, nxt = (torch.full((b,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    B.verify_drafts(target, _dev(tokens), _dev(u, np.float32), path, acc, nxt, draft_probs=draft,
                    parents=None if parents is None else _dev(parents), workspace=ws, stream=stream)
    if stream is not None:
        stream.synchronize()
    return path.cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy()


def _same(got, ref):
    for g, r, what in zip(got, ref, ("path", "accepted", "next")):
        assert np.array_equal(g, r), (what, np.argwhere(g != r)[:5], g[g != r][:5], r[g != r][:5])


@pytest.mark.parametrize("B,W,V", [(1, 1, 1), (1, 1, 7), (2, 2, 3), (5, 4, 300), (3, 5, 32001), (40, 8, 1000),
                                   (2, 64, 4097), (300, 3, 2050), (1, 2, 200001), (9, 33, 31)])
@pytest.mark.parametrize("form", ["sampled", "chain", "tree"])
def test_verify(B, W, V, form):
    rng = np.random.default_rng(B * W + V)
    target = _rows(rng, B, W, V)
    draft = parents = None
    if form == "sampled":
        draft = _rows(rng, B, W, V) * np.float32(0.5) + target[:, [max(i - 1, 0) for i in range(W)]] * np.float32(0.5)
        pick = draft
    else:
        parents = _tree(rng, B, W, 5) if form == "tree" else None
        pick = target[:, [max(i - 1, 0) for i in range(W)]] if parents is None else \
            np.take_along_axis(target, np.maximum(parents, 0)[..., None], 1)
    # drafts that the target likes about as often as not; among siblings one token may come twice
    tokens = (np.cumsum(pick, -1) > rng.random((B, W, 1)) * pick.sum(-1, keepdims=True)).argmax(-1)
    u = rng.random((B, W)).astype(np.float32)
    u[::3, 0] = 0.0
    ref = S.verify(target, tokens, u, draft, parents)
    got = _verify(_dev(target, np.float32), tokens, u, None if draft is None else _dev(draft, np.float32), parents)
    _same(got, ref)


def test_verify_keeps_the_targets_distribution():
    # sampled and chosen drafts alike: over many numbers the first token after draft 0 is distributed as the target
    rng = np.random.default_rng(1)
    n, V = 20000, 5
    p = np.array([0.4, 0.3, 0.2, 0.1, 0.0], dtype=np.float32)
    q = np.array([0.1, 0.2, 0.3, 0.2, 0.2], dtype=np.float32)
    target = np.broadcast_to(p, (n, 3, V))
    for form in ("sampled", "tree"):
        u = rng.random((n, 3)).astype(np.float32)
        tokens = np.zeros((n, 3), dtype=np.int64)
        if form == "sampled":
            tokens[:, 1] = (np.cumsum(q) > rng.random((n, 1)) * q.sum()).argmax(-1)
            tokens[:, 2] = 0
            got = _verify(_dev(target, np.float32), tokens, u, _dev(np.broadcast_to(q, (n, 3, V)), np.float32))
        else:
            tokens[:, 1:] = [2, 0]
            got = _verify(_dev(target, np.float32), tokens, u, parents=np.tile([-1, 0, 0], (n, 1)))
        path, acc, nxt = got
        first = np.where(acc > 1, tokens[np.arange(n), np.maximum(path[:, 1], 0)], nxt)
        share = np.bincount(first, minlength=V) / n
        # five standard deviations of a share of n draws
        assert (np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / n) + 1e-12).all(), (form, share)


def test_verify_at_the_borders():
    # equal numbers do not pass; a ratio of one, zeros on either side, all mass on one token
    V = 8
    t = np.zeros((6, 2, V), dtype=np.float32)
    q = np.zeros((6, 2, V), dtype=np.float32)
    u = np.zeros((6, 2), dtype=np.float32)
    tokens = np.tile([0, 3], (6, 1))
    t[:, 0, 3], t[:, 0, 5], q[:, 1, 3] = 0.5, 0.5, 1.0
    u[0, 1] = 0.5                                   # 0.5 * 1 < 0.5 does not hold: rejected, 5 is left
    u[1, 1] = np.nextafter(np.float32(0.5), np.float32(0))     # accepted
    t[2, 0], q[2, 1] = 0, 0
    t[2, 0, 1], q[2, 1, 3] = 1.0, 0.25              # t(x) = 0: rejected at u = 0
    t[3, 0, 3], t[3, 0, 5], q[3, 1, 3] = 1.0, 0.0, 0.0        # q(x) = 0 < t(x): accepted at any u
    u[3, 1] = 0.999
    q[4, 1] = t[4, 0]                               # equal rows: a ratio of one
    u[4, 1] = 0.9999999
    t[5, 0], q[5, 1] = 0, 0
    q[5, 1, 3] = 1.0                                # nothing there at all: rejected, and nothing left
    t[:, 1, 6] = 1.0
    got = _verify(_dev(t, np.float32), tokens, u, _dev(q, np.float32))
    _same(got, S.verify(t, tokens, u, q))
    assert got[1].tolist() == [1, 2, 1, 2, 2, 1] and got[2].tolist() == [5, 6, 1, 6, 6, -1]


def test_verify_of_odd_values():
    # NaN, infinities, negative values and numbers outside [0, 1)
    rng = np.random.default_rng(2)
    B, W, V = 24, 4, 515
    t, q = _rows(rng, B, W, V), _rows(rng, B, W, V)
    for x in (t, q):
        x[rng.random(x.shape) < 0.05] = np.nan
        x[rng.random(x.shape) < 0.05] = -1.0
        x[rng.random(x.shape) < 0.01] = np.inf
        x[rng.random(x.shape) < 0.01] = -np.inf
    u = rng.random((B, W)).astype(np.float32)
    u[0], u[1], u[2], u[3, 0], u[4, 0] = np.nan, 1.0, -0.5, 7.0, -3.0
    tokens = rng.integers(0, V, (B, W))
    for kw in (dict(draft=q), dict(), dict(parents=_tree(rng, B, W, 3))):
        dev = {k: _dev(v, np.float32) if k == "draft" else v for k, v in kw.items()}
        _same(_verify(_dev(t, np.float32), tokens, u, **dev), S.verify(t, tokens, u, **kw))


def test_verify_records_bad_tokens_and_trees():
    torch, B = _t()
    rng = np.random.default_rng(3)
    t = _rows(rng, 4, 6, 64)
    u = (rng.random((4, 6)) * 0.01).astype(np.float32)
    tokens = rng.integers(0, 64, (4, 6))
    tokens[:, 0] = -5                                # (the first is not looked at)
    parents = _tree(rng, 4, 6, 2)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    _same(_verify(_dev(t, np.float32), tokens, u, parents=parents, ws=ws), S.verify(t, tokens, u, parents=parents))
    assert B.check_errors(ws) == 0
    tokens[1, 2], tokens[2, 1], tokens[3, 5] = 64, -1, 2 ** 31 - 1
    _same(_verify(_dev(t, np.float32), tokens, u, parents=parents, ws=ws), S.verify(t, tokens, u, parents=parents))
    assert B.check_errors(ws) == 6
    tokens = rng.integers(0, 64, (4, 6))
    parents[0, 0], parents[1, 3], parents[2, 2], parents[3, 4] = 0, 3, -2, -1
    _same(_verify(_dev(t, np.float32), tokens, u, parents=parents, ws=ws), S.verify(t, tokens, u, parents=parents))
    assert B.check_errors(ws) == 8


@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_verify_of_strided_and_broadcast_rows(off):
    # rows cut out of a wider vocabulary, at any alignment; one distribution for all requests
    torch, _ = _t()
    rng = np.random.default_rng(off)
    B, W, V = 6, 3, 4099
    wide = _dev(_rows(rng, B, W, V + 9), np.float32)
    t = wide[..., off:off + V]
    q = _dev(_rows(rng, W, V), np.float32)[None].expand(B, -1, -1)
    tokens, u = rng.integers(0, V, (B, W)), rng.random((B, W)).astype(np.float32)
    tokens[:, 1] = t[:, 0].argmax(-1).cpu().numpy()
    ref = S.verify(t.cpu().numpy(), tokens, u, q.cpu().numpy())
    _same(_verify(t, tokens, u, q), ref)
    swapped = wide.transpose(0, 1).contiguous().transpose(0, 1)[..., off:off + V]      # rows outside, requests inside
    _same(_verify(swapped, tokens, u, q), ref)


def test_verify_on_a_stream_and_replayed():
    torch, B = _t()
    rng = np.random.default_rng(5)
    t, q = _rows(rng, 7, 5, 2000), _rows(rng, 7, 5, 2000)
    tokens, u = rng.integers(0, 2000, (7, 5)), rng.random((7, 5)).astype(np.float32)
    tokens[:, 1:] = np.argmax(t[:, :-1] - q[:, 1:], -1)
    td, qd, kd, ud = _dev(t, np.float32), _dev(q, np.float32), _dev(tokens), _dev(u, np.float32)
    torch.cuda.synchronize()
    _same(_verify(td, tokens, u, qd, stream=torch.cuda.Stream()), S.verify(t, tokens, u, q))
    path, acc, nxt = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((7, 5), (7,), (7,)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.verify_drafts(td, kd, ud, path, acc, nxt, draft_probs=qd)
    for k in range(2):
        u = rng.random((7, 5)).astype(np.float32)
        ud.copy_(_dev(u, np.float32))
        graph.replay()
        _same([x.cpu().numpy() for x in (path, acc, nxt)], S.verify(t, tokens, u, q))


# ------------------------------------------------------------------ request lists

def _repack(indptr, indices, sources, slots, path=None, accepted=None, room=None, freed_room=None, keep=False, ws=None):
    torch, B = _t()
    fill = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
    if ws is None:
        ws = torch.zeros(B.slots_workspace_bytes(slots), dtype=torch.uint8, device="cuda")
    n = len(indices)
    new_indptr, new_indices = fill(len(sources) + 1), fill(4 * n + 8 if room is None else room)
    freed, count = (None, None) if keep else (fill(n if freed_room is None else freed_room), fill(1))
    B.repack_requests(_dev(indptr), _dev(indices), _dev(sources), new_indptr, new_indices, slots, ws,
                      path=None if path is None else _dev(path), accepted=None if path is None else _dev(accepted),
                      freed=freed, freed_count=count)
    status = B.check_errors(ws)
    assert not ws.any(), "the workspace is empty between calls"
    return [x.cpu().numpy() if x is not None else None for x in (new_indptr, new_indices, freed, count)] + [status]


def _check_repack(got, rows, free):
    new_indptr, new_indices, freed, count, status = got
    flat = [x for mine in rows for x in mine]
    assert new_indptr.tolist() == np.concatenate(([0], np.cumsum([len(r) for r in rows]))).astype(int).tolist()
    assert new_indices[:len(flat)].tolist() == flat and (new_indices[len(flat):] == -9).all()
    if freed is not None:
        assert count[0] == len(free) and freed[:len(free)].tolist() == free and (freed[len(free):] == -9).all()
    assert status == 0


def _lists(rng, lens, slots, shared=0):
    """Distinct slots, but for `shared` first rows that all requests have in common."""
    n = sum(lens)
    idx = rng.permutation(slots)[:n]
    ptr = np.concatenate(([0], np.cumsum(lens)))
    for b in range(len(lens)):
        k = min(shared, lens[b], lens[0])
        idx[ptr[b]:ptr[b] + k] = idx[:k]
    return ptr, idx


@pytest.mark.parametrize("lens,sources", [
    ([5], [0]), ([5], []), ([0], [0, 0]), ([3, 0, 70, 1], [2, 2, 0, -1, 3]), ([300, 1, 2000], [1, -1, 1]),
    ([7] * 300, list(range(299, -1, -1))), ([1025, 4096, 33], [0, 1, 2, 2, 2, 1]), ([40000], [-1]), ([40000, 9], [0, 0, 1]),
])
@pytest.mark.parametrize("shared", [0, 20])
def test_repack(lens, sources, shared):
    rng = np.random.default_rng(len(lens) + shared)
    slots = sum(lens) + 100
    ptr, idx = _lists(rng, lens, slots, shared)
    rows, free = S.repack(ptr, idx, sources)
    _check_repack(_repack(ptr, idx, sources, slots), rows, free)
    _check_repack(_repack(ptr, idx, sources, slots, keep=True), rows, free)


@pytest.mark.parametrize("W", [1, 2, 8, 33, 64])
@pytest.mark.parametrize("B", [1, 5, 200])
def test_repack_of_accepted_drafts(W, B):
    rng = np.random.default_rng(W * B)
    lens = [W + int(x) for x in rng.integers(0, 400, B)]
    lens[0] = W                                      # drafts only
    slots = sum(lens) + 1000
    ptr, idx = _lists(rng, lens, slots)
    accepted = rng.integers(0, W + 1, B)
    path = np.full((B, W), -1)
    for b in range(B):
        path[b, :accepted[b]] = np.sort(rng.choice(W, accepted[b], replace=False))
    sources = [int(x) for x in rng.integers(-1, B, B + 3)]
    _check_repack(_repack(ptr, idx, sources, slots, path, accepted), *S.repack(ptr, idx, sources, path, accepted))


@pytest.mark.parametrize("slots", [1, 31, 32, 33, 1000, 262144, 262145, 2 ** 21 + 5])
def test_repack_frees_whole_pools_of_any_size(slots):
    # every word of the set, its last one included
    n = min(slots, 70000)
    idx = np.unique(np.concatenate((np.linspace(0, slots - 1, n).astype(np.int64), [slots - 1])))
    np.random.default_rng(slots).shuffle(idx)
    ptr = np.array([0, len(idx)])
    _check_repack(_repack(ptr, idx, [-1], slots), [[]], sorted(idx.tolist()))


def test_repack_records_what_does_not_fit_and_goes_on():
    rng = np.random.default_rng(8)
    ptr, idx = _lists(rng, [50, 60], 500)
    got = _repack(ptr, idx, [1, 0], 500, room=70)                       # the second list is cut
    assert got[4] == 3 and got[0].tolist() == [0, 60, 70] and got[1].tolist() == idx[50:].tolist() + idx[:10].tolist()
    got = _repack(ptr, idx, [1], 500, freed_room=7)                     # 50 are free, 7 are listed
    assert got[4] == 3 and got[3][0] == 50 and got[2].tolist() == sorted(idx[:50].tolist())[:7]
    got = _repack(ptr, idx, [1, 2, -2, 0], 500)                         # sources that are none
    assert got[4] == 7 and got[0].tolist() == [0, 60, 60, 60, 110]
    bad = idx.copy()
    bad[3], bad[70] = 500, -4                                           # slots outside the pool
    got = _repack(ptr, bad, [0], 500)
    assert got[4] == 6 and got[1][:50].tolist() == bad[:50].tolist()
    assert got[2][:got[3][0]].tolist() == sorted(x for x in bad[50:].tolist() if x >= 0)
    got = _repack(np.array([0, 50, 111]), idx, [1], 500)                # past the entries
    assert got[4] == 7 and got[0].tolist() == [0, 60]
    got = _repack(np.array([0, 50, 40]), idx, [1, 0], 500)              # falling
    assert got[4] == 7 and got[0].tolist() == [0, 0, 50]
    path, accepted = np.array([[0, 1, 2, 3], [0, 9, -1, 3]]), np.array([5, 2])
    got = _repack(ptr, idx, [0, 1], 500, path, accepted)                # a count and a step that are none
    assert got[4] == 8 and got[0].tolist() == [0, 50, 108]
    got = _repack(np.array([0, 3, 63]), idx, [0, 1], 500, np.zeros((2, 4), int), np.array([1, 1]))
    assert got[4] == 7 and got[0].tolist() == [0, 3, 60]                # fewer rows than drafts: all of them


def test_repack_replayed_and_sharing_a_workspace():
    torch, B = _t()
    rng = np.random.default_rng(9)
    slots, lens = 5000, [700, 20, 1500]
    ptr, idx = _lists(rng, lens, slots)
    ws = torch.zeros(B.slots_workspace_bytes(slots), dtype=torch.uint8, device="cuda")
    fill = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
    dptr, didx, graphs = _dev(ptr), _dev(idx), []
    for sources in ([0, 0, 2], [1, -1, -1]):
        dsrc = _dev(sources)
        out = (fill(4), fill(4500), fill(2220), fill(1))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.repack_requests(dptr, didx, dsrc, out[0], out[1], slots, ws, freed=out[2], freed_count=out[3])
        graphs.append((g, sources, out, dsrc))
    for g, sources, out, _ in graphs * 2:
        g.replay()
        _check_repack([x.cpu().numpy() for x in out] + [B.check_errors(ws)], *S.repack(ptr, idx, sources))
        for x in out:
            x.fill_(-9)


# ---------------------------------------------------------------------- row moves

def _pool(seed, L, N, dtype):
    torch, _ = _t()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if dtype == "bf16":
        return torch.randn((L, N, 576), generator=g, device="cuda").bfloat16(), None
    return (torch.randint(0, 256, (L, N, 576), generator=g, device="cuda", dtype=torch.uint8),
            torch.rand((L, N), generator=g, device="cuda") if dtype == "rows8" else None)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "rows8"])
@pytest.mark.parametrize("L,N,n", [(1, 2, 1), (3, 41, 20), (2, 5000, 2500), (7, 129, 3), (1, 30000, 9999), (3, 18002, 9001),
                                   (8, 5000, 2049)])
def test_copy_rows(L, N, n, dtype):
    torch, B = _t()
    cache, scales = _pool(N, L, N, dtype)
    rng = np.random.default_rng(n)
    order = rng.permutation(N)
    src, dst = order[:n].copy(), order[n:2 * n]
    src[n // 2:] = src[:n - n // 2]                   # a source may come twice
    ref, ref_s = cache.clone(), None if scales is None else scales.clone()
    ref[:, _dev(dst).long()] = cache[:, _dev(src).long()]
    if scales is not None:
        ref_s[:, _dev(dst).long()] = scales[:, _dev(src).long()]
    B.copy_rows(cache, _dev(src), cache, _dev(dst), src_scales=scales, dst_scales=scales)
    assert torch.equal(cache, ref) and (scales is None or torch.equal(scales, ref_s))


def test_copy_rows_between_pools_and_out_of_range():
    torch, B = _t()
    a, sa = _pool(1, 4, 60, "rows8")
    b, sb = _pool(2, 4, 100, "rows8")
    part, ps = a[1:3, :50], sa[1:3, :50]              # two layers, a part of the slots
    was, was_s = b.clone(), sb.clone()
    src, dst = [0, 49, 50, 7, -1, 3], [99, 0, 5, 100, 6, 2]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.copy_rows(part, _dev(src), b[2:], _dev(dst), src_scales=ps, dst_scales=sb[2:], workspace=ws)
    assert B.check_errors(ws) == 6
    for s, d in ((0, 99), (49, 0), (3, 2)):
        was[2:, d], was_s[2:, d] = a[1:3, s], sa[1:3, s]
    assert torch.equal(b, was) and torch.equal(sb, was_s)
    one, _ = _pool(3, 1, 10, "bf16")                  # a cache of one layer
    B.copy_rows(one[0], _dev([1]), one[0], _dev([9]))
    assert torch.equal(one[0, 1], one[0, 9])


@pytest.mark.parametrize("dtype", ["bf16", "rows8"])
def test_copy_many_rows_skips_those_out_of_range(dtype):
    torch, B = _t()
    cache, scales = _pool(7, 4, 12000, dtype)
    ref, ref_s = cache.clone(), None if scales is None else scales.clone()
    order = np.random.default_rng(7).permutation(12000)
    src, dst = order[:5000].copy(), order[5000:10000].copy()
    src[::7], dst[3::11] = 12000, -1
    ok = (src < 12000) & (dst >= 0)
    ref[:, _dev(dst[ok]).long()] = cache[:, _dev(src[ok]).long()]
    if scales is not None:
        ref_s[:, _dev(dst[ok]).long()] = scales[:, _dev(src[ok]).long()]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.copy_rows(cache, _dev(src), cache, _dev(dst), src_scales=scales, dst_scales=scales, workspace=ws)
    assert B.check_errors(ws) == 6
    assert torch.equal(cache, ref) and (scales is None or torch.equal(scales, ref_s))


def _compact(idx, N, L=2, dtype="bf16", extra=0, in_place=False, ws=None, seed=0):
    torch, B = _t()
    cache, scales = _pool(seed, L, N, dtype)
    was, was_s = cache.clone(), None if scales is None else scales.clone()
    n_live, to = S.compact(idx)
    ptr = [0, len(idx) // 3, len(idx)]
    indices = _dev(list(idx) + [-9] * extra)
    out = indices if in_place else torch.full_like(indices, -9)
    count = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.zeros(B.slots_workspace_bytes(N), dtype=torch.uint8, device="cuda")
    B.compact_cache(cache, _dev(ptr), indices, out, count, ws, kv_scales=scales)
    assert B.check_errors(ws) == 0
    assert count.item() == n_live
    assert out.tolist() == [to.get(int(x), int(x)) for x in idx] + [-9] * extra
    if to:
        a, z = (torch.tensor(list(x), device="cuda") for x in (to.keys(), to.values()))
        was[:, z] = was[:, a]
        if scales is not None:
            was_s[:, z] = was_s[:, a]
    assert torch.equal(cache, was) and (scales is None or torch.equal(scales, was_s))
    return ws


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "rows8"])
@pytest.mark.parametrize("N,live", [(1, 0), (1, 1), (32, 32), (33, 33), (40, 7), (100, 64), (4099, 1300), (4099, 4000)])
def test_compact(N, live, dtype):
    rng = np.random.default_rng(N + live)
    idx = rng.permutation(N)[:live]
    if live > 4:
        idx = np.concatenate((idx, idx[:live // 2]))   # a shared prefix
    _compact(idx, N, dtype=dtype, extra=5)
    _compact(idx, N, dtype=dtype, in_place=True)


@pytest.mark.parametrize("where", ["low", "high", "every second", "one far"])
def test_compact_of_patterns(where):
    N = 70000
    idx = {"low": np.arange(1000), "high": np.arange(N - 999, N), "every second": np.arange(0, N, 2),
           "one far": np.concatenate((np.arange(63), [N - 1]))}[where]
    _compact(np.random.default_rng(1).permutation(idx), N, L=1, dtype="fp8")


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "rows8"])
@pytest.mark.parametrize("live", [5000, 20000, 39000])
def test_compact_of_many_rows(live, dtype):
    _compact(np.random.default_rng(live).permutation(40000)[:live], 40000, L=3, dtype=dtype)


def test_compact_of_a_pool_wider_than_one_pass():
    rng = np.random.default_rng(3)
    _compact(rng.permutation(300001)[:5000], 300001, L=1, dtype="fp8")


def test_compact_takes_a_workspace_again_and_records_bad_slots():
    torch, B = _t()
    rng = np.random.default_rng(4)
    ws = _compact(rng.permutation(900)[:400], 900)
    _compact(rng.permutation(900)[:100], 900, ws=ws, seed=1)
    _compact(rng.permutation(500)[:300], 500, ws=ws, seed=2)           # a smaller pool
    cache, _ = _pool(5, 1, 50, "bf16")
    idx = _dev([40, 50, -1, 2])
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.compact_cache(cache, _dev([0, 4]), idx, idx, count, ws)
    assert B.check_errors(ws) == 6 and count.item() == 2 and idx.tolist() == [1, 50, -1, 0]


# ------------------------------------------------------------------ as they are used

def test_one_workspace_serves_pools_of_two_sizes():
    torch, B = _t()
    ws = torch.zeros(B.slots_workspace_bytes(50000), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(9)
    for N in (50000, 300, 50000, 7000, 50000):
        idx = rng.permutation(N)[:2 * N // 3].astype(np.int32)
        cache = torch.zeros((N, 576), dtype=torch.uint8, device="cuda")
        new, live, ip = _dev(idx * 0), _dev([0]), _dev([0, len(idx)])
        B.compact_cache(cache, ip, _dev(idx), new, live, ws)
        n, to = S.compact(idx)
        assert int(live) == n and new.cpu().tolist() == [to.get(int(x), int(x)) for x in idx]
        nip, nidx, freed, count = _dev([0]), _dev([0]), _dev(np.full(N, -1)), _dev([0])
        B.repack_requests(ip, _dev(idx), _dev([]), nip, nidx, N, ws, freed=freed, freed_count=count)
        assert int(count) == len(idx) and freed[:len(idx)].cpu().tolist() == sorted(idx.tolist())
    assert B.check_errors(ws) == 0


@pytest.mark.parametrize("H,form", [(16, "tree"), (8, "chain")])
def test_a_speculative_step(H, form):
    """Drafts appended, attended to in one pass, verified; the lists cut, a request forked and one freed, the pool made
    contiguous, and the next step decoded: over the rewritten lists it gives what it gives over lists made by hand."""
    torch, B = _t()
    rng = np.random.default_rng(H)
    W = 8 if form == "tree" else 4
    heads = H // W if form == "tree" else 4
    slots, lens = 3000, [200, 65, 0, 700]
    lens = [x + W for x in lens]
    ptr, idx = _lists(rng, lens, slots)
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    cache = rand(slots, 576).bfloat16()
    Bn = len(lens)
    parents = _tree(rng, Bn, W, 3)
    dptr, didx = _dev(ptr), _dev(idx)
    rows = rand(Bn * W, 576).bfloat16()
    at = np.concatenate([idx[ptr[b + 1] - W:ptr[b + 1]] for b in range(Bn)])
    B.append_kv(cache, _dev(at), rows)
    n_heads = W * heads
    dec = B.Decoder(ptr.astype(np.int32), n_heads)
    q, r = rand(Bn, W, heads, 512).bfloat16(), rand(Bn, W, heads, 64).bfloat16()
    out, lse = torch.empty((Bn, W, heads, 512), device="cuda"), torch.empty((Bn, W, heads), device="cuda")
    sm = 1 / math.sqrt(192)
    if form == "tree":
        masks = torch.zeros((Bn, W), dtype=torch.int64, device="cuda")
        B.decode_run_tree(dec.plan_host, dec.plan_dev, _dev(parents), masks, q, r, cache, dptr, didx, sm, out, lse,
                          dec.workspace)
    else:
        B.decode_run_multi_query(dec.plan_host, dec.plan_dev, W, q, r, cache, dptr, didx, sm, out, lse, dec.workspace)
    assert dec.check() == 0
    head = rand(heads * 512, 999) / 20                                # what turns the attention's output into logits
    target = torch.softmax(out.flatten(2) @ head, -1).contiguous()
    up = parents if form == "tree" else np.tile(np.arange(-1, W - 1), (Bn, 1))
    tokens = np.take_along_axis(target.argmax(-1).cpu().numpy(), np.maximum(up, 0), 1)
    u = rng.random((Bn, W)).astype(np.float32)
    path, acc, nxt = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((Bn, W), (Bn,), (Bn,)))
    B.verify_drafts(target, _dev(tokens), _dev(u, np.float32), path, acc, nxt,
                    parents=_dev(parents) if form == "tree" else None)
    ref = S.verify(target.cpu().numpy(), tokens, u, parents=parents if form == "tree" else None)
    _same([x.cpu().numpy() for x in (path, acc, nxt)], ref)
    sources = [3, 0, 3]
    ws = torch.zeros(B.slots_workspace_bytes(slots), dtype=torch.uint8, device="cuda")
    fill = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
    nptr, nidx, freed, count = fill(4), fill(2 * len(idx)), fill(len(idx)), fill(1)
    B.repack_requests(dptr, didx, _dev(sources), nptr, nidx, slots, ws, path=path, accepted=acc, freed=freed,
                      freed_count=count)
    want, free = S.repack(ptr, idx, sources, ref[0], ref[1])
    _check_repack([x.cpu().numpy() for x in (nptr, nidx, freed, count)] + [B.check_errors(ws)], want, free)
    # the next step over lists made by hand, and over the compacted pool
    flat = np.array([x for mine in want for x in mine])
    hand = np.concatenate(([0], np.cumsum([len(x) for x in want]))).astype(np.int32)
    Hn = 16
    qn, qr = rand(3, Hn, 512).bfloat16(), rand(3, Hn, 64).bfloat16()
    results = []
    for k in range(2):
        if k:
            B.compact_cache(cache, nptr, nidx, nidx, count, ws)
            assert B.check_errors(ws) == 0 and count.item() == len(set(flat.tolist()))
            assert nidx[:len(flat)].max().item() == count.item() - 1
        d2 = B.Decoder(hand, Hn)
        o, l = torch.empty((3, Hn, 512), device="cuda"), torch.empty((3, Hn), device="cuda")
        d2.run(qn, qr, cache, nptr, nidx if k else _dev(flat), sm, o, l)
        assert d2.check() == 0
        results.append((o, l))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
