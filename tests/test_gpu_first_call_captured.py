"""GPU test: the library's first calls in a process are captured ones (kernels are
loaded, attributes set and clusters asked for inside the capture), then replayed."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys
sys.path.insert(0, sys.argv[1])
import numpy as np, torch
from mla_latent_kv_absorbed_gb300 import binding as B
from oracle import serving_oracle as S
rng = np.random.default_rng(3)
N, L, H, W, V = 40000, 1, 16, 4, 500
dev = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).cuda()
fill = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")
lens = [300 + W, 20 + W, 25000 + W]
ptr, idx = np.concatenate(([0], np.cumsum(lens))), rng.permutation(N)[:sum(lens)]
codes = torch.randint(0, 64, (L, N, 576), device="cuda", dtype=torch.uint8)
scales = torch.rand((L, N), device="cuda") + 0.5
was, was_s = codes.clone(), scales.clone()
target = torch.softmax(torch.randn(3, W, V, device="cuda"), -1)
tokens, u = rng.integers(0, V, (3, W)), rng.random((3, W)).astype(np.float32)
dptr, didx, dtok, du, dsrc = dev(ptr), dev(idx), dev(tokens), dev(u, np.float32), dev([2, 0])
path, acc, nxt = fill(3 * W).view(3, W), fill(3), fill(3)
nptr, nidx, freed, count, live = fill(3), fill(len(idx)), fill(len(idx)), fill(1), fill(1)
ws = torch.zeros(B.slots_workspace_bytes(N), dtype=torch.uint8, device="cuda")
plan = B.decode_plan(ptr, H)[0]
pd, wd = torch.from_numpy(plan).cuda(), torch.zeros(B.decode_fp8_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
qn, qr = torch.randn(3, H, 512, device="cuda").bfloat16(), torch.randn(3, H, 64, device="cuda").bfloat16()
out, lse = torch.empty(3, H, 512, device="cuda"), torch.empty(3, H, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.decode_run_fp8_rows(plan, pd, qn, qr, codes[0], scales[0], dptr, didx, 0.01, out, lse, wd)
    B.verify_drafts(target, dtok, du, path, acc, nxt)
    B.repack_requests(dptr, didx, dsrc, nptr, nidx, N, ws, path=path, accepted=acc, freed=freed, freed_count=count)
    B.compact_cache(codes, nptr, nidx, nidx, live, ws, kv_scales=scales)
g.replay()
torch.cuda.synchronize()
assert B.check_errors(ws) == 0 and B.check_errors(wd) == 0
p, a, x, _ = S.verify(target.cpu().numpy(), tokens, u)
assert (path.cpu().numpy() == p).all() and (acc.cpu().numpy() == a).all() and (nxt.cpu().numpy() == x).all()
rows, free = S.repack(ptr, idx, [2, 0], p, a)
flat = [s for r in rows for s in r]
n, to = S.compact(flat)
assert freed[:count.item()].tolist() == free and live.item() == n
assert nidx[:len(flat)].tolist() == [to.get(s, s) for s in flat]
assert torch.equal(codes[0, nidx[:len(flat)].long()], was[0, dev(flat).long()])
assert torch.equal(scales[0, nidx[:len(flat)].long()], was_s[0, dev(flat).long()])
for b in range(3):
    at = dev(idx[ptr[b]:ptr[b + 1]]).long()
    x = was[0, at].view(torch.float8_e4m3fn).double() * was_s[0, at].double()[:, None]
    s = (torch.cat((qn[b], qr[b]), -1).double() @ x.t()) * 0.01
    ref = torch.softmax(s, -1) @ x[:, :512]
    assert ((out[b].double() - ref).norm() <= 1e-3 * ref.norm()), b
print("fine")
"""


def test_first_calls_in_a_capture():
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]
