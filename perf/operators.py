"""The prompt side of latent attention: what its operators are asked to do, and their plain forms.

Four operators, each named by a case's "op":

  rope_query   rotary positions on the 64-wide part of every head's query, in a dense copy;
               with "split" the rest of the head is laid out dense beside it, as the query
               absorption takes it;
  rope_append  a step's or a prompt's rows (512-wide latent, 64-wide rope key) on their way into
               the cache: RMS norm of the latent, rotation of the key, write to the row's slot of
               a bf16 or an FP8 (E4M3) cache;
  expand       cached rows, named by slot, to every head's keys (c . w_kc[h]^T) and values
               (c . w_vc[h]), with the rope key all heads share;
  prefill      attention of ragged sequences over expanded keys (128 per head and 64 shared) and
               values: causal, aligned at the sequences' ends, or full; output and log-sum-exp.

`own` says which side runs: the plain forms below (elementary torch operations in 32 bits, angles
in 64), or the library's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

ROPE, NOPE, LATENT, ROW = 64, 128, 512, 576
THETA, FACTOR, ORIGINAL, FAST, SLOW = 10000.0, 40.0, 4096, 32.0, 1.0   # rotary base and YaRN scaling
EPS = 1e-6
KV_SCALE = 2.0 ** -5                                                     # FP8 cache: value = code x scale
SM_SCALE = 1.0 / math.sqrt(192.0)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the query of a decode step of 64 requests: rotated, and split for the absorption
        dict(name="rope_query_step", op="rope_query", tokens=64, heads=128, nope=128, split=True, interleaved=True,
             scaling="yarn", near=False),
        # the queries of a long prompt, only the rotary part rewritten
        dict(name="rope_query_prompt", op="rope_query", tokens=8191, heads=128, nope=128, split=False,
             interleaved=False, scaling="none", near=True),
        # the smallest call: four requests' new rows, where latency is all
        dict(name="rope_append_step", op="rope_append", tokens=4, slots=512, fp8=False, norm=True, interleaved=True,
             scaling="yarn", near=False, stride=576),
        # a prompt's rows, cut out of the wider projection that also holds the query's low-rank part
        dict(name="rope_append_prompt", op="rope_append", tokens=16384, slots=20000, fp8=False, norm=True,
             interleaved=True, scaling="yarn", near=True, stride=2112),
        # the same into an FP8 cache, half layout
        dict(name="rope_append_fp8", op="rope_append", tokens=5000, slots=8192, fp8=True, norm=True,
             interleaved=False, scaling="linear", near=True, stride=576),
        # a short prompt of the 16-head shape: two tiles of rows and one row more
        dict(name="expand_short", op="expand", tokens=257, heads=16, slots=4096, fp8=False),
        # a prompt of the 128-head shape
        dict(name="expand_prompt", op="expand", tokens=4096, heads=128, slots=8192, fp8=False),
        # a cached prefix in FP8, for a chunk that continues it
        dict(name="expand_fp8", op="expand", tokens=8191, heads=32, slots=16384, fp8=True),
        # four short prompts: the smallest attention
        dict(name="prefill_tiny", op="prefill", lengths="1 7 33 100", context="0 0 0 0", heads=32, causal=True),
        # one prompt of the 128-head shape
        dict(name="prefill_prompt", op="prefill", lengths="4096", context="0", heads=128, causal=True),
        # a batch of ragged prompts: some continue a cached context, one is empty, one is a single token, one
        # lost the oldest of its keys (a negative context), so that its first rows see nothing
        dict(name="prefill_ragged", op="prefill", heads=32, causal=True,
             lengths="1500 1 640 2047 333 16 0 1024 129 800 257 64", context="0 2000 0 0 512 1500 77 1 1300 0 64 -20"),
        # a short chunk over long cached contexts: few rows, many keys
        dict(name="prefill_chunk", op="prefill", lengths="64 64", context="65472 32000", heads=16, causal=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_query", "rope_append", "rope_append", "expand", "expand", "prefill", "prefill", "prefill"])
    if op == "rope_query":
        heads = rng.choice([16, 24, 32, 64, 128])
        return dict(op=op, tokens=max(1, _log_uniform(rng, 1, 8191 * 128 // heads // 2)), heads=heads,
                    nope=rng.choice([64, 128, 192]), split=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "yarn"]), near=rng.random() < 0.5)
    if op == "rope_append":
        tokens = _log_uniform(rng, 1, 16384)
        return dict(op=op, tokens=tokens, slots=tokens + rng.randint(1, 4000), fp8=rng.random() < 0.5,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "yarn"]), near=rng.random() < 0.5,
                    stride=rng.choice([576, 584, 1344, 2112]))
    if op == "expand":
        heads = rng.choice([1, 5, 16, 32, 128])
        tokens = _log_uniform(rng, 1, 4096 * 128 // max(heads, 32))
        return dict(op=op, tokens=tokens, heads=heads, slots=tokens + rng.randint(1, 4000), fp8=rng.random() < 0.5)
    n = rng.choice([1, 1, 2, 5, 9])                     # sequences of a prefill
    heads = rng.choice([5, 16, 32, 128])
    most = int(4096 * math.sqrt(128 / heads / n) / 1.5)
    lengths, context = [], []
    for _ in range(n):
        length = _log_uniform(rng, 1, most)
        lengths.append(0 if lengths and rng.random() < 0.05 else length)
        few = -rng.randint(0, length // 2) if rng.random() < 0.1 else 0
        context.append(_log_uniform(rng, 1, max(2, most - length)) if rng.random() < 0.5 else few)
    return dict(op="prefill", lengths=" ".join(map(str, lengths)), context=" ".join(map(str, context)), heads=heads,
                causal=rng.random() < 0.8)


def _lens(case):
    """Queries and keys of each sequence."""
    q = [int(x) for x in case["lengths"].split()]
    return q, [max(0, a + int(b)) for a, b in zip(q, case["context"].split())]


def work(case):
    op = case["op"]
    if op == "rope_query":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * (ROPE + (case["nope"] if case["split"] else 0)) * 4 + 4 * case["tokens"], "flops": n * ROPE * 3}
    if op == "rope_append":
        return {"bytes": case["tokens"] * (ROW * 2 + ROW * (1 if case["fp8"] else 2) + 8) + LATENT * 2 * case["norm"],
                "flops": case["tokens"] * ROW * 4}
    if op == "expand":
        t, h = case["tokens"], case["heads"]
        return {"bytes": t * (ROW * (1 if case["fp8"] else 2) + 4 + ROPE * 2 + h * 2 * NOPE * 2) + h * 2 * NOPE * LATENT * 2,
                "flops": 2.0 * t * h * LATENT * 2 * NOPE}
    ql, kl = _lens(case)
    h, pairs, read = case["heads"], 0, 0
    for a, b in zip(ql, kl):
        first = b - a + 1                                # keys that the first row sees, if any
        pairs += sum(max(0, first + i) for i in range(a)) if case["causal"] else a * b
        read += b if a else 0
    return {"bytes": sum(ql) * h * (192 * 2 + NOPE * 2 + 4) + read * (h * 2 * NOPE * 2 + ROPE * 2),
            "flops": 2.0 * h * pairs * (192 + NOPE)}


# --------------------------------------------------------------- the inputs

def _positions(case, gen):
    """A prompt's positions follow one another; a step's requests are anywhere in their contexts."""
    t = case["tokens"]
    if case["near"]:
        start = torch.randint(0, 1000, (1,), generator=gen, device="cuda", dtype=torch.int32)
        return torch.arange(t, device="cuda", dtype=torch.int32) + start
    return torch.randint(0, 163840, (t,), generator=gen, device="cuda", dtype=torch.int32)


def _normal(gen, *shape, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(torch.bfloat16)


def _codes(gen, rows):
    """E4M3 codes of values about N(0, 1) / KV_SCALE (no NaN code)."""
    x = torch.randn((rows, ROW), generator=gen, device="cuda", dtype=torch.float32) / KV_SCALE
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=case)
    op = case["op"]
    if op == "rope_query":
        t, h, d = case["tokens"], case["heads"], case["nope"] + ROPE
        s.update(q=_normal(gen, t, h, d), positions=_positions(case, gen))
    elif op == "rope_append":
        t, n = case["tokens"], case["slots"]
        wide = _normal(gen, t, case["stride"], scale=2.0)
        s.update(rows=wide[:, case["stride"] - ROW:], positions=_positions(case, gen),
                 slots=torch.randperm(n, generator=gen, device="cuda")[:t].to(torch.int32),
                 weight=(1.0 + 0.1 * _normal(gen, LATENT).float()).to(torch.bfloat16) if case["norm"] else None,
                 cache=_codes(gen, n) if case["fp8"] else _normal(gen, n, ROW))
    elif op == "expand":
        t, h, n = case["tokens"], case["heads"], case["slots"]
        s.update(cache=_codes(gen, n) if case["fp8"] else _normal(gen, n, ROW),
                 indices=torch.randperm(n, generator=gen, device="cuda")[:t].to(torch.int32),
                 w_kc=_normal(gen, h, NOPE, LATENT, scale=LATENT ** -0.5),
                 w_vc=_normal(gen, h, LATENT, NOPE, scale=LATENT ** -0.5))
    else:
        ql, kl = _lens(case)
        h = case["heads"]
        qp, kp = np.cumsum([0] + ql), np.cumsum([0] + kl)
        s.update(q=_normal(gen, int(qp[-1]), h, 192), k_nope=_normal(gen, int(kp[-1]), h, NOPE),
                 k_rope=_normal(gen, int(kp[-1]), ROPE), v=_normal(gen, int(kp[-1]), h, NOPE),
                 q_indptr=torch.tensor(qp, dtype=torch.int32, device="cuda"),
                 kv_indptr=torch.tensor(kp, dtype=torch.int32, device="cuda"), longest=(max(ql), max(kl)))
    if own:
        # what a user's program keeps: the model's rotary frequencies, a batch's plan, buffers it writes into
        from mla_latent_kv_absorbed_gb300 import binding
        bf = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        if op.startswith("rope"):
            s["freqs"] = binding.rope_frequencies(THETA, case["scaling"], FACTOR, ORIGINAL, FAST, SLOW)
        if op == "rope_query":
            s["out"] = bf(t, h, ROPE)
            s["nope"] = bf(t, h, case["nope"]) if case["split"] else None
        elif op == "expand":
            s.update(k=bf(t, h, NOPE), kr=bf(t, ROPE), vo=bf(t, h, NOPE))
        elif op == "prefill":
            s["plan"] = binding.Prefiller(qp, kp, h, causal=case["causal"])
            s["out"] = bf(int(qp[-1]), h, NOPE)
            s["lse"] = torch.empty((int(qp[-1]), h), dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------- the plain forms

def _inv_freq(scaling):
    """The rotary frequencies of the 32 pairs, float64."""
    i = torch.arange(ROPE // 2, dtype=torch.float64, device="cuda")
    f = THETA ** (-2.0 * i / ROPE)
    if scaling == "none":
        return f
    if scaling == "linear":
        return f / FACTOR
    turn = lambda beta: ROPE * math.log(ORIGINAL / (beta * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
    low, high = max(math.floor(turn(FAST)), 0), min(math.ceil(turn(SLOW)), ROPE - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / FACTOR * ramp + f * (1 - ramp)


def _rotate(x, positions, case):
    """x [T, ..., 64] float32, rotated by its positions."""
    angle = positions.double()[:, None] * _inv_freq(case["scaling"])
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (ROPE // 2,)
    cos, sin = angle.cos().float().view(shape), angle.sin().float().view(shape)
    if case["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)


def _plain_rope_query(s):
    case, q = s["case"], s["q"]
    r = _rotate(q[..., case["nope"]:].float(), s["positions"], case).to(torch.bfloat16)
    return [r, q[..., :case["nope"]].contiguous()] if case["split"] else [r]


def _plain_rope_append(s):
    case = s["case"]
    x = s["rows"].float()
    c = x[:, :LATENT]
    if case["norm"]:
        c = c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat((c, _rotate(x[:, LATENT:], s["positions"], case)), dim=1)
    if case["fp8"]:
        code = (row / KV_SCALE).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        s["cache"][s["slots"].long()] = code.view(torch.uint8)
        return s["cache"].view(torch.float8_e4m3fn)
    s["cache"][s["slots"].long()] = row.to(torch.bfloat16)
    return s["cache"]


def _plain_expand(s):
    rows = s["cache"][s["indices"].long()]
    x = rows.view(torch.float8_e4m3fn).float() * KV_SCALE if s["case"]["fp8"] else rows.float()
    c = x[:, :LATENT]
    k = torch.einsum("tr,hnr->thn", c, s["w_kc"].float())
    v = torch.einsum("tr,hrn->thn", c, s["w_vc"].float())
    return [k.to(torch.bfloat16), x[:, LATENT:].to(torch.bfloat16), v.to(torch.bfloat16)]


def _padded(x, indptr, longest):
    """Rows of ragged sequences as [B, longest, ...] float32 (zero past a sequence's end), the places they
    came from, and which of them are there."""
    at = indptr[:-1, None].long() + torch.arange(longest, device=x.device)
    there = at < indptr[1:, None]
    at = at.clamp(max=max(x.shape[0] - 1, 0))
    return x[at].float() * there.view(there.shape + (1,) * (x.dim() - 1)), at, there


def _plain_prefill(s):
    nq, nk = s["longest"]
    q, at, q_there = _padded(s["q"], s["q_indptr"], nq)
    kn, _, k_there = _padded(s["k_nope"], s["kv_indptr"], nk)
    kr, _, _ = _padded(s["k_rope"], s["kv_indptr"], nk)
    v, _, _ = _padded(s["v"], s["kv_indptr"], nk)
    score = torch.einsum("bihd,bjhd->bhij", q[..., :NOPE], kn)
    score += torch.einsum("bihd,bjd->bhij", q[..., NOPE:], kr)
    score *= SM_SCALE
    seen = k_there[:, None, :].expand(-1, nq, -1)
    if s["case"]["causal"]:
        lead = (s["kv_indptr"][1:] - s["kv_indptr"][:-1]) - (s["q_indptr"][1:] - s["q_indptr"][:-1])
        i = torch.arange(nq, device=q.device)[None, :, None] + lead[:, None, None]
        seen = seen & (torch.arange(nk, device=q.device)[None, None, :] <= i)
    score.masked_fill_(~seen[:, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = torch.einsum("bhij,bjhd->bhid", p, v) / total.clamp(min=1e-37)
    lse = (total.log() + top).squeeze(-1)                       # -inf where nothing is seen
    lse = torch.where(total.squeeze(-1) > 0, lse, torch.full_like(lse, -math.inf))
    return [out.transpose(1, 2)[q_there].to(torch.bfloat16), lse.transpose(1, 2)[q_there]]


# ------------------------------------------------------------------ the run

def _own_run(s):
    from mla_latent_kv_absorbed_gb300 import binding
    case = s["case"]
    op = case["op"]
    if op == "rope_query":
        binding.rope_query(s["q"], s["positions"], s["freqs"], s["out"], q_nope=s["nope"],
                           interleaved=case["interleaved"])
        return [s["out"], s["nope"]] if case["split"] else [s["out"]]
    if op == "rope_append":
        if case["fp8"]:
            binding.rope_append_kv_fp8(s["cache"], s["slots"], s["rows"], s["positions"], s["freqs"], KV_SCALE,
                                       norm_weight=s["weight"], eps=EPS, interleaved=case["interleaved"])
            return s["cache"].view(torch.float8_e4m3fn)
        binding.rope_append_kv(s["cache"], s["slots"], s["rows"], s["positions"], s["freqs"],
                               norm_weight=s["weight"], eps=EPS, interleaved=case["interleaved"])
        return s["cache"]
    if op == "expand":
        if case["fp8"]:
            binding.expand_kv_fp8(s["cache"], KV_SCALE, s["indices"], s["w_kc"], s["w_vc"], s["k"], s["kr"], s["vo"])
        else:
            binding.expand_kv(s["cache"], s["indices"], s["w_kc"], s["w_vc"], s["k"], s["kr"], s["vo"])
        return [s["k"], s["kr"], s["vo"]]
    s["plan"].run(s["q"], s["k_nope"], s["k_rope"], s["v"], SM_SCALE, s["out"], s["lse"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own_run(state)
    return {"rope_query": _plain_rope_query, "rope_append": _plain_rope_append, "expand": _plain_expand,
            "prefill": _plain_prefill}[state["case"]["op"]](state)


# ------------------------------------------------------------- in 64 bits

def _exact_rotate(x, positions, case):
    """Rotation as a product of complex numbers, from the definition of the frequencies."""
    freq = []
    for i in range(32):
        f = 1.0 / math.pow(THETA, i / 32.0)
        if case["scaling"] == "linear":
            f /= FACTOR
        elif case["scaling"] == "yarn":
            bound = [32.0 * math.log(ORIGINAL / (2.0 * math.pi * beta)) / math.log(THETA) for beta in (FAST, SLOW)]
            lo, hi = max(0, math.floor(bound[0])), min(63, math.ceil(bound[1]))
            mix = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = (1.0 - mix) * f + mix * (f / FACTOR)
        freq.append(f)
    turn = torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64, device=x.device))
    turn = torch.polar(torch.ones_like(turn), turn).reshape((x.shape[0],) + (1,) * (x.dim() - 2) + (32,))
    pairs = x.reshape(x.shape[:-1] + (32, 2)) if case["interleaved"] else x.reshape(x.shape[:-1] + (2, 32)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    return (y if case["interleaved"] else y.transpose(-1, -2)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope_query":
        q = s["q"].double()
        got = [_exact_rotate(q[..., case["nope"]:], s["positions"], case)]
        return got + [q[..., :case["nope"]]] if case["split"] else got
    if op == "rope_append":
        cache = s["cache"].view(torch.float8_e4m3fn).double() if case["fp8"] else s["cache"].double()
        x = s["rows"].double()
        lat = x[:, :LATENT]
        if case["norm"]:
            lat = lat / (lat.pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
        row = torch.cat((lat, _exact_rotate(x[:, LATENT:], s["positions"], case)), 1)
        cache[s["slots"].long()] = (row / KV_SCALE).clamp(-448, 448) if case["fp8"] else row
        return cache
    if op == "expand":
        rows = s["cache"][s["indices"].long()]
        x = rows.view(torch.float8_e4m3fn).double() * KV_SCALE if case["fp8"] else rows.double()
        k = torch.stack([x[:, :LATENT] @ w.double().t() for w in s["w_kc"]], 1)
        v = torch.stack([x[:, :LATENT] @ w.double() for w in s["w_vc"]], 1)
        return [k, x[:, LATENT:], v]
    ql, kl = _lens(case)
    h = case["heads"]
    out = torch.zeros((sum(ql), h, NOPE), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(ql), h), -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for a, b in zip(ql, kl):
        step = max(1, int(2e9 // max(1, a * b * 8)))
        hidden = None
        if case["causal"]:
            hidden = torch.ones((a, b), dtype=torch.bool, device="cuda").tril_(b - a).logical_not_()
        for g in range(0, h if a and b else 0, step):
            hs = slice(g, min(h, g + step))
            keys = torch.cat((s["k_nope"][k0:k0 + b, hs].double(),
                              s["k_rope"][k0:k0 + b, None].double().expand(-1, hs.stop - hs.start, -1)), -1)
            w = torch.matmul(s["q"][q0:q0 + a, hs].double().permute(1, 0, 2), keys.permute(1, 2, 0)) * SM_SCALE
            if hidden is not None:
                w.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(w, -1, keepdim=True)
            p = torch.where(torch.isneginf(z), torch.zeros_like(w), (w - z).exp())
            out[q0:q0 + a, hs] = torch.matmul(p, s["v"][k0:k0 + b, hs].double().permute(1, 0, 2)).permute(1, 0, 2)
            lse[q0:q0 + a, hs] = z[..., 0].t()
        q0 += a
        k0 += b
    return [out, lse]
