"""A cache in 8 bits with a scale for every row, and what a serving loop does with a cache between two steps:
what these operators are asked to do, and their plain forms.

Six operators, each named by a case's "op":

  append8   a step's or a prompt's rows (512-wide latent, 64-wide rope key) on their way into a cache of
            E4M3 codes: RMS norm of the latent, rotation of the key, a scale of the row's own from its
            largest magnitude, write of codes and scale to the row's slot;
  expand8   cached rows of that kind, named by slot, to every head's keys and values, with the rope key;
  decode8   absorbed latent attention of one query token a request over such a cache: output, log-sum-exp;
  verify    the drafts of a speculative step against the target's probabilities, from given random numbers:
            "sampled" chains with the probabilities they were drawn from, "chain" and "tree" of chosen drafts;
            the accepted drafts, their number, and the token that follows them;
  requests  the lists of cache rows of a batch's requests after a step: forked, freed, and cut to the accepted
            drafts, with the slots that no request holds any more;
  move      rows in all layers of a cache: "copy" by pairs of slots, "compact" into the lowest slots, with the
            lists of rows rewritten.

`own` says which side runs: the plain forms below (elementary torch operations in 32 bits, in 64 where a
comparison is close: angles, probabilities and their running sums), or the library's entry points.
"""
import math
import random

import torch

own = False

ROPE, NOPE, LATENT, ROW = 64, 128, 512, 576
THETA, FACTOR, ORIGINAL, FAST, SLOW = 10000.0, 40.0, 4096, 32.0, 1.0   # rotary base and YaRN scaling
EPS = 1e-6
TOP = 448.0                                                              # largest E4M3 value
LOW_SCALE, HIGH_SCALE = 2.0 ** -64, 2.0 ** 64                            # a row's scale lies between these
SM_SCALE = 1.0 / math.sqrt(192.0)


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the smallest call: four requests' new rows, where latency is all
        dict(name="append8_step", op="append8", tokens=4, slots=512, norm=True, interleaved=True, scaling="yarn",
             near=False, stride=576),
        # a prompt's rows, cut out of the wider projection that also holds the query's low-rank part
        dict(name="append8_prompt", op="append8", tokens=16384, slots=20000, norm=True, interleaved=False,
             scaling="yarn", near=True, stride=2112),
        # a short prompt of the 16-head shape: two tiles of rows and one row more
        dict(name="expand8_short", op="expand8", tokens=257, heads=16, slots=4096),
        # a cached prefix of the 128-head shape, for a chunk that continues it
        dict(name="expand8_prefix", op="expand8", tokens=4095, heads=128, slots=16384),
        # a decode step of the 16-head shape: 64 requests over 512 to 4096 rows
        dict(name="decode8_step", op="decode8", heads=16, batch=64, shortest=512, longest=4096, which=1,
             slots=1 << 19, bf16=True),
        # a ragged serving batch of the 128-head shape
        dict(name="decode8_ragged", op="decode8", heads=128, batch=256, shortest=16, longest=16384, which=2,
             slots=1 << 20, bf16=False),
        # one request whose small draft model proposed four tokens, a vocabulary of odd size
        dict(name="verify_one", op="verify", form="sampled", batch=1, width=5, vocab=32001),
        # a serving batch with chains of seven drafts and a wide vocabulary
        dict(name="verify_batch", op="verify", form="sampled", batch=64, width=8, vocab=129280),
        # drafts of a ragged batch as trees, 15 drafts below the last token: lists cut to the accepted ones
        dict(name="requests_accept", op="requests", form="tree", batch=256, shortest=16, longest=16384, which=2,
             width=16, slots=1 << 20),
        # a beam search of 16 requests of four beams: some beams are forked, some freed
        dict(name="requests_fork", op="requests", form="fork", batch=64, shortest=512, longest=4096, which=1,
             width=0, slots=1 << 19),
        # a pool that is three tenths full, made contiguous in eight layers
        dict(name="compact_pool", op="move", form="compact", layers=8, slots=1 << 16, live=20001, bytes8=False),
        # 300 rows of a shared prefix copied for a request that leaves it, 8-bit rows with their scales
        dict(name="copy_rows", op="move", form="copy", layers=8, slots=1 << 13, live=300, bytes8=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append8", "expand8", "decode8", "decode8", "verify", "verify", "verify", "requests", "move", "move"])
    if op == "append8":
        tokens = _log_uniform(rng, 1, 16384)
        return dict(op=op, tokens=tokens, slots=tokens + rng.randint(1, 4000), norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]),
                    near=rng.random() < 0.5, stride=rng.choice([576, 584, 1344, 2112]))
    if op == "expand8":
        heads = rng.choice([1, 5, 16, 32, 128])
        tokens = _log_uniform(rng, 1, 4095 * 128 // max(heads, 32))
        return dict(op=op, tokens=tokens, heads=heads, slots=tokens + rng.randint(1, 4000))
    if op == "decode8":
        batch = _log_uniform(rng, 1, 256)
        longest = _log_uniform(rng, 2, min(131072, 400000 // batch))
        return dict(op=op, heads=rng.choice([16, 32, 48, 64, 96, 112, 128]), batch=batch,
                    shortest=_log_uniform(rng, 1, longest), longest=longest, which=rng.randint(0, 10 ** 6),
                    slots=batch * longest + rng.randint(1, 10 ** 5), bf16=rng.random() < 0.5)
    if op == "verify":
        width, vocab = _log_uniform(rng, 1, 64), _log_uniform(rng, 300, 200001)
        most = max(1, 64 * 8 * 129280 // (width * vocab))
        return dict(op=op, form=rng.choice(["sampled", "sampled", "chain", "tree"]), width=width, vocab=vocab,
                    batch=_log_uniform(rng, 1, min(256, most)))
    if op == "requests":
        batch = _log_uniform(rng, 1, 256)
        form = rng.choice(["fork", "chain", "tree"])
        longest = _log_uniform(rng, 64, min(16384, 10 ** 6 // batch))
        return dict(op=op, form=form, batch=batch, shortest=_log_uniform(rng, 1, longest), longest=longest,
                    which=rng.randint(0, 10 ** 6), width=0 if form == "fork" else rng.randint(1, 32),
                    slots=batch * (longest + 32) + rng.randint(1, 50000))
    form, layers, bytes8 = rng.choice(["compact", "copy"]), rng.randint(1, 8), rng.random() < 0.5
    slots = _log_uniform(rng, 40, 1 << 16)
    live = _log_uniform(rng, 1, slots // 2 if form == "copy" else slots)
    return dict(op="move", form=form, layers=layers, slots=slots, bytes8=bytes8,
                live=min(live, 20001) if form == "copy" else live)


def _lens(case):
    """The requests' numbers of rows: log-uniform, one stream of numbers for each case."""
    rng = random.Random(case["which"])
    return [_log_uniform(rng, case["shortest"], case["longest"]) for _ in range(case["batch"])]


def work(case):
    op = case["op"]
    if op == "append8":
        return {"bytes": case["tokens"] * (ROW * 2 + ROW + 4 + 8) + LATENT * 2 * case["norm"],
                "flops": case["tokens"] * ROW * 6}
    if op == "expand8":
        t, h = case["tokens"], case["heads"]
        return {"bytes": t * (ROW + 4 + 4 + ROPE * 2 + h * 2 * NOPE * 2) + h * 2 * NOPE * LATENT * 2,
                "flops": 2.0 * t * h * LATENT * 2 * NOPE}
    if op == "decode8":
        n, b, h = sum(_lens(case)), case["batch"], case["heads"]
        return {"bytes": n * (ROW + 4 + 4) + b * h * (ROW * 2 + LATENT * (2 if case["bf16"] else 4) + 4) + 4 * b,
                "flops": 2.0 * n * h * (ROW + LATENT)}
    if op == "verify":
        # the row that the next token is drawn from, and where a rejected draft was sampled its own as well
        b, v = case["batch"], case["vocab"]
        rows = 2 if case["form"] == "sampled" and case["width"] > 1 else 1
        return {"bytes": b * (4 * v * rows + 20 * case["width"] + 8), "flops": 3.0 * b * v * rows}
    if op == "requests":
        n = sum(_lens(case))
        return {"bytes": 8 * n + 12 * case["batch"] * (1 + case["width"]), "flops": n}
    row = ROW + 4 if case["bytes8"] else ROW * 2
    if case["form"] == "copy":
        return {"bytes": case["live"] * (case["layers"] * 2 * row + 8), "flops": case["live"]}
    moved = case["live"] * (1.0 - case["live"] / case["slots"])       # live rows in slots past the live ones
    return {"bytes": int(moved * case["layers"] * 2 * row) + 8 * case["live"], "flops": case["live"]}


# --------------------------------------------------------------- the inputs

def _positions(case, gen):
    """A prompt's positions follow one another; a step's requests are anywhere in their contexts."""
    t = case["tokens"]
    if case["near"]:
        start = torch.randint(0, 1000, (1,), generator=gen, device="cuda", dtype=torch.int32)
        return torch.arange(t, device="cuda", dtype=torch.int32) + start
    return torch.randint(0, 163840, (t,), generator=gen, device="cuda", dtype=torch.int32)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _normal(gen, *shape, scale=1.0):
    return _randn(gen, *shape).mul_(scale).to(torch.bfloat16)


def _loud(gen, rows):
    """How loud rows are: most about alike, one in 64 eight times as loud."""
    x = torch.exp(0.4 * _randn(gen, rows))
    return torch.where(torch.rand(rows, generator=gen, device="cuda") < 1 / 64, 8 * x, x)


def _cache8(gen, rows):
    """Codes and scales of rows about N(0, 1), a row's largest magnitude at the largest code."""
    x = _randn(gen, rows, ROW)
    top = x.abs().amax(dim=1)
    codes = x.mul_((TOP / top)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, top.mul_(1 / TOP).mul_(_loud(gen, rows))


def _slots(gen, count, slots):
    return torch.randperm(slots, generator=gen, device="cuda")[:count].to(torch.int32)


def _indptr(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


def _tree(rng, width, chain):
    """Parents of one request's drafts: draft 0 is the last token, the others extend an earlier draft."""
    return [-1] + [i - 1 if chain or rng.random() < 0.4 else rng.randint(max(0, i - 6), i - 1) for i in range(1, width)]


def _prepare_verify(case, gen, seed, s):
    b, w, v = case["batch"], case["width"], case["vocab"]
    form = case["form"]
    logits = _randn(gen, b, w, v).mul_(3.0)
    target = torch.softmax(logits, dim=-1)
    logits.add_(_randn(gen, b, w, v), alpha=0.8)                  # what a draft model makes of it
    s["uniforms"] = torch.rand((b, w), generator=gen, device="cuda")
    s["draft"], s["parents"] = None, None
    tokens = torch.zeros((b, w), dtype=torch.int64, device="cuda")
    if form == "sampled":
        # draft i was drawn from the draft model's row i - 1; one request in eight decodes greedily (its
        # target holds all mass on one token)
        draft = torch.empty_like(logits)
        draft[:, 1:] = torch.softmax(logits[:, :-1], dim=-1)
        draft[:, 0] = 0
        race = torch.empty((b, v), device="cuda")
        for i in range(1, w):
            race.exponential_(generator=gen)
            tokens[:, i] = (draft[:, i] / race).argmax(dim=-1)
        greedy = target[::8]
        best = greedy.argmax(dim=-1, keepdim=True)
        greedy.zero_().scatter_(-1, best, 1.0)
        s["draft"] = draft
    else:
        rng = random.Random(seed)
        parents = [_tree(rng, w, form == "chain") for _ in range(b)]
        rank = [[row[:i].count(p) for i, p in enumerate(row)] for row in parents]   # a draft's place among siblings
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda") if form == "tree" else None
        top = logits.topk(min(w + 1, v), dim=-1).indices
        at = torch.tensor(parents, device="cuda").clamp(min=0)
        pick = torch.gather(top, 1, at[..., None].expand(-1, -1, top.shape[-1]))
        tokens = torch.gather(pick, 2, torch.tensor(rank, device="cuda")[..., None])[..., 0]
    s.update(target=target, tokens=tokens.to(torch.int32),
             path=torch.empty((b, w), dtype=torch.int32, device="cuda"),
             accepted=torch.empty(b, dtype=torch.int32, device="cuda"),
             next=torch.empty(b, dtype=torch.int32, device="cuda"))


def _prepare_requests(case, gen, seed, s):
    lens, b, w = _lens(case), case["batch"], case["width"]
    lens = [x + w for x in lens]
    indptr, n = _indptr(lens), sum(lens)
    indices = _slots(gen, n, case["slots"])
    if case["form"] == "fork":
        # beams of four share the first half of the shortest of them
        for g in range(0, b - 3, 4):
            half = min(lens[g:g + 4]) // 2
            start = [sum(lens[:g + k]) for k in range(4)]
            for k in range(1, 4):
                indices[start[k]:start[k] + half] = indices[start[0]:start[0] + half]
        rng = random.Random(seed)
        sources = [4 * (r // 4) + rng.randrange(4) if 4 * (r // 4) + 3 < b else r for r in range(b)]
        s["path"] = s["accepted"] = None
    else:
        # one request in sixteen is done after this step
        rng = random.Random(seed)
        sources = [-1 if rng.random() < 1 / 16 else r for r in range(b)]
        path, accepted = [], []
        for _ in range(b):
            tree = _tree(rng, w, case["form"] == "chain")
            walk = [0]
            while True:
                below = [i for i in range(walk[-1] + 1, w) if tree[i] == walk[-1]]
                if not below or rng.random() < 0.35:
                    break
                walk.append(rng.choice(below))
            accepted.append(len(walk))
            path.append(walk + [-1] * (w - len(walk)))
        s["path"] = torch.tensor(path, dtype=torch.int32, device="cuda")
        s["accepted"] = torch.tensor(accepted, dtype=torch.int32, device="cuda")
    room = max(lens) * b if case["form"] == "fork" else n
    fill = lambda k: torch.full((k,), -1, dtype=torch.int32, device="cuda")  # noqa: E731
    s.update(indptr=indptr, indices=indices, sources=torch.tensor(sources, dtype=torch.int32, device="cuda"),
             new_indptr=fill(b + 1), new_indices=fill(room), freed=fill(n), count=fill(1))


def _prepare_move(case, gen, s):
    layers, slots, live = case["layers"], case["slots"], case["live"]
    if case["bytes8"]:
        parts = [_cache8(gen, slots) for _ in range(layers)]
        s["cache"], s["scales"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    else:
        s["cache"], s["scales"] = _normal(gen, layers, slots, ROW), None
    order = torch.randperm(slots, generator=gen, device="cuda").to(torch.int32)
    if case["form"] == "copy":
        s["src"], s["dst"] = order[:live].contiguous(), order[live:2 * live].contiguous()
    else:
        # two requests, the second with the first one's oldest rows as well: shared rows are named twice
        half = live // 2
        s["indices"] = torch.cat((order[:half], order[:half // 2], order[half:live])).contiguous()
        s["indptr"] = _indptr([half, live - half + half // 2])
        s["new_indices"] = torch.empty_like(s["indices"])
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=case)
    op = case["op"]
    if op == "append8":
        t, n = case["tokens"], case["slots"]
        wide = (_randn(gen, t, case["stride"]) * (2 * _loud(gen, t))[:, None]).to(torch.bfloat16)
        codes, scales = _cache8(gen, n)
        s.update(rows=wide[:, case["stride"] - ROW:], positions=_positions(case, gen), slots=_slots(gen, t, n),
                 weight=(1.0 + 0.1 * _normal(gen, LATENT).float()).to(torch.bfloat16) if case["norm"] else None,
                 cache=codes, scales=scales)
    elif op == "expand8":
        t, h, n = case["tokens"], case["heads"], case["slots"]
        s["cache"], s["scales"] = _cache8(gen, n)
        s.update(indices=_slots(gen, t, n), w_kc=_normal(gen, h, NOPE, LATENT, scale=LATENT ** -0.5),
                 w_vc=_normal(gen, h, LATENT, NOPE, scale=LATENT ** -0.5))
    elif op == "decode8":
        lens, b, h = _lens(case), case["batch"], case["heads"]
        s["cache"], s["scales"] = _cache8(gen, case["slots"])
        s.update(q_nope=_normal(gen, b, h, LATENT), q_rope=_normal(gen, b, h, ROPE), lens=lens,
                 indptr=_indptr(lens), indices=_slots(gen, sum(lens), case["slots"]))
    elif op == "verify":
        _prepare_verify(case, gen, int(seed), s)
    elif op == "requests":
        _prepare_requests(case, gen, int(seed), s)
    else:
        _prepare_move(case, gen, s)
    if own:
        # what a user's program keeps: the model's rotary frequencies, a batch's plan, buffers and workspaces
        from mla_latent_kv_absorbed_gb300 import binding
        bf = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        if op == "append8":
            s["freqs"] = binding.rope_frequencies(THETA, case["scaling"], FACTOR, ORIGINAL, FAST, SLOW)
        elif op == "expand8":
            s.update(k=bf(t, h, NOPE), kr=bf(t, ROPE), vo=bf(t, h, NOPE))
        elif op == "decode8":
            plan = binding.decode_plan(s["indptr"].cpu().numpy(), h)[0]
            s.update(plan=plan, plan_dev=torch.from_numpy(plan).cuda(),
                     workspace=zeros(binding.decode_fp8_workspace_bytes(plan)),
                     out=torch.empty((b, h, LATENT), dtype=torch.bfloat16 if case["bf16"] else torch.float32,
                                     device="cuda"),
                     lse=torch.empty((b, h), dtype=torch.float32, device="cuda"))
        elif op in ("requests", "move"):
            s["workspace"] = zeros(binding.slots_workspace_bytes(case["slots"]))
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


def _plain_append8(s):
    case = s["case"]
    x = s["rows"].float()
    c = x[:, :LATENT]
    if case["norm"]:
        c = c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    angle = s["positions"].double()[:, None] * _inv_freq(case["scaling"])
    cos, sin, r = angle.cos().float(), angle.sin().float(), x[:, LATENT:]
    if case["interleaved"]:
        a, b = r[:, 0::2], r[:, 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = r[:, :32], r[:, 32:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    row = torch.cat((c, r), dim=1)
    scale = (row.abs().amax(dim=1) / TOP).clamp(LOW_SCALE, HIGH_SCALE)
    code = (row / scale[:, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    at = s["slots"].long()
    s["cache"][at] = code.view(torch.uint8)
    s["scales"][at] = scale
    return [s["cache"].view(torch.float8_e4m3fn), s["scales"]]


def _values(s, at):
    """Rows of the 8-bit cache as float32."""
    return s["cache"][at].view(torch.float8_e4m3fn).float() * s["scales"][at][:, None]


def _plain_expand8(s):
    x = _values(s, s["indices"].long())
    c = x[:, :LATENT]
    k = torch.einsum("tr,hnr->thn", c, s["w_kc"].float())
    v = torch.einsum("tr,hrn->thn", c, s["w_vc"].float())
    return [k.to(torch.bfloat16), x[:, LATENT:].to(torch.bfloat16), v.to(torch.bfloat16)]


def _plain_decode8(s):
    q = torch.cat((s["q_nope"], s["q_rope"]), dim=-1).float()
    out = torch.empty(s["q_nope"].shape, device="cuda")
    lse = torch.empty(out.shape[:2], device="cuda")
    start = 0
    for i, n in enumerate(s["lens"]):
        x = _values(s, s["indices"][start:start + n].long())
        start += n
        score = (q[i] @ x.t()).mul_(SM_SCALE)
        top = score.amax(dim=-1, keepdim=True)
        p = score.sub_(top).exp_()
        total = p.sum(dim=-1, keepdim=True)
        out[i] = p @ x[:, :LATENT] / total
        lse[i] = (total.log() + top)[:, 0]
    return [out.to(torch.bfloat16) if s["case"]["bf16"] else out, lse]


def _plain_verify(s):
    """The walk down the drafts in their order: a draft whose parent is the node reached so far is accepted when
    its random number, times the draft's own probability (chosen drafts: the mass that rejected siblings left),
    is below the target's probability.  The next token is drawn from what is left of the node's row."""
    target, draft, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["uniforms"].double()
    b, w, v = target.shape
    every = torch.arange(b, device="cuda")
    node = torch.zeros(b, dtype=torch.int64, device="cuda")
    accepted = torch.ones_like(node)
    path = torch.full((b, w), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    rejected = torch.zeros((b, w), dtype=torch.bool, device="cuda")     # of the node's children
    left = torch.ones(b, dtype=torch.float64, device="cuda")
    for c in range(1, w):
        parent = s["parents"][:, c].long() if s["parents"] is not None else torch.full_like(node, c - 1)
        tried = parent == node
        again = (rejected & (tokens == tokens[:, c:c + 1])).any(dim=1)  # a rejected sibling had the same token
        t = target[every, node, tokens[:, c]].double()
        t = torch.where(again, torch.zeros_like(t), t)
        against = draft[every, c, tokens[:, c]].double() if draft is not None else left
        yes = tried & (u[:, c] * against < t)
        no = tried & ~yes
        left = torch.where(yes, torch.ones_like(left), torch.where(no, (left - t).clamp(min=0), left))
        rejected = rejected & ~yes[:, None]
        rejected[:, c] = no
        path.scatter_(1, torch.where(yes, accepted, torch.zeros_like(node))[:, None],
                      torch.where(yes, torch.full_like(node, c), torch.zeros_like(node))[:, None])
        accepted = accepted + yes
        node = torch.where(yes, torch.full_like(node, c), node)
    row = target[every, node].double()
    if draft is not None:
        below = (node + 1).clamp(max=w - 1)                             # the draft that was rejected, if any was
        less = row - draft[every, below].double()
        row = torch.where(rejected.any(dim=1, keepdim=True), less.clamp(min=0), row)
    else:
        for c in range(1, w):                                           # one after another: a token may come twice
            at = tokens[:, c:c + 1]
            row.scatter_(1, at, torch.where(rejected[:, c:c + 1], torch.zeros_like(left)[:, None], row.gather(1, at)))
    run_sum = row.cumsum(dim=1)
    total = run_sum[:, -1:]
    pick = (run_sum <= u[:, :1] * total).sum(dim=1)
    pick = torch.where(total[:, 0] > 0, pick.clamp(max=v - 1), torch.full_like(pick, -1))
    return [path.to(torch.int32), accepted.to(torch.int32), pick.to(torch.int32)]


def _plain_requests(s):
    indptr, indices, sources = s["indptr"].long(), s["indices"], s["sources"].long()
    w, path = s["case"]["width"], s["path"]
    src = sources.clamp(min=0)
    whole = (indptr[1:] - indptr[:-1])[src]
    kept = whole if path is None else whole - w + s["accepted"].long()[src]
    kept = torch.where(sources >= 0, kept, torch.zeros_like(kept))
    new_indptr = torch.cat((torch.zeros_like(kept[:1]), kept.cumsum(0)))
    s["new_indptr"].copy_(new_indptr)
    pos = torch.arange(s["new_indices"].numel(), device="cuda")
    r = (torch.searchsorted(new_indptr, pos, right=True) - 1).clamp(max=kept.numel() - 1)
    there, at, parent = pos < new_indptr[-1], pos - new_indptr[r], src[r]
    if path is not None:
        base = (indptr[1:] - indptr[:-1])[parent] - w                  # rows before the drafts
        step = (at - base).clamp(0, w - 1)
        at = torch.where(at < base, at, base + path[parent, step].long())
    got = indices[(indptr[parent] + at).clamp(0, indices.numel() - 1)]
    s["new_indices"].copy_(torch.where(there, got, s["new_indices"]))
    held = torch.zeros(s["case"]["slots"] + 1, dtype=torch.bool, device="cuda")
    held[indices.long()] = True
    held[torch.where(there, got.long(), torch.full_like(pos, s["case"]["slots"]))] = False
    free = held[:-1]
    rank = free.cumsum(0)
    n = s["freed"].numel()
    ext = torch.cat((s["freed"], s["freed"][:1]))
    where = torch.where(free, rank - 1, torch.full_like(rank, n))
    ext[where] = torch.arange(free.numel(), device="cuda", dtype=torch.int32)
    s["freed"].copy_(ext[:-1])
    s["count"].copy_(rank[-1:])
    return [s["new_indptr"], s["new_indices"], s["freed"], s["count"]]


def _plain_move(s):
    cache, scales = s["cache"], s["scales"]
    if s["case"]["form"] == "copy":
        src, dst, out = s["src"].long(), s["dst"].long(), []
    else:
        slots, old = cache.shape[1], s["indices"].long()
        live = torch.zeros(slots, dtype=torch.bool, device="cuda")
        live[old] = True
        n = live.sum()
        at = torch.arange(slots, device="cuda")
        # the k-th live slot past the live ones goes to the k-th free slot among them
        away, hole = live & (at >= n), ~live & (at < n)
        src, dst = away.nonzero()[:, 0], hole.nonzero()[:, 0]
        to = at.clone()
        to[src] = dst
        s["new_indices"].copy_(to[old])
        s["count"].copy_(n)
        out = [s["new_indices"], s["count"]]
    cache[:, dst] = cache[:, src]
    if scales is None:
        return [cache] + out
    scales[:, dst] = scales[:, src]
    return [cache.view(torch.float8_e4m3fn), scales] + out


# ------------------------------------------------------------------ the run

def _own_run(s):
    from mla_latent_kv_absorbed_gb300 import binding
    case = s["case"]
    op = case["op"]
    if op == "append8":
        binding.rope_append_kv_fp8_rows(s["cache"], s["scales"], s["slots"], s["rows"], s["positions"], s["freqs"],
                                        norm_weight=s["weight"], eps=EPS, interleaved=case["interleaved"])
        return [s["cache"].view(torch.float8_e4m3fn), s["scales"]]
    if op == "expand8":
        binding.expand_kv_fp8_rows(s["cache"], s["scales"], s["indices"], s["w_kc"], s["w_vc"], s["k"], s["kr"], s["vo"])
        return [s["k"], s["kr"], s["vo"]]
    if op == "decode8":
        binding.decode_run_fp8_rows(s["plan"], s["plan_dev"], s["q_nope"], s["q_rope"], s["cache"], s["scales"],
                                    s["indptr"], s["indices"], SM_SCALE, s["out"], s["lse"], s["workspace"])
        return [s["out"], s["lse"]]
    if op == "verify":
        binding.verify_drafts(s["target"], s["tokens"], s["uniforms"], s["path"], s["accepted"], s["next"],
                              draft_probs=s["draft"], parents=s["parents"])
        return [s["path"], s["accepted"], s["next"]]
    if op == "requests":
        binding.repack_requests(s["indptr"], s["indices"], s["sources"], s["new_indptr"], s["new_indices"],
                                case["slots"], s["workspace"], path=s["path"], accepted=s["accepted"],
                                freed=s["freed"], freed_count=s["count"])
        return [s["new_indptr"], s["new_indices"], s["freed"], s["count"]]
    cache = s["cache"].view(torch.float8_e4m3fn) if case["bytes8"] else s["cache"]
    held = [cache] if s["scales"] is None else [cache, s["scales"]]
    if case["form"] == "copy":
        binding.copy_rows(s["cache"], s["src"], s["cache"], s["dst"], src_scales=s["scales"], dst_scales=s["scales"],
                          workspace=s["workspace"])
        return held
    binding.compact_cache(s["cache"], s["indptr"], s["indices"], s["new_indices"], s["count"], s["workspace"],
                          kv_scales=s["scales"])
    return held + [s["new_indices"], s["count"]]


def run(state):
    if own:
        return _own_run(state)
    return {"append8": _plain_append8, "expand8": _plain_expand8, "decode8": _plain_decode8, "verify": _plain_verify,
            "requests": _plain_requests, "move": _plain_move}[state["case"]["op"]](state)


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
    turn = torch.polar(torch.ones_like(turn), turn)
    pairs = x.reshape(-1, 32, 2) if case["interleaved"] else x.reshape(-1, 2, 32).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    return (y if case["interleaved"] else y.transpose(-1, -2)).reshape(x.shape)


def _exact_verify(s):
    """Request by request on the host, as the operator's words have it."""
    target, draft = s["target"], s["draft"]
    tokens, u = s["tokens"].tolist(), s["uniforms"].double().tolist()
    b, w, v = target.shape
    parents = s["parents"].tolist() if s["parents"] is not None else [[i - 1 for i in range(w)]] * b
    at = s["tokens"].long()
    p_at = torch.gather(target, 2, at[:, None].expand(-1, w, -1)).double().tolist()      # [b][node][draft]
    q_at = torch.gather(draft, 2, at[..., None])[..., 0].double().tolist() if draft is not None else None
    path, accepted, following = [], [], []
    for i in range(b):
        walk, out = [0], None
        while out is None:
            node, lost, gone = walk[-1], 1.0, []
            for c in [k for k in range(node + 1, w) if parents[i][k] == node]:
                mass = 0.0 if tokens[i][c] in [tokens[i][g] for g in gone] else p_at[i][node][c]
                if u[i][c] * (q_at[i][c] if q_at else lost) < mass:
                    walk.append(c)
                    break
                lost = max(0.0, lost - mass)
                gone.append(c)
            else:
                out = gone
        row = target[i, walk[-1]].double()
        if out and draft is not None:
            row = torch.relu(row - draft[i, out[0]].double())
        elif out:
            row[[tokens[i][g] for g in out]] = 0.0
        upto = row.cumsum(0)
        total = float(upto[-1])
        following.append(int(torch.searchsorted(upto, u[i][0] * total, right=True).clamp(max=v - 1)) if total > 0 else -1)
        path.append(walk + [-1] * (w - len(walk)))
        accepted.append(len(walk))
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (path, accepted, following)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append8":
        codes, scales = s["cache"].view(torch.float8_e4m3fn).double(), s["scales"].double()
        x = s["rows"].double()
        lat = x[:, :LATENT]
        if case["norm"]:
            lat = lat / (lat.pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
        row = torch.cat((lat, _exact_rotate(x[:, LATENT:], s["positions"], case)), 1)
        scale = torch.linalg.vector_norm(row, ord=math.inf, dim=1) / TOP
        scale = scale.clamp(LOW_SCALE, HIGH_SCALE)
        codes[s["slots"].long()] = (row / scale.unsqueeze(1)).clamp(-TOP, TOP)
        scales[s["slots"].long()] = scale
        return [codes, scales]
    if op == "expand8":
        at = s["indices"].long()
        x = s["cache"][at].view(torch.float8_e4m3fn).double() * s["scales"][at].double().unsqueeze(1)
        k = torch.stack([x[:, :LATENT] @ w.double().t() for w in s["w_kc"]], 1)
        v = torch.stack([x[:, :LATENT] @ w.double() for w in s["w_vc"]], 1)
        return [k, x[:, LATENT:], v]
    if op == "decode8":
        b, h = case["batch"], case["heads"]
        out = torch.zeros((b, h, LATENT), dtype=torch.float64, device="cuda")
        lse = torch.zeros((b, h), dtype=torch.float64, device="cuda")
        for i, at in enumerate(torch.split(s["indices"].long(), s["lens"])):
            x = s["cache"][at].view(torch.float8_e4m3fn).double() * s["scales"][at].double().unsqueeze(1)
            z = (s["q_nope"][i].double() @ x[:, :LATENT].t() + s["q_rope"][i].double() @ x[:, LATENT:].t()) * SM_SCALE
            lse[i] = torch.logsumexp(z, 1)
            out[i] = torch.exp(z - lse[i].unsqueeze(1)) @ x[:, :LATENT]
        return [out, lse]
    if op == "verify":
        return _exact_verify(s)
    if op == "requests":
        ptr, idx, w = s["indptr"].tolist(), s["indices"].tolist(), case["width"]
        path = s["path"].tolist() if s["path"] is not None else None
        rows = []
        for src in s["sources"].tolist():
            mine = idx[ptr[src]:ptr[src + 1]] if src >= 0 else []
            if path is not None and src >= 0:
                mine = mine[:len(mine) - w] + [mine[len(mine) - w + i] for i in path[src] if i >= 0]
            rows.append(mine)
        flat = [x for mine in rows for x in mine]
        free = sorted(set(idx) - set(flat))
        put = lambda buf, vals: torch.tensor(vals + [-1] * (buf.numel() - len(vals)), dtype=torch.int32, device="cuda")  # noqa: E731
        ends = [0]
        for mine in rows:
            ends.append(ends[-1] + len(mine))
        return [put(s["new_indptr"], ends), put(s["new_indices"], flat), put(s["freed"], free),
                torch.tensor([len(free)], dtype=torch.int32, device="cuda")]
    cache = (s["cache"].view(torch.float8_e4m3fn) if case["bytes8"] else s["cache"]).double()
    extra = []
    if case["form"] == "copy":
        moves = list(zip(s["src"].tolist(), s["dst"].tolist()))
    else:
        old = s["indices"].tolist()
        live = sorted(set(old))
        n, there = len(live), set(live)
        moves = list(zip([x for x in live if x >= n], [x for x in range(n) if x not in there]))
        to = dict(moves)
        extra = [torch.tensor([to.get(x, x) for x in old], dtype=torch.int32, device="cuda"),
                 torch.tensor([n], dtype=torch.int32, device="cuda")]
    if moves:
        a, z = (torch.tensor(x, device="cuda") for x in zip(*moves))
        cache.index_copy_(1, z, cache.index_select(1, a))
    if s["scales"] is None:
        return [cache] + extra
    scales = s["scales"].double()
    if moves:
        scales.index_copy_(1, z, scales.index_select(1, a))
    return [cache, scales] + extra
