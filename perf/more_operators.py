"""Cases that measure the operators of the 8-bit paged cache and of rotary positions: rotation of
queries and keys and its gradient, the quantising append to a cache of 8-bit codes with a scale
for each page of 16 tokens and KV head, and attention of new tokens over that cache.

With `own` false, run() computes them from elementary torch operations in 32 bits (angles in 64)
over a padded batch; with `own` true it makes the library's calls. Sizes are those of this
repository's own workloads (28 query and 4 KV heads of 128, 14 and 2 of 64, 4 and 2 of 64, blocks
of 8 and 16 positions, prefixes up to 8192, streams of 512 and 4096, pages of 16 tokens) and
generic ones. The lengths of a case's sequences come from its "layout", so that they are the same
for every seed; inputs come from the seed."""
import math
import random

import torch

own = False

PAGE = 16
TOP = 448.0                  # the largest value of a code (e4m3)
BIAS, LEAST, MOST = 127, 87, 167      # scale byte x: 2^(x - BIAS); the bytes in use
LARGEST_FLOPS = 1.2e12       # the largest listed case's, which drawn ones stay below
LARGEST_SCORES = 2.0e9       # elements of a padded score matrix
LARGEST_CACHE = 5.5e8        # elements of K in a padded batch


def listed():
    return [
        # a scheduler's step of a small model: a few tokens of each of four sequences (latency)
        {"name": "rotary_few_tokens", "op": "rotary", "hq": 14, "hkv": 2, "d": 64, "batch": 4,
         "lo": 1, "hi": 13, "plo": 37, "phi": 512, "fused": False, "tail": 3, "rot": 64,
         "interleaved": False, "inverse": False, "stretch": 1.0, "layout": 1},
        # prompts of the 7B-class heads, from a fused projection's output
        {"name": "rotary_prompts_7b", "op": "rotary", "hq": 28, "hkv": 4, "d": 128, "batch": 8,
         "lo": 512, "hi": 2048, "plo": 0, "phi": 0, "fused": True, "tail": 0, "rot": 128,
         "interleaved": False, "inverse": False, "stretch": 1.0, "layout": 2},
        # the gradient for one long example: pairs side by side, half of the head, a stretched
        # context
        {"name": "rotary_grad_long_7b", "op": "rotary", "hq": 28, "hkv": 4, "d": 128, "batch": 1,
         "lo": 8191, "hi": 8191, "plo": 24576, "phi": 24576, "fused": True, "tail": 0, "rot": 64,
         "interleaved": True, "inverse": True, "stretch": 8.0, "layout": 3},
        # a few tokens of each of four sequences into pages that hold some already (latency)
        {"name": "append8_few_tokens", "op": "append8", "hq": 14, "hkv": 2, "d": 64, "batch": 4,
         "lo": 1, "hi": 13, "plo": 37, "phi": 512, "fused": False, "tail": 3, "layout": 4},
        # the serving step: one token of each of 128 sequences
        {"name": "append8_tokens_7b_b128", "op": "append8", "hq": 28, "hkv": 4, "d": 128,
         "batch": 128, "lo": 1, "hi": 1, "plo": 512, "phi": 2048, "fused": True, "tail": 0,
         "layout": 5},
        # prompts into an empty cache
        {"name": "append8_prompts_7b", "op": "append8", "hq": 28, "hkv": 4, "d": 128, "batch": 8,
         "lo": 512, "hi": 2048, "plo": 0, "phi": 0, "fused": True, "tail": 0, "layout": 6},
        # one new token after a short prompt (latency)
        {"name": "chunk8_one_token", "op": "chunk8", "hq": 4, "hkv": 2, "d": 64, "batch": 1,
         "lo": 1, "hi": 1, "plo": 50, "phi": 50, "fused": False, "tail": 0, "layout": 7},
        # single tokens of a batch over long caches: the serving step, bound by the cache's bytes
        {"name": "chunk8_tokens_7b_b32", "op": "chunk8", "hq": 28, "hkv": 4, "d": 128, "batch": 32,
         "lo": 1, "hi": 1, "plo": 2048, "phi": 8192, "fused": True, "tail": 0, "layout": 8},
        # a block of 8 masked positions for each of 32 sequences
        {"name": "chunk8_block8_7b_b32", "op": "chunk8", "hq": 28, "hkv": 4, "d": 128, "batch": 32,
         "lo": 8, "hi": 8, "plo": 512, "phi": 2048, "fused": True, "tail": 0, "layout": 9},
        # blocks of 16 positions, 128 sequences with long caches: the sustained decode
        {"name": "chunk8_block16_7b_b128", "op": "chunk8", "hq": 28, "hkv": 4, "d": 128,
         "batch": 128, "lo": 16, "hi": 16, "plo": 2048, "phi": 8192, "fused": True, "tail": 0,
         "layout": 10},
        # a scheduler's mixed step: chunks of every length from one token on, ragged caches
        {"name": "chunk8_mixed_7b_b12", "op": "chunk8", "hq": 28, "hkv": 4, "d": 128, "batch": 12,
         "lo": 1, "hi": 700, "plo": 0, "phi": 2048, "fused": True, "tail": 5, "layout": 11},
        # the last chunk of one long prompt
        {"name": "chunk8_long_7b", "op": "chunk8", "hq": 28, "hkv": 4, "d": 128, "batch": 1,
         "lo": 2048, "hi": 2048, "plo": 30001, "phi": 30001, "fused": True, "tail": 0,
         "layout": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append8", "chunk8", "chunk8"])
    hq, hkv, d = rng.choice([(28, 4, 128), (28, 4, 128), (14, 2, 64), (4, 2, 64), (8, 8, 64),
                             (8, 1, 128), (16, 16, 128)])
    case = {"op": op, "hq": hq, "hkv": hkv, "d": d, "batch": _log_int(rng, 1, 128),
            "fused": rng.random() < 0.5, "tail": rng.choice([0, 0, 1, 9]),
            "layout": rng.randrange(1 << 30)}
    case["hi"] = 1 if rng.random() < 0.3 else _log_int(rng, 1, 1024 if op == "chunk8" else 8192)
    case["lo"] = rng.randint(1, case["hi"])
    case["phi"] = _log_int(rng, 1, 65536 if op == "rotary" else 16384)
    case["plo"] = rng.randint(0, case["phi"])
    if op == "rotary":
        case.update(rot=rng.choice([d, d, d // 2, 16]), interleaved=rng.random() < 0.4,
                    inverse=rng.random() < 0.4, stretch=rng.choice([1.0, 1.0, 4.0]))
    while case["batch"] > 1 and _cost(case) > 0.5:
        case["batch"] -= 1
    while case["hi"] > 1 and _cost(case) > 0.5:
        case["hi"] = max(1, case["hi"] // 2)
        case["lo"] = min(case["lo"], case["hi"])
    return case


def _cost(case):
    """The larger share of the largest case's work and memory that a case takes."""
    rows = case["batch"] * case["hi"]
    if case["op"] == "rotary":
        return rows * (case["hq"] + case["hkv"]) * case["d"] / 6e7
    cached = case["batch"] * (case["phi"] + case["hi"]) * case["hkv"] * case["d"] / LARGEST_CACHE
    if case["op"] == "append8":
        return max(rows * case["hkv"] * case["d"] / 2e7, cached)
    scores = case["batch"] * case["hq"] * case["hi"] * (case["hi"] + case["phi"])
    return max(scores / LARGEST_SCORES, work(case)["flops"] / LARGEST_FLOPS, cached)


def _lengths(case):
    """(new tokens, cached tokens) of each sequence: the first has the most new tokens, and where
    there is room one has none."""
    rng = random.Random(case["layout"])
    new = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    new[0] = case["hi"]
    if case["batch"] > 3 and case["lo"] == 1 and case["hi"] > 1:
        new[2] = 0
    old = [rng.randint(case["plo"], case["phi"]) for _ in range(case["batch"])]
    return new, old


def work(case):
    new, old = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n, p = sum(new), sum(old)
    if case["op"] == "rotary":
        return {"bytes": 4.0 * n * (hq + hkv) * d, "flops": 3.0 * n * (hq + hkv) * case["rot"]}
    if case["op"] == "append8":
        pages = sum(-(-(a + b) // PAGE) - b // PAGE for a, b in zip(new, old) if a)
        return {"bytes": (4.0 + 2.0) * n * hkv * d + 2.0 * pages * hkv, "flops": 0.0}
    pairs = hq * sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
    pages = sum(-(-b // PAGE) for b in old)
    return {"bytes": 2.0 * d * n * (2 * hq + 2 * hkv) + 2.0 * hkv * (d * p + pages),
            "flops": 4.0 * d * pairs}


class State:
    pass


def _exponent(amax):
    """The smallest e with amax <= TOP * 2^e, in the range of the scale bytes."""
    m, x = torch.frexp(amax)
    e = torch.where(amax > 0, x - 9 + (m > TOP / 512), LEAST - BIAS)
    return e.clamp_(LEAST - BIAS, MOST - BIAS)


def _codes(x, e):
    """Codes of x over scales 2^e. Finite values beyond the range end at its border."""
    y = torch.ldexp(x, -e)
    return torch.where(x.isfinite(), y.clamp(-TOP, TOP), x).to(torch.float8_e4m3fn)


def _pool(g, pages, hkv, d, spread):
    """Pages as an append leaves them: codes and scale bytes. Their sizes differ page by page."""
    codes = torch.empty(pages, hkv, PAGE, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(pages, hkv, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (hkv * PAGE * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn(n, hkv, PAGE, d, generator=g, device="cuda")
        x *= (spread * torch.randn(n, hkv, 1, 1, generator=g, device="cuda")).exp_()
        e = _exponent(x.abs().amax((2, 3)))
        codes[i:i + n] = _codes(x, e[:, :, None, None])
        scale[i:i + n] = (e + BIAS).to(torch.uint8)
    return codes, scale


def prepare(case, seed):
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["batch"]
    new, old = _lengths(case)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    s = State()
    s.case = case
    s.rows = n = sum(new) + case["tail"]
    s.max_new, s.max_old = max(new), max(old)
    s.max_len = max(x + y for x, y in zip(new, old))
    # Q, K and V as the views of a fused projection's output, or as tensors of their own
    if case["fused"]:
        qkv = normal(n, hq + 2 * hkv, d)
        s.q, s.k, s.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s.q, s.k, s.v = normal(n, hq, d), normal(n, hkv, d), normal(n, hkv, d)
    ends = [0]
    for x in new:
        ends.append(ends[-1] + x)
    s.cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s.old = torch.tensor(old, dtype=torch.int32, device="cuda")
    s.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "rotary":
        rot = case["rot"]
        j = torch.arange(0, rot, 2, dtype=torch.float64)
        s.inv_freq = (10000.0 ** (-j / rot) / case["stretch"]).float().cuda()
        s.factor = 1.0 + 0.1 * math.log(case["stretch"])
        s.q_out = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        s.k_out = torch.zeros(n, hkv, d, dtype=torch.bfloat16, device="cuda")
        return s
    need = [-(-(x + y) // PAGE) for x, y in zip(new, old)]
    pages = max(1, sum(need))
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((b, max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = perm[at:at + m]
        at += m
    s.table = table.cuda()
    s.k_pool, s.k_scale = _pool(g, pages, hkv, d, 0.3)
    s.v_pool, s.v_scale = _pool(g, pages, hkv, d, 0.7)
    s.new_lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    s.slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    if case["op"] == "chunk8":
        s.o = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    s.ws = None
    return s


def run(s):
    if own:
        return _run_own(s, s.case["op"])
    if s.case["op"] == "rotary":
        return _plain_rotary(s)
    if s.case["op"] == "append8":
        return _plain_append(s)
    return {"o": _plain_chunk(s)}


def _run_own(s, op):
    from block_masked_token_gb300 import packed
    c = s.case
    if op == "rotary":
        packed.mars_rotary(s.q, s.k, s.cu, s.inv_freq, s.q_out, s.k_out, seq_lens=s.old,
                           interleaved=c["interleaved"], factor=s.factor, inverse=c["inverse"],
                           status=s.status)
        return {"q": s.q_out, "k": s.k_out}
    if op == "append8":
        packed.mars_kv_append_q8(s.k, s.v, s.cu, s.old, s.table, s.k_pool, s.v_pool, s.k_scale,
                                 s.v_scale, new_lens=s.new_lens, slots=s.slots, status=s.status)
        return {"k_pool": s.k_pool, "v_pool": s.v_pool, "k_scale": s.k_scale,
                "v_scale": s.v_scale, "new_lens": s.new_lens, "slots": s.slots}
    if s.ws is None:         # the workspace that a program keeps for a batch of this shape
        size = packed.mars_packed_workspace_bytes(packed.OP_ATTN_CHUNK_Q8, c["batch"], s.rows,
                                                  c["hq"], c["hkv"], c["d"], s.max_len)
        s.ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    packed.mars_attn_chunk_q8(s.q, s.k, s.v, s.cu, s.k_pool, s.v_pool, s.k_scale, s.v_scale,
                              s.table, s.old, s.max_len, s.o, s.ws, status=s.status)
    return {"o": s.o}


# ------------------------------------------------------------------------- plain forms


def _grid(s):
    """Row numbers of a padded batch [b, max_new] and which of its places hold a row."""
    cu = s.cu.long()
    i = torch.arange(s.max_new, device="cuda")
    live = i < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + i).clamp_(max=s.rows - 1), live, i


def _plain_rotary(s):
    c, rot = s.case, s.case["rot"]
    rows, live, i = _grid(s)
    r = rows[live]
    angle = (s.old.long()[:, None] + i)[live].double()[:, None] * s.inv_freq.double()
    cos, sin = (angle.cos() * s.factor).float()[:, None], (angle.sin() * s.factor).float()[:, None]
    if c["inverse"]:
        sin = -sin
    for x, out in ((s.q, s.q_out), (s.k, s.k_out)):
        y = x[r].float()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        out[r] = torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16)
    return {"q": s.q_out, "k": s.k_out}


def _power(scale):
    """Exponents of scale bytes."""
    return scale.int().clamp(LEAST, MOST) - BIAS


def _plain_append(s):
    n = (s.cu[1:] - s.cu[:-1]).long()
    old, cu = s.old.long(), s.cu.long()
    first = old // PAGE
    # the pages that get rows: [pages, PAGE] places, which of them are new and which held a token
    lp = torch.arange(s.table.shape[1], device="cuda")
    seq, page = torch.nonzero((lp >= first[:, None]) & (lp * PAGE < (old + n)[:, None]) &
                              (n > 0)[:, None], as_tuple=True)
    pos = page[:, None] * PAGE + torch.arange(PAGE, device="cuda")
    fresh = (pos >= old[seq, None]) & (pos < (old + n)[seq, None])
    held = pos < old[seq, None]
    row = (cu[seq, None] + pos - old[seq, None]).clamp_(0, max(0, s.rows - 1))
    at = s.table[seq, page].long()
    for x, pool, scale in ((s.k, s.k_pool, s.k_scale), (s.v, s.v_pool, s.v_scale)):
        y = x[row].float().transpose(1, 2)                      # [pages, hkv, PAGE, d]
        size = torch.where(y.isfinite() & fresh[:, None, :, None], y.abs(), 0.0).amax((2, 3))
        before = _power(scale[at])
        e = torch.maximum(_exponent(size), torch.where(held[:, :1], before, LEAST - BIAS))
        was = pool[at].float()
        codes = torch.where(fresh[:, None, :, None], _codes(y, e[:, :, None, None]).view(torch.uint8),
                            _codes(was, (e - before)[:, :, None, None]).view(torch.uint8))
        keep = (fresh | held)[:, None, :, None]
        pool.view(torch.uint8)[at] = torch.where(keep, codes, pool.view(torch.uint8)[at])
        scale[at] = (e + BIAS).to(torch.uint8)
    slots = torch.full_like(s.slots, -1)
    slots[row[fresh]] = (at[:, None] * PAGE + pos % PAGE)[fresh].int()
    return {"k_pool": s.k_pool, "v_pool": s.v_pool, "k_scale": s.k_scale, "v_scale": s.v_scale,
            "new_lens": (old + n).int(), "slots": slots}


def _plain_chunk(s):
    rows, live, i = _grid(s)
    groups = s.case["hq"] // s.case["hkv"]

    def heads(x, per):       # [n, h, d] rows -> [b, hkv, per, max_new, d]
        return x[rows].float().transpose(1, 2).unflatten(1, (-1, per))

    pos = torch.arange(s.max_old, device="cuda")
    cached = pos < s.old[:, None]
    wide = -(-max(1, s.max_old) // PAGE)
    lp = torch.arange(wide, device="cuda")
    page = torch.where(lp * PAGE < s.old[:, None], s.table[:, :wide], 0).long()

    def keys(pool, scale, x):
        y = torch.ldexp(pool[page].float(), _power(scale[page])[..., None, None])
        y = y.transpose(1, 2).flatten(2, 3)[:, :, :s.max_old].unsqueeze(2)
        return torch.cat([y, heads(x, 1)], 3)

    hidden = torch.cat([~cached[:, None, :].expand(-1, s.max_new, -1),
                        (i > i[:, None]) | ~live[:, None, :]], 2)[:, None, None]
    p = (heads(s.q, groups) @ keys(s.k_pool, s.k_scale, s.k).transpose(-1, -2)).mul_(
        1.0 / math.sqrt(s.case["d"]))
    p.masked_fill_(hidden, -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    y = (p @ keys(s.v_pool, s.v_scale, s.v)) / p.sum(-1, keepdim=True)
    s.o[rows[live]] = y.flatten(1, 2).transpose(1, 2)[live].to(torch.bfloat16)
    return s.o


# ------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append8": _exact_append, "chunk8": _exact_chunk}[case["op"]](
        s, case, *_lengths(case))


def _exact_rotary(s, case, new, old):
    """Each pair as a complex number, times exp(i angle)."""
    at, rot, out = 0, case["rot"], []
    turn = []
    for n, p in zip(new, old):
        pos = torch.arange(p, p + n, dtype=torch.float64, device="cuda")
        turn.append(torch.outer(pos, s.inv_freq.double()))
        at += n
    angle = torch.cat(turn) * (-1.0 if case["inverse"] else 1.0)
    z = torch.polar(torch.full_like(angle, s.factor), angle)[:, None]
    for x in (s.q, s.k):
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        y[:at] = x[:at].double()
        w = y[:at, :, :rot]
        w = w.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else w.unflatten(
            -1, (2, rot // 2)).transpose(-1, -2)
        w = torch.view_as_real(torch.view_as_complex(w.contiguous()) * z)
        y[:at, :, :rot] = (w if case["interleaved"] else w.transpose(-1, -2)).flatten(-2)
        out.append(y)
    return {"q": out[0], "k": out[1]}


def _exact_append(s, case, new, old):
    """What the codes would be without their last rounding, page by page."""
    pools, at = [], 0
    spans = []
    for i, (n, p) in enumerate(zip(new, old)):
        if n:
            spans.append((i, at, n, p))
        at += n
    tables = s.table.cpu().tolist()
    for x, pool, scale in ((s.k, s.k_pool, s.k_scale), (s.v, s.v_pool, s.v_scale)):
        values = pool.double()
        for i, row, n, p in spans:
            # the whole run of rows laid over its pages
            first, last = p // PAGE, (p + n - 1) // PAGE
            ids = torch.tensor(tables[i][first:last + 1], device="cuda")
            m, skip = len(ids), p % PAGE
            run_ = torch.zeros(m * PAGE, *x.shape[1:], dtype=torch.float64, device="cuda")
            run_[skip:skip + n] = x[row:row + n].double()
            run_ = run_.unflatten(0, (m, PAGE)).transpose(1, 2)
            e = torch.ceil(torch.log2(run_.abs().amax((2, 3)) / TOP)).clamp(LEAST - BIAS, MOST - BIAS)
            was = values[ids]
            if skip:
                e0 = scale[ids[0]].double() - BIAS
                e[0] = torch.maximum(e[0], e0)
                was[0, :, :skip] *= torch.exp2(e0 - e[0])[:, None, None]
            run_ *= torch.exp2(-e)[:, :, None, None]
            fresh = torch.zeros(m * PAGE, dtype=torch.bool, device="cuda")
            fresh[skip:skip + n] = True
            values[ids] = torch.where(fresh.view(m, 1, PAGE, 1), run_, was)
        pools.append(values)
    return {"k_pool": pools[0], "v_pool": pools[1], "k_scale": None, "v_scale": None,
            "new_lens": None, "slots": None}


def _exact_chunk(s, case, new, old):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    o = torch.zeros(s.rows, hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, p) in enumerate(zip(new, old)):
        span = slice(at, at + n)
        at += n
        if n == 0:
            continue
        ids = s.table[i, :-(-p // PAGE)].long()
        seen = torch.ones(n, n + p, dtype=torch.bool, device="cuda").tril_(p)
        for u in range(hkv):
            k, v = ((torch.exp2(scale[ids, u].double() - BIAS)[:, None, None] * pool[ids, u].double())
                    .reshape(-1, d)[:p] for pool, scale in ((s.k_pool, s.k_scale), (s.v_pool, s.v_scale)))
            k, v = torch.cat([k, s.k[span, u].double()]), torch.cat([v, s.v[span, u].double()])
            per = hq // hkv
            step = max(1, min(per, (1 << 28) // (n * (n + p))))
            for h in range(u * per, (u + 1) * per, step):
                hs = slice(h, min(h + step, (u + 1) * per))
                q = s.q[span, hs].double().transpose(0, 1)
                z = (q @ k.T / math.sqrt(d)).masked_fill_(~seen, -math.inf)
                o[span, hs] = (torch.softmax(z, -1) @ v).transpose(0, 1)
    return {"o": o}
