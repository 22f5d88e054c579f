"""Cases that measure the prompt operators: attention over packed prompts and its gradient,
attention of new tokens over the paged cache, and the append of their K/V to it.

With `own` false, run() computes them from elementary torch operations in 32 bits over a padded
batch; with `own` true it makes the library's calls. Sizes are those of this repository's own
workloads (28 query and 4 KV heads of 128, 14 and 2 of 64, 4 and 2 of 64, prefixes up to 8192,
streams of 512 and 4096, pages of 16 tokens) and generic ones. The lengths of a case's sequences
come from its "layout", so that they are the same for every seed; inputs come from the seed."""
import math
import random

import torch

own = False

PAGE = 16
LOG2E = 1.4426950408889634
LARGEST_FLOPS = 1.2e12       # the largest listed case's, which drawn ones stay below
LARGEST_SCORES = 2.0e9       # elements of a padded score matrix


def listed():
    return [
        # a prompt's K/V into an empty cache: eight prompts of the 7B-class heads
        {"name": "append_prompts_7b", "op": "append", "hq": 28, "hkv": 4, "d": 128, "batch": 8,
         "lo": 512, "hi": 2048, "plo": 0, "phi": 0, "fused": True, "tail": 0, "layout": 1},
        # a scheduler's step of a small model: a few tokens of each of four sequences (latency)
        {"name": "append_few_tokens", "op": "append", "hq": 14, "hkv": 2, "d": 64, "batch": 4,
         "lo": 1, "hi": 13, "plo": 37, "phi": 512, "fused": False, "tail": 3, "layout": 2},
        # one new token after a short prompt (latency)
        {"name": "chunk_one_token", "op": "chunk", "hq": 4, "hkv": 2, "d": 64, "batch": 1,
         "lo": 1, "hi": 1, "plo": 50, "phi": 50, "fused": False, "tail": 0, "layout": 3},
        # single tokens of a batch over long caches: the serving step, bound by the cache's bytes
        {"name": "chunk_tokens_7b_b32", "op": "chunk", "hq": 28, "hkv": 4, "d": 128, "batch": 32,
         "lo": 1, "hi": 1, "plo": 2048, "phi": 8192, "fused": True, "tail": 0, "layout": 4},
        # a scheduler's mixed step: chunks of every length from one token on, ragged caches
        {"name": "chunk_mixed_7b_b12", "op": "chunk", "hq": 28, "hkv": 4, "d": 128, "batch": 12,
         "lo": 1, "hi": 700, "plo": 0, "phi": 2048, "fused": True, "tail": 5, "layout": 5},
        # the last chunk of one long prompt
        {"name": "chunk_long_7b", "op": "chunk", "hq": 28, "hkv": 4, "d": 128, "batch": 1,
         "lo": 2048, "hi": 2048, "plo": 30001, "phi": 30001, "fused": True, "tail": 0, "layout": 6},
        # prompts of a small model, prefilled together
        {"name": "packed_0.5b_b4", "op": "packed", "hq": 14, "hkv": 2, "d": 64, "batch": 4,
         "lo": 1, "hi": 512, "plo": 0, "phi": 0, "fused": False, "tail": 7, "layout": 7},
        # ragged prompts packed into one batch, 7B-class heads
        {"name": "packed_7b_b12", "op": "packed", "hq": 28, "hkv": 4, "d": 128, "batch": 12,
         "lo": 64, "hi": 2048, "plo": 0, "phi": 0, "fused": True, "tail": 0, "layout": 8},
        # one long prompt
        {"name": "packed_7b_long", "op": "packed", "hq": 28, "hkv": 4, "d": 128, "batch": 1,
         "lo": 8191, "hi": 8191, "plo": 0, "phi": 0, "fused": True, "tail": 0, "layout": 9},
        # training steps (forward with its row statistics, then the gradient) of packed examples
        {"name": "train_0.5b_b4", "op": "train", "hq": 14, "hkv": 2, "d": 64, "batch": 4,
         "lo": 1, "hi": 512, "plo": 0, "phi": 0, "fused": False, "tail": 7, "layout": 10},
        {"name": "train_7b_b8", "op": "train", "hq": 28, "hkv": 4, "d": 128, "batch": 8,
         "lo": 100, "hi": 2048, "plo": 0, "phi": 0, "fused": True, "tail": 0, "layout": 11},
        {"name": "train_7b_L4096", "op": "train", "hq": 28, "hkv": 4, "d": 128, "batch": 1,
         "lo": 4096, "hi": 4096, "plo": 0, "phi": 0, "fused": True, "tail": 0, "layout": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "packed", "train"])
    hq, hkv, d = rng.choice([(28, 4, 128), (28, 4, 128), (14, 2, 64), (4, 2, 64), (8, 8, 64),
                             (8, 1, 128), (16, 16, 128)])
    case = {"op": op, "hq": hq, "hkv": hkv, "d": d, "batch": _log_int(rng, 1, 48), "plo": 0,
            "phi": 0, "fused": rng.random() < 0.5, "tail": rng.choice([0, 0, 1, 9]),
            "layout": rng.randrange(1 << 30)}
    case["hi"] = 1 if op == "chunk" and rng.random() < 0.35 else _log_int(
        rng, 1, 1024 if op == "chunk" else 8192)
    case["lo"] = rng.randint(1, case["hi"])
    if op in ("chunk", "append"):
        case["phi"] = _log_int(rng, 1, 16384)
        case["plo"] = rng.randint(0, case["phi"])
    while case["batch"] > 1 and _cost(case) > 0.5:
        case["batch"] -= 1
    while case["hi"] > 1 and _cost(case) > 0.5:
        case["hi"] = max(1, case["hi"] // 2)
        case["lo"] = min(case["lo"], case["hi"])
    return case


def _cost(case):
    """The larger share of the largest case's work and memory that a case takes."""
    rows = case["batch"] * case["hi"]
    scores = case["batch"] * case["hq"] * case["hi"] * (case["hi"] + case["phi"])
    copied = rows * case["hkv"] * case["d"] / 4e8
    cached = case["batch"] * (case["phi"] + case["hi"]) * case["hkv"] * case["d"] / 1e9
    if case["op"] == "append":
        return max(copied, cached)
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
    if case["op"] == "append":
        return {"bytes": 8.0 * n * hkv * d, "flops": 0.0}
    pairs = hq * sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
    io = 2.0 * d * n * (2 * hq + 2 * hkv)
    if case["op"] == "chunk":
        return {"bytes": io + 4.0 * d * hkv * p, "flops": 4.0 * d * pairs}
    if case["op"] == "packed":
        return {"bytes": io + 4.0 * hq * n, "flops": 4.0 * d * pairs}
    return {"bytes": io + 4.0 * hq * n + 2.0 * d * n * (2 * hq + 2 * hkv), "flops": 14.0 * d * pairs}


class State:
    pass


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
    s.o = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    s.lse = torch.zeros(hq, n, dtype=torch.float32, device="cuda")
    s.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "train":
        s.d_o = normal(n, hq, d)
        s.dq, s.dk, s.dv = torch.zeros_like(s.q), torch.zeros_like(s.k), torch.zeros_like(s.v)
    if case["op"] in ("chunk", "append"):
        need = [-(-(x + y) // PAGE) for x, y in zip(new, old)]
        pages = max(1, sum(need))
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
        table = torch.full((b, max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = perm[at:at + m]
            at += m
        s.table = table.cuda()
        s.k_pool, s.v_pool = normal(pages, hkv, PAGE, d), normal(pages, hkv, PAGE, d)
        s.old = torch.tensor(old, dtype=torch.int32, device="cuda")
        s.new_lens = torch.zeros(b, dtype=torch.int32, device="cuda")
        s.slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    s.ws = None
    return s


def run(s):
    op = s.case["op"]
    if own:
        return _run_own(s, op)
    if op == "append":
        return _plain_append(s)
    if op == "chunk":
        return {"o": _plain_chunk(s)}
    if op == "packed":
        o, lse = _plain_packed(s)[:2]
        return {"o": o, "lse": lse}
    return _plain_train(s)


def _run_own(s, op):
    from block_masked_token_gb300 import packed
    c = s.case
    if op == "append":
        packed.mars_kv_append(s.k, s.v, s.cu, s.old, s.table, s.k_pool, s.v_pool,
                              new_lens=s.new_lens, slots=s.slots, status=s.status)
        return {"k_pool": s.k_pool, "v_pool": s.v_pool, "new_lens": s.new_lens, "slots": s.slots}
    if s.ws is None:         # the workspace that a program keeps for a batch of this shape
        code = {"chunk": packed.OP_ATTN_CHUNK, "packed": packed.OP_ATTN_PACKED,
                "train": packed.OP_ATTN_PACKED}[op]
        size = packed.mars_packed_workspace_bytes(code, c["batch"], s.rows, c["hq"], c["hkv"],
                                                  c["d"], s.max_len)
        if op == "train":
            size = max(size, packed.mars_packed_workspace_bytes(
                packed.OP_ATTN_PACKED_GRAD, c["batch"], s.rows, c["hq"], c["hkv"], c["d"],
                s.max_len))
        s.ws = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    if op == "chunk":
        packed.mars_attn_chunk(s.q, s.k, s.v, s.cu, s.k_pool, s.v_pool, s.table, s.old,
                               s.max_len, s.o, s.ws, status=s.status)
        return {"o": s.o}
    packed.mars_attn_packed(s.q, s.k, s.v, s.cu, s.o, s.ws, lse=s.lse, status=s.status)
    if op == "packed":
        return {"o": s.o, "lse": s.lse}
    packed.mars_attn_packed_grad(s.q, s.k, s.v, s.o, s.d_o, s.lse, s.cu, s.dq, s.dk, s.dv, s.ws,
                                 status=s.status)
    return {"o": s.o, "lse": s.lse, "dq": s.dq, "dk": s.dk, "dv": s.dv}


# ------------------------------------------------------------------------- plain forms


def _grid(s):
    """Row numbers of a padded batch [b, max_new] and which of its places hold a row."""
    cu = s.cu.long()
    i = torch.arange(s.max_new, device="cuda")
    live = i < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + i).clamp_(max=s.rows - 1), live, i


def _heads(x, rows, groups):
    """[n, h, d] rows -> [b, h, 1, max_new, d] in 32 bits (queries: [b, hkv, groups, ...])."""
    y = x[rows].float().transpose(1, 2)
    return y.unflatten(1, (-1, groups))


def _unpad(x, rows, live, like):
    """[b, hkv, groups, max_new, d] -> the rows of a tensor like `like`, zero where no row is."""
    out = torch.zeros(like.shape, dtype=like.dtype, device="cuda")
    out[rows[live]] = x.flatten(1, 2).transpose(1, 2)[live].to(like.dtype)
    return out


def _weights(q, k, hidden):
    """exp(score - row's maximum), the rows' sums and maxima; hidden: what a row does not see."""
    p = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(q.shape[-1]))
    p.masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(m).exp_()
    return p, p.sum(-1, keepdim=True), m


def _plain_packed(s):
    rows, live, i = _grid(s)
    groups = s.case["hq"] // s.case["hkv"]
    q, k, v = _heads(s.q, rows, groups), _heads(s.k, rows, 1), _heads(s.v, rows, 1)
    hidden = (i > i[:, None]) | ~live[:, None, :]
    p, total, m = _weights(q, k, hidden[:, None, None])
    o = _unpad((p @ v) / total, rows, live, s.o)
    lse = torch.zeros_like(s.lse)
    lse[:, rows[live]] = ((m + total.log()) * LOG2E)[..., 0].flatten(1, 2).transpose(1, 2)[live].t()
    return o, lse, p.div_(total), (rows, live, groups, q, k, v)


def _plain_train(s):
    o, lse, p, (rows, live, groups, q, k, v) = _plain_packed(s)
    keep = live[:, None, None, :, None]
    p = p.masked_fill_(~keep, 0.0)            # places without a row take part in no sum
    g = _heads(s.d_o, rows, groups)
    dv = (p.transpose(-1, -2) @ g).sum(2, keepdim=True)
    ds = g @ v.transpose(-1, -2)
    ds.sub_((p * ds).sum(-1, keepdim=True)).mul_(p).mul_(1.0 / math.sqrt(q.shape[-1]))
    dq, dk = ds @ k, (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
    return {"o": o, "lse": lse, "dq": _unpad(dq, rows, live, s.q),
            "dk": _unpad(dk, rows, live, s.k), "dv": _unpad(dv, rows, live, s.v)}


def _plain_chunk(s):
    rows, live, i = _grid(s)
    groups = s.case["hq"] // s.case["hkv"]
    q = _heads(s.q, rows, groups)
    pos = torch.arange(s.max_old, device="cuda")
    cached = pos < s.old[:, None]
    page = torch.where(cached, s.table[:, pos // PAGE], 0).long()

    def keys(pool, x):
        old = pool[page, :, pos % PAGE].float().transpose(1, 2).unsqueeze(2)
        return torch.cat([old, _heads(x, rows, 1)], 3)

    hidden = torch.cat([~cached[:, None, :].expand(-1, s.max_new, -1),
                        (i > i[:, None]) | ~live[:, None, :]], 2)
    p, total, _ = _weights(q, keys(s.k_pool, s.k), hidden[:, None, None])
    return _unpad((p @ keys(s.v_pool, s.v)) / total, rows, live, s.o)


def _plain_append(s):
    rows, live, i = _grid(s)
    pos = (s.old[:, None] + i)[live]
    seq = torch.arange(len(s.old), device="cuda")[:, None].expand_as(live)[live]
    page, at, r = s.table[seq, pos // PAGE].long(), pos % PAGE, rows[live]
    s.k_pool[page, :, at] = s.k[r]
    s.v_pool[page, :, at] = s.v[r]
    slots = torch.full_like(s.slots, -1)
    slots[r] = (page * PAGE + at).int()
    return {"k_pool": s.k_pool, "v_pool": s.v_pool, "new_lens": s.old + (s.cu[1:] - s.cu[:-1]),
            "slots": slots}


# ------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    if op == "append":
        return None          # copies: there is nothing that a rounding could change
    new, old = _lengths(case)
    per, scale = hq // hkv, 1.0 / math.sqrt(d)
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(s.rows, hq, d, **f64), torch.zeros(hq, s.rows, **f64)
    dq = torch.zeros(s.rows, hq, d, **f64)
    dk, dv = torch.zeros(s.rows, hkv, d, **f64), torch.zeros(s.rows, hkv, d, **f64)
    at = 0
    for i, (n, p) in enumerate(zip(new, old)):
        span = slice(at, at + n)
        at += n
        if n == 0:
            continue
        for h in range(hq):
            u = h // per
            k, v = s.k[span, u].double(), s.v[span, u].double()
            if p:
                ids = s.table[i, :-(-p // PAGE)].long()
                k = torch.cat([s.k_pool[ids, u].reshape(-1, d)[:p].double(), k])
                v = torch.cat([s.v_pool[ids, u].reshape(-1, d)[:p].double(), v])
            q = s.q[span, h].double()
            seen = torch.ones(n, n + p, dtype=torch.bool, device="cuda").tril_(p)
            z = torch.where(seen, q @ k.T * scale, -math.inf)
            top = torch.logsumexp(z, 1)
            a = torch.exp(z - top[:, None])
            o[span, h] = a @ v
            lse[h, span] = top / math.log(2.0)
            if op == "train":
                g = s.d_o[span, h].double()
                w = g @ v.T
                z = a * (w - (a * w).sum(1, keepdim=True)) * scale
                dq[span, h] = z @ k
                dk[span, u] += z.T @ q
                dv[span, u] += a.T @ g
    if op == "chunk":
        return {"o": o}
    if op == "packed":
        return {"o": o, "lse": lse}
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
