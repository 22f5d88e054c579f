"""Inputs, runs and error bounds for the packed-sequence tests."""
import numpy as np
import torch

from block_masked_token_gb300 import mars, packed
from parity_util import U_BF16, UPSTREAM_REL, product_error_bound

PAGE = mars.PAGE_SIZE


def make(lens, hq, hkv, d, seed=0, old=None, tail=0, lead=0, fused=True, spare_pages=2):
    """CPU tensors of a packed batch: q, k, v as views of one tensor (fused) or apart, cu, and
    with `old` (cached tokens per sequence) pools and a block table with room for the append."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16)

    n = lead + sum(lens) + tail
    x = {"n": n, "lens": lens}
    x["qkv"] = normal(n, hq + 2 * hkv, d)
    q, k, v = x["qkv"].split([hq, hkv, hkv], dim=1)
    x["q"], x["k"], x["v"] = (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())
    x["fused"] = fused
    x["cu"] = torch.tensor(np.cumsum([lead] + list(lens)), dtype=torch.int32)
    x["do"] = normal(n, hq, d)
    if old is not None:
        need = [-(-(p + m) // PAGE) for p, m in zip(old, lens)]
        pages = sum(need) + spare_pages
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = perm[at:at + m]
            at += m
        x["table"], x["old"] = table, torch.tensor(old, dtype=torch.int32)
        x["k_pool"], x["v_pool"] = normal(pages, hkv, PAGE, d), normal(pages, hkv, PAGE, d)
        x["unused"] = perm[at:]
    return x


def cuda(x):
    """The same on the GPU, views kept as views."""
    y = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    if x["fused"]:
        hq, hkv = x["q"].shape[1], x["k"].shape[1]
        y["q"], y["k"], y["v"] = y["qkv"].split([hq, hkv, hkv], dim=1)
    return y


def workspace(op, batch, n, hq, hkv, d, max_len=0):
    size = packed.mars_packed_workspace_bytes(op, batch, n, hq, hkv, d, max_len)
    return torch.empty(size + 16, dtype=torch.uint8, device="cuda")


def run_packed(y, fill=7.0, scale=0.0, **kw):
    n, hq, d = y["q"].shape
    o = torch.full((n, hq, d), fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, n), fill, dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = workspace(packed.OP_ATTN_PACKED, len(y["cu"]) - 1, n, hq, y["k"].shape[1], d)
    packed.mars_attn_packed(y["q"], y["k"], y["v"], y["cu"], o, ws, lse=lse, status=st, scale=scale, **kw)
    torch.cuda.synchronize()
    return o, lse, int(st.item())


def run_chunk(y, fill=7.0, hint=None, scale=0.0, **kw):
    n, hq, d = y["q"].shape
    o = torch.full((n, hq, d), fill, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if hint is None:
        hint = max(int(p) + m for p, m in zip(y["old"].tolist(), y["lens"]))
    ws = workspace(packed.OP_ATTN_CHUNK, len(y["cu"]) - 1, n, hq, y["k"].shape[1], d, hint)
    packed.mars_attn_chunk(y["q"], y["k"], y["v"], y["cu"], y["k_pool"], y["v_pool"], y["table"],
                         y["old"], hint, o, ws, status=st, scale=scale, **kw)
    torch.cuda.synchronize()
    return o, int(st.item())


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def output_bound(P, V, ref):
    """Elementwise bound of a row block O = P V [rows, D] of the kernels: P rounded to bf16
    before the product (product_error_bound, one rounding), then O rounded to bf16, which is off
    by at most half a step, 2^-8 of the value."""
    b = product_error_bound(P @ np.abs(V), (P * P) @ (V * V), P.shape[1])
    return b + U_BF16 * (np.abs(ref) + b)


# lse = log2 sum exp2(s): an absolute error e of the scaled scores in natural units (the model's
# 2^-14, parity_util) moves it by log2(e) e, ex2.approx by 2^-22 log2(e), the fp32 result by
# 2^-24 of values below 32; together below 9.1e-5.
LSE_TOL = UPSTREAM_REL * 1.4426950408889634 + 2.0 ** -21 + 32 * 2.0 ** -24


def causal_weights(q, k, scale=None):
    n, D = q.shape
    z = (1.0 / np.sqrt(D) if scale is None else scale) * (q @ k.T)
    i = np.arange(len(k))[None, :] - (len(k) - n)
    z = np.where(i <= np.arange(n)[:, None], z, -np.inf)
    e = np.exp(z - z.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def run_grad(y, o, lse, d_o, fill=7.0, scale=0.0, wide=True, ws=None, out=None, **kw):
    """dq, dk, dv of run_packed's o and lse; `wide`: as slices of one tensor."""
    n, hq, d = y["q"].shape
    hkv = y["k"].shape[1]
    if out is None:
        all_ = torch.full((n, hq + 2 * hkv, d), fill, dtype=torch.bfloat16, device="cuda")
        out = all_.split([hq, hkv, hkv], dim=1)
        if not wide:
            out = [t.contiguous() for t in out]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = workspace(packed.OP_ATTN_PACKED_GRAD, len(y["cu"]) - 1, n, hq, hkv, d)
    packed.mars_attn_packed_grad(y["q"], y["k"], y["v"], o, d_o, lse, y["cu"], *out, ws, status=st,
                                 scale=scale, **kw)
    torch.cuda.synchronize()
    return [*out, int(st.item())]


def gradient_bounds(x, a, b, u):
    """Reference and elementwise bounds of dq [heads of group u], dk and dv of KV head u for the
    sequence in rows [a, b). The model of parity_util with one rounding (dS is formed from the
    unrounded P), to which D = rowsum(dO * o) adds: o carries output_bound, so D is off by at
    most sum_c |dO_c| output_bound_c, which enters dS times P. The results are rounded to bf16."""
    g = x["q"].shape[1] // x["k"].shape[1]
    k, v = f64(x["k"][a:b, u]), f64(x["v"][a:b, u])
    scale, n = 1.0 / np.sqrt(k.shape[1]), b - a
    dq, dq_b = [], []
    dk, dv = np.zeros_like(k), np.zeros_like(k)
    s1 = {"k": 0.0, "v": 0.0}
    s2 = {"k": 0.0, "v": 0.0}
    up = 0.0
    for h in range(u * g, u * g + g):
        q, do = f64(x["q"][a:b, h]), f64(x["do"][a:b, h])
        P = causal_weights(q, k)
        dP = do @ v.T
        D = (P * dP).sum(axis=1, keepdims=True)
        dS = scale * P * (dP - D)
        off = (np.abs(do) * output_bound(P, v, P @ v)).sum(axis=1, keepdims=True)
        slack = scale * P * (UPSTREAM_REL * (np.abs(dP) + np.abs(D)) + off)
        slack[0] = 0.0                                  # row 0: dS is 0, exactly
        dq.append(dS @ k)
        dq_b.append(product_error_bound(np.abs(dS) @ np.abs(k), dS ** 2 @ k ** 2, n, slack @ np.abs(k)))
        dk, dv = dk + dS.T @ q, dv + P.T @ do
        s1["k"], s2["k"] = s1["k"] + np.abs(dS).T @ np.abs(q), s2["k"] + (dS ** 2).T @ q ** 2
        s1["v"], s2["v"] = s1["v"] + P.T @ np.abs(do), s2["v"] + (P ** 2).T @ do ** 2
        up = up + slack.T @ np.abs(q)
    dk_b = product_error_bound(s1["k"], s2["k"], g * n, up, extra_roundings=g)
    dv_b = product_error_bound(s1["v"], s2["v"], g * n, extra_roundings=g)

    def rounded(r, e):
        return e + U_BF16 * (np.abs(r) + e)

    return ([(r, rounded(r, e)) for r, e in zip(dq, dq_b)], (dk, rounded(dk, dk_b)),
            (dv, rounded(dv, dv_b)))
