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
