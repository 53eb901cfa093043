"""Plain 64-bit forms of the windowed attention and of the paged cache's
attention, on whatever device their inputs are, and the elementwise bounds that
the kernels' roundings give.

A rounding to a type is off by at most eps / 2 of the value (bf16 2^-8, fp16
2^-11).  The kernels round P and dS to bf16 before the second products, keep P
as fp16 between the backward's two phases (without dropout), and round every
output to bf16; sums, softmax statistics and D are fp32.  FP32 stands for what
the fp32 steps add (scores up to about 40 in log2 units, each off by 2^-24 of
that and of the d products, then exp2): 1e-5 of P covers them."""

import math

import torch

BF16, FP16, FP32 = 2.0 ** -8, 2.0 ** -11, 1e-5


def visible(nq, nk, device, causal=True, window=0, sinks=0, kv_len=None, block_mask=None):
    """bool [nq, nk]: which keys each query sees."""
    i = torch.arange(nq, device=device)[:, None]
    j = torch.arange(nk, device=device)[None, :]
    pos = i + nk - nq
    m = torch.ones((nq, nk), dtype=torch.bool, device=device)
    if causal:
        m &= j <= pos
    if window:
        m &= (j > pos - window) | (j < sinks)
    if kv_len is not None:
        m &= j < kv_len
    if block_mask is not None:
        m &= block_mask.to(device).bool()[i // 128, j // 128]
    return m


def head(q, k, v, scale, mask, do=None, keep=None, rscale=1.0):
    """One head in 64 bits: dict of o, lse (dq, dk, dv) and of the bound of each.

    q, do [n, d], k, v [m, d] float64; mask [n, m]; keep: dropout's kept entries."""
    s = scale * (q @ k.T)
    s = s.masked_fill(~mask, -math.inf)
    m = s.amax(1, keepdim=True) if k.shape[0] else torch.full((q.shape[0], 1), -math.inf).to(q)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(s - m)
    l = e.sum(1, keepdim=True)
    p = torch.where(l > 0, e / torch.where(l > 0, l, torch.ones_like(l)), torch.zeros_like(e))
    z = torch.ones_like(p) if keep is None else keep.to(p) * rscale
    pd = p * z
    o = pd @ v
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))[:, 0]
    o_tol = (BF16 + FP32) * (pd @ v.abs()) * (1 + BF16) + BF16 * o.abs()
    out = dict(o=o, o_tol=o_tol, lse=lse)
    if do is None:
        return out
    dp = (do @ v.T) * z
    dsum = (do * o).sum(1, keepdim=True)
    ds = p * (dp - dsum)
    ds_tol = (BF16 + FP16 + FP32) * (1 + BF16) * ds.abs() + p * (
        (do.abs() * o_tol).sum(1, keepdim=True) + FP32 * ((do.abs() @ v.abs().T) * z + dsum.abs()))
    out.update(dq=scale * (ds @ k), dk=scale * (ds.T @ q), dv=pd.T @ do)
    out["dq_tol"] = scale * (ds_tol @ k.abs()) * (1 + BF16) + BF16 * out["dq"].abs()
    out["dk_tol"] = scale * (ds_tol.T @ q.abs()) * (1 + BF16) + BF16 * out["dk"].abs()
    out["dv_tol"] = (BF16 + FP32) * (pd.T @ do.abs()) * (1 + BF16) + BF16 * out["dv"].abs()
    return out


def padded(q, k, v, scale, mask_of, do=None, keep=None, rscale=1.0):
    """All heads of [B, H, N, d] tensors; mask_of(b) the mask of entry b; the
    gradients of a shared K / V head (and their bounds) are summed over its
    query heads."""
    B, H = q.shape[:2]
    G = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    do = None if do is None else do.double()
    out = {}
    for b in range(B):
        mask = mask_of(b)
        for h in range(H):
            r = head(q[b, h], k[b, h // G], v[b, h // G], scale, mask,
                     None if do is None else do[b, h], None if keep is None else keep[b, h], rscale)
            for name, x in r.items():
                kv = name[:2] in ("dk", "dv")
                shape = (B, H // G if kv else H) + tuple(x.shape)
                t = out.setdefault(name, torch.zeros(shape, dtype=torch.float64, device=q.device))
                t[b, h // G if kv else h] += x
    # the sum over a group is rounded once more
    for name in ("dk", "dv"):
        if name in out and G > 1:
            out[name + "_tol"] = out[name + "_tol"] + BF16 * out[name].abs()
    return out


def check(name, got, ref, tol):
    """Every element within its bound (tiny absolute slack for exact zeros)."""
    got = got.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - (tol + 1e-7)
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{name}: {worst:.3g} over its bound at {over.argmax().item()}"


def check_lse(got, ref, tol=2e-5):
    """LSE: fp32 scores and sums (2^-24 of values up to about 60, and of the sum)."""
    got = got.double()
    empty = ref == -math.inf
    assert torch.equal(got == -math.inf, empty), "rows without keys differ"
    d = (got - ref)[~empty].abs()
    assert d.numel() == 0 or d.max().item() <= tol, f"lse: {d.max().item():.3g}"
