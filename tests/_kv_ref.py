"""Plain 64-bit forms of the cache operators, and the error bounds of their kernels.

Bounds (u = 2^-8, half a step of bf16 relative to the value).  A kernel's weights are
rounded to bf16 before they meet V and the sum they are divided by is that of the rounded
weights, so the output is off by at most sum_j p_j u |v_j - out| <= u (sum_j p_j |v_j| +
|out|); a bf16 output adds u |out|.  Scores are fp32 sums of D exact products: an error of
at most D 2^-24 sum_d |q_d k_d| scale, below 1e-4 for unit normal inputs at D = 128
(sum_d |q_d k_d| scale is about 128 * 0.64 / 11.3 = 7.2, times 128 * 2^-24 = 5.5e-5), which is
a relative error of the weights of as much, as are the exponential's 2^-22 and the sums'
order; 2^-12 covers them together for scores up to four times that size.
"""
import torch

U = 2.0 ** -8


def attention_row(q, k, v, scale):
    """(out, sum_j p_j |v_j|, lse) of one row over the keys k, v [n, D] (fp64)."""
    D = q.shape[-1]
    if k.shape[0] == 0:
        z = torch.zeros(D, dtype=torch.float64)
        return z, z, torch.tensor(-float("inf"), dtype=torch.float64)
    s = (k @ q) * scale
    lse = torch.logsumexp(s, 0)
    p = torch.exp(s - lse)
    return p @ v, p @ v.abs(), lse


def check_attention(out, lse, ref, label=""):
    """out [.., D] and lse against ref = (out, weighted |v|, lse) within the bounds above."""
    ro, ra, rl = ref
    o, l = out.detach().double().cpu(), lse.detach().double().cpu()
    assert torch.isfinite(o).all(), f"{label}: non-finite output"
    tol = U * (ra + ro.abs()) + 2.0 ** -12 * ra + 1e-30
    if out.dtype == torch.bfloat16:
        tol = tol + U * (ro.abs() + tol)
    worst = ((o - ro).abs() / tol).max()
    assert worst <= 1.0, f"{label}: output {worst:.3f} of its bound"
    empty = rl == -float("inf")
    assert torch.equal(l == -float("inf"), empty), f"{label}: empty rows"
    assert (o[empty] == 0).all(), f"{label}: empty rows must give 0"
    d = (l - rl)[~empty].abs()
    # the scores' error above (2^-12) and the logarithm's rounding
    assert (d <= 2.0 ** -12 + 2.0 ** -20 * rl[~empty].abs()).all(), f"{label}: lse {d.max():.2e}"


def paged_keys(pages, table, n):
    """The first n rows of a table's pages: [n, H_kv, D] in fp64."""
    ps = pages.shape[1]
    return torch.stack([pages[int(table[j // ps]), j % ps] for j in range(n)]).double() if n else \
        torch.zeros((0, *pages.shape[2:]), dtype=torch.float64)


def prefix_attention(q, kp, vp, cu, lens, tables, ptable, plen, scale):
    """CPU tensors -> (out [N, H, D], weighted |v|, lse [H, N]) over the rows < cu[-1]."""
    N, H, D = q.shape
    g = H // kp.shape[2]
    out = torch.zeros(N, H, D, dtype=torch.float64)
    wa = torch.zeros_like(out)
    lse = torch.zeros(H, N, dtype=torch.float64)
    pk, pv = paged_keys(kp, ptable, plen), paged_keys(vp, ptable, plen)
    for b in range(len(lens)):
        n, ln = int(cu[b + 1] - cu[b]), int(lens[b])
        ok, ov = paged_keys(kp, tables[b], ln), paged_keys(vp, tables[b], ln)
        for i in range(n):
            see = max(0, ln - n + i + 1)
            k, v = torch.cat([pk, ok[:see]]), torch.cat([pv, ov[:see]])
            t = int(cu[b]) + i
            for h in range(H):
                out[t, h], wa[t, h], lse[h, t] = attention_row(q[t, h].double(), k[:, h // g],
                                                               v[:, h // g], scale)
    return out, wa, lse


def cross_attention(q, k, v, lens, scale):
    """CPU tensors -> (out [B, Lq, H, D], weighted |v|, lse [B, H, Lq])."""
    B, Lq, H, D = q.shape
    g = H // k.shape[2]
    out = torch.zeros(B, Lq, H, D, dtype=torch.float64)
    wa = torch.zeros_like(out)
    lse = torch.full((B, H, Lq), -float("inf"), dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        kk = k[b, :n].double().repeat_interleave(g, 1).transpose(0, 1)
        vv = v[b, :n].double().repeat_interleave(g, 1).transpose(0, 1)
        s = (q[b].double().transpose(0, 1) @ kk.mT) * scale
        l = torch.logsumexp(s, -1)
        p = torch.exp(s - l[..., None])
        out[b], wa[b], lse[b] = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1), l
    return out, wa, lse


def rotate(x, pos, inv_freq, interleaved):
    """x [N, H, D] rotated to positions pos [N]: fp64."""
    x = x.double().clone()
    half = 0 if inv_freq is None else len(inv_freq)
    if half == 0:
        return x
    ang = pos.double()[:, None] * inv_freq.double()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    xa, xb = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    return x


def cross_backward(q, k, v, lens, do, scale):
    """CPU tensors -> (dq, dk, dv) in fp64, and a bound of each element's error by the
    kernel's roundings: P and dS are rounded to bf16 (u each) before their products with dO,
    k and q; Delta = rowsum(dO * O) is taken from O rounded to bf16, an error of at most
    u sum_d |dO O| that P weighs; scores and exponentials add 2^-12 of P (see above)."""
    B, Lq, H, D = q.shape
    Hk = k.shape[2]
    g = H // Hk
    grads = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v)]
    bounds = [torch.zeros_like(x) for x in grads]
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        qq, dd = q[b].double().transpose(0, 1), do[b].double().transpose(0, 1)
        kk = k[b, :n].double().repeat_interleave(g, 1).transpose(0, 1)
        vv = v[b, :n].double().repeat_interleave(g, 1).transpose(0, 1)
        p = torch.softmax((qq @ kk.mT) * scale, -1)
        o = p @ vv
        dp = dd @ vv.mT
        delta = (dd * o).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        e = 2.0 ** -12
        ds_err = (U + e) * ds.abs() + p * U * (dd * o).abs().sum(-1, keepdim=True) \
            + p * 2.0 ** -16 * (dd.abs() @ vv.abs().mT)
        p_err = (U + e) * p

        def group(x):  # sum over the query heads of a kv head
            return x.view(Hk, g, n, D).sum(1).transpose(0, 1)

        grads[0][b] = (ds @ kk * scale).transpose(0, 1)
        bounds[0][b] = (ds_err @ kk.abs() * scale).transpose(0, 1)
        grads[1][b, :n] = group(ds.mT @ qq * scale)
        bounds[1][b, :n] = group(ds_err.mT @ qq.abs() * scale)
        grads[2][b, :n] = group(p.mT @ dd)
        bounds[2][b, :n] = group(p_err.mT @ dd.abs())
    return grads, bounds


def check_grads(got, ref, label=""):
    for name, x, want, tol in zip(("dq", "dk", "dv"), got, *ref):
        x0, x = x, x.detach().double().cpu()
        assert torch.isfinite(x).all(), f"{label} {name}: non-finite"
        if x0.dtype == torch.bfloat16:
            tol = tol + U * (want.abs() + tol)
        err = (x - want).abs()
        assert (err <= tol + 1e-30).all(), \
            f"{label} {name}: {float((err / (tol + 1e-30)).max()):.3f} of its bound"
