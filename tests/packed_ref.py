"""Packed sequences: a plain 64-bit reference and the bounds on how far the
kernels' outputs may be from it.

u = 2^-8 is half a step of bf16, relative.  The forward rounds each softmax
weight (u) and the output (u); scores, exponentials and sums are in fp32, whose
errors together stay below 2^-11 of a weight for the scores used here (products
of Dh values of a few units: 256 * 2^-24 * 256 * 3 at most for the largest
head, an exponential's 2^-22, a sum's n * 2^-24).  So, with a = sum_j p |v_j|:
    |o - ref| <= (1 + u) (u + 2^-11) a + u |ref|.
The backward starts from that o and from log-sum-exps in fp32.  D_i = dO_i . o_i
is off by at most sum_d |dO_id| times the bound of o; p by 2^-11 of itself; dP
by 2^-11 of sum_d |dO_id| |v_jd|.  p (for dV) and dS are rounded to bf16, and so
are the gradients.
"""
import torch

U, F = 2.0 ** -8, 2.0 ** -11


def hidden(n, causal, window, device):
    i = torch.arange(n, device=device)
    m = torch.zeros(n, n, dtype=torch.bool, device=device)
    if causal:
        m |= i[None] > i[:, None]
        if window > 0:
            m |= i[None] <= i[:, None] - window
    return m


def attention(q, k, v, cu, causal=True, window=0, scale=0.0, dout=None):
    """(o, lse, bound of o) or, with dout, also ((dq, dk, dv), their bounds); q [T,Hq,Dh], k and
    v [T,Hkv,Dh] any float type; rows of no sequence are zero."""
    T, Hq, Dh = q.shape
    Hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    scale = scale or Dh ** -0.5
    d64 = dict(dtype=torch.float64, device=q.device)
    o, bo = torch.zeros(T, Hq, Dh, **d64), torch.zeros(T, Hq, Dh, **d64)
    lse = torch.zeros(Hq, T, **d64)
    if dout is not None:
        dq, bq = torch.zeros(T, Hq, Dh, **d64), torch.zeros(T, Hq, Dh, **d64)
        dk, dv, bk, bv = (torch.zeros(T, Hkv, Dh, **d64) for _ in range(4))
    for a, z in zip(cu, cu[1:]):
        if z == a:
            continue
        m = hidden(z - a, causal, window, q.device)
        for h in range(Hq):
            g = h // G
            Q, K, V = q[a:z, h].double(), k[a:z, g].double(), v[a:z, g].double()
            s = (Q @ K.t() * scale).masked_fill(m, -torch.inf)
            L = torch.logsumexp(s, -1)
            p = torch.exp(s - L[:, None])
            y = p @ V
            o[a:z, h], lse[h, a:z] = y, L
            by = (1 + U) * (U + F) * (p @ V.abs()) + U * y.abs()
            bo[a:z, h] = by
            if dout is None:
                continue
            dO = dout[a:z, h].double()
            D = (dO * y).sum(-1, keepdim=True)
            dP = dO @ V.t()
            ds = p * (dP - D)
            off = (dO.abs() * by).sum(-1, keepdim=True) + F * (dO.abs() @ V.abs().t())
            e = (U + F) * ds.abs() + p * (1 + U) * off          # of dS before the last product
            dq[a:z, h] = scale * ds @ K
            bq[a:z, h] = scale * e @ K.abs()
            dk[a:z, g] += scale * ds.t() @ Q
            bk[a:z, g] += scale * e.t() @ Q.abs()
            dv[a:z, g] += p.t() @ dO
            bv[a:z, g] += (U + F) * p.t() @ dO.abs()
    if dout is None:
        return o, lse, bo
    bounds = tuple((1 + U) * b + U * x.abs() for b, x in ((bq, dq), (bk, dk), (bv, dv)))
    return o, lse, bo, (dq, dk, dv), bounds


def check(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    assert not torch.isnan(err).any(), what
    # (a result next to zero may underflow in fp32: 1e-30)
    over = err - bound
    assert bool((over <= 1e-30).all()), (what, float(over.max()), float(err.max()))


def layouts(T, Hq, Hkv, Dh, kind, gen, device="cuda"):
    """q, k, v as slices of one projection's output, contiguous, heads first, or of wider heads."""
    def normal(*shape):
        return torch.randn(shape, generator=gen, device=device).to(torch.bfloat16)
    if kind == "fused":
        x = normal(T, Hq + 2 * Hkv, Dh)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if kind == "heads_first":
        return tuple(normal(h, T, Dh).transpose(0, 1) for h in (Hq, Hkv, Hkv))
    if kind == "wide":
        return tuple(normal(T, h, Dh + 24)[..., 8:8 + Dh] for h in (Hq, Hkv, Hkv))
    return normal(T, Hq, Dh), normal(T, Hkv, Dh), normal(T, Hkv, Dh)


def offsets(lens, ahead=0):
    cu = [ahead]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu
