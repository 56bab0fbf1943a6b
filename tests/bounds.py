"""Elementwise error bounds of the attention kernels, from the roundings they make.

u = 2^-24 (fp32 half step).  A dot product of n terms summed in fp32 in any order errs by at
most n u sum|terms|; the tensor cores may truncate instead of rounding, which doubles it: 2 n u.
The exponential is one hardware instruction (2^-22 relative) of an argument that errs as the
score does plus u times each of its operands.  bf16 rounds by at most 2^-8 relative.
"""
import numpy as np

U = 2.0 ** -24
BF16, F32 = 2.0 ** -8, 2.0 ** -24


def _probability(q, k, s, scale, lse, D):
    """Relative error of exp(s - lse) per (row, key)."""
    dot = scale * np.einsum("bhid,bhjd->bhij", np.abs(q), np.abs(k))
    return 2 * D * U * dot + 4 * U * (np.abs(s) + np.abs(lse)[..., None]) + 2.0 ** -21


def backward(q, k, v, o, lse, do, dlse, sel, scale, out_u):
    """(dq, dk, dv) bounds.  out_u: half step of the outputs; bf16 outputs also mean that P and
    dS are rounded to bf16 for the products."""
    B, H, N, D = q.shape
    mid = BF16 if out_u == BF16 else 0.0
    live = sel & ~np.isneginf(lse)[..., None]
    lse0 = np.where(np.isneginf(lse), 0.0, lse)
    s = scale * np.einsum("bhid,bhjd->bhij", q, k)
    p = np.where(live, np.exp(np.where(live, s - lse0[..., None], 0.0)), 0.0)
    ep = p * _probability(q, k, s, scale, lse0, D)
    dp = np.einsum("bhid,bhjd->bhij", do, v)
    delta = (do * o).sum(-1) - (0.0 if dlse is None else dlse)
    mag = (np.abs(do) * np.abs(o)).sum(-1) + (0.0 if dlse is None else np.abs(dlse))
    edp = 2 * D * U * (np.einsum("bhid,bhjd->bhij", np.abs(do), np.abs(v)) + mag[..., None])
    ds = np.abs(p * (dp - delta[..., None]))
    eds = ep * np.abs(dp - delta[..., None]) + (p + ep) * edp + 4 * U * ds
    eds = eds + mid * (ds + eds)
    ep = ep + mid * (p + ep)

    def out(w, ew, x, spec, val):
        e = np.einsum(spec, ew + 2 * (N + 2) * U * (w + ew), np.abs(x))
        return e + out_u * (np.abs(val) + e) + 2.0 ** -126

    sc = scale
    dq = sc * np.einsum("bhij,bhjd->bhid", np.where(live, p * (dp - delta[..., None]), 0), k)
    dk = sc * np.einsum("bhij,bhid->bhjd", np.where(live, p * (dp - delta[..., None]), 0), q)
    dv = np.einsum("bhij,bhid->bhjd", p, do)
    return (out(sc * ds, sc * eds, k, "bhij,bhjd->bhid", dq), out(sc * ds, sc * eds, q, "bhij,bhid->bhjd", dk),
            out(p, ep, do, "bhij,bhid->bhjd", dv))


def attention(q, k, v, lens, scale, out_u):
    """(o, lse) bounds of attention over the first lens[b] keys; q [B, H, Nq, D], k and v
    [B, Hk, M, D].  The weights and their sum carry the same error; with bf16 outputs the
    weights are rounded to bf16 for the second product only."""
    B, H, Nq, D = q.shape
    share = H // k.shape[1]
    mid = BF16 if out_u == BF16 else 0.0
    eo, el = np.zeros(q.shape), np.zeros((B, H, Nq))
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        for h in range(H):
            kk, vv = k[b, h // share, :n], v[b, h // share, :n]
            s = scale * q[b, h] @ kk.T
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(axis=1, keepdims=True)
            p = p / z
            ep = _probability(q[b:b + 1, h:h + 1], kk[None, None], s[None, None], scale,
                              m[None, None, :, 0], D)[0, 0]
            ez = (p * ep).sum(axis=1) + 2 * (n + 4) * U         # relative error of the sum
            el[b, h] = 2 * ez + 4 * U * (np.abs(m[:, 0]) + np.abs(np.log(z[:, 0]))) + 2.0 ** -21
            val = p @ vv
            e = (p * (ep + ez[:, None] + mid + 2 * (n + 4) * U)) @ np.abs(vv)
            eo[b, h] = 1.01 * e + out_u * (np.abs(val) + 1.01 * e) + 2.0 ** -126
    return eo, el


def check(name, got, want, bound):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= bound) | (np.isneginf(got) & np.isneginf(want)))
    if bad.any():
        i = tuple(int(x[0]) for x in np.nonzero(bad))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside the bound, first at {i}: "
                             f"got {got[i]}, want {want[i]}, bound {np.broadcast_to(bound, got.shape)[i]}")
