"""Inputs and error bounds of the attention tests.

The bounds count roundings.  u = 2^-24 is fp32's half step, b = 2^-8 bf16's.
A scaled score is a sum of d products of at most `size` in total magnitude
(sum |q_e k_e| scale): its error is at most (d + 2) u size, and that of the
exponent's argument, base-2 factor included, at most (d + 6) u size + 4 u |lse|.
The exponential adds 2^-21.  A weight is therefore off by a factor of at most
1 + e, e = (d + 8) u (size + |lse|) + 2^-21, and the sum of n of them by
another n u.
"""
import numpy as np
import torch

U, B = 2.0 ** -24, 2.0 ** -8


def weight_err(size, lse, d, n):
    return (d + 8) * U * (size + np.abs(np.where(np.isfinite(lse), lse, 0.0))) + 2.0 ** -21 + n * U


def check_attention(out, lse, ref, d, n, bf16):
    """out, lse against oracle (out, lse, abs_out, size)."""
    o, l, ab, size = ref[:4]
    e = weight_err(size, l, d, n)[..., None]
    # weights off by e in numerator and denominator, n products summed; bf16: each weight and the
    # result rounded once more
    tol = ab * (2 * e + n * U) + 4 * U * np.abs(o)
    if bf16:
        tol = tol + 1.01 * B * (ab + np.abs(o))
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    bad = np.abs(got - o) - tol
    assert np.all(bad <= 1e-30), (float(bad.max()), np.argwhere(bad > 0)[:4].tolist())
    if lse is not None:
        g = lse.cpu().numpy().astype(np.float64)
        empty = ~np.isfinite(l)
        assert np.array_equal(empty, ~np.isfinite(g)) and np.all(g[empty] == -np.inf)
        t = e[..., 0] + 4 * U * (np.abs(np.where(empty, 0, l)) + size + 1)
        assert np.all(np.abs(g - l)[~empty] <= t[~empty]), float((np.abs(g - l) - t)[~empty].max())


def rows(rng, n, h, d, dtype, loud=False):
    x = rng.normal(size=(n, h, d)).astype(np.float32)
    if loud:
        x[..., ::29] *= 5
    return torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def table(rng, kv_lens, page, spare=2, extra=1):
    """Permuted page table with `extra` unused columns (a page number that names none), and the page count."""
    per = [-(-k // page) for k in kv_lens]
    pages = sum(per) + spare
    perm = rng.permutation(pages)
    t = np.full((len(kv_lens), max(per, default=0) + extra), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, pages


def filled_cache(rng, kv_lens, page, hk, d):
    """A cache on the GPU whose visible slots hold quantised rows and whose other slots hold the bytes
    that hurt most (NaN scales), and its host copy for the oracle."""
    import exact_top_token_amd as E
    from oracle import attention as A

    t, pages = table(rng, kv_lens, page)
    h = {n: np.full((pages, page, hk, w), 0xFF, np.uint8) for n, w in (
        ("k_codes", d // 2), ("k_scales", d // 32), ("v_codes", d // 2), ("v_scales", d // 32))}
    for b, n in enumerate(kv_lens):
        at = A.slots(t, b, n, page, pages)
        for which in "kv":
            c, s = A.mx_encode(rows(rng, n, hk, d, "bf16", loud=True).float().numpy())
            h[which + "_codes"].reshape(-1, hk, d // 2)[at] = c
            h[which + "_scales"].reshape(-1, hk, d // 32)[at] = s
    g = {n: torch.from_numpy(x).cuda() for n, x in h.items()}
    h["table"] = t
    return E.Cache(g["k_codes"], g["k_scales"], g["v_codes"], g["v_scales"], torch.from_numpy(t).cuda()), h
