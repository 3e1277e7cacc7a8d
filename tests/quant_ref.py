"""The quantised paged cache in plain 64-bit arithmetic (numpy), written from the format's
definition in include/decode_attn.h: the oracle of tests/test_quant_cache.py."""
import numpy as np
import torch


def row_bytes(D, bits, group):
    return 2 * D * bits // 8 + 8 * (D // group)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bf16_up(x):
    """The smallest bf16 (as float64) that is >= x, for x >= 0."""
    b = np.asarray(x, np.float64).view(np.int64)
    up = (-(-b // 2 ** 45) * 2 ** 45).view(np.float64)          # 7 fraction bits
    return np.where(up < 2.0 ** -126, 0.0, up)                  # subnormals count as nothing


def quantise(x, bits, group):
    """x float64 [..., D] holding bf16 values -> (codes, scale, minimum)."""
    x = x.reshape(x.shape[:-1] + (-1, group))
    with np.errstate(invalid="ignore", over="ignore"):
        lo, hi = x.min(-1), x.max(-1)
        lo = lo + 0.0
        fine = np.isfinite(lo) & np.isfinite(hi) & (hi - lo <= np.finfo(np.float32).max)
        s = bf16_up(np.where(fine, hi - lo, 0.0) / (2 ** bits - 1))
        c = np.rint((x - lo[..., None]) / np.where(s > 0, s, 1.0)[..., None])
        c = np.where((fine & (s > 0))[..., None], c, 0.0)
    nan = np.float64("nan")
    return (c.astype(np.int64).reshape(c.shape[:-2] + (-1,)), np.where(fine, s, nan),
            np.where(fine, lo, nan))


def places(D, value):
    """Index in the stored row of each element's code."""
    e, S = np.arange(D), D // 16
    if value:
        return ((e % 16) // 2 * S + e // 16) * 2 + e % 2
    return ((e % 16) // 4 * S + e // 16) * 4 + e % 4


def pack(codes, bits, value):
    D = codes.shape[-1]
    stored = np.empty_like(codes)
    stored[..., places(D, value)] = codes
    if bits == 4:
        stored = stored[..., 0::2] | (stored[..., 1::2] << 4)
    return stored.astype(np.uint8)


def bf16_bytes(x):
    t = torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.bfloat16).contiguous()
    b = t.view(torch.int16).numpy().astype(np.int64) & 0xFFFF
    b = np.where(np.isnan(x), 0x7FC0, b)
    return np.stack((b & 255, b >> 8), -1).astype(np.uint8)


def append(pool, k, v, slots, D, P, bits, group):
    """pool uint8 numpy [pages, Hkv, page_bytes], changed in place."""
    rb, pb = D * bits // 8, 8 * (D // group)
    n = pool.shape[0] * P
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= n:
            continue
        page, r = divmod(int(slot), P)
        kc, ks, kl = quantise(k[t], bits, group)
        vc, vs, vl = quantise(v[t], bits, group)
        pool[page, :, r * rb:(r + 1) * rb] = pack(kc, bits, False)
        pool[page, :, (P + r) * rb:(P + r + 1) * rb] = pack(vc, bits, True)
        par = bf16_bytes(np.stack((ks, kl, vs, vl), -1)).reshape(pool.shape[1], pb)
        pool[page, :, 2 * P * rb + r * pb:2 * P * rb + (r + 1) * pb] = par


def rows(pool, pages, offs, D, P, bits, group):
    """(K, V) float64 [n, Hkv, D] of the given pages and rows, with their scales and minima."""
    rb, pb = D * bits // 8, 8 * (D // group)
    out = []
    for value in (0, 1):
        at = (value * P + offs)[:, None] * rb + np.arange(rb)
        raw = pool[pages[:, None], :, at].transpose(0, 2, 1).astype(np.int64)
        if bits == 4:
            raw = np.stack((raw & 15, raw >> 4), -1).reshape(raw.shape[:2] + (D,))
        codes = raw[..., places(D, value)]
        at = 2 * P * rb + offs[:, None] * pb + np.arange(pb)
        par = pool[pages[:, None], :, at].transpose(0, 2, 1).astype(np.uint32)
        par = (par[..., 0::2] | (par[..., 1::2] << 8)) << 16
        with np.errstate(invalid="ignore"):      # signalling NaN
            par = par.astype(np.uint32).view(np.float32).astype(np.float64)
        par = par.reshape(par.shape[:2] + (-1, 4))
        s = np.repeat(par[..., 2 * value], group, -1)
        lo = np.repeat(par[..., 2 * value + 1], group, -1)
        out.append((lo + s * codes, s, lo))
    return out


def attend(q, pool, table, lens, D, P, bits, group, scale, causal):
    """q float64 [B, Hq, Sq, D]; pool, table, lens numpy.  Returns (out, allowed error) float64.

    The allowed error: bf16 rounding of the output, half a step: 2^-8 |out|.  The weights p * vs
    are rounded to fp16, half a step 2^-11 of sum p * vs * c, at most the span of V; ex2.approx and
    the fp32 sums and products stay below 2^-15 of the same and of |min|.  A score's fp32 error, d =
    2^-18 * |scale| * sum|q| * max(|kmin| + span K) (its products are exact, its sums of at most D
    terms and three roundings lose below D / 8 + 4 units of 2^-24 of that), changes a weight by the
    factor e^d and the output by at most 2 d max|V|."""
    B, Hq, Sq, _ = q.shape
    Hkv = pool.shape[1]
    G = Hq // Hkv
    cap = table.shape[1] * P
    out = np.zeros_like(q)
    tol = np.zeros_like(q)
    for b in range(B):
        n = min(int(np.uint32(lens[b])), cap)
        if n == 0:
            continue
        pages = table[b, :-(-n // P)]
        key = np.arange(n)
        pg = pages[key // P]
        good = (pg >= 0) & (pg < pool.shape[0])
        if not good.any():
            continue
        key = key[good]
        (K, ks, kl), (V, vs, vl) = rows(pool, pg[good], key % P, D, P, bits, group)
        for h in range(Hkv):
            qq = q[b, h * G:(h + 1) * G].reshape(G * Sq, D)
            with np.errstate(invalid="ignore", over="ignore"):
                x = scale * (qq @ K[:, h].T)
                token = np.arange(G * Sq) % Sq
                seen = key[None] <= (n - Sq + token)[:, None] if causal else np.ones_like(x, bool)
                x = np.where(seen, x, -np.inf)
                top = x.max(-1, keepdims=True)
                p = np.where(seen, np.exp(x - np.where(np.isneginf(top), 0.0, top)), 0.0)
                total = p.sum(-1, keepdims=True)
                w = p / np.where(total == 0, 1.0, total)
                Vz = np.where(np.isnan(V[:, h]) & ~seen.any(0)[:, None], 0.0, V[:, h])
                if np.isnan(Vz).any():       # only the rows a column sees reach it
                    o = np.stack([w[i, seen[i]] @ Vz[seen[i]] for i in range(G * Sq)])
                else:
                    o = w @ Vz
                span = (2 ** bits - 1) * np.nanmax(vs[:, h])
                most = span + np.nanmax(np.abs(vl[:, h]))
                d = 2.0 ** -18 * abs(scale) * np.abs(qq).sum(-1, keepdims=True) * np.nanmax(
                    np.abs(kl[:, h]) + (2 ** bits - 1) * ks[:, h])
                t = 2.0 ** -8 * np.abs(o) + 2.0 ** -11 * span + (2.0 ** -15 + 2 * d) * most
            out[b, h * G:(h + 1) * G] = o.reshape(G, Sq, D)
            tol[b, h * G:(h + 1) * G] = np.broadcast_to(t, o.shape).reshape(G, Sq, D)
    return out, tol


def check(got, ref, tol, what=""):
    """Elementwise |got - ref| <= tol, NaN exactly where the reference has one."""
    got = got.detach().float().cpu().numpy().astype(np.float64)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    bad = ~nan & ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; first {i}: got {got[i]!r} "
                             f"ref {ref[i]!r} allowed {tol[i]!r}")
