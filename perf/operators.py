"""The quantised paged KV cache, measured: writing it, reading it back, and attending over it.

Three operators share one cache format.

* append: new K/V rows (bf16) are quantised as they are written to the slots of a paged cache, and
  the written rows are read back (a chunk of a prompt attends to the values that later steps will
  see, so the prefill wants them back at once).
* read: the rows of given slots, dequantised to bf16 (a cached prefix leaving the cache).
* attend: decode attention of a few query tokens per sequence over the cached rows, lengths and
  block table on the device.

A page of one KV head holds ``page`` rows: the K codes, the V codes, then per row and group of
``group`` elements the four bf16 numbers (k_scale, k_min, v_scale, v_min); a code c stands for
min + scale * c.  A row's codes are stored in the order the kernels read them: K as [D/16][4][4]
transposed to [4][D/16][4], V as [D/16][8][2] transposed to [8][D/16][2], two 4-bit codes per byte
with the first one in the low half.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _append(name, T, Hkv, D, page, bits, group):
    return dict(name=name, op="append", T=T, Hkv=Hkv, D=D, page=page, bits=bits, group=group)


def _read(name, T, Hkv, D, page, bits, group):
    return dict(name=name, op="read", T=T, Hkv=Hkv, D=D, page=page, bits=bits, group=group)


def _attend(name, B, Hq, Hkv, D, page, kv_min, kv_max, bits, group, sq=1):
    return dict(name=name, op="attend", B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, kv_min=kv_min,
                kv_max=kv_max, bits=bits, group=group, sq=sq)


def listed():
    return [
        # one decode step of 64 sequences: a new row each, latency counts
        _append("append_step", 64, 8, 128, 16, 4, 128),
        # a prompt chunk written at once, small groups
        _append("append_chunk", 8192, 8, 128, 16, 4, 32),
        # an odd number of rows, the small head dim, 8 bits
        _append("append_odd_8bit", 777, 2, 64, 32, 8, 64),
        # a short cached prefix read back before the rest of its prompt is prefilled
        _read("read_prefix", 1000, 8, 128, 16, 4, 128),
        # a long context leaving the cache
        _read("read_long", 131071, 8, 128, 64, 4, 64),
        # one short sequence: the smallest decode step
        _attend("attend_short", 1, 8, 2, 64, 16, 300, 300, 4, 64),
        # a batch of equal lengths
        _attend("attend_batched", 16, 32, 8, 128, 16, 4096, 4096, 4, 128),
        # a serving batch of ragged lengths
        _attend("attend_ragged", 64, 32, 8, 128, 16, 128, 32768, 4, 128),
        # few long sequences, 8 query heads per KV head, small groups
        _attend("attend_long", 4, 64, 8, 128, 64, 131071, 131071, 4, 32),
        # the ragged batch with 8-bit codes
        _attend("attend_ragged_8bit", 64, 32, 8, 128, 16, 128, 32768, 8, 128),
        # a four-token verify step, causal among the new tokens
        _attend("attend_verify4", 16, 32, 8, 128, 32, 1, 8192, 4, 64, sq=4),
        # every query head on one KV head
        _attend("attend_mqa", 32, 64, 1, 128, 16, 1024, 16384, 4, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    D = rng.choice([64, 128, 128])
    bits = rng.choice([4, 4, 8])
    group = rng.choice([g for g in (32, 64, 128) if g <= D])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8])
    op = rng.choice(["append", "read", "attend", "attend"])
    if op == "append":
        c = _append("", _log(rng, 1, 8192), Hkv, D, page, bits, group)
    elif op == "read":
        c = _read("", _log(rng, 1, 65536), Hkv, D, page, bits, group)
    else:
        sq = rng.choice([1, 1, 1, 2, 3, 4])
        G = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16, 32, 64) if g * sq <= 64])
        B = _log(rng, 1, 64)
        longest = max(16, min(131072, 64 * 32768 * 8 // (B * Hkv * max(4, G * sq // 4))))
        top = _log(rng, 16, longest)
        c = _attend("", B, G * Hkv, Hkv, D, page, rng.choice([0, 1, top // 2, top]), top, bits,
                    group, sq)
    del c["name"]
    return c


def _row_bytes(c):
    return 2 * c["D"] * c["bits"] // 8 + 8 * (c["D"] // c["group"])


def _lengths(c):
    """The live rows of each sequence: the same for every seed, so that work() can count them."""
    span = c["kv_max"] - c["kv_min"]
    # a fixed low-discrepancy spread over [kv_min, kv_max]
    return [c["kv_min"] + int(round(span * ((0.5 + b * 0.6180339887498949) % 1.0)))
            for b in range(c["B"])]


def work(case):
    c = case
    if c["op"] in ("append", "read"):
        moved = c["T"] * c["Hkv"]
        # K and V rows of bf16: out of the cache, and for an append into it as well
        rows = moved * c["D"] * 4 * (2 if c["op"] == "append" else 1)
        return {"bytes": rows + moved * _row_bytes(c) + 8 * c["T"], "flops": 4 * moved * c["D"]}
    rows = sum(_lengths(c))
    io = 2 * 2 * c["B"] * c["Hq"] * c["sq"] * c["D"]
    table = 4 * sum(-(-n // c["page"]) for n in _lengths(c)) + 4 * c["B"]
    return {"bytes": rows * c["Hkv"] * _row_bytes(c) + io + table,
            "flops": 4 * rows * c["Hq"] * c["sq"] * c["D"]}


# ------------------------------------------------------------------ the format in plain operations
def _quantise(x, bits, group):
    """x [..., D] bf16 -> (codes uint8 [..., D], scale, minimum fp32 [..., D/group])."""
    qmax = float(2 ** bits - 1)
    x = x.float().unflatten(-1, (-1, group))
    lo, hi = x.amin(-1) + 0.0, x.amax(-1)
    span = hi - lo
    fine = torch.isfinite(span)
    # (a tensor divided by a tensor: by a plain number it would be multiplied by the reciprocal)
    s = torch.where(fine, span, torch.zeros_like(span)) / torch.full_like(span, qmax)
    # up to the next bf16, so the largest element never needs a code past the last one
    s = (((s.view(torch.int32) + 0xFFFF) >> 16) << 16).view(torch.float32)
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    live = (s > 0) & fine
    c = torch.round((x - lo[..., None]) / torch.where(live, s, torch.ones_like(s))[..., None])
    c = torch.where(live[..., None], c, torch.zeros_like(c)).to(torch.uint8).flatten(-2)
    nan = torch.full_like(s, float("nan"))
    return c, torch.where(fine, s, nan), torch.where(fine, lo, nan)


def _stored(codes, bits, value):
    """Codes [..., D] in the order of a stored K or V row, packed to bytes."""
    S = codes.shape[-1] // 16
    shape = (S, 8, 2) if value else (S, 4, 4)
    codes = codes.unflatten(-1, shape).transpose(-3, -2).flatten(-3)
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes


def _codes(rows, bits, value):
    """The inverse of _stored, as fp32 codes [..., D]."""
    if bits == 4:
        rows = torch.stack((rows & 15, rows >> 4), -1).flatten(-2)
    S = rows.shape[-1] // 16
    shape = (8, S, 2) if value else (4, S, 4)
    return rows.unflatten(-1, shape).transpose(-3, -2).flatten(-3).float()


def _regions(pool, c):
    """Views of the K codes, V codes and parameter bytes of pages [..., page_bytes]."""
    P, rb, par = c["page"], c["D"] * c["bits"] // 8, 8 * (c["D"] // c["group"])
    return (pool[..., :P * rb].unflatten(-1, (P, rb)),
            pool[..., P * rb:2 * P * rb].unflatten(-1, (P, rb)),
            pool[..., 2 * P * rb:].unflatten(-1, (P, par)))


def _params(par):
    """Parameter bytes [..., 8 * groups] -> fp32 [..., groups, 4]."""
    return par.contiguous().view(torch.bfloat16).float().unflatten(-1, (-1, 4))


def _values(codes, scale, low, group):
    return (codes.unflatten(-1, (-1, group)) * scale[..., None] + low[..., None]).flatten(-2)


def _write(pool, k, v, slots, c):
    """Quantises rows k, v [T, Hkv, D] into the slots of the pool; a negative slot writes nothing."""
    keep = slots >= 0
    page, off = slots[keep] // c["page"], slots[keep] % c["page"]
    kreg, vreg, preg = _regions(pool, c)
    kc, ks, kl = _quantise(k[keep], c["bits"], c["group"])
    vc, vs, vl = _quantise(v[keep], c["bits"], c["group"])
    kreg[page, :, off] = _stored(kc, c["bits"], False)
    vreg[page, :, off] = _stored(vc, c["bits"], True)
    par = torch.stack((ks, kl, vs, vl), -1).to(torch.bfloat16).flatten(-2)
    preg[page, :, off] = par.contiguous().view(torch.uint8)


def _gather(pool, slots, c):
    """The rows of the slots as bf16 (k, v) [T, Hkv, D]; a negative slot gives a zero row."""
    keep = slots >= 0
    at = slots.clamp(min=0)
    page, off = at // c["page"], at % c["page"]
    kreg, vreg, preg = _regions(pool, c)
    par = _params(preg[page, :, off])
    k = _values(_codes(kreg[page, :, off], c["bits"], False), par[..., 0], par[..., 1], c["group"])
    v = _values(_codes(vreg[page, :, off], c["bits"], True), par[..., 2], par[..., 3], c["group"])
    zero = torch.zeros((), device=k.device)
    keep = keep[:, None, None]
    return (torch.where(keep, k, zero).to(torch.bfloat16),
            torch.where(keep, v, zero).to(torch.bfloat16))


def _attention(s, c):
    """Decode attention over the pages of every sequence, padded to the longest one."""
    q, pool, table, lens = s["q"], s["pool"], s["block_table"], s["kv_lens"].long()
    B, Hq, sq, D = q.shape
    Hkv, P = c["Hkv"], c["page"]
    good = (table >= 0) & (table < pool.shape[0])
    pages = pool[torch.where(good, table, torch.zeros_like(table)).long()]    # [B, M, Hkv, bytes]
    kreg, vreg, preg = _regions(pages, c)
    par = _params(preg)
    k = _values(_codes(kreg, c["bits"], False), par[..., 0], par[..., 1], c["group"])
    k = k.permute(0, 2, 1, 3, 4).flatten(2, 3)                                # [B, Hkv, L, D]
    x = torch.matmul(q.float().reshape(B, Hkv, -1, D), k.transpose(-1, -2)) * s["scale"]
    del k
    L = x.shape[-1]
    key = torch.arange(L, device=q.device)
    tok = torch.arange(x.shape[2], device=q.device) % sq
    last = lens[:, None] - sq + tok                                           # causal: last row seen
    seen = (key <= last[..., None]) & good.repeat_interleave(P, 1)[:, None]   # [B, G*sq, L]
    x = torch.where(seen[:, None], x, torch.full((), -math.inf, device=q.device))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    v = _values(_codes(vreg, c["bits"], True), par[..., 2], par[..., 3], c["group"])
    v = v.permute(0, 2, 1, 3, 4).flatten(2, 3)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return out.reshape(B, Hq, sq, D).to(torch.bfloat16)


# ------------------------------------------------------------------ inputs
def _normals(g, *shape, channels=None):
    x = torch.randn(*shape, generator=g, device=DEV)
    if channels is not None:
        x *= channels
    return x.to(torch.bfloat16)


def _fill(pool, g, c, channels):
    """Quantised normal rows in every slot, some pages at a time (page by page order, no scatter)."""
    kreg, vreg, preg = _regions(pool, c)
    step = max(1, (1 << 26) // (c["Hkv"] * c["page"] * c["D"]))
    for a in range(0, pool.shape[0], step):
        n = min(step, pool.shape[0] - a)
        for reg, value in ((kreg, False), (vreg, True)):
            x = _normals(g, n, c["Hkv"], c["page"], c["D"], channels=None if value else channels)
            codes, s, lo = _quantise(x, c["bits"], c["group"])
            reg[a:a + n] = _stored(codes, c["bits"], value)
            par = torch.stack((s, lo), -1).to(torch.bfloat16).contiguous().view(torch.uint8)
            at = 4 if value else 0
            preg[a:a + n].unflatten(-1, (-1, 8))[..., at:at + 4] = par


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    Hkv, D, P = c["Hkv"], c["D"], c["page"]
    # K has channels of unlike size, as after a rotary embedding; one profile per KV head
    channels = torch.exp(0.5 * torch.randn(Hkv, 1, D, generator=g, device=DEV))
    page_bytes = P * _row_bytes(c)
    if c["op"] in ("append", "read"):
        T = c["T"]
        pages = -(-T // P) + 7
        pool = torch.zeros(pages, Hkv, page_bytes, dtype=torch.uint8, device=DEV)
        # consecutive positions on pages in random order, as a prompt or a batch lies in the cache
        order = torch.randperm(pages, generator=g, device=DEV)
        pos = torch.arange(T, device=DEV)
        slots = order[pos // P] * P + pos % P
        s = dict(case=c, pool=pool, slots=slots,
                 k_out=torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV),
                 v_out=torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV))
        if c["op"] == "append":
            if T >= 16:
                slots[5::16] = -1        # padding rows of a fixed-size step
            s["k"] = _normals(g, T, Hkv, D, channels=channels[:, 0])
            s["v"] = _normals(g, T, Hkv, D)
        else:
            _fill(pool, g, c, channels)
        return s
    B, Hq, sq = c["B"], c["Hq"], c["sq"]
    lens = _lengths(c)
    need = [-(-n // P) for n in lens]
    wide = max(1, max(need))
    pages = sum(need) + 5
    pool = torch.zeros(pages, Hkv, page_bytes, dtype=torch.uint8, device=DEV)
    _fill(pool, g, c, channels)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    count = torch.tensor(need, device=DEV)
    first = torch.cumsum(count, 0) - count
    col = torch.arange(wide, device=DEV)
    at = (first[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < count[:, None], order[at], torch.full((), -1, dtype=torch.int32, device=DEV))
    return dict(case=c, pool=pool, block_table=table.contiguous(),
                kv_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                q=_normals(g, B, Hq, sq, D), scale=D ** -0.5,
                out=torch.empty(B, Hq, sq, D, dtype=torch.bfloat16, device=DEV), workspace=None)


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "append":
            _write(s["pool"], s["k"], s["v"], s["slots"], c)
        if c["op"] in ("append", "read"):
            k, v = _gather(s["pool"], s["slots"], c)
            return {"k": k, "v": v}
        return {"out": _attention(s, c)}
    from token_decode_attention_split_gb300 import binding as da
    if c["op"] == "append":
        da.decode_attn_append_paged_quant(s["k"], s["v"], s["pool"], s["slots"], c["bits"], c["group"])
    if c["op"] in ("append", "read"):
        da.decode_attn_read_paged_quant(s["pool"], s["slots"], s["k_out"], s["v_out"], c["bits"],
                                        c["group"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["workspace"] is None:
        s["workspace"] = da.new_workspace(da.decode_attn_workspace_size(
            da.DA_VARIANT_PAGED_QUANT, c["B"], c["Hq"] * c["sq"], c["Hkv"], c["D"]), DEV)
    da.decode_attn_paged_quant(s["q"], s["pool"], s["out"], s["block_table"], s["kv_lens"], 1,
                               c["bits"], c["group"], c["sq"] > 1, s["scale"], s["workspace"])
    return {"out": s["out"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_row_values(x, bits, group):
    """What a quantised bf16 row stands for, from the definition: the nearest of the 2^bits levels
    min + scale * c, the even c on a tie; scale: the smallest bf16 >= range / (2^bits - 1)."""
    T, H, D = x.shape
    x = x.double().reshape(T, H, D // group, group)
    lo = x.min(dim=-1, keepdim=True).values
    step = (x.max(dim=-1, keepdim=True).values - lo) / (2 ** bits - 1)
    # bf16 keeps 7 of the 52 fraction bits: up to the next multiple of 2^45 in the bit pattern
    scale = (-(-step.view(torch.int64) // 2 ** 45) * 2 ** 45).view(torch.float64)
    code = torch.where(scale > 0, torch.round((x - lo) / torch.where(scale > 0, scale, 1.0)), 0.0)
    return (lo + scale * code).reshape(T, H, D)


def _exact_page_rows(pages, c, value):
    """The K or V rows (fp64) [n * page, Hkv, D] that n pages [n, Hkv, page_bytes] stand for."""
    D, P, bits, group = c["D"], c["page"], c["bits"], c["group"]
    n, H, rb, S, NG = pages.shape[0], pages.shape[1], D * bits // 8, D // 16, D // group
    raw = pages[:, :, P * rb * value:P * rb * (value + 1)].reshape(n, H, P, rb).to(torch.int64)
    e = torch.arange(D, device=pages.device)
    if value:    # pair (e / 16, (e % 16) / 2) is stored at pair position ((e % 16) / 2) * S + e / 16
        place = ((e % 16) // 2 * S + e // 16) * 2 + e % 2
    else:        # quad (e / 16, (e % 16) / 4) is stored at quad position ((e % 16) / 4) * S + e / 16
        place = ((e % 16) // 4 * S + e // 16) * 4 + e % 4
    codes = (raw[..., place // 2] >> (4 * (place % 2))) & 15 if bits == 4 else raw[..., place]
    par = pages[:, :, 2 * P * rb:].reshape(n, H, P, NG, 4, 2).to(torch.int32)
    par = ((par[..., 0] | (par[..., 1] << 8)) << 16).view(torch.float32).double()
    rows = par[..., e // group, 2 * value + 1] + par[..., e // group, 2 * value] * codes.double()
    return rows.permute(0, 2, 1, 3).reshape(n * P, H, D)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "append":
        keep = (s["slots"] >= 0)[:, None, None]
        return {n: torch.where(keep, _exact_row_values(s[n], c["bits"], c["group"]), 0.0)
                for n in ("k", "v")}
    if c["op"] == "read":
        k, v = (torch.empty(c["T"], c["Hkv"], c["D"], dtype=torch.float64, device=DEV) for _ in "kv")
        for a in range(0, c["T"], 8192):
            at = s["slots"][a:a + 8192]
            page, inv = torch.unique(at // c["page"], return_inverse=True)
            row = inv * c["page"] + at % c["page"]
            k[a:a + 8192] = _exact_page_rows(s["pool"][page], c, 0)[row]
            v[a:a + 8192] = _exact_page_rows(s["pool"][page], c, 1)[row]
        return {"k": k, "v": v}
    B, Hq, sq, D = s["q"].shape
    G = Hq // c["Hkv"]
    out = torch.zeros(B, Hq, sq, D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(c)):
        if n == 0:
            continue
        pages = s["pool"][s["block_table"][b, :-(-n // c["page"])].long()]
        k = _exact_page_rows(pages, c, 0)[:n]
        v = _exact_page_rows(pages, c, 1)[:n]
        q = s["q"][b].double().reshape(c["Hkv"], G * sq, D)
        x = torch.bmm(q, k.permute(1, 2, 0)) * s["scale"]                      # [Hkv, G * sq, n]
        token = torch.arange(G * sq, device=DEV) % sq
        dark = torch.arange(n, device=DEV)[None] > (n - sq + token)[:, None]
        x = x.masked_fill(dark[None], -math.inf)
        p = torch.nan_to_num(torch.softmax(x, -1))                             # a token with no row: 0
        out[b] = torch.bmm(p, v.permute(1, 0, 2)).reshape(Hq, sq, D)
    return {"out": out}
