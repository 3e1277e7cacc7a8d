"""The quantised paged cache on the GPU against the 64-bit oracle of tests/quant_ref.py: the writer
byte for byte, the reader bit for bit, the attention within a bound derived there; then all three
together as a serving loop uses them."""
import numpy as np
import pytest
import torch

import quant_ref as R
from token_decode_attention_split_gb300 import binding as B_

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normals(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


def noise_pool(pages, Hkv, D, P, bits, group, g):
    """A pool of random bytes (parameters too: infinities, NaN, anything)."""
    pool = B_.new_quant_pool(pages, Hkv, D, P, bits, group, DEV)
    return pool.random_(0, 256, generator=g)


FORMATS = [(64, 4, 32), (64, 4, 64), (64, 8, 32), (64, 8, 64), (128, 4, 32), (128, 4, 64),
           (128, 4, 128), (128, 8, 32), (128, 8, 64), (128, 8, 128)]


# ------------------------------------------------------------------ writing
@pytest.mark.parametrize("D,bits,group", FORMATS)
@pytest.mark.parametrize("T,Hkv,P", [(1, 1, 8), (37, 3, 16), (130, 8, 64)])
def test_append_bytes(D, bits, group, T, Hkv, P):
    g = gen(T * 1000 + D + bits + group)
    pages = -(-T // P) + 2
    pool = noise_pool(pages, Hkv, D, P, bits, group, g)
    want = pool.cpu().numpy().copy()
    k = normals(g, T, Hkv, D, scale=3.0)
    v = normals(g, T, Hkv, D) + torch.tensor(5.0, device=DEV, dtype=BF)
    slots = torch.randperm(pages * P, generator=g, device=DEV)[:T]
    if T > 8:
        slots[3], slots[5], slots[7] = -1, pages * P, -(1 << 40)   # skipped
    R.append(want, R.f64(k), R.f64(v), slots.tolist(), D, P, bits, group)
    B_.decode_attn_append_paged_quant(k, v, pool, slots, bits, group)
    assert np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("D,bits,group", FORMATS)
def test_append_special_rows(D, bits, group):
    """Constant groups, both zeros, NaN, infinities, the largest and the smallest numbers, and
    values that lie exactly half way between two codes."""
    rows = []

    def row(fill):
        x = torch.empty(D).normal_(generator=torch.Generator().manual_seed(len(rows)))
        rows.append(fill(x).to(BF).reshape(1, D))

    def at(x, i, val):
        x = x.clone()
        x[i] = val
        return x

    row(lambda x: torch.zeros(D))
    row(lambda x: -torch.zeros(D))
    row(lambda x: torch.where(x > 0, torch.zeros(D), -torch.zeros(D)))
    row(lambda x: torch.full((D,), 3.14159))
    row(lambda x: at(x, 7, float("nan")))
    row(lambda x: at(x, D - 1, float("inf")))
    row(lambda x: at(at(x, 0, float("-inf")), 33, float("nan")))
    row(lambda x: at(at(x, 1, 3e38), 2, -3e38))       # the range overflows: NaN
    row(lambda x: at(at(x, 1, 1.6e38), 2, -1.6e38))   # the range is finite
    row(lambda x: x * 1e-38)
    row(lambda x: x * 1e-40)                          # subnormal inputs: scale 0
    row(lambda x: x * 2e-37)
    row(lambda x: x * 1e30)
    row(lambda x: 1000.0 + x)
    n = 2 ** bits - 1
    # scale exactly 2 (or 1.5): the even numbers are half way for 4 and 8 bits
    row(lambda x: at(at(torch.randint(0, 31, (D,), generator=torch.Generator().manual_seed(5)).float(),
                        slice(0, None, 32), 0.0), slice(1, None, 32), 2.0 * n))
    row(lambda x: at(at(torch.randint(0, 240, (D,), generator=torch.Generator().manual_seed(6)) * 0.25,
                        slice(0, None, 32), 0.0), slice(1, None, 32), 1.5 * n))
    row(lambda x: at(at(torch.randint(0, 31, (D,), generator=torch.Generator().manual_seed(7)) - 17.0,
                        slice(0, None, 32), -17.0), slice(1, None, 32), 2.0 * n - 17.0))
    k = torch.cat(rows)[:, None].to(DEV)
    v = torch.cat(rows[::-1])[:, None].to(DEV)
    T, P = len(rows), 16
    pool = B_.new_quant_pool(2, 1, D, P, bits, group, DEV)
    want = pool.cpu().numpy().copy()
    slots = torch.arange(T, device=DEV) + 5
    R.append(want, R.f64(k), R.f64(v), slots.tolist(), D, P, bits, group)
    B_.decode_attn_append_paged_quant(k, v, pool, slots, bits, group)
    got = pool.cpu().numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, bad[:8]


def test_append_ties_in_bulk():
    """Small integers over ranges of 15, 30, 45, ... hit every tie; 2^17 groups at once."""
    g = gen(9)
    T, Hkv, D, P, bits, group = 1024, 32, 128, 256, 4, 32
    k = torch.randint(-100, 100, (T, Hkv, D), generator=g, device=DEV).to(BF)
    v = (torch.randint(-128, 128, (T, Hkv, D), generator=g, device=DEV) * 0.0625).to(BF)
    pool = B_.new_quant_pool(T // P, Hkv, D, P, bits, group, DEV)
    want = pool.cpu().numpy().copy()
    slots = torch.arange(T, device=DEV)
    R.append(want, R.f64(k), R.f64(v), slots.tolist(), D, P, bits, group)
    B_.decode_attn_append_paged_quant(k, v, pool, slots, bits, group)
    assert np.array_equal(pool.cpu().numpy(), want)


def test_append_strided_rows():
    """K and V as parts of one projection's rows."""
    g = gen(10)
    T, Hq, Hkv, D, P, bits, group = 33, 4, 2, 128, 16, 4, 64
    qkv = normals(g, T, (Hq + 2 * Hkv) * D + 8)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(-1, (Hkv, D))
    slots = torch.randperm(64, generator=g, device=DEV)[:T]
    a = B_.new_quant_pool(4, Hkv, D, P, bits, group, DEV)
    b = torch.zeros_like(a)
    B_.decode_attn_append_paged_quant(k, v, a, slots, bits, group)
    B_.decode_attn_append_paged_quant(k.contiguous(), v.contiguous(), b, slots, bits, group)
    assert torch.equal(a, b) and bool(a.any())


# ------------------------------------------------------------------ reading
@pytest.mark.parametrize("D,bits,group", FORMATS)
@pytest.mark.parametrize("T,Hkv,P", [(1, 1, 8), (61, 3, 16), (300, 8, 128)])
def test_read_rows(D, bits, group, T, Hkv, P):
    """Any bytes: every finite parameter and code, NaN and infinities; duplicate and bad slots."""
    g = gen(T + D + bits + group)
    pages = 5
    pool = noise_pool(pages, Hkv, D, P, bits, group, g)
    slots = torch.randint(0, pages * P, (T,), generator=g, device=DEV)
    if T > 8:
        slots[2], slots[4], slots[6] = -1, pages * P, 1 << 50
    k = torch.full((T, Hkv, D), 7.0, dtype=BF, device=DEV)
    v = torch.full_like(k, 7.0)
    B_.decode_attn_read_paged_quant(pool, slots, k, v, bits, group)
    s = slots.cpu().numpy()
    ok = (s >= 0) & (s < pages * P)
    at = np.where(ok, s, 0)
    for got, (_, scale, low), value in zip((k, v), R.rows(pool.cpu().numpy(), at // P, at % P, D, P,
                                                         bits, group), (0, 1)):
        with np.errstate(all="ignore"):
            codes = R.rows(pool.cpu().numpy(), at // P, at % P, D, P, bits, group)[value]
            x = codes[0].astype(np.float32)        # min + scale * code, rounded once to fp32
        want = torch.from_numpy(x).to(BF)
        want[torch.from_numpy(~ok)] = 0
        got = got.cpu()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], want[~nan])


def test_append_then_read_is_within_half_a_step():
    g = gen(12)
    T, Hkv, D, P = 200, 4, 128, 32
    k, v = normals(g, T, Hkv, D, scale=4.0), normals(g, T, Hkv, D)
    slots = torch.randperm(256, generator=g, device=DEV)[:T]
    for bits in (4, 8):
        for group in (32, 64, 128):
            pool = B_.new_quant_pool(8, Hkv, D, P, bits, group, DEV)
            B_.decode_attn_append_paged_quant(k, v, pool, slots, bits, group)
            ko, vo = torch.empty_like(k), torch.empty_like(v)
            B_.decode_attn_read_paged_quant(pool, slots, ko, vo, bits, group)
            for x, y in ((k, ko), (v, vo)):
                x, y = (t.double().unflatten(-1, (-1, group)) for t in (x, y))
                step = (x.amax(-1) - x.amin(-1)) / (2 ** bits - 1) * (1 + 2 ** -7)
                # half a step of the codes, half a step of bf16
                allowed = step[..., None] / 2 + y.abs() * 2 ** -8
                assert bool(((x - y).abs() <= allowed).all())


# ------------------------------------------------------------------ attention
def make(B, Hq, Hkv, D, P, bits, group, lens, seed, sq=1, k_scale=1.0, v_scale=1.0, spare=3):
    """Quantised normal rows in every live slot; NaN rows behind each sequence's end and in every
    unused page."""
    g = gen(seed)
    need = [-(-n // P) for n in lens]
    pages = sum(need) + spare
    pool = torch.full((pages, Hkv, B_.decode_attn_quant_page_bytes(D, P, bits, group)), 0xFF,
                      dtype=torch.uint8, device=DEV)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if n:
            pos = torch.arange(n, device=DEV)
            slots = table[b, pos // P].long() * P + pos % P
            B_.decode_attn_append_paged_quant(normals(g, n, Hkv, D, scale=k_scale),
                                              normals(g, n, Hkv, D, scale=v_scale), pool, slots,
                                              bits, group)
    return dict(q=normals(g, B, Hq, sq, D), pool=pool, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), D=D, P=P, bits=bits,
                group=group, scale=D ** -0.5)


def workspace(c):
    B, Hq, sq, D = c["q"].shape
    return B_.new_workspace(B_.decode_attn_workspace_size(B_.DA_VARIANT_PAGED_QUANT, B, Hq * sq,
                                                          c["pool"].shape[1], D), DEV)


def run(c, causal=True, ws=None, out=None):
    if out is None:
        out = torch.full_like(c["q"], float("nan"))
    ws = workspace(c) if ws is None else ws
    B_.decode_attn_paged_quant(c["q"], c["pool"], out, c["table"], c["lens"], c.get("stride", 1),
                               c["bits"], c["group"], causal, c["scale"], ws)
    return out


def oracle(c, causal=True):
    lens = c["lens"].cpu().numpy()[::c.get("stride", 1)]
    return R.attend(R.f64(c["q"]), c["pool"].cpu().numpy(), c["table"].cpu().numpy(), lens, c["D"],
                    c["P"], c["bits"], c["group"], c["scale"], causal)


def check(c, causal=True, what=""):
    out = run(c, causal)
    R.check(out, *oracle(c, causal), what)
    assert B_.decode_attn_read_device_error() == 0
    return out


@pytest.mark.parametrize("D,bits,group", FORMATS)
@pytest.mark.parametrize("G,Hkv", [(1, 1), (4, 8), (8, 2), (16, 4), (24, 1), (64, 1)])
def test_attention_formats(D, bits, group, G, Hkv):
    """Every kernel: narrow and wide columns, one to four column slices, one to eight heads a unit."""
    c = make(3, G * Hkv, Hkv, D, 16, bits, group, [1, 333, 150], seed=D + bits + group + G)
    check(c)


@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hkv", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("bits", [4, 8])
def test_attention_page_sizes(P, Hkv, bits):
    """Pages shorter and longer than a stage's rows of a head, and every unit width."""
    check(make(4, 4 * Hkv, Hkv, 128, P, bits, 64, [0, 17, P, 700 + P // 2], seed=P + Hkv))


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257, 1000])
def test_attention_lengths(n):
    check(make(2, 8, 2, 64, 8, 4, 32, [n, max(0, n - 1)], seed=n))
    check(make(1, 32, 8, 128, 64, 8, 128, [n], seed=n))


@pytest.mark.parametrize("sq,G,Hkv", [(2, 4, 8), (4, 4, 2), (3, 5, 1), (4, 16, 1), (7, 1, 3), (64, 1, 2)])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_several_tokens(sq, G, Hkv, causal):
    """Lengths below the token count leave the first tokens without a row: zero rows."""
    c = make(5, G * Hkv, Hkv, 128, 16, 4, 64, [0, 1, sq - 1, sq, 300], seed=sq + G, sq=sq)
    out = check(c, causal)
    assert not bool(out[0].any())
    if causal and sq > 1:
        assert not bool(out[1, :, :sq - 1].any())


@pytest.mark.parametrize("limit", [1, 2, 3, 5, 7, 40])
@pytest.mark.parametrize("G,Hkv", [(4, 8), (16, 2), (64, 1)])
def test_attention_splits(limit, G, Hkv):
    """Fewer CTAs: units in one piece, in many, and across CTAs; a unit's merge counter returns to zero."""
    c = make(5, G * Hkv, Hkv, 128, 16, 4, 128, [900, 0, 64, 2500, 1], seed=limit)
    ws = workspace(c)
    B_.decode_attn_set_grid_limit(limit)
    try:
        a = run(c, ws=ws)
        b = run(c, ws=ws)
    finally:
        B_.decode_attn_set_grid_limit(0)
    R.check(a, *oracle(c))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("B", [31, 32, 33, 100, 1024])
def test_attention_many_sequences(B):
    """More sequences than lanes and than CTAs, with empty ones at both ends, in runs and alone."""
    rng = np.random.RandomState(B)
    lens = [int(n) if keep else 0 for n, keep in zip(rng.randint(1, 90, B), rng.rand(B) < 0.7)]
    lens[0] = lens[-1] = 0
    lens[B // 2] = 700
    check(make(B, 8, 2, 64, 16, 4, 64, lens, seed=B))
    lens = [0] * B
    lens[-1] = 40
    out = check(make(B, 4, 4, 128, 8, 8, 128, lens, seed=B + 1))
    assert not bool(out[:-1].any()) and bool(out[-1].any())


@pytest.mark.parametrize("seed", range(40))
def test_attention_random(seed):
    """Drawn shapes: head counts, page sizes, tokens, lengths, grids, bad pages."""
    rng = np.random.RandomState(1000 + seed)
    D = int(rng.choice([64, 128]))
    bits = int(rng.choice([4, 8]))
    group = int(rng.choice([g for g in (32, 64, 128) if g <= D]))
    P = int(2 ** rng.randint(3, 9))
    Hkv = int(rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16]))
    sq = int(rng.choice([1, 1, 2, 3, 5]))
    G = int(rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 11, 16, 20, 32, 64) if g * sq <= 64]))
    B = int(rng.randint(1, 9))
    top = int(rng.choice([20, 300, 3000]))
    lens = [int(n) for n in rng.randint(0, top + 1, B)]
    c = make(B, G * Hkv, Hkv, D, P, bits, group, lens, seed=seed, sq=sq, k_scale=float(rng.choice([1, 4])))
    if rng.rand() < 0.3:
        hit = torch.from_numpy(rng.rand(*c["table"].shape) < 0.1).to(DEV)
        c["table"] = torch.where(hit, torch.full_like(c["table"], 1 << 29), c["table"])
    B_.decode_attn_set_grid_limit(int(rng.choice([0, 0, 1, 3, 17])))
    try:
        check(c, bool(rng.rand() < 0.7), f"D={D} bits={bits} group={group} P={P} Hkv={Hkv} G={G} sq={sq} {lens}")
    finally:
        B_.decode_attn_set_grid_limit(0)


@pytest.mark.parametrize("D,bits", [(64, 4), (64, 8), (128, 4), (128, 8)])
@pytest.mark.parametrize("G,sq", [(33, 1), (64, 1), (8, 5), (1, 64)])
@pytest.mark.parametrize("P", [8, 64, 256])
def test_attention_wide_units(D, bits, G, sq, P):
    """33 to 64 columns of rows with one group: lengths around a stage, several KV heads, lost pages, causal or
    not, units in one piece and in many."""
    lens = [0, 1, 63, 64, 65, 700, 128, sq, 0]
    c = make(len(lens), 3 * G, 3, D, P, bits, D, lens, seed=D + bits + G + P, sq=sq)
    ws = workspace(c)
    for limit in (0, 1, 5):
        B_.decode_attn_set_grid_limit(limit)
        try:
            for causal in (True, False):
                R.check(run(c, causal, ws), *oracle(c, causal), f"limit {limit} causal {causal}")
        finally:
            B_.decode_attn_set_grid_limit(0)
    c["table"][5, ::2] = 1 << 30
    c["table"][2] = -5
    check(c)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(30.0, 1.0, 1.0), (1.0, 1e-6, 1.0), (1.0, 1e20, 1.0),
                                                     (1e-3, 1.0, 1e4), (1.0, 1.0, 1e-30), (1e-25, 1.0, 1e25)])
def test_attention_wide_magnitudes(bits, k_scale, v_scale, q_scale):
    c = make(2, 80, 2, 128, 16, bits, 128, [500, 33], seed=42, k_scale=k_scale, v_scale=v_scale)
    c["q"] = (c["q"].float() * q_scale).to(BF)
    check(c)
    for scale in (0.0, -0.125):
        check(dict(c, scale=scale * c["scale"]))


def test_attention_wide_rows_of_unlike_scale():
    """Scores and V scales that grow along the sequence, together and against each other: the references
    rise many times, in either half of a tile."""
    D, P, n = 128, 16, 640
    c = make(1, 40, 1, D, P, 4, D, [n], seed=53)
    g = gen(54)
    q = normals(g, 1, 40, 1, D)
    q[:] = q[:, :1]
    pos = torch.arange(n, device=DEV)
    grow = torch.linspace(-1.0, 1.0, n, device=DEV)[:, None, None]
    slots = c["table"][0, pos // P].long() * P + pos % P
    for sign, order in ((1.0, 1.0), (1.0, -1.0), (-1.0, 1.0)):
        k = (sign * grow * q[0, 0].float() * 4.0 + 0.1 * torch.randn(n, 1, D, generator=g, device=DEV)).to(BF)
        v = (torch.randn(n, 1, D, generator=g, device=DEV) * torch.exp2(order * 30.0 * grow)).to(BF)
        v[5::7] = 0
        B_.decode_attn_append_paged_quant(k, v, c["pool"], slots, 4, D)
        c["q"] = q
        out = run(c)
        ref, _ = oracle(c)
        kk, vv = R.rows(c["pool"].cpu().numpy(), (slots // P).cpu().numpy(), (slots % P).cpu().numpy(), D, P, 4, D)
        x = c["scale"] * (R.f64(q)[0, 0, 0] @ kk[0][:, 0].T)
        p = np.exp(x - x.max())
        w = (p / p.sum())[:, None]
        # as above: weights to fp16 (subnormals: half of 2^-24 of the largest weight * scale), scores to fp32
        d = 2.0 ** -18 * c["scale"] * np.abs(R.f64(q)[0, 0, 0]).sum() * (np.abs(kk[2]) + 15 * kk[1]).max()
        tol = 2.0 ** -8 * np.abs(ref[0, 0, 0]) + (w * (
            (2.0 ** -11 + 2.0 ** -15 + 2 * d) * (15 * vv[1][:, 0] + np.abs(vv[2][:, 0])))).sum(0)
        tol = tol + 2.0 ** -25 * 15 * n * (w * vv[1][:, 0]).max(0)
        for i in range(40):
            R.check(out[0, i, 0], ref[0, i, 0], tol, f"sign {sign} order {order}")


def test_attention_wide_nan_rows():
    """A NaN in the last row reaches the last token's columns only, of its sequence."""
    D, P = 64, 16
    c = make(3, 40, 2, D, P, 8, D, [100, 100, 100], seed=63, sq=2)
    g = gen(64)
    for b, which in ((0, 0), (1, 1)):
        kv = [normals(g, 1, 2, D), normals(g, 1, 2, D)]
        kv[which][0, 1, 40] = float("nan")
        slot = c["table"][b, 99 // P].long() * P + 99 % P
        B_.decode_attn_append_paged_quant(kv[0], kv[1], c["pool"], slot.reshape(1), 8, D)
    out = check(c, True).float()
    assert bool(torch.isnan(out[:2, 20:, 1]).all())
    assert not bool(torch.isnan(out[:, :20]).any()) and not bool(torch.isnan(out[:, :, 0]).any())
    assert not bool(torch.isnan(out[2]).any())


def test_attention_wide_mixed_with_narrow():
    """Calls of both kernels one behind the other on one stream and one workspace."""
    a = make(3, 64, 1, 128, 16, 4, 128, [2000, 31, 450], seed=81)
    b = make(5, 32, 8, 128, 16, 4, 128, [900, 0, 64, 2500, 1], seed=82)
    ws = max(workspace(a), workspace(b), key=lambda t: t.numel())
    want = [run(c).view(torch.int16).clone() for c in (a, b)]
    outs = []
    for i in range(20):
        outs.append(run((a, b)[i % 2], ws=ws))
    for i, out in enumerate(outs):
        assert torch.equal(out.view(torch.int16), want[i % 2])


def test_attention_one_long_sequence():
    """One sequence on every CTA: the merge of many partial rows."""
    check(make(1, 8, 1, 128, 64, 4, 128, [60000], seed=3))
    check(make(2, 8, 2, 64, 256, 8, 32, [30001, 12345], seed=4))
    check(make(1, 64, 1, 128, 16, 4, 128, [40001], seed=5))


def test_attention_stride_3_and_clamped_lengths():
    c = make(4, 16, 4, 128, 16, 4, 64, [100, 37, 64, 200], seed=21)
    rec = torch.tensor([[100, 9, 9], [37, 9, 9], [0, 9, 9], [200, 9, 9]], dtype=torch.int32, device=DEV)
    check(dict(c, lens=rec.flatten(), stride=3))
    cap = c["table"].shape[1] * 16
    full = make(2, 16, 4, 128, 16, 4, 64, [96, 96], seed=22)
    full["lens"] = torch.tensor([97, -1], dtype=torch.int32, device=DEV)     # past the capacity: clamped
    check(full)
    assert cap >= 200


@pytest.mark.parametrize("P", [8, 16, 128])
def test_attention_bad_pages(P):
    """Pages outside the pool are skipped, whatever else the stage holds; all of them: zero rows."""
    c = make(4, 8, 2, 128, P, 4, 64, [500, 500, 3, 40], seed=P)
    t = c["table"].clone()
    t[0, 1], t[0, -1] = -1, 1 << 30
    t[1, ::2] = -7
    t[2, 0] = c["pool"].shape[0]
    c["table"] = t
    out = check(c)
    assert not bool(out[2].any())


def test_attention_same_page_twice():
    c = make(2, 8, 2, 128, 16, 4, 64, [160, 160], seed=31)
    c["table"][0, 3] = c["table"][0, 1]
    c["table"][1] = c["table"][0]
    check(c)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(30.0, 1.0, 1.0), (1.0, 1e-6, 1.0), (1.0, 1e20, 1.0),
                                                     (1e-3, 1.0, 1e4), (1.0, 1.0, 1e-30), (1e-25, 1.0, 1e25)])
def test_attention_magnitudes(bits, k_scale, v_scale, q_scale):
    c = make(2, 8, 2, 128, 16, bits, 64, [500, 33], seed=41, k_scale=k_scale, v_scale=v_scale)
    c["q"] = (c["q"].float() * q_scale).to(BF)
    check(c)


def test_attention_rows_of_unlike_scale():
    """V rows 2^60 apart, the largest ones with the smallest weights, constant rows, zero rows; and
    a score that grows along the sequence, so that every reference is raised many times."""
    D, P, n, Hkv = 128, 16, 640, 2
    c = make(1, 8, Hkv, D, P, 4, 32, [n], seed=51)
    g = gen(52)
    q = normals(g, 1, 8, 1, D)
    q[:] = q[:, :1]
    grow = torch.linspace(-1.0, 1.0, n, device=DEV)[:, None, None]
    k = (grow * q[0, 0].float() * 4.0 + 0.1 * torch.randn(n, Hkv, D, generator=g, device=DEV)).to(BF)
    for order in (1.0, -1.0):
        e = order * 30.0 * grow
        v = (torch.randn(n, Hkv, D, generator=g, device=DEV) * torch.exp2(e)).to(BF)
        v[5::7] = 0
        v[6::7] = 2.5
        slots = c["table"][0, torch.arange(n, device=DEV) // P].long() * P + torch.arange(n, device=DEV) % P
        B_.decode_attn_append_paged_quant(k, v, c["pool"], slots, 4, 32)
        c["q"] = q
        out = run(c)
        ref, _ = oracle(c)
        # per row bounds instead of the largest row's: weights to fp16, scores to fp32
        kk, vv = R.rows(c["pool"].cpu().numpy(), (slots // P).cpu().numpy(), (slots % P).cpu().numpy(), D, P, 4, 32)
        for h in range(Hkv):
            x = c["scale"] * (R.f64(q)[0, 0, 0] @ kk[0][:, h].T)
            p = np.exp(x - x.max())
            w = (p / p.sum())[:, None]
            d = 2.0 ** -18 * c["scale"] * np.abs(R.f64(q)[0, 0, 0]).sum() * (np.abs(kk[2]) + 15 * kk[1]).max()
            tol = 2.0 ** -8 * np.abs(ref[0, 4 * h, 0]) + (w * (
                (2.0 ** -11 + 2.0 ** -15 + 2 * d) * (15 * vv[1][:, h] + np.abs(vv[2][:, h])))).sum(0)
            # fp16 subnormals: half of 2^-24 relative to the largest weight * scale
            tol = tol + 2.0 ** -25 * 15 * n * (w * vv[1][:, h]).max(0)
            for i in range(4):
                R.check(out[0, 4 * h + i, 0], ref[0, 4 * h + i, 0], tol, f"order {order}")


def test_attention_nan_rows_and_infinite_parameters():
    """A NaN in K reaches the heads that read the row; one in V its group's elements; neither
    reaches other sequences, nor tokens that do not see the row."""
    D, P, group = 128, 16, 32
    c = make(3, 8, 2, D, P, 4, group, [100, 100, 100], seed=61, sq=2)
    g = gen(62)
    for b, which in ((0, 0), (1, 1)):
        kv = [normals(g, 1, 2, D), normals(g, 1, 2, D)]
        kv[which][0, 1, 40] = float("nan")
        slot = c["table"][b, 99 // P].long() * P + 99 % P       # the last row: only the last token sees it
        B_.decode_attn_append_paged_quant(kv[0], kv[1], c["pool"], slot.reshape(1), 4, group)
    out = check(c, True).float()
    assert bool(torch.isnan(out[0, 4:, 1]).all()) and not bool(torch.isnan(out[0, :4]).any())
    assert not bool(torch.isnan(out[:, :, 0]).any()) and not bool(torch.isnan(out[2]).any())
    assert bool(torch.isnan(out[1, 4:, 1, 32:64]).all())
    assert not bool(torch.isnan(out[1, 4:, 1, :32]).any()) and not bool(torch.isnan(out[1, 4:, 1, 64:]).any())


def test_attention_scale_zero_and_negative():
    c = make(2, 8, 2, 64, 16, 4, 64, [200, 31], seed=71)
    for scale in (0.0, -0.125):
        check(dict(c, scale=scale))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, rows in its last pages."""
    Hkv, D, P, bits, group = 8, 128, 64, 8, 128
    nbytes = B_.decode_attn_quant_page_bytes(D, P, bits, group)
    pages = (1 << 32) // (Hkv * nbytes) + 9
    pool = torch.empty(pages, Hkv, nbytes, dtype=torch.uint8, device=DEV)
    g = gen(81)
    n = 200
    table = torch.tensor([[pages - 1, 3, pages - 2, pages - 7]], dtype=torch.int32, device=DEV)
    pos = torch.arange(n, device=DEV)
    slots = table[0, pos // P].long() * P + pos % P
    k, v = normals(g, n, Hkv, D), normals(g, n, Hkv, D)
    B_.decode_attn_append_paged_quant(k, v, pool, slots, bits, group)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    B_.decode_attn_read_paged_quant(pool, slots, ko, vo, bits, group)
    assert float((ko.float() - k.float()).abs().max()) < 0.05
    assert float((vo.float() - v.float()).abs().max()) < 0.05
    c = dict(q=normals(g, 1, 32, 1, D), pool=pool, table=table, D=D, P=P, bits=bits, group=group,
             lens=torch.tensor([n], dtype=torch.int32, device=DEV), scale=D ** -0.5)
    out = run(c)
    small = pool[table[0].long()].contiguous()
    ref = dict(c, pool=small, table=torch.arange(4, dtype=torch.int32, device=DEV)[None])
    R.check(out, *oracle(ref))


# ------------------------------------------------------------------ together, streams and graphs
@pytest.mark.parametrize("bits,group", [(4, 32), (4, 128), (8, 64)])
def test_serving_loop(bits, group):
    """A prompt written and read back, then decode steps that append one row per sequence and attend:
    captured once, replayed with lengths and slots rewritten in place."""
    B, Hq, Hkv, D, P, steps = 3, 16, 4, 128, 16, 5
    g = gen(91)
    start = [0, 37, 90]
    pool = B_.new_quant_pool(40, Hkv, D, P, bits, group, DEV)
    table = torch.randperm(40, generator=g, device=DEV)[:B * 8].reshape(B, 8).to(torch.int32)
    for b, n in enumerate(start):
        pos = torch.arange(n, device=DEV)
        slots = table[b, pos // P].long() * P + pos % P
        k, v = normals(g, n, Hkv, D), normals(g, n, Hkv, D)
        B_.decode_attn_append_paged_quant(k, v, pool, slots, bits, group)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        B_.decode_attn_read_paged_quant(pool, slots, ko, vo, bits, group)
    q = torch.empty(B, Hq, 1, D, dtype=BF, device=DEV)
    k, v = (torch.empty(B, Hkv, D, dtype=BF, device=DEV) for _ in "kv")
    slots = torch.empty(B, dtype=torch.int64, device=DEV)
    lens = torch.empty(B, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    c = dict(q=q, pool=pool, table=table, lens=lens, D=D, P=P, bits=bits, group=group, scale=D ** -0.5)
    ws = workspace(c)

    def step():
        B_.decode_attn_append_paged_quant(k, v, pool, slots, bits, group)
        run(c, ws=ws, out=out)

    def inputs(i):
        pos = torch.tensor([n + i for n in start], device=DEV)
        slots.copy_(table.gather(1, (pos // P)[:, None])[:, 0].long() * P + pos % P)
        lens.copy_(pos + 1)
        for x in (q, k, v):
            x.copy_(normals(g, *x.shape))

    inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    R.check(out, *oracle(c), "eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, steps):
        inputs(i)
        graph.replay()
        torch.cuda.synchronize()
        R.check(out, *oracle(c), f"replay {i}")
    assert B_.decode_attn_read_device_error() == 0


def test_two_graphs_share_a_workspace():
    """Two captured calls of unlike shapes on one workspace, replayed in turn."""
    a = make(4, 32, 8, 128, 16, 4, 128, [3000, 17, 0, 900], seed=101)
    b = make(9, 16, 1, 64, 32, 8, 32, [500, 1, 40, 2000, 0, 7, 64, 333, 90], seed=102)
    ws = max(workspace(a), workspace(b), key=lambda w: w.numel())
    want = [run(c).view(torch.int16).clone() for c in (a, b)]
    outs, graphs = [], []
    for c in (a, b):
        out = torch.empty_like(c["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, ws=ws, out=out)
        outs.append(out)
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        outs[i].fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i].view(torch.int16), want[i])


FIRST_CALL = """
import torch
from token_decode_attention_split_gb300 import binding as B
k = torch.randn(40, 2, 64, device="cuda").to(torch.bfloat16)
pool = B.new_quant_pool(4, 2, 64, 16, 4, 64, "cuda")
slots = torch.arange(40, device="cuda")
table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
lens = torch.tensor([40], dtype=torch.int32, device="cuda")
q = torch.randn(1, 8, 1, 64, device="cuda").to(torch.bfloat16)
out, back = torch.zeros_like(q), torch.empty_like(k)
ws = B.new_workspace(B.decode_attn_workspace_size(B.DA_VARIANT_PAGED_QUANT, 1, 8, 2, 64), "cuda")
def calls():
    B.decode_attn_append_paged_quant(k, k, pool, slots, 4, 64)
    B.decode_attn_read_paged_quant(pool, slots, back, torch.empty_like(k), 4, 64)
    B.decode_attn_paged_quant(q, pool, out, table, lens, 1, 4, 64, False, 0.125, ws)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    calls()
g.replay()
torch.cuda.synchronize()
captured = out.clone()
calls()
torch.cuda.synchronize()
assert torch.equal(captured, out) and bool(out.any())
"""


def test_first_call_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_streams_at_once():
    """Two calls in flight together on one pool, each with a workspace of its own."""
    c = make(4, 32, 8, 128, 16, 4, 128, [3000, 17, 2000, 900], seed=95)
    d = dict(c, q=normals(gen(96), *c["q"].shape))
    want = [run(x).clone() for x in (c, d)]
    spaces = [workspace(x) for x in (c, d)]
    outs = [torch.empty_like(c["q"]) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for x, ws, o, st in zip((c, d), spaces, outs, streams):
            with torch.cuda.stream(st):
                run(x, ws=ws, out=o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.int16), w.view(torch.int16))


def test_same_result_every_time():
    c = make(6, 32, 8, 128, 16, 4, 32, [5000, 100, 2222, 1, 0, 777], seed=97)
    ws = workspace(c)
    a = run(c, ws=ws).view(torch.int16).clone()
    for _ in range(30):
        assert torch.equal(run(c, ws=ws).view(torch.int16), a)


def test_nothing_to_do():
    pool = B_.new_quant_pool(2, 2, 64, 16, 4, 64, DEV)
    e = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    s = torch.empty(0, dtype=torch.int64, device=DEV)
    B_.decode_attn_append_paged_quant(e, e, pool, s, 4, 64)
    B_.decode_attn_read_paged_quant(pool, s, e, e, 4, 64)
    q = torch.empty(0, 4, 1, 64, dtype=BF, device=DEV)
    B_.decode_attn_paged_quant(q, pool, q, torch.empty(0, 1, dtype=torch.int32, device=DEV),
                               torch.empty(1, dtype=torch.int32, device=DEV), 1, 4, 64, False, 0.1,
                               B_.new_workspace(256, DEV))
    assert not bool(pool.any())


def test_refused_workspace_and_shapes():
    c = make(2, 8, 2, 64, 16, 4, 64, [20, 3], seed=99)
    out = torch.full_like(c["q"], 3.0)
    with pytest.raises(B_.DecodeAttnError) as e:
        run(c, ws=torch.zeros(256, dtype=torch.uint8, device=DEV), out=out)
    assert e.value.status == 3 and bool((out == 3.0).all())
    with pytest.raises(ValueError):
        run(dict(c, q=c["q"].float()), ws=workspace(c), out=out)
    with pytest.raises(ValueError):
        run(dict(c, q=c["q"].transpose(1, 2)), ws=workspace(c), out=out)
    with pytest.raises(ValueError):
        run(dict(c, lens=c["lens"].cpu()), ws=workspace(c), out=out)
    with pytest.raises(ValueError):
        run(dict(c, lens=c["lens"].float()), ws=workspace(c), out=out)
    with pytest.raises(ValueError):
        run(dict(c, lens=c["lens"][:1]), ws=workspace(c), out=out)
    with pytest.raises(ValueError):
        run(dict(c, group=128), ws=workspace(c), out=out)
