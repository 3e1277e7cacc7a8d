"""The quantised cache's calls on the host, no GPU needed: sizes, and what they refuse before
anything touches the device."""
import ctypes
import math

import numpy as np
import pytest
import torch

import quant_ref as R
from token_decode_attention_split_gb300 import binding as B_
from token_decode_attention_split_gb300 import build

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B_.load_library()


@pytest.mark.parametrize("D,P,bits,group,want", [(128, 16, 4, 128, 16 * 136), (128, 64, 4, 32, 64 * 160),
                                                 (64, 8, 4, 64, 8 * 72), (128, 256, 8, 64, 256 * 272)])
def test_page_bytes(lib, D, P, bits, group, want):
    assert B_.decode_attn_quant_page_bytes(D, P, bits, group) == want == P * R.row_bytes(D, bits, group)


@pytest.mark.parametrize("D,P,bits,group", [(96, 16, 4, 32), (128, 12, 4, 32), (128, 4, 4, 32),
                                            (128, 512, 4, 32), (128, 16, 2, 32), (128, 16, 16, 32),
                                            (64, 16, 4, 128), (128, 16, 4, 16), (128, 16, 4, 0),
                                            (0, 16, 4, 32), (128, 0, 4, 32), (128, -16, 4, 32)])
def test_formats_refused(lib, D, P, bits, group):
    assert B_.decode_attn_quant_page_bytes(D, P, bits, group) == 0
    with pytest.raises(ValueError):
        B_.new_quant_pool(1, 1, D, P, bits, group, "cpu")


def append(lib, k=FAKE, v=FAKE, ks=256, vs=256, pool=FAKE, slots=FAKE, T=4, Hkv=2, D=128, P=16,
           pages=8, bits=4, group=64):
    return lib.decode_attn_append_paged_quant(k, v, ks, vs, pool, slots, T, Hkv, D, P, pages, bits,
                                              group, None)


def test_append_rejects(lib):
    for name in ("k", "v", "pool", "slots"):
        assert append(lib, **{name: None}) == INVALID
    assert append(lib, k=FAKE + 8) == INVALID
    assert append(lib, pool=FAKE + 8) == INVALID
    assert append(lib, slots=FAKE + 4) == INVALID
    assert append(lib, T=-1) == INVALID
    assert append(lib, Hkv=0) == INVALID
    assert append(lib, pages=-1) == INVALID
    assert append(lib, P=0) == INVALID
    assert append(lib, ks=255) == INVALID            # rows would overlap
    assert append(lib, vs=128) == INVALID
    assert append(lib, ks=257) == UNSUPPORTED        # rows must start on 16 bytes
    assert append(lib, ks=(1 << 62)) == UNSUPPORTED
    assert append(lib, D=96) == UNSUPPORTED
    assert append(lib, P=24) == UNSUPPORTED
    assert append(lib, bits=3) == UNSUPPORTED
    assert append(lib, group=16) == UNSUPPORTED
    assert append(lib, Hkv=4096, ks=1 << 20, vs=1 << 20) == UNSUPPORTED
    assert append(lib, pages=1 << 31) == UNSUPPORTED
    assert append(lib, T=0) == OK                    # nothing to write


def test_read_rejects(lib):
    def read(pool=FAKE, slots=FAKE, k=FAKE, v=FAKE, T=4, Hkv=2, D=128, P=16, pages=8, bits=4, group=64):
        return lib.decode_attn_read_paged_quant(pool, slots, k, v, T, Hkv, D, P, pages, bits, group, None)
    for name in ("k", "v", "pool", "slots"):
        assert read(**{name: None}) == INVALID
    assert read(k=FAKE + 2) == INVALID
    assert read(T=-1) == INVALID
    assert read(D=32) == UNSUPPORTED
    assert read(bits=5) == UNSUPPORTED
    assert read(group=128, D=64) == UNSUPPORTED
    assert read(T=1 << 41) == UNSUPPORTED
    assert read(T=0) == OK


def test_attention_rejects(lib):
    def call(q=FAKE, pool=FAKE, out=FAKE, bt=FAKE, maxp=4, P=16, pages=16, kl=FAKE, stride=1, B=2, Hq=8,
             Hkv=2, D=128, Sq=1, bits=4, group=64, scale=0.1, ws=FAKE):
        return lib.decode_attn_paged_quant(q, pool, out, bt, maxp, P, pages, kl, stride, B, Hq, Hkv, D,
                                           Sq, 0, bits, group, scale, ws, 1 << 20, None)
    for name in ("q", "pool", "out", "bt", "kl", "ws"):
        assert call(**{name: None}) == INVALID
    assert call(pool=FAKE + 8) == INVALID
    assert call(kl=FAKE + 2) == INVALID
    assert call(stride=2) == INVALID
    assert call(Hq=7) == INVALID
    assert call(Sq=0) == INVALID
    assert call(maxp=0) == INVALID
    assert call(pages=0) == INVALID
    assert call(scale=math.nan) == INVALID
    assert call(B=-1) == INVALID
    assert call(D=96) == UNSUPPORTED
    assert call(Hq=130, Hkv=2) == UNSUPPORTED        # 65 columns
    assert call(Sq=17) == UNSUPPORTED                # 68 columns
    assert call(Sq=1 << 30) == UNSUPPORTED
    assert call(P=48) == UNSUPPORTED
    assert call(bits=6) == UNSUPPORTED
    assert call(group=256) == UNSUPPORTED
    assert call(B=1025) == UNSUPPORTED
    assert call(pages=1 << 31) == UNSUPPORTED
    assert call(maxp=1 << 23, P=256) == UNSUPPORTED  # 2^31 rows of capacity
    assert call(B=0) == OK


def test_binding_refuses_host_tensors(lib):
    """Wrong devices, types and shapes never reach the library."""
    bf = torch.bfloat16
    pool = B_.new_quant_pool(2, 2, 128, 16, 4, 64, "cpu")
    rows, slots = torch.zeros(3, 2, 128, dtype=bf), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        B_.decode_attn_append_paged_quant(rows, rows, pool, slots, 4, 64)
    with pytest.raises(ValueError):
        B_.decode_attn_read_paged_quant(pool, slots, rows, rows, 4, 64)
    q = torch.zeros(1, 4, 1, 128, dtype=bf)
    with pytest.raises(ValueError):
        B_.decode_attn_paged_quant(q, pool, q, torch.zeros(1, 1, dtype=torch.int32),
                                   torch.zeros(1, dtype=torch.int32), 1, 4, 64, False, 0.1,
                                   torch.zeros(256, dtype=torch.uint8))


# ------------------------------------------------------------------ the oracle itself
def test_oracle_quantiser_by_brute_force():
    """Nearest of all levels, ties to the even code; the smallest bf16 scale that covers the range."""
    rng = np.random.RandomState(3)
    for bits in (4, 8):
        x = torch.from_numpy(rng.randn(6, 64)).to(torch.bfloat16).double().numpy()
        x[0] = rng.randint(-50, 50, 64)
        x[1] = 2.5
        c, s, lo = R.quantise(x, bits, 32)
        for r in range(6):
            for g in range(2):
                v = x[r, 32 * g:32 * g + 32]
                assert lo[r, g] == v.min()
                if v.max() == v.min():
                    assert s[r, g] == 0
                    continue
                assert s[r, g] * (2 ** bits - 1) >= v.max() - v.min()
                below = torch.tensor(s[r, g]).to(torch.bfloat16).view(torch.int16) - 1
                assert float(below.view(torch.bfloat16)) * (2 ** bits - 1) < v.max() - v.min()
                for i, e in enumerate(v):
                    d = np.abs(lo[r, g] + s[r, g] * np.arange(2 ** bits) - e)
                    best = np.flatnonzero(d == d.min())
                    code = c[r, 32 * g + i]
                    assert code in best and (len(best) == 1 or code % 2 == 0)


def test_oracle_pack_and_rows_agree():
    rng = np.random.RandomState(4)
    for D, bits, group, P in ((64, 4, 32, 8), (128, 8, 128, 16), (128, 4, 64, 32)):
        pool = np.zeros((2, 3, P * R.row_bytes(D, bits, group)), np.uint8)
        k, v = (torch.from_numpy(rng.randn(P + 3, 3, D)).to(torch.bfloat16).double().numpy() for _ in "kv")
        slots = np.arange(P + 3)
        R.append(pool, k, v, slots, D, P, bits, group)
        for x, (y, s, lo) in zip((k, v), R.rows(pool, slots // P, slots % P, D, P, bits, group)):
            assert np.all(np.abs(x - y) <= s / 2 + 1e-12)
