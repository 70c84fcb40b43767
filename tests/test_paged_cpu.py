"""CPU checks of the paged-cache entry points: struct layouts, exports, and
refusals (every check runs before any CUDA call, on fake addresses)."""
import os
import struct

import pytest
import torch

import io_aware_exact_18_b200 as fa
from io_aware_exact_18_b200 import build as fa_build
from io_aware_exact_18_b200 import paged
from tests.test_rotary_cpu import INCLUDE, c_sizes


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def test_structs_match_the_header(tmp_path):
    got = c_sizes(tmp_path, "fa_paged.h", ["fa_paged_cache_t", "fa_block_table_t",
                                           "fa_paged_append_t", "fa_paged_decode_t"])
    assert got == [struct.calcsize("@" + paged.CACHE), struct.calcsize("@" + paged.TABLE),
                   paged._APPEND.size, paged._DECODE.size]


def test_library_exports_the_header(lib):
    names = fa.declared_symbols(os.path.join(INCLUDE, "fa_paged.h"))
    assert names == ["fa_copy_pages", "fa_paged_append", "fa_paged_decode",
                     "fa_paged_decode_workspace_bytes"]
    for n in names:
        assert hasattr(lib, n)


P = 1 << 40
G = 1 << 32
# 100 pages of 16 tokens, 2 heads of 128
CACHE = dict(kc=P, vc=P + G, sp=2 * 16 * 128, sh=16 * 128, st=128, pages=100, page=16, H_kv=2,
             d=128, elem=2, ks=1.0, vs=1.0, table=P + 2 * G, ts=40, seqs=4, width=40)


def cache_fields(a):
    return (a["kc"], a["vc"], a["sp"], a["sh"], a["st"], a["pages"], a["page"], a["H_kv"], a["d"],
            a["elem"], a["ks"], a["vs"], 0)


def table_fields(a):
    return (a["table"], a["ts"], a["seqs"], a["width"])


BAD_CACHE = [
    (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(elem=4), fa.FA_ERR_UNSUPPORTED),
    (dict(page=0), fa.FA_ERR_INVALID_ARG),
    (dict(page=65537), fa.FA_ERR_INVALID_ARG),
    (dict(pages=-1), fa.FA_ERR_INVALID_ARG),
    (dict(H_kv=-1), fa.FA_ERR_INVALID_ARG),
    (dict(ks=0.5), fa.FA_ERR_INVALID_ARG),                  # bf16 pages have no descale
    (dict(elem=1, ks=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(elem=1, vs=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(elem=1, vs=float("inf")), fa.FA_ERR_INVALID_ARG),
    (dict(kc=0), fa.FA_ERR_INVALID_ARG),
    (dict(vc=P + G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(vc=P), fa.FA_ERR_INVALID_ARG),                    # K is V
    (dict(st=132), fa.FA_ERR_INVALID_ARG),                  # 264 bytes
    (dict(st=64), fa.FA_ERR_INVALID_ARG),                   # rows run into one another
    (dict(sh=15 * 128), fa.FA_ERR_INVALID_ARG),             # heads run into one another
    (dict(sp=16 * 128), fa.FA_ERR_INVALID_ARG),             # pages run into one another
    (dict(sp=-4096), fa.FA_ERR_INVALID_ARG),
]
BAD_TABLE = [
    (dict(table=0), fa.FA_ERR_INVALID_ARG),
    (dict(table=P + 2 * G + 2), fa.FA_ERR_INVALID_ARG),
    (dict(ts=-1), fa.FA_ERR_INVALID_ARG),
    (dict(seqs=-1), fa.FA_ERR_INVALID_ARG),
    (dict(width=-1), fa.FA_ERR_INVALID_ARG),
]

AP = dict(CACHE, k=P + 3 * G, v=P + 4 * G, q=P + 5 * G, qo=P + 6 * G, pos=P + 7 * G, psb=1, psn=1,
          seq=0, freqs=P + 8 * G, wq=0, wk=0, rot=128, inter=0, norm=0, w32=0, scale=1.0, eps=0.0,
          B=4, H=8, N=1, ks_=(256, 128, 128), qs=(1024, 128, 128), qos=(1024, 128, 128))


def append(lib, **over):
    a = dict(AP, **over)
    args = paged._APPEND.pack(*cache_fields(a), *table_fields(a), a["k"], *a["ks_"], a["v"],
                              *a["ks_"], a["q"], *a["qs"], a["qo"], *a["qos"], a["pos"], a["psb"],
                              a["psn"], a["seq"], a["freqs"], a["wq"], a["wk"], a["rot"],
                              a["inter"], a["norm"], a["w32"], a["scale"], a["eps"], a["B"],
                              a["H"], a["N"], 0)
    return lib.fa_paged_append(args, None)


@pytest.mark.parametrize("over,status", BAD_CACHE + BAD_TABLE + [
    (dict(rot=20), fa.FA_ERR_INVALID_ARG),
    (dict(norm=1, eps=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(pos=0), fa.FA_ERR_INVALID_ARG),
    (dict(pos=0, rot=0), fa.FA_ERR_INVALID_ARG),            # positions place the tokens too
    (dict(seq=P + 1), fa.FA_ERR_INVALID_ARG),
    (dict(qo=0), fa.FA_ERR_INVALID_ARG),                    # q without q_out
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(k=0), fa.FA_ERR_INVALID_ARG),
    (dict(v=P + 4 * G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(k=P + 1024), fa.FA_ERR_INVALID_ARG),              # inside the cache
    (dict(qo=P + G + 64), fa.FA_ERR_INVALID_ARG),
    (dict(qo=P + 3 * G), fa.FA_ERR_INVALID_ARG),            # over k
    (dict(qo=P + 5 * G + 256), fa.FA_ERR_INVALID_ARG),      # shifted over q
    (dict(qos=(1024, 0, 128)), fa.FA_ERR_INVALID_ARG),
    (dict(pos=P + 64), fa.FA_ERR_INVALID_ARG),              # positions in the cache
    (dict(table=P + G), fa.FA_ERR_INVALID_ARG),
    (dict(seq=P + 6 * G), fa.FA_ERR_INVALID_ARG),           # under q_out
    (dict(freqs=P + 6 * G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(B=-1), fa.FA_ERR_INVALID_ARG),
    (dict(N=1 << 30), fa.FA_ERR_INVALID_ARG),
    (dict(B=0), fa.FA_OK),
    (dict(N=0, k=0, v=0, q=0, qo=0), fa.FA_OK),
    (dict(q=0, qo=0, H_kv=0, kc=0, vc=0, k=0, v=0), fa.FA_OK),
])
def test_append_refusals(lib, over, status):
    assert append(lib, **over) == status


DE = dict(CACHE, q=P + 3 * G, qsb=1024, qsh=128, o=P + 4 * G, lse=P + 5 * G, lens=P + 6 * G,
          B=4, H=8, scale=0.088, ws=P + 7 * G, ws_bytes=1 << 28)


def decode(lib, **over):
    a = dict(DE, **over)
    args = paged._DECODE.pack(*cache_fields(a), *table_fields(a), a["q"], a["qsb"], a["qsh"],
                              a["o"], a["lse"], a["lens"], a["B"], a["H"], a["scale"], 0)
    return lib.fa_paged_decode(args, a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("over,status", BAD_CACHE + BAD_TABLE + [
    (dict(H=7), fa.FA_ERR_INVALID_ARG),
    (dict(H=1), fa.FA_ERR_INVALID_ARG),
    (dict(H_kv=0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(seqs=3), fa.FA_ERR_INVALID_ARG),                  # fewer table rows than sequences
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(q=P + 3 * G + 4), fa.FA_ERR_INVALID_ARG),
    (dict(qsh=132), fa.FA_ERR_INVALID_ARG),
    (dict(qsb=-1024), fa.FA_ERR_INVALID_ARG),
    (dict(o=0), fa.FA_ERR_INVALID_ARG),
    (dict(lse=P + 5 * G + 2), fa.FA_ERR_INVALID_ARG),
    (dict(lens=0), fa.FA_ERR_INVALID_ARG),
    (dict(ws=0), fa.FA_ERR_INVALID_ARG),
    (dict(ws=P + 7 * G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(ws_bytes=1000), fa.FA_ERR_INVALID_ARG),
    (dict(ws=P + 4 * G), fa.FA_ERR_INVALID_ARG),            # over o
    (dict(ws=P + 2 * G), fa.FA_ERR_INVALID_ARG),            # over the table
    (dict(o=P + 512), fa.FA_ERR_INVALID_ARG),               # in the cache
    (dict(o=P + 3 * G), fa.FA_ERR_INVALID_ARG),             # over q
    (dict(lse=P + 4 * G + 64), fa.FA_ERR_INVALID_ARG),      # in o
    (dict(lse=P + 6 * G), fa.FA_ERR_INVALID_ARG),           # over kv_len
    (dict(B=1 << 24), fa.FA_ERR_INVALID_ARG),
    (dict(B=0), fa.FA_OK),
    (dict(H=0, q=0, o=0, lse=0, ws=0), fa.FA_OK),
])
def test_decode_refusals(lib, over, status):
    assert decode(lib, **over) == status


@pytest.mark.parametrize("over,status", [(o, s) for o, s in BAD_CACHE] + [
    (dict(src=0), fa.FA_ERR_INVALID_ARG),
    (dict(dst=P + 5 * G + 2), fa.FA_ERR_INVALID_ARG),
    (dict(src=P + 64), fa.FA_ERR_INVALID_ARG),              # in the cache
    (dict(n=-1), fa.FA_ERR_INVALID_ARG),
    (dict(n=1 << 30), fa.FA_ERR_INVALID_ARG),
    (dict(n=0, src=0, dst=0), fa.FA_OK),
    (dict(pages=0, kc=0, vc=0), fa.FA_OK),
])
def test_copy_refusals(lib, over, status):
    a = dict(CACHE, src=P + 4 * G, dst=P + 5 * G, n=3)
    a.update(over)
    assert lib.fa_copy_pages(paged._COPY.pack(*cache_fields(a)), a["src"], a["dst"], a["n"],
                             None) == status


def test_null_args(lib):
    assert lib.fa_paged_append(None, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_paged_decode(None, None, 0, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_copy_pages(None, None, None, 0, None) == fa.FA_ERR_INVALID_ARG


def test_workspace_bytes(lib):
    """Bounded by the blocks, not by lengths; a row more per sequence."""
    f = lib.fa_paged_decode_workspace_bytes
    assert f(0, 8, 2, 128) == 0 and f(4, 8, 3, 128) == 0 and f(4, 8, 2, 96) == 0
    assert f(4, 8, 2, 128) >= 148 * 2 * 8 * 129 * 4
    assert f(1024, 8, 2, 128) - f(4, 8, 2, 128) < 1 << 15


def test_wrappers_refuse():
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.paged_append(x, x, kc, kc.clone(), t, t[:, :1])
    with pytest.raises(TypeError):
        fa.paged_decode_attention(x, kc.float(), kc.float(), t, t[0, :1])
    with pytest.raises(ValueError):
        fa.copy_pages(kc, kc.clone(), t[0], t[0])


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("descale", [2.0 ** -149, 2.0 ** -130, 2.0 ** -128])
def test_append_refuses_descales_without_a_reciprocal(lib, which, descale):
    """Codes are products with 1 / descale: infinite below 2^-128, and zeros would
    be stored as NaN."""
    assert append(lib, elem=1, **{which: descale}) == fa.FA_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on fake pointers")
def test_small_descales_are_accepted(lib):
    """Append from the first descale on whose reciprocal is finite; reading any."""
    assert append(lib, elem=1, ks=2.0 ** -127, vs=2.0 ** -127) != fa.FA_ERR_INVALID_ARG
    assert append(lib, elem=1, ks=2.0 ** 127, vs=1e38) != fa.FA_ERR_INVALID_ARG
    assert decode(lib, elem=1, ks=2.0 ** -140, vs=2.0 ** -140) != fa.FA_ERR_INVALID_ARG


def kv_layouts():
    """(cache fields, whether K and V share an element) for V at many offsets from K
    in buffers that hold both, by counting the elements themselves."""
    H, page, d = 2, 4, 64
    cases = []
    for pages, sp, sh, st in ((3, 2 * H * page * d, page * d, d),          # [pages, 2, H, page, d]
                              (3, 2 * H * page * d, 2 * page * d, d),      # [pages, H, 2, page, d]
                              (3, 2 * H * page * d, 2 * d, 2 * H * d),     # [pages, page, H, 2, d]
                              (3, 2 * H * page * d, d, 2 * H * d),         # [pages, page, 2, H, d]
                              (3, H * page * d, page * d, d),              # dense
                              (1, 0, page * d + 32, d)):                   # one page, padded heads
        rows = {p * sp + h * sh + t * st for p in range(pages) for h in range(H) for t in range(page)}
        taken = {r + j for r in rows for j in range(0, d, 8)}
        for off in range(-2 * max(taken), 2 * max(taken), 8 * 4):
            shared = any(r + off + j in taken for r in rows for j in range(0, d, 8))
            cases.append((dict(vc=P + (1 << 24) + 2 * off, kc=P + (1 << 24), sp=sp, sh=sh, st=st,
                               pages=pages, page=page, H_kv=H, d=d), shared))
    return cases


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on fake pointers")
def test_keys_and_values_that_share_elements_are_refused(lib):
    """K and V may lie in one buffer as long as no element is both."""
    a = dict(CACHE, src=P + 4 * G, dst=P + 5 * G)
    some = {True: 0, False: 0}
    for over, shared in kv_layouts():
        a.update(over)
        st = lib.fa_copy_pages(paged._COPY.pack(*cache_fields(a)), a["src"], a["dst"], 3, None)
        assert (st == fa.FA_ERR_INVALID_ARG) == shared, over
        some[shared] += 1
    assert min(some.values()) > 100


@pytest.mark.parametrize("over", [dict(vc=P + 256), dict(vc=P + 2 * 16 * 128 * 2),
                                  dict(vc=P - 99 * 2 * 16 * 128 * 2),
                                  dict(sp=4 * 16 * 128, vc=P + 2 * 16 * 128 * 2 - 256)])
def test_overlapping_caches_are_refused(lib, over):
    """V a row, a page or 99 pages of K away, or a row into its half of a buffer."""
    assert append(lib, **over) == fa.FA_ERR_INVALID_ARG
    a = dict(CACHE, **over)
    assert lib.fa_copy_pages(paged._COPY.pack(*cache_fields(a)), P + 4 * G, P + 5 * G, 3,
                             None) == fa.FA_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on fake pointers")
def test_reading_overlapping_caches_is_accepted(lib):
    """Values that are part of the keys' rows, or a page away, are only read."""
    assert decode(lib, vc=P + 2 * 16 * 128 * 2) != fa.FA_ERR_INVALID_ARG
    assert decode(lib, st=192, sh=16 * 192, sp=2 * 16 * 192, vc=P + 128) != fa.FA_ERR_INVALID_ARG
