"""GPU parity of paged_append, paged_decode_attention and copy_pages against the
fp64 oracles (oracle/rotary.py, oracle/paged.py).

Tolerances of the attention. A score is an fp32 sum of d exact products: off by
at most e = scale d 2^-23 sum |q_i k_i| (each addition by one unit, truncating),
and each exponential by 2^-21 relative besides. lse is then off by at most
e + 2^-20 plus the fp32 sums' chains (under 2^12 additions a thread, then trees):
2^-12 at the very worst, in practice far less; the bound takes 2^-17 for chains
under 2^7. The weights are off by the rounding of p, u = 2^-16 (two bf16 parts,
half a step 2^-8 of the rest, itself at most 2^-8 of p) or 2^-11 (f16), e and
2^-21: O by twice that times sum w |v - O|. bf16 divides by the sum of the exact
p: u sum w |v| more. f16 probabilities under 2^-14 are off by 2^-25 each instead:
sum |v - O| / sum exp. The fp32 sums of O add 2^-17 sum w |v|, the last rounding
2^-8 |O|. Append: see tests/test_rotary_gpu.py; an e4m3 code is off by half a
step, 2^-4 of the value or 2^-10 among subnormals."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as opaged
from oracle import rotary as orot
from tests.test_rotary_gpu import DEV, TINY, U, fa, np64, partner_sum, weights  # noqa: F401

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def pages_of(P, H_kv, page, d, elem, token_major=False, seed=0, ks=0.02, vs=0.01, mult=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (P, page, H_kv, d) if token_major else (P, H_kv, page, d)
    out = []
    for s in (ks, vs):
        x = torch.randn(shape, generator=g, device=DEV) * mult
        x = (x / s).clamp(-448, 448).to(E4M3) if elem == 1 else x.to(torch.bfloat16)
        out.append(x.transpose(1, 2) if token_major else x)
    return out[0], out[1], (ks if elem == 1 else 1.0), (vs if elem == 1 else 1.0)


def decode_and_check(fa, q, kc, vc, ks, vs, table, lens, what="", scale=None, **kw):
    d = q.shape[-1]
    o, lse = fa.paged_decode_attention(q, kc, vc, table, lens, scale=scale, k_descale=ks,
                                       v_descale=vs, **kw)
    torch.cuda.synchronize()
    scale = 1 / math.sqrt(d) if scale is None else scale
    ro, rl, x = opaged.decode(np64(q)[:, :, 0], np64(kc) * ks, np64(vc) * vs,
                              table.cpu().numpy(), lens.cpu().numpy(), scale)
    e = scale * d * 2.0 ** -23 * x["mag"]
    empty = np.isneginf(rl)
    gl, go = np64(lse)[..., 0], np64(o)[:, :, 0]
    assert np.array_equal(np.isneginf(gl), empty), what
    lerr = np.abs(gl[~empty] - rl[~empty])
    assert np.all(lerr <= (e + 2.0 ** -20 + 2.0 ** -17)[~empty] + U * np.abs(rl[~empty])), \
        f"{what}: lse {lerr.max()}"
    u = 2.0 ** -16 if kc.dtype == torch.bfloat16 else 2.0 ** -11
    tol = 2 * (u + e[..., None] + 2.0 ** -21) * x["dev"] + 2.0 ** -17 * x["absv"] \
        + 2.0 ** -8 * np.abs(ro) + TINY
    if kc.dtype == torch.bfloat16:
        tol = tol + u * x["absv"]
    if kc.dtype != torch.bfloat16:
        tol = tol + 2.0 ** -24 * x["flat"]
    err = np.abs(go - ro)
    assert np.all(err <= tol), f"{what}: O off by {err.max()} ({(err - tol).max()} over)"
    return o, lse


def shuffled_table(P, B, width, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(P, generator=g)[:B * width].view(B, width).to(torch.int32).to(DEV)


def queries(B, H, d, seed=1, mult=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, H, 1, d, generator=g) * mult).to(torch.bfloat16).to(DEV)


HEADS = [(1, 1), (4, 4), (6, 2), (8, 1), (9, 1), (16, 1), (20, 1), (40, 2)]


@pytest.mark.parametrize("elem", [2, 1])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,H_kv", HEADS)
def test_decode_heads(fa, H, H_kv, d, elem):  # noqa: F811
    """Every head grouping on both sides of the 8- and 16-head tiles, lengths
    0, 1 and around the tiles."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]
    B, page = len(lens), 16
    width = -(-max(lens) // page)
    kc, vc, ks, vs = pages_of(B * width + 3, H_kv, page, d, elem, seed=d + H)
    decode_and_check(fa, queries(B, H, d), kc, vc, ks, vs, shuffled_table(B * width + 3, B, width),
                     torch.tensor(lens, dtype=torch.int32, device=DEV), f"H{H} H_kv{H_kv} d{d}")


@pytest.mark.parametrize("elem", [2, 1])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 128, 200])
def test_decode_pages(fa, page, token_major, elem):  # noqa: F811
    """Page sizes that end inside a tile and hold several; both page orders."""
    lens = [37, 513, 1, 200]
    width = -(-max(lens) // page)
    P = 4 * width + 2
    kc, vc, ks, vs = pages_of(P, 2, page, 128, elem, token_major, seed=page)
    decode_and_check(fa, queries(4, 8, 128), kc, vc, ks, vs, shuffled_table(P, 4, width, page),
                     torch.tensor(lens, dtype=torch.int32, device=DEV), f"page {page}")


@pytest.mark.parametrize("elem", [2, 1])
def test_decode_shared_out(fa, elem):  # noqa: F811
    """One long sequence over all blocks among short ones, and a tail."""
    lens = [3, 9000, 40, 0, 7, 1111]
    width = -(-9000 // 32)
    kc, vc, ks, vs = pages_of(6 * width, 2, 32, 128, elem, seed=4)
    decode_and_check(fa, queries(6, 8, 128), kc, vc, ks, vs, shuffled_table(6 * width, 6, width),
                     torch.tensor(lens, dtype=torch.int32, device=DEV))


def test_decode_many_sequences(fa):  # noqa: F811
    """More sequences than threads of a block (several a thread in the scan)."""
    rng = np.random.default_rng(0)
    B, width = 700, 3
    lens = rng.integers(0, 40, B).astype(np.int32)
    kc, vc, _, _ = pages_of(B * width, 1, 16, 64, 2, seed=5)
    decode_and_check(fa, queries(B, 2, 64), kc, vc, 1.0, 1.0, shuffled_table(B * width, B, width),
                     torch.from_numpy(lens).to(DEV))


@pytest.mark.parametrize("elem", [2, 1])
def test_decode_hidden_slots_hold_anything(fa, elem):  # noqa: F811
    """NaN in every slot past a sequence's length and in every page that no
    sequence lists; table entries past the length that name no page."""
    B, page, width = 3, 16, 8
    lens = torch.tensor([5, 33, 100], dtype=torch.int32, device=DEV)
    kc, vc, ks, vs = pages_of(B * width + 4, 2, page, 128, elem, seed=6)
    table = shuffled_table(B * width + 4, B, width)
    used = torch.zeros(B * width + 4, page, dtype=torch.bool, device=DEV)
    for b in range(B):
        for j in range(int(lens[b])):
            used[table[b, j // page], j % page] = True
    for c in (kc, vc):
        raw = c.view(torch.uint8) if elem == 1 else c.view(torch.int16)
        nan = 0x7F if elem == 1 else 0x7FC0
        raw.masked_fill_(~used[:, None, :, None], nan)
    for b in range(B):
        last = -(-int(lens[b]) // page)
        table[b, last:] = torch.tensor([-1, 1 << 30], dtype=torch.int32).repeat(8)[:width - last]
    o, _ = decode_and_check(fa, queries(B, 6, 128), kc, vc, ks, vs, table, lens)
    assert torch.isfinite(o).all()


def test_decode_bad_pages_hide_keys(fa):  # noqa: F811
    """A listed page outside the cache hides its keys; a sequence with no other
    is empty; kv_len is clamped to the table's width and to 0."""
    kc, vc, _, _ = pages_of(12, 2, 16, 64, 2, seed=7)
    table = torch.tensor([[0, -1, 2], [99, -5, 12], [3, 4, 5], [6, 7, 8]], dtype=torch.int32,
                         device=DEV)
    lens = torch.tensor([45, 48, 1000000, -3], dtype=torch.int32, device=DEV)
    o, lse = fa.paged_decode_attention(queries(4, 4, 64), kc, vc, table, lens)
    clamped = torch.tensor([45, 48, 48, 0], dtype=torch.int32, device=DEV)
    o2, lse2 = decode_and_check(fa, queries(4, 4, 64), kc, vc, 1.0, 1.0, table, clamped)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b in (1, 3):
        assert (o[b] == 0).all() and torch.isneginf(lse[b]).all()


@pytest.mark.parametrize("elem", [2, 1])
def test_decode_moving_reference(fa, elem):  # noqa: F811
    """Scores that rise by 16 log2 units from one 16-key group to the next, and
    fall again: the reference moves in every group; and flat scores."""
    d, n, page = 128, 640, 16
    kc, vc, ks, vs = pages_of(n // page, 1, page, d, elem, seed=8, ks=1.0, vs=0.01)
    step = torch.cat([torch.arange(20), torch.arange(20).flip(0)]).float()
    k = torch.zeros(n // page, 1, page, d, device=DEV)
    k[..., 0] = (step[:n // page, None, None] * 2).to(DEV)
    kc = k.to(E4M3 if elem == 1 else torch.bfloat16)
    q = torch.zeros(1, 4, 1, d, device=DEV)
    q[..., 0] = torch.tensor([1.0, 64.0, 512.0, -64.0], device=DEV)[None, :, None]
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    decode_and_check(fa, q.to(torch.bfloat16), kc, vc, 1.0, vs, table, lens)


@pytest.mark.parametrize("mult", [2.0 ** -60, 2.0 ** 60, 0.0])
def test_decode_e4m3_query_range(fa, mult):  # noqa: F811
    """Queries far outside f16's range: the power-of-two scaling keeps them."""
    kc, vc, ks, vs = pages_of(8, 1, 16, 128, 1, seed=9)
    q = queries(1, 5, 128, mult=mult)
    scale = 0.1 / mult if mult else 0.1
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([120], dtype=torch.int32, device=DEV)
    decode_and_check(fa, q, kc, vc, ks, vs, table, lens, scale=scale)


def test_decode_nan_queries_and_visible_nan(fa):  # noqa: F811
    """A NaN in one head's query or in a visible key or value reaches the rows
    that use it and no others."""
    kc, vc, _, _ = pages_of(60, 2, 16, 64, 2, seed=10)
    q = queries(3, 4, 64)
    q[0, 1] = float("nan")
    kc[5, 1, 3, 7] = float("nan")        # in sequences 0 and 1, heads 2 and 3
    vc[45, 0, 2, 9] = float("nan")       # sequence 2, heads 0 and 1, column 9
    table = torch.arange(60, dtype=torch.int32, device=DEV).view(3, 20)
    table[1, 0] = 5
    lens = torch.tensor([300, 300, 300], dtype=torch.int32, device=DEV)
    o, lse = fa.paged_decode_attention(q, kc, vc, table, lens)
    bad = torch.isnan(lse[..., 0]).nonzero().tolist()
    assert bad == [[0, 1], [0, 2], [0, 3], [1, 2], [1, 3]]
    assert torch.isnan(o[0, 1]).all() and torch.isnan(o[1, 2:]).all()
    assert torch.isnan(o[2, :2, 0, 9]).all()
    o[2, :2, 0, 9] = 0
    assert torch.isfinite(o[2]).all() and torch.isfinite(o[1, :2]).all()


def test_decode_views_and_outputs(fa):  # noqa: F811
    """q as heads of a fused buffer, K and V as slices of one tensor, table rows
    cut from a wider one, caller's outputs and workspace, repeated calls equal."""
    B, H, H_kv, d, page = 5, 8, 2, 128, 16
    both = torch.randn(30, 2, H_kv, page, d, device=DEV).to(torch.bfloat16)
    kc, vc = both[:, 0], both[:, 1]
    fused = torch.randn(B, 1, H + 2 * H_kv, d, device=DEV).to(torch.bfloat16).transpose(1, 2)
    q = fused[:, :H]
    table = shuffled_table(30, 6, 5)[:, 1:4]
    lens = torch.tensor([48, 1, 20, 33, 0], dtype=torch.int32, device=DEV)
    ws = torch.full((fa.load_library().fa_paged_decode_workspace_bytes(B, H, H_kv, d),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    out = torch.empty(B, H, 1, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, H, 1, device=DEV)
    a = decode_and_check(fa, q, kc, vc, 1.0, 1.0, table, lens, workspace=ws, out=out, lse=lse)
    assert a[0] is out and a[1] is lse
    o2, l2 = fa.paged_decode_attention(q, kc, vc, table, lens, workspace=ws)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_decode_offsets_beyond_32_bits(fa):  # noqa: F811
    """Pages more than 2^32 bytes and 2^31 elements into the cache."""
    P, H_kv, page, d = 150000, 8, 16, 128
    kc = torch.empty(P, H_kv, page, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    assert kc.numel() > 1 << 31
    small_k, small_v, _, _ = pages_of(8, H_kv, page, d, 2, seed=11)
    where = torch.tensor([149999, 140000, 131072, 131071, 3, 149998, 70000, 0], device=DEV)
    q = queries(1, 16, d)
    lens = torch.tensor([121], dtype=torch.int32, device=DEV)
    # the pages get there by copies from the cache's start, as compaction makes them
    kc[100:108], vc[100:108] = small_k, small_v
    fa.copy_pages(kc, vc, torch.arange(100, 108, dtype=torch.int32, device=DEV),
                  where.to(torch.int32))
    assert torch.equal(kc[where], small_k) and torch.equal(vc[where], small_v)
    o, lse = fa.paged_decode_attention(q, kc, vc, where.to(torch.int32)[None], lens)
    o2, lse2 = decode_and_check(fa, q, small_k, small_v, 1.0, 1.0,
                                torch.arange(8, dtype=torch.int32, device=DEV)[None], lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    new = torch.randn(1, H_kv, 1, d, device=DEV).to(torch.bfloat16)
    pos = torch.tensor([[121]], dtype=torch.int32, device=DEV)
    fa.paged_append(new, new, kc, vc, where.roll(1).to(torch.int32)[None], pos)
    assert torch.equal(kc[70000, :, 9], new[0, :, 0])


# ---------------------------------------------------------------- append
def check_stored(got, ref, descale, elem, mag):
    """Stored values (codes, before descale) against fp64 values."""
    want = ref / descale
    extra = 32 * U * mag / descale
    if elem == 2:
        tol = 2.0 ** -8 * np.abs(want) + extra + TINY
    else:
        want = np.clip(want, -448, 448)
        tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + extra + 2.0 ** -22 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()


APPENDS = [  # B, H, H_kv, N, d, page, rot, norm, inter, elem, token_major
    (1, 1, 1, 1, 64, 16, 64, False, False, 2, False),
    (16, 32, 8, 1, 128, 16, 128, True, False, 2, False),
    (3, 6, 2, 37, 128, 24, 32, True, True, 1, True),
    (2, 4, 4, 100, 256, 8, 256, False, False, 1, False),
    (2, 0, 3, 19, 64, 1, 16, True, False, 2, True),
    (5, 8, 1, 3, 64, 64, 0, False, False, 1, False),
    (130, 2, 1, 1, 256, 16, 64, True, True, 2, False),
]


@pytest.mark.parametrize("B,H,H_kv,N,d,page,rot,norm,inter,elem,token_major", APPENDS)
def test_append(fa, B, H, H_kv, N, d, page, rot, norm, inter, elem, token_major):  # noqa: F811
    """New tokens at ragged starts; slots that no token goes to, and q_out rows
    of padding, stay as they were bit for bit."""
    g = torch.Generator().manual_seed(B + N)
    x = torch.randn(B, N, H + 2 * H_kv, d, generator=g).to(torch.bfloat16).to(DEV).transpose(1, 2)
    q, k, v = x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]
    rng = np.random.default_rng(B)
    start = rng.integers(0, 200, B)
    pos = (start[:, None] + np.arange(N)).astype(np.int32)
    if N > 2:
        pos[:, -1] = -1                                      # padding
        pos[0, 0] = -7
    width = -(-(200 + N) // page)
    P = B * width + 2
    table = shuffled_table(P, B, width, seed=N)
    kc, vc, ks, vs = pages_of(P, H_kv, page, d, elem, token_major, seed=1)
    k0, v0 = kc.clone(), vc.clone()
    eps = 1e-6 if norm else None
    wq, wk = weights(d, False) if norm else (None, None)
    freqs = fa.rotary_frequencies(rot) if rot else None
    f64 = np64(freqs) if rot else np.zeros(0)
    q_out = torch.full((B, H, N, d), 7.0, dtype=torch.bfloat16, device=DEV)
    got = fa.paged_append(k, v, kc, vc, table, torch.from_numpy(pos).to(DEV),
                          q=q if H else None, freqs=freqs, interleaved=inter, norm_eps=eps,
                          q_weight=wq, k_weight=wk, k_descale=ks, v_descale=vs,
                          q_out=q_out if H else None)
    torch.cuda.synchronize()
    live = pos >= 0
    if H:
        assert got is q_out
        w64 = None if wq is None else np64(wq)
        ref = orot.forward(np64(q), pos, f64, inter, 1.0, eps, w64)
        mag = partner_sum(orot.norm(np64(q), eps, w64), len(f64), inter)
        o = np64(q_out)
        tol = 2.0 ** -8 * np.abs(ref) + 32 * U * mag + TINY
        rows = np.broadcast_to(live[:, None], (B, H, N))
        assert np.all((np.abs(o - ref) <= tol)[rows])
        assert np.all(o[~rows] == 7.0)
    else:
        assert got is None
    wk64 = None if wk is None else np64(wk)
    rk = orot.forward(np64(k), pos, f64, inter, 1.0, eps, wk64)
    mk = partner_sum(orot.norm(np64(k), eps, wk64), len(f64), inter)
    b, n = np.nonzero(live)
    page_of = table.cpu().numpy()[b, pos[b, n] // page]
    slot = pos[b, n] % page
    at = (torch.from_numpy(page_of).long().to(DEV), slice(None), torch.from_numpy(slot).to(DEV))

    def raw(c):
        return c.view(torch.uint8) if elem == 1 else c

    check_stored(raw(kc)[at].view(kc.dtype).double().cpu().numpy(), rk[b, :, n], ks, elem,
                 mk[b, :, n])
    if elem == 2:
        assert torch.equal(vc[at], v[torch.from_numpy(b).to(DEV), :, torch.from_numpy(n).to(DEV)])
    else:
        check_stored(raw(vc)[at].view(vc.dtype).double().cpu().numpy(), np64(v)[b, :, n], vs, elem,
                     0 * mk[b, :, n])
    for c, c0 in ((kc, k0), (vc, v0)):                       # everything else untouched
        raw(c0)[at] = raw(c)[at]
        assert torch.equal(raw(c), raw(c0))


def test_append_special_values(fa):  # noqa: F811
    """e4m3 saturates (infinities too) and keeps NaN; bf16 keeps them all."""
    d = 64
    k = torch.zeros(1, 1, 1, d, dtype=torch.bfloat16, device=DEV)
    vals = [float("inf"), float("-inf"), float("nan"), 1000.0, -449.0, 448.0, 2.0 ** -9, 1e-4]
    k[0, 0, 0, :8] = torch.tensor(vals)
    pos = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    kc = torch.zeros(1, 1, 4, d, dtype=E4M3, device=DEV)
    vc = torch.zeros_like(kc)
    fa.paged_append(k, k, kc, vc, table, pos)
    for c in (kc, vc):
        got = c[0, 0, 0, :8].float().tolist()
        assert got[:2] == [448.0, -448.0] and math.isnan(got[2])
        assert got[3:7] == [448.0, -448.0, 448.0, 2.0 ** -9] and got[7] == 0.0
    kb = torch.zeros(1, 1, 4, d, dtype=torch.bfloat16, device=DEV)
    vb = torch.zeros_like(kb)
    fa.paged_append(k, k, kb, vb, table, pos)
    for c in (kb, vb):
        assert torch.equal(c[0, 0, 0].view(torch.int16), k[0, 0, 0].view(torch.int16))


def test_append_drops_what_has_no_page(fa):  # noqa: F811
    """Unknown sequences, positions past the table and bad pages write nothing
    to the cache; their queries come out all the same."""
    kc, vc, _, _ = pages_of(6, 2, 8, 64, 2, seed=2)
    k0, v0 = kc.clone(), vc.clone()
    x = torch.randn(6, 4, 1, 64, device=DEV).to(torch.bfloat16)
    table = torch.tensor([[0, 1], [-1, 6], [2, 1 << 29]], dtype=torch.int32, device=DEV)
    seq = torch.tensor([3, -1, 0, 1, 1, 2], dtype=torch.int32, device=DEV)
    pos = torch.tensor([[0], [0], [16], [3], [9], [8]], dtype=torch.int32, device=DEV)
    q = fa.paged_append(x[:, :2], x[:, 2:], kc, vc, table, pos, q=x, seq=seq)
    assert torch.equal(q, x) and torch.equal(kc, k0) and torch.equal(vc, v0)
    seq[0], pos[0] = 2, 5
    fa.paged_append(x[:, :2], x[:, 2:], kc, vc, table, pos, seq=seq)
    assert torch.equal(kc[2, :, 5], x[0, :2, 0]) and torch.equal(vc[2, :, 5], x[0, 2:, 0])
    far = torch.full((6, 1), (1 << 31) - 1, dtype=torch.int32, device=DEV)
    fa.paged_append(x[:, :2], x[:, 2:], kc, vc, table, far)


# ---------------------------------------------------------------- copies
@pytest.mark.parametrize("elem", [2, 1])
@pytest.mark.parametrize("H_kv,page,d", [(1, 1, 64), (3, 5, 64), (2, 16, 128), (8, 64, 256)])
@pytest.mark.parametrize("layout", ["heads", "tokens", "padded"])
def test_copy(fa, H_kv, page, d, elem, layout):  # noqa: F811
    P = 41
    kc, vc, _, _ = pages_of(P, H_kv, page, d, elem, layout == "tokens", seed=3)
    if layout == "padded":                                   # rows wider than a head
        wide = [torch.zeros(P, H_kv, page + 1, d + 16, device=DEV).to(kc.dtype) for _ in range(2)]
        for w, c in zip(wide, (kc, vc)):
            w[:, :, :page, :d] = c
        kc, vc = (w[:, :, :page, :d] for w in wide)
    g = torch.Generator().manual_seed(page)
    perm = torch.randperm(P, generator=g).to(torch.int32).to(DEV)
    src, dst = perm[:15].clone(), perm[20:35].clone()
    src[3] = src[2]                                          # one source, two copies
    src[7] = dst[7]                                          # onto itself
    src[9], dst[11] = -1, P                                  # skipped

    def raw(c):
        return c.view(torch.uint8) if elem == 1 else c

    want = [raw(c).clone() for c in (kc, vc)]
    for w, c in zip(want, (kc, vc)):
        for i, (s, t) in enumerate(zip(src.tolist(), dst.tolist())):
            if 0 <= s < P and 0 <= t < P:
                w[t] = raw(c)[s]
    fa.copy_pages(kc, vc, src, dst)
    for w, c in zip(want, (kc, vc)):
        assert torch.equal(raw(c), w)
    if layout == "padded":
        assert all((w[:, :, page:].float() == 0).all() and (w[..., d:].float() == 0).all()
                   for w in wide)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("elem", [2, 1])
def test_prompt_fork_decode_compact(fa, elem):  # noqa: F811
    """A serving run: two prompts appended as one padded batch; the second forked
    (full pages shared, the last one copied); three sequences decode two tokens
    each; the live pages are moved down and decoding gives the same bits. Each
    step's attention is checked on the cache as it stands, and, for bf16, the
    cache against the contiguous path."""
    H, H_kv, d, page, P = 8, 2, 128, 16, 64
    kc, vc, ks, vs = pages_of(P, H_kv, page, d, elem, seed=5)
    freqs = fa.rotary_frequencies(128, scaling="linear", factor=2.0)
    wq, wk = weights(d, False)
    kw = dict(freqs=freqs, norm_eps=1e-6, q_weight=wq, k_weight=wk, k_descale=ks, v_descale=vs)
    g = torch.Generator().manual_seed(9)
    lens = [45, 70]
    x = torch.randn(2, 70, H + 2 * H_kv, d, generator=g).to(torch.bfloat16).to(DEV).transpose(1, 2)
    pos = torch.arange(70, dtype=torch.int32).repeat(2, 1)
    pos[0, 45:] = -1
    table = torch.full((3, 8), -1, dtype=torch.int32)
    order = iter(np.random.default_rng(1).permutation(P).tolist())
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b, i] = next(order)
    table = table.to(DEV)
    fa.paged_append(x[:, H:H + H_kv], x[:, H + H_kv:], kc, vc, table, pos.to(DEV), q=x[:, :H], **kw)
    # fork sequence 1: four full pages shared, page 4 copied
    table[2] = table[1]
    table[2, 4] = next(order)
    fa.copy_pages(kc, vc, table[1, 4:5].clone(), table[2, 4:5].clone())
    kv_len = torch.tensor([45, 70, 70], dtype=torch.int32, device=DEV)
    fresh = []
    for step in range(2):
        y = torch.randn(3, 1, H + 2 * H_kv, d, generator=g).to(torch.bfloat16).to(DEV).transpose(1, 2)
        for b in range(3):
            if int(kv_len[b]) % page == 0:
                table[b, int(kv_len[b]) // page] = next(order)
        q = fa.paged_append(y[:, H:H + H_kv], y[:, H + H_kv:], kc, vc, table, kv_len[:, None],
                            q=y[:, :H], **kw)
        kv_len += 1
        o, lse = decode_and_check(fa, q, kc, vc, ks, vs, table, kv_len, f"step {step}")
        fresh.append(y)
    assert not torch.equal(o[1], o[2])                       # the fork went its own way
    # compaction: every live page to a free page below the live count
    live = torch.unique(table[table >= 0])
    n = len(live)
    low = torch.zeros(P, dtype=torch.bool, device=DEV)
    low[live.long()] = True
    src = live[live >= n]
    dst = (~low[:n]).nonzero().flatten().to(torch.int32)
    assert len(src) == len(dst) > 0
    fa.copy_pages(kc, vc, src, dst)
    new_id = torch.arange(P, dtype=torch.int32, device=DEV)
    new_id[src.long()] = dst
    moved = torch.where(table >= 0, new_id[table.clamp(min=0).long()], table)
    assert int(moved.max()) < n
    o2, lse2 = fa.paged_decode_attention(q, kc, vc, moved, kv_len, k_descale=ks, v_descale=vs)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if elem == 2:
        # the contiguous path over the same keys (sequence 0): qk_rotary + decode_attention
        ks_all = torch.cat([x[:1, H:H + H_kv, :45]] + [y[:1, H:H + H_kv] for y in fresh], 2)
        vs_all = torch.cat([x[:1, H + H_kv:, :45]] + [y[:1, H + H_kv:] for y in fresh], 2)
        _, kr = fa.qk_rotary(ks_all[:, :0], ks_all, torch.arange(47, dtype=torch.int32, device=DEV),
                             freqs, norm_eps=1e-6, q_weight=wq, k_weight=wk)
        oc, lc = fa.decode_attention(q[:1].contiguous(), kr.contiguous(), vs_all.contiguous())
        assert (oc.float() - o[:1].float()).abs().max() <= 2e-2
        assert (lc - lse[:1]).abs().max() <= 1e-3


def test_streams_and_graphs(fa):  # noqa: F811
    """Decoding on a named stream; two captured steps (append, then attention)
    replayed in turn, each with its own workspace, over a growing cache."""
    B, H, H_kv, d, page = 4, 8, 2, 128, 16
    kc, vc, _, _ = pages_of(200, H_kv, page, d, 2, seed=6)
    table = shuffled_table(200, B, 40)
    kv_len = torch.tensor([5, 300, 600, 1], dtype=torch.int32, device=DEV)
    q = queries(B, H, d)
    want = fa.paged_decode_attention(q, kc, vc, table, kv_len)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.paged_decode_attention(q, kc, vc, table, kv_len, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])

    new = torch.randn(B, H + 2 * H_kv, 1, d, device=DEV).to(torch.bfloat16)
    freqs = fa.rotary_frequencies(64)

    def step():
        qq = fa.paged_append(new[:, H:H + H_kv], new[:, H + H_kv:], kc, vc, table, kv_len[:, None],
                             q=new[:, :H], freqs=freqs)
        n = kv_len + 1
        return (*fa.paged_decode_attention(qq, kc, vc, table, n), n)

    step()
    torch.cuda.synchronize()
    graphs, kept = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            kept.append(step())
        graphs.append(gr)
    for i in range(4):
        new.copy_(torch.randn(B, H + 2 * H_kv, 1, d, device=DEV).to(torch.bfloat16))
        graphs[i % 2].replay()
        o, lse, n = kept[i % 2]
        decode_and = step()
        assert torch.equal(o, decode_and[0]) and torch.equal(lse, decode_and[1])
        kv_len.copy_(n)


def test_empty_calls(fa):  # noqa: F811
    """No sequences, no tokens, no heads, no pages to copy, no pages at all."""
    kc, vc, _, _ = pages_of(4, 2, 16, 64, 2, seed=1)
    k0, v0 = kc.clone(), vc.clone()
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    table = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    o, lse = fa.paged_decode_attention(queries(0, 4, 64), kc, vc, table[:0], none)
    assert o.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)
    x = torch.zeros(1, 2, 0, 64, dtype=torch.bfloat16, device=DEV)
    fa.paged_append(x, x, kc, vc, table, none[None])
    fa.copy_pages(kc, vc, none, none)
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    o, lse = fa.paged_decode_attention(queries(1, 4, 64), kc[:0], vc[:0], table,
                                       torch.tensor([9], dtype=torch.int32, device=DEV))
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = fa.paged_decode_attention(queries(1, 4, 64), kc, vc, table[:, :0],
                                       torch.tensor([9], dtype=torch.int32, device=DEV))
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_decode_shared_table_rows(fa):  # noqa: F811
    """One table row for all sequences (stride 0), pages listed twice."""
    kc, vc, _, _ = pages_of(6, 2, 16, 128, 2, seed=2)
    row = torch.tensor([3, 1, 3, 5], dtype=torch.int32, device=DEV)
    lens = torch.tensor([64, 10, 33], dtype=torch.int32, device=DEV)
    decode_and_check(fa, queries(3, 4, 128), kc, vc, 1.0, 1.0, row.expand(3, 4), lens)


def test_append_in_place_queries(fa):  # noqa: F811
    """q_out is q: the same bits as into a new tensor; keys alone without q."""
    x = torch.randn(3, 12, 5, 128, device=DEV).to(torch.bfloat16)
    kc, vc, _, _ = pages_of(20, 2, 16, 128, 2, seed=3)
    k2, v2 = kc.clone(), vc.clone()
    table = shuffled_table(20, 3, 4)
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    kw = dict(freqs=fa.rotary_frequencies(128), norm_eps=1e-6)
    q = x[:, :8].clone()
    want = fa.paged_append(x[:, 8:10], x[:, 10:], kc, vc, table, pos, q=q, **kw)
    got = fa.paged_append(x[:, 8:10], x[:, 10:], k2, v2, table, pos, q=q, q_out=q, **kw)
    assert got is q and torch.equal(q, want) and torch.equal(kc, k2) and torch.equal(vc, v2)
    k2.zero_()
    assert fa.paged_append(x[:, 8:10], x[:, 10:], k2, v2, table, pos, **kw) is None
    used = table[:, :1].long()
    assert torch.equal(k2[used, :, :5], kc[used, :, :5])


def test_decode_two_streams_at_once(fa):  # noqa: F811
    """Calls in flight together on two streams, each with its own workspace."""
    kc, vc, _, _ = pages_of(1200, 2, 16, 128, 2, seed=4)
    table = shuffled_table(1200, 4, 300)
    lens = [torch.tensor(x, dtype=torch.int32, device=DEV)
            for x in ([4800, 100, 4000, 1], [7, 4700, 0, 2500])]
    qs = [queries(4, 16, 128, seed=s) for s in (1, 2)]
    want = [fa.paged_decode_attention(q, kc, vc, table, n) for q, n in zip(qs, lens)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fa.paged_decode_attention(qs[i], kc, vc, table, lens[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


N_CASES = 40


@pytest.mark.parametrize("case", range(N_CASES))
def test_random_decoding(fa, case):  # noqa: F811
    """Seeded random shapes: heads, head dim, page size and order, type, lengths."""
    rng = np.random.default_rng(1009 + 7919 * case)
    d = int(rng.choice([64, 128, 256]))
    H_kv = int(rng.integers(1, 5))
    H = H_kv * int(rng.choice([1, 2, 3, 4, 7, 8, 12, 16, 18]))
    page = int(rng.choice([1, 2, 5, 8, 16, 16, 32, 48, 64, 100, 256]))
    elem = int(rng.choice([1, 2]))
    B = int(rng.choice([1, 2, 3, 7, 33]))
    most = int(rng.choice([1, 30, 300, 2000])) if B < 33 else 90
    lens = rng.integers(0, most + 1, B).astype(np.int32)
    width = -(-most // page)
    P = B * width + 1
    kc, vc, ks, vs = pages_of(P, H_kv, page, d, elem, bool(rng.integers(2)), seed=case,
                              mult=float(rng.choice([0.25, 1.0, 3.0])))
    decode_and_check(fa, queries(B, H, d, seed=case, mult=float(rng.choice([0.5, 1.0, 4.0]))),
                     kc, vc, ks, vs, shuffled_table(P, B, width, seed=case),
                     torch.from_numpy(lens).to(DEV),
                     f"case {case}: B{B} H{H} H_kv{H_kv} d{d} page{page} elem{elem} {lens.tolist()}")


def test_calls_in_a_row_wait_for_one_another(fa):  # noqa: F811
    """The kernels start before their predecessors end and wait inside: a chain
    in which each call reads what the one before wrote (torch kernels among
    them), run without and with a synchronisation after every call."""
    B, H, H_kv, d, page = 3, 8, 2, 128, 16
    freqs = fa.rotary_frequencies(128)
    table = shuffled_table(120, B, 20)
    spare = torch.tensor([x for x in range(120) if x not in set(table.flatten().tolist())][:B],
                         dtype=torch.int32, device=DEV)
    start = torch.randn(B, H + 2 * H_kv, 1, d, device=DEV).to(torch.bfloat16)

    def chain(wait):
        def step(value):
            if wait:
                torch.cuda.synchronize()
            return value

        kc = torch.zeros(120, H_kv, page, d, dtype=torch.bfloat16, device=DEV)
        vc = torch.zeros_like(kc)
        t = table.clone()
        n = torch.zeros(B, dtype=torch.int32, device=DEV)
        x = start.clone()
        outs = []
        for i in range(60):
            q = step(fa.paged_append(x[:, H:H + H_kv], x[:, H + H_kv:], kc, vc, t, n[:, None],
                                     q=x[:, :H], freqs=freqs, norm_eps=1e-6))
            n = step(n + 1)
            o, lse = step(fa.paged_decode_attention(q, kc, vc, t, n))
            if i == 30:                                      # the last pages move away
                old = t[:, 1].contiguous()
                step(fa.copy_pages(kc, vc, old, spare))
                t[:, 1] = step(spare)
            qr, kr = step(fa.qk_rotary(o, o[:, :H_kv], n[:, None], freqs))
            dq, dk, dw, _ = step(fa.qk_rotary_bwd(qr, kr, o, o[:, :H_kv], n[:, None], freqs,
                                                  norm_eps=1e-6))
            x = step(torch.cat([dq, dk, kr], 1))             # the next token
            outs.append((o, lse, dw))
        torch.cuda.synchronize()
        return outs, kc, vc

    a, b = chain(True), chain(False)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    for u, v in zip(a[0], b[0]):
        for p, r in zip(u, v):
            assert torch.equal(p, r)


# ---------------------------------------------------------------- e4m3 pages: bits of q and P
def e4m3_tail(n, d):
    """n keys and values: value 0 is zero, the others' are positive; the others'
    keys are 0 to 4 in element 0."""
    k = torch.zeros(n, d)
    k[1:, 0] = (torch.arange(n - 1) % 9) * 0.5
    v = torch.zeros(n, d)
    v[1:] = 1 + 0.125 * ((torch.arange(n - 1)[:, None] + torch.arange(d)) % 8)
    return k, v


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 3, 12])
@pytest.mark.parametrize("top", [20.0, 26.0, 28.0])
@pytest.mark.parametrize("B,n", [(1, 40), (60, 5000)])
def test_decode_e4m3_small_probabilities(fa, B, n, top, heads, d):  # noqa: F811
    """One key outweighs each of the others by 2^16 to 2^28, and O is the others'
    alone; one step a warp, and several. Codes, values and, but for the scale's
    rounding (2^-24 of 28), scores (scale ln 2: log2 units) are exact. A weight is
    off by 2^-19 (that and the exponential) and 2^-11 (f16) relative, and by 2^-32
    of the largest (half an f16 step, 2^-24, at p taken 2^7 larger): O by that
    times |v - O|. The sums add 2^-17 as in decode_and_check, O's rounding 2^-8."""
    page = 16
    k, v = e4m3_tail(n, d)
    k[0, 0] = top
    width = -(-n // page)
    kc, vc = (torch.zeros(width * page, d) for _ in range(2))
    kc[:n], vc[:n] = k, v
    kc, vc = (c.view(width, 1, page, d).to(E4M3).to(DEV) for c in (kc, vc))
    q = torch.zeros(B, heads, 1, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1
    table = torch.arange(width, dtype=torch.int32, device=DEV).expand(B, width)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    o, lse = fa.paged_decode_attention(q, kc, vc, table, lens, scale=math.log(2.0))
    k, v = np64(k), np64(v)
    w = np.exp2(k[:, 0] - top)
    want = w @ v / w.sum()
    away = np.abs(v - want)
    tol = (2.0 ** -19 + 2.0 ** -11) * (w @ away) / w.sum() + 2.0 ** -32 * away.sum(0) / w.sum() \
        + (2.0 ** -17 + 2.0 ** -8) * want
    err = np.abs(np64(o)[:, :, 0] - want)
    assert np.all(err <= tol), f"{(err / want).max()} of O"
    want = math.log(w.sum()) + top * math.log(2.0)
    assert np.all(np.abs(np64(lse) - want) <= 2.0 ** -16 + U * want)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("below", [18, 21, 24, 30])
def test_decode_e4m3_query_spread(fa, below, d):  # noqa: F811
    """The scores come from elements 2^-below of the query's largest one, which
    meets zeros: bf16 elements down to 2^-31 of the largest count in full."""
    heads, n, page = 5, 200, 16
    kc, vc, ks, vs = pages_of(-(-n // page), 1, page, d, 1, seed=below, ks=0.02)
    kc = kc.float()
    kc[..., 0] = 0
    kc = kc.to(E4M3)
    q = queries(1, heads, d, seed=below).float().clamp(-2, 2)
    q = (q.abs().clamp(min=0.5) * q.sign() * 2.0 ** -below)
    q[..., 0] = 1.5
    table = torch.arange(kc.shape[0], dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    decode_and_check(fa, q.to(torch.bfloat16), kc, vc, ks, vs, table, lens,
                     scale=2.0 ** below / math.sqrt(d))


@pytest.mark.parametrize("mult", [2.0 ** -122, 2.0 ** -90, 2.0 ** 100, 2.0 ** 118])
def test_decode_e4m3_query_extremes(fa, mult):  # noqa: F811
    """Magnitudes near both ends of bf16: the power of two follows them there."""
    kc, vc, ks, vs = pages_of(8, 1, 16, 128, 1, seed=9)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([120], dtype=torch.int32, device=DEV)
    decode_and_check(fa, queries(1, 5, 128, mult=mult), kc, vc, ks, vs, table, lens,
                     scale=0.1 / mult)


def test_decode_e4m3_infinite_query_element(fa):  # noqa: F811
    """An infinite element beside large finite ones: only what meets it is not a
    number; a head beside it is as without it."""
    kc, vc, ks, vs = pages_of(8, 1, 16, 64, 1, seed=9)
    q = queries(1, 3, 64)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([120], dtype=torch.int32, device=DEV)
    want = fa.paged_decode_attention(q, kc, vc, table, lens, k_descale=ks, v_descale=vs)
    q[0, 1, 0, 5] = float("inf")
    o, lse = fa.paged_decode_attention(q, kc, vc, table, lens, k_descale=ks, v_descale=vs)
    for h in (0, 2):
        assert torch.equal(o[:, h], want[0][:, h]) and torch.equal(lse[:, h], want[1][:, h])
    assert torch.isnan(lse[0, 1]).all() and torch.isnan(o[0, 1]).all()


@pytest.mark.parametrize("elem", [2, 1])
@pytest.mark.parametrize("d,H,H_kv", [(64, 12, 12), (128, 32, 8), (128, 16, 1), (256, 40, 2)])
def test_decode_repeats_itself(fa, d, H, H_kv, elem):  # noqa: F811
    """The same bits every time: into other outputs, over other workspace
    contents, after other calls."""
    page, lens = 16, [777, 1, 0, 2000, 64, 350]
    B, width = len(lens), -(-2000 // page)
    kc, vc, ks, vs = pages_of(B * width, H_kv, page, d, elem, seed=d + H)
    table = shuffled_table(B * width, B, width)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q, other = queries(B, H, d, seed=1), queries(B, H, d, seed=2)
    need = fa.load_library().fa_paged_decode_workspace_bytes(B, H, H_kv, d)
    kw = dict(k_descale=ks, v_descale=vs)
    o, lse = fa.paged_decode_attention(q, kc, vc, table, n, **kw)
    for fill in (0, 0xFF, 0x3C):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        for _ in range(3):
            fa.paged_decode_attention(other, kc, vc, table, n.flip(0), workspace=ws, **kw)
            o2, lse2 = fa.paged_decode_attention(q, kc, vc, table, n, workspace=ws, **kw)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_captured_forks_joins_and_copies(fa):  # noqa: F811
    """One captured step whose calls follow two branches at once, a copy and a fill:
    replayed on changing inputs it gives the eager step's bits. A second graph
    holds the same step over the same workspace."""
    B, H, H_kv, d, page = 3, 8, 2, 128, 16
    kc, vc, _, _ = pages_of(100, H_kv, page, d, 2, seed=7)
    table = shuffled_table(100, B, 30)
    freqs = fa.rotary_frequencies(128)
    x = torch.randn(B, H + 2 * H_kv, 1, d, device=DEV).to(torch.bfloat16)
    n = torch.tensor([470, 3, 100], dtype=torch.int32, device=DEV)
    held, left = torch.zeros_like(n), torch.zeros_like(n)
    need = fa.load_library().fa_paged_decode_workspace_bytes(B, H, H_kv, d)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        left.fill_(0)
        held.copy_(n)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            fa.paged_append(x[:, H:H + H_kv], x[:, H + H_kv:], kc, vc, table, held[:, None],
                            freqs=freqs, norm_eps=1e-6)
        q, k = fa.qk_rotary(x[:, :H], x[:, H:H + H_kv], held[:, None], freqs, norm_eps=1e-6)
        main.wait_stream(side)                               # both are read next
        left.add_(held).add_(1)
        o, lse = fa.paged_decode_attention(q, kc, vc, table, left, workspace=ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            dq, dk, dw, _ = fa.qk_rotary_bwd(o, k, x[:, :H], x[:, H:H + H_kv], held[:, None], freqs,
                                             norm_eps=1e-6)
        o2, lse2 = fa.paged_decode_attention(q, kc, vc, table, held, workspace=ws)
        main.wait_stream(side)
        return o, lse, dq, dk, dw, o2, lse2

    step()
    torch.cuda.synchronize()
    graphs, kept = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(step())
        graphs.append(g)
    for i in range(6):
        x.copy_(torch.randn(B, H + 2 * H_kv, 1, d, device=DEV).to(torch.bfloat16))
        graphs[i % 2].replay()
        got = [t.clone() for t in kept[i % 2]]
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        n.add_(1)
