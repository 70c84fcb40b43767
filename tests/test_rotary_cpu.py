"""CPU checks of the rotary entry points: the headers are C, the binding packs
their structs as C lays them out, bad arguments are refused before any CUDA
call, and the fp64 oracle's gradients agree with differences."""
import os
import struct
import subprocess

import numpy as np
import pytest
import torch

import io_aware_exact_18_b200 as fa
from io_aware_exact_18_b200 import build as fa_build
from io_aware_exact_18_b200 import rotary
from oracle import rotary as orot

INCLUDE = os.path.dirname(fa.HEADER_PATH)


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def c_sizes(tmp_path, header, names):
    """sizeof of each struct, compiled as plain C11."""
    src = tmp_path / "sizes.c"
    body = "".join(f'printf("%zu\\n", sizeof({n}));' for n in names)
    src.write_text(f'#include <stdio.h>\n#include "{header}"\nint main(void) {{ {body} return 0; }}\n')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-I", INCLUDE, str(src),
                    "-o", str(exe)], check=True)
    return [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                           text=True).stdout.split()]


def test_structs_match_the_header(tmp_path):
    got = c_sizes(tmp_path, "fa_rotary.h",
                  ["fa_heads_t", "fa_rotary_t", "fa_qk_rotary_t", "fa_qk_rotary_bwd_t"])
    assert got == [struct.calcsize("@" + rotary.HEADS), struct.calcsize("@" + rotary.ROTARY),
                   rotary._QK.size, rotary._QK_BWD.size]


def test_library_exports_the_header(lib):
    names = fa.declared_symbols(os.path.join(INCLUDE, "fa_rotary.h"))
    assert names == ["fa_qk_rotary", "fa_qk_rotary_bwd", "fa_qk_rotary_bwd_workspace_bytes"]
    for n in names:
        assert hasattr(lib, n)


# Fake, never-dereferenced addresses: every check runs before any CUDA call.
P = 1 << 40
G = 1 << 32
GOOD = dict(q=P, k=P + G, qo=P + 2 * G, ko=P + 3 * G, pos=P + 4 * G, psb=100, psn=1,
            freqs=P + 5 * G, wq=P + 6 * G, wk=P + 7 * G, rot=64, inter=0, norm=1, w32=0, scale=1.0,
            eps=1e-6, B=2, H=8, H_kv=2, N=100, d=128, qs=None, ks=None, qos=None, kos=None)


def strides(a, heads):
    return (heads * a["N"] * a["d"], a["N"] * a["d"], a["d"])


def pack_fwd(a):
    qs, ks = strides(a, a["H"]), strides(a, a["H_kv"])
    return rotary._QK.pack(a["q"], *(a["qs"] or qs), a["k"], *(a["ks"] or ks),
                           a["qo"], *(a["qos"] or qs), a["ko"], *(a["kos"] or ks),
                           a["pos"], a["psb"], a["psn"], a["freqs"], a["wq"], a["wk"], a["rot"],
                           a["inter"], a["norm"], a["w32"], a["scale"], a["eps"], a["B"], a["H"],
                           a["H_kv"], a["N"], a["d"], 0)


BAD = [
    (dict(d=96, rot=32), fa.FA_ERR_UNSUPPORTED),
    (dict(rot=24), fa.FA_ERR_INVALID_ARG),
    (dict(rot=144), fa.FA_ERR_INVALID_ARG),
    (dict(rot=-16), fa.FA_ERR_INVALID_ARG),
    (dict(inter=2), fa.FA_ERR_INVALID_ARG),
    (dict(norm=-1), fa.FA_ERR_INVALID_ARG),
    (dict(w32=3), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(eps=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(eps=float("inf")), fa.FA_ERR_INVALID_ARG),
    (dict(freqs=0), fa.FA_ERR_INVALID_ARG),
    (dict(freqs=P + 5 * G + 4), fa.FA_ERR_INVALID_ARG),
    (dict(wq=P + 1), fa.FA_ERR_INVALID_ARG),
    (dict(w32=1, wk=P + 7 * G + 2), fa.FA_ERR_INVALID_ARG),
    (dict(pos=0), fa.FA_ERR_INVALID_ARG),
    (dict(pos=P + 4 * G + 2), fa.FA_ERR_INVALID_ARG),
    (dict(psb=-1), fa.FA_ERR_INVALID_ARG),
    (dict(B=-1), fa.FA_ERR_INVALID_ARG),
    (dict(H=-1), fa.FA_ERR_INVALID_ARG),
    (dict(N=-1), fa.FA_ERR_INVALID_ARG),
    (dict(B=1 << 20, N=1 << 20), fa.FA_ERR_INVALID_ARG),       # too many tokens
    (dict(H=70000), fa.FA_ERR_INVALID_ARG),
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(q=P + 8), fa.FA_ERR_INVALID_ARG),
    (dict(ko=P + 3 * G + 4), fa.FA_ERR_INVALID_ARG),
    (dict(qs=(102400, 12804, 128)), fa.FA_ERR_INVALID_ARG),    # stride not a multiple of 8
    (dict(qs=(-102400, 12800, 128)), fa.FA_ERR_INVALID_ARG),
    (dict(qos=(102400, 0, 128)), fa.FA_ERR_INVALID_ARG),       # heads written over one another
    (dict(qos=(102400, 12800, 64)), fa.FA_ERR_INVALID_ARG),    # rows run into one another
    (dict(qo=P + 128), fa.FA_ERR_INVALID_ARG),                 # shifted over its input
    (dict(qo=P + G), fa.FA_ERR_INVALID_ARG),                   # over k
    (dict(ko=P + 2 * G), fa.FA_ERR_INVALID_ARG),               # over the other output
    (dict(pos=P + 2 * G + 4), fa.FA_ERR_INVALID_ARG),          # read from under an output
    (dict(freqs=P + 3 * G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(wk=P + 2 * G), fa.FA_ERR_INVALID_ARG),
    (dict(B=0), fa.FA_OK),
    (dict(N=0, q=0, k=0, qo=0, ko=0), fa.FA_OK),
    (dict(H=0, H_kv=0), fa.FA_OK),
]


@pytest.mark.parametrize("over,status", BAD)
def test_forward_refusals(lib, over, status):
    assert lib.fa_qk_rotary(pack_fwd(dict(GOOD, **over)), None) == status


def accepted(lib, **over):
    """Past the argument checks: the call then fails for want of a GPU here."""
    st = lib.fa_qk_rotary(pack_fwd(dict(GOOD, **over)), None)
    return st != fa.FA_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on fake pointers")
def test_accepted_overlaps(lib):
    """In place, and in place on the q and k views of one fused buffer."""
    assert accepted(lib)
    assert accepted(lib, qo=P, ko=P + G)
    heads, d, N = 8 + 2 + 2, 128, 100
    fused = (N * heads * d, d, heads * d)
    v = dict(q=P, k=P + 2 * 8 * d, qs=fused, ks=fused, qos=fused, kos=fused)
    assert accepted(lib, **v)
    assert accepted(lib, qo=P, ko=P + 2 * 8 * d, **v)
    # k's output on v's place is apart from q and k; one head earlier it is not
    assert accepted(lib, qo=P, ko=P + 2 * 10 * d, **v)
    assert not accepted(lib, qo=P, ko=P + 2 * 9 * d, **v)
    assert accepted(lib, qs=(0, 0, 0), ks=(0, 0, 0))           # inputs may repeat


@pytest.mark.skipif(torch.cuda.is_available(), reason="the good call would launch on fake pointers")
def test_null_args(lib):
    assert lib.fa_qk_rotary(None, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_qk_rotary_bwd(None, None, 0, None) == fa.FA_ERR_INVALID_ARG


BWD = dict(GOOD, gq=P + 8 * G, gk=P + 9 * G, dwq=P + 10 * G, dwk=P + 11 * G, ws=P + 12 * G,
           ws_bytes=1 << 24)


@pytest.mark.parametrize("over,status", [
    (dict(dwq=0), fa.FA_ERR_INVALID_ARG),
    (dict(dwk=P + 11 * G + 2), fa.FA_ERR_INVALID_ARG),
    (dict(dwk=P + 10 * G + 256), fa.FA_ERR_INVALID_ARG),       # inside the other
    (dict(norm=0), fa.FA_ERR_INVALID_ARG),                     # weight gradients without a norm
    (dict(ws=0), fa.FA_ERR_INVALID_ARG),
    (dict(ws_bytes=100), fa.FA_ERR_INVALID_ARG),
    (dict(ws=P + 12 * G + 8), fa.FA_ERR_INVALID_ARG),
    (dict(ws=P), fa.FA_ERR_INVALID_ARG),                       # over q
    (dict(ws=P + 10 * G), fa.FA_ERR_INVALID_ARG),              # over dq_weight
    (dict(dwq=P + 2 * G), fa.FA_ERR_INVALID_ARG),              # over dq
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(qo=P), fa.FA_ERR_INVALID_ARG),                       # dq over q
    (dict(gq=0), fa.FA_ERR_INVALID_ARG),
    (dict(rot=40), fa.FA_ERR_INVALID_ARG),
    (dict(d=32, rot=16), fa.FA_ERR_UNSUPPORTED),
    (dict(norm=0, dwq=0, dwk=0, B=0), fa.FA_OK),
])
def test_backward_refusals(lib, over, status):
    a = dict(BWD, **over)
    qs, ks = strides(a, a["H"]), strides(a, a["H_kv"])
    args = rotary._QK_BWD.pack(a["gq"], *qs, a["gk"], *ks, a["q"], *qs, a["k"], *ks, a["qo"], *qs,
                               a["ko"], *ks, a["pos"], a["psb"], a["psn"], a["freqs"], a["wq"],
                               a["wk"], a["rot"], a["inter"], a["norm"], a["w32"], a["scale"],
                               a["eps"], a["dwq"], a["dwk"], a["B"], a["H"], a["H_kv"], a["N"],
                               a["d"], 0)
    assert lib.fa_qk_rotary_bwd(args, a["ws"], a["ws_bytes"], None) == status


def test_backward_workspace_bytes(lib):
    f = lib.fa_qk_rotary_bwd_workspace_bytes
    assert f(2, 8, 2, 100, 128, 0) == 0
    assert f(2, 8, 2, 0, 128, 1) == 0
    assert f(2, 8, 2, 100, 96, 1) == 0
    assert f(-1, 8, 2, 100, 128, 1) == 0
    one = f(1, 1, 0, 1, 128, 1)
    assert one >= 128 * 4 and one % 16 == 0
    assert f(8, 64, 64, 16384, 128, 1) % one == 0 and f(8, 64, 64, 16384, 128, 1) < 1 << 21


def test_wrappers_refuse():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.qk_rotary(x, x, pos, None)
    with pytest.raises(TypeError):
        fa.qk_rotary(x.float(), x.float(), pos, None)
    with pytest.raises(ValueError):
        fa.rotary_frequencies(20, device="cpu")
    with pytest.raises(ValueError):
        fa.rotary_frequencies(32, scaling="ramp", factor=4.0, device="cpu")
    with pytest.raises(ValueError):
        fa.rotary_frequencies(32, scaling="other", device="cpu")


def test_frequencies():
    f = fa.rotary_frequencies(64, base=10000.0, device="cpu").numpy()
    i = np.arange(32)
    np.testing.assert_allclose(f, 10000.0 ** (-2.0 * i / 64), rtol=1e-14)
    np.testing.assert_allclose(
        fa.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu").numpy(), f / 4)
    ntk = fa.rotary_frequencies(64, scaling="ntk", factor=8.0, device="cpu").numpy()
    assert ntk[0] == 1.0
    np.testing.assert_allclose(ntk[-1], f[-1] / 8, rtol=1e-12)
    ramp = fa.rotary_frequencies(64, scaling="ramp", factor=8.0, original_length=4096, low=1.0,
                                 high=32.0, device="cpu").numpy()
    turns = 4096 * f / (2 * np.pi)
    assert np.array_equal(ramp[turns >= 32], f[turns >= 32])
    np.testing.assert_allclose(ramp[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((ramp[mid] < f[mid]) & (ramp[mid] > f[mid] / 8))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("eps", [None, 1e-5])
def test_oracle_gradient_by_differences(interleaved, eps):
    """Central differences of the fp64 forward, step 1e-6: truncation about
    1e-12 and cancellation about 1e-10 against gradients of order one."""
    rng = np.random.default_rng(5)
    x, dy = rng.standard_normal((2, 2, 3, 64)), rng.standard_normal((2, 2, 3, 64))
    w = None if eps is None else 1 + 0.2 * rng.standard_normal(64)
    pos = rng.integers(-50, 5000, (2, 3))
    freqs = 10000.0 ** (-np.arange(16) / 16)

    def loss(x, w):
        return (dy * orot.forward(x, pos, freqs, interleaved, 1.25, eps, w)).sum()

    dx, dw = orot.backward(dy, x, pos, freqs, interleaved, 1.25, eps, w)
    for _ in range(40):
        at = tuple(int(rng.integers(n)) for n in x.shape)
        step = np.zeros_like(x)
        step[at] = 1e-6
        num = (loss(x + step, w) - loss(x - step, w)) / 2e-6
        assert abs(num - dx[at]) < 1e-7, (at, num, dx[at])
    if eps is not None:
        for j in (0, 17, 63):
            step = np.zeros(64)
            step[j] = 1e-6
            num = (loss(x, w + step) - loss(x, w - step)) / 2e-6
            assert abs(num - dw[j]) < 1e-6, (j, num, dw[j])


@pytest.mark.parametrize("over", [dict(pos=0), dict(pos=P + 4 * G + 2), dict(psb=-1), dict(psn=-1),
                                  dict(pos=P + 2 * G + 4)])
@pytest.mark.parametrize("norm", [0, 1])
def test_positions_are_checked_whatever_is_turned(lib, over, norm):
    """The kernels read positions with rotary_dim 0 too: NULL, misaligned ones,
    and ones under an output are refused there as anywhere, forward and backward."""
    a = dict(GOOD, rot=0, freqs=0, norm=norm, **over)
    assert lib.fa_qk_rotary(pack_fwd(a), None) == fa.FA_ERR_INVALID_ARG
    none = {} if norm else dict(dwq=0, dwk=0)
    assert backward(lib, rot=0, freqs=0, norm=norm, **none, **over) == fa.FA_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on fake pointers")
def test_norm_alone_is_accepted(lib):
    assert accepted(lib, rot=0, freqs=0)
    assert backward(lib, rot=0, freqs=0) != fa.FA_ERR_INVALID_ARG
    assert backward(lib, rot=0, freqs=0, norm=0, dwq=0, dwk=0) != fa.FA_ERR_INVALID_ARG


def backward(lib, **over):
    a = dict(BWD, **over)
    qs, ks = strides(a, a["H"]), strides(a, a["H_kv"])
    args = rotary._QK_BWD.pack(a["gq"], *qs, a["gk"], *ks, a["q"], *qs, a["k"], *ks, a["qo"], *qs,
                               a["ko"], *ks, a["pos"], a["psb"], a["psn"], a["freqs"], a["wq"],
                               a["wk"], a["rot"], a["inter"], a["norm"], a["w32"], a["scale"],
                               a["eps"], a["dwq"], a["dwk"], a["B"], a["H"], a["H_kv"], a["N"],
                               a["d"], 0)
    return lib.fa_qk_rotary_bwd(args, a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("what", ["ws", "dwq", "dwk"])
@pytest.mark.parametrize("under", ["pos", "freqs", "wq", "wk"])
@pytest.mark.parametrize("rot", [64, 0])
def test_backward_refuses_to_write_over_what_it_reads(lib, what, under, rot):
    """The workspace and the weight gradients, over the start and the last element
    of positions, frequencies and norm weights (bf16 and fp32)."""
    last = dict(pos=4 * 199, freqs=8 * 31, wq=2 * 127, wk=2 * 127)[under]
    for w32 in (0, 1):
        for off in (0, last * (2 if w32 and under[0] == "w" else 1)):
            over = {what: (BWD[under] + off) & ~15, "rot": rot, "w32": w32}
            if rot == 0 and under == "freqs":
                continue                                     # not read
            assert backward(lib, **over) == fa.FA_ERR_INVALID_ARG, (what, under, off)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on fake pointers")
def test_backward_accepts_neighbours(lib):
    """Right behind what is read, and over frequencies that rotary_dim 0 leaves unread."""
    for what in ("ws", "dwq", "dwk"):
        for under, size in (("pos", 4 * 200), ("freqs", 8 * 32), ("wq", 2 * 128), ("wk", 2 * 128)):
            assert backward(lib, **{what: BWD[under] + size}) != fa.FA_ERR_INVALID_ARG, (what, under)
        assert backward(lib, **{what: BWD["freqs"], "rot": 0}) != fa.FA_ERR_INVALID_ARG
