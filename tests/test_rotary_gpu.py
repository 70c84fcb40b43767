"""GPU parity of qk_rotary and qk_rotary_bwd against the fp64 oracle
(oracle/rotary.py).

Tolerances. The result is rounded once to bf16: half a step, 2^-8 of the value
(plus half the smallest bf16 subnormal). Before that the arithmetic is fp32:
the angle (2^-25 turns, 3.2 units of 2^-24 rad), sincospi (2 units), the
products with s and w (3), the two-term sum (2), r = rsqrt of a mean of d <= 256
squares (8 + 5 additions halved by the square root, rsqrt 2) and its product (1)
stay below 32 units of 2^-24 of the pair's magnitude |a| + |b|. Backward: the two row sums and
the same factors stay below 64 units of r (|g| |w| + |n| mean |g w n|). A weight's
gradient is an fp32 sum whose chains (a thread's heads and items, 32 slots, then
fp64 over blocks) are below 256 terms here: 256 units of 2^-24 of the sum of
magnitudes."""
import numpy as np
import pytest
import torch

from oracle import rotary as orot

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -134
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import io_aware_exact_18_b200 as fa
    from io_aware_exact_18_b200 import build
    build.build()
    fa.load_library()
    return fa


def np64(t):
    return t.detach().double().cpu().numpy()


def partner_sum(y, half, interleaved):
    """|a| + |b| of the pair an element belongs to (|y| where it is not turned)."""
    y = np.abs(y)
    out = y.copy()
    if half:
        if interleaved:
            a, b = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
        else:
            a, b = slice(0, half), slice(half, 2 * half)
        out[..., a] = out[..., b] = y[..., a] + y[..., b]
    return out


def check_forward(got, x, pos, freqs, inter, scale, eps, w, what):
    ref = orot.forward(x, pos, freqs, inter, scale, eps, w)
    mag = partner_sum(orot.norm(x, eps, w), len(freqs), inter) * max(abs(scale), 1.0)
    tol = 2.0 ** -8 * np.abs(ref) + 32 * U * mag + TINY
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - ref).max()}"


def make(B, H, H_kv, N, d, seed, fused=False, mult=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, N, H + 2 * H_kv, d, generator=g) * mult).to(torch.bfloat16).to(DEV)
    x = x.transpose(1, 2)
    if not fused:
        return x[:, :H].contiguous(), x[:, H:H + H_kv].contiguous()
    return x[:, :H], x[:, H:H + H_kv]


def weights(d, w32, seed=3):
    g = torch.Generator().manual_seed(seed)
    t = torch.float32 if w32 else torch.bfloat16
    return [(1 + 0.3 * torch.randn(d, generator=g)).to(t).to(DEV) for _ in range(2)]


SHAPES = [  # B, H, H_kv, N, d, rot
    (1, 1, 1, 1, 64, 64),
    (2, 3, 1, 5, 64, 32),
    (1, 12, 12, 33, 64, 64),
    (3, 8, 2, 17, 128, 128),
    (1, 5, 5, 100, 128, 48),
    (2, 6, 2, 9, 256, 64),
    (1, 2, 1, 40, 256, 256),
    (1, 40, 8, 1, 128, 16),
    (65, 4, 1, 1, 128, 128),
    (1, 0, 3, 7, 128, 64),       # keys only
    (1, 3, 0, 7, 64, 64),        # queries only
]


@pytest.mark.parametrize("B,H,H_kv,N,d,rot", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [None, "bf16", "f32", "ones"])
def test_forward(fa, B, H, H_kv, N, d, rot, inter, norm):
    q, k = make(B, H, H_kv, N, d, seed=B * 1000 + N, fused=N % 2 == 1)
    rng = np.random.default_rng(N)
    pos = torch.from_numpy(rng.integers(-300, 200000, (B, N)).astype(np.int32)).to(DEV)
    freqs = fa.rotary_frequencies(rot, base=500000.0, scaling="linear", factor=3.0)
    eps = None if norm is None else 1e-5
    wq, wk = weights(d, norm == "f32") if norm in ("bf16", "f32") else (None, None)
    qo, ko = fa.qk_rotary(q, k, pos, freqs, interleaved=inter, rotary_scale=1.1, norm_eps=eps,
                          q_weight=wq, k_weight=wk)
    torch.cuda.synchronize()
    for x, w, o, name in ((q, wq, qo, "q"), (k, wk, ko, "k")):
        if x.shape[1]:
            check_forward(np64(o), np64(x), np64(pos), np64(freqs), inter, 1.1, eps,
                          None if w is None else np64(w), name)


def test_far_positions(fa):
    """Positions up to 2^31 - 1: the angle is exact to 2^-25 turns there too."""
    q, k = make(1, 2, 1, 8, 128, seed=1)
    pos = torch.tensor([0, 1, -1, 131071, 1 << 24, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)],
                       dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(128)
    qo, _ = fa.qk_rotary(q, k, pos, freqs)
    # fp64 p f itself is off by up to 2^-52 of 2^31 radians: 5e-7, 8 units more
    ref = orot.forward(np64(q), np64(pos)[None], np64(freqs), False)
    mag = partner_sum(np64(q), 64, False)
    assert np.all(np.abs(np64(qo) - ref) <= 2.0 ** -8 * np.abs(ref) + 48 * U * mag)


def test_norm_alone_and_nothing(fa):
    """freqs=None: the norm alone; without a norm either, a copy, bit for bit."""
    q, k = make(2, 3, 2, 11, 128, seed=2, fused=True)
    pos = torch.zeros(11, dtype=torch.int32, device=DEV)
    qo, ko = fa.qk_rotary(q, k, pos, None)
    assert torch.equal(qo, q) and torch.equal(ko, k)
    wq, wk = weights(128, False)
    qo, _ = fa.qk_rotary(q, k, pos, None, norm_eps=1e-6, q_weight=wq, k_weight=wk)
    check_forward(np64(qo), np64(q), np.zeros((2, 11)), [], False, 1.0, 1e-6, np64(wq), "norm")


def test_special_values(fa):
    """Infinities and NaN stay in their pair; elements that are not turned pass
    through bit for bit; a row of zeros with eps > 0 stays zero."""
    q, k = make(1, 2, 2, 4, 64, seed=4)
    q[0, 0, 0, 40] = float("inf")        # not turned (rot 32)
    q[0, 0, 1, 50] = float("nan")
    q[0, 1, 2, 3] = float("inf")         # turned, pair (3, 19)
    k[0, 0, 0] = 0
    pos = torch.arange(1, 5, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(32)
    for inter in (False, True):
        qo, ko = fa.qk_rotary(q, k, pos, freqs, interleaved=inter)
        assert torch.equal(qo[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16))
        bad = ~torch.isfinite(qo[0, 1, 2])
        assert bad.nonzero().flatten().tolist() == ([2, 3] if inter else [3, 19])
        assert torch.isfinite(qo[0, 0, 0, :32]).all()
        _, kn = fa.qk_rotary(k, k, pos, freqs, interleaved=inter, norm_eps=1e-6)
        assert (kn[0, 0, 0] == 0).all()


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place(fa, fused, inter):
    B, H, H_kv, N, d = 2, 8, 2, 37, 128
    q, k = make(B, H, H_kv, N, d, seed=6, fused=fused)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(128)
    wq, wk = weights(d, True)
    kw = dict(interleaved=inter, norm_eps=1e-6, q_weight=wq, k_weight=wk)
    qo, ko = fa.qk_rotary(q, k, pos, freqs, **kw)
    fa.qk_rotary(q, k, pos, freqs, q_out=q, k_out=k, **kw)
    assert torch.equal(q, qo) and torch.equal(k, ko)


BWD_SHAPES = [
    (1, 1, 1, 1, 64, 64),
    (2, 3, 1, 21, 64, 32),
    (3, 8, 2, 17, 128, 128),
    (1, 5, 5, 100, 128, 48),
    (2, 6, 2, 9, 256, 64),
    (1, 40, 8, 1, 128, 16),
    (130, 4, 1, 1, 128, 128),
    (1, 0, 3, 7, 128, 64),
    (1, 3, 0, 7, 64, 0),
]


@pytest.mark.parametrize("B,H,H_kv,N,d,rot", BWD_SHAPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [None, "bf16", "f32", "ones"])
def test_backward(fa, B, H, H_kv, N, d, rot, inter, norm):
    q, k = make(B, H, H_kv, N, d, seed=B * 77 + N, fused=N % 2 == 1)
    gq, gk = make(B, H, H_kv, N, d, seed=B * 78 + N, fused=N % 2 == 0)
    rng = np.random.default_rng(N + 1)
    pos = torch.from_numpy(rng.integers(0, 100000, (B, N)).astype(np.int32)).to(DEV)
    freqs = fa.rotary_frequencies(rot) if rot else None
    f64 = np64(freqs) if rot else np.zeros(0)
    eps = None if norm is None else 1e-5
    wq, wk = weights(d, norm == "f32") if norm in ("bf16", "f32") else (None, None)
    got = fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, interleaved=inter, rotary_scale=0.9,
                           norm_eps=eps, q_weight=wq, k_weight=wk)
    torch.cuda.synchronize()
    for x, dy, w, dx, dw, name in ((q, gq, wq, got[0], got[2], "q"),
                                   (k, gk, wk, got[1], got[3], "k")):
        w64 = None if w is None else np64(w)
        if not x.shape[1]:
            assert norm is None or (dw == 0).all()
            continue
        x64, dy64 = np64(x), np64(dy)
        rx, rw = orot.backward(dy64, x64, np64(pos), f64, inter, 0.9, eps, w64)
        g = partner_sum(dy64, len(f64), inter)
        if norm is None:
            assert dw is None
            tol = 2.0 ** -8 * np.abs(rx) + 32 * U * g
        else:
            ww = np.ones(d) if w64 is None else np.abs(w64)
            r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
            n = np.abs(x64 * r)
            gw = g * ww
            tol = 2.0 ** -8 * np.abs(rx) + 64 * U * r * (gw + n * (gw * n).mean(-1, keepdims=True))
            mag = (g * n).reshape(-1, d).sum(0)
            assert np.all(np.abs(np64(dw) - rw) <= 256 * U * mag), f"d{name}_weight"
        assert np.all(np.abs(np64(dx) - rx) <= tol + TINY), f"d{name}"


def test_backward_of_an_empty_batch(fa):
    x = torch.zeros(0, 4, 8, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(8, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(64)
    _, _, dwq, dwk = fa.qk_rotary_bwd(x, x, x, x, pos, freqs, norm_eps=1e-6)
    assert (dwq == 0).all() and (dwk == 0).all()
    fa.qk_rotary(x, x, pos, freqs)


def test_many_rows(fa):
    """More items than blocks (each block takes several): the weight gradients
    of 8192 x 40 rows, and repeated calls bit for bit."""
    B, H, H_kv, N, d = 2, 8, 2, 4099, 128
    q, k = make(B, H, H_kv, N, d, seed=12, fused=True)
    gq, gk = make(B, H, H_kv, N, d, seed=13)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(128)
    wq, wk = weights(d, True)
    kw = dict(norm_eps=1e-6, q_weight=wq, k_weight=wk)
    got = fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, **kw)
    again = fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, **kw)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    p64 = np.broadcast_to(np64(pos), (B, N))
    for x, dy, w, dx, dw in ((q, gq, wq, got[0], got[2]), (k, gk, wk, got[1], got[3])):
        rx, rw = orot.backward(np64(dy), np64(x), p64, np64(freqs), False, 1.0, 1e-6, np64(w))
        g = partner_sum(np64(dy), 64, False)
        n = np.abs(orot.norm(np64(x), 1e-6))
        assert np.all(np.abs(np64(dw) - rw) <= 256 * U * (g * n).reshape(-1, d).sum(0))
        r = 1 / np.sqrt((np64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        gw = g * np.abs(np64(w))
        tol = 2.0 ** -8 * np.abs(rx) + 64 * U * r * (gw + n * (gw * n).mean(-1, keepdims=True))
        assert np.all(np.abs(np64(dx) - rx) <= tol + TINY)


def test_other_stream_and_graph(fa):
    """A call on a named stream, and one captured and replayed on new inputs."""
    q, k = make(2, 4, 2, 50, 64, seed=20)
    gq, gk = make(2, 4, 2, 50, 64, seed=21)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(64)

    def step(**kw):
        return (*fa.qk_rotary(q, k, pos, freqs, norm_eps=1e-6, **kw),
                *fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, norm_eps=1e-6, **kw))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side.cuda_stream)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    q2, k2 = make(2, 4, 2, 50, 64, seed=22)
    q.copy_(q2)
    k.copy_(k2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(kept, step()):
        assert torch.equal(a, b)


def test_with_attention(fa):
    """A training step's path: qk_rotary, attention, its backward, qk_rotary's
    backward, against torch's fp64 autograd of the same definition. The attention works on
    bf16 queries, keys and gradients, so the bound is its own: 2e-2 of the largest
    gradient (tests/test_bwd_gpu.py), doubled for the rounded dq, dk that pass
    through the second backward."""
    B, H, H_kv, N, d = 1, 4, 2, 200, 64
    q, k = make(B, H, H_kv, N, d, seed=30, fused=True)
    g = torch.Generator().manual_seed(31)
    v = torch.randn(B, H_kv, N, d, generator=g).to(torch.bfloat16).to(DEV)
    do = torch.randn(B, H, N, d, generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(64)
    wq, wk = weights(d, True)
    kw = dict(norm_eps=1e-6, q_weight=wq, k_weight=wk)
    qr, kr = fa.qk_rotary(q, k, pos, freqs, **kw)
    o, lse = fa.attention(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.attention_bwd(qr, kr, v, o, lse, do, causal=True)
    dq, dk, dwq, dwk = fa.qk_rotary_bwd(dqr, dkr, q, k, pos, freqs, **kw)

    leaves = [t.double().requires_grad_() for t in (q, k, v, wq, wk)]
    q6, k6, v6, wq6, wk6 = leaves
    angle = pos.double()[:, None] * freqs

    def turn(x, w):
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = y.chunk(2, -1)
        return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1)

    kk = turn(k6, wk6).repeat_interleave(H // H_kv, 1)
    s = turn(q6, wq6) @ kk.transpose(-1, -2) / d ** 0.5
    s = s.masked_fill(torch.ones(N, N, device=DEV).triu(1).bool(), float("-inf"))
    oo = s.softmax(-1) @ v6.repeat_interleave(H // H_kv, 1)
    ref = torch.autograd.grad(oo, leaves, do.double())
    for got, want, name in zip((dq, dk, dv, dwq, dwk), ref, ("dq", "dk", "dv", "dwq", "dwk")):
        err = (got.double() - want).abs().max().item()
        assert err <= 4e-2 * want.abs().max().item(), f"{name}: {err}"
    err = (o.double() - oo).abs().max().item()
    assert err <= 2e-2 + 2.0 ** -8 * oo.abs().max().item()


def test_backward_in_place_and_repeated_gradients(fa):
    """dq, dk in the place of dq_out, dk_out; output gradients that are one row
    repeated (strides 0, as a sum's gradient comes); positions one row for all."""
    B, H, H_kv, N, d = 3, 5, 2, 21, 128
    q, k = make(B, H, H_kv, N, d, seed=40, fused=True)
    pos = torch.arange(7, 7 + N, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(96)
    wq, wk = weights(d, True)
    row = torch.randn(d, generator=torch.Generator().manual_seed(41)).to(torch.bfloat16).to(DEV)
    for kw in (dict(norm_eps=1e-6, q_weight=wq, k_weight=wk), dict()):
        gq, gk = row.expand(B, H, N, d), row.expand(B, H_kv, N, d)
        got = fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, **kw)
        want = fa.qk_rotary_bwd(gq.contiguous(), gk.contiguous(), q, k,
                                pos.expand(B, N).contiguous(), freqs, **kw)
        gq, gk = gq.contiguous(), gk.contiguous()
        place = fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, dq=gq, dk=gk, **kw)
        assert place[0] is gq and place[1] is gk
        for a, b, c in zip(got, want, place):
            assert (a is None and b is None and c is None) or \
                (torch.equal(a, b) and torch.equal(a, c))


@pytest.mark.parametrize("norm", [None, 1e-6])
def test_gradient_by_differences(fa, norm):
    """The backward against differences of the forward itself: along a random
    direction, (f(x + h v) - f(x - h v)) / 2h from the fp64 oracle's forward at
    the same bf16 point, whose step errors (1e-10) are far below the bound of the
    kernel's own rounding: 2^-8 of sum |dx v| for its bf16 result."""
    B, H, N, d = 1, 2, 6, 64
    q, k = make(B, H, H, N, d, seed=42)
    gq, gk = make(B, H, H, N, d, seed=43)
    pos = torch.arange(100, 100 + N, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(64)
    dq, dk, _, _ = fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, norm_eps=norm)
    p64, f64 = np64(pos)[None], np64(freqs)
    rng = np.random.default_rng(44)
    for x, g, dx in ((q, gq, dq), (k, gk, dk)):
        x, g, dx = np64(x), np64(g), np64(dx)
        for _ in range(4):
            v = rng.standard_normal(x.shape)
            h = 1e-6
            up = (g * orot.forward(x + h * v, p64, f64, False, 1.0, norm)).sum()
            down = (g * orot.forward(x - h * v, p64, f64, False, 1.0, norm)).sum()
            assert abs((up - down) / (2 * h) - (dx * v).sum()) <= 2.0 ** -8 * np.abs(dx * v).sum()


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 48), (256, 256)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("power,eps", [(50, 1e-6), (30, 1e-6), (-50, 0.0), (-44, 1e-30)])
def test_backward_of_large_and_small_rows(fa, power, eps, inter, d, rot):
    """Rows of rms 2^50 and 2^-50, where r^3 leaves fp32 while r, the row sums and
    the gradients are ordinary numbers; gradients along x, so that the mean's term
    counts. Each product is rounded as in test_backward: its bound."""
    B, H, H_kv, N = 2, 3, 1, 11
    q, k = make(B, H, H_kv, N, d, seed=d)
    gq, gk = make(B, H, H_kv, N, d, seed=d + 1)
    gq, gk = (0.5 * gq + q).to(torch.bfloat16), (0.5 * gk + k).to(torch.bfloat16)
    q, k = q * 2.0 ** power, k * 2.0 ** power
    pos = torch.arange(N, dtype=torch.int32, device=DEV).expand(B, N)
    freqs = fa.rotary_frequencies(rot)
    wq, wk = weights(d, True)
    got = fa.qk_rotary_bwd(gq, gk, q, k, pos, freqs, interleaved=inter, norm_eps=eps, q_weight=wq,
                           k_weight=wk)
    for x, dy, w, dx, dw, name in ((q, gq, wq, got[0], got[2], "q"),
                                   (k, gk, wk, got[1], got[3], "k")):
        x64, dy64, w64 = np64(x), np64(dy), np64(w)
        eps64 = float(np.float32(eps))
        rx, rw = orot.backward(dy64, x64, np64(pos), np64(freqs), inter, 1.0, eps64, w64)
        g = partner_sum(dy64, len(freqs), inter)
        r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps64)
        n = np.abs(x64 * r)
        gw = g * np.abs(w64)
        tol = 2.0 ** -8 * np.abs(rx) + 64 * U * r * (gw + n * (gw * n).mean(-1, keepdims=True))
        assert np.all(np.abs(np64(dx) - rx) <= tol + TINY), f"d{name}"
        assert np.all(np.abs(np64(dw) - rw) <= 256 * U * (g * n).reshape(-1, d).sum(0)), name


@pytest.mark.parametrize("inter", [False, True])
def test_infinite_weight_stays_in_its_pair(fa, inter):
    """An infinite weight of one element: those that are not turned, and the other
    pairs, do not see it."""
    q, k = make(1, 2, 2, 5, 64, seed=50)
    pos = torch.arange(1, 6, dtype=torch.int32, device=DEV)
    freqs = fa.rotary_frequencies(32)
    w = torch.ones(64, device=DEV)
    want, _ = fa.qk_rotary(q, k, pos, freqs, interleaved=inter, norm_eps=1e-6, q_weight=w)
    for at in (40, 63, 3):
        u = w.clone()
        u[at] = float("inf")
        got, _ = fa.qk_rotary(q, k, pos, freqs, interleaved=inter, norm_eps=1e-6, q_weight=u)
        here = [at] if at >= 32 else [2, 3] if inter else [3, 19]
        bad = ~torch.isfinite(got)
        assert bad[..., here].all()
        bad[..., here] = False
        assert not bad.any()
        rest = [i for i in range(64) if i not in here]
        assert torch.equal(got[..., rest], want[..., rest])
