"""Cases of the operators around the attention kernels: queries and keys on
their way in (per-head norm and rotary position, forward and backward), the
paged key-value cache (append, page copies) and one-token attention over it.

``run`` computes a case in plain torch operations, in 32 bits (angles in 64),
rounded once at the end; with ``own`` set it calls the library instead.
``exact`` gives the same results from the definitions in 64 bits.

Layouts are the library's: activations bf16 [B, heads, N, d]; cache pages
[pages, H_kv, page_size, d] (``token_major``: stored [pages, page_size, H_kv,
d] and viewed transposed); block_table int32 [B, pages per sequence].
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # query and key projections of the GPT-2-shaped training batch, read as
        # views of one fused projection output
        dict(name="rotary_gpt2_d64", kind="rotary", B=8, H=12, H_kv=12, N=1024, d=64, rot=64,
             interleaved=False, norm=False, w32=False, first=0, base=10000.0, factor=1.0),
        # the long-context workload with grouped heads: normed queries and keys
        # at far positions, linearly scaled
        dict(name="rotary_norm_long_context", kind="rotary", B=1, H=32, H_kv=8, N=16384, d=128,
             rot=128, interleaved=False, norm=True, w32=False, first=100000, base=500000.0,
             factor=4.0),
        # backward of the long-range training shape, with the norms' weight gradients
        dict(name="rotary_bwd_long_range", kind="rotary_bwd", B=2, H=16, H_kv=16, N=4096, d=128,
             rot=128, interleaved=False, norm=True, w32=True, first=0, base=10000.0, factor=1.0),
        # a small odd batch: wide heads, interleaved pairs, a quarter of the head rotated
        dict(name="rotary_bwd_odd_d256", kind="rotary_bwd", B=3, H=6, H_kv=2, N=333, d=256,
             rot=64, interleaved=True, norm=True, w32=False, first=17, base=10000.0, factor=1.0),
        # one new token of each of 16 sequences: a decoding step's entry into the cache
        dict(name="append_decode_step", kind="append", B=16, H=32, H_kv=8, N=1, d=128, page=16,
             elem=2, token_major=False, rot=128, interleaved=False, norm=True, w32=False,
             first=5000, base=500000.0, factor=1.0),
        # a prompt of 8192 tokens written into an e4m3 cache
        dict(name="append_prompt_e4m3", kind="append", B=1, H=32, H_kv=8, N=8192, d=128, page=64,
             elem=1, token_major=True, rot=64, interleaved=True, norm=False, w32=False, first=0,
             base=10000.0, factor=1.0),
        # one short sequence, one query head per key head: latency
        dict(name="decode_one_short_d64", kind="decode", B=1, H=12, H_kv=12, d=64, page=16, elem=2,
             token_major=False, lo=777, hi=777),
        # a serving batch of 16 with grouped heads and lengths 2048 to 8192
        dict(name="decode_gqa_ragged", kind="decode", B=16, H=32, H_kv=8, d=128, page=16, elem=2,
             token_major=False, lo=2048, hi=8192),
        # one sequence against a cache of 131072 tokens
        dict(name="decode_long_cache", kind="decode", B=1, H=32, H_kv=8, d=128, page=64, elem=2,
             token_major=False, lo=131072, hi=131072),
        # a wide batch over an e4m3 cache, some sequences just begun
        dict(name="decode_e4m3_ragged", kind="decode", B=32, H=32, H_kv=8, d=128, page=32, elem=1,
             token_major=True, lo=9, hi=8192),
        # copy-on-write of a few shared last pages when sequences fork
        dict(name="copy_fork_pages", kind="copy", H_kv=12, d=64, page=16, elem=2,
             token_major=False, pages=64, moved=7),
        # compaction: a third of a pool's pages moved down
        dict(name="copy_compact_pool", kind="copy", H_kv=8, d=128, page=16, elem=2,
             token_major=False, pages=6000, moved=2000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "rotary_bwd", "append", "decode", "decode", "copy"])
    d = rng.choice([64, 128, 256])
    H_kv = rng.choice([1, 2, 3, 4, 8, 12])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128, 256])
    elem = rng.choice([1, 2])
    token_major = rng.choice([False, True])
    if kind == "copy":
        most = max(8, 60_000_000 // (H_kv * page * d))
        pages = _log_int(rng, 8, min(most, 8000))
        return dict(kind=kind, H_kv=H_kv, d=d, page=page, elem=elem, token_major=token_major,
                    pages=pages, moved=rng.randint(1, pages // 2))
    H = H_kv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    if kind == "decode":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(131072, max(2, 130_000_000 // (B * H_kv * d))))
        return dict(kind=kind, B=B, H=H, H_kv=H_kv, d=d, page=page, elem=elem,
                    token_major=token_major, lo=rng.randint(1, hi), hi=hi)
    rotary = dict(rot=16 * rng.randint(1, d // 16), interleaved=rng.choice([False, True]),
                  norm=rng.choice([False, True]), w32=rng.choice([False, True]),
                  first=rng.choice([0, 1, 4097, 1_000_003]), base=rng.choice([10000.0, 500000.0]),
                  factor=rng.choice([1.0, 4.0]))
    most = max(4, 60_000_000 // ((H + H_kv) * d))
    if kind == "append":
        B = _log_int(rng, 1, 128)
        N = rng.choice([1, _log_int(rng, 1, max(1, min(8192, most // B)))])
        return dict(kind=kind, B=B, H=H, H_kv=H_kv, N=N, d=d, page=page, elem=elem,
                    token_major=token_major, **dict(rotary, first=min(rotary["first"], 4097)))
    B = _log_int(rng, 1, 8)
    N = _log_int(rng, 1, max(2, min(16384, most // B)))
    return dict(kind=kind, B=B, H=H, H_kv=H_kv, N=N, d=d, **rotary)


def _lengths(c):
    """Key counts of the sequences, spread evenly from lo to hi."""
    return [c["hi"] if c["B"] == 1 else c["lo"] + (c["hi"] - c["lo"]) * i // (c["B"] - 1)
            for i in range(c["B"])]


def _cache(g, pages, c, zero=False):
    """K and V pages as the cache holds them, and their descales."""
    shape = (pages, c["page"], c["H_kv"], c["d"]) if c["token_major"] else \
            (pages, c["H_kv"], c["page"], c["d"])
    descales = (0.0125, 0.009) if c["elem"] == 1 else (1.0, 1.0)
    got = []
    for s in descales:
        if zero:
            x = torch.zeros(shape, dtype=torch.uint8 if c["elem"] == 1 else torch.bfloat16,
                            device="cuda")
            x = x.view(torch.float8_e4m3fn) if c["elem"] == 1 else x
        else:
            x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
            if c["elem"] == 1:
                x = (x / s).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        got.append(x.transpose(1, 2) if c["token_major"] else x)
    return got[0], got[1], descales[0], descales[1]


def _rotary_inputs(g, c, s):
    """Positions, frequencies (radians per position, 64 bits) and norm weights."""
    B, N, d, rot = c["B"], c["N"], c["d"], c["rot"]
    i = torch.arange(0, rot, 2, device="cuda", dtype=torch.float64)
    s["freqs"] = torch.pow(torch.tensor(c["base"], device="cuda", dtype=torch.float64),
                           -i / rot) / c["factor"]
    s["positions"] = (c["first"] + torch.arange(N, device="cuda", dtype=torch.int32)
                      ).expand(B, N)
    if c["kind"] == "append" and N == 1:   # sequences of a decoding step differ in length
        s["positions"] = (c["first"] + 37 * torch.arange(B, device="cuda", dtype=torch.int32)
                          )[:, None].contiguous()
    s["eps"] = 1e-6 if c["norm"] else None
    s["wq"] = s["wk"] = None
    if c["norm"]:
        t = torch.float32 if c["w32"] else torch.bfloat16
        s["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(t)
        s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(t)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c, "scale": 1.0 / math.sqrt(c["d"])}
    kind = c["kind"]

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    if kind in ("rotary", "rotary_bwd", "append"):
        B, H, H_kv, N, d = (c[n] for n in ("B", "H", "H_kv", "N", "d"))
        # the fused projection's output, [B, N, heads, d]; q, k, v are views of it
        qkv = rand(B, N, H + 2 * H_kv, d).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
        _rotary_inputs(g, c, s)
    if kind == "rotary_bwd":
        s["dq_out"], s["dk_out"] = rand(B, H, N, d), rand(B, H_kv, N, d)
    if kind == "append":
        last = int(s["positions"].max())
        width = last // c["page"] + 1
        # pages of a running cache: only those that this call writes have to differ
        pages = B * (N // c["page"] + 2) + 3
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(g, pages, c, zero=True)
        per = N // c["page"] + 2
        own_pages = torch.randperm(pages - 3, generator=g, device="cuda").view(B, per)
        start = s["positions"][:, :1] // c["page"]
        col = torch.arange(width, device="cuda")[None] - start
        s["table"] = torch.where((col >= 0) & (col < per),
                                 own_pages.gather(1, col.clamp(0, per - 1)),
                                 torch.full_like(col, pages - 1)).to(torch.int32)
    if kind == "decode":
        B, H, d = c["B"], c["H"], c["d"]
        s["q"] = rand(B, H, 1, d)
        order = torch.randperm(B, generator=g, device="cuda")
        s["kv_len"] = torch.tensor(_lengths(c), device="cuda", dtype=torch.int32)[order]
        width = -(-c["hi"] // c["page"])
        pages = B * width + 5
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(g, pages, c)
        s["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * width].view(
            B, width).to(torch.int32)
    if kind == "copy":
        s["kc"], s["vc"], _, _ = _cache(g, c["pages"], c)
        p = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
        s["src"], s["dst"] = p[:c["moved"]], p[c["moved"]:2 * c["moved"]]
    return s


# ------------------------------------------------------------------ plain forms
def _cos_sin(s):
    angle = s["positions"].double()[:, None, :, None] * s["freqs"]
    return angle.cos().float(), angle.sin().float()


def _pairs(x, rot, interleaved):
    """The first and second members of the rotated pairs, and the untouched rest."""
    r = x[..., :rot]
    if interleaved:
        return r[..., 0::2], r[..., 1::2], x[..., rot:]
    return r[..., :rot // 2], r[..., rot // 2:], x[..., rot:]


def _join(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _rotated(x, cos, sin, rot, interleaved):
    a, b, rest = _pairs(x, rot, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, interleaved)


def _normed(x, w, eps):
    if eps is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _head_bwd(dy, x, w, eps, cos, sin, rot, interleaved):
    """Gradient through the rotation (its transpose), then through the norm."""
    g = _rotated(dy.float(), cos, -sin, rot, interleaved)
    if eps is None:
        return g.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    xn = x * r
    dw = (g * xn).double().sum((0, 1, 2)).float()
    gw = g * w.float()
    dx = r * (gw - xn * (gw * xn).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dw


def _store(cache, page, slot, x, descale):
    if cache.dtype == torch.float8_e4m3fn:
        code = (x.float() / descale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache.view(torch.uint8)[page, :, slot] = code.view(torch.uint8).transpose(1, 2)
    else:
        cache[page, :, slot] = x.to(torch.bfloat16).transpose(1, 2)


def _gathered(cache, table):
    """[B, H_kv, keys, d] in 32 bits of the pages a table names."""
    x = cache.view(torch.uint8)[table].view(cache.dtype) if cache.dtype == torch.float8_e4m3fn \
        else cache[table]
    x = x.float().transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _plain(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind == "rotary":
        cos, sin = _cos_sin(s)
        return tuple(_rotated(_normed(x.float(), w, s["eps"]), cos, sin, c["rot"],
                              c["interleaved"]).to(torch.bfloat16)
                     for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    if kind == "rotary_bwd":
        cos, sin = _cos_sin(s)
        dq, dwq = _head_bwd(s["dq_out"], s["q"], s["wq"], s["eps"], cos, sin, c["rot"],
                            c["interleaved"])
        dk, dwk = _head_bwd(s["dk_out"], s["k"], s["wk"], s["eps"], cos, sin, c["rot"],
                            c["interleaved"])
        return (dq, dk) if s["eps"] is None else (dq, dk, dwq, dwk)
    if kind == "append":
        cos, sin = _cos_sin(s)
        q = _rotated(_normed(s["q"].float(), s["wq"], s["eps"]), cos, sin, c["rot"],
                     c["interleaved"]).to(torch.bfloat16)
        k = _rotated(_normed(s["k"].float(), s["wk"], s["eps"]), cos, sin, c["rot"],
                     c["interleaved"])
        page = s["table"].gather(1, (s["positions"] // c["page"]).long()).long()
        slot = (s["positions"] % c["page"]).long()
        _store(s["kc"], page, slot, k, s["ks"])
        _store(s["vc"], page, slot, s["v"], s["vs"])
        return q, s["kc"], s["vc"]
    if kind == "decode":
        B, H, H_kv, d = c["B"], c["H"], c["H_kv"], c["d"]
        k, v = _gathered(s["kc"], s["table"]), _gathered(s["vc"], s["table"])
        q = s["q"].float().view(B, H_kv, H // H_kv, d)
        score = (q @ k.transpose(-1, -2)) * (s["scale"] * s["ks"])
        hidden = torch.arange(k.shape[2], device="cuda")[None] >= s["kv_len"][:, None]
        score = score.masked_fill(hidden[:, None, None], -math.inf)
        m = score.amax(-1, keepdim=True)
        p = torch.exp(score - m)
        total = p.sum(-1, keepdim=True)
        o = (p @ v) / total * s["vs"]
        return o.to(torch.bfloat16).view(B, H, 1, d), (m + total.log()).view(B, H, 1)
    s["kc"].view(torch.uint8)[s["dst"].long()] = s["kc"].view(torch.uint8)[s["src"].long()]
    s["vc"].view(torch.uint8)[s["dst"].long()] = s["vc"].view(torch.uint8)[s["src"].long()]
    return s["kc"], s["vc"]


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import io_aware_exact_18_b200 as fa
    c, kind = s["case"], s["case"]["kind"]
    if kind == "rotary":
        return fa.qk_rotary(s["q"], s["k"], s["positions"], s["freqs"],
                            interleaved=c["interleaved"], norm_eps=s["eps"], q_weight=s["wq"],
                            k_weight=s["wk"])
    if kind == "rotary_bwd":
        dq, dk, dwq, dwk = fa.qk_rotary_bwd(
            s["dq_out"], s["dk_out"], s["q"], s["k"], s["positions"], s["freqs"],
            interleaved=c["interleaved"], norm_eps=s["eps"], q_weight=s["wq"], k_weight=s["wk"])
        return (dq, dk) if s["eps"] is None else (dq, dk, dwq, dwk)
    if kind == "append":
        q = fa.paged_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["positions"],
                            q=s["q"], freqs=s["freqs"], interleaved=c["interleaved"],
                            norm_eps=s["eps"], q_weight=s["wq"], k_weight=s["wk"],
                            k_descale=s["ks"], v_descale=s["vs"])
        return q, s["kc"], s["vc"]
    if kind == "decode":
        return fa.paged_decode_attention(s["q"], s["kc"], s["vc"], s["table"], s["kv_len"],
                                         k_descale=s["ks"], v_descale=s["vs"])
    fa.copy_pages(s["kc"], s["vc"], s["src"], s["dst"])
    return s["kc"], s["vc"]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    c, kind = case, case["kind"]
    d, H_kv = c["d"], c["H_kv"]
    if kind == "copy":
        return {"bytes": 2 * 2 * c["moved"] * H_kv * c["page"] * d * c["elem"] + 8 * c["moved"],
                "flops": 0}
    if kind == "decode":
        keys = sum(_lengths(c))
        return {"bytes": 2 * keys * H_kv * d * c["elem"] + c["B"] * c["H"] * (4 * d + 4)
                + 4 * c["B"] + 4 * sum(-(-n // c["page"]) for n in _lengths(c)),
                "flops": 4 * keys * c["H"] * d}
    rows = c["B"] * c["N"] * (c["H"] + H_kv)
    tokens = c["B"] * c["N"]
    per = 3 * c["rot"] + (4 * d if c["norm"] else 0)     # operations of a row, forward
    small = 4 * tokens + 4 * c["rot"] + (4 * d * (2 if c["w32"] else 1) if c["norm"] else 0)
    if kind == "rotary":
        return {"bytes": rows * d * 4 + small, "flops": rows * per}
    if kind == "rotary_bwd":
        grads = 8 * d if c["norm"] else 0
        return {"bytes": rows * d * (6 if c["norm"] else 4) + small + grads,
                "flops": rows * (3 * c["rot"] + (12 * d if c["norm"] else 0))}
    store = tokens * H_kv * d * (4 + 2 * c["elem"])      # k and v read, their codes written
    return {"bytes": tokens * c["H"] * d * 4 + store + small + 4 * tokens, "flops": rows * per}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_head(x, pos, s, w):
    """Norm (if any), then each pair (a, b) turned by its angle, one pair at a time."""
    c = s["case"]
    y = x.double().clone()
    if s["eps"] is not None:
        ms = (y * y).sum(-1) / c["d"] + s["eps"]
        y = y / ms.sqrt()[..., None] * w.double()
    out = y.clone()
    for i in range(c["rot"] // 2):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rot"] // 2)
        t = (pos.double() * s["freqs"][i])[:, None]
        out[..., a] = y[..., a] * torch.cos(t) - y[..., b] * torch.sin(t)
        out[..., b] = y[..., a] * torch.sin(t) + y[..., b] * torch.cos(t)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, kind = s["case"], case["kind"]
    if kind == "rotary":
        return (_exact_head(s["q"], s["positions"], s, s["wq"]),
                _exact_head(s["k"], s["positions"], s, s["wk"]))
    if kind == "rotary_bwd":      # by differentiating the definition
        grads, weights = [], []
        for x, dy, w in ((s["q"], s["dq_out"], s["wq"]), (s["k"], s["dk_out"], s["wk"])):
            x = x.double().requires_grad_()
            w = None if w is None else w.double().requires_grad_()
            leaves = (x,) if w is None else (x, w)
            with torch.enable_grad():
                got = torch.autograd.grad(_exact_head(x, s["positions"], s, w), leaves,
                                          dy.double())
            grads.append(got[0])
            weights += got[1:]
        return (*grads, *weights)
    if kind == "append":
        q = _exact_head(s["q"], s["positions"], s, s["wq"])
        k = _exact_head(s["k"], s["positions"], s, s["wk"])
        kc, vc = s["kc"].double().contiguous(), s["vc"].double().contiguous()
        limit = E4M3_MAX if c["elem"] == 1 else math.inf
        for b in range(c["B"]):
            pos = s["positions"][b].long()
            page, slot = s["table"][b].long()[pos // c["page"]], pos % c["page"]
            kc[page, :, slot] = (k[b] / s["ks"]).clamp(-limit, limit).transpose(0, 1)
            vc[page, :, slot] = (s["v"][b].double() / s["vs"]).clamp(-limit, limit).transpose(0, 1)
        return q, kc, vc
    if kind == "decode":
        o = torch.zeros(c["B"], c["H"], 1, c["d"], dtype=torch.float64, device="cuda")
        lse = torch.zeros(c["B"], c["H"], 1, dtype=torch.float64, device="cuda")
        group = c["H"] // c["H_kv"]
        for b, n in enumerate(s["kv_len"].tolist()):
            pos = torch.arange(n, device="cuda")
            page, slot = s["table"][b].long()[pos // c["page"]], pos % c["page"]
            pages, at = torch.unique(page, return_inverse=True)
            for h in range(c["H_kv"]):
                k = s["kc"][:, h].view(torch.uint8)[pages].view(s["kc"].dtype).double()[at, slot]
                v = s["vc"][:, h].view(torch.uint8)[pages].view(s["vc"].dtype).double()[at, slot]
                rows = slice(h * group, (h + 1) * group)
                z = s["scale"] * (s["q"][b, rows, 0].double() @ (k * s["ks"]).T)
                lse[b, rows, 0] = torch.logsumexp(z, -1)
                o[b, rows, 0] = torch.softmax(z, -1) @ (v * s["vs"])
        return o, lse
    kc, vc = s["kc"].clone(), s["vc"].clone()
    for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
        kc[j], vc[j] = s["kc"][i], s["vc"][i]
    return kc.double(), vc.double()
