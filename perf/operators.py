"""Cases of the serving operators: products with 4-bit weights, their quantiser,
the append to a paged 8-bit key/value cache, and attention over that cache.

`own` false: the operators in elementary torch operations; true: the same calls
through dense_tiled_gemm_fp8_amd.gemm355.

Buffers, as the library has them:
  codes    uint8 [N][ldw / 2], two 4-bit codes a byte, element 2i in the low nibble
  k, v     uint8 E4M3, k [pages][heads][page][dim], v [pages][heads][dim][page]
  *_scale  uint8 E8M0 [pages][heads]
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def _w4(name, M, N, K, fmt, group, zeros, out):
    return {"name": name, "op": "w4_gemm", "M": M, "N": N, "K": K, "fmt": fmt, "group": group, "zeros": zeros, "out": out}


def _q4(name, N, K, fmt, group, zeros, src):
    return {"name": name, "op": "w4_quantize", "N": N, "K": K, "fmt": fmt, "group": group, "zeros": zeros, "src": src}


def _app(name, B, new, L, Hq, H, D, page, rot, interleaved):
    return {"name": name, "op": "kv_append", "B": B, "new": new, "L": L, "Hq": Hq, "H": H, "D": D, "page": page,
            "rot": rot, "interleaved": interleaved}


def _att(name, B, new, L, Hq, H, D, page, window, sinks):
    return {"name": name, "op": "attention", "B": B, "new": new, "L": L, "Hq": Hq, "H": H, "D": D, "page": page,
            "window": window, "sinks": sinks}


def listed():
    return [
        # one token through a small projection: what a call costs at least
        _w4("w4_gemm-m1-1024x1024", 1, 1024, 1024, "int", 128, False, "bf16"),
        # one token through a wide feed-forward matrix with zero points: the stream of codes counts
        _w4("w4_gemm-m1-16384x8192", 1, 16384, 8192, "int", 64, True, "bf16"),
        # five draft tokens, sizes that no tile divides, odd K, sums kept in 32 bits
        _w4("w4_gemm-m5-3000x777", 5, 3000, 777, "int", 32, False, "f32"),
        # a decode batch over block-scaled FP4 weights
        _w4("w4_gemm-m32-8192x8192", 32, 8192, 8192, "mxfp4", 32, False, "bf16"),
        # quantising a layer's bf16 weights with zero points when a model is loaded
        _q4("w4_quantize-8192x8192", 8192, 8192, "int", 64, True, "bf16"),
        # a small fp32 matrix into block-scaled FP4, last block short
        _q4("w4_quantize-1000x3000", 1000, 3000, "mxfp4", 32, False, "f32"),
        # a decode step of 32 sequences: one new token each
        _app("kv_append-32x1", 32, 1, 4096, 32, 8, 128, 64, 128, False),
        # prompts of up to 1000 tokens behind cached prefixes, half of each head rotated
        _app("kv_append-8x1000", 8, 1000, 4096, 16, 4, 128, 32, 64, True),
        # one short sequence, as many key heads as query heads: latency
        _att("attention-1x700", 1, 1, 700, 8, 8, 64, 16, 0, 0),
        # a decode batch at length
        _att("attention-64x8192", 64, 1, 8192, 32, 8, 128, 64, 0, 0),
        # two long documents: few rows, a long axis
        _att("attention-2x65536", 2, 1, 65536, 16, 2, 128, 128, 0, 0),
        # chunks of prompts with a sliding window and four tokens that stay visible
        _att("attention-4x512-window", 4, 512, 8192, 16, 4, 128, 32, 2048, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("w4_gemm", "w4_gemm", "w4_quantize", "kv_append", "attention", "attention"))
    fmt = rng.choice(("int", "int", "mxfp4"))
    group = 32 if fmt == "mxfp4" else rng.choice((32, 64, 128))
    zeros = fmt == "int" and rng.random() < 0.5
    if op == "w4_gemm":
        N, K = _log(rng, 256, 16384), _log(rng, 256, 8192)
        if rng.random() < 0.6:
            N, K = N // 64 * 64, K // 128 * 128
        M = rng.choice((1, 1, 2, 4, _log(rng, 2, 64)))
        c = _w4("", M, N, K, fmt, group, zeros, rng.choice(("bf16", "f32")))
    elif op == "w4_quantize":
        N, K = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.5:
            K = -(-K // 128) * 128
        c = _q4("", N, min(K, 8192), fmt, group, zeros, rng.choice(("bf16", "f32")))
    else:
        H, D = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128, 256))
        Hq, page = H * rng.choice((1, 2, 4, 5, 8)), rng.choice((16, 32, 64, 128))
        new = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 16, 512)))
        if op == "kv_append":
            B = _log(rng, 1, max(1, min(64, 4096 // new)))
            c = _app("", B, new, _log(rng, 600, 8192), Hq, H, D, page, rng.choice((D, D // 2)), rng.random() < 0.5)
        else:
            B = _log(rng, 1, 64 if new < 9 else 4)
            L = max(new, _log(rng, 64, min(65536, (1 << 28) // (B * H * D)) if new < 9 else 4096))
            window = rng.choice((0, 0, _log(rng, 16, 4096)))
            c = _att("", B, new, L, Hq, H, D, page, window, rng.choice((0, 4)) if window else 0)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that follow from a case

def _news(c):
    """New tokens of each sequence: one, or from half of `new` to `new`."""
    B, new = c["B"], c["new"]
    return [new - (i * (new // 2)) // B for i in range(B)]


def _lens(c):
    """Lengths with the new tokens: from half of L to L."""
    B, L = c["B"], c["L"]
    return [max(n, L - (i * (L // 2)) // B) for i, n in enumerate(_news(c))]


def _visible(c, p):
    """Tokens that a query at position p sees."""
    if not c["window"] or p + 1 <= c["window"]:
        return p + 1
    return c["window"] + min(c["sinks"], p + 1 - c["window"])


def work(case):
    c = case
    if c["op"] in ("w4_gemm", "w4_quantize"):
        N, K = c["N"], c["K"]
        ng = -(-K // c["group"])
        packed = N * (K / 2 + ng * ((1 if c["fmt"] == "mxfp4" else 2) + (1 if c["zeros"] else 0)))
        if c["op"] == "w4_gemm":
            M = c["M"]
            return {"bytes": packed + 2 * M * K + M * N * (2 if c["out"] == "bf16" else 4), "flops": 2 * M * N * K}
        # the weights in, codes and scales out and in again, the values that they stand for out
        return {"bytes": N * K * (2 if c["src"] == "bf16" else 4) + 2 * packed + 2 * N * K, "flops": 4 * N * K}
    news, lens, H, Hq, D = _news(c), _lens(c), c["H"], c["Hq"], c["D"]
    T = sum(news)
    if c["op"] == "kv_append":
        return {"bytes": T * D * (2 * H * 3 + Hq * 4 + 8), "flops": T * D * (H + Hq) * 6}
    read = sum(min(n_t, c["window"] + n - 1 + c["sinks"]) if c["window"] else n_t for n_t, n in zip(lens, news))
    pairs = sum(_visible(c, p) for n_t, n in zip(lens, news) for p in range(n_t - n, n_t))
    return {"bytes": read * H * D * 2 + T * Hq * (D * 4 + 4), "flops": pairs * Hq * D * 4}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "w4_gemm":
        _prepare_w4_gemm(c, s, g)
    elif c["op"] == "w4_quantize":
        N, K = c["N"], c["K"]
        w = torch.randn(N, K, generator=g, device="cuda") * 0.02
        w *= torch.exp(0.5 * torch.randn(1, K, generator=g, device="cuda"))    # channels of uneven size
        s["w"] = w.to(torch.bfloat16) if c["src"] == "bf16" else w
        _packed_buffers(c, s)
        s["values"] = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    else:
        _prepare_cache(c, s, g)
    if own:
        _handles(c, s)
    return s


def _packed_buffers(c, s):
    N, K = c["N"], c["K"]
    ng = -(-K // c["group"])
    s["codes"] = torch.zeros(N, -(-K // 32) * 16, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.zeros(N, ng, dtype=torch.uint8 if c["fmt"] == "mxfp4" else torch.bfloat16, device="cuda")
    s["zeros"] = torch.zeros(N, ng, dtype=torch.uint8, device="cuda") if c["zeros"] else None


def _prepare_w4_gemm(c, s, g):
    M, N, K = c["M"], c["N"], c["K"]
    _packed_buffers(c, s)
    s["x"] = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    if c["fmt"] == "mxfp4":
        s["codes"].random_(0, 256, generator=g)
        s["scales"].random_(118, 122, generator=g)
    else:
        u = torch.randn(N, s["codes"].shape[1] * 2, generator=g, device="cuda").mul_(2.3).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        s["codes"].copy_(u[:, 0::2] | (u[:, 1::2] << 4))
        s["scales"].copy_(0.004 + 0.008 * torch.rand(s["scales"].shape, generator=g, device="cuda"))
        if c["zeros"]:
            s["zeros"].random_(5, 11, generator=g)
    s["y"] = torch.empty(M, N, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device="cuda")


def _prepare_cache(c, s, g):
    B, H, Hq, D, page = c["B"], c["H"], c["Hq"], c["D"], c["page"]
    news, lens = _news(c), _lens(c)
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    news, lens = [news[i] for i in order], [lens[i] for i in order]
    T, cols = sum(news), -(-max(lens) // page)
    start = [0]
    for n in news:
        start.append(start[-1] + n)
    pages = sum(-(-n // page) for n in lens)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    rows = []
    for n in lens:
        k = -(-n // page)
        rows.append([ids.pop() for _ in range(k)] + [0] * (cols - k))
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s["table"], s["lens"], s["start"] = torch.tensor(rows, **i32), torch.tensor(lens, **i32), torch.tensor(start, **i32)
    s["T"], s["max_new"], s["max_len"], s["pages"] = T, max(news), max(lens), pages
    for name, shape in (("k", (pages, H, page, D)), ("v", (pages, H, D, page))):
        codes = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(107.0).clamp_(-448.0, 448.0)
        s[name] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_scale"] = torch.randint(119, 122, (pages, H), generator=g, device="cuda", dtype=torch.uint8)
    if c["op"] == "attention":
        s["q"] = (2.0 * torch.randn(T, Hq, D, generator=g, device="cuda")).to(torch.bfloat16)
        s["o"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
        return
    for name, heads in (("xk", H), ("xv", H), ("q", Hq)):
        s[name] = torch.randn(T, heads, D, generator=g, device="cuda").to(torch.bfloat16)
    s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    half = c["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(c["L"] + c["new"], device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()


# ------------------------------------------------------------------ the framework's calls

def _handles(c, s):
    """Descriptors that a serving program makes once: of a weight matrix, of a cache and of a step's buffers."""
    from dense_tiled_gemm_fp8_amd import gemm355 as lib
    s["lib"] = lib
    if c["op"] in ("w4_gemm", "w4_quantize"):
        s["matrix"] = lib.make_w4_matrix(c["N"], c["K"], s["codes"], s["scales"], s["zeros"],
                                         fmt=lib.W4_MXFP4 if c["fmt"] == "mxfp4" else lib.W4_INT, group=c["group"])
        return
    cache = lib.make_kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], pages=s["pages"], heads=c["H"], head_dim=c["D"],
                              page=c["page"], table=s["table"], lens=s["lens"], batch=c["B"], max_len=s["max_len"],
                              q_start=s["start"], tokens=s["T"], max_new=s["max_new"])
    if c["op"] == "kv_append":
        s["args"] = lib.make_kv_append_args(cache, s["xk"], s["xv"], q=s["q"], q_out=s["q_out"], q_heads=c["Hq"], cos=s["cos"],
                                            sin=s["sin"], rot_dim=c["rot"], rot_len=s["cos"].shape[0], interleaved=c["interleaved"])
    else:
        s["args"] = lib.make_attention_args(cache, s["q"], s["o"], q_heads=c["Hq"], lse=s["lse"], scale=c["D"] ** -0.5,
                                            window=c["window"], sinks=c["sinks"])


def _run_own(c, s):
    lib = s["lib"]
    if c["op"] == "w4_gemm":
        lib.gemm355_w4_gemm(c["M"], s["x"], s["matrix"], s["y"], out=lib.SRC_BF16 if c["out"] == "bf16" else lib.SRC_F32)
        return {"y": s["y"]}
    if c["op"] == "w4_quantize":
        lib.gemm355_w4_quantize(s["w"], s["matrix"], src=lib.SRC_BF16 if c["src"] == "bf16" else lib.SRC_F32)
        lib.gemm355_w4_dequantize(s["matrix"], s["values"], dst=lib.SRC_BF16)
        return _packed_outputs(s)
    if c["op"] == "kv_append":
        lib.gemm355_kv_append(s["args"])
        return _cache_outputs(s)
    lib.gemm355_attention(s["args"])
    return {"o": s["o"], "lse": s["lse"]}


def _packed_outputs(s):
    return {"values": s["values"], "scales": s["scales"], "zeros": s["zeros"]}


def _cache_outputs(s):
    f8 = torch.float8_e4m3fn
    return {"q": s["q_out"], "k": s["k"].view(f8), "v": s["v"].view(f8), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    c = state["c"]
    if own:
        return _run_own(c, state)
    if c["op"] == "w4_gemm":
        w = _weights(c, state)
        return {"y": torch.matmul(state["x"].float(), w.t()).to(state["y"].dtype)}
    if c["op"] == "w4_quantize":
        return _plain_quantize(c, state)
    if c["op"] == "kv_append":
        return _plain_append(c, state)
    return _plain_attention(c, state)


# ------------------------------------------------------------------ plain forms

def _pow2(e):
    """2^e for whole e in [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _weights(c, s):
    """The values that a packed matrix stands for, in 32 bits."""
    K = c["K"]
    u = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).reshape(c["N"], -1)[:, :K]
    if c["fmt"] == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=u.device)
        return table[u.long()] * _pow2(s["scales"].int() - 127).repeat_interleave(32, 1)[:, :K]
    z = s["zeros"].float().repeat_interleave(c["group"], 1)[:, :K] if c["zeros"] else 8.0
    return (u.float() - z) * s["scales"].float().repeat_interleave(c["group"], 1)[:, :K]


def _quotient(a, b):
    """a / b of 32-bit values, rounded to 32 bits once."""
    return (a.double() / b.double()).float()


def _plain_quantize(c, s):
    N, K, G = c["N"], c["K"], c["group"]
    ng = -(-K // G)
    w = torch.nn.functional.pad(s["w"].float(), (0, ng * G - K)).reshape(N, ng, G)
    if c["fmt"] == "mxfp4":
        a = w.abs().amax(2, keepdim=True)
        e = (torch.frexp(a).exponent - 3).clamp(-127, 127)
        e = torch.where(a == 0, -127, e)
        t = (w.double() * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=w.device), -e.double())).abs().float()
        mag = ((t > 0.25).int() + (t >= 0.75).int() + (t > 1.25).int() + (t >= 1.75).int() + (t > 2.5).int() + (t >= 3.5).int()
               + (t > 5.0).int())
        u = mag + 8 * torch.signbit(w).int()
        s["scales"].copy_(e[:, :, 0] + 127)
    else:
        if c["zeros"]:
            lo, hi = w.amin(2, keepdim=True).clamp(max=0), w.amax(2, keepdim=True).clamp(min=0)
            a, steps = hi - lo, 15.0
        else:
            a, steps = w.abs().amax(2, keepdim=True), 7.0
        sc = torch.where(a < 2.0 ** -100, 1.0, _quotient(a, torch.full_like(a, steps)).to(torch.bfloat16).float())
        z = _quotient(-lo, sc).round().clamp(0, 15) if c["zeros"] else torch.full_like(sc, 8.0)
        r = _quotient(w, sc).round()
        u = ((r + z).clamp(0, 15) if c["zeros"] else r.clamp(-8, 7) + 8).int()
        s["scales"].copy_(sc[:, :, 0])
        if c["zeros"]:
            s["zeros"].copy_(z[:, :, 0])
    u = u.reshape(N, ng * G)[:, :K].to(torch.uint8)
    u = torch.nn.functional.pad(u, (0, s["codes"].shape[1] * 2 - K))
    s["codes"].copy_(u[:, 0::2] | (u[:, 1::2] << 4))
    s["values"].copy_(_weights(c, s))
    return _packed_outputs(s)


def _rows(c, s):
    """Of each new token: its sequence, its place among that sequence's new tokens, its position."""
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["start"], t, right=True) - 1
    i = t - s["start"][b]
    return b, i, s["lens"][b] - (s["start"][b + 1] - s["start"][b]) + i


def _rotated(c, s, x, pos):
    cos, sin = s["cos"][pos].double()[:, None], s["sin"][pos].double()[:, None]
    rot = c["rot"]
    head, rest = x[..., :rot].double(), x[..., rot:].float()
    if c["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).reshape(head.shape)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y.float(), rest), -1)


def _plain_append(c, s):
    page, new = c["page"], s["max_new"]
    _, _, pos = _rows(c, s)
    pos = pos.long()
    lens, n = s["lens"].long(), (s["start"][1:] - s["start"][:-1]).long()
    J = (new + page - 2) // page + 1
    # pages that get new tokens; one past a sequence's last stands for the last again
    pg = torch.minimum((lens - n)[:, None] // page + torch.arange(J, device="cuda"), (lens - 1)[:, None] // page)
    at = s["table"].long().gather(1, pg)
    p = pg[:, :, None] * page + torch.arange(page, device="cuda")
    old, fresh = p < (lens - n)[:, None, None], (p >= (lens - n)[:, None, None]) & (p < lens[:, None, None])
    t = (s["start"][:-1].long()[:, None, None] + p - (lens - n)[:, None, None]).clamp(0, s["T"] - 1)
    begins = (pg * page >= (lens - n)[:, None])[:, :, None]
    s["q_out"].copy_(_rotated(c, s, s["q"], pos))
    for name, x in (("k", _rotated(c, s, s["xk"], pos)), ("v", s["xv"].float())):
        x = torch.where(fresh[..., None, None], x[t], 0.0)                      # [B, J, page, H, D]
        m, e = torch.frexp(x.abs().amax((2, 4)))
        e = torch.where(m == 0, -100, (e - 9 + (m > 0.875).int()).clamp(-100, 120))
        e_old = s[name + "_scale"][at].int() - 127
        e = torch.where(begins, e, torch.maximum(e, e_old))
        codes = s[name][at] if name == "k" else s[name][at].transpose(3, 4)     # [B, J, H, page, D]
        f8 = torch.float8_e4m3fn
        moved = (codes.view(f8).float() * _pow2((e_old - e).clamp(-60, 0))[..., None, None]).to(f8).view(torch.uint8)
        made = (x.permute(0, 1, 3, 2, 4) * _pow2(-e)[..., None, None]).clamp(-448, 448).to(f8).view(torch.uint8)
        out = torch.where(fresh[:, :, None, :, None], made, torch.where(old[:, :, None, :, None], moved, codes))
        s[name][at] = out if name == "k" else out.transpose(3, 4)
        s[name + "_scale"][at] = (e + 127).to(torch.uint8)
    return _cache_outputs(s)


def _plain_attention(c, s):
    B, H, Hq, D, page, T, n = c["B"], c["H"], c["Hq"], c["D"], c["page"], s["T"], s["max_new"]
    at, group = s["table"].long(), Hq // H
    f8 = torch.float8_e4m3fn
    k = s["k"][at].view(f8).float() * _pow2(s["k_scale"][at].int() - 127)[..., None, None]
    v = s["v"][at].view(f8).float() * _pow2(s["v_scale"][at].int() - 127)[..., None, None]
    k = k.transpose(1, 2).reshape(B, H, -1, D)                                  # [B, np, H, page, D]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, H, -1, D)                           # [B, np, H, D, page]
    b, i, pos = _rows(c, s)
    row = (s["start"][:-1].long()[:, None] + torch.arange(n, device="cuda")).clamp(max=T - 1)
    q = s["q"].float()[row].reshape(B, n, H, group, D).transpose(1, 2).reshape(B, H, n * group, D)
    score = torch.matmul(q * D ** -0.5, k.transpose(2, 3)).reshape(B, H, n, group, -1)
    t = torch.arange(k.shape[2], device="cuda")
    p = pos[row][:, :, None]
    seen = t <= p
    if c["window"]:
        seen &= (t > p - c["window"]) | (t < c["sinks"])
    seen = seen[:, None, :, None]
    score = torch.where(seen, score, -math.inf)
    m = score.amax(-1, keepdim=True)
    w = torch.where(seen, torch.exp(score - m), 0.0)
    total = w.sum(-1, keepdim=True)
    v = torch.where((t < s["lens"][:, None])[:, None, :, None], v, 0.0)         # what lies behind a sequence is not read
    o = torch.matmul((w / total).reshape(B, H, n * group, -1), v).reshape(B, H, n, group, D)
    lse = (m + total.log())[..., 0]
    o = o.transpose(1, 2).reshape(B, n, Hq, D)[b.long(), i.long()]
    lse = lse.transpose(1, 2).reshape(B, n, Hq)[b.long(), i.long()]
    return {"o": o.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "w4_gemm":
        return {"y": s["x"].double() @ _exact_weights(c, s["codes"], s["scales"], s["zeros"]).T}
    if c["op"] == "w4_quantize":
        return _exact_quantize(c, s)
    if c["op"] == "kv_append":
        return _exact_append(c, s)
    return _exact_attention(c, s)


def _exact_weights(c, codes, scales, zeros):
    N, K, G = c["N"], c["K"], c["group"]
    j = torch.arange(K, device="cuda")
    u = (codes[:, j // 2].int() >> (4 * (j % 2))[None].int()) & 15
    if c["fmt"] == "mxfp4":
        e, m = (u >> 1) & 3, (u & 1).double()
        mag = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
        return torch.where(u > 7, -mag, mag) * torch.exp2(scales[:, j // G].double() - 127)
    z = zeros[:, j // G].double() if c["zeros"] else 8.0
    return (u.double() - z) * scales[:, j // G].double()


def _exact_quantize(c, s):
    N, K, G = c["N"], c["K"], c["group"]
    w, parts, scales, zeros = s["w"].double(), [], [], []
    for k in range(0, K, G):
        x = w[:, k:k + G]
        if c["fmt"] == "mxfp4":
            a = x.abs().max(1, keepdim=True).values
            e = torch.where(a > 0, torch.floor(torch.log2(torch.where(a > 0, a, 1.0))) - 2, -127.0).clamp(min=-127)
            t, ulp = x / torch.exp2(e), torch.exp2(torch.floor(torch.log2((x / torch.exp2(e)).abs().clamp(min=1.0))) - 1)
            parts.append((torch.round(t / ulp) * ulp).clamp(-6, 6) * torch.exp2(e))
            scales.append((e + 127).to(torch.uint8))
            continue
        lo, hi = x.min(1, keepdim=True).values.clamp(max=0), x.max(1, keepdim=True).values.clamp(min=0)
        a = (hi - lo).float().double() / 15 if c["zeros"] else torch.maximum(-lo, hi) / 7
        sc = a.float().to(torch.bfloat16).double()
        sc = torch.where(((hi - lo) if c["zeros"] else torch.maximum(-lo, hi)) < 2.0 ** -100, 1.0, sc)
        z = torch.round((-lo / sc).float()).clamp(0, 15).double() if c["zeros"] else torch.full_like(sc, 8)
        u = (torch.round((x / sc).float()).double() + z).clamp(0, 15)
        parts.append((u - z) * sc)
        scales.append(sc)
        zeros.append(z.to(torch.uint8))
    return {"values": torch.cat(parts, 1), "scales": torch.cat(scales, 1), "zeros": torch.cat(zeros, 1) if c["zeros"] else None}


def _e4m3_values():
    """What the codes 0 to 126 stand for."""
    return [m / 512.0 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def _e4m3(codes):
    """Codes to values in 64 bits."""
    pos = torch.tensor(_e4m3_values() + [math.nan], dtype=torch.float64, device=codes.device)
    mag = pos[(codes & 127).long()]
    return torch.where(codes > 127, -mag, mag)


def _to_e4m3(x):
    """The value of the code nearest to x (at most 448 in size), ties to the even code."""
    pos = torch.tensor(_e4m3_values(), dtype=torch.float64, device=x.device)
    a = x.abs().contiguous()
    hi = torch.searchsorted(pos, a).clamp(1, 126)
    below, above = a - pos[hi - 1], pos[hi] - a
    mag = pos[torch.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)]
    return torch.copysign(mag, x)


def _exact_append(c, s):
    H, D, page, rot = c["H"], c["D"], c["page"], c["rot"]
    lens, start, table = s["lens"].tolist(), s["start"].tolist(), s["table"].tolist()
    got = {"k": _e4m3(s["k"]), "v": _e4m3(s["v"])}
    scale = {n: s[n + "_scale"].clone() for n in "kv"}
    cos, sin = s["cos"].double(), s["sin"].double()
    half = rot // 2
    first = [2 * j if c["interleaved"] else j for j in range(half)]
    second = [2 * j + 1 if c["interleaved"] else j + half for j in range(half)]

    def turned(x, at):
        y = x.double().clone()
        y[..., first] = x[..., first].double() * cos[at, None] - x[..., second].double() * sin[at, None]
        y[..., second] = x[..., second].double() * cos[at, None] + x[..., first].double() * sin[at, None]
        return y

    where = torch.cat([torch.arange(n - (start[b + 1] - start[b]), n) for b, n in enumerate(lens)]).cuda()
    rows = {"k": turned(s["xk"], where).float().double(), "v": s["xv"].double()}
    for b, n in enumerate(lens):
        p0 = n - (start[b + 1] - start[b])
        for pg in range(p0 // page, (n - 1) // page + 1):
            lo, hi, at = max(p0, pg * page), min(n, (pg + 1) * page), table[b][pg]
            for name in "kv":
                x = rows[name][start[b] + lo - p0:start[b] + hi - p0].transpose(0, 1)     # [H, tokens, D]
                a = x.abs().amax((1, 2))
                e = torch.ceil(torch.log2(torch.where(a > 0, a, 2.0 ** -200) / 448)).clamp(-100, 120)
                e_old = scale[name][at].double() - 127
                e = e if lo == pg * page else torch.maximum(e, e_old)
                block = got[name][at] if name == "k" else got[name][at].transpose(1, 2)
                ahead = lo - pg * page
                block[:, :ahead] = _to_e4m3(block[:, :ahead] * torch.exp2(e_old - e)[:, None, None])
                block[:, ahead:ahead + hi - lo] = _to_e4m3(x * torch.exp2(-e)[:, None, None])
                scale[name][at] = (e + 127).to(torch.uint8)
    return {"q": turned(s["q"], where), "k": got["k"], "v": got["v"], "k_scale": scale["k"], "v_scale": scale["v"]}


def _exact_attention(c, s):
    H, Hq, D, page = c["H"], c["Hq"], c["D"], c["page"]
    lens, start = s["lens"].tolist(), s["start"].tolist()
    o, lse = [], []
    for b, n in enumerate(lens):
        at = s["table"][b, :-(-n // page)].long()
        k = _e4m3(s["k"][at]) * torch.exp2(s["k_scale"][at].double() - 127)[..., None, None]
        v = _e4m3(s["v"][at]) * torch.exp2(s["v_scale"][at].double() - 127)[..., None, None]
        q = s["q"][start[b]:start[b + 1]].double()
        pos = torch.arange(n - q.shape[0], n, device="cuda")
        t = torch.arange(n, device="cuda")
        hidden = t[None] > pos[:, None]
        if c["window"]:
            hidden |= (t[None] <= pos[:, None] - c["window"]) & (t[None] >= c["sinks"])
        heads_o, heads_l = [], []
        for h in range(Hq):
            j = h // (Hq // H)
            keys = k[:, j].reshape(-1, D)[:n]
            vals = v[:, j].transpose(1, 2).reshape(-1, D)[:n]
            x = (q[:, h] @ keys.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            heads_l.append(torch.logsumexp(x, 1))
            heads_o.append(torch.softmax(x, 1) @ vals)
        o.append(torch.stack(heads_o, 1))
        lse.append(torch.stack(heads_l, 1))
    return {"o": torch.cat(o), "lse": torch.cat(lse)}
