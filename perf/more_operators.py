"""Cases of the block-scaled operators: the quantiser that gives a matrix one
scale for each block of 128, the root-mean-square norm with the residual's
addition, the product of two such matrices, and the gated pair of products.

`own` false: the operators in elementary torch operations; true: the same calls
through dense_tiled_gemm_fp8_amd.gemm355.

Buffers, as the library has them (K blocks of 128, the last of a row may be short):
  codes    uint8 E4M3 [rows][ld], ld = K rounded up to 16
  scales   fp32: rows with a scale of their own [K blocks][rows], rows that share
           one by 128 [ceil(rows / 128)][K blocks]
"""
import math

import torch

own = False

EPS = 1e-5
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def _quant(name, rows, K, block, src):
    return {"name": name, "op": "block_quantize", "rows": rows, "K": K, "block": block, "src": src}


def _norm(name, rows, K, src, residual, out):
    return {"name": name, "op": "rmsnorm", "rows": rows, "K": K, "src": src, "residual": residual, "out": out}


def _gemm(name, M, N, K, out):
    return {"name": name, "op": "block_gemm", "M": M, "N": N, "K": K, "out": out}


def _gated(name, M, N, K, act, out):
    return {"name": name, "op": "block_gated", "M": M, "N": N, "K": K, "act": act, "out": out}


def listed():
    return [
        # a layer's weights when a model is loaded: one scale a 128 x 128 block
        _quant("block_quantize-weights-8192x8192", 8192, 8192, 128, "bf16"),
        # a few rows of activations kept in 32 bits, last block short, odd row length
        _quant("block_quantize-rows-100x4001", 100, 4001, 1, "f32"),
        # one token between two layers: what a call costs at least
        _norm("rmsnorm-1x4096-8bit", 1, 4096, "bf16", True, "8bit"),
        # a prompt's rows, the residual stream read and written, codes for the next product
        _norm("rmsnorm-4096x8192-8bit", 4096, 8192, "bf16", True, "8bit"),
        # the final norm of a batch in 32 bits, no residual, a width that no vector divides
        _norm("rmsnorm-1000x777-bf16", 1000, 777, "f32", False, "bf16"),
        # one token through a wide matrix: the stream of codes counts
        _gemm("block_gemm-m1-16384x8192", 1, 16384, 8192, "bf16"),
        # some draft tokens, sizes that no tile divides, odd K, sums kept in 32 bits
        _gemm("block_gemm-m37-3000x777", 37, 3000, 777, "f32"),
        # a decode batch
        _gemm("block_gemm-m128-8192x8192", 128, 8192, 8192, "bf16"),
        # a long prompt: the matrix units count
        _gemm("block_gemm-m4096-8192x8192", 4096, 8192, 8192, "bf16"),
        # one token through both projections of a feed-forward block
        _gated("block_gated-m1-8192x4096", 1, 8192, 4096, "silu", "8bit"),
        # a decode batch, ragged, rows of bf16 out
        _gated("block_gated-m50-5000x4096", 50, 5000, 4096, "gelu", "bf16"),
        # a prompt, codes for the product that follows
        _gated("block_gated-m2048-8192x4096", 2048, 8192, 4096, "silu", "8bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("block_quantize", "rmsnorm", "block_gemm", "block_gemm", "block_gated"))
    whole = rng.random() < 0.6
    if op == "block_quantize":
        src = rng.choice(("bf16", "f32"))
        K = _log(rng, 64, 8192)
        K = -(-K // 128) * 128 if whole else K
        c = _quant("", _log(rng, 1, 8192 if src == "bf16" else 4096), K, rng.choice((1, 128)), src)
    elif op == "rmsnorm":
        K = _log(rng, 64, 8192)
        K = -(-K // 128) * 128 if whole else K
        c = _norm("", rng.choice((1, _log(rng, 2, 2048))), K, rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.7,
                  rng.choice(("8bit", "8bit", "bf16")))
    else:
        M = rng.choice((1, _log(rng, 2, 64), _log(rng, 64, 4096)))
        gated = op == "block_gated"
        N, K = _log(rng, 128, 8192 if gated else 16384), _log(rng, 128, 4096 if gated else 8192)
        if whole:
            N, K = -(-N // 128) * 128, -(-K // 128) * 128
        M = max(1, min(M, (2048 * 8192 * 4096 if gated else 4096 * 8192 * 8192) // (N * K)))
        if gated:
            c = _gated("", M, N, K, rng.choice(("silu", "silu", "gelu")), rng.choice(("8bit", "8bit", "bf16")))
        else:
            c = _gemm("", M, N, K, rng.choice(("bf16", "bf16", "f32")))
    del c["name"]
    return c


BYTES = {"8bit": 1, "bf16": 2, "f32": 4}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _blocks(n):
    return -(-n // 128)


def _packed(rows, K, block):
    """Bytes of a matrix of codes and its scales."""
    return rows * K + 4 * _blocks(K) * (rows if block == 1 else _blocks(rows))


def work(case):
    c = case
    if c["op"] == "block_quantize":
        n = c["rows"] * c["K"]
        return {"bytes": n * BYTES[c["src"]] + _packed(c["rows"], c["K"], c["block"]), "flops": 3 * n}
    if c["op"] == "rmsnorm":
        rows, K = c["rows"], c["K"]
        out = _packed(rows, K, 1) if c["out"] == "8bit" else rows * K * BYTES[c["out"]]
        return {"bytes": rows * K * BYTES[c["src"]] * (3 if c["residual"] else 1) + 2 * K + out, "flops": 7 * rows * K}
    M, N, K = c["M"], c["N"], c["K"]
    out = _packed(M, N, 1) if c["out"] == "8bit" else M * N * BYTES[c["out"]]
    two = 2 if c["op"] == "block_gated" else 1
    return {"bytes": _packed(M, K, 1) + two * _packed(N, K, 128) + out, "flops": 2 * two * M * N * K}


# ------------------------------------------------------------------ inputs

def _uneven(g, rows, K, size):
    """Values with channels of uneven size, as activations and weights have them."""
    x = torch.randn(rows, K, generator=g, device="cuda") * size
    return x * torch.exp(0.7 * torch.randn(1, K, generator=g, device="cuda"))


def _empty_codes(rows, K, block):
    codes = torch.zeros(rows, -(-K // 16) * 16, dtype=torch.uint8, device="cuda")
    shape = (_blocks(K), rows) if block == 1 else (_blocks(rows), _blocks(K))
    return codes, torch.zeros(shape, dtype=torch.float32, device="cuda")


def _held(x, block):
    """Codes and scales that stand for x: what a checkpoint or the step before has left."""
    rows, K = x.shape
    codes, scales = _empty_codes(rows, K, block)
    for k in range(_blocks(K)):
        part = x[:, k * 128:(k + 1) * 128]
        a = part.abs().amax(1, keepdim=True)
        if block == 128:
            a = torch.stack([t.amax() for t in a.split(128)])
            scales[:, k] = a / 448
            a = a.repeat_interleave(128)[:rows, None]
        else:
            scales[k] = a[:, 0] / 448
        codes[:, k * 128:k * 128 + part.shape[1]] = (part * (448 / a)).clamp(-448, 448).to(F8).view(torch.uint8)
    return codes, scales


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    K = c["K"]
    if c["op"] == "block_quantize":
        s["x"] = _uneven(g, c["rows"], K, 1.0 if c["block"] == 1 else 0.02).to(TYPES[c["src"]])
        s["q"], s["q_scale"] = _empty_codes(c["rows"], K, c["block"])
    elif c["op"] == "rmsnorm":
        t = TYPES[c["src"]]
        s["x"] = _uneven(g, c["rows"], K, 0.3).to(t)
        s["residual"] = _uneven(g, c["rows"], K, 2.0).to(t) if c["residual"] else None
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
        _out(c, s, c["rows"], K)
    else:
        s["x"], s["x_scale"] = _held(_uneven(g, c["M"], K, 1.0), 1)
        for name in ("w", "up") if c["op"] == "block_gated" else ("w",):
            w = torch.randn(c["N"], K, generator=g, device="cuda") * (1.5 / math.sqrt(K))
            s[name], s[name + "_scale"] = _held(w, 128)
            del w
        _out(c, s, c["M"], c["N"])
    if own:
        _handles(c, s)
    return s


def _out(c, s, rows, width):
    s["y"] = s["q"] = s["q_scale"] = None
    if c["out"] == "8bit":
        s["q"], s["q_scale"] = _empty_codes(rows, width, 1)
    else:
        s["y"] = torch.empty(rows, width, dtype=TYPES[c["out"]], device="cuda")


# ------------------------------------------------------------------ the framework's calls

def _handles(c, s):
    """Descriptors that a program makes once: of its matrices and of a step's buffers."""
    from dense_tiled_gemm_fp8_amd import gemm355 as lib
    s["lib"] = lib
    kinds = {"bf16": lib.SRC_BF16, "f32": lib.SRC_F32, "8bit": lib.SRC_BF16}
    K = c["K"]
    if c["op"] == "block_quantize":
        s["matrix"] = lib.make_block_matrix(c["rows"], K, s["q"], s["q_scale"], block_rows=c["block"])
        s["src"] = kinds[c["src"]]
        return
    rows, width = (c["rows"], K) if c["op"] == "rmsnorm" else (c["M"], c["N"])
    q = lib.make_block_matrix(rows, width, s["q"], s["q_scale"]) if c["out"] == "8bit" else None
    if c["op"] == "rmsnorm":
        t = kinds[c["src"]]
        s["args"] = lib.make_rmsnorm_args(rows, width, x=s["x"], x_type=t, residual=s["residual"], sum=s["sum"], r_type=t,
                                          weight=s["weight"], w_type=lib.SRC_BF16, eps=EPS, y=s["y"],
                                          y_type=kinds[c["out"]], q=q)
        return
    x = lib.make_block_matrix(rows, K, s["x"], s["x_scale"])
    w = lib.make_block_matrix(width, K, s["w"], s["w_scale"], block_rows=128)
    if c["op"] == "block_gemm":
        s["args"] = lib.make_block_gemm_args(x, w, y=s["y"], out=kinds[c["out"]])
    else:
        up = lib.make_block_matrix(width, K, s["up"], s["up_scale"], block_rows=128)
        s["args"] = lib.make_block_gated_args(x, w, up, act=lib.ACT_SILU if c["act"] == "silu" else lib.ACT_GELU_TANH,
                                              y=s["y"], out=kinds[c["out"]], q=q)


def _outputs(c, s, width):
    out = {}
    if c["op"] == "rmsnorm" and c["residual"]:
        out["sum"] = s["sum"]
    if s.get("q") is not None:
        out["q"], out["q_scale"] = s["q"][:, :width].view(F8), s["q_scale"]
    else:
        out["y"] = s["y"]
    return out


def _run_own(c, s):
    lib = s["lib"]
    if c["op"] == "block_quantize":
        lib.gemm355_block_quantize(s["x"], s["matrix"], src=s["src"])
        return _outputs(c, s, c["K"])
    if c["op"] == "rmsnorm":
        lib.gemm355_rmsnorm(s["args"])
        return _outputs(c, s, c["K"])
    if c["op"] == "block_gemm":
        lib.gemm355_block_gemm(s["args"])
    else:
        lib.gemm355_block_gated(s["args"])
    return _outputs(c, s, c["N"])


def run(state):
    c = state["c"]
    if own:
        return _run_own(c, state)
    if c["op"] == "block_quantize":
        _plain_quantize(state, state["x"].float(), c["block"])
        return _outputs(c, state, c["K"])
    if c["op"] == "rmsnorm":
        return _plain_norm(c, state)
    x = _values(state["x"], state["x_scale"], c["M"], c["K"], 1)
    y = torch.matmul(x, _values(state["w"], state["w_scale"], c["N"], c["K"], 128).t())
    if c["op"] == "block_gated":
        y = _act(c, y) * torch.matmul(x, _values(state["up"], state["up_scale"], c["N"], c["K"], 128).t())
    return _store(c, state, y)


# ------------------------------------------------------------------ plain forms

def _values(codes, scales, rows, K, block):
    """What codes and scales stand for, in 32 bits."""
    v = codes[:, :K].view(F8).float()
    per = scales.t() if block == 1 else scales.repeat_interleave(128, 0)[:rows]
    return v * per.repeat_interleave(128, 1)[:, :K]


def _act(c, g):
    if c["act"] == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_quantize(s, x, block):
    """Codes and scales of 32-bit x into the state's buffers."""
    rows, K = x.shape
    nb, nr = _blocks(K), _blocks(rows) if block == 128 else rows
    x = torch.nn.functional.pad(x, (0, nb * 128 - K, 0, nr * block - rows)).reshape(nr, block, nb, 128)
    a = x.abs().amax((1, 3), keepdim=True)
    none = a < 2.0 ** -100
    scale, inverse = torch.where(none, 1.0, a / 448), torch.where(none, 1.0, 448 / a)
    q = (x * inverse).clamp(-448, 448).to(F8).reshape(nr * block, nb * 128)[:rows, :K]
    s["q"][:, :K] = q.view(torch.uint8)
    scale = scale[:, 0, :, 0]
    s["q_scale"].copy_(scale.t() if block == 1 else scale)


def _store(c, s, y):
    if c["out"] == "8bit":
        _plain_quantize(s, y, 1)
    else:
        s["y"].copy_(y)
    return _outputs(c, s, y.shape[1])


def _plain_norm(c, s):
    h = s["x"].float()
    if c["residual"]:
        s["sum"].copy_(h + s["residual"].float())
        h = s["sum"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    return _store(c, s, y)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _e4m3_values():
    """What the codes 0 to 126 stand for."""
    return [m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]


def _decode(codes):
    table = torch.tensor(_e4m3_values() + [math.nan], dtype=torch.float64, device=codes.device)
    return torch.where(codes >= 128, -1.0, 1.0) * table[(codes & 127).long()]


def _nearest(x):
    """The value of the code nearest to x, ties to the even code."""
    size = x.abs().clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(size / step) * step).clamp(max=448), x)


def _exact_matrix(codes, scales, rows, K, block):
    v = _decode(codes[:, :K])
    j, i = torch.arange(K, device="cuda") // 128, torch.arange(rows, device="cuda")
    at = scales.double()[j][:, i].T if block == 1 else scales.double()[i // 128][:, j]
    return v * at


def _exact_codes(x, block):
    rows, K = x.shape
    q, scales = torch.empty_like(x), []
    for k in range(0, K, 128):
        part, column = x[:, k:k + 128], []
        for r in range(0, rows, 128) if block == 128 else (0,):
            t = part[r:r + 128] if block == 128 else part
            a = t.abs().max() if block == 128 else t.abs().max(1, keepdim=True).values
            scale = torch.where(a < 2.0 ** -100, 1.0, a / 448)
            q[r:r + t.shape[0], k:k + 128] = _nearest(t / scale)
            column.append(scale.reshape(-1))
        scales.append(torch.cat(column))
    return q, torch.stack(scales, 0 if block == 1 else 1)


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    out = {}
    if c["op"] == "block_quantize":
        out["q"], out["q_scale"] = _exact_codes(s["x"].double(), c["block"])
        return out
    if c["op"] == "rmsnorm":
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["residual"].double()).to(TYPES[c["src"]]).double()
            out["sum"] = h
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / c["K"] + EPS) * s["weight"].double()
    else:
        M, N, K = c["M"], c["N"], c["K"]
        x = _exact_matrix(s["x"], s["x_scale"], M, K, 1)
        y = x @ _exact_matrix(s["w"], s["w_scale"], N, K, 128).T
        if c["op"] == "block_gated":
            u = x @ _exact_matrix(s["up"], s["up_scale"], N, K, 128).T
            if c["act"] == "silu":
                y = y * torch.sigmoid(y) * u
            else:
                y = torch.nn.functional.gelu(y, approximate="tanh") * u
    if c["out"] == "8bit":
        out["q"], out["q_scale"] = _exact_codes(y, 1)
    else:
        out["y"] = y
    return out
