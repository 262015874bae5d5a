"""The 4-bit linear layer and attention over an 8-bit cache: what one pass of each computes, and what it has to move.

Four operators, each beside the 8-bit form that the library has already:

quant   a matrix to microscaled 4-bit floating point (E2M1 codes, a scale for each block of 16 or 32 of a row) and
        back to the 16-bit values that the codes stand for
gemm    Y = A B^T of two such matrices, with a scale per row and column and a bias
append  new tokens' K and V into a paged int8 cache with one scale per block of tokens and head
attn    attention over that cache: single tokens, a few tokens for each sequence, and prompts

Formats ("nv": block 16, scale E4M3, and one power of two per row; "mx": block 32, scale E8M0). Block scales are held
in tiles of 128 rows x 4 blocks: the scale of row r, block c sits at byte (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4 of
tile (r // 128, c // 4), tiles of one row group back to back. Rows and blocks that fill up a tile hold zeros.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BLOCK = {"nv": 16, "mx": 32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # a decode batch's hidden states before a linear layer of the 6.7B shapes
        dict(name="quant_act_16x4096", op="quant", fmt="nv", M=16, K=4096, dt="bf16", what="act", smooth=False),
        # the prompt of the 175B-shaped block
        dict(name="quant_act_4096x12288", op="quant", fmt="nv", M=4096, K=12288, dt="bf16", what="act", smooth=False),
        # out projection of the 6.7B shapes for a decode batch of 16
        dict(name="gemm_16x4096x4096", op="gemm", fmt="nv", M=16, N=4096, K=4096, dt="bf16", bias=False),
        # odd sizes: rows, columns and blocks that end inside a tile
        dict(name="gemm_333x1001x1056", op="gemm", fmt="nv", M=333, N=1001, K=1056, dt="fp16", bias=True),
        # FC2 of the 30B shapes at 1024 tokens
        dict(name="gemm_mx_1024x7168x28672", op="gemm", fmt="mx", M=1024, N=7168, K=28672, dt="fp16", bias=True),
        # out projection of the 175B-shaped block
        dict(name="gemm_4096x12288x12288", op="gemm", fmt="nv", M=4096, N=12288, K=12288, dt="bf16", bias=False),
        # one new token for each of 64 sequences
        dict(name="append_64x1", op="append", B=64, new=1, ragged=False, ctx=1024, Hkv=8, D=128, block=16, dt="bf16"),
        # prompts of different lengths, 8192 tokens at most
        dict(name="append_4x2048", op="append", B=4, new=2048, ragged=True, ctx=2048, Hkv=8, D=128, block=16, dt="bf16"),
        # one sequence answers: the shortest call
        dict(name="attn_1x1_ctx1000", op="attn", B=1, new=1, ragged=False, ctx=1000, Hq=32, Hkv=8, D=128, block=16,
             dt="bf16"),
        # a full decode batch, sequences of different lengths up to 8192
        dict(name="attn_64x1_ctx8192", op="attn", B=64, new=1, ragged=True, ctx=8192, Hq=32, Hkv=8, D=128, block=16,
             dt="bf16"),
        # four drafted tokens of each sequence checked at once, one K/V head for each query head, narrow heads
        dict(name="attn_16x4_ctx4000", op="attn", B=16, new=4, ragged=True, ctx=4000, Hq=16, Hkv=16, D=64, block=32,
             dt="fp16"),
        # prompts
        dict(name="attn_2x2048_ctx4096", op="attn", B=2, new=2048, ragged=True, ctx=4096, Hq=32, Hkv=8, D=128, block=64,
             dt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "gemm", "append", "attn"))
    fmt = rng.choice(("nv", "mx"))
    if op == "quant":
        return dict(op=op, fmt=fmt, M=_log(rng, 1, 4096), K=32 * _log(rng, 2, 384), dt=rng.choice(("bf16", "fp16", "fp32")),
                    what=rng.choice(("act", "weight")), smooth=rng.random() < 0.5)
    if op == "gemm":
        return dict(op=op, fmt=fmt, M=_log(rng, 1, 2048), N=_log(rng, 8, 8192), K=32 * _log(rng, 2, 256),
                    dt=rng.choice(("bf16", "fp16")), bias=rng.random() < 0.5)
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    block = rng.choice((16, 32, 64, 128))
    dt = rng.choice(("bf16", "fp16"))
    new = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 16, 1024)))
    ctx = new + _log(rng, 1, 6000)
    B = max(1, min(_log(rng, 1, 128), 80000 // ctx, 6000 // new))
    c = dict(op=op, B=B, new=new, ragged=rng.random() < 0.7, ctx=ctx, Hkv=Hkv, D=D, block=block, dt=dt)
    if op == "attn":
        c["Hq"] = Hkv * rng.choice((1, 2, 4, 8))
        c["B"] = max(1, min(B, 500_000_000 // (new * ctx * c["Hq"])))
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _matrix(rows, K, g, what):
    """Hidden states with a few loud channels, or weights."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    if what == "act":
        loud = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 1000)]
        x[:, loud] *= 20.0
        return x
    return x.mul_(0.03)


def _lengths(case):
    """New tokens and length (after them) of each sequence, on the host: a case has the same ones whatever the seed."""
    g = torch.Generator().manual_seed(case["B"] + case["new"] + case["ctx"])
    B, new, ctx = case["B"], case["new"], case["ctx"]
    n = torch.full((B,), new)
    length = torch.full((B,), ctx)
    if case["ragged"]:
        n = torch.randint(max(1, new // 2), new + 1, (B,), generator=g)
        length = torch.maximum(n, torch.randint(max(1, ctx // 8), ctx + 1, (B,), generator=g))
    return n, length


def _cache(case, g):
    """Lengths, block table (blocks in any order) and a cache whose first tokens are there."""
    n, length = _lengths(case)
    B, bs, Hkv, D = case["B"], case["block"], case["Hkv"], case["D"]
    width = (case["ctx"] + bs - 1) // bs
    num = B * width + 3
    table = torch.randperm(num, generator=g, device="cuda")[: B * width].to(torch.int32).view(B, width)
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = n.cumsum(0)
    s = dict(cu=cu.cuda(), lens=length.to(torch.int32).cuda(), table=table, T=int(n.sum()))
    for name in ("k", "v"):
        code = torch.randn((num, Hkv, bs, D), generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127)
        s[name + "c"] = code.to(torch.int8)
        s[name + "qs"] = 127.0 / (3.0 + torch.rand((num, Hkv), generator=g, device="cuda"))
    return s


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], _DT[case["dt"]]
    if op == "quant":
        M, K = case["M"], case["K"]
        s = dict(x=_matrix(M, K, g, case["what"]).to(dt), s=None)
        if case["smooth"]:
            s["s"] = torch.rand(K, generator=g, device="cuda") + 0.5
        blocks = K // _BLOCK[case["fmt"]]
        s["codes"] = torch.empty((M, K // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((M + 127) // 128 * ((blocks + 3) // 4) * 512, dtype=torch.uint8, device="cuda")
        s["qs"] = torch.empty(M, device="cuda") if case["fmt"] == "nv" else None
        s["values"] = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s = {}
        for name, rows, what in (("x", M, "act"), ("w", N, "weight")):
            code, sb, qs = _to_fp4(_matrix(rows, K, g, what), case["fmt"])
            s[name] = code[:, 0::2] | (code[:, 1::2] << 4)
            s[name + "s"] = _tiled(sb, case["fmt"])
            s[name + "qs"] = qs
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["y"] = torch.empty((M, N), dtype=dt, device="cuda")
    else:
        s = _cache(case, g)
        T, Hkv, D = s["T"], case["Hkv"], case["D"]
        if op == "append":
            s["k"] = torch.randn((T, Hkv, D), generator=g, device="cuda").to(dt)
            s["v"] = torch.randn((T, Hkv, D), generator=g, device="cuda").to(dt)
        else:
            s["q"] = torch.randn((T, case["Hq"], D), generator=g, device="cuda").to(dt)
            s["y"] = torch.empty_like(s["q"])
    s["case"] = case
    return s


# ---------------------------------------------------------------- plain forms
def _pow2(field):
    """2^(field - 127) from the exponent field."""
    return (field.to(torch.int32) << 23).view(torch.float32)


def _field(x):
    """The exponent field of non-negative fp32 values."""
    return x.contiguous().view(torch.int32) >> 23


def _to_fp4(v, fmt):
    """fp32 [rows, K] -> (E2M1 codes [rows, K], block scales [rows, K / block] as values, power of two per row or None)."""
    rows, K = v.shape
    qs = None
    if fmt == "nv":
        qs = _pow2(264 - _field(v.abs().amax(1)).clamp(min=27))
        u = (v * qs[:, None]).view(rows, -1, 16)
        sb = (u.abs().amax(2) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        t = torch.where(sb[..., None] > 0, u / sb[..., None], torch.zeros_like(u))
    else:
        u = v.view(rows, -1, 32)
        field = (_field(u.abs().amax(2)) - 2).clamp(min=0)
        t = u * _pow2(254 - field)[..., None]
        sb = torch.ldexp(torch.ones_like(field, dtype=torch.float64), field - 127).float()
    a = t.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code |= (t < 0).to(torch.uint8) << 3
    return code.view(rows, K), sb, qs


def _tiled(sb, fmt):
    """Block scales [rows, blocks] as bytes in tiles of 128 rows x 4 blocks."""
    byte = sb.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "nv" else torch.frexp(sb)[1].add(126).to(torch.uint8)
    rows, blocks = byte.shape
    byte = torch.nn.functional.pad(byte, (0, -blocks % 4, 0, -rows % 128))
    byte = byte.view(byte.shape[0] // 128, 4, 32, byte.shape[1] // 4, 4)
    return byte.permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _values(packed, tiles, fmt):
    """What packed codes and tiled scales stand for, fp32 [rows, K]."""
    rows, K = packed.shape[0], packed.shape[1] * 2
    code = torch.stack((packed & 15, packed >> 4), 2).view(rows, K)
    value = torch.tensor(_E2M1, device="cuda")[code.int()]
    blocks = K // _BLOCK[fmt]
    byte = tiles.view((rows + 127) // 128, (blocks + 3) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    byte = byte.reshape((rows + 127) // 128 * 128, -1)[:rows, :blocks].contiguous()
    sb = byte.view(torch.float8_e4m3fn if fmt == "nv" else torch.float8_e8m0fnu).float()
    return (value.view(rows, blocks, -1) * sb[..., None]).view(rows, K)


def _plain_quant(s, case):
    v = s["x"].float()
    if s["s"] is not None:
        v = v * s["s"] if case["what"] == "weight" else v / s["s"]
    code, sb, qs = _to_fp4(v, case["fmt"])
    packed, tiles = code[:, 0::2] | (code[:, 1::2] << 4), _tiled(sb, case["fmt"])
    y = _values(packed, tiles, case["fmt"])
    if qs is not None:
        y = y / qs[:, None]
    return {"values": y.to(torch.bfloat16), "qs": qs}


def _plain_gemm(s, case):
    y = _values(s["x"], s["xs"], case["fmt"]) @ _values(s["w"], s["ws"], case["fmt"]).t()
    if s["xqs"] is not None:
        y = y / (s["xqs"][:, None] * s["wqs"])
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(_DT[case["dt"]])


def _tokens(s):
    """The sequence and the position in it of each new token, and the number of new tokens of each sequence."""
    n = s["cu"][1:] - s["cu"][:-1]
    sid = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["T"])
    pos = s["lens"][sid] - n[sid] + torch.arange(s["T"], device="cuda") - s["cu"][sid]
    return sid, pos, n


def _plain_append(s, case):
    bs = case["block"]
    sid, pos, n = _tokens(s)
    blk, off = s["table"][sid, pos // bs].long(), pos % bs
    start = s["lens"] - n
    # each sequence's first new token may enter a block that holds tokens already
    first = s["table"][torch.arange(n.numel(), device="cuda"), torch.where(n > 0, start // bs, 0)].long()
    kept = torch.where(n > 0, start % bs, 0)
    for new, codes, qs in ((s["k"], s["kc"], s["kqs"]), (s["v"], s["vc"], s["vqs"])):
        x = new.float()
        peak = torch.zeros_like(qs).scatter_reduce_(0, blk[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
        now = 127.0 / peak.clamp(min=1e-8)
        before = qs[first]
        after = torch.where(kept[:, None] > 0, torch.minimum(before, now[first]), now[first])
        after = torch.where(n[:, None] > 0, after, before)
        ratio = torch.where(after < before, after / before, 1.0)
        old = codes[first]
        mask = torch.arange(bs, device="cuda") < kept[:, None]
        scaled = (old.float() * ratio[:, :, None, None]).round().clamp(-127, 127).to(torch.int8)
        codes[first] = torch.where(mask[:, None, :, None], scaled, old)
        now[first] = after
        qs[blk] = now[blk]
        codes[blk, :, off] = (x * now[blk][..., None]).round().clamp(-127, 127).to(torch.int8)
    return {"k": s["kc"], "v": s["vc"], "kqs": s["kqs"], "vqs": s["vqs"]}


def _plain_attn(s, case):
    B, Hq, Hkv, D, L = case["B"], case["Hq"], case["Hkv"], case["D"], s["table"].shape[1] * case["block"]
    sid, pos, n = _tokens(s)
    table = s["table"].long()
    k = (s["kc"][table] / s["kqs"][table][..., None, None]).transpose(1, 2).reshape(B, Hkv, L, D)
    v = (s["vc"][table] / s["vqs"][table][..., None, None]).transpose(1, 2).reshape(B, Hkv, L, D)
    at = s["cu"][:-1, None] + torch.arange(case["new"], device="cuda")
    q = s["q"].float()[at.clamp(max=s["T"] - 1)]  # [B, new, Hq, D], rows past a sequence's end unused
    q = q.view(B, -1, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (q @ k.transpose(2, 3)).view(B, Hkv, Hq // Hkv, -1, L) * (1.0 / math.sqrt(D))
    seen = s["lens"][:, None] - n[:, None] + torch.arange(case["new"], device="cuda") + 1
    score.masked_fill_((torch.arange(L, device="cuda") >= seen[..., None])[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, Hkv, -1, L)
    y = (p @ v).view(B, Hkv, Hq // Hkv, -1, D).permute(0, 3, 1, 2, 4).reshape(B, -1, Hq, D)
    return y[sid, torch.arange(s["T"], device="cuda") - s["cu"][sid]].to(_DT[case["dt"]])


# ---------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"quant": _plain_quant, "gemm": _plain_gemm, "append": _plain_append, "attn": _plain_attn}[op](s, case)
    import w8a8_post_quantization_sq_b200 as sq

    if op in ("quant", "gemm"):
        fmt = sq.SQ_NVFP4 if case["fmt"] == "nv" else sq.SQ_MXFP4
    if op == "quant":
        if case["what"] == "act":
            sq.sq_quantize_act_fp4(s["x"], s["s"], fmt, True, None, s["codes"], s["scales"], s["qs"])
        else:
            sq.sq_quantize_weight_fp4(s["x"], s["s"], fmt, s["codes"], s["scales"], s["qs"])
        sq.sq_dequantize_fp4(s["codes"], s["scales"], fmt, s["qs"], s["values"])
        return {"values": s["values"], "qs": s["qs"]}
    if op == "append":
        sq.sq_kv8_append(s["k"], s["v"], s["cu"], s["lens"], s["table"], s["kc"], s["vc"], s["kqs"], s["vqs"])
        return {"k": s["kc"], "v": s["vc"], "kqs": s["kqs"], "vqs": s["vqs"]}
    if "work" not in s:  # a workspace, kept by a program from its first call on
        sizes = (case["M"], case["N"], case["K"]) if op == "gemm" else (s["T"], case["Hq"], case["D"])
        s["work"] = sq.workspace(sq.SQ_OP_GEMM_FP4 if op == "gemm" else sq.SQ_OP_KV8_ATTENTION, *sizes)
    if op == "gemm":
        sq.sq_gemm_fp4(s["x"], s["xs"], s["w"], s["ws"], fmt, s["xqs"], s["wqs"], s["bias"], s["y"], s["work"])
    else:
        sq.sq_kv8_attention(s["q"], s["kc"], s["vc"], s["kqs"], s["vqs"], s["cu"], s["lens"], s["table"],
                            1.0 / math.sqrt(case["D"]), True, case["new"], s["y"], s["work"])
    return s["y"]


def _visible(case):
    """Query rows x keys that attention of the batch sees, the keys of all its sequences, and the new tokens."""
    n, length = _lengths(case)
    return int((n * length - n * (n - 1) // 2).sum()), int(length.sum()), int(n.sum())


def work(case):
    op = case["op"]
    if op == "quant":
        M, K, eb = case["M"], case["K"], 4 if case["dt"] == "fp32" else 2
        held = M * K // 2 + M * K // _BLOCK[case["fmt"]]
        return {"bytes": M * K * eb + held + 2 * M * K + (4 * M if case["fmt"] == "nv" else 0), "flops": 3 * M * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        held = (M + N) * K // 2 + (M + N) * K // _BLOCK[case["fmt"]]
        return {"bytes": held + 2 * M * N + 4 * (M + N), "flops": 2 * M * N * K}
    pairs, keys, tokens = _visible(case)
    if op == "append":
        scales = 8 * case["Hkv"] * (tokens // case["block"] + case["B"])
        return {"bytes": 2 * tokens * case["Hkv"] * case["D"] * 3 + scales, "flops": 6 * tokens * case["Hkv"] * case["D"]}
    bs, Hq, Hkv, D = case["block"], case["Hq"], case["Hkv"], case["D"]
    return {"bytes": keys * Hkv * 2 * D + keys // bs * Hkv * 8 + 4 * tokens * Hq * D, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- in 64 bits
def _exact_fp4(x, fmt):
    """Values of the codes nearest to x / scale, in 64 bits, and the power of two per row."""
    amax = x.abs().amax(1)
    ex = torch.where(amax > 0, torch.frexp(amax)[1], -99).clamp(min=-99)
    one = torch.ones((), dtype=torch.float64, device="cuda")
    row = torch.ldexp(one, 11 - ex) if fmt == "nv" else torch.ones_like(amax)
    u = (x * row[:, None]).unflatten(1, (-1, _BLOCK[fmt]))
    top = u.abs().amax(2)
    if fmt == "nv":
        # nearest multiple of the E4M3 step at this size, ties to even
        step = torch.ldexp(one, torch.frexp(top / 6)[1].clamp(min=-5) - 4)
        sb = torch.round(top / 6 / step) * step
    else:
        sb = torch.ldexp(one, (torch.frexp(top)[1] - 3).clamp(min=-127))
    t = torch.where(sb[..., None] > 0, u / sb[..., None], 0.0)
    step = torch.ldexp(one, torch.frexp(t)[1].clamp(min=1) - 2)
    y = (torch.round(t / step) * step).clamp(-6, 6) * sb[..., None]
    return y.flatten(1) / row[:, None], row.float() if fmt == "nv" else None


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = s["x"].double()
        if s["s"] is not None:
            x = x * s["s"].double() if case["what"] == "weight" else x / s["s"].double()
        y, row = _exact_fp4(x, case["fmt"])
        return {"values": y, "qs": row}
    if op == "gemm":
        sides = []
        for name in ("x", "w"):
            rows, half = s[name].shape
            c = torch.arange(2 * half // _BLOCK[case["fmt"]], device="cuda")
            r = torch.arange(rows, device="cuda")[:, None]
            at = (r // 128 * ((c.numel() + 3) // 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4
            b = s[name + "s"][at].double()
            if case["fmt"] == "nv":
                low, e = b % 8, b // 8
                sb = torch.where(e > 0, (8 + low) * 2.0 ** (e - 10), low * 2.0**-9)
            else:
                sb = 2.0 ** (b - 127)
            two = torch.stack((s[name] % 16, s[name] // 16), 2).flatten(1).double()
            mag = two % 8
            mag = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
            y = torch.where(two < 8, mag, -mag) * sb.repeat_interleave(_BLOCK[case["fmt"]], 1)
            sides.append(y if s[name + "qs"] is None else y / s[name + "qs"].double()[:, None])
        y = sides[0] @ sides[1].T
        return y if s["bias"] is None else y + s["bias"].double()
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    bs = case["block"]
    if op == "append":
        out = {"k": None, "v": None}
        for name in ("k", "v"):
            new, qs = s[name].double(), s[name + "qs"].double()
            for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
                at = lens[b] - (hi - lo)
                while lo < hi:
                    take = min(hi - lo, bs - at % bs)
                    one = 127 / new[lo : lo + take].abs().amax((0, 2)).clamp(min=1e-8)
                    row = table[b][at // bs]
                    qs[row] = torch.minimum(qs[row], one) if at % bs else one
                    lo, at = lo + take, at + take
            out[name + "qs"] = qs
        return out
    group = case["Hq"] // case["Hkv"]
    y = torch.zeros_like(s["q"], dtype=torch.float64)
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        rows = torch.tensor(table[b][: (lens[b] + bs - 1) // bs], device="cuda")
        k, v = ((s[c][rows].double() / s[c[0] + "qs"][rows].double()[..., None, None]).transpose(0, 1).flatten(1, 2)
                for c in ("kc", "vc"))
        late = torch.arange(lens[b], device="cuda") > lens[b] - (hi - lo) + torch.arange(hi - lo, device="cuda")[:, None]
        for h in range(case["Hq"]):
            sc = s["q"][lo:hi, h].double() @ k[h // group, : lens[b]].T / math.sqrt(case["D"])
            y[lo:hi, h] = torch.softmax(sc.masked_fill(late, -math.inf), 1) @ v[h // group, : lens[b]]
    return y
