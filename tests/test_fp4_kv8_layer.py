"""The 4-bit linear layers and the int8 cache together, as a decoder layer runs them: a prompt, then single tokens.

Each step's result is checked against its definition in 64 bits on the inputs that the step before it produced.
"""
import math

import numpy as np
import pytest
import torch

import fp4_ref
import kv8_ref
import w8a8_post_quantization_sq_b200 as sq
from test_fp4 import check_gemm
from test_kv8 import check_attention

BF = torch.bfloat16


def weight(N, K, fmt, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((N, K), generator=g) * 0.05).to(BF).cuda()
    codes, scales, qs = sq.fp4_buffers(N, K, fmt)
    sq.sq_quantize_weight_fp4(w, None, fmt, codes, scales, qs)
    return codes, scales, qs


def values(t, rows, K, fmt):
    """What quantised operands stand for, fp64 on the GPU, from their bytes."""
    codes, scales, qs = t
    b = codes.cpu().numpy()
    c = np.stack([b & 15, b >> 4], 2).reshape(rows, K)
    blocks = K // fp4_ref.BLOCK[fmt]
    r, k = np.arange(rows)[:, None], np.arange(blocks)[None]
    at = (r // 128 * ((blocks + 3) // 4) + k // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + k % 4
    v = fp4_ref.values(c, scales.cpu().numpy()[at], fmt)
    return torch.from_numpy(v / (qs.cpu().double().numpy()[:, None] if qs is not None else 1.0)).cuda()


class Linear:
    def __init__(self, N, K, fmt, seed, rows):
        self.w, self.N, self.K, self.fmt = weight(N, K, fmt, seed), N, K, fmt
        self.wv = values(self.w, N, K, fmt)
        self.x = sq.fp4_buffers(rows, K, fmt)
        self.ws = sq.workspace(sq.SQ_OP_GEMM_FP4, rows, N, K)

    def __call__(self, x, check):
        M = x.shape[0]
        codes, scales, qs = self.x
        codes, qs = codes[:M], None if qs is None else qs[:M]
        sq.sq_quantize_act_fp4(x, None, self.fmt, True, None, codes, scales, qs)
        y = torch.empty((M, self.N), dtype=BF, device="cuda")
        sq.sq_gemm_fp4(codes, scales, self.w[0], self.w[1], self.fmt, qs, self.w[2], None, y, self.ws)
        if check:
            c, b, q = fp4_ref.quantise(x.double().cpu().numpy(), self.fmt)
            xv = values((codes, scales, qs), M, self.K, self.fmt)
            want = fp4_ref.values(c, b, self.fmt) / (q[:, None] if q is not None else 1.0)
            assert torch.equal(xv.cpu(), torch.from_numpy(want))
            check_gemm(y, xv, self.wv, None, self.K)
        return y


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [sq.SQ_NVFP4, sq.SQ_MXFP4])
def test_decoder_layer(fmt):
    hidden, hq, hkv, D, inner, bs = 512, 8, 2, 64, 768, 32
    lens = [150, 70, 3]
    T = sum(lens)
    qkv = Linear((hq + 2 * hkv) * D, hidden, fmt, 1, T)
    out = Linear(hidden, hq * D, fmt, 2, T)
    up = Linear(2 * inner, hidden, fmt, 3, T)
    down = Linear(hidden, inner, fmt, 4, T)
    gamma = (1 + 0.1 * torch.randn(hidden, generator=torch.Generator().manual_seed(5))).cuda()
    batch = kv8_ref.Batch(lens, lens, hkv, D, bs, seed=6, width=8)
    dev = batch.gpu()
    attn_ws = sq.workspace(sq.SQ_OP_KV8_ATTENTION, T, hq, D)

    def layer(h, check):
        n = h.shape[0]
        v = torch.empty_like(h)
        sq.sq_norm_smooth_quant(h, sq.SQ_RMSNORM, gamma, None, 1e-6, True, None, None, None, None, v)
        z = qkv(v, check)  # K and V go to the cache as slices of the projection's output
        q, k, vv = (z[:, a * D : b * D].unflatten(1, (b - a, D)) for a, b in
                    ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        sq.sq_kv8_append(k, vv, dev["cu"], dev["lens"], dev["table"], dev["k"], dev["v"], dev["kqs"], dev["vqs"])
        y = torch.empty((n, hq, D), dtype=BF, device="cuda")
        sq.sq_kv8_attention(q, dev["k"], dev["v"], dev["kqs"], dev["vqs"], dev["cu"], dev["lens"], dev["table"],
                            1 / math.sqrt(D), True, max(batch.new), y, attn_ws)
        if check:
            kv8_ref.append(batch, k.cpu().double().numpy(), vv.cpu().double().numpy())
            assert np.array_equal(dev["k"].cpu().numpy(), batch.k) and np.array_equal(dev["v"].cpu().numpy(), batch.v)
            check_attention(batch, q.cpu(), 1 / math.sqrt(D), y=y)
        h = h + out(y.flatten(1), check)
        sq.sq_norm_smooth_quant(h, sq.SQ_RMSNORM, gamma, None, 1e-6, True, None, None, None, None, v)
        a = up(v, check)
        m = torch.empty((n, inner), dtype=BF, device="cuda")
        sq.sq_act_quant(a, sq.SQ_ACT_SWIGLU, True, None, None, None, None, m)
        return h + down(m, check)

    x = torch.randn((T, hidden), generator=torch.Generator().manual_seed(7)).to(BF).cuda()
    h = layer(x, True)
    last = torch.tensor(np.cumsum(lens) - 1, device="cuda")
    x = h[last].contiguous()
    batch.new, batch.cu = [1] * 3, np.arange(4, dtype=np.int32)
    dev["cu"] = torch.arange(4, dtype=torch.int32, device="cuda")
    for step in range(4):
        batch.lens = [n + 1 + step for n in lens]
        dev["lens"] = torch.tensor(batch.lens, dtype=torch.int32, device="cuda")
        x = layer(x, True)
        assert bool(x.isfinite().all())
    sq.sq_workspace_status(attn_ws)


@pytest.mark.gpu
def test_two_streams():
    """Two layers at once, each with its own buffers and workspace, on streams of their own."""
    fmt, M, N, K = sq.SQ_NVFP4, 48, 640, 1024
    layers = [Linear(N, K, fmt, s, M) for s in (1, 2)]
    batches = [kv8_ref.Batch([1, 3, 90], [500, 40, 300], 2, 128, 16, seed=s) for s in (3, 4)]
    devs = [b.gpu() for b in batches]
    xs = [torch.randn((M, K), generator=torch.Generator().manual_seed(s)).to(BF).cuda() for s in (5, 6)]
    qs = [torch.randn((94, 8, 128), generator=torch.Generator().manual_seed(s)).to(BF).cuda() for s in (7, 8)]
    ws = [sq.workspace(sq.SQ_OP_KV8_ATTENTION, 94, 8, 128) for _ in range(2)]

    def run(i, y):
        for _ in range(5):
            z = layers[i](xs[i], False)
            d = devs[i]
            sq.sq_kv8_attention(qs[i], d["k"], d["v"], d["kqs"], d["vqs"], d["cu"], d["lens"], d["table"], 0.1, True, 90,
                                y, ws[i])
        return z, y

    alone = [run(i, torch.empty_like(qs[i])) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            both.append(run(i, torch.empty_like(qs[i])))
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
