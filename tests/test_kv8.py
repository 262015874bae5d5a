"""The paged int8 K/V cache: appending and attention against their definition in 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv8_ref as ref
import w8a8_post_quantization_sq_b200 as sq

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def L():
    from w8a8_post_quantization_sq_b200 import build

    build.build()
    return sq.lib()


def rows16(T, heads, D, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, heads, D), generator=g) * scale).to(dt)


# ---------------------------------------------------------------- without a GPU
def test_refusals(L):
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)

    def expect(status, code, text):
        assert status == code and text in L.sq_last_error_string().decode(), L.sq_last_error_string()

    ok = [p, p, 2, 4, 2, 64, 128, 128, p, p, 1, p, 4, 4, p, p, p, p, 8, 16, None]
    for at, v, code, text in [(2, 0, 1, "dtype"), (3, -1, 2, "need"), (4, 0, 2, "need"), (5, 96, 2, "head width"),
                              (19, 24, 2, "block must"), (6, 64, 2, "strides"), (6, 132, 3, "aligned"),
                              (0, None, 1, "null"), (8, None, 1, "null"), (14, odd, 3, "aligned"), (12, 0, 2, "need"),
                              (13, 3, 2, "table stride"), (18, 0, 2, "need"), (12, 1 << 28, 2, "table stride"),
                              (10, -1, 2, "need")]:
        bad = list(ok)
        bad[at] = v
        expect(L.sq_kv8_append(*bad), code, text)
    bad = list(ok)
    bad[12] = bad[13] = 1 << 28
    expect(L.sq_kv8_append(*bad), 2, "2^31")
    for at in (3, 10):  # no tokens, no sequences
        none = list(ok)
        none[at] = 0
        none[0] = None
        assert L.sq_kv8_append(*none) == 0
    big = 1 << 24
    ok = [p, 2, 4, 8, 2, 64, 512, p, p, p, p, 8, 16, p, p, 1, p, 4, 4, 0.125, 1, 4, p, 512, p, big, None]
    for at, v, code, text in [(1, 0, 1, "dtype"), (3, 7, 2, "multiple of Hkv"), (5, 32, 2, "head width"),
                              (12, 8, 2, "block must"), (6, 256, 2, "strides"), (6, 516, 3, "aligned"),
                              (0, None, 1, "null"), (2, 1 << 28, 2, "2^31"), (22, None, 1, "null"), (16, None, 1, "null"), (21, -1, 1, "max_q"),
                              (24, None, 1, "workspace"), (25, 256, 1, "workspace"), (7, odd, 3, "aligned"),
                              (23, 8, 2, "strides")]:
        bad = list(ok)
        bad[at] = v
        expect(L.sq_kv8_attention(*bad), code, text)
    for at in (2, 15):
        none = list(ok)
        none[at] = 0
        none[0] = None
        assert L.sq_kv8_attention(*none) == 0


def test_binding_refusals():
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.int8)
    s = torch.ones((4, 2))
    cu, lens, tab = (torch.zeros(n, dtype=torch.int32) for n in (2, 1, 2))
    x = torch.zeros((3, 2, 64), dtype=BF)
    with pytest.raises(ValueError, match="block_table"):
        sq.sq_kv8_append(x, x, cu, lens, tab, kc, kc, s, s)
    with pytest.raises(ValueError, match="kqs"):
        sq.sq_kv8_append(x, x, cu, lens, tab.view(1, 2), kc, kc, s[:2], s)
    with pytest.raises(ValueError, match="int8"):
        sq.sq_kv8_append(x, x, cu, lens, tab.view(1, 2), kc.float(), kc, s, s)


def test_reference_against_plain_softmax():
    """The 64-bit attention of the tests against a direct double loop."""
    b = ref.Batch([2, 1], [5, 20], 1, 64, 16, seed=1)
    q = rows16(3, 2, 64, FP, 2).double()
    y, _ = ref.attention(b, q, 0.125)
    t = 0
    for s in range(2):
        for i in range(b.new[s]):
            vis = b.lens[s] - b.new[s] + i + 1
            for h in range(2):
                num, den = np.zeros(64), 0.0
                for j in range(vis):
                    blk, o = b.table[s, j // 16], j % 16
                    k, v = b.k[blk, 0, o] / b.kqs[blk, 0], b.v[blk, 0, o] / b.vqs[blk, 0]
                    e = math.exp(0.125 * float(q[t, h].numpy() @ k))
                    num, den = num + e * v, den + e
                assert np.allclose(y[t, h].numpy(), num / den, rtol=1e-12, atol=1e-12)
            t += 1


# ---------------------------------------------------------------- append
def check_append(batch, k, v, dev, ldk=0):
    T, H, D = k.shape

    def strided(x):
        base = torch.full((T, H * D + ldk), 5.0, dtype=x.dtype, device="cuda")
        base[:, : H * D] = x.cuda().reshape(T, H * D)
        return base[:, : H * D].unflatten(1, (H, D))

    sq.sq_kv8_append(strided(k), strided(v), dev["cu"], dev["lens"], dev["table"], dev["k"], dev["v"], dev["kqs"],
                     dev["vqs"])
    ref.append(batch, k.double().numpy(), v.double().numpy())
    for c, s, gc, gs in ((batch.k, batch.kqs, dev["k"], dev["kqs"]), (batch.v, batch.vqs, dev["v"], dev["vqs"])):
        gs = gs.cpu().double().numpy()
        assert np.array_equal(gs, s, equal_nan=True)
        good = ~np.isnan(s)
        assert np.array_equal(gc.cpu().numpy()[good], c[good])  # untouched blocks among them


APPEND = [
    # new, lens, block
    ([1], [1], 16), ([1], [17], 16), ([5], [21], 16), ([16], [16], 16), ([33], [40], 16), ([1, 1, 1], [16, 33, 100], 32),
    ([0, 3, 0, 70], [9, 3, 0, 90], 64), ([200, 1, 31], [200, 128, 160], 128), ([1] * 70, list(range(1, 71)), 16),
    ([300, 280], [300, 500], 16), ([2] * 40, [50] * 40, 64), ([64, 1, 1, 1, 1], [64, 5, 6, 7, 8], 16),
    ([600], [700], 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt,D,heads", [(BF, 128, 2), (FP, 64, 3), (FP, 128, 1), (BF, 64, 8)])
@pytest.mark.parametrize("new,lens,block", APPEND)
def test_append(new, lens, block, dt, D, heads):
    batch = ref.Batch(new, lens, heads, D, block, seed=len(new) + block)
    dev = batch.gpu()
    # large enough that kept codes are rescaled in some blocks and not in others
    check_append(batch, rows16(batch.T, heads, D, dt, 1, 1.2), rows16(batch.T, heads, D, dt, 2, 0.8), dev, 64)


@pytest.mark.gpu
def test_append_steps():
    """Token by token, growing values: a block is rescaled many times; then a second prompt in recycled blocks."""
    H, D, bs = 2, 128, 16
    batch = ref.Batch([1, 1], [1, 6], H, D, bs, seed=3, width=4)
    dev = batch.gpu()
    for step in range(40):
        batch.lens = [1 + step, 6 + step]
        dev["lens"] = torch.tensor(batch.lens, dtype=torch.int32, device="cuda")
        amp = 0.1 * (step + 1) if step % 3 else 0.05
        check_append(batch, rows16(2, H, D, BF, step, amp), rows16(2, H, D, BF, 100 + step, 1 / (step + 1)), dev)
    batch.new, batch.lens = [20, 9], [20, 9]
    batch.cu = np.array([0, 20, 29], np.int32)
    dev["cu"], dev["lens"] = torch.from_numpy(batch.cu).cuda(), torch.tensor([20, 9], dtype=torch.int32, device="cuda")
    check_append(batch, rows16(29, H, D, BF, 7, 1e-3), rows16(29, H, D, BF, 8, 1e-3), dev)


@pytest.mark.gpu
def test_append_edge_values():
    """Zeros, subnormals, the largest values, NaN and infinity (each in a block of its own)."""
    for dt in (BF, FP):
        H, D, bs = 1, 64, 16
        batch = ref.Batch([96, 3], [96, 20], H, D, bs, seed=4)
        dev = batch.gpu()
        k = rows16(99, H, D, dt, 5)
        k[:16] = 0
        k[16:32] *= torch.finfo(dt).tiny
        k[32:48] = torch.finfo(dt).max
        k[50, 0, 3] = float("nan")
        k[70, 0, 3] = float("inf")
        check_append(batch, k, rows16(99, H, D, dt, 6), dev)
        # the scale of a block stays NaN until the block is started anew
        batch.new, batch.lens, batch.cu = [1, 0], [56, 20], np.array([0, 1, 1], np.int32)
        dev["cu"], dev["lens"] = torch.from_numpy(batch.cu).cuda(), torch.tensor([56, 20], dtype=torch.int32).cuda()
        check_append(batch, rows16(1, H, D, dt, 9), rows16(1, H, D, dt, 9), dev)


@pytest.mark.gpu
def test_append_leaves_the_rest():
    """Tokens behind the last sequence, positions past the table, and blocks outside the cache are not written."""
    H, D, bs = 2, 64, 16
    batch = ref.Batch([2, 4, 1], [18, 20, 5], H, D, bs, seed=5, width=2)
    dev = batch.gpu()
    before = {n: dev[n].clone() for n in ("k", "v", "kqs", "vqs")}
    x = rows16(12, H, D, BF, 1).cuda()
    dev["lens"] = torch.tensor([34, 40, 0], dtype=torch.int32).cuda()  # past the table, past it, shorter than its tokens
    sq.sq_kv8_append(x, x, dev["cu"], dev["lens"], dev["table"], dev["k"], dev["v"], dev["kqs"], dev["vqs"])
    dev["lens"] = torch.tensor([18, 20, 5], dtype=torch.int32).cuda()
    dev["table"] = torch.tensor([[0, -1], [0, batch.num], [-5, 0]], dtype=torch.int32).cuda()
    sq.sq_kv8_append(x, x, dev["cu"], dev["lens"], dev["table"], dev["k"], dev["v"], dev["kqs"], dev["vqs"])
    assert all(torch.equal(before[n], dev[n]) for n in before)


# ---------------------------------------------------------------- attention
def run_attention(batch, q, scale, causal, dev=None, max_q=None, ws=None, pad=0):
    dev = dev or batch.gpu()
    T, H, D = q.shape

    def strided(fill):
        base = torch.full((T, H * D + pad), fill, dtype=q.dtype, device="cuda")
        return base, base[:, : H * D].unflatten(1, (H, D))

    _, qs = strided(3.0)
    qs.copy_(q)
    base, y = strided(-7.0)
    ws = sq.workspace(sq.SQ_OP_KV8_ATTENTION, T, H, D) if ws is None else ws
    sq.sq_kv8_attention(qs, dev["k"], dev["v"], dev["kqs"], dev["vqs"], dev["cu"], dev["lens"], dev["table"], scale,
                        causal, max(batch.new) if max_q is None else max_q, y, ws)
    sq.sq_workspace_status(ws)
    if pad:
        assert bool((base[:, H * D :] == -7).all())
    return y


def check_attention(batch, q, scale=None, causal=True, y=None, **kw):
    """Against 64 bits. Half a step of the output type of |y|, and of the sum over keys of weight x |value| (mass):
    the softmax weights' rounding to fp16 (2^-11), the scores' error and fp32 sums. A score of magnitude S (log2)
    has an fp32 error of at most (D + 8) 2^-24 of its |q||k| mass: with the sizes here (mass below 2^7) under 2^-10;
    its exponential and the sum of weights double that. In all 2^-11 + 2 * 2^-10 + 2^-11 < 3.1e-3 of mass."""
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    if y is None:
        y = run_attention(batch, q, scale, causal, **kw)
    want, mass = ref.attention(batch, q.double().cuda(), scale, causal)
    half = 2.0**-8 if q.dtype == BF else 2.0**-11
    T = batch.T
    err = (y[:T].double() - want[:T]).abs()
    tol = half * want[:T].abs() + 3.1e-3 * mass[:T] + 2.0**-25
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-30)).max())


ATTN = [
    # new, lens, block, Hkv, group, D
    ([1], [1], 16, 1, 1, 64), ([1], [1000], 16, 8, 4, 128), ([1, 1, 1], [16, 17, 15], 16, 2, 8, 128),
    ([1], [63], 32, 1, 16, 64), ([1, 1], [64, 65], 64, 3, 5, 128), ([1], [129], 128, 1, 7, 64),
    ([4, 4], [300, 77], 32, 2, 4, 64), ([1, 0, 3], [40, 9, 3], 16, 2, 2, 128), ([7], [7], 16, 1, 3, 128),
    ([40], [64], 16, 2, 1, 64), ([129, 1, 17], [129, 700, 300], 64, 2, 4, 128), ([1] * 33, [5 * i + 1 for i in range(33)], 16, 1, 8, 64),
    ([1, 1], [5000, 3], 16, 1, 2, 128), ([1], [3000], 128, 2, 32, 64), ([300], [1500], 16, 1, 2, 128),
    # prompts (many rows per K/V head), among shorter sequences
    ([700, 3, 257, 1], [1500, 300, 257, 90], 64, 2, 4, 128), ([64], [64], 16, 1, 1, 64), ([65], [193], 32, 2, 1, 64),
    ([513, 128], [600, 128], 16, 1, 3, 128), ([1000], [1000], 128, 3, 1, 64), ([9, 2], [400, 2], 32, 1, 32, 128),
    ([256, 0, 255, 1025], [257, 0, 2000, 1100], 16, 1, 2, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("new,lens,block,hkv,group,D", ATTN)
def test_attention(new, lens, block, hkv, group, D, dt):
    batch = ref.Batch(new, lens, hkv, D, block, seed=sum(lens))
    check_attention(batch, rows16(batch.T, hkv * group, D, dt, 1), pad=8 * (block == 16))


@pytest.mark.gpu
@pytest.mark.parametrize("new,lens,block,hkv,group,D", [ATTN[1], ATTN[6], ATTN[10], ATTN[15], ATTN[21]])
def test_attention_not_causal(new, lens, block, hkv, group, D):
    batch = ref.Batch(new, lens, hkv, D, block, seed=sum(lens))
    check_attention(batch, rows16(batch.T, hkv * group, D, BF, 1), causal=False)


@pytest.mark.gpu
def test_attention_rows_without_keys():
    """Sequences of length zero, and more new tokens than the length holds: those rows are zero."""
    batch = ref.Batch([2, 1, 5, 20], [10, 0, 3, 7], 2, 128, 16, seed=1)
    q = rows16(batch.T, 4, 128, BF, 1)
    y = run_attention(batch, q, 0.09, True)
    check_attention(batch, q, 0.09, y=y)
    assert bool((y[2] == 0).all() and (y[3:5] == 0).all() and (y[8:21] == 0).all())
    batch = ref.Batch([1, 3], [0, 0], 1, 64, 16, seed=1)
    assert bool((run_attention(batch, rows16(4, 2, 64, FP, 1), 0.1, False) == 0).all())


@pytest.mark.gpu
def test_prompt_rows_without_keys():
    """The same for sequences of many rows."""
    batch = ref.Batch([2, 1, 50, 200, 90], [10, 0, 30, 70, 0], 2, 128, 16, seed=1)
    q = rows16(batch.T, 8, 128, BF, 1)
    y = run_attention(batch, q, 0.09, True)
    check_attention(batch, q, 0.09, y=y)
    assert bool((y[2:23] == 0).all() and (y[53:183] == 0).all() and (y[253:343] == 0).all())
    check_attention(batch, q, 0.09, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_attention_any_scale(scale):
    """Scale zero (equal weights), negative, and large."""
    batch = ref.Batch([1, 100], [90, 150], 2, 64, 16, seed=3)
    check_attention(batch, rows16(101, 4, 64, FP, 2, 0.2), scale)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1e-6, 1e5])
def test_attention_scales_far_apart(spread):
    """Blocks whose V (and K) scales differ by many orders of magnitude; a block of zeros."""
    batch = ref.Batch([1, 40], [400, 300], 2, 128, 16, seed=2)
    g = np.random.default_rng(0)
    batch.vqs = ref.f32(batch.vqs * spread ** g.uniform(-1, 1, batch.vqs.shape))
    blk = batch.table[0, 3]
    batch.k[blk] = batch.v[blk] = 0
    batch.kqs[blk] = batch.vqs[blk] = ref.f32(127 / 1e-8)
    check_attention(batch, rows16(41, 8, 128, BF, 3))


@pytest.mark.gpu
def test_attention_peaked_and_shifted_scores():
    """Scores far from zero, growing along the sequence (the running maximum moves all the time) or falling."""
    for sign, new in ((1.0, [1, 3]), (-1.0, [1, 3]), (1.0, [150, 130]), (-1.0, [150, 130])):
        batch = ref.Batch(new, [600, 200], 1, 64, 16, seed=4)
        for b in range(2):
            for j, blk in enumerate(batch.table[b]):
                batch.k[blk, :, :, 0] = 100
                batch.kqs[blk] = ref.f32(100.0 / (j + 1))
                batch.k[blk, :, :, 1:] = np.clip(batch.k[blk, :, :, 1:] // 32, -1, 1)
        q = rows16(batch.T, 4, 64, BF, 5, 0.25)
        q[:, :, 0] = sign * 4.0
        check_attention(batch, q, 0.5)


@pytest.mark.gpu
def test_attention_small_and_large_queries():
    batch = ref.Batch([1, 4], [100, 50], 2, 64, 16, seed=6)
    for amp in (1e-30, 1e-6, 1e4):
        q = rows16(5, 4, 64, BF, 7, amp)
        check_attention(batch, q, 0.125 / max(amp, 1e-9))
    q = rows16(5, 4, 64, BF, 7)
    q[1] = 0  # equal weights
    check_attention(batch, q)


@pytest.mark.gpu
def test_attention_bad_values_stay_where_they_are_read():
    """NaN scales and missing blocks make NaN of the rows that read them, and of no others; what lies behind a
    sequence's end (any codes, NaN scales, numbers outside the cache) is not read."""
    H, D, bs = 2, 128, 16
    batch = ref.Batch([3, 1, 1, 2], [40, 50, 20, 18], H, D, bs, seed=7, width=6)
    batch.kqs[batch.table[0, 3:]] = np.nan
    batch.vqs[batch.table[0, 3:]] = np.nan
    batch.table[2, 2:] = [-1, 1 << 30, -(1 << 31), batch.num]
    q = rows16(7, 4, D, BF, 8)
    dev = batch.gpu()
    clean = run_attention(batch, q, 0.1, True, dev=dev)
    check_attention(batch, q, 0.1, y=clean)
    dev["kqs"][batch.table[1, 1], 0] = float("nan")  # sequence 1, head 0
    dev["table"][3, 1] = -1  # the second block of sequence 3: positions 16, 17
    y = run_attention(batch, q, 0.1, True, dev=dev)
    bad = torch.zeros((7, 4, D), dtype=torch.bool)
    bad[3, :2] = True
    bad[5:7] = True
    assert torch.equal(y.isnan().cpu(), bad)
    assert torch.equal(y[~bad.cuda()], clean[~bad.cuda()])
    q[4, 1, 5] = float("nan")
    bad[4, 1] = True
    y = run_attention(batch, q, 0.1, True, dev=dev)
    assert torch.equal(y.isnan().cpu(), bad)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_bad_values_stay_where_they_are_read(D):
    """The same for sequences of many rows: only the rows from the bad block on."""
    bs = 16
    batch = ref.Batch([80, 70, 1], [130, 70, 40], 1, D, bs, seed=7, width=12)
    for b, used in enumerate((9, 5, 3)):
        batch.kqs[batch.table[b, used:]] = batch.vqs[batch.table[b, used:]] = np.nan
        batch.table[b, used + 1 :] = -1
    q = rows16(151, 2, D, BF, 8)
    dev = batch.gpu()
    clean = run_attention(batch, q, 0.1, True, dev=dev)
    check_attention(batch, q, 0.1, y=clean)
    for name in ("kqs", "vqs"):
        spoilt = batch.gpu()
        spoilt[name][batch.table[0, 5]] = float("nan")  # positions 80 .. 95
        spoilt["table"][1, 3] = batch.num  # positions 48 .. 63: outside the cache
        q2 = q.clone()
        q2[3, 1, 7] = float("inf")
        y = run_attention(batch, q2, 0.1, True, dev=spoilt)
        bad = torch.zeros((151, 2, D), dtype=torch.bool)
        bad[30:80] = True  # tokens at positions 50 + i
        bad[80 + 48 : 150] = True
        bad[3, 1] = True
        assert torch.equal(y.isnan().cpu(), bad)
        assert torch.equal(y[~bad.cuda()], clean[~bad.cuda()])


@pytest.mark.gpu
def test_attention_rows_behind_the_last_sequence():
    batch = ref.Batch([2, 1], [30, 70], 1, 64, 16, seed=8)
    q = rows16(9, 2, 64, BF, 1)
    y = run_attention(batch, q, 0.125, True)
    check_attention(batch, q[:3], 0.125, y=y)
    assert bool((y[3:] == -7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [0, 1, 3, 200, 1 << 40])
def test_attention_with_any_max_q(max_q):
    batch = ref.Batch([1, 5, 170, 0, 30], [77, 300, 200, 4, 31], 2, 128, 16, seed=11)
    check_attention(batch, rows16(batch.T, 6, 128, BF, 1), max_q=max_q)


@pytest.mark.gpu
def test_attention_many_sequences():
    """More sequences than are looked at together (32), with empty ones and prompts among them."""
    g = np.random.default_rng(12)
    new = g.integers(0, 3, 150)
    new[[3, 40, 41, 130]] = [90, 33, 70, 65]
    lens = np.maximum(new, g.integers(0, 200, 150))
    batch = ref.Batch(new.tolist(), lens.tolist(), 1, 64, 16, seed=12)
    check_attention(batch, rows16(batch.T, 4, 64, FP, 1))
    batch.new = [min(n, 1) for n in batch.new]
    batch.cu = np.concatenate([[0], np.cumsum(batch.new)]).astype(np.int32)
    batch.T = int(batch.cu[-1])
    check_attention(batch, rows16(batch.T, 4, 64, FP, 2))


@pytest.mark.gpu
def test_prompts_of_half_a_block_of_rows():
    """Several blocks of rows to an SM, one after another, all (or only some) with rows in their first half alone."""
    lens = np.random.default_rng(13).integers(700, 1000, 64)
    for new in ([70] * 64, [70, 300] * 32):
        batch = ref.Batch(new, lens.tolist(), 8, 64, 16, seed=13)
        check_attention(batch, rows16(batch.T, 8, 64, BF, 1))


LONG = [
    # few rows on many keys (cut into pieces by keys): new, lens, block, Hkv, group, D
    ([70], [6000], 16, 1, 1, 128), ([33], [9000], 64, 2, 4, 64), ([257, 3, 90], [5000, 200, 3000], 32, 2, 2, 128),
    ([65], [1153], 16, 1, 1, 64), ([66, 1, 70] * 14, [1500, 4000, 100] * 14, 64, 3, 1, 64), ([17], [20000], 128, 8, 16, 128),
    ([300, 2000], [8000, 2000], 16, 1, 3, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,block,hkv,group,D", LONG)
def test_prompts_on_many_keys(new, lens, block, hkv, group, D, causal):
    """Twice the same bits, and the counters zero again."""
    batch = ref.Batch(new, lens, hkv, D, block, seed=14)
    dev = batch.gpu()
    q = rows16(batch.T, hkv * group, D, BF if D == 128 else FP, 2)
    ws = sq.workspace(sq.SQ_OP_KV8_ATTENTION, batch.T, hkv * group, D)
    y = run_attention(batch, q, 0.09, causal, dev=dev, ws=ws, pad=8)
    assert torch.equal(y, run_attention(batch, q, 0.09, causal, dev=dev, ws=ws))
    check_attention(batch, q, 0.09, causal, y=y)
    assert int(ws[256 : 256 + 4096].sum()) == 0


@pytest.mark.gpu
def test_prompts_on_many_keys_bad_values():
    """In a piece of a long sequence's keys: all rows that see the block, and no row of another sequence or head."""
    batch = ref.Batch([80, 70], [5000, 3000], 2, 128, 16, seed=15)
    q = rows16(150, 4, 128, BF, 8)
    clean = run_attention(batch, q, 0.1, True)
    for name in ("kqs", "vqs"):
        spoilt = batch.gpu()
        spoilt[name][batch.table[0, 200], 1] = float("nan")  # positions 3200 .. 3215, head 1
        y = run_attention(batch, q, 0.1, True, dev=spoilt)
        bad = torch.zeros((150, 4, 128), dtype=torch.bool)
        bad[:80, 2:] = True
        assert torch.equal(y.isnan().cpu(), bad)
        assert torch.equal(y[~bad.cuda()], clean[~bad.cuda()])


@pytest.mark.gpu
def test_attention_same_bits_every_time():
    """One workspace for batches of different lengths in turn; equal bits; the counters are zero again."""
    ws = sq.workspace(sq.SQ_OP_KV8_ATTENTION, 64, 16, 128)
    for new, lens in (([1], [4000]), ([1] * 5, [900, 1, 64, 333, 2000]), ([9, 1], [100, 1500]),
                      ([300, 1, 400], [900, 1500, 400]), ([1], [4000])):
        batch = ref.Batch(new, lens, 2, 128, 16, seed=9)
        dev = batch.gpu()
        q = rows16(batch.T, 8, 128, BF, 1)
        first = run_attention(batch, q, 0.1, True, dev=dev, ws=ws)
        for _ in range(3):
            assert torch.equal(first, run_attention(batch, q, 0.1, True, dev=dev, ws=ws))
        check_attention(batch, q, 0.1, y=first)
        assert int(ws[256 : 256 + 4096].sum()) == 0


@pytest.mark.gpu
def test_append_then_attend_in_a_graph():
    """Decode steps captured once and replayed with growing lengths, on a stream of its own."""
    H, G, D, bs, B = 2, 4, 128, 16, 3
    batch = ref.Batch([1] * B, [20, 31, 64], H, D, bs, seed=10, width=8)
    dev = batch.gpu()
    kn, vn = (torch.zeros((B, H, D), dtype=BF, device="cuda") for _ in range(2))
    q, y = (torch.zeros((B, H * G, D), dtype=BF, device="cuda") for _ in range(2))
    ws = sq.workspace(sq.SQ_OP_KV8_ATTENTION, B, H * G, D)

    def step():
        sq.sq_kv8_append(kn, vn, dev["cu"], dev["lens"], dev["table"], dev["k"], dev["v"], dev["kqs"], dev["vqs"])
        sq.sq_kv8_attention(q, dev["k"], dev["v"], dev["kqs"], dev["vqs"], dev["cu"], dev["lens"], dev["table"], 0.1,
                            True, 1, y, ws)

    saved = {n: dev[n].clone() for n in ("k", "v", "kqs", "vqs")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    for n in saved:
        dev[n].copy_(saved[n])
    for t in range(20):
        k, v, qq = (rows16(B, h, D, BF, 3 * t + i) for i, h in enumerate((H, H, H * G)))
        kn.copy_(k)
        vn.copy_(v)
        q.copy_(qq)
        g.replay()
        torch.cuda.synchronize()
        ref.append(batch, k.double().numpy(), v.double().numpy())
        check_attention(batch, qq, 0.1, y=y)
        batch.lens = [n + 1 for n in batch.lens]
        dev["lens"] += 1
    sq.sq_workspace_status(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,lens", [([70, 130, 1], [75, 200, 9]), ([70, 3], [3000, 40])])
@pytest.mark.parametrize("kind", ["zeros", "zero_block", "tiny_keys", "zero_scale"])
def test_prompt_of_equal_scores(kind, new, lens, D, causal):
    """Rows whose scores are all equal because q, K or the scale is zero: equal weights. The blocks of zero (or
    1e-7 sized) keys have the largest scales that there are, and rows end inside a block; whole and cut by keys."""
    batch = ref.Batch(new, lens, 2, D, 16, seed=21)
    dev = batch.gpu()
    q = rows16(batch.T, 4, D, BF, 1)
    k, v = rows16(batch.T, 2, D, BF, 2), rows16(batch.T, 2, D, BF, 3)
    if kind == "zeros":
        q, k, v = (torch.zeros_like(x) for x in (q, k, v))
    elif kind == "tiny_keys":
        q, k = torch.zeros_like(q), k * 1e-7
    else:
        k[19:60] = 0  # a whole block of the first sequence and more
        if kind == "zero_block":
            q = torch.zeros_like(q)
    check_append(batch, k, v, dev)
    check_attention(batch, q, 0.0 if kind == "zero_scale" else None, causal, dev=dev)


@pytest.mark.gpu
def test_prompt_of_zeros_with_bad_scales():
    """A NaN scale of a block reaches the zero rows that see it, and a NaN score scale every row that sees a key."""
    batch = ref.Batch([80, 90], [80, 2000], 1, 64, 16, seed=22)
    q = torch.zeros((170, 2, 64), dtype=BF)
    for name in ("kqs", "vqs"):
        spoilt = batch.gpu()
        spoilt[name][batch.table[0, 2]] = float("nan")  # positions 32 .. 47
        y = run_attention(batch, q, 0.1, True, dev=spoilt)
        bad = torch.zeros((170, 2, 64), dtype=torch.bool)
        bad[32:80] = True
        assert torch.equal(y.isnan().cpu(), bad)
    assert bool(run_attention(batch, rows16(170, 2, 64, BF, 1), float("nan"), True).isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 5, 70])
def test_attention_one_high_score_before_a_long_tail(new, D):
    """A first key whose weight is 2^26 times each other's and whose value is zero, so the output is the tail's alone;
    heads enough that nobody's keys are cut into parts (which have maxima of their own). A weight below 2^-21 of the
    largest is an fp16 subnormal once it is lifted by 2^7: off by 2^-25 2^-7 of the largest at most (all values have one
    scale here), in all 2^-32 sum |v|, beside what check_attention counts."""
    B, H, N = 64, 8, 2005
    batch = ref.Batch([new] * B, [N] * B, H, D, 128, seed=23)
    batch.table[:] = batch.table[0]  # all sequences read the same blocks
    batch.k[:] = 0
    batch.kqs[:] = 127.0
    batch.vqs[:] = 31.75
    batch.v = np.maximum(np.abs(batch.v), 1)  # nothing cancels
    first = batch.table[0, 0]
    batch.k[first, :, 0, 0] = 127
    batch.v[first, :, 0] = 0
    q = torch.zeros((batch.T, 2 * H, D), dtype=BF)
    q[:, :, 0] = 18.0  # 25.97 in log2
    y = run_attention(batch, q, 1.0, False).double()
    one = ref.Batch([new], [N], H, D, 128)
    for name in ("k", "v", "kqs", "vqs"):
        setattr(one, name, getattr(batch, name))
    one.table = batch.table[:1]
    want, mass = ref.attention(one, q[:new].double().cuda(), 1.0, False)
    used = batch.v[batch.table[0]].transpose(1, 0, 2, 3).reshape(H, -1, D)[:, :N].astype(np.float64).sum(1)
    floor = torch.from_numpy(2.0**-32 * used / 31.75).cuda().repeat_interleave(2, 0)
    tol = 2.0**-8 * want + 3.1e-3 * mass + floor
    assert bool((want > 50 * floor).all())
    err = (y.view(B, new, 2 * H, D) - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_refuses_an_unaligned_workspace(L):
    """Its counters and sums are accessed up to 16 bytes at a time: host error, no launch."""
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
    status = L.sq_kv8_attention(p, 2, 4, 8, 2, 64, 512, p, p, p, p, 8, 16, p, p, 1, p, 4, 4, 0.125, 1, 4, p, 512, odd,
                                1 << 24, None)
    assert status == 3 and "workspace must be 16-byte aligned" in L.sq_last_error_string().decode()
