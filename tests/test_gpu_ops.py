"""The operators of include/vit_ops.h against plain implementations in 64 bits, at the sizes, masks,
strides and values where they can go wrong.  Tolerances count the roundings: u = eps / 2 of the type,
half a step relative to the value."""
import math

import pytest
import torch

from parity import gpu, need_cuda

pytestmark = gpu

E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NAN = float("nan")


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def lib():
    need_cuda()
    import vision_transformer_encoder_fwd_b200 as V
    return V


# ------------------------------------------------------------------ norm and 8-bit rows
# fp32 arithmetic of the norm, relative: the sum of squares of a row has at most 64 terms in a thread
# and 6 + 32 joining steps, each off by 2^-24 (half of it after the root); the root (2 units in the
# last place), the residual's addition and four products: below 100 / 2 + 2 * 2 + 6 half steps.
NORM32 = 64 * 2.0 ** -24


def check_rows8(out, scales, y, what):
    """8-bit rows against y in 64 bits: half a step of e4m3 (2^-4 relative, or half of its smallest
    step 2^-9) of the scaled value, the scale's and the norm's fp32 roundings."""
    want_s = y.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
    assert ((scales.double() - want_s).abs() <= NORM32 * want_s).all(), what
    err = (out.double() * scales.double()[:, None] - y).abs()
    tol = y.abs() * (2.0 ** -4 + 4 * NORM32) + want_s[:, None] * 2.0 ** -10
    assert (err <= tol).all(), (what, (err - tol).max().item())


@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 64), (2, 129), (9, 256), (4, 264), (3, 1000), (7, 1024), (2, 4096),
                                    (130, 1536), (2, 12285), (3, 12288), (2, 16384), (1, 16392), (2, 32768), (1, 32767)])
@pytest.mark.parametrize("xt,rt,wt,e4m3", [("bf16", "fp32", "bf16", True), ("bf16", "bf16", "fp32", False),
                                           ("fp16", None, "fp16", True), ("fp32", "fp32", "fp32", False),
                                           ("fp32", None, "fp32", True), ("fp16", "fp32", "fp16", False)])
def test_rms_norm(rows, D, xt, rt, wt, e4m3):
    V, g = lib(), gen(rows * 131 + D)
    x = randn(g, rows, D, dtype=DT[xt], scale=2.0)
    w = (1 + randn(g, D, scale=0.3)).to(DT[wt])
    r = None if rt is None else randn(g, rows, D, dtype=DT[rt], scale=3.0)
    out, scales, h = V.rms_norm(x, w, 1e-5, residual=r, fp8=e4m3)
    hd = x.double() + (0 if r is None else r.double())
    y = hd / torch.sqrt(hd.square().mean(dim=1, keepdim=True) + 1e-5) * w.double()
    if r is not None:
        assert h.dtype == r.dtype
        uh = u_of(r.dtype) + 2.0 ** -24
        assert ((h.double() - hd).abs() <= uh * 1.01 * (x.double().abs() + r.double().abs())).all()
    # the residual's sum in fp32 is off by 2^-24 of its parts, where they cancel too
    part = x.double().abs() + (0 if r is None else r.double().abs())
    slack = part * w.double().abs() * 2.0 ** -23 / torch.sqrt(hd.square().mean(dim=1, keepdim=True) + 1e-5)
    if e4m3:
        s = scales.double()[:, None]
        want_s = y.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
        assert ((scales.double() - want_s).abs() <= NORM32 * want_s + slack.amax(dim=1) / 448).all()
        err = (out.double() * s - y).abs()
        assert (err <= y.abs() * (2.0 ** -4 + 4 * NORM32) + 2 * slack + s * 2.0 ** -10).all()
    else:
        assert scales is None and out.dtype == x.dtype
        err = (out.double() - y).abs()
        # fp16 has its smallest step of 2^-24 below 2^-14
        tiny = 2.0 ** -25 if xt == "fp16" else 0.0
        assert (err <= y.abs() * (u_of(x.dtype) + NORM32) * 1.01 + 2 * slack + tiny).all()


def test_rms_norm_strides_in_place_and_stream():
    """Rows of wider matrices (16-byte accesses and not), the residual updated in place, `out` over x, another stream."""
    V, g = lib(), gen(5)
    for pad in (8, 3):
        big = randn(g, 33, 200 + pad, dtype=torch.bfloat16)
        res = randn(g, 33, 208 + pad)
        x, r = big[:, :200], res[:, 4:204]
        before_big, before_res = big.clone(), res.clone()
        w = randn(g, 200, dtype=torch.bfloat16)
        hd = x.double() + r.double()
        y = hd / torch.sqrt(hd.square().mean(dim=1, keepdim=True) + 1e-6) * w.double()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out, _, h = V.rms_norm(x, w, 1e-6, residual=r, residual_out=r, out=x, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert out is x and h is r
        assert ((r.double() - hd).abs() <= 2.0 ** -23 * (hd.abs() + 6)).all()
        assert ((x.double() - y).abs() <= y.abs() * (2.0 ** -8 + NORM32) * 1.01 + 1e-5).all()
        # what lies between the rows is untouched
        assert torch.equal(big[:, 200:], before_big[:, 200:])
        assert torch.equal(res[:, :4], before_res[:, :4]) and torch.equal(res[:, 204:], before_res[:, 204:])


@pytest.mark.parametrize("rt", [None, "same", "fp32"])
@pytest.mark.parametrize("xt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [1, 9, 65, 263, 497, 519, 1003, 2055, 4090, 8179, 8199, 16391, 20007, 32767])
def test_rows_that_begin_anywhere(D, xt, rt):
    """Rows of any width behind one another and with gaps (NaN, which stays), the operands' strides the same modulo
    8 elements or not."""
    V, g = lib(), gen(D)
    rows, dt = 9, DT[xt]
    w = (1 + randn(g, D, scale=0.3)).to(dt)
    x = randn(g, rows, D, dtype=dt, scale=2.0)
    r = None if rt is None else randn(g, rows, D, dtype=dt if rt == "same" else torch.float32)
    xd, rd = x.double(), 0 if r is None else r.double()
    hd = xd + rd
    rms = torch.sqrt(hd.square().mean(dim=1, keepdim=True) + 1e-5)
    y = hd / rms * w.double()
    # the residual's sum in fp32 is off by 2^-24 of its parts, where they cancel too
    slack = (xd.abs() + (0 if r is None else rd.abs())) * w.double().abs() * 2.0 ** -23 / rms

    def wide(t, gap):
        big = torch.full((rows, D + gap), NAN, device="cuda").to(t)
        return big, big[:, :D]

    for e4m3 in (False, True):
        for gaps in ((0, 0, 0, 0), (3, 11, 3, 19), (3, 3, 4, 5)):
            xb, xv = wide(dt, gaps[0])
            xv.copy_(x)
            ob, ov = wide(E4M3 if e4m3 else dt, gaps[1])
            rv = hv = hb = None
            if r is not None:
                rv = wide(r.dtype, gaps[2])[1]
                rv.copy_(r)
                hb, hv = wide(r.dtype, gaps[3])
            out, scales, h = V.rms_norm(xv, w, 1e-5, residual=rv, residual_out=hv, out=ov, fp8=e4m3)
            if r is not None:
                assert torch.equal(h, (x.float() + r.float()).to(r.dtype))
            if e4m3:
                want_s = y.abs().amax(dim=1).clamp_min(2.0 ** -100) / 448
                assert ((scales.double() - want_s).abs() <= NORM32 * want_s + slack.amax(dim=1) / 448).all()
                s = scales.double()[:, None]
                assert ((out.double() * s - y).abs() <= y.abs() * (2.0 ** -4 + 4 * NORM32) + 2 * slack + s * 2.0 ** -10).all()
            else:
                tiny = 2.0 ** -25 if xt == "fp16" else 0.0  # half of fp16's smallest step
                assert ((out.double() - y).abs() <= y.abs() * (u_of(dt) + NORM32) * 1.01 + 2 * slack + tiny).all()
            assert ob[:, D:].float().isnan().all() and (hb is None or hb[:, D:].isnan().all())
            assert xb[:, D:].isnan().all()


@pytest.mark.parametrize("D", [64, 1024, 16384, 7])
def test_rows_with_nan_infinity_and_zeros(D):
    """A NaN or an infinity reaches its own row only; rows of zeros and of tiny values stay finite."""
    V, g = lib(), gen(6)
    x = randn(g, 6, D)
    x[1, D // 2] = NAN
    x[2, D - 1] = math.inf
    x[3] = 0
    x[4] = 1e-42
    w = torch.ones(D, device="cuda")
    for e4m3 in (False, True):
        out, scales, _ = V.rms_norm(x, w, 1e-6, fp8=e4m3)
        o = out.float()
        assert torch.isfinite(o[[0, 3, 4, 5]]).all()
        assert o[1].isnan().all() and o[2, D - 1].isnan()
        assert (o[3] == 0).all()
        if e4m3:
            assert scales[1].isnan() and torch.isfinite(scales[[0, 3, 4, 5]]).all()
    q, s = V.quant_rows(x)
    assert s[1].isnan() and q.float()[1].isnan().all() and torch.isinf(s[2])
    assert torch.isfinite(q.float()[[0, 3, 4, 5]]).all() and (q.float()[3] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,D", [(1, 16), (17, 384), (5, 4097), (64, 4096), (3, 20000), (0, 64)])
def test_quant_rows(dtype, rows, D):
    V, g = lib(), gen(rows + D)
    x = randn(g, rows, D, dtype=DT[dtype], scale=5.0)
    q, s = V.quant_rows(x)
    assert q.shape == x.shape and s.shape == (rows,)
    if rows:
        check_rows8(q, s, x.double(), (dtype, rows, D))
        # the largest value of a row is held exactly as 448
        assert (q.float().abs().amax(dim=1) == 448).all()


# ------------------------------------------------------------------ linear
def make_linear(M, N, K, seed, bias):
    V, g = lib(), gen(seed)
    a, sa = V.quant_rows(randn(g, M, K, dtype=torch.bfloat16))
    w, sw = V.quant_rows(randn(g, N, K, scale=K ** -0.5))
    return a, sa, w, sw, (randn(g, N) if bias else None)


def check_linear(out, a, sa, w, sw, b):
    """bf16 rounding of the result, and fp32 sums: K / 32 steps and 32 products within one, each off by
    at most 2^-23 of the sum of magnitudes (a step that is cut, not rounded)."""
    K = a.shape[1]
    ad, wd = a.double() * sa.double()[:, None], w.double() * sw.double()[:, None]
    ref, mag = ad @ wd.T, ad.abs() @ wd.abs().T
    if b is not None:
        ref, mag = ref + b.double(), mag + b.double().abs()
    err = (out.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() * 1.01 + (K / 32 + 36) * 2.0 ** -23 * mag
    assert (err <= tol).all(), (err - tol).max().item()


@pytest.mark.parametrize("M,N,K,bias", [
    (1, 8, 16, True), (1, 64, 64, False), (2, 136, 48, True), (7, 6144, 4096, False), (8, 256, 144, True), (9, 512, 1024, True),
    (16, 4096, 4096, False), (17, 1000, 400, True), (31, 264, 8192, False), (32, 72, 112, True), (33, 640, 256, False),
    (64, 1152, 384, True), (65, 384, 1536, False), (127, 128, 128, True), (128, 256, 4080, False), (129, 136, 64, True),
    (300, 1000, 528, True), (1000, 1024, 4096, False), (2500, 2048, 1024, True), (4101, 3080, 1040, True),
    (8191, 520, 256, False), (8200, 4096, 512, True)])
def test_linear_fp8(M, N, K, bias):
    V = lib()
    a, sa, w, sw, b = make_linear(M, N, K, M + N + K, bias)
    out = V.linear_fp8(a, sa, w, sw, bias=b)
    V.op_poll()
    assert torch.isfinite(out.float()).all()
    check_linear(out, a, sa, w, sw, b)


@pytest.mark.parametrize("M,N,K", [(3, 64, 128), (20, 256, 512), (200, 320, 256), (2600, 1024, 256)])
def test_linear_fp8_strides_status_and_what_it_leaves(M, N, K):
    V = lib()
    a, sa, w, sw, b = make_linear(M, N, K, 3, True)
    abig = torch.full((M, K + 32), NAN, device="cuda").to(E4M3)
    wbig = torch.full((N, K + 16), NAN, device="cuda").to(E4M3)
    abig[:, 16:16 + K] = a
    wbig[:, :K] = w
    obig = torch.full((M + 2, N + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    V.linear_fp8(abig[:, 16:16 + K], sa, wbig[:, :K], sw, bias=b, out=obig[:M, :N], status=st, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert int(st.item()) == 0
    check_linear(obig[:M, :N], a, sa, w, sw, b)
    assert (obig[M:] == 7).all() and (obig[:, N:] == 7).all()


@pytest.mark.parametrize("M", [5, 150])
def test_linear_fp8_nan_row(M):
    """A NaN in a row of a, or an infinite scale, stays in that row."""
    V = lib()
    a, sa, w, sw, _ = make_linear(M, 128, 256, 4, False)
    clean = V.linear_fp8(a, sa, w, sw)
    af = a.float()
    af[2, 100] = NAN
    out = V.linear_fp8(af.to(E4M3), sa, w, sw)
    assert out[2].isnan().all()
    keep = [i for i in range(M) if i != 2]
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("M", [5, 200, 2600])
def test_linear_fp8_is_repeatable(M):
    """Two calls give the same bits (no sums in an order of arrival)."""
    V = lib()
    a, sa, w, sw, b = make_linear(M, 1024, 2048, 9, True)
    assert torch.equal(V.linear_fp8(a, sa, w, sw, bias=b), V.linear_fp8(a, sa, w, sw, bias=b))


# ------------------------------------------------------------------ rotary positions
def rope_ref(x, pos, freqs, layout, gain, inverse):
    """In 64 bits; positions [axes, T]."""
    n = freqs.shape[0]
    per = n // pos.shape[0]
    x, y = x.double(), x.double().clone()
    turn = freqs.to(x.device) / (2 * math.pi)
    for i in range(n):
        p = pos[i // per]
        # whole turns of the high and low halves of the position drop out one by one
        hi, lo = p >> 20, p & ((1 << 20) - 1)
        t = torch.remainder(hi.double() * torch.remainder(turn[i] * 2.0 ** 20, 1.0), 1.0) + lo.double() * turn[i]
        t = t * (2 * math.pi) * (-1 if inverse else 1)
        c, s = (torch.cos(t) * gain)[:, None], (torch.sin(t) * gain)[:, None]
        a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def check_rope(out, x, pos, freqs, layout, gain=1.0, inverse=False, far=0.0):
    """Rounding to the type, and fp32: the angle's conversion (2^-25 of at most pi), sine and cosine (2 units
    each) and three roundings of the products, below 5e-7 of |a| + |b|; `far`: the reference's own
    angle error (2^-53 of the turns at 64 bits)."""
    n, ref = freqs.shape[0], rope_ref(x, pos if pos.dim() == 2 else pos[None], freqs, layout, gain, inverse)
    xd = x.double().abs()
    mag = torch.zeros_like(xd)
    if layout == "half":
        mag[..., :n] = mag[..., n:2 * n] = xd[..., :n] + xd[..., n:2 * n]
    else:
        mag[..., 0:2 * n:2] = mag[..., 1:2 * n:2] = xd[..., 0:2 * n:2] + xd[..., 1:2 * n:2]
    tiny = 2.0 ** -25 if out.dtype == torch.float16 else 0.0
    tol = u_of(out.dtype) * 1.01 * ref.abs() + (5e-7 + far) * gain * mag + tiny
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), (err - tol).max().item()
    assert torch.equal(out[..., 2 * n:], x[..., 2 * n:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hkv,d,rd,axes", [
    (1, 1, 1, 2, 2, 1), (1, 32, 8, 128, 128, 1), (3, 4, 2, 64, 32, 1), (65, 6, 6, 64, 64, 2), (37, 3, 1, 80, 80, 2),
    (513, 8, 2, 96, 48, 1), (130, 2, 1, 256, 256, 4), (7, 5, 5, 66, 34, 1), (2000, 1, 1, 72, 72, 3), (4, 2, 1, 258, 256, 1)])
def test_rope(dtype, layout, T, hq, hkv, d, rd, axes):
    V, g = lib(), gen(T + d)
    qk = randn(g, T, hq + hkv, d, dtype=DT[dtype])
    q, k = qk[:, :hq], qk[:, hq:]
    pos = torch.randint(0, 5000, (axes, T), generator=g, device="cuda", dtype=torch.int32)
    f = V.rope_freqs(10000.0, rd, axes)
    qo, ko = V.rope(q, k, pos if axes > 1 else pos[0], f, layout=layout)
    check_rope(qo, q, pos, f, layout)
    check_rope(ko, k, pos, f, layout)


@pytest.mark.parametrize("far", [1 << 22, (1 << 31) - 1, 1 << 40])
def test_rope_far_and_negative_positions(far):
    V, g = lib(), gen(11)
    q = randn(g, 50, 2, 128)
    pos = torch.randint(-far, far, (50,), generator=g, device="cuda", dtype=torch.int64)
    pos[0], pos[1] = far, -far
    f = V.rope_freqs(500000.0, 128, scaling="parts", factor=32.0, original_len=8192)
    qo, _ = V.rope(q, None, pos, f)
    # the reference's turn fraction: hi (at most 2^20) times a remainder good to 2^-33 - 2^-53 of 2^20
    check_rope(qo, q, pos, f, "half", far=2 * math.pi * 2.0 ** 20 * 2.0 ** -33 if far > 1 << 32 else 2 * math.pi * 2.0 ** -21)
    if far < 1 << 31:
        same, _ = V.rope(q, None, pos.to(torch.int32), f)
        assert torch.equal(qo, same)


def test_rope_far_positions_agree_with_whole_turns():
    """A frequency of a binary fraction of a turn: positions 2^k apart give the same bits, however far."""
    V, g = lib(), gen(12)
    x = randn(g, 1, 1, 8).expand(6, 1, 8).contiguous()
    f = torch.tensor([2 * math.pi / 64, 2 * math.pi / 256, 2 * math.pi / 8, 2 * math.pi / 4], dtype=torch.float64)
    base = 37
    pos = torch.tensor([base, base + 256, base + (1 << 20), base + (1 << 30), base - 256, base + (1 << 33)], device="cuda")
    out, _ = V.rope(x, None, pos, f)
    # 2 pi / 64 in 64 bits is off by up to 2^-53 of itself: 2^33 positions on, 2^-26 of a turn
    assert ((out - out[:1]).abs() <= 2 * math.pi * 2.0 ** -25 * 8 * x.abs().amax()).all()
    assert torch.equal(out[0], out[1])


def test_rope_in_place_strided_inverse_gain_and_capture():
    V, g = lib(), gen(13)
    T, hq, hkv, d = 77, 4, 2, 64
    qkv = randn(g, T, hq + 2 * hkv, d, dtype=torch.bfloat16)
    before = qkv.clone()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    f = V.rope_freqs(10000.0, d)
    V.rope(q, k, pos, f, out=(q, k))
    check_rope(q, before[:, :hq], pos, f, "half")
    check_rope(k, before[:, hq:hq + hkv], pos, f, "half")
    assert torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:])
    # heads outside tokens, values at odd offsets
    x = randn(g, 3, T, 2 * d + 1)[..., 1:1 + d].permute(1, 0, 2)
    y, _ = V.rope(x, None, pos, f, layout="interleaved", gain=1.25)
    check_rope(y, x, pos, f, "interleaved", gain=1.25)
    z, _ = V.rope(x, None, pos, f, layout="interleaved", gain=0.8, inverse=True)
    check_rope(z, x, pos, f, "interleaved", gain=0.8, inverse=True)
    # the inverse is the transpose (the gradient's rotation): <rope x, w> = <x, rope^-1 w>
    w = randn(g, T, 3, d)
    lhs = (V.rope(x, None, pos, f)[0].double() * w.double()).sum()
    rhs = (x.double() * V.rope(w, None, pos, f, inverse=True)[0].double()).sum()
    n = T * 3 * d
    assert abs(lhs - rhs) <= 1e-6 * 8 * n
    # captured: new positions and values on replay, the frequencies of the capture
    out = torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        V.rope(w, None, pos, f, out=(out, None))
    w.copy_(randn(g, T, 3, d))
    pos.add_(1000)
    f0 = f.clone()
    f.zero_()
    graph.replay()
    check_rope(out, w, pos, f0, "half")


def test_rope_empty():
    V = lib()
    q = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    f = V.rope_freqs(10000.0, 64)
    qo, ko = V.rope(q, q, torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert qo.shape == q.shape and ko.shape == q.shape


# ------------------------------------------------------------------ attention
def cum(v):
    return torch.tensor([0] + list(v), dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def attn_ref(q, k, v, q0, k0, lq, lk, causal, scale):
    """Sequence by sequence in 64 bits: {row: (result, sum of p |v|, number of keys)}."""
    Hq, Hk = q.shape[1], k.shape[1]
    res = []
    for b in range(len(lq)):
        if lq[b] == 0:
            continue
        qs = q[q0[b]:q0[b] + lq[b]].double().permute(1, 0, 2)
        ks = k[k0[b]:k0[b] + lk[b]].double().permute(1, 0, 2).repeat_interleave(Hq // Hk, dim=0)
        vs = v[k0[b]:k0[b] + lk[b]].double().permute(1, 0, 2).repeat_interleave(Hq // Hk, dim=0)
        z = qs @ ks.transpose(1, 2) * scale
        if causal:
            i = torch.arange(lq[b], device="cuda")[:, None]
            j = torch.arange(lk[b], device="cuda")[None]
            z = z.masked_fill(j > i + lk[b] - lq[b], -math.inf)
        if lk[b] == 0:
            o = a = torch.zeros_like(qs)
        else:
            top = z.amax(dim=-1, keepdim=True)
            p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            den = p.sum(dim=-1, keepdim=True)
            p = torch.where(den == 0, 0.0, p / den)
            o, a = p @ vs, p @ vs.abs()
        res.append((b, o.permute(1, 0, 2), a.permute(1, 0, 2)))
    return res


def check_attn(out, q, k, v, q0, k0, lq, lk, causal, scale, zmax=32.0):
    """The weights and the result are rounded to the type (u each; the denominator's weights too: u); an
    exponential is off by 1e-4 at most (numerator and denominator); a score of magnitude up to
    zmax by d 2^-24 of its products' sum, taken as 8 zmax; fp16 weights below 2^-14 by 2^-25."""
    u = u_of(out.dtype)
    tiny = 2.0 ** -25 if out.dtype == torch.float16 else 0.0
    score = 2 * 8 * zmax * 2.0 ** -24 * 8
    for b, o, a in attn_ref(q, k, v, q0, k0, lq, lk, causal, scale):
        got = out[q0[b]:q0[b] + lq[b]].double()
        vmax = v[k0[b]:k0[b] + lk[b]].double().abs().max().item() if lk[b] else 0.0
        tol = u * 1.01 * o.abs() + (2 * u * 1.01 + 2e-4 + score) * a + tiny * (2 + 2 * lk[b] * vmax)
        err = (got - o).abs()
        assert (err <= tol).all(), (b, lq[b], lk[b], (err - tol).max().item())


KERNELS = ["tile", "split", "short"]


def by_kernel(kernel, k, v, cu_q, cu_k, len_k=None):
    """The arguments that make a call take the named kernel, without changing its result: key rows of nobody
    (NaN) or empty sequences behind the others, and a max_q that need not be true."""
    n = cu_q.shape[0] - 1
    if kernel == "split":
        pad = torch.full((600 * n, *k.shape[1:]), NAN, dtype=k.dtype, device="cuda")
        return dict(k=torch.cat([k, pad]), v=torch.cat([v, pad]), cu_q=cu_q, cu_k=cu_k, len_k=len_k, max_q=1)
    if kernel == "short":
        more = max(0, -(-k.shape[0] // 64) - n)
        cu_q, cu_k = (torch.cat([c, c[-1:].expand(more)]) for c in (cu_q, cu_k))
        if len_k is not None:
            len_k = torch.cat([len_k, torch.zeros(more, dtype=torch.int32, device="cuda")])
        return dict(k=k, v=v, cu_q=cu_q, cu_k=cu_k, len_k=len_k, max_q=1)
    return dict(k=k, v=v, cu_q=cu_q, cu_k=cu_k, len_k=len_k, max_q=0)


LENS = {  # (query length, key length) of each sequence
    "one": [(1, 1)],
    "edges": [(1, 64), (64, 64), (65, 65), (63, 63), (127, 127), (128, 128), (129, 129), (2, 2)],
    "holes": [(0, 5), (5, 0), (0, 0), (3, 3), (1, 0), (0, 0), (200, 0), (4, 70)],
    "longer_keys": [(1, 300), (17, 290), (130, 333), (2, 65)],
    "longer_queries": [(300, 1), (140, 130), (65, 64), (129, 1), (20, 3)],
    "many": [(i % 23 + 1, i % 23 + 1) for i in range(150)],
    "prompt": [(513, 513), (40, 40)],
    "tokens": [(1, 33), (1, 1), (1, 700), (1, 64), (1, 65), (1, 129), (1, 0)],
    "few": [(4, 100), (0, 9), (2, 2), (3, 1000), (1, 5)],
}


@pytest.mark.parametrize("d,dtype,hq,hkv", [(64, "bf16", 4, 4), (64, "fp16", 6, 2), (128, "bf16", 8, 2), (128, "fp16", 3, 1),
                                            (128, "bf16", 12, 1)])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kernel", KERNELS + ["rule"])
def test_attention_packed(d, dtype, hq, hkv, lens, causal, kernel):
    """Packed sequences behind one another, each followed by rows of nobody (NaN) that have to stay."""
    V = lib()
    lq, lk = [x[0] for x in LENS[lens]], [x[1] for x in LENS[lens]]
    g, dt, tail = gen(d + len(lens)), DT[dtype], 3
    same = lq == lk
    Tq, Tk = sum(lq) + tail, sum(lk) + tail
    q = randn(g, Tq, hq, d, dtype=dt)
    k, v = randn(g, Tk, hkv, d, dtype=dt), randn(g, Tk, hkv, d, dtype=dt)
    if same:  # the fused projection's output, read in place
        qkv = torch.cat([q, k, v], dim=1)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    k[-tail:], v[-tail:], q[-tail:] = NAN, NAN, NAN
    out = torch.full((Tq, hq, d), 0.5, dtype=dt, device="cuda")
    cu_q, cu_k = cum(lq), cum(lk)
    args = dict(k=k, v=v, cu_q=cu_q, cu_k=cu_k, max_q=max(lq)) if kernel == "rule" else by_kernel(kernel, k, v, cu_q, cu_k)
    res = V.attention_packed(q, **args, causal=causal, out=out)
    V.op_poll()
    assert res is out and (out[-tail:] == 0.5).all()
    check_attn(out, q, k, v, cu_q.tolist(), cu_k.tolist(), lq, lk, causal, d ** -0.5)


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 8, 1), (128, 2, 2)])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("room,lens", [(64, [1, 64, 0, 63]), (100, [100, 99, 65, 1, 64]), (1037, [1037, 3, 512, 1000])])
def test_attention_over_a_cache(d, hq, hkv, single, kernel, room, lens):
    """New tokens over caches with room, in a larger buffer with heads outside tokens: what lies past a length
    is NaN, queries of different numbers (none among them)."""
    V, g = lib(), gen(room)
    n = len(lens)
    lq = [1 if single else min(lens[i], (1, 3, 0, 5, 2)[i]) for i in range(n)]
    Tk = n * room + 7
    kv = randn(g, 2, hkv, Tk, d, dtype=torch.bfloat16)
    for i, ln in enumerate(lens):
        kv[:, :, i * room + ln:(i + 1) * room] = NAN
    kv[:, :, n * room:] = NAN
    k, v = kv[0].permute(1, 0, 2), kv[1].permute(1, 0, 2)
    q = randn(g, sum(lq) + 2, hq, d, dtype=torch.bfloat16)
    out = torch.full_like(q, 0.5)
    cu_q, cu_k = cum(lq), cum([room] * n)
    len_k = torch.tensor(lens, dtype=torch.int32, device="cuda")
    V.attention_packed(q, **by_kernel(kernel, k, v, cu_q, cu_k, len_k), causal=True, scale=0.2, out=out)
    V.op_poll()
    check_attn(out, q, k, v, cu_q.tolist(), cu_k.tolist(), lq, lens, True, 0.2)
    assert (out[sum(lq):] == 0.5).all()


@pytest.mark.parametrize("n,hq,hkv,d,lk,dtype", [(1, 8, 8, 128, 30011, "bf16"), (1, 1, 1, 64, 65536, "fp16"), (3, 16, 2, 128, 20000, "fp16"),
                                                 (40, 4, 2, 64, 3000, "bf16"), (97, 2, 1, 128, 777, "bf16")])
def test_attention_tokens_long_cache(n, hq, hkv, d, lk, dtype):
    """Single tokens over long caches: the keys' axis is split and joined; twice the same bits."""
    V, g = lib(), gen(lk)
    lens = [max(1, lk - 97 * i) for i in range(n)]
    k, v = randn(g, n * lk, hkv, d, dtype=DT[dtype]), randn(g, n * lk, hkv, d, dtype=DT[dtype])
    q = randn(g, n, hq, d, dtype=DT[dtype])
    cu_q, cu_k = cum([1] * n), cum([lk] * n)
    len_k = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = V.attention_packed(q, k, v, cu_q, cu_k, len_k=len_k, causal=True, max_q=1)
    V.op_poll()
    check_attn(out, q, k, v, list(range(n)), [i * lk for i in range(n)], [1] * n, lens, True, d ** -0.5)
    assert torch.equal(out, V.attention_packed(q, k, v, cu_q, cu_k, len_k=len_k, causal=True, max_q=1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_sharp_and_large_scores(d, kernel):
    """Scores that grow along the keys by far more than the rescaling step, up to 1e6, and a sink that takes all
    the weight."""
    V, g = lib(), gen(d)
    lk, lq = 700, 130
    q = torch.ones(lq, 2, d, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(lk, 2, d, device="cuda", dtype=torch.bfloat16)
    # exact in bf16 and fp32: scores 0, 64, 128, ... on every 50th key; the second head falls instead
    for i, j in enumerate(range(0, lk, 50)):
        k[j, 0, 0], k[lk - 1 - j, 1, 0] = 64.0 * i, 64.0 * i
    v = randn(g, lk, 2, d, dtype=torch.bfloat16)
    cu_q, cu_k = cum([lq]), cum([lk])
    for causal in (False, True):
        out = V.attention_packed(q, **by_kernel(kernel, k, v, cu_q, cu_k), causal=causal, scale=1.0)
        check_attn(out, q, k, v, [0], [0], [lq], [lk], causal, 1.0, zmax=1.0)
    k[:, :, 0] = 0
    k[123, :, 0] = 1.0e6
    out = V.attention_packed(q, **by_kernel(kernel, k, v, cu_q, cu_k), scale=1.0)
    # one weight, rounded (u), over an unrounded or rounded sum, and the result's rounding
    assert ((out.double() - v[123].double()).abs() <= 2.02 * 2.0 ** -8 * v[123].double().abs()).all()
    V.op_poll()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("at", range(60, 80))
def test_attention_nan_and_infinite_keys(d, kernel, at):
    """A NaN in a key, or a score of +infinity, reaches exactly the rows that see it; -infinity is weight 0."""
    V, g = lib(), gen(at)
    n = 150
    q, k, v = (randn(g, n, 2, d, dtype=torch.bfloat16) for _ in range(3))
    q[..., 0] = q[..., 0].abs() + 0.1
    cu = cum([n])
    clean = V.attention_packed(q, **by_kernel(kernel, k, v, cu, cu), causal=True)
    for bad in (NAN, math.inf, -math.inf):
        k2 = k.clone()
        k2[at, 0, 0] = bad
        out = V.attention_packed(q, **by_kernel(kernel, k2, v, cu, cu), causal=True)
        assert torch.equal(out[:at], clean[:at]) and torch.equal(out[:, 1], clean[:, 1])
        if bad == -math.inf:
            assert torch.isfinite(out.float()).all()
        else:
            assert out[at:, 0].isnan().all()
    V.op_poll()


@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_clamps_bad_bounds(kernel):
    """Bounds outside the buffers (stale tables) read and write nothing outside them; a length past a
    sequence's room is its room."""
    V, g = lib(), gen(20)
    keys = 2000 if kernel == "split" else 90
    q = randn(g, 6, 2, 64, dtype=torch.bfloat16)
    k, v = randn(g, keys, 2, 64, dtype=torch.bfloat16), randn(g, keys, 2, 64, dtype=torch.bfloat16)
    cu_q = torch.tensor([0, 1, 2, 999], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([-50, 30, 60, 100000], dtype=torch.int32, device="cuda")
    len_k = torch.tensor([500, 30, -3], dtype=torch.int32, device="cuda")
    out = V.attention_packed(q, k, v, cu_q, cu_k, len_k=len_k, max_q=0 if kernel == "tile" else 1)
    V.op_poll()
    check_attn(out, q, k, v, [0, 1, 2], [0, 30, 60], [1, 1, 4], [30, 30, 0], False, 0.125)


@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_streams_and_two_captured_graphs(kernel):
    """Calls side by side on two streams, and two captured graphs replayed side by side with new lengths."""
    V, g = lib(), gen(21)
    n, hq, hkv, d, room = 9, 8, 2, 128, 60 if kernel == "short" else 600
    max_q = 0 if kernel == "tile" else 1
    lens = [[(37 * i + s) % room + 1 for i in range(n)] for s in (1, 200, 411)]
    work = []
    for s in range(2):
        q = randn(g, n, hq, d, dtype=torch.bfloat16)
        k, v = randn(g, n * room, hkv, d, dtype=torch.bfloat16), randn(g, n * room, hkv, d, dtype=torch.bfloat16)
        len_k = torch.tensor(lens[s], dtype=torch.int32, device="cuda")
        work.append([q, k, v, len_k, torch.empty_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph()])
    cu_q, cu_k = cum([1] * n), cum([room] * n)
    at_q, at_k = cu_q.tolist(), cu_k.tolist()

    def call(w, **kw):
        return V.attention_packed(w[0], w[1], w[2], cu_q, cu_k, len_k=w[3], causal=True, max_q=max_q, out=w[4], **kw)

    def verify(which):
        torch.cuda.synchronize()
        for w, ln in zip(work, which):
            check_attn(w[4], w[0], w[1], w[2], at_q, at_k, [1] * n, ln, True, d ** -0.5)
            w[4].fill_(NAN)
        torch.cuda.synchronize()
    torch.cuda.synchronize()
    for _ in range(3):
        for w in work:
            call(w, stream=w[5])
    verify(lens[:2])
    for w in work:
        with torch.cuda.graph(w[6]):
            call(w)
    torch.cuda.synchronize()
    for _ in range(3):
        for w in work:
            with torch.cuda.stream(w[5]):
                w[6].replay()
    verify(lens[:2])
    for w in work:
        w[3].copy_(torch.tensor(lens[2], dtype=torch.int32))
    torch.cuda.synchronize()
    for w in work:
        with torch.cuda.stream(w[5]):
            w[6].replay()
    verify([lens[2], lens[2]])
    V.op_poll()


def test_attention_wait_expiry_is_reported():
    """A pipeline wait cut to 200 ns runs out on purpose: the status tells, later calls on the word return
    without work until it is cleared, and the next call is right."""
    V, g = lib(), gen(22)
    n = 500
    q, k, v = (randn(g, n, 2, 128, dtype=torch.bfloat16) for _ in range(3))
    cu = cum([n])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    V.attention_packed(q, k, v, cu, cu, status=st, wait_ns=200)
    torch.cuda.synchronize()
    assert 0x400 < int(st.item()) < 0x500
    out = torch.full_like(q, 0.5)
    V.attention_packed(q, k, v, cu, cu, status=st, out=out)
    assert (out == 0.5).all()
    V.attention_packed(q, k, v, cu, cu, wait_ns=200)
    with pytest.raises(V.VitError) as e:
        V.op_poll()
    assert e.value.status == V.VIT_E_DEVICE_TIMEOUT
    V.op_poll()
    V.attention_packed(q, k, v, cu, cu, out=out)
    V.op_poll()
    check_attn(out, q, k, v, [0], [0], [n], [n], False, 128 ** -0.5)


def test_linear_wait_expiry_is_reported():
    V = lib()
    a, sa, w, sw, b = make_linear(3000, 2048, 4096, 23, True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    V.linear_fp8(a, sa, w, sw, status=st, wait_ns=200)
    torch.cuda.synchronize()
    assert 0x300 < int(st.item()) < 0x400
    out = V.linear_fp8(a, sa, w, sw, bias=b)
    V.op_poll()
    check_linear(out, a, sa, w, sw, b)


# ------------------------------------------------------------------ together
def test_prompt_and_token_steps_of_a_layer():
    """The attention half of a pre-norm layer with 8-bit weights, as a decoder runs it: packed prompts first,
    their keys and values into a cache, then new tokens one by one.  Every stage is compared with 64 bits
    on the inputs it had, and the new tokens' results with those of the whole prompt at once."""
    V, g = lib(), gen(30)
    dim, hq, hkv, d, room = 512, 8, 2, 64, 96
    lens, steps = [50, 1, 33, 71], 3
    n, T = len(lens), sum(lens)
    w_norm = (1 + randn(g, dim, scale=0.1)).to(torch.bfloat16)
    w_qkv = V.quant_rows(randn(g, (hq + 2 * hkv) * d, dim, scale=dim ** -0.5, dtype=torch.bfloat16))
    w_out = V.quant_rows(randn(g, dim, hq * d, scale=dim ** -0.5, dtype=torch.bfloat16))
    freqs = V.rope_freqs(10000.0, d)
    cache = torch.full((2, n * room, hkv, d), NAN, device="cuda", dtype=torch.bfloat16)
    cu_k = cum([room] * n)

    def layer(x, res, pos, rows, cu_q, len_k, max_q):
        a, sa, h = V.rms_norm(x, w_norm, 1e-6, residual=res, fp8=True)
        qkv = V.linear_fp8(a, sa, *w_qkv).view(-1, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        V.rope(q, k, pos, freqs, out=(q, k))
        cache[0, rows], cache[1, rows] = k, v
        o = V.attention_packed(q, cache[0], cache[1], cu_q, cu_k, len_k=len_k, causal=True, max_q=max_q)
        oq, os = V.quant_rows(o.view(-1, hq * d))
        y = V.linear_fp8(oq, os, *w_out)
        hd = x.double() + res.double()
        assert ((h.double() - hd).abs() <= 2.0 ** -23 * (x.double().abs() + res.double().abs())).all()
        yn = hd / torch.sqrt(hd.square().mean(dim=1, keepdim=True) + 1e-6) * w_norm.double()
        assert ((a.double() * sa.double()[:, None] - yn).abs()
                <= yn.abs() * (2.0 ** -4 + 1e-5) + sa.double()[:, None] * 2.0 ** -9).all()
        lq = (cu_q[1:] - cu_q[:-1]).tolist()
        check_attn(o, q, cache[0], cache[1], cu_q.tolist(), cu_k.tolist(), lq, len_k.tolist(), True, d ** -0.5)
        check_linear(y, oq, os, *w_out, None)
        return y, h, o

    total = [ln + steps for ln in lens]
    xs = [randn(g, t, dim, dtype=torch.bfloat16) for t in total]
    rs = [randn(g, t, dim, scale=2.0) for t in total]

    def batch(parts):
        """Rows [from, to) of each sequence, packed."""
        pos = torch.cat([torch.arange(a, b) for a, b in parts]).to(torch.int32).cuda()
        rows = torch.cat([torch.arange(a, b) + i * room for i, (a, b) in enumerate(parts)]).cuda()
        return (torch.cat([x[a:b] for x, (a, b) in zip(xs, parts)]), torch.cat([r[a:b] for r, (a, b) in zip(rs, parts)]), pos,
                rows, cum([b - a for a, b in parts]), torch.tensor([b for _, b in parts], dtype=torch.int32, device="cuda"))
    y, h, o = layer(*batch([(0, ln) for ln in lens]), 0)
    token_o, token_y = [], []
    for s in range(steps):
        y, h, o = layer(*batch([(ln + s, ln + s + 1) for ln in lens]), 1)
        token_o.append(o)
        token_y.append(y)
    y, h, o = layer(*batch([(0, t) for t in total]), 0)
    at = cum(total).tolist()
    for s in range(steps):
        for i, ln in enumerate(lens):
            whole, token = o[at[i] + ln + s].double(), token_o[s][i].double()
            # two kernels, the same inputs: each within its tolerance of the exact result (values up to 5)
            assert (whole - token).abs().max() <= 2 * (3 * 2.0 ** -8 + 3e-4) * 5
    V.op_poll()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_rows_wait_expiry_is_reported(d):
    """The same for the kernel of few query rows, whose warps meet at the end of each item."""
    V, g = lib(), gen(24)
    n, lk = 40, 900
    q = randn(g, n, 4, d, dtype=torch.bfloat16)
    k, v = randn(g, n * lk, 2, d, dtype=torch.bfloat16), randn(g, n * lk, 2, d, dtype=torch.bfloat16)
    cu_q, cu_k = cum([1] * n), cum([lk] * n)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    V.attention_packed(q, k, v, cu_q, cu_k, max_q=1, status=st, wait_ns=200)
    torch.cuda.synchronize()
    assert 0x500 < int(st.item()) < 0x600
    out = torch.full_like(q, 0.5)
    V.attention_packed(q, k, v, cu_q, cu_k, max_q=1, status=st, out=out)
    assert (out == 0.5).all()
    V.attention_packed(q, k, v, cu_q, cu_k, max_q=1, out=out)
    V.op_poll()
    check_attn(out, q, k, v, list(range(n)), cu_k.tolist(), [1] * n, [lk] * n, False, d ** -0.5)


@pytest.mark.parametrize("M,N,K", [(17, 4096, 4096), (33, 4096, 2064), (100, 1000, 4096), (128, 72, 8192), (129, 2056, 1008),
                                   (257, 640, 2048), (1000, 1024, 1024), (1024, 4096, 4096), (4096, 1024, 1024), (255, 8, 160)])
def test_linear_fp8_by_every_kernel(M, N, K):
    """Sizes on both sides of the choices between the kernels; rows and columns past the ends are left."""
    V = lib()
    a, sa, w, sw, b = make_linear(M, N, K, M + K, True)
    big = torch.full((M + 3, N + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    V.linear_fp8(a, sa, w, sw, bias=b, out=big[:M, :N])
    V.op_poll()
    check_linear(big[:M, :N], a, sa, w, sw, b)
    assert (big[M:] == 7).all() and (big[:, N:] == 7).all()
    again = V.linear_fp8(a, sa, w, sw, bias=b)
    assert torch.equal(again, big[:M, :N])


@pytest.mark.parametrize("M,N,K", [(200, 1024, 4096), (3000, 512, 8192)])
def test_linear_split_and_tile_wait_expiry_is_reported(M, N, K):
    V = lib()
    a, sa, w, sw, b = make_linear(M, N, K, 25, True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    V.linear_fp8(a, sa, w, sw, status=st, wait_ns=200)
    torch.cuda.synchronize()
    assert 0x300 < int(st.item()) < 0x400
    out = torch.full((M, N), 7.0, device="cuda", dtype=torch.bfloat16)
    V.linear_fp8(a, sa, w, sw, status=st, out=out)
    assert (out == 7).all()
    V.linear_fp8(a, sa, w, sw, bias=b, out=out)
    V.op_poll()
    check_linear(out, a, sa, w, sw, b)


@pytest.mark.parametrize("rows,D", [(6000, 64), (9000, 256), (7001, 512), (5003, 1024), (6001, 2048), (3001, 4096), (2001, 8200),
                                    (1500, 16384), (5000, 1023)])
@pytest.mark.parametrize("xt", ["bf16", "fp16"])
def test_many_rows(rows, D, xt):
    """As many rows as run through the ring of copies: every row is right, quantised and normed."""
    V, g = lib(), gen(rows)
    x = randn(g, rows, D, dtype=DT[xt], scale=4.0)
    x[rows // 2] = 0
    q, s = V.quant_rows(x)
    check_rows8(q, s, x.double(), (rows, D))
    w = (1 + randn(g, D, scale=0.3)).to(DT[xt])
    for weight in (w, w.float()):
        for e4m3 in (True, False):
            out, scales, _ = V.rms_norm(x, weight, 1e-6, fp8=e4m3)
            y = x.double() / torch.sqrt(x.double().square().mean(dim=1, keepdim=True) + 1e-6) * w.double()
            if e4m3:
                check_rows8(out, scales, y, (rows, D))
            else:
                tiny = 2.0 ** -25 if xt == "fp16" else 0.0
                assert ((out.double() - y).abs() <= y.abs() * (u_of(x.dtype) + NORM32) * 1.01 + tiny).all()
    few, _, _ = V.rms_norm(x[:3], w, 1e-6)
    many, _, _ = V.rms_norm(x, w, 1e-6)
    assert ((few.double() - many[:3].double()).abs() <= 2 * u_of(x.dtype) * many[:3].double().abs()).all()


# ------------------------------------------------------------------ calls at the edges of what is allowed
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_broadcast_heads_and_tokens(kernel, d):
    """Keys and values that are one head's seen as several (a head stride of 0): right, or refused."""
    V, g = lib(), gen(40)
    q = randn(g, 70, 4, d, dtype=torch.bfloat16)
    k1, v1 = randn(g, 70, 1, d, dtype=torch.bfloat16), randn(g, 70, 1, d, dtype=torch.bfloat16)
    args = by_kernel(kernel, k1, v1, cum([30, 40]), cum([30, 40]))
    args["k"], args["v"] = args["k"].expand(-1, 2, -1), args["v"].expand(-1, 2, -1)
    try:
        out = V.attention_packed(q, **args, causal=True)
    except V.VitError as e:
        assert e.status in (V.VIT_E_CUDA, V.VIT_E_SHAPE)
        return
    V.op_poll()
    check_attn(out, q, k1.expand(-1, 2, -1), v1.expand(-1, 2, -1), [0, 30], [0, 30], [30, 40], [30, 40], True, d ** -0.5)


@pytest.mark.parametrize("kernel", KERNELS)
def test_attention_offsets_past_32_bits(kernel):
    """A cache of more than 2^31 values: the last sequence begins behind them."""
    V, g = lib(), gen(41)
    hkv, d, room = 8, 128, 2_200_000
    lens = [70, 50]
    kv = torch.empty(2, 2 * room, hkv, d, dtype=torch.bfloat16, device="cuda")
    for i, ln in enumerate(lens):
        kv[:, i * room:i * room + ln] = randn(g, 2, ln, hkv, d, dtype=torch.bfloat16)
        kv[:, i * room + ln:i * room + ln + 64] = NAN
    k, v = kv[0], kv[1]
    assert k.stride(0) * room > 1 << 31
    q = randn(g, 2, 16, d, dtype=torch.bfloat16)
    cu_q, cu_k = cum([1, 1]), cum([room, room])
    len_k = torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = dict(k=k, v=v, cu_q=cu_q, cu_k=cu_k, len_k=len_k, max_q=0 if kernel == "tile" else 1)
    if kernel == "short":
        args = by_kernel(kernel, k, v, cu_q, cu_k, len_k)
    out = V.attention_packed(q, **args, causal=True)
    V.op_poll()
    check_attn(out, q, k, v, [0, 1], [0, room], [1, 1], lens, True, d ** -0.5)


def test_rows_offsets_past_32_bits():
    """Rows of a matrix of more than 2^31 values, at its end, through the norm, rope and the 8-bit layer."""
    V, g = lib(), gen(42)
    rows, D, ld = 3, 256, 1 << 30
    big = torch.empty(2 * ld + D, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (rows, D), (ld, 1))
    x.copy_(randn(g, rows, D, dtype=torch.bfloat16))
    q, s = V.quant_rows(x)
    check_rows8(q, s, x.double(), "far rows")
    heads = torch.as_strided(big, (rows, 2, 128), (ld, 128, 1))
    pos = torch.arange(rows, device="cuda", dtype=torch.int32) + 7
    f = V.rope_freqs(10000.0, 128)
    out, _ = V.rope(heads, None, pos, f)
    check_rope(out, heads, pos, f, "half")
    del big, x, heads
    a = torch.empty(2 * ld + D, dtype=torch.uint8, device="cuda").view(E4M3)
    far = torch.as_strided(a, (rows, D), (ld, 1))
    far.copy_(q)
    w, sw = V.quant_rows(randn(g, 64, D))
    check_linear(V.linear_fp8(far, s, w, sw), q, s, w, sw, None)


def test_first_calls_inside_a_capture():
    """In a fresh process the first call of every operator may be a captured one."""
    lib()
    import os
    import subprocess
    import sys
    code = """
import torch, vision_transformer_encoder_fwd_b200 as V
bf = torch.bfloat16
x = torch.randn(40, 1024, device="cuda", dtype=bf)
w = torch.ones(1024, device="cuda", dtype=bf)
wf = torch.zeros(256, 1024, device="cuda").to(torch.float8_e4m3fn)
sw = torch.ones(256, device="cuda")
q = torch.randn(40, 4, 64, device="cuda", dtype=bf)
k = torch.randn(4000, 4, 64, device="cuda", dtype=bf)
cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
ck = torch.tensor([0, 4000], dtype=torch.int32, device="cuda")
pos = torch.arange(40, device="cuda")
f = V.rope_freqs(10000.0, 64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a, s, _ = V.rms_norm(x, w, fp8=True)
    y = V.linear_fp8(a, s, wf, sw)
    y1 = V.linear_fp8(a[:4], s[:4], wf, sw)
    r, _ = V.rope(q, None, pos, f)
    o = [V.attention_packed(r, k, k, cu, ck, max_q=m) for m in (0, 1)]
    o.append(V.attention_packed(r, k[:40], k[:40], cu, cu, max_q=40))
g.replay()
torch.cuda.synchronize()
V.op_poll()
for i, t in enumerate([y, y1, r] + o):
    assert torch.isfinite(t.float()).all(), i
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "fine" in res.stdout, res.stderr[-2000:]


@pytest.mark.parametrize("xt,rt", [("fp32", None), ("bf16", None), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,D", [(6, 7), (6, 64), (6, 1003), (6, 4096), (6, 16392), (9000, 256), (3001, 4096)])
def test_rows8_for_a_small_eps(rows, D, xt, rt):
    """Rows of zeros and of values so small that the factor which takes them to 8 bits is past fp32's range: the
    definition is finite there.  Widths and numbers of rows of each of the kernel's forms."""
    V, g = lib(), gen(50)
    dt = DT[xt]
    x = randn(g, rows, D, dtype=dt)
    x[1] = 0
    x[2] = 0
    x[2, D // 2] = 3e-19
    x[3] = (randn(g, D) * 1e-19).to(dt)
    r = None if rt is None else torch.zeros(rows, D, device="cuda", dtype=DT[rt])
    for eps in (1e-12, 1e-30):
        for scale in (1.0, 1e-18):
            w = (1 + 0.3 * torch.rand(D, generator=g, device="cuda")) * scale
            out, s, _ = V.rms_norm(x, w, eps, residual=r, fp8=True)
            xd = x.double()
            # eps as the call takes it: in fp32
            y = xd / torch.sqrt(xd.square().mean(dim=1, keepdim=True) + float(torch.tensor(eps))) * w.double()
            assert (out.float()[1] == 0).all() and s[1] == torch.tensor(2.0 ** -100 / 448)
            assert torch.isfinite(out.float()).all() and torch.isfinite(s).all()
            # h w of 1e-19 x 1e-18 is held to 2^-149 of fp32's range, relative to 1e-37 less than 2^-24
            check_rows8(out, s, y, (eps, scale))


@pytest.mark.parametrize("rows,D", [(3, 64), (3, 1003), (3, 4096), (6000, 256)])
def test_rows8_of_an_infinity(rows, D):
    """With an infinity in a row the norm's scale is NaN (0 times infinity), and so is all that is divided by it; without
    the norm the scale is infinity, finite values are 0 and the infinity NaN."""
    V, g = lib(), gen(51)
    x = randn(g, rows, D)
    x[1, D // 3] = -math.inf
    for t in (torch.float32, torch.bfloat16):
        out, s, _ = V.rms_norm(x.to(t), torch.ones(D, device="cuda"), 1e-6, fp8=True)
        assert s[1].isnan() and out.float()[1].isnan().all()
        assert torch.isfinite(out.float()[[0, 2]]).all() and torch.isfinite(s[[0, 2]]).all()
        q, s = V.quant_rows(x.to(t))
        assert torch.isinf(s[1]) and q.float()[1, D // 3].isnan()
        assert (q.float()[1, torch.arange(D, device="cuda") != D // 3] == 0).all()


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_wait_that_ran_out_leaves_other_calls_alone(kernel):
    """Without a status word of their own, calls after one whose wait ran out do their work; the poll still tells."""
    V, g = lib(), gen(52)
    n = 500
    q, k, v = (randn(g, n, 2, 128, dtype=torch.bfloat16) for _ in range(3))
    cu = cum([n])
    V.attention_packed(q, k, v, cu, cu, wait_ns=200)
    out = torch.full_like(q, 0.5)
    V.attention_packed(q, **by_kernel(kernel, k, v, cu, cu), out=out)
    lin = []
    for M in (5, 200, 2600):
        a, sa, w, sw, b = make_linear(M, 1024, 2048, 9, True)
        lin.append((V.linear_fp8(a, sa, w, sw, bias=b, out=torch.full((M, 1024), 7.0, device="cuda", dtype=torch.bfloat16)),
                    a, sa, w, sw, b))
    with pytest.raises(V.VitError) as e:
        V.op_poll()
    assert e.value.status == V.VIT_E_DEVICE_TIMEOUT
    V.op_poll()
    check_attn(out, q, k, v, [0], [0], [n], [n], False, 128 ** -0.5)
    for r in lin:
        check_linear(*r)


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", [(1, 64), (7, 64), (9, 1003), (8, 4096), (6000, 256), (3001, 4096), (2000, 1023)])
def test_rows_on_their_inputs(rows, D, xt):
    """out on x (of x's type, and 8-bit rows at the start of x's rows), few rows and as many as the ring kernel takes: the
    same bits as into memory of their own with the same strides (by which the order of a row's sum goes)."""
    V, g = lib(), gen(53)
    dt = DT[xt]
    x = randn(g, rows, D, dtype=dt)
    w = (1 + randn(g, D, scale=0.3)).to(dt)
    want = V.rms_norm(x, w, 1e-6)[0]
    apart = [torch.empty_like(x).view(torch.uint8)[:, :D].view(E4M3) for _ in range(2)]
    want8, want_s, _ = V.rms_norm(x, w, 1e-6, out=apart[0])
    wq, wqs = V.quant_rows(x, out=apart[1])
    y = x.clone()
    assert torch.equal(V.rms_norm(y, w, 1e-6, out=y)[0], want)
    for call, a, s in ((lambda x, o: V.rms_norm(x, w, 1e-6, out=o)[:2], want8, want_s),
                       (lambda x, o: V.quant_rows(x, out=o), wq, wqs)):
        y = x.clone()
        o = y.view(torch.uint8)[:, :D].view(E4M3)
        got, gs = call(y, o)
        assert got.data_ptr() == y.data_ptr() and torch.equal(got.float(), a.float()) and torch.equal(gs, s)


@pytest.mark.parametrize("what", ["kv head", "kv token", "q head", "q token"])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_reads_broadcast_heads_and_tokens(kernel, d, what):
    """A stride of 0 in q, or in k and v, is right in every kernel."""
    V, g = lib(), gen(54)
    n, hkv = 70, 2
    q = randn(g, n, 4, d, dtype=torch.bfloat16)
    k, v = randn(g, n, hkv, d, dtype=torch.bfloat16), randn(g, n, hkv, d, dtype=torch.bfloat16)
    if what == "q head":
        q = q[:, :1].expand(-1, 4, -1)
    if what == "q token":
        q = q[:1].expand(n, -1, -1)
    if what == "kv token":
        k, v = k[:1].expand(n, -1, -1), v[:1].expand(n, -1, -1)
    args = by_kernel(kernel, k, v, cum([30, 40]), cum([30, 40]))
    if what == "kv head":
        args["k"], args["v"] = (t[:, :1].expand(-1, hkv, -1) for t in (args["k"], args["v"]))
        k, v = k[:, :1].expand(-1, hkv, -1), v[:, :1].expand(-1, hkv, -1)
    if what == "kv token":
        args["k"], args["v"] = (t[:1].expand(args["k"].shape[0], -1, -1) for t in (k, v))
    out = V.attention_packed(q, **args, causal=True)
    V.op_poll()
    check_attn(out, q, k, v, [0, 30], [0, 30], [30, 40], [30, 40], True, d ** -0.5)


def test_outputs_that_overlap_are_refused():
    V, g = lib(), gen(55)
    q = randn(g, 20, 4, 64, dtype=torch.bfloat16)
    cu = cum([20])
    pos = torch.arange(20, device="cuda")
    f = V.rope_freqs(10000.0, 64)
    for shared in (torch.zeros(20, 1, 64, device="cuda", dtype=q.dtype).expand(-1, 4, -1),
                   torch.zeros(1, 4, 64, device="cuda", dtype=q.dtype).expand(20, -1, -1)):
        for call in (lambda: V.attention_packed(q, q, q, cu, cu, out=shared), lambda: V.rope(q, None, pos, f, out=(shared, None)),
                     lambda: V.rope(shared, None, pos, f, out=(shared, None))):
            with pytest.raises(V.VitError) as e:
                call()
            assert e.value.status == V.VIT_E_SHAPE
        assert (shared == 0).all()
    # read, they are fine
    x = q[:, :1].expand(-1, 4, -1)
    y, _ = V.rope(x, None, pos, f)
    check_rope(y, x, pos, f, "half")


def test_written_tensors_show_in_autograd():
    """What a call writes into counts as changed: a backward pass that saved it says so instead of using it."""
    V, g = lib(), gen(56)
    x, w = randn(g, 8, 64, dtype=torch.bfloat16), torch.ones(64, device="cuda")
    q, cu = randn(g, 8, 2, 64, dtype=torch.bfloat16), cum([8])
    pos, f = torch.arange(8, device="cuda"), V.rope_freqs(100.0, 64)
    q8, s8 = V.quant_rows(randn(g, 8, 64))
    res, out, o8, sc, k = randn(g, 8, 64), x.clone(), q8.clone(), s8.clone(), q.clone()
    o2, s2, lin, att = q8.clone(), s8.clone(), torch.zeros(8, 8, device="cuda", dtype=torch.bfloat16), q.clone()
    given = [res, out, o8, sc, q, k, o2, s2, lin, att]
    before = [t._version for t in given]
    V.rms_norm(x, w, residual=res, residual_out=res, out=out)
    V.rms_norm(x, w, out=o8, scales=sc)
    V.rope(q, k, pos, f, out=(q, k))
    V.quant_rows(x, out=o2, scales=s2)
    V.linear_fp8(q8, s8, q8, s8, out=lin)
    V.attention_packed(q, q, q, cu, cu, out=att)
    assert [t._version for t in given] == [v + 1 for v in before]
    assert x._version == 0 and q8._version == 0
    p = torch.ones(8, 64, device="cuda", requires_grad=True)
    y = (p * res).sum()  # keeps res for p's gradient
    V.rms_norm(x, w, residual=res, residual_out=res)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        frozen = torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16)
    V.rms_norm(x, w, out=frozen)  # has no version to count
    assert torch.equal(frozen, V.rms_norm(x, w)[0])


def test_rope_rounds_the_angle():
    """Angles of a few 2^-32 turns: the fraction of a turn is rounded to 2^-32, not cut, so that it is off by at most
    2^-33 turns (and the sine by two units in its last place)."""
    V = lib()
    k = torch.arange(0, 64, dtype=torch.float64)
    f = 2 * math.pi * (k + 0.75) * 2.0 ** -32
    x = torch.zeros(2, 1, 128, device="cuda")
    x[..., :64] = 1
    pos = torch.tensor([1, -1], device="cuda")
    out, _ = V.rope(x, None, pos, f)
    t = torch.stack([f, -f]).cuda()
    err = (out[:, 0, 64:].double() - torch.sin(t)).abs()
    assert (err <= 2 * math.pi * 2.0 ** -33 * 1.01 + 4 * 2.0 ** -24 * t.abs()).all(), err.max().item()


def _fresh_process(code, **env):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300,
                          env={**os.environ, **env})


EVERY_KERNEL = """
import torch, vision_transformer_encoder_fwd_b200 as V
torch.manual_seed(0)
bf, dev = torch.bfloat16, "cuda"
W = V.quant_rows(torch.randn(1024, 2048, device=dev))
xs = {M: torch.randn(M, 2048, device=dev, dtype=bf) for M in (3, 40, 300, 9000)}
res = {M: torch.randn(M, 2048, device=dev) for M in xs}
wn = torch.rand(2048, device=dev) + 0.5
k = torch.randn(5000, 2, 128, device=dev, dtype=bf)
q = torch.randn(90, 4, 128, device=dev, dtype=bf)
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
f = V.rope_freqs(10000.0, 128)
pos = torch.arange(90, device=dev)

def every():
    out = []
    for M, x in xs.items():  # rows, K split, tile and pair kernels; rows in registers and through the ring
        a, s, h = V.rms_norm(x, wn, 1e-6, residual=res[M], fp8=True)
        out += [a.float(), s, h, V.linear_fp8(a, s, *W), V.linear_fp8(*V.quant_rows(x), *W)]
    r, kr = V.rope(q, k[:90], pos, f)
    out += [r, kr, V.attention_packed(r, kr, kr, i32(0, 50, 90), i32(0, 50, 90), causal=True, max_q=0)]
    out.append(V.attention_packed(r[:2], k, k, i32(0, 1, 2), i32(0, 2500, 5000), max_q=1))
    out.append(V.attention_packed(r[:40], k[:40], k[:40], i32(0, 20, 40), i32(0, 20, 40), causal=True, max_q=20))
    return out
"""


def test_operators_without_early_starts(tmp_path):
    """Launched in plain stream order (VIT_B200_PDL=0) the operators give the same bits."""
    lib()
    for pdl in ("0", "1"):
        res = _fresh_process(EVERY_KERNEL + f"torch.save([t.cpu() for t in every()], {str(tmp_path / pdl)!r})\nV.op_poll()",
                             VIT_B200_PDL=pdl)
        assert res.returncode == 0, res.stderr[-2000:]
    a, b = (torch.load(tmp_path / p) for p in "01")
    assert len(a) == len(b) and all(torch.isfinite(x.float()).all() and torch.equal(x, y) for x, y in zip(a, b))


def test_operators_from_several_threads():
    """First calls and later ones from four threads at once, each on a stream of its own: the bits of calls one by one."""
    lib()
    res = _fresh_process(EVERY_KERNEL + """
import threading
start, bad, got = threading.Barrier(4), [], {}
torch.cuda.synchronize()

def work(me):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            got[me] = [every() for _ in range(8)]
            torch.cuda.current_stream().synchronize()
    except BaseException as e:
        bad.append(e)

threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not bad, bad
V.op_poll()
want = every()
for me, rounds in got.items():
    for r in rounds:
        assert all(torch.equal(x, y) for x, y in zip(r, want)), me
print("fine")
""")
    assert res.returncode == 0 and "fine" in res.stdout, res.stderr[-2000:]


def test_rows_and_layers_captured():
    """The norm, 8-bit rows and 8-bit layers of every size captured into one graph and replayed on new values."""
    V, g = lib(), gen(57)
    w, sw = V.quant_rows(randn(g, 1024, 2048))
    wn = 1 + randn(g, 2048, scale=0.2)
    xs = [randn(g, M, 2048, dtype=torch.bfloat16) for M in (3, 40, 300, 9000)]

    def run():
        res = []
        for x in xs:
            a, s, _ = V.rms_norm(x, wn, 1e-6, fp8=True)
            q, t = V.quant_rows(x)
            res.append((a, s, V.linear_fp8(a, s, w, sw), q, t, V.linear_fp8(q, t, w, sw)))
        return res
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for x in xs:
            x.copy_(randn(g, *x.shape, dtype=torch.bfloat16, scale=3.0))
        graph.replay()
        for a, b in zip(got, run()):
            assert all(torch.equal(x.float(), y.float()) for x, y in zip(a, b))
    V.op_poll()
