"""afd_ffn_add_rmsnorm against the float64 definition.

Bounds, fixed before the first run.  u = 2^-24 is half a step of fp32, relative.
  sum   fp32: one correctly rounded addition of two values; bf16: half a step of bf16, 2^-8, on top.
  y     the sum of H squares adds at most 32 terms in a thread, 5 + 5 between lanes and warps, each a
        step u of a sum of positive terms, 2 more for the square of the rounded s and 1 for the
        multiply-add: 45 u; mean, + eps, reciprocal root halves that: 23 u + 3 u; two products 2 u,
        s itself 1 u: 29 u, taken as 32 u.
  out   + half a step of bf16 (2^-8, relative).
  scale 32 u + 2 u (the product and the quotient), taken as 40 u.
  codes |code * scale - y| <= half an e4m3 step (2^-4 of |y|, or 2^-10 of the scale below the
        normal range) + 80 u |y|.
"""
import math

import numpy as np
import pytest
import torch

import ffn_side_expert_b200 as afd
import synth
from layer_support import FP8_TOL, Layer, rel_max_err
from oracle import moe
from oracle import operators as op

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
DT = {BF16: afd.AFD_DT_BF16, F32: afd.AFD_DT_F32}


def f64(t):
    return t.double().cpu().numpy()


def strided(T, H, pad, dtype, gen=None, scale=1.0, fill=7.0):
    """[T][H] rows of a wider buffer; the gaps hold `fill`."""
    base = torch.full((T, H + pad), fill, dtype=dtype, device="cuda")
    rows = base[:, :H]
    if gen is not None:
        rows.copy_((scale * torch.randn((T, H), generator=gen)).to(dtype))
    return base, rows


def call(x, r, g, total, out, codes, scale, eps=1e-6, **kw):
    T, H = x.shape
    st = lambda t: t.stride(0) if t is not None and T > 1 else 0                # noqa: E731
    cfg = afd.afd_ffn_norm_cfg(T=T, H=H, residual_dtype=DT[r.dtype] if r is not None else 0, gamma_dtype=DT[g.dtype],
                               x_stride=st(x), residual_stride=st(r), sum_stride=st(total), out_stride=st(out), eps=eps)
    assert afd.afd_ffn_add_rmsnorm(cfg, x, r, g, total, out, codes, scale, **kw) == afd.AFD_OK


def check(x, r, g, total, out, codes, scale, eps=1e-6):
    s, y, sc = op.add_rmsnorm(f64(x), f64(r) if r is not None else None, f64(g), eps)
    if total is not None:
        half = 2.0 ** -8 if total.dtype == BF16 else 0.0
        assert (np.abs(f64(total) - s) <= np.abs(s) * (U + half) * (1 + 1e-6)).all()
    if out is not None:
        assert (np.abs(f64(out) - y) <= np.abs(y) * (2.0 ** -8 + 33 * U) + 1e-38).all()
    if codes is not None:
        assert (np.abs(f64(scale) - sc) <= 40 * U * sc).all()
        got = f64(codes.float()) * f64(scale)[:, None]
        step = np.maximum(np.abs(y) * 2.0 ** -4, sc[:, None] * 2.0 ** -10)
        assert (np.abs(got - y) <= step * (1 + 80 * U) + 80 * U * np.abs(y)).all()


@pytest.mark.parametrize("H", [1, 7, 8, 100, 256, 1001, 4097, 7168, 8200, 16383, 32768])
@pytest.mark.parametrize("rdt,gdt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_sizes_and_types(H, rdt, gdt):
    gen = torch.Generator().manual_seed(H)
    for T, pad in ((1, 0), (5, 0), (3, 8), (4, 3)):
        _, x = strided(T, H, pad, BF16, gen)
        _, r = strided(T, H, pad, rdt, gen, 3.0)
        g = (1 + 0.3 * torch.randn((H,), generator=gen)).to(gdt).cuda()
        sb, total = strided(T, H, pad, rdt)
        ob, out = strided(T, H, pad, BF16)
        codes = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.zeros((T,), device="cuda")
        call(x, r, g, total, out, codes, scale)
        check(x, r, g, total, out, codes, scale)
        for b in (sb, ob):                                      # the gaps between rows stay as they were
            assert (b[:, H:].float() == 7.0).all()


@pytest.mark.parametrize("parts", ["out", "codes", "sum+out", "no residual"])
def test_optional_parts(parts):
    gen = torch.Generator().manual_seed(3)
    T, H = 9, 640
    _, x = strided(T, H, 0, BF16, gen)
    _, r = strided(T, H, 0, BF16, gen)
    g = torch.randn((H,), generator=gen).cuda()
    out = torch.empty((T, H), dtype=BF16, device="cuda") if parts != "codes" else None
    codes = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda") if parts == "codes" else None
    scale = torch.empty((T,), device="cuda") if parts == "codes" else None
    total = torch.empty_like(r) if parts == "sum+out" else None
    r = None if parts == "no residual" else r
    call(x, r, g, total, out, codes, scale)
    check(x, r, g, total, out, codes, scale)


@pytest.mark.parametrize("H", [77, 2048])
def test_in_place(H):
    gen = torch.Generator().manual_seed(4)
    _, x = strided(6, H, 0, BF16, gen)
    _, r = strided(6, H, 0, BF16, gen)
    g = torch.ones((H,), device="cuda")
    x0, r0 = x.clone(), r.clone()
    call(x, r, g, r, x, None, None)              # sum over the residual, out over x
    check(x0, r0, g, r, x, None, None)


def test_special_rows():
    """A zero row (scale 1, codes 0), rows with an infinity or a NaN: only those rows are affected."""
    T, H = 6, 512
    gen = torch.Generator().manual_seed(5)
    _, x = strided(T, H, 0, BF16, gen)
    x[1] = 0
    x[2, 17] = math.inf
    x[4, 300] = math.nan
    g = torch.ones((H,), device="cuda")
    out = torch.empty((T, H), dtype=BF16, device="cuda")
    codes = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((T,), device="cuda")
    call(x, None, g, None, out, codes, scale)
    assert scale[1] == 1 and (out[1] == 0).all() and (codes[1].float() == 0).all()
    assert torch.isnan(out[2, 17]) and (out[2, :17] == 0).all() and torch.isnan(codes[2].float()[17])
    assert torch.isnan(out[4]).all() and torch.isnan(codes[4].float()).all()
    ok = [0, 3, 5]
    check(x[ok], None, g, None, out[ok], codes[ok], scale[ok])


def test_unaligned_pointers():
    """Buffers that start on odd elements take the element path."""
    T, H = 4, 264
    gen = torch.Generator().manual_seed(6)
    x = torch.randn((T * H + 1,), generator=gen).to(BF16).cuda()[1:].view(T, H)
    r = torch.randn((T * H + 1,), generator=gen).cuda()[1:].view(T, H)
    g = torch.randn((H + 1,), generator=gen).to(BF16).cuda()[1:]
    total = torch.empty((T * H + 1,), device="cuda")[1:].view(T, H)
    out = torch.empty((T * H + 1,), dtype=BF16, device="cuda")[1:].view(T, H)
    codes = torch.empty((T * H + 1,), dtype=torch.uint8, device="cuda")[1:].view(torch.float8_e4m3fn).view(T, H)
    scale = torch.empty((T + 1,), device="cuda")[1:]
    call(x, r, g, total, out, codes, scale)
    check(x, r, g, total, out, codes, scale)


def test_row_offsets_past_32_bits():
    H, far = 264, (1 << 31) + 16                 # the second row starts 2^31 + 16 elements in
    buf = torch.empty((far + H,), dtype=BF16, device="cuda")
    x = buf.as_strided((2, H), (far, 1))
    gen = torch.Generator().manual_seed(7)
    x.copy_(torch.randn((2, H), generator=gen).to(BF16))
    g = torch.ones((H,), device="cuda")
    out = torch.empty((2, H), dtype=BF16, device="cuda")
    call(x, None, g, None, out, None, None)
    check(x, None, g, None, out, None, None)


def test_stream_and_graph():
    gen = torch.Generator().manual_seed(8)
    T, H = 33, 1024
    _, x = strided(T, H, 0, BF16, gen)
    _, r = strided(T, H, 0, BF16, gen)
    g = torch.randn((H,), generator=gen).cuda()
    out, total = torch.zeros_like(x), torch.zeros_like(r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(x, r, g, total, out, None, None)
    torch.cuda.synchronize()
    assert (out == 0).all()
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    check(x, r, g, total, out, None, None)
    again = torch.zeros_like(out)
    call(x, r, g, total, again, None, None, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


@pytest.mark.parametrize("H", [8, 33, 100, 1001, 1032, 4097, 4096, 5000, 7168, 8192, 8200, 9001])
@pytest.mark.parametrize("rdt,gdt", [(BF16, F32), (F32, BF16)])
def test_many_rows(H, rdt, gdt):
    """Rows enough to fill the SMs many times take other shapes of the kernel."""
    gen = torch.Generator().manual_seed(H)
    T = 300
    for pad in (0, 3):
        _, x = strided(T, H, pad, BF16, gen)
        _, r = strided(T, H, pad, rdt, gen, 3.0)
        g = (1 + 0.3 * torch.randn((H,), generator=gen)).to(gdt).cuda()
        sb, total = strided(T, H, pad, rdt)
        ob, out = strided(T, H, pad, BF16)
        codes = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.zeros((T,), device="cuda")
        call(x, r, g, total, out, codes, scale)
        check(x, r, g, total, out, codes, scale)
        for b in (sb, ob):
            assert (b[:, H:].float() == 7.0).all()


@pytest.mark.parametrize("H", [1024, 1025])
@pytest.mark.parametrize("unit", [1.0, 2.0 ** -90, 2.0 ** -105, 2.0 ** 90, 2.0 ** 110])
def test_codes_are_those_of_the_quotient(H, unit):
    """With s = +-1 and eps = 0 the factor is 1 and y is gamma itself: each code is that of gamma / scale,
    rounded to fp32 first as a division rounds it, over rows of many sizes."""
    gen = torch.Generator().manual_seed(H)
    sign = (torch.randint(0, 2, (1, H), generator=gen) * 2 - 1).to(BF16)
    for _ in range(20):
        g = (torch.randn((H,), generator=gen) * 2.0 ** torch.randint(-12, 1, (H,), generator=gen)).float() * unit
        codes = torch.zeros((1, H), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.zeros((1,), device="cuda")
        call(sign.cuda(), None, g.cuda(), None, None, codes, scale, eps=0.0)
        y, s = (sign[0].float() * g), scale.cpu()
        assert s[0] == (g.abs().max() / 448.0)
        assert torch.equal(codes[0].cpu().float(), (y / s).clamp(-448, 448).to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("H", [513, 700, 1001, 2046, 4097, 8185, 32767])
@pytest.mark.parametrize("rdt,gdt", [(BF16, F32), (F32, BF16)])
def test_rows_of_any_start_into_contiguous_outputs(H, rdt, gdt):
    """Inputs with gaps of any size, outputs without: rows start anywhere; gamma one element off a boundary."""
    gen = torch.Generator().manual_seed(H)
    for T, pad in ((1, 0), (19, 0), (19, 1), (9, 5), (300 if H < 5000 else 12, 13)):
        _, x = strided(T, H, pad, BF16, gen)
        _, r = strided(T, H, pad + 2, rdt, gen, 3.0)
        g = torch.ones((H + 1,), dtype=gdt, device="cuda")[1:]
        g.copy_((1 + 0.3 * torch.randn((H,), generator=gen)).to(gdt))
        room = lambda dt: torch.full((T * H + 16,), 7.0, device="cuda").to(dt)                      # noqa: E731
        sb, ob, cb = room(rdt), room(BF16), room(torch.float8_e4m3fn)
        total, out, codes = (t[:T * H].view(T, H) for t in (sb, ob, cb))
        scale = torch.zeros((T,), device="cuda")
        call(x, r, g, total, out, codes, scale)
        check(x, r, g, total, out, codes, scale)
        call(x, None, g, None, out, None, None)
        check(x, None, g, None, out, None, None)
        for b in (sb, ob, cb):                                  # nothing behind the last row
            assert (b[T * H:].float() == 7.0).all()


@pytest.mark.parametrize("H", [1001, 7001])
@pytest.mark.parametrize("rdt", [BF16, F32])
def test_in_place_rows_of_any_start(H, rdt):
    gen = torch.Generator().manual_seed(9)
    for T in (7, 400):
        x = torch.randn((T, H), generator=gen).to(BF16).cuda()
        r = torch.randn((T, H), generator=gen).to(rdt).cuda()
        g = torch.ones((H,), device="cuda")
        x0, r0 = x.clone(), r.clone()
        call(x, r, g, r, x, None, None)
        check(x0, r0, g, r, x, None, None)


@pytest.mark.parametrize("H", [256, 257, 513, 1024])
def test_codes_of_rows_next_to_nothing(H):
    """max |y| of 2^-149, whose 448th part is no fp32 number: the scale stays above zero, so the zeros of the
    row have code 0 and not that of 0 / 0.  y: x gamma = 2^-133 1e-5 rounds to 2^-149, and the factor is 1."""
    for T in (1, 300):
        x = torch.zeros((T, H), dtype=BF16, device="cuda")
        x[:, H // 2] = 2.0 ** -133
        g = torch.full((H,), 1e-5, device="cuda")
        codes = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.zeros((T,), device="cuda")
        call(x, None, g, None, None, codes, scale, eps=1.0)
        got = f64(codes.float()) * f64(scale)[:, None]
        assert (f64(scale) > 0).all() and np.isfinite(got).all()
        assert (got[:, H // 2] == 2.0 ** -149).all() and np.count_nonzero(got) == T


@pytest.mark.parametrize("H", [8201, 9001, 16001, 24001, 32753, 32767])
def test_scales_of_wide_rows_of_any_start(H):
    """The derivation above counts at most 32 squares a thread: so too in the shifted form's longest rows.  The
    row scale is the one fp32 result that shows the factor: within 34 u (32 u, the product and the quotient)."""
    gen = torch.Generator().manual_seed(H)
    for T in (3, 300):
        _, x = strided(T, H, 1, BF16, gen)
        _, r = strided(T, H, 3, F32, gen, 3.0)
        g = torch.ones((H,), device="cuda")
        codes = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.zeros((T,), device="cuda")
        call(x, r, g, None, None, codes, scale)
        check(x, r, g, None, None, codes, scale)
        want = op.add_rmsnorm(f64(x), f64(r), f64(g), 1e-6)[2]
        assert (np.abs(f64(scale) - want) <= 34 * U * want).all()


def test_codes_feed_a_dense_w8a8_expert():
    """Codes and scales as they come, in token order, into an expert that takes every row (a dense FFN or a
    replicated shared expert): against the definition of the expert on the dequantised rows."""
    T, H, I = 40, 512, 256
    cfg = synth.MoEConfig("dense", T=T, H=H, E=1, k=1, I=I, S=0, seed=51, dtype="fp8")
    L = Layer(cfg, redraws={})
    try:
        gen = torch.Generator().manual_seed(52)
        _, x = strided(T, H, 0, BF16, gen)
        _, r = strided(T, H, 0, BF16, gen)
        g = (1 + 0.2 * torch.randn((H,), generator=gen)).cuda()
        total, codes = torch.empty_like(r), torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        scale, Y = torch.empty((T,), device="cuda"), torch.empty((T, H), dtype=BF16, device="cuda")
        call(x, r, g, total, None, codes, scale)
        counts = torch.tensor([T], dtype=torch.int32, device="cuda")
        assert afd.afd_ffn_expert_rows_fp8(L.mod.h, codes, scale, counts, T, Y) == afd.AFD_OK
        torch.cuda.synchronize()
        assert L.mod.get_error() == afd.AFD_OK
        check(x, r, g, total, None, codes, scale)
        w13, w2 = moe.expert_weights_f64(L.expert_fn(0))
        ref = moe.swiglu_ffn(f64(codes.float()) * f64(scale)[:, None], w13, w2, quant_act=True)[0]
        assert rel_max_err(f64(Y), ref) <= FP8_TOL
    finally:
        L.close()


@pytest.mark.parametrize("H", [16384, 16385])
def test_outputs_past_32_bits(H):
    """More than 2^31 elements in the rows that are read and written, on 16-byte boundaries and off them."""
    T = (1 << 31) // H + 200
    x = torch.empty((T, H), dtype=BF16, device="cuda")
    out, codes = torch.empty_like(x), torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((T,), device="cuda")
    g = torch.ones((H,), device="cuda")
    gen = torch.Generator().manual_seed(H)
    rows = [0, 1, (1 << 31) // H - 1, (1 << 31) // H, (1 << 31) // H + 1, T - 1]
    x.zero_()
    for r in rows:
        x[r] = torch.randn((H,), generator=gen).to(BF16)
    call(x, None, g, None, out, codes, scale)
    torch.cuda.synchronize()
    check(x[rows], None, g, None, out[rows], codes[rows], scale[rows])
    empty = torch.ones((T,), dtype=torch.bool)
    empty[rows] = False
    assert (scale.cpu()[empty] == 1).all() and float(out[2:100].abs().max()) == 0
