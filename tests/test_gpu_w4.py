"""afd_ffn_w4_rows and afd_ffn_w4_expert_rows against the float64 definition, and the chain
norm -> selection -> dispatch -> 4-bit experts -> combine.

Bounds, fixed before the first run (u = 2^-24).  The weights q - z and the inputs are exact in bf16
and their products exact in fp32.  A sum of K products, taken in any order with fp32 accumulators
(a tensor-core step of 16 products may truncate, 2 u a step) and scaled once per group, is within
(K / 8 + 32) u of the sum of |x| |W|: K / 16 steps of 2 u at most one after another, one product and
one addition per group of at least 32 (K / 16 u), the parts' joining (<= 32 u).
bf16 results: half a step, 2^-8 relative, more.  SwiGLU: |silu'| <= 1.1, so act is within
1.1 |u| dg + |silu(g)| du + (2^-16 + 2^-20) |act| of the exact one (two bf16 terms: 2^-16 at most;
expf, quotient and products below 2^-20), which the down product spreads by |W2|.
"""
import numpy as np
import pytest
import torch

import ffn_side_expert_b200 as afd
from oracle import moe
from oracle import operators as op

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


class W4:
    """Seeded 4-bit weights [E][N][K] on the device and as float64 on the host."""

    def __init__(self, gen, E, N, K, group, zeros=False, scales=BF16):
        self.codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=gen)
        self.scale = ((0.7 + 0.6 * torch.rand((E, N, K // group), generator=gen)) * (0.22 / K ** 0.5)).to(scales)
        self.zero = torch.randint(0, 16, (E, N, K // group), dtype=torch.uint8, generator=gen) if zeros else None
        self.group = group
        dev = [None if t is None else t.cuda() for t in (self.codes, self.scale, self.zero)]
        self.plan = afd.w4_weights(*dev, group)

    def __call__(self, e):
        return op.w4_dequant(self.codes[e].numpy(), self.scale[e].double().numpy(),
                             None if self.zero is None else self.zero[e].numpy(), self.group)


def f64(t):
    return t.double().cpu().numpy()


def rows_of(gen, n, K):
    return torch.randn((n, K), generator=gen).to(BF16)


def rows_tol(a, y, K, dtype):
    return (K / 8 + 32) * U * a + (2.0 ** -8 * np.abs(y) if dtype == BF16 else U * np.abs(y)) + 1e-38


def run_rows(w, E, x, counts, n, dtype, N, spare=3, **kw):
    y = torch.full((n + spare, N), 7.0, dtype=dtype, device="cuda")
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    assert afd.afd_ffn_w4_rows(w.plan, E, x, c, n, y, **kw) == afd.AFD_OK
    torch.cuda.synchronize()
    return y


def check_rows(w, E, x, counts, dtype, N, K):
    n = x.shape[0]
    y = run_rows(w, E, x.cuda(), counts, n, dtype, N)
    used = n if counts is None else sum(counts)
    ref, a = op.w4_rows(f64(x), w, [n] if counts is None else counts)
    err = np.abs(f64(y[:used]) - ref)
    assert (err <= rows_tol(a, ref, K, dtype)).all(), np.max(err / rows_tol(a, ref, K, dtype))
    assert (y[used:].float() == 7.0).all()
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (96, 96), (128, 128), (160, 32), (480, 96), (2080, 32), (7168, 128),
                                     (7168, 64), (7168, 7168), (1024, 1024), (18432, 128),
                                     (320, 160), (1440, 160)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_matrix(K, group, dtype):
    gen = torch.Generator().manual_seed(K + group)
    for N, n, zeros, scales in ((1, 1, False, BF16), (40, 3, True, F32), (131, 9, True, BF16), (257, 1, False, F32)):
        w = W4(gen, 1, N, K, group, zeros, scales)
        check_rows(w, 1, rows_of(gen, n, K), None, dtype, N, K)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 63, 65, 100, 200])
def test_row_counts_of_one_matrix(n):
    gen = torch.Generator().manual_seed(n)
    for group, zeros in ((32, True), (128, False)):
        w = W4(gen, 1, 200, 640, group, zeros)
        check_rows(w, 1, rows_of(gen, n, 640), None, F32, 200, 640)


@pytest.mark.parametrize("counts", [[0, 3, 0, 1], [5], [0, 0, 0], [1] * 40, [33, 0, 8, 17, 64, 2], [0, 0, 70], [0] * 255 + [2], [1] * 256])
def test_experts_with_any_rows(counts):
    gen = torch.Generator().manual_seed(len(counts))
    E, N, K = len(counts), 72, 256
    w = W4(gen, E, N, K, 64, True)
    n = sum(counts)
    if n == 0:
        y = run_rows(w, E, rows_of(gen, 4, K).cuda(), counts, 4, F32, N)
        assert (y == 7.0).all()
        return
    check_rows(w, E, rows_of(gen, n, K), counts, F32, N, K)
    # rows behind the last expert's are left as they were
    x = rows_of(gen, n + 5, K)
    y = run_rows(w, E, x.cuda(), counts, n + 5, BF16, N)
    ref, a = op.w4_rows(f64(x), w, counts)
    assert (np.abs(f64(y[:n]) - ref) <= rows_tol(a, ref, K, BF16)).all()
    assert (y[n:].float() == 7.0).all()


def test_counts_that_do_not_fit_are_flagged():
    gen = torch.Generator().manual_seed(1)
    E, N, K = 3, 64, 128
    w = W4(gen, E, N, K, 32)
    x = rows_of(gen, 6, K)
    for counts, real in (([2, -4, 1], [2, 0, 1]), ([4, 9, 2], [4, 2, 0]), ([2000000000, 2000000000, 1], [6, 0, 0])):
        y = run_rows(w, E, x.cuda(), counts, 6, F32, N)
        used = sum(real)
        ref, a = op.w4_rows(f64(x), w, real)
        assert (np.abs(f64(y[:used]) - ref) <= rows_tol(a, ref, K, F32)).all()
        assert (y[used:] == 7.0).all()
        assert afd.afd_ffn_rows_error() == afd.AFD_ERR_DEVICE_FLAG
        assert afd.afd_ffn_rows_error() == afd.AFD_OK


def test_infinities_and_nans_stay_in_their_rows():
    gen = torch.Generator().manual_seed(2)
    w = W4(gen, 2, 64, 256, 64)
    x = rows_of(gen, 11, 256)
    x[3, 5] = float("inf")
    x[7, 200] = float("nan")
    counts = [6, 5]
    y = run_rows(w, 2, x.cuda(), counts, 11, F32, 64)
    clean = x.clone()
    clean[3], clean[7] = 0, 0
    ref, a = op.w4_rows(f64(clean), w, counts)
    ok = [r for r in range(11) if r not in (3, 7)]
    assert (np.abs(f64(y[:11]) - ref) <= rows_tol(a, ref, 256, F32))[ok].all()
    assert not torch.isfinite(y[3]).any() and torch.isnan(y[7]).all()


def test_extreme_codes_and_zero_points():
    """Every code and zero point: W of one group is (q - z) exactly."""
    K = 32
    q = np.tile(np.arange(16, dtype=np.uint8), (16, 2))
    w = W4(torch.Generator().manual_seed(0), 1, 16, K, K, True, F32)
    w.codes = torch.from_numpy(op.w4_pack(q))[None]
    w.zero = torch.arange(16, dtype=torch.uint8).view(1, 16, 1) + 16 * 5      # the high four bits do not count
    w.scale = torch.ones((1, 16, 1))
    w.plan = afd.w4_weights(w.codes.cuda(), w.scale.cuda(), w.zero.cuda(), K)
    for k in range(K):                                  # a unit row reads one column of the weights
        x = torch.zeros((1, K), dtype=BF16)
        x[0, k] = 1
        y = run_rows(w, 1, x.cuda(), None, 1, F32, 16)
        assert torch.equal(y[0].cpu(), torch.from_numpy(q[:, k].astype(np.float32) - np.arange(16, dtype=np.float32)))


def test_weights_past_32_bits():
    """Codes of the last expert start more than 2^32 bytes in."""
    E, N, K = 5, 65536, 32768                            # 1 GiB of codes an expert
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    codes.fill_(0x88)
    codes[4, N - 3:] = torch.randint(0, 256, (3, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.full((E, N, K // 1024), 0.01, dtype=BF16, device="cuda")
    plan = afd.w4_weights(codes, scale, None, 1024)
    x = rows_of(torch.Generator().manual_seed(3), 1, K)
    y = torch.full((1, N), 7.0, device="cuda")
    counts = torch.tensor([0, 0, 0, 0, 1], dtype=torch.int32, device="cuda")
    assert afd.afd_ffn_w4_rows(plan, E, x.cuda(), counts, 1, y) == afd.AFD_OK
    torch.cuda.synchronize()
    w = op.w4_dequant(codes[4, N - 3:].cpu().numpy(), scale[4, N - 3:].double().cpu().numpy(), None, 1024)
    ref, a = f64(x) @ w.T, np.abs(f64(x)) @ np.abs(w).T
    assert (np.abs(f64(y[:, N - 3:]) - ref) <= rows_tol(a, ref, K, F32)).all()
    assert (y[:, :N - 3] == 0).all()


# ------------------------------------------------------------------ whole experts
def experts_tol(x, w13, w2, counts, y, H, I, dtype):
    gu, a = op.w4_rows(x, w13, counts)
    d = (H / 8 + 32) * U * a
    g, u = np.split(gu, 2, axis=1)
    dg, du = np.split(d, 2, axis=1)
    act = op.swiglu(gu)
    silu = moe.silu(g)
    dact = 1.1 * np.abs(u) * dg + np.abs(silu) * du + 1.1 * dg * du + (2.0 ** -16 + 2.0 ** -20) * np.abs(act)
    at, tol = 0, []
    for e, m in enumerate(counts):
        if m:
            aw = np.abs(w2(e)).T
            tol.append((dact[at:at + m] + (I / 8 + 32) * U * (np.abs(act[at:at + m]) + dact[at:at + m])) @ aw)
            at += m
    return np.concatenate(tol) + (2.0 ** -8 if dtype == BF16 else U) * np.abs(y) + 1e-38


@pytest.mark.parametrize("H,I,g13,g2", [(32, 32, 32, 32), (256, 512, 64, 128), (1056, 96, 32, 96), (2048, 320, 128, 64),
                                        (7168, 256, 128, 128)])
@pytest.mark.parametrize("counts", [[1], [0, 2, 0, 1], [9, 0, 40, 1], [1] * 8])
def test_experts(H, I, g13, g2, counts):
    gen = torch.Generator().manual_seed(H + I)
    E, n = len(counts), sum(counts)
    w13, w2 = W4(gen, E, 2 * I, H, g13, True), W4(gen, E, H, I, g2, False, F32)
    x = rows_of(gen, n, H)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    scratch = torch.full((afd.afd_ffn_w4_scratch_bytes(n + 2, I),), 255, dtype=torch.uint8, device="cuda")
    ref = op.w4_expert_rows(f64(x), w13, w2, counts)
    xd = torch.cat([x, x.new_full((2, H), float("nan"))]).cuda()
    for dtype in (F32, BF16):
        y = torch.full((n + 2, H), 7.0, dtype=dtype, device="cuda")
        assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, xd, c, n + 2, y, scratch) == afd.AFD_OK
        torch.cuda.synchronize()
        tol = experts_tol(f64(x), w13, w2, counts, ref, H, I, dtype)
        err = np.abs(f64(y[:n]) - ref)
        assert (err <= tol).all(), np.max(err / tol)
        assert (y[n:].float() == 7.0).all()
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


def test_experts_with_large_gates():
    """Gates far beyond expf's range: silu is 0 or the gate itself, never NaN."""
    gen = torch.Generator().manual_seed(9)
    H, I = 64, 64
    w13, w2 = W4(gen, 1, 2 * I, H, 32), W4(gen, 1, H, I, 32)
    x = (rows_of(gen, 4, H).float() * 1000).to(BF16)
    y = torch.empty((4, H), device="cuda")
    scratch = torch.empty((afd.afd_ffn_w4_scratch_bytes(4, I),), dtype=torch.uint8, device="cuda")
    assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, 1, x.cuda(), None, 4, y, scratch) == afd.AFD_OK
    torch.cuda.synchronize()
    ref = op.w4_expert_rows(f64(x), w13, w2, [4])
    assert (np.abs(f64(y) - ref) <= experts_tol(f64(x), w13, w2, [4], ref, H, I, F32)).all()


def test_same_bits_every_time_on_any_stream_and_in_graphs():
    """Two captured graphs with a scratch each, replayed together on two streams, and plain calls in between."""
    gen = torch.Generator().manual_seed(10)
    E, H, I, counts = 6, 512, 256, [3, 0, 20, 1, 9, 2]
    n = sum(counts)
    w13, w2 = W4(gen, E, 2 * I, H, 64), W4(gen, E, H, I, 64)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    xs = [rows_of(gen, n, H).cuda() for _ in range(2)]
    size = afd.afd_ffn_w4_scratch_bytes(n, I)
    scratch = [torch.empty((size,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want, ys, graphs, streams = [], [], [], []
    for i in range(2):
        y = torch.empty((n, H), dtype=BF16, device="cuda")
        assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, xs[i], c, n, y, scratch[i]) == afd.AFD_OK
        want.append(y)
    torch.cuda.synchronize()
    for i in range(2):
        s = torch.cuda.Stream()
        y = torch.zeros((n, H), dtype=BF16, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, xs[i], c, n, y, scratch[i]) == afd.AFD_OK
        ys.append(y); graphs.append(graph); streams.append(s)
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])


def test_a_row_does_not_depend_on_the_rows_beside_it():
    """Row by row gives the bits of one call, except that the split of the sums may go by the row count:
    within twice the sums' bound."""
    gen = torch.Generator().manual_seed(11)
    K, N = 1024, 96
    w = W4(gen, 1, N, K, 128)
    x = rows_of(gen, 20, K).cuda()
    whole = run_rows(w, 1, x, None, 20, F32, N)[:20]
    a = np.abs(f64(x)) @ np.abs(w(0)).T
    for r in range(20):
        one = run_rows(w, 1, x[r:r + 1].contiguous(), None, 1, F32, N)[:1]
        assert (np.abs(f64(one - whole[r:r + 1])) <= 2 * (K / 8 + 32) * U * a[r]).all()


@pytest.mark.parametrize("K,group,scales", [(4096, 256, BF16), (2048, 512, F32), (2560, 128, F32), (1024, 32, F32),
                                            (1536, 64, BF16), (2048, 1024, BF16)])
@pytest.mark.parametrize("n", [1, 4, 6, 13])
def test_groups_in_whole_pieces(K, group, scales, n):
    """Rows of scales that 16-byte pieces cover, and the same weights with scales and zero points that start
    four bytes later, which are read group by group: equal bits."""
    gen = torch.Generator().manual_seed(K + group + n)
    N = 144
    w = W4(gen, 1, N, K, group, True, scales)
    x = rows_of(gen, n, K)
    check_rows(w, 1, x, None, F32, N, K)
    want = run_rows(w, 1, x.cuda(), None, n, F32, N)
    off = 4 // w.scale.element_size()
    scale = torch.empty((w.scale.numel() + off,), dtype=scales, device="cuda")[off:].view(w.scale.shape)
    zero = torch.empty((w.zero.numel() + 4,), dtype=torch.uint8, device="cuda")[4:].view(w.zero.shape)
    scale.copy_(w.scale)
    zero.copy_(w.zero)
    w.plan = afd.w4_weights(w.codes.cuda(), scale, zero, group)
    assert torch.equal(run_rows(w, 1, x.cuda(), None, n, F32, N), want)


@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_few_and_many_rows_in_one_call(group):
    """Weights large enough that experts with few rows and with many go to kernels of their own."""
    gen = torch.Generator().manual_seed(group)
    E, N, K, counts = 8, 2304, 4096, [3, 16, 0, 17, 8, 1, 70, 9]
    w = W4(gen, E, N, K, group, group != 64)
    n = sum(counts)
    check_rows(w, E, rows_of(gen, n, K), counts, F32, N, K)
    few = [2, 0, 4, 1, 0, 0, 8, 1]                       # every expert in few rows: units of 64 and 32 rows
    check_rows(w, E, rows_of(gen, sum(few), K), few, F32, N, K)
    ones = [1, 0, 0, 4, 0, 0, 0, 0]
    check_rows(w, E, rows_of(gen, sum(ones), K), ones, BF16, N, K)


@pytest.mark.parametrize("counts", [[1, 0, 9, 4, 33, 8, 2, 5], [1] * 8])
def test_large_experts_with_few_and_many_rows(counts):
    gen = torch.Generator().manual_seed(12)
    E, H, I, n = 8, 4096, 2304, sum(counts)
    w13, w2 = W4(gen, E, 2 * I, H, 128, True), W4(gen, E, H, I, 64)
    x = rows_of(gen, n, H)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    scratch = torch.empty((afd.afd_ffn_w4_scratch_bytes(n, I),), dtype=torch.uint8, device="cuda")
    ref = op.w4_expert_rows(f64(x), w13, w2, counts)
    tol = experts_tol(f64(x), w13, w2, counts, ref, H, I, F32)
    first = None
    for _ in range(3):
        y = torch.full((n, H), 7.0, device="cuda")
        assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, x.cuda(), c, n, y, scratch) == afd.AFD_OK
        torch.cuda.synchronize()
        assert (np.abs(f64(y) - ref) <= tol).all()
        assert first is None or torch.equal(first, y)
        first = y
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


def test_two_calls_at_once():
    """Calls on two streams over the same weights, each with rows and scratch of its own."""
    gen = torch.Generator().manual_seed(13)
    E, H, I, counts = 4, 1024, 512, [2, 20, 0, 5]
    n = sum(counts)
    w13, w2 = W4(gen, E, 2 * I, H, 32, True), W4(gen, E, H, I, 128)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    xs = [rows_of(gen, n, H).cuda() for _ in range(2)]
    scratch = [torch.empty((afd.afd_ffn_w4_scratch_bytes(n, I),), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [torch.zeros((n, H), dtype=BF16, device="cuda") for _ in range(4)]
    call = lambda i, y, **kw: afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, xs[i], c, n, y, scratch[i], **kw)  # noqa: E731
    for i in range(2):
        assert call(i, ys[i]) == afd.AFD_OK
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        for i in range(2):
            assert call(i, ys[2 + i], stream=streams[i]) == afd.AFD_OK
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[2]) and torch.equal(ys[1], ys[3])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_norm_selection_experts_and_combine_together(T):
    """The FFN half of a layer with 4-bit experts, on device data only, against the float64 chain (the
    selection's indices taken from the device, their scores held against the definition)."""
    gen = torch.Generator().manual_seed(20 + T)
    H, I, E, k, eps = 512, 256, 32, 4, 1e-6
    x, res = torch.randn((T, H), generator=gen).to(BF16).cuda(), torch.randn((T, H), generator=gen).cuda()
    gamma = (1 + 0.1 * torch.randn((H,), generator=gen)).cuda()
    wr = (torch.randn((E, H), generator=gen) / H ** 0.5).cuda()
    bias = (0.05 * torch.randn((E,), generator=gen)).cuda()
    w13, w2 = W4(gen, E, 2 * I, H, 128, True), W4(gen, E, H, I, 64)
    r = dict(sigmoid=True, n_groups=4, topk_groups=2, group_best=2, renormalise=True, weight_scale=2.5)

    total, hidden, out = torch.empty_like(res), torch.empty_like(x), torch.empty_like(x)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")                  # noqa: E731
    idx, w, counts, offsets, pos, src = i32(T, k), torch.empty((T, k), device="cuda"), i32(E), i32(E + 1), i32(T, k), i32(T * k)
    rows, Y = torch.empty((T * k, H), dtype=BF16, device="cuda"), torch.empty((T * k, H), device="cuda")
    scratch_d = i32(2 * ((T + 127) // 128) * E)
    scratch_w = torch.empty((afd.afd_ffn_w4_scratch_bytes(T * k, I),), dtype=torch.uint8, device="cuda")
    cfg = afd.afd_ffn_norm_cfg(T=T, H=H, residual_dtype=afd.AFD_DT_F32, gamma_dtype=afd.AFD_DT_F32, eps=eps)
    route = afd.afd_ffn_routing(score=1, n_groups=4, topk_groups=2, group_best=2, renormalise=1, weight_scale=2.5)

    ok = afd.AFD_OK
    assert afd.afd_ffn_add_rmsnorm(cfg, x, res, gamma, total, hidden) == ok
    logits = hidden.float() @ wr.T
    assert afd.afd_ffn_select_experts(logits, bias, T, E, k, route, idx, w) == ok
    assert afd.afd_ffn_dispatch_rows(hidden, idx, T, k, E, H, counts, offsets, pos, src, rows, scratch_d) == ok
    assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, rows, counts, T * k, Y, scratch_w) == ok
    assert afd.afd_ffn_combine_rows(Y, None, w, pos, T, k, H, out) == ok
    torch.cuda.synchronize()
    assert afd.afd_ffn_rows_error() == ok

    s, y, _ = op.add_rmsnorm(f64(x), f64(res), f64(gamma), eps)
    assert (np.abs(f64(total) - s) <= U * np.abs(s) * (1 + 1e-6)).all()
    assert (np.abs(f64(hidden) - y) <= (2.0 ** -8 + 33 * U) * np.abs(y)).all()
    ri, rw = op.select_experts(f64(logits), f64(bias), k, **r)
    assert np.array_equal(idx.cpu().numpy(), ri)
    h = f64(hidden)                                    # what the device's experts read
    order = np.argsort(ri.reshape(-1), kind="stable")
    cnt = np.bincount(ri.reshape(-1), minlength=E).tolist()
    xr = h[order // k]
    ref_rows = op.w4_expert_rows(xr, w13, w2, cnt)
    tol_rows = experts_tol(xr, w13, w2, cnt, ref_rows, H, I, F32)
    yr, tr = np.empty_like(ref_rows), np.empty_like(ref_rows)
    yr[order], tr[order] = ref_rows, tol_rows
    yr, tr = yr.reshape(T, k, H), tr.reshape(T, k, H)
    ref = (rw[:, :, None] * yr).sum(1)
    # the rows' own error, the weights' (64 u), the sum's (k + 1 steps), half a bf16 step
    tol = (rw[:, :, None] * (tr + (64 + k + 1) * U * np.abs(yr))).sum(1) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(f64(out) - ref) <= tol).all()


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("counts", [[0, 0, 64, 0, 0], [64, 0, 0, 0], [17, 1, 30, 16], [20, 0, 0, 0, 33, 0, 1, 9], [13, 19],
                                    [0, 32, 0], [33, 0, 32], [0, 65, 0, 0], [32], [33]])
@pytest.mark.parametrize("N,K", [(88, 512), (1208, 2048)])
def test_few_columns_over_several_tiles(group, counts, N, K):
    """Calls of at most 64 columns, and of one more, with experts of up to all of them."""
    gen = torch.Generator().manual_seed(group + sum(counts))
    E, n = len(counts), sum(counts)
    w = W4(gen, E, N, K, group, group != 64)
    x = rows_of(gen, n, K)
    check_rows(w, E, x, counts, F32, N, K)
    # counts that do not fit the rows are flagged; the rows stay in bounds
    y = run_rows(w, E, x[:-1].cuda(), [c + 1 for c in counts], n - 1, F32, N)
    assert afd.afd_ffn_rows_error() != afd.AFD_OK
    assert (y[n - 1:] == 7.0).all()
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


# ------------------------------------------------------------------ split units, one after another in a block
def scattered(gen, shape, dtype, span=6):
    """Scales that differ by up to 2^(2 span) from row to row and group to group."""
    return (torch.exp2((2 * span) * torch.rand(shape, generator=gen) - span) / 64).to(dtype)


def off_a_piece(t, n):
    """The same values, contiguous, n elements behind a 16-byte boundary: scales like these are read one by one."""
    to = torch.empty((t.numel() + n,), dtype=t.dtype, device="cuda")[n:].view(t.shape)
    return to.copy_(t)


@pytest.mark.parametrize("group,scales,zeros", [(32, F32, True), (32, BF16, False), (64, F32, False), (128, F32, True),
                                                (128, BF16, True), (256, F32, False)])
def test_split_units_one_after_another(group, scales, zeros):
    """Three tokens, units of 128 weight rows, two a block, each split by K over the block's warpgroups: with
    32 or 16 steps a unit, 2 rounds of a share (8 or 6 steps) cost less than whole units or ones of 64 or 32 rows.
    A share that ends inside K must not ask for scales behind it: they would land, in no order, where the next
    unit's first ones go.  The scales read in pieces give the bits of the scales read one by one, and the
    definition's values (evaluated on the device in 64 bits)."""
    gen = torch.Generator().manual_seed(group)
    K = 4096
    N = 2 * 128 * torch.cuda.get_device_properties(0).multi_processor_count - 40
    codes = torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, generator=gen).cuda()
    scale = scattered(gen, (1, N, K // group), scales).cuda()
    zero = torch.randint(0, 16, scale.shape, dtype=torch.uint8, generator=gen).cuda() if zeros else None
    x = rows_of(gen, 3, K).cuda()
    one_by_one = afd.w4_weights(codes, off_a_piece(scale, 4 // scale.element_size()),
                                None if zero is None else off_a_piece(zero, 4), group)
    pieces = afd.w4_weights(codes, scale, zero, group)

    q = torch.stack((codes[0] & 15, codes[0] >> 4), 2).view(N, K // group, group).double()
    z = 8.0 if zero is None else zero[0].double()[:, :, None]
    w = ((q - z) * scale[0].double()[:, :, None]).view(N, K)
    ref, a = f64(x.double() @ w.T), f64(x.double().abs() @ w.abs().T)
    want = torch.empty((3, N), device="cuda")
    assert afd.afd_ffn_w4_rows(one_by_one, 1, x, None, 3, want) == afd.AFD_OK
    assert (np.abs(f64(want) - ref) <= rows_tol(a, ref, K, F32)).all()
    ys = [torch.full((3, N), 7.0, device="cuda") for _ in range(10)]
    for y in ys:
        assert afd.afd_ffn_w4_rows(pieces, 1, x, None, 3, y) == afd.AFD_OK
    assert all(torch.equal(y, want) for y in ys)
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


@pytest.mark.parametrize("group", [32, 128])
def test_split_units_of_a_whole_expert(group):
    """The same in the down product (rows of two bf16 terms, moved by cp.async) of a dense expert."""
    gen = torch.Generator().manual_seed(group + 1)
    I = 4096
    H = 2 * 128 * torch.cuda.get_device_properties(0).multi_processor_count - 128
    made = []
    for N, K in ((2 * I, H), (H, I)):
        codes = torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, generator=gen).cuda()
        scale = (scattered(gen, (1, N, K // group), F32, 3) * K ** -0.5).cuda()
        made.append((afd.w4_weights(codes, scale, None, group), afd.w4_weights(codes, off_a_piece(scale, 1), None, group)))
    x = rows_of(gen, 3, H).cuda()
    scratch = torch.empty((afd.afd_ffn_w4_scratch_bytes(3, I),), dtype=torch.uint8, device="cuda")
    want = torch.empty((3, H), device="cuda")
    assert afd.afd_ffn_w4_expert_rows(made[0][1], made[1][1], 1, x, None, 3, want, scratch) == afd.AFD_OK
    ys = [torch.full((3, H), 7.0, device="cuda") for _ in range(10)]
    for y in ys:
        assert afd.afd_ffn_w4_expert_rows(made[0][0], made[1][0], 1, x, None, 3, y, scratch) == afd.AFD_OK
    assert torch.isfinite(want).all() and all(torch.equal(y, want) for y in ys)
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


def test_swiglu_value_above_the_last_bf16():
    """A SwiGLU value of 3.4e38 is an fp32 number but rounds to an infinite bf16: its two terms stay finite.
    gate = 2^64, up = 3.4e38 / 2^64, a down weight of 2^-64 beside zeros."""
    act = float(np.float32(3.4e38))
    codes = lambda q: torch.from_numpy(op.w4_pack(q))[None].cuda()                     # noqa: E731
    q13, q2 = np.full((64, 32), 8, np.uint8), np.full((32, 32), 8, np.uint8)
    q13[0, 0] = q13[32, 0] = 9
    q2[5, 0] = 9
    s13 = torch.ones((1, 64, 1), device="cuda")
    s13[0, 0], s13[0, 32] = 2.0 ** 64, act * 2.0 ** -64
    w13 = afd.w4_weights(codes(q13), s13, None, 32)
    w2 = afd.w4_weights(codes(q2), torch.full((1, 32, 1), 2.0 ** -64, device="cuda"), None, 32)
    for n in (1, 40):                                    # few columns, and many
        x = torch.zeros((n, 32), dtype=BF16, device="cuda")
        x[:, 0] = 1
        y = torch.full((n, 32), 7.0, device="cuda")
        scratch = torch.empty((afd.afd_ffn_w4_scratch_bytes(n, 32),), dtype=torch.uint8, device="cuda")
        assert afd.afd_ffn_w4_expert_rows(w13, w2, 1, x, None, n, y, scratch) == afd.AFD_OK
        ref = np.zeros((n, 32))
        ref[:, 5] = act * 2.0 ** -64
        assert (np.abs(f64(y) - ref) <= 2.0 ** -16 * ref).all()


# ------------------------------------------------------------------ calls that follow one another at once
@pytest.mark.parametrize("captured", [False, True])
def test_calls_that_nothing_waits_between(captured):
    """Whole experts with few and with many rows, two kernels a product, on one scratch: the rows come from a
    norm and the counts from a copy just before, other rows and counts of another call follow at once, and what
    the call read and its scratch are overwritten behind it.  Each call's results are those of a call alone."""
    gen = torch.Generator().manual_seed(14)
    E, H, I, rounds = 6, 2048, 1600, 12
    w13, w2 = W4(gen, E, 2 * I, H, 128, True), W4(gen, E, H, I, 64)
    lots = [[70, 3, 0, 20, 1, 9], [1, 0, 40, 2, 60, 0], [0, 103, 0, 0, 0, 0]]
    n = 103
    counts = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in lots]
    xs = [rows_of(gen, n, H).cuda() for _ in lots]
    gamma = (1 + 0.2 * torch.randn((H,), generator=gen)).cuda()
    cfg = afd.afd_ffn_norm_cfg(T=n, H=H, residual_dtype=afd.AFD_DT_BF16, gamma_dtype=afd.AFD_DT_F32, eps=1e-6)
    rows, now = torch.empty((n, H), dtype=BF16, device="cuda"), torch.empty((E,), dtype=torch.int32, device="cuda")
    scratch = torch.empty((afd.afd_ffn_w4_scratch_bytes(n, I),), dtype=torch.uint8, device="cuda")

    def one(i, y):
        now.copy_(counts[i])
        assert afd.afd_ffn_add_rmsnorm(cfg, xs[i], None, gamma, None, rows) == afd.AFD_OK
        assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, rows, now, n, y, scratch) == afd.AFD_OK

    want = []
    for i in range(3):
        y = torch.full((n, H), 7.0, device="cuda")
        torch.cuda.synchronize()
        one(i, y)
        torch.cuda.synchronize()
        want.append(y)
        used = sum(lots[i])
        ref = op.w4_expert_rows(f64(rows[:used]), w13, w2, lots[i])
        tol = experts_tol(f64(rows[:used]), w13, w2, lots[i], ref, H, I, F32)
        assert (np.abs(f64(y[:used]) - ref) <= tol).all() and (y[used:] == 7.0).all()
    ys = [torch.full((n, H), 7.0, device="cuda") for _ in range(rounds)]

    def chain():
        for r, y in enumerate(ys):
            one(r % 3, y)
            if r % 2:                                    # else the next call's own kernels follow
                scratch.fill_(255)
                rows.fill_(float("nan"))
                now.fill_(-1)

    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            chain()
        for _ in range(3):
            graph.replay()
    else:
        chain()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[r % 3]) for r, y in enumerate(ys))
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


# ------------------------------------------------------------------ as many rows as a prompt has
@pytest.mark.parametrize("group,zeros,scales", [(32, True, F32), (64, False, BF16), (128, True, BF16), (256, False, F32)])
def test_thousands_of_rows(group, zeros, scales):
    gen = torch.Generator().manual_seed(group + 7)
    N, K = 328, 512
    w = W4(gen, 1, N, K, group, zeros, scales)
    check_rows(w, 1, rows_of(gen, 5001, K), None, F32, N, K)
    E, counts = 7, [1500, 0, 17, 2049, 1, 64, 900]
    w = W4(gen, E, N, K, group, zeros, scales)
    check_rows(w, E, rows_of(gen, sum(counts), K), counts, BF16, N, K)


@pytest.mark.parametrize("H,I,counts", [(256, 128, [4096] * 15 + [4095]), (1024, 384, [2900, 0, 1, 33, 5, 700, 0, 16]),
                                        (512, 2048, [0, 0, 3000])])
def test_experts_with_thousands_of_rows(H, I, counts):
    gen = torch.Generator().manual_seed(H + len(counts))
    E, n = len(counts), sum(counts)
    w13, w2 = W4(gen, E, 2 * I, H, 128, True), W4(gen, E, H, I, 64, False, F32)
    x = rows_of(gen, n, H)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    scratch = torch.empty((afd.afd_ffn_w4_scratch_bytes(n, I),), dtype=torch.uint8, device="cuda")
    ref = op.w4_expert_rows(f64(x), w13, w2, counts)
    y = torch.full((n, H), 7.0, device="cuda")
    assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, x.cuda(), c, n, y, scratch) == afd.AFD_OK
    torch.cuda.synchronize()
    assert (np.abs(f64(y) - ref) <= experts_tol(f64(x), w13, w2, counts, ref, H, I, F32)).all()
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


@pytest.mark.parametrize("T", [3, 70])
def test_tokens_with_no_expert_left(T):
    """Selection, dispatch, 4-bit experts and combine where masks leave a token fewer experts than k, or none: the
    empty slots are skipped and flagged, the rows behind the last expert's are nobody's, and a token with no
    expert gets zeros."""
    gen = torch.Generator().manual_seed(30 + T)
    H, I, E, k = 256, 128, 8, 4
    hidden = torch.randn((T, H), generator=gen).to(BF16).cuda()
    logits = torch.randn((T, E), generator=gen)
    logits[0] = float("-inf")
    logits[1, 2:] = torch.finfo(F32).min                  # the type's lowest value is a number: chosen last
    logits[2, 1:] = float("nan")
    w13, w2 = W4(gen, E, 2 * I, H, 64, True), W4(gen, E, H, I, 32)
    r = dict(sigmoid=False, n_groups=1, topk_groups=1, group_best=1, renormalise=True, weight_scale=1.0)
    route = afd.afd_ffn_routing(score=0, n_groups=1, topk_groups=1, group_best=1, renormalise=1, weight_scale=1.0)
    i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")               # noqa: E731
    idx, w, counts, offsets, pos, src = i32(T, k), torch.empty((T, k), device="cuda"), i32(E), i32(E + 1), i32(T, k), i32(T * k)
    rows = torch.full((T * k, H), float("nan"), dtype=BF16, device="cuda")
    Y, out = torch.full((T * k, H), float("nan"), device="cuda"), torch.full((T, H), 7.0, dtype=BF16, device="cuda")
    scratch_d = i32(2 * ((T + 127) // 128) * E)
    scratch_w = torch.empty((afd.afd_ffn_w4_scratch_bytes(T * k, I),), dtype=torch.uint8, device="cuda")
    ok = afd.AFD_OK
    assert afd.afd_ffn_select_experts(logits.cuda(), None, T, E, k, route, idx, w) == ok
    assert afd.afd_ffn_dispatch_rows(hidden, idx, T, k, E, H, counts, offsets, pos, src, rows, scratch_d) == ok
    assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, rows, counts, T * k, Y, scratch_w) == ok
    assert afd.afd_ffn_combine_rows(Y, None, w, pos, T, k, H, out) == ok
    torch.cuda.synchronize()
    assert afd.afd_ffn_rows_error() == afd.AFD_ERR_DEVICE_FLAG          # the slots without an expert
    assert afd.afd_ffn_rows_error() == ok
    ri, rw = op.select_experts(logits.double().numpy(), None, k, **r)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert (ri[0] == -1).all() and (ri[2] == [0, -1, -1, -1]).all() and (ri[1] >= 0).all()
    used = int((ri >= 0).sum())
    assert torch.isnan(Y[used:]).all() and torch.isfinite(Y[:used]).all()
    flat = ri.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:used]
    cnt = np.bincount(flat[flat >= 0], minlength=E).tolist()
    assert counts.tolist() == cnt
    xr = f64(hidden)[order // k]
    ref_rows = op.w4_expert_rows(xr, w13, w2, cnt)
    yr, tr = np.zeros((T * k, H)), np.zeros((T * k, H))
    yr[order], tr[order] = ref_rows, experts_tol(xr, w13, w2, cnt, ref_rows, H, I, F32)
    yr, tr = yr.reshape(T, k, H), tr.reshape(T, k, H)
    ref = (rw[:, :, None] * yr).sum(1)
    tol = (rw[:, :, None] * (tr + (64 + k + 1) * U * np.abs(yr))).sum(1) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(f64(out) - ref) <= tol).all() and (out[0] == 0).all()


# ------------------------------------------------------------------ the ends of the ranges
def test_rows_and_results_past_32_bits():
    """The most rows that are taken, with more than 2^31 inputs and more than 2^31 results."""
    gen = torch.Generator().manual_seed(40)
    n, K, N, E = 1 << 22, 544, 520, 3
    w = W4(gen, E, N, K, 32, True, F32)
    counts = [n - 70, 0, 65]
    x = torch.zeros((n, K), dtype=BF16, device="cuda")
    at = [0, 63, 64, (1 << 31) // K, (1 << 31) // K + 1, (1 << 31) // N, n - 71, n - 70, n - 6]
    some = rows_of(gen, len(at), K)
    x[at] = some.cuda()
    y = torch.full((n, N), 7.0, device="cuda")
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    assert afd.afd_ffn_w4_rows(w.plan, E, x, c, n, y) == afd.AFD_OK
    torch.cuda.synchronize()
    ref, a = op.w4_rows(f64(some), w, [7, 0, 2])
    assert (np.abs(f64(y[at]) - ref) <= rows_tol(a, ref, K, F32)).all()
    assert (y[n - 5:] == 7.0).all() and (y[(1 << 31) // N + 1: n - 71] == 0).all()
    assert afd.afd_ffn_rows_error() == afd.AFD_OK


def test_scratch_past_32_bits():
    """SwiGLU rows with more than 2^31 terms between the two products."""
    gen = torch.Generator().manual_seed(41)
    n, H, I = (1 << 21) + 33, 64, 544
    w13, w2 = W4(gen, 1, 2 * I, H, 32), W4(gen, 1, H, I, 32, True)
    x = torch.zeros((n, H), dtype=BF16, device="cuda")
    at = [0, (1 << 31) // (2 * I) - 1, (1 << 31) // (2 * I), (1 << 31) // (2 * I) + 1, n - 1]
    some = rows_of(gen, len(at), H)
    x[at] = some.cuda()
    y = torch.full((n, H), 7.0, device="cuda")
    scratch = torch.empty((afd.afd_ffn_w4_scratch_bytes(n, I),), dtype=torch.uint8, device="cuda")
    assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, 1, x, None, n, y, scratch) == afd.AFD_OK
    torch.cuda.synchronize()
    ref = op.w4_expert_rows(f64(some), w13, w2, [len(at)])
    assert (np.abs(f64(y[at]) - ref) <= experts_tol(f64(some), w13, w2, [len(at)], ref, H, I, F32)).all()
    assert (y[1:1000] == 0).all()


def test_captured_behind_a_fork_and_a_join():
    """A graph in which the norm and the selection run on streams of their own and the experts wait for both:
    kernels that may start early behind more than one other."""
    gen = torch.Generator().manual_seed(42)
    T, H, I, E, k = 24, 512, 256, 8, 2
    x = torch.randn((T, H), generator=gen).to(BF16).cuda()
    logits = torch.randn((T, E), generator=gen).cuda()
    gamma = torch.ones((H,), device="cuda")
    w13, w2 = W4(gen, E, 2 * I, H, 128, True), W4(gen, E, H, I, 64)
    cfg = afd.afd_ffn_norm_cfg(T=T, H=H, residual_dtype=afd.AFD_DT_BF16, gamma_dtype=afd.AFD_DT_F32, eps=1e-6)
    route = afd.afd_ffn_routing(score=1, n_groups=1, topk_groups=1, group_best=1, renormalise=1, weight_scale=1.0)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")                  # noqa: E731
    hidden, out = torch.zeros_like(x), torch.zeros_like(x)
    idx, w, counts, offsets, pos, src = i32(T, k), torch.zeros((T, k), device="cuda"), i32(E), i32(E + 1), i32(T, k), i32(T * k)
    rows, Y = torch.zeros((T * k, H), dtype=BF16, device="cuda"), torch.zeros((T * k, H), device="cuda")
    scratch_d = i32(2 * E)
    scratch_w = torch.zeros((afd.afd_ffn_w4_scratch_bytes(T * k, I),), dtype=torch.uint8, device="cuda")
    dense, scratch_s = torch.zeros((T, H), device="cuda"), torch.zeros((afd.afd_ffn_w4_scratch_bytes(T, I),), dtype=torch.uint8, device="cuda")
    ok = afd.AFD_OK

    def layer(main, side):
        side.wait_stream(main)
        assert afd.afd_ffn_select_experts(logits, None, T, E, k, route, idx, w, stream=side) == ok
        assert afd.afd_ffn_add_rmsnorm(cfg, x, None, gamma, None, hidden, stream=main) == ok
        main.wait_stream(side)
        assert afd.afd_ffn_add_rmsnorm(cfg, hidden, None, gamma, None, hidden, stream=main) == ok      # behind both
        side.wait_stream(main)
        one = afd.afd_ffn_w4(w13.plan.codes, w13.plan.scale, w13.plan.zero, 2 * I, H, 128, afd.AFD_DT_BF16)
        two = afd.afd_ffn_w4(w2.plan.codes, w2.plan.scale, w2.plan.zero, H, I, 64, afd.AFD_DT_BF16)
        assert afd.afd_ffn_w4_expert_rows(one, two, 1, hidden, None, T, dense, scratch_s, stream=side) == ok
        assert afd.afd_ffn_dispatch_rows(hidden, idx, T, k, E, H, counts, offsets, pos, src, rows, scratch_d, stream=main) == ok
        assert afd.afd_ffn_w4_expert_rows(w13.plan, w2.plan, E, rows, counts, T * k, Y, scratch_w, stream=main) == ok
        main.wait_stream(side)
        assert afd.afd_ffn_combine_rows(Y, dense, w, pos, T, k, H, out, stream=main) == ok

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    layer(main, side)
    torch.cuda.synchronize()
    want, wi = out.clone(), idx.clone()
    assert torch.isfinite(want).all() and want.abs().max() > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        layer(main, side)
    for t in (hidden, out, idx, w, rows, Y, dense):
        t.zero_()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(idx, wi)
    assert afd.afd_ffn_rows_error() == ok
