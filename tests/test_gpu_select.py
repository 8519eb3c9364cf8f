"""afd_ffn_select_experts and afd_ffn_set_routing against the float64 definition.

idx is compared exactly.  Bounds of w, fixed before the first run (u = 2^-24): a sigmoid is within
6 u; a softmax term exp(l - top) within 4 u + u |l - top| <= 20 u for |l - top| <= 16, its sum 13 u
more; renormalising adds 5 + 1 u and the terms' own share, the scale 1 u.  Together under 50 u,
taken as 64 u relative, with 1e-37 for weights near fp32's smallest.
"""
import math

import numpy as np
import pytest
import torch

import ffn_side_expert_b200 as afd
import synth
from ffn_side_expert_b200.service import FfnService, Mailbox
from layer_support import BF16_TOL, FP8_TOL, Layer, rel_max_err, to64
from oracle import moe
from oracle import operators as op

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
PLAIN = dict(sigmoid=False, n_groups=1, topk_groups=1, group_best=1, renormalise=True, weight_scale=1.0)


def routing(r):
    return afd.afd_ffn_routing(score=int(r["sigmoid"]), n_groups=r["n_groups"], topk_groups=r["topk_groups"],
                               group_best=r["group_best"], renormalise=int(r["renormalise"]), weight_scale=r["weight_scale"])


def select(logits, bias, k, r, **kw):
    T, E = logits.shape
    idx = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 99.0, device="cuda")
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).cuda()
    st = afd.afd_ffn_select_experts(logits, b, T, E, k, routing(r), idx, w, **kw)
    assert st == afd.AFD_OK
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.double().cpu().numpy()


def check(logits, bias, k, r):
    idx, w = select(logits, bias, k, r)
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).double().numpy()
    ri, rw = op.select_experts(logits.double().cpu().numpy(), b, k, **r)
    assert np.array_equal(idx, ri), np.argwhere(idx != ri)[:5]
    assert (np.abs(w - rw) <= 64 * U * rw + 1e-37).all(), np.max(np.abs(w - rw) / np.maximum(rw, 1e-37))


@pytest.mark.parametrize("E,k,groups,keep", [
    (1, 1, 1, 1), (2, 2, 1, 1), (7, 3, 1, 1), (33, 4, 1, 1), (64, 32, 1, 1), (256, 8, 1, 1), (256, 32, 1, 1),
    (256, 8, 8, 4), (160, 6, 8, 3), (96, 5, 3, 2), (66, 4, 22, 7), (256, 8, 32, 4), (32, 2, 32, 2), (250, 3, 5, 1),
    (24, 4, 4, 4)])
@pytest.mark.parametrize("sigmoid,renorm", [(False, False), (False, True), (True, False), (True, True)])
def test_against_the_definition(E, k, groups, keep, sigmoid, renorm):
    gen = torch.Generator().manual_seed(E * 31 + k)
    for n, (T, biased, best) in enumerate(((1, True, 2), (37, False, 2), (65, True, 1), (9, False, 1))):
        wide = torch.randn((T, E + 5 * (n % 2)), generator=gen) * 1.5
        logits = wide.cuda()[:, :E]
        bias = 0.1 * torch.randn((E,), generator=gen) if biased else None
        r = dict(sigmoid=sigmoid, n_groups=groups, topk_groups=keep, group_best=best, renormalise=renorm, weight_scale=1.0 + n)
        check(logits, bias, k, r)
        if best == 1 or groups == 1:   # coarse logits: sums of two could be equal but for their rounding
            check(logits.to(torch.bfloat16), bias, k, r)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_ties_go_to_the_lower_index(sigmoid):
    logits = torch.zeros((3, 64), device="cuda")
    logits[1, 10:] = 1.0
    logits[2, 5] = -0.0
    for groups, keep in ((1, 1), (8, 2)):
        for bias in (None, torch.zeros(64), torch.full((64,), 0.25)):
            check(logits, bias, 6, {**PLAIN, "sigmoid": sigmoid, "n_groups": groups, "topk_groups": keep, "group_best": 2})


@pytest.mark.parametrize("sigmoid", [False, True])
def test_choices_closer_than_fp32(sigmoid):
    """Choices that differ by about 1e-9, far less than an fp32 score resolves: the order is still that of
    64 bits.  The bias brings every choice next to one value; its own fp32 rounding spreads them."""
    rng = np.random.default_rng(6)
    T, E = 1, 48
    for trial in range(40):
        l = rng.normal(size=(T, E)).astype(np.float32)
        s = np.array(op.scores(l[0].tolist(), sigmoid)[1])
        bias = (0.7 - s).astype(np.float32)                       # s + bias = 0.7 +- 3e-8
        r = dict(PLAIN, sigmoid=sigmoid, n_groups=1 if trial % 2 else 4, topk_groups=1 if trial % 2 else 2, group_best=2)
        check(torch.from_numpy(l).cuda(), torch.from_numpy(bias), 8, r)


def test_group_sums_closer_than_fp32():
    """Groups whose two best sigmoid scores add up to nearly the same: no bias, sums of two."""
    rng = np.random.default_rng(7)
    for _ in range(40):
        a = rng.uniform(0.2, 0.6, size=4)
        p = np.stack([0.6 + a / 2, 0.6 - a / 2], 1)               # each pair sums to 1.2
        l = np.log(p / (1 - p)).reshape(1, 8).astype(np.float32)
        check(torch.from_numpy(l).cuda(), None, 3, dict(PLAIN, sigmoid=True, n_groups=4, topk_groups=2, group_best=2))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_experts_out_of_service(sigmoid, biased):
    gen = torch.Generator().manual_seed(8)
    logits = torch.randn((8, 32), generator=gen)
    inf, nan = math.inf, math.nan
    logits[0] = -inf                                  # nothing is left
    logits[1, 1:] = -inf                              # one expert
    logits[2, ::2] = nan
    logits[3, 4] = inf
    logits[4, 4] = logits[4, 20] = inf
    logits[5, :24] = -inf                             # whole groups out
    logits[6, 3] = 3e38
    logits[7] = nan
    bias = 0.1 * torch.randn((32,), generator=gen) if biased else None
    if biased:
        bias[9], bias[10] = -inf, nan
    for groups, keep, best in ((1, 1, 1), (4, 2, 2), (4, 3, 1), (16, 3, 2)):
        for renorm in (False, True):
            check(logits.cuda(), bias, 6, dict(sigmoid=sigmoid, n_groups=groups, topk_groups=keep, group_best=best,
                                               renormalise=renorm, weight_scale=2.0))


@pytest.mark.parametrize("at", [-100.0, -60.0, -39.0, 30.0])
def test_far_logits(at):
    """Scores near the ends of fp32: renormalised weights keep their ratios."""
    gen = torch.Generator().manual_seed(9)
    logits = (at + torch.rand((17, 40), generator=gen)).cuda()
    for sigmoid in (False, True):
        check(logits, None, 5, dict(PLAIN, sigmoid=sigmoid))


def test_many_tokens():
    gen = torch.Generator().manual_seed(10)
    logits = torch.randn((3001, 256), generator=gen)
    bias = 0.05 * torch.randn((256,), generator=gen)
    check(logits.cuda(), bias, 8, dict(sigmoid=True, n_groups=8, topk_groups=4, group_best=2, renormalise=True, weight_scale=2.5))
    check(logits.to(torch.bfloat16).cuda(), None, 8, PLAIN)


def test_logit_offsets_past_32_bits():
    far = (1 << 31) + 3
    buf = torch.empty((far + 64,), dtype=torch.bfloat16, device="cuda")
    logits = buf.as_strided((2, 64), (far, 1))
    logits.copy_(torch.randn((2, 64), generator=torch.Generator().manual_seed(11)).to(torch.bfloat16))
    check(logits, None, 4, PLAIN)


def test_nothing_behind_the_last_token_and_graph_replay():
    gen = torch.Generator().manual_seed(12)
    logits = torch.randn((5, 64), generator=gen).cuda()
    idx = torch.full((7, 4), 99, dtype=torch.int32, device="cuda")
    w = torch.full((7, 4), 99.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            assert afd.afd_ffn_select_experts(logits, None, 5, 64, 4, routing(PLAIN), idx, w) == afd.AFD_OK
    logits.neg_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    ri, _ = op.select_experts(logits.double().cpu().numpy(), None, 4, **PLAIN)
    assert np.array_equal(idx[:5].cpu().numpy(), ri) and (idx[5:] == 99).all() and (w[5:] == 99).all()


# ------------------------------------------------------------------ on a handle
@pytest.mark.parametrize("T", [64, 37, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_handle_routes_as_told(T, biased):
    """afd_ffn_route and afd_ffn_forward with a routing set.  The router's logits are within 1e-5 of the
    float64 ones, so a token is compared where no decision is nearer than 1e-4 (for scores of slope at most
    1, and sums of two); the seeds leave most tokens."""
    cfg = synth.MoEConfig("routed", T=64, H=256, E=16, k=2, I=128, S=1, seed=41)
    L = Layer(cfg, redraws={})
    try:
        r = dict(sigmoid=True, n_groups=4, topk_groups=2, group_best=2, renormalise=True, weight_scale=2.5)
        bias = torch.linspace(-0.2, 0.2, 16) if biased else None
        dbias = None if bias is None else bias.cuda()
        T0 = L.h[:T].contiguous()
        plain = torch.empty_like(T0)
        L.mod.forward(T0, plain)
        L.mod.set_routing(routing(r), dbias)
        idx = torch.empty((T, 2), dtype=torch.int32, device="cuda")
        w = torch.empty((T, 2), device="cuda")
        L.mod.route(T0, T, idx, w)
        out = torch.empty_like(T0)
        L.mod.forward(T0, out)
        torch.cuda.synchronize()
        assert L.mod.get_error() == afd.AFD_OK
        logits = moe.router_logits(L.hidden[:T], L.Wr, L.bias)
        b = None if bias is None else bias.double().numpy()
        ri, rw = op.select_experts(logits, b, 2, **r)
        clear = []
        for t in range(T):
            c = np.array(op.select_token(logits[t].tolist(), b, 2, **r)[2])
            worth = np.sort([np.sort(c[4 * g:4 * g + 4])[-2:].sum() for g in range(4)])
            kept = np.sort(np.concatenate([c[4 * g:4 * g + 4] for g in range(4)
                                           if np.sort(c[4 * g:4 * g + 4])[-2:].sum() >= worth[2]]))[::-1]
            clear.append(worth[2] - worth[1] > 1e-4 and kept[0] - kept[1] > 1e-4 and kept[1] - kept[2] > 1e-4)
        clear = np.array(clear)
        assert clear.sum() >= T // 2
        assert np.array_equal(idx.cpu().numpy()[clear], ri[clear])
        assert np.abs(w.double().cpu().numpy() - rw)[clear].max() <= 2.5 * 2e-5
        ref = L.oracle(tokens=np.arange(T), routing=(idx.cpu().numpy(), w.double().cpu().numpy()))["out"]
        got = out.double().cpu().numpy()
        assert np.abs(got - ref).max() <= 2e-2 * np.sqrt(np.mean(ref ** 2))
        L.mod.set_routing(None)                       # back to the softmax top-k, bit for bit
        again = torch.empty_like(T0)
        L.mod.forward(T0, again)
        torch.cuda.synchronize()
        assert torch.equal(plain, again)
    finally:
        L.close()


def test_set_routing_refuses_what_the_handle_cannot():
    cfg = synth.MoEConfig("routed", T=8, H=256, E=16, k=4, I=128, S=0, seed=42)
    L = Layer(cfg, redraws={})
    try:
        for kw in (dict(n_groups=3), dict(n_groups=8, topk_groups=1), dict(score=5)):
            r = routing(PLAIN)
            for name, v in kw.items():
                setattr(r, name, v)
            with pytest.raises(afd.AfdError):
                L.mod.set_routing(r)
        assert afd.afd_ffn_set_routing(L.mod.h, None, 4096) == afd.AFD_ERR_INVALID_ARG
    finally:
        L.close()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k", [(40, 8), (256, 8), (256, 32)])
def test_more_equal_choices_than_lanes(sigmoid, E, k):
    """Equal logits, biases a few 1e-9 apart: every expert is a candidate."""
    rng = np.random.default_rng(11)
    for trial in range(4):
        logits = torch.full((3, E), 0.25)
        logits[1, : E // 2] = -3.0
        bias = torch.from_numpy((0.3 + 1e-9 * rng.normal(size=E)).astype(np.float32))
        r = dict(PLAIN, sigmoid=sigmoid, n_groups=1 if trial % 2 else 4, topk_groups=1 if trial % 2 else 4)
        check(logits.cuda(), bias, k, r)


@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
def test_logits_that_differ_in_their_last_bits(groups, keep):
    """fp32 logits next to one another, in every order and with equal ones among them."""
    rng = np.random.default_rng(12)
    for at in (1.0, -1.0, 1e-3, -77.0):
        base = np.float32(at).view(np.int32)
        l = (base + rng.integers(0, 24, size=(40, 64))).astype(np.int32).view(np.float32)
        check(torch.from_numpy(l.copy()).cuda(), None, 9, dict(PLAIN, n_groups=groups, topk_groups=keep))


@pytest.mark.parametrize("top", [-39.5, -30.0, -5.0, 0.5, 20.0])
def test_sigmoid_scores_far_below_the_best(top):
    """Renormalised weights of scores whose 1 + exp(-l) overflows beside one that is less far down: they keep
    their ratio.  Bound: exp(l - a) with |l - a| < 64 is within 32 u (half a step of l - a) and expf's 4 u, the
    factor exp(a) / sum within 4 + 16 + 1 u, two products 2 u: 59 u, taken as 64 u, and 1e-37 as above."""
    l = torch.tensor([[top, -79.0, -85.0, -88.5, -89.0, -91.0, -95.0, -100.0],
                      [-100.0, -99.0, top, -90.0, top, -80.5, -81.0, -88.8]])
    for scale in (1.0, 2.5):
        check(l.cuda(), None, 8, dict(PLAIN, sigmoid=True, weight_scale=scale))


GROUPED = dict(sigmoid=True, n_groups=4, topk_groups=2, group_best=2, renormalise=True, weight_scale=2.5)


def clear_tokens(logits, bias, k, r, margin=1e-4):
    """Tokens whose groups and choices are decided by more than `margin` (4 groups, the best two of each)."""
    got = []
    for l in logits:
        c = np.array(op.select_token(l.tolist(), bias, k, **r)[2]).reshape(4, -1)
        worth = np.sort(c, 1)[:, -2:].sum(1)
        kept = np.sort(c[worth >= np.sort(worth)[2]].reshape(-1))[::-1][: k + 1]
        got.append(np.sort(worth)[2] - np.sort(worth)[1] > margin and (kept[:-1] - kept[1:]).min() > margin)
    return np.array(got)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 64, 700])
def test_forward_under_a_routing(dtype, T):
    """Both kinds of weights, small and large micro-batches: the layer's output is that of the experts and
    weights that afd_ffn_route reports, and those are the definition's where the logits' error (1e-5, as above)
    cannot matter."""
    cfg = synth.MoEConfig("routed", T=T, H=256, E=16, k=2, I=128, S=1, seed=43, dtype=dtype)
    L = Layer(cfg, redraws={})
    try:
        bias = torch.linspace(-0.2, 0.2, 16)
        L.mod.set_routing(routing(GROUPED), bias.cuda())
        idx, w = L.route()
        got = to64(L.forward())
        assert L.mod.get_error() == afd.AFD_OK
        b = bias.double().numpy()
        logits = moe.router_logits(L.hidden, L.Wr, L.bias)
        ri, rw = op.select_experts(logits, b, 2, **GROUPED)
        clear = clear_tokens(logits, b, 2, GROUPED)
        assert clear.sum() >= T // 2
        assert np.array_equal(idx.cpu().numpy()[clear], ri[clear])
        assert np.abs(w.double().cpu().numpy() - rw)[clear].max(initial=0) <= 2.5 * 2e-5
        some = np.arange(T)[:: max(1, T // 64)]
        ref = L.oracle(tokens=some, routing=(idx.cpu().numpy(), w.double().cpu().numpy()))["out"]
        # the bars of the layer tests, times the weights' own scale
        assert rel_max_err(got[some], ref) <= (FP8_TOL if dtype == "fp8" else BF16_TOL)
    finally:
        L.close()


def test_a_captured_forward_keeps_its_routing():
    """A graph captured under one routing, replayed after another was set and the caller's bias is gone."""
    cfg = synth.MoEConfig("routed", T=48, H=256, E=16, k=2, I=128, S=1, seed=44)
    L = Layer(cfg, redraws={})
    try:
        def both(stream=None):
            i = torch.zeros((48, 2), dtype=torch.int32, device="cuda")
            w, out = torch.zeros((48, 2), device="cuda"), torch.zeros_like(L.h)
            return (i, w, out), lambda: (L.mod.route(L.h, 48, i, w, stream), L.mod.forward(L.h, out, stream=stream))
        plain, call = both()
        call()
        L.mod.set_routing(routing(GROUPED), torch.linspace(0.2, -0.2, 16, device="cuda"))
        want, call = both()
        call()
        torch.cuda.synchronize()
        assert not torch.equal(plain[0], want[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        captured, call = both(s)
        with torch.cuda.graph(graph, stream=s):
            call()
        L.mod.set_routing(None)
        junk = [torch.full((16,), 9.0 * n, device="cuda") for n in range(64)]    # what a freed bias would become
        again, call = both()
        call()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert len(junk) == 64
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
        assert all(torch.equal(a, b) for a, b in zip(again, plain))
    finally:
        L.close()


def test_a_service_serves_under_the_routing_that_was_set():
    cfg = synth.MoEConfig("routed", T=32, H=256, E=16, k=2, I=128, S=1, seed=45)
    L = Layer(cfg, redraws={})
    try:
        L.mod.set_routing(routing(GROUPED), torch.linspace(0.2, -0.2, 16, device="cuda"))
        want = L.forward().cpu()
        mb = Mailbox(2, 32, 256)
        svc = FfnService(L.mod, mb)
        try:
            for slot, rows in ((0, 32), (1, 7)):
                mb.write_input(slot, L.hidden[:rows])
                mb.post(slot, rows)
            got = []
            for slot, rows in ((0, 32), (1, 7)):
                mb.wait(slot, 60.0)
                got.append(mb.output(slot)[:rows].clone())
        finally:
            stats = svc.stop()
            mb.close()
        assert stats.status == afd.AFD_OK and stats.device_status == afd.AFD_OK
        assert torch.equal(got[0], want)
        assert torch.equal(got[1], L.forward(T=7).cpu())
    finally:
        L.close()


def test_stage_events_around_a_routing():
    """Timing events between the stages, the router's two among them: the same output, and times in order."""
    cfg = synth.MoEConfig("routed", T=64, H=256, E=16, k=2, I=128, S=1, seed=46)
    L = Layer(cfg, redraws={})
    try:
        L.mod.set_routing(routing(GROUPED), torch.linspace(0.2, -0.2, 16, device="cuda"))
        want = L.forward()
        events = [torch.cuda.Event(enable_timing=True) for _ in range(afd.AFD_FFN_NUM_STAGES + 1)]
        for e in events:
            e.record()                                   # so that they exist
        torch.cuda.synchronize()
        L.mod.set_stage_events(events)
        got = [L.forward() for _ in range(3)]
        torch.cuda.synchronize()
        L.mod.set_stage_events([])
        assert all(torch.equal(g, want) for g in got)
        assert all(a.elapsed_time(b) >= 0 for a, b in zip(events, events[1:]))
    finally:
        L.close()


def test_tokens_past_32_bits():
    """More than 2^31 logits and more than 2^31 / 4 results."""
    E, k = 8, 2
    T = (1 << 28) + 77
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 28) - 1, 1 << 28, T - 1]
    some = torch.randn((len(at), E), generator=torch.Generator().manual_seed(13)).to(torch.bfloat16)
    logits[at] = some.cuda()
    idx = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 99.0, device="cuda")
    assert afd.afd_ffn_select_experts(logits, None, T, E, k, routing(PLAIN), idx, w) == afd.AFD_OK
    torch.cuda.synchronize()
    ri, rw = op.select_experts(some.double().numpy(), None, k, **PLAIN)
    assert np.array_equal(idx[at].cpu().numpy(), ri)
    assert (np.abs(w[at].double().cpu().numpy() - rw) <= 64 * U * rw).all()
    assert (idx[1: 1000] == torch.tensor([0, 1], device="cuda")).all() and int(idx.max()) < E and float(w.max()) <= 1
