"""Host-side refusals of the norm, the expert selection and the 4-bit products (CPU: no call here
reaches the device)."""
import ctypes
import math
import weakref

import pytest
import torch

import ffn_side_expert_b200 as afd

A = 4096          # a 16-byte aligned stand-in address, never used
BAD, NO, OK = afd.AFD_ERR_INVALID_ARG, afd.AFD_ERR_UNSUPPORTED, afd.AFD_OK


def _norm(x=A, residual=A, gamma=A, sum=A, out=A, codes=A, scale=A, **kw):
    base = dict(T=4, H=256, residual_dtype=afd.AFD_DT_BF16, gamma_dtype=afd.AFD_DT_BF16, eps=1e-6)
    base.update(kw)
    return afd.afd_ffn_add_rmsnorm(afd.afd_ffn_norm_cfg(**base), x, residual, gamma, sum, out, codes, scale)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(H=0), BAD), (dict(H=32769), NO), (dict(residual_dtype=afd.AFD_DT_FP8_E4M3), BAD),
    (dict(gamma_dtype=9), BAD), (dict(eps=-1e-6), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD),
    (dict(x_stride=255), BAD), (dict(residual_stride=-256), BAD), (dict(sum_stride=1), BAD), (dict(out_stride=255), BAD),
    (dict(x=None), BAD), (dict(gamma=None), BAD), (dict(residual=None), BAD),      # sum without a residual
    (dict(out=None, codes=None, scale=None), BAD), (dict(scale=None), BAD), (dict(codes=None), BAD),
    (dict(x=A + 1), BAD), (dict(residual=A + 2, residual_dtype=afd.AFD_DT_F32), BAD), (dict(gamma=A + 1), BAD),
    (dict(out=A + 1), BAD), (dict(scale=A + 2), BAD), (dict(T=0, x=None), OK),
])
def test_norm_refuses(kw, status):
    assert _norm(**kw) == status


def test_norm_refuses_no_cfg():
    assert afd.afd_ffn_add_rmsnorm(None, A, A, A, A, A) == BAD


def _routing(**kw):
    base = dict(score=afd.AFD_SCORE_SIGMOID, n_groups=8, topk_groups=4, group_best=2, renormalise=1, weight_scale=2.5)
    base.update(kw)
    return afd.afd_ffn_routing(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(score=2), BAD), (dict(n_groups=0), BAD), (dict(n_groups=7), BAD), (dict(n_groups=64), NO),
    (dict(n_groups=512), BAD), (dict(topk_groups=0), BAD), (dict(topk_groups=9), BAD), (dict(group_best=0), BAD),
    (dict(group_best=3), BAD), (dict(renormalise=2), BAD), (dict(weight_scale=0.0), BAD),
    (dict(weight_scale=-1.0), BAD), (dict(weight_scale=math.nan), BAD), (dict(weight_scale=math.inf), BAD),
])
def test_selection_refuses_a_routing(kw, status):
    call = lambda r: afd.afd_ffn_select_experts(A, A, 4, 256, 8, r, A, A, afd.AFD_DT_F32, 0)     # noqa: E731
    assert call(_routing(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(E=0), BAD), (dict(k=0), BAD), (dict(E=4, k=5), BAD), (dict(E=264), NO), (dict(k=33), NO),
    (dict(logits_dtype=afd.AFD_DT_FP8_E4M3), BAD), (dict(logits_stride=255), BAD), (dict(logits=None), BAD),
    (dict(topk_idx=None), BAD), (dict(topk_w=None), BAD), (dict(logits=A + 2), BAD), (dict(topk_w=A + 2), BAD),
    (dict(logits=A + 1, logits_dtype=afd.AFD_DT_BF16), BAD), (dict(choice_bias=A + 1), BAD), (dict(T=0, logits=None), OK),
    (dict(k=20, routing=_routing(topk_groups=1, group_best=1), E=128), BAD),     # 16 experts in the groups that stay
    (dict(routing=None), BAD),
])
def test_selection_refuses(kw, status):
    base = dict(logits=A, choice_bias=None, T=4, E=256, k=8, routing=_routing(), topk_idx=A, topk_w=A,
                logits_dtype=afd.AFD_DT_F32, logits_stride=0)
    base.update(kw)
    assert afd.afd_ffn_select_experts(**base) == status


def test_set_routing_needs_a_handle():
    assert afd.afd_ffn_set_routing(None, _routing()) == BAD


def _w4(N=64, K=128, group=32, codes=A, scale=A, zero=None, scale_dtype=afd.AFD_DT_BF16):
    return afd.afd_ffn_w4(codes, scale, zero, N, K, group, scale_dtype)


@pytest.mark.parametrize("w,status", [
    (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=48), BAD), (dict(group=16), BAD), (dict(group=48), BAD),
    (dict(group=256), BAD), (dict(group=0), BAD), (dict(K=96, group=64), BAD), (dict(scale_dtype=afd.AFD_DT_FP8_E4M3), BAD),
    (dict(codes=None), BAD), (dict(scale=None), BAD), (dict(codes=A + 8), BAD), (dict(scale=A + 1), BAD),
    (dict(scale=A + 2, scale_dtype=afd.AFD_DT_F32), BAD), (dict(scale=A + 2), BAD), (dict(zero=A + 2), BAD), (dict(N=1 << 28), NO), (dict(K=1 << 21), NO),
])
def test_w4_refuses_weights(w, status):
    assert afd.afd_ffn_w4_rows(_w4(**w), 8, A, A, 4, A, afd.AFD_DT_BF16) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), BAD), (dict(E=0), BAD), (dict(E=257), NO), (dict(n_rows=-1), BAD), (dict(n_rows=(1 << 22) + 1), NO),
    (dict(counts=None), BAD), (dict(x=None), BAD), (dict(y=None), BAD), (dict(x=A + 8), BAD), (dict(y=A + 8), BAD),
    (dict(y_dtype=afd.AFD_DT_FP8_E4M3), BAD), (dict(n_rows=0, x=None), OK), (dict(counts=A + 2), BAD),
])
def test_w4_rows_refuses(kw, status):
    base = dict(w=_w4(), E=8, x=A, counts=A, n_rows=4, y=A, y_dtype=afd.AFD_DT_F32)
    base.update(kw)
    assert afd.afd_ffn_w4_rows(**base) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w13=None), BAD), (dict(w2=None), BAD), (dict(w13=_w4(N=128, K=64)), BAD),      # N = 2I, K = H
    (dict(w13=_w4(N=192, K=64)), BAD), (dict(E=257), NO), (dict(n_rows=-1), BAD), (dict(scratch=None), BAD),
    (dict(scratch=A + 4), BAD), (dict(rows=None), BAD), (dict(Y=A + 2), BAD), (dict(y_dtype=1), BAD), (dict(counts=None), BAD),
    (dict(n_rows=0, rows=None), OK),
])
def test_w4_expert_rows_refuses(kw, status):
    base = dict(w13=_w4(N=256, K=64), w2=_w4(N=64, K=128), E=8, rows=A, counts=A, n_rows=4, Y=A, scratch=A,
                y_dtype=afd.AFD_DT_BF16)
    base.update(kw)
    assert afd.afd_ffn_w4_expert_rows(**base) == status


def test_w4_scratch_bytes():
    assert afd.afd_ffn_w4_scratch_bytes(0, 128) >= 0 and afd.afd_ffn_w4_scratch_bytes(-1, 128) == 0
    assert afd.afd_ffn_w4_scratch_bytes(100, 2048) >= 2 * 100 * 2048 * 2
    assert afd.afd_ffn_w4_scratch_bytes(1 << 24, 4096) >= (1 << 24) * 4096 * 4     # past 32 bits


def test_w4_weights_checks_its_tensors():
    codes = torch.zeros((2, 6, 32), dtype=torch.uint8)
    scale, zero = torch.ones((2, 6, 2)), torch.zeros((2, 6, 2), dtype=torch.uint8)
    w = afd.w4_weights(codes, scale, zero)
    assert (w.N, w.K, w.group, w.scale_dtype) == (6, 64, 32, afd.AFD_DT_F32) and w.codes == codes.data_ptr()
    assert w._keep[1] is scale
    for bad in (dict(codes=codes.int()), dict(scale=scale[:, :, :1], group=32), dict(zero=zero.int()),
                dict(codes=codes[:, :, ::2]), dict(scale=scale.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            afd.w4_weights(**{**dict(codes=codes, scale=scale, zero=zero), **bad})


def test_struct_sizes_match_the_header():
    # natural alignment of the declared fields on a 64-bit host
    assert ctypes.sizeof(afd.afd_ffn_routing) == 24
    assert ctypes.sizeof(afd.afd_ffn_w4) == 40
    assert ctypes.sizeof(afd.afd_ffn_norm_cfg) == 56


def test_w4_refuses_more_experts_than_its_tensors_hold():
    """The library cannot see where the weights end; the binding knows the tensors it described."""
    def plan(E, N, K):
        shape = (E, N) if E else (N,)
        return afd.w4_weights(torch.zeros(shape + (K // 2,), dtype=torch.uint8), torch.ones(shape + (K // 32,)))
    for E, n in ((3, 3), (0, 1)):                        # a stack, one matrix
        w13, w2 = plan(E, 256, 64), plan(E, 64, 128)
        for e in (n, 1):                                 # the first ones of a stack are a stack
            assert afd.afd_ffn_w4_rows(w2, e, A, A, 0, A, afd.AFD_DT_F32) == OK
            assert afd.afd_ffn_w4_expert_rows(w13, w2, e, A, A, 0, A, A, afd.AFD_DT_F32) == OK
        assert afd.afd_ffn_w4_rows(w2, n + 1, A, A, 0, A, afd.AFD_DT_F32) == BAD
        assert afd.afd_ffn_w4_expert_rows(w13, w2, n + 1, A, A, 0, A, A, afd.AFD_DT_F32) == BAD
        assert afd.afd_ffn_w4_expert_rows(plan(5, 256, 64), w2, n + 1, A, A, 0, A, A, afd.AFD_DT_F32) == BAD
        assert afd.afd_ffn_w4_expert_rows(w13, plan(5, 64, 128), n + 1, A, A, 0, A, A, afd.AFD_DT_F32) == BAD


@pytest.mark.parametrize("logits", [
    torch.zeros((16, 4)).t(),                        # experts 4 elements apart
    torch.zeros((4, 32))[:, ::2],
    torch.zeros((1, 16)).expand(4, 16),              # one row for every token: its stride of 0 would mean E
    torch.zeros((4, 1)).expand(4, 16),
])
def test_selection_refuses_logits_that_are_no_rows(logits):
    """The stride is the tensor's own, so the binding can see that the rows are not there to be read."""
    idx, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    r = _routing(n_groups=1, topk_groups=1)
    assert afd.afd_ffn_select_experts(logits, None, 4, 16, 2, r, idx, w) == BAD


def test_a_layer_keeps_the_biases_that_its_graphs_read(monkeypatch):
    """A graph captured under an earlier routing reads that routing's bias: it lives as long as the layer."""
    status = [OK]
    monkeypatch.setattr(afd, "afd_ffn_set_routing", lambda h, routing, bias=None: status[0])
    monkeypatch.setattr(afd, "afd_ffn_destroy", lambda h: None)
    layer = object.__new__(afd.AfdFfn)
    layer.h, layer._choice_biases = 1, []
    first, second, refused = torch.zeros(4), torch.ones(4), torch.ones(4)
    alive = [weakref.ref(t) for t in (first, second, refused)]
    for bias in (first, second, first, None):
        layer.set_routing(_routing(), bias)
    assert len(layer._choice_biases) == 2                # a tensor set twice is held once
    status[0] = BAD
    with pytest.raises(afd.AfdError):
        layer.set_routing(_routing(), refused)
    del first, second, refused, bias
    assert [r() is not None for r in alive] == [True, True, False]
    layer.close()
    assert [r() is not None for r in alive] == [False] * 3
