"""CPU tests of the routed-expert layer: the oracle on hand-worked cases, and the refusals of
awq_moe_route, awq_moe_workspace, awq_moe_gate_up, awq_moe_down and awq_moe_mlp, all made
before any device work."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import w4a16_weight_only_amd as awq
from oracle import awq_ref as oracle
from w4a16_weight_only_amd import _lib, synth

OK, NULL, SHAPE, GROUP, ALIGN, UNSUP = (_lib.AWQ_OK, _lib.AWQ_ERR_NULL, _lib.AWQ_ERR_SHAPE, _lib.AWQ_ERR_GROUP,
                                        _lib.AWQ_ERR_ALIGN, _lib.AWQ_ERR_UNSUPPORTED)


def test_route_ref_by_hand():
    """Softmax of log(1, 2, 5) is (1, 2, 5) / 8; the two best renormalised are 5/7 and 2/7; a
    bias of 1 on expert 0 makes it the first without changing its score."""
    l = np.log([[1.0, 2.0, 5.0]])
    w, i = oracle.route_ref(l, 2, renormalize=False)
    assert i.tolist() == [[2, 1]] and np.allclose(w, [[5 / 8, 2 / 8]], rtol=1e-15)
    w, i = oracle.route_ref(l, 2, scale=2.0)
    assert i.tolist() == [[2, 1]] and np.allclose(w, [[10 / 7, 4 / 7]], rtol=1e-15)
    w, i = oracle.route_ref(l, 2, bias=np.array([1.0, 0, 0]), renormalize=False)
    assert i.tolist() == [[0, 2]] and np.allclose(w, [[1 / 8, 5 / 8]], rtol=1e-15)
    w, i = oracle.route_ref(np.zeros((1, 4)), 3, score="sigmoid", renormalize=False)
    assert i.tolist() == [[0, 1, 2]] and w.tolist() == [[0.5] * 3]  # ties: the lowest index


def test_route_ref_groups_and_masks_by_hand():
    """Scores (sigmoid of l) rise with l.  Groups {0, 1}, {2, 3}, {4, 5}: the best expert is 4,
    the best sums of two are group 1's (its two are 2 and 2) and then group 2's."""
    l = np.array([[1.0, 0.5, 2.0, 2.0, 3.0, -np.inf]])
    assert oracle.route_ref(l, 2, score="sigmoid", groups=3, topk_groups=1)[1].tolist() == [[4, -1]]
    assert oracle.route_ref(l, 3, score="sigmoid", groups=3, topk_groups=2)[1].tolist() == [[4, 2, 3]]
    assert oracle.route_ref(l, 2, score="sigmoid", groups=3, topk_groups=1, group_top=2)[1].tolist() == [[2, 3]]
    none = np.full((2, 4), -np.inf)
    none[1, 2] = np.nan
    w, i = oracle.route_ref(none, 2)
    assert (i == -1).all() and (w[0] == 0).all() and np.isnan(w[1]).all()


def test_expert_refs_by_hand():
    """One expert of W = [[1, 2], ...]: codes equal to their value, zeros 0, scale 1."""
    codes = np.array([[1, 0, 2, 0, 0, 0, 0, 0], [0, 3, 0, 1, 0, 0, 0, 0]])  # [K = 2, 8]
    qw, qz, sc = oracle.pack_awq(codes)[None], oracle.pack_awq(np.zeros((1, 8), dtype=int))[None], np.ones((1, 1, 8), np.float16)
    x = np.array([[2.0, 1.0]], dtype=np.float16)
    # x . W = (2, 3, 4, 1 | 0, 0, 0, 0): the up half is zero, so h is zero; with the halves of
    # the columns exchanged the gate is zero and silu(0) = 0.
    assert (oracle.gate_up_ref(x, qw, qz, sc, [0], 1, -1) == 0).all()
    y = oracle.down_ref(x, qw, qz, sc, [0], [[0.5]], 1, -1)
    assert y.tolist() == [[1.0, 1.5, 2.0, 0.5, 0, 0, 0, 0]]
    y = oracle.down_ref(np.repeat(x, 2, axis=0), qw, qz, sc, [0, 1], [[0.5, np.nan]], 2, -1)  # expert 1: not there
    assert y.tolist() == [[1.0, 1.5, 2.0, 0.5, 0, 0, 0, 0]]
    codes[:, 4:] = [[1, 1, 1, 1], [0, 0, 0, 0]]  # up half: x . (1, 0) = 2
    qw = oracle.pack_awq(codes)[None]
    g = np.array([2.0, 3.0, 4.0, 1.0])
    assert np.allclose(oracle.gate_up_ref(x, qw, qz, sc, [0], 1, -1), 2 * g / (1 + np.exp(-g)), rtol=1e-15)


P = ctypes.c_void_p(1 << 20)  # an aligned address that is never read
ODD = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 40


def route(logits=P, type=_lib.AWQ_F16, T=4, E=8, stride=8, bias=None, score=0, groups=1, topk_groups=1, group_top=1,
          topk=2, weights=P, ids=P):
    return _lib.load().awq_moe_route(logits, type, T, E, stride, bias, score, groups, topk_groups, group_top, topk, 1,
                                     1.0, weights, ids, None)


def test_route_refusals():
    assert route(T=0, logits=None) == OK  # nothing to do
    assert route(T=-1) == SHAPE
    assert route(E=0, stride=0) == SHAPE
    assert route(stride=7) == SHAPE
    assert route(topk=0) == SHAPE
    assert route(topk=9) == SHAPE
    assert route(groups=3) == SHAPE
    assert route(groups=4, topk_groups=5) == SHAPE
    assert route(groups=4, topk_groups=0) == SHAPE
    assert route(groups=4, topk_groups=1, topk=3) == SHAPE
    assert route(group_top=3) == SHAPE
    assert route(E=1025, stride=1025) == UNSUP
    assert route(E=512, stride=512, topk=65) == UNSUP
    assert route(E=256, stride=256, groups=128, topk_groups=2) == UNSUP
    assert route(T=(1 << 24) + 1) == UNSUP
    assert route(type=3) == UNSUP
    assert route(score=2) == UNSUP
    for name in ("logits", "weights", "ids"):
        assert route(**{name: None}) == NULL
        assert route(**{name: ctypes.c_void_p((1 << 20) + 1)}) == ALIGN
    assert route(bias=ODD) == ALIGN
    assert route(logits=ODD, type=_lib.AWQ_F32) == ALIGN


def test_workspace_sizes():
    ws = _lib.load().awq_moe_workspace
    assert ws(0, 2, 8, 4096, 1408, 0, 128) == 0
    up, down, both = ws(16, 2, 8, 4096, 1408, 0, 128), ws(16, 2, 8, 0, 1408, 4096, 128), ws(16, 2, 8, 4096, 1408, 4096, 128)
    assert 0 < up < both and 0 < down < both
    assert ws(16, 2, 8, 0, 1408, 0, 128) == SHAPE      # neither half
    assert ws(16, 2, 8, -32, 1408, 0, 128) == SHAPE
    assert ws(-1, 2, 8, 4096, 1408, 0, 128) == SHAPE
    assert ws(16, 0, 8, 4096, 1408, 0, 128) == SHAPE
    assert ws(16, 2, 0, 4096, 1408, 0, 128) == SHAPE
    assert ws(16, 2, 8, 4096, 0, 0, 128) == SHAPE
    assert ws(16, 2, 1025, 4096, 1408, 0, 128) == UNSUP
    assert ws(16, 2, 8, 4096, 1424, 0, 128) == UNSUP    # halves of 16 (mod 32) columns
    assert ws(16, 2, 8, 4112, 1408, 0, -1) == UNSUP     # K % 32
    assert ws(16, 2, 8, 4096, 1408, 0, 16) == UNSUP     # groups of 16
    assert ws(16, 2, 8, 4096, 1408, 0, 100) == GROUP
    assert ws(16, 2, 8, 4096, 1440, 4096, 128) == GROUP  # the second product's K = 1440
    assert ws(1 << 20, 2, 8, 4096, 1408, 0, 128) == UNSUP  # x of 8 GiB
    assert ws(1 << 21, 1, 8, 0, 1024, 4096, 128) == UNSUP  # h of 4 GiB
    assert ws(BIG, BIG, 8, 4096, 1408, 4096, 128) == UNSUP
    assert ws(1 << 24, 1 << 24, 8, 4096, 1408, 4096, 128) == UNSUP
    assert ws(16, 2, 8, 4096, BIG, 4096, 128) == UNSUP


@pytest.mark.parametrize("T", [1, 4096])
def test_one_experts_weight_below_4_gib(T):
    """32-bit offsets into one expert's weight, in either kernel."""
    ws = _lib.load().awq_moe_workspace
    assert ws(T, 1, 1, 1 << 16, 1 << 16, 0, 128) == UNSUP
    assert ws(T, 1, 1, 0, 1 << 16, 1 << 17, 128) == UNSUP
    assert ws(T, 1, 1, 1 << 16, 1 << 15, 0, 128) > 0
    assert ws(T, 1, 1, 0, 1 << 16, 1 << 16, 128) > 0


def gate_up(x=P, act=_lib.AWQ_F16, qw=P, qz=P, sc=P, ids=P, T=4, topk=2, E=8, K=256, inner=64, g=64, h=P, ws=P, nb=BIG):
    return _lib.load().awq_moe_gate_up(x, act, qw, qz, sc, ids, T, topk, E, K, inner, g, h, ws, nb, None)


def down(h=P, act=_lib.AWQ_F16, qw=P, qz=P, sc=P, ids=P, w=P, T=4, topk=2, E=8, K=256, N=64, g=64, y=P, ws=P, nb=BIG):
    return _lib.load().awq_moe_down(h, act, qw, qz, sc, ids, w, T, topk, E, K, N, g, y, ws, nb, None)


def mlp(x=P, act=_lib.AWQ_F16, a=P, b=P, c=P, d=P, e=P, f=P, ids=P, w=P, T=4, topk=2, E=8, K=256, inner=64, N=96, g=64,
        y=P, ws=P, nb=BIG):
    return _lib.load().awq_moe_mlp(x, act, a, b, c, d, e, f, ids, w, T, topk, E, K, inner, N, g, y, ws, nb, None)


@pytest.mark.parametrize("call,pointers,need", [
    (gate_up, ("x", "qw", "qz", "sc", "h", "ws"), (4, 2, 8, 256, 64, 0, 64)),
    (down, ("h", "qw", "qz", "sc", "y", "ws"), (4, 2, 8, 0, 256, 64, 64)),
    (mlp, ("x", "a", "b", "c", "d", "e", "f", "y", "ws"), (4, 2, 8, 256, 64, 96, 64)),
], ids=["gate_up", "down", "mlp"])
def test_expert_refusals(call, pointers, need):
    assert call(T=0, ids=None) == OK  # nothing to do
    assert call(T=-1) == SHAPE
    assert call(topk=0) == SHAPE
    assert call(E=0) == SHAPE
    assert call(K=0) == SHAPE
    assert call(g=0) == GROUP
    assert call(g=16) == UNSUP
    assert call(K=272, g=-1) == UNSUP
    assert call(E=1025) == UNSUP
    assert call(T=1 << 24, topk=2) == UNSUP
    assert call(act=_lib.AWQ_F32) == UNSUP
    assert call(act=7) == UNSUP
    for name in pointers:
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ODD}) == ALIGN, name
    for name in ("ids",) if call is gate_up else ("ids", "w"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: ODD}) == ALIGN, name
    assert call(nb=_lib.load().awq_moe_workspace(*need) - 1) == UNSUP


def test_python_refusals_without_a_device():
    """Wrong types and host tensors are refused before the library is called."""
    x = torch.zeros(2, 64, dtype=torch.float16)
    w = (torch.zeros(4, 64, 8, dtype=torch.int32), torch.zeros(4, 1, 8, dtype=torch.int32),
         torch.zeros(4, 1, 64, dtype=torch.float16))
    ids, wt = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    with pytest.raises(ValueError):
        awq.awq_moe_route(x, 2)  # on the host
    with pytest.raises(TypeError):
        awq.awq_moe_route(x.double(), 2)
    with pytest.raises(TypeError):
        awq.awq_moe_route([1.0], 2)
    with pytest.raises(ValueError):
        awq.awq_moe_gate_up(x, *w, ids, 64)
    with pytest.raises(TypeError):
        awq.awq_moe_gate_up(x.float(), *w, ids, 64)
    with pytest.raises(TypeError):
        awq.awq_moe_down(None, *w, ids, wt, 64)
    with pytest.raises(ValueError):
        awq.awq_moe_mlp(x, w, w, ids, wt, 64)


def test_synth_routing_inputs():
    """The generator's layers: as many distinct experts per token as asked for."""
    d = synth.make_moe_custom(6, 5, 3, 64, 32, 32, seed=3)
    assert all(len(set(r)) == 3 for r in d["expert_ids"].reshape(6, 3).tolist())


def test_nan_weights_flag():
    """A flag of act, for the products that have weights; nothing else is one."""
    keep = _lib.AWQ_NAN_WEIGHTS
    for act in (_lib.AWQ_F16, _lib.AWQ_BF16):
        assert down(act=act | keep, h=None) == NULL and mlp(act=act | keep, x=None) == NULL
        assert gate_up(act=act | keep) == UNSUP
        assert down(act=act | 2 * keep) == UNSUP and mlp(act=act | keep | 2) == UNSUP
    assert down(act=_lib.AWQ_F32 | keep) == UNSUP and down(act=-1) == UNSUP


@pytest.mark.parametrize("score,l", [("sigmoid", [[40.0, 50.0, 0.0, 0.0]]), ("softmax", [[-900.0, -800.0, 0.0, -950.0]])])
def test_route_ref_chooses_by_the_logits_without_a_bias(score, l):
    """Scores that round to the same number (1.0, or 0.0) still have their logits' order, also where
    groups are worth sums of two."""
    l = np.array(l)
    for top in (1, 2):
        ids = oracle.route_ref(l, 2, score=score, groups=2, topk_groups=2, group_top=top)[1]
        assert ids.tolist() == ([[1, 0]] if score == "sigmoid" else [[2, 1]])


def test_gate_up_refuses_an_h_that_overlaps_x():
    """h is written while other workgroups still read x.  Refused before any launch."""
    x = 1 << 20
    size_x, size_h = 4 * 256 * 2, 8 * 64 * 2  # T K, T topk inner
    for at in (x, x + size_x - 16, x - size_h + 16):
        assert gate_up(h=ctypes.c_void_p(at)) == UNSUP
