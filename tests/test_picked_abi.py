"""Router, experts and adapters without a GPU: every refusal of the C ABI comes before any HIP call, the binding refuses
what it cannot marshal, and the plain forms that the GPU tests compare with are pinned by hand-worked values."""
import math

import numpy as np
import pytest
import torch

import oracle
from mxfp4_block_scaled_02_amd import ops
from tests import picked

P = 1 << 20  # a fake, aligned "device pointer": validation never dereferences it
INF, NAN = math.inf, math.nan
R = dict(logits=P, ldl=16, dtype=2, bias=None, score=0, renorm=1, scale=1.0, weights=P, ids=P, T=4, E=16, k=4)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), 1), (dict(weights=None), 1), (dict(ids=None), 1),
    (dict(dtype=3), 8), (dict(dtype=-1), 8), (dict(score=2), 8), (dict(score=-1), 8), (dict(scale=NAN), 8),
    (dict(scale=INF), 8), (dict(scale=-INF), 8),
    (dict(T=0), 2), (dict(T=(1 << 24) + 1), 2), (dict(E=0), 2), (dict(E=1025, ldl=2048), 2), (dict(k=0), 2),
    (dict(k=17), 2), (dict(k=65, E=128, ldl=128), 2), (dict(ldl=15), 2), (dict(ldl=(1 << 36) + 1), 2), (dict(ldl=-16), 2),
    (dict(logits=P + 2), 3), (dict(logits=P + 1, dtype=0), 3), (dict(bias=P + 2), 3), (dict(weights=P + 1), 3),
    (dict(ids=P + 2), 3),
])
def test_moe_route_refusals(change, status):
    a = dict(R, **change)
    assert ops.lib().moe_route(a["logits"], a["ldl"], a["dtype"], a["bias"], a["score"], a["renorm"], a["scale"],
                               a["weights"], a["ids"], a["T"], a["E"], a["k"], None) == status


E = dict(x=P, ldx=64, ids=P, weights=P, w13=P, s13=1 << 20, w2=P, s2=1 << 20, y=P, ldy=64, T=4, k=2, E=8, H=64, I=32,
         ws=P, nbytes=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(ids=None), 1), (dict(weights=None), 1), (dict(w13=None), 1), (dict(w2=None), 1),
    (dict(y=None), 1),
    (dict(T=0), 2), (dict(k=0), 2), (dict(E=0), 2), (dict(E=1025), 2), (dict(T=2049), 2), (dict(T=1 << 62, k=4), 2),
    (dict(T=4, k=1 << 62), 2), (dict(H=0), 2), (dict(H=48), 2), (dict(I=0), 2), (dict(I=40), 2),
    (dict(H=(1 << 20) + 32, ldx=1 << 21, ldy=1 << 21, s13=1 << 39, s2=1 << 39), 2), (dict(I=(1 << 20) + 32), 2),
    (dict(ldx=56), 2), (dict(ldy=60), 2), (dict(ldx=(1 << 36) + 8), 2), (dict(ldy=(1 << 36) + 8), 2), (dict(ldx=-64), 2),
    (dict(s13=ops.lib().mxfp4_pack_B_bytes(64, 64) - 16), 2), (dict(s2=ops.lib().mxfp4_pack_B_bytes(64, 32) - 16), 2),
    (dict(s13=-16), 2), (dict(s2=(1 << 40) + 16), 2),
    (dict(x=P + 8), 3), (dict(ldx=68), 3), (dict(ids=P + 2), 3), (dict(weights=P + 1), 3), (dict(w13=P + 8), 3),
    (dict(s13=(1 << 20) + 8), 3), (dict(w2=P + 4), 3), (dict(s2=(1 << 20) + 4), 3), (dict(y=P + 4), 3), (dict(ldy=66), 3),
    (dict(ws=None), 4), (dict(ws=P + 8), 4), (dict(nbytes=64), 4),
])
def test_moe_a16w4_refusals(change, status):
    a = dict(E, **change)
    assert ops.lib().moe_a16w4(a["x"], a["ldx"], a["ids"], a["weights"], a["w13"], a["s13"], a["w2"], a["s2"], a["y"],
                               a["ldy"], a["T"], a["k"], a["E"], a["H"], a["I"], a["ws"], a["nbytes"], None) == status


@pytest.mark.parametrize("T,k,H,I", [(0, 1, 64, 64), (1, 0, 64, 64), (4097, 1, 64, 64), (1 << 40, 1 << 40, 64, 64),
                                     (1, 1, 33, 64), (1, 1, 64, 16), (1, 1, 1 << 21, 64)])
def test_moe_workspace_of_a_rejected_shape(T, k, H, I):
    assert ops.lib().moe_a16w4_workspace_bytes(T, k, H, I) == 0
    assert ops.lib().moe_a16w4_workspace_bytes(3, 2, 64, 32) > 0


L = dict(y=P, ldy=48, yt=0, x=P, ldx=64, xt=0, a=P, b=P, index=P, scale=None, T=4, N=48, K=64, R=16, n=3, ws=P,
         nbytes=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(y=None), 1), (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(index=None), 1),
    (dict(xt=2), 8), (dict(xt=-1), 8), (dict(yt=1), 8), (dict(yt=3), 8), (dict(xt=1, yt=0), 8),
    (dict(T=0), 2), (dict(N=0), 2), (dict(n=0), 2), (dict(T=(1 << 20) + 1), 2), (dict(n=4097), 2),
    (dict(N=(1 << 20) + 1, ldy=1 << 21), 2), (dict(K=0), 2), (dict(K=4), 2), (dict(K=60), 2),
    (dict(K=(1 << 20) + 8, ldx=1 << 21), 2), (dict(R=0), 2), (dict(R=12), 2), (dict(R=136), 2), (dict(ldx=56), 2),
    (dict(ldy=47), 2), (dict(ldx=(1 << 36) + 8), 2), (dict(ldy=(1 << 36) + 1), 2), (dict(ldx=-64), 2),
    (dict(x=P + 8), 3), (dict(ldx=68), 3), (dict(a=P + 8), 3), (dict(b=P + 4), 3), (dict(y=P + 1), 3),
    (dict(y=P + 2, yt=2), 3), (dict(index=P + 2), 3), (dict(scale=P + 2), 3),
    (dict(ws=None), 4), (dict(ws=P + 4), 4), (dict(nbytes=0), 4),
])
def test_lora_add_refusals(change, status):
    a = dict(L, **change)
    assert ops.lib().lora_add(a["y"], a["ldy"], a["yt"], a["x"], a["ldx"], a["xt"], a["a"], a["b"], a["index"], a["scale"],
                              a["T"], a["N"], a["K"], a["R"], a["n"], a["ws"], a["nbytes"], None) == status


@pytest.mark.parametrize("T,K,R,n", [(0, 64, 16, 1), (1, 0, 16, 1), (1, 60, 16, 1), (1, 64, 0, 1), (1, 64, 12, 1),
                                     (1, 64, 136, 1), (1 << 21, 64, 16, 1), (1, 1 << 21, 16, 1), (1, 64, 16, 0),
                                     (1, 64, 16, 4097)])
def test_lora_workspace_of_a_rejected_shape(T, K, R, n):
    assert ops.lib().lora_add_workspace_bytes(T, K, R, n) == 0
    assert ops.lib().lora_add_workspace_bytes(1, 64, 16, 1) > 0


def test_binding_refuses_what_it_cannot_marshal():
    f = torch.zeros(2, 32)
    x, i = f.bfloat16(), torch.zeros(2, 2, dtype=torch.int32)
    w = torch.zeros(3, 4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        ops.moe_route(f, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ops.moe_a16w4(x, i, f[:, :2], w, w, 32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.lora_add(f, x, x[None], x[None], i[0])
    with pytest.raises(ValueError, match="E, N, K/2"):
        ops.pack_experts(w, w)
    with pytest.raises(ValueError, match="contiguous torch.int32"):
        ops._dense(i.long(), "ids", torch.int32, (2, 2), -1)
    with pytest.raises(ValueError, match="contiguous torch.int32"):
        ops._dense(i.t(), "ids", torch.int32, (2, 2), 0)
    with pytest.raises(ValueError, match="pack_experts of 64 x 32"):
        ops._experts(w[:, :100], "w13", 2304, 64, 32, -1)
    with pytest.raises(ValueError, match="pack_experts of 64 x 33"):
        ops._experts(w, "w13", 0, 64, 33, -1)
    assert ops._experts(w[:, :2600], "w13", 2304, 64, 32, -1) == (3, 4096)


def test_plain_forms_dequantise_as_the_oracle():
    g = np.random.default_rng(0)
    codes = g.integers(0, 256, (5, 32), dtype=np.uint8)
    scales = g.integers(120, 131, (5, 2), dtype=np.uint8)
    want = oracle.dequant_mx(codes, scales)
    assert np.array_equal(picked.dequantised(torch.from_numpy(codes), torch.from_numpy(scales)).numpy(), want)


def test_plain_route_by_hand():
    ln = math.log
    l = torch.tensor([[ln(1.0), ln(4.0), ln(3.0), -INF], [2.0, 2.0, 2.0, 2.0], [-INF] * 4, [0.0, NAN, 1.0, 2.0]]).double()
    w, i = picked.route(l, 2, None, "softmax", False, 1.0)
    assert i.tolist() == [[1, 2], [0, 1], [-1, -1], [0, 1]]
    assert np.allclose(w[:3].numpy(), [[0.5, 0.375], [0.25, 0.25], [0.0, 0.0]], rtol=1e-7) and w[3].isnan().all()
    w, i = picked.route(l[:1], 4, torch.tensor([0.5, 0.0, 0.0, 9.0]), "softmax", True, 2.0)
    assert i.tolist() == [[0, 1, 2, -1]]  # 0.125 + 0.5, 0.5, 0.375; a logit of -inf is never chosen
    assert np.allclose(w.numpy(), [[0.25, 1.0, 0.75, 0.0]], rtol=1e-7)
    w, i = picked.route(torch.tensor([[0.0, ln(3.0)]]), 1, None, "sigmoid", False, 1.0)
    assert i.tolist() == [[1]] and abs(w.item() - 0.75) < 1e-7


def test_plain_experts_and_adapters_by_hand():
    # one expert, H = I = 1 in effect: g = 2, u = 3, silu(2) * 3 * 0.5
    w13 = torch.tensor([[[2.0], [3.0]]], dtype=torch.float64)
    w2 = torch.tensor([[[0.5]]], dtype=torch.float64)
    x, ids = torch.tensor([[1.0], [1.0]]).bfloat16(), torch.tensor([[0, -1], [0, 0]], dtype=torch.int32)
    y, off = picked.experts(x, ids, torch.tensor([[1.0, 9.0], [0.25, 0.5]]), w13, w2)
    one = 2 / (1 + math.exp(-2)) * 1.5
    assert np.allclose(y.numpy(), [[one], [0.75 * one]]) and (off > 0).all() and (off < 0.02 * one).all()
    y, off = picked.adapters(torch.ones(3, 1), torch.tensor([[2.0], [3.0], [4.0]]).half(), torch.full((2, 1, 1), 0.5).half(),
                             torch.tensor([[[3.0]], [[5.0]]]).half(), torch.tensor([1, -1, 0]), torch.tensor([2.0, 0.5]))
    # the bound: 3 * 32 additions of 2^-23 on 2.5, and little else
    assert y[:, 0].tolist() == [3.5, 1.0, 13.0] and off[1, 0] == 0 and 0 < off[0, 0] < 4e-5
