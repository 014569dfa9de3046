"""The example layer runs its operators together: training lowers the loss,
the gradient of the projection agrees with differences of the loss, and the
paged cache serves the training forward's outputs."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples", "block_sparse_layer.py")
    spec = importlib.util.spec_from_file_location("block_sparse_layer", path)
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["block_sparse_layer"] = m
    spec.loader.exec_module(m)
    return m


def test_trains_and_serves(example):
    losses, o, served = example.main()
    assert all(b < a for a, b in zip(losses, losses[1:]))
    # The same inputs through other tile shapes and splits: q and k are equal
    # to the bit; the weights' roundings (2^-8 each) and the result's differ.
    # Where a block mean is a near tie the selection is the same, as both
    # sides feed the indexer the same bits.
    a, b = o.float(), served.float()
    assert bool(torch.isfinite(b).all())
    close = (a - b).abs() <= 2.0 ** -6 * (a.abs() + a.abs().amax(-1, keepdim=True))
    assert bool(close.all())


def test_gradient_of_the_projection(example):
    """The chain of the operators' backwards against a 64-bit autograd of the
    same layer with the same selection.  Four roundings to bf16 (2^-8 each)
    lie between them in a row: of q and k, of o (which delta is made of), of
    dS, and of the gradients of q and k; as a share of the gradient's norm
    they add to 2^-6 at most."""
    layer = example.Layer(hidden=128)
    g = torch.Generator(device="cuda").manual_seed(2)
    S, H, Hk, D = 200, layer.heads, layer.kv_heads, layer.dim
    x = torch.randn((S, 1, 128), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn((S, 1, H, D), generator=g, device="cuda")
    _, gw, o = layer.train_step(x, target)

    dsa = example.dsa
    q0, k0, _ = layer.qkv(x)
    q1, k1 = dsa.dsa_norm_rope_fwd(q0, k0, layer.inv_freq, wq=layer.wq,
                                   wk=layer.wk, **layer.rope())
    ids = layer.select(q1, layer.index_keys(k1))[0].cpu()

    # the projection's output is bf16 in both; its gradient passes through
    w = layer.w.double().cpu().requires_grad_(True)
    y = x[:, 0].double().cpu() @ w
    exact = (x @ layer.w)[:, 0].double().cpu()
    y = y + (exact - y).detach()
    y = y.view(S, H + 2 * Hk, D)

    def turned(t, weight):
        n = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6)
        n = n * weight.double().cpu()
        R = D // 2
        a = torch.arange(S, dtype=torch.float64)[:, None] * layer.inv_freq.cpu()
        c = (a.cos() * layer.rot_scale)[:, None]
        s = (a.sin() * layer.rot_scale)[:, None]
        lo, hi, rest = n[..., :R // 2], n[..., R // 2:R], n[..., R:]
        return torch.cat([lo * c - hi * s, lo * s + hi * c, rest], -1)
    q, k = turned(y[:, :H], layer.wq), turned(y[:, H:H + Hk], layer.wk)
    v = y[:, H + Hk:]
    nblk = -(-S // layer.block)
    holds = torch.zeros((S, nblk + 1), dtype=torch.bool)
    holds.scatter_(1, torch.where(ids >= 0, ids, nblk).long(), True)
    pos = torch.arange(S)
    holds[pos, pos // layer.block] = True
    seen = holds[:, pos // layer.block] & (pos[None] <= pos[:, None])
    outs = []
    for h in range(H):
        z = layer.scale * q[:, h] @ k[:, h // (H // Hk)].t()
        z = z.masked_fill(~seen, float("-inf"))
        outs.append(torch.softmax(z, 1) @ v[:, h // (H // Hk)])
    want_o = torch.stack(outs, 1)
    loss = (want_o - target[:, 0].double().cpu()).square().mean()
    (want,) = torch.autograd.grad(loss, w)
    err = float((gw.double().cpu() - want).norm() / want.norm())
    assert err <= 2.0 ** -6, err
