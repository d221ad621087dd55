"""A two-layer block trained with the sharded Muon step, its F ranks on one GPU.

    python examples/muon_block.py [--steps N]

Every rank holds 1/F of the unit (W1, norm weight, W2). A step, as a training program makes it:

* forward and backward of  y = norm(x + residual) W1^T -> SiLU -> W2^T  on each rank's batch
  (rms_norm, rms_norm_backward; the products are torch's);
* the ranks' bf16 gradient rows into each rank's momentum   (reduce_momentum_shard);
* the bf16 updates gathered into whole tensors              (cast_unflatten);
* the matrices orthogonalised                               (orthogonalize);
* each rank's window of the master weights stepped          (muon_apply_shard);
* the bf16 parameters gathered for the next forward pass    (cast_unflatten).
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sharded_flatparameter_flatten_amd as fsdp  # noqa: E402

SHAPES = [(1024, 256), (256,), (256, 1024)]     # W1, the norm's weight, W2
F, ROWS = 4, 512


def train(steps: int = 20, seed: int = 0):
    torch.manual_seed(seed)
    dev, bf = "cuda", torch.bfloat16
    new = lambda *s, t=bf: torch.empty(*s, dtype=t, device=dev)  # noqa: E731
    units = [fsdp.Unit(SHAPES, F, r) for r in range(F)]
    S, U = units[0].S, units[0].U
    params = [0.06 * torch.randn(SHAPES[0], device=dev), torch.ones(SHAPES[1], device=dev),
              0.03 * torch.randn(SHAPES[2], device=dev)]
    masters, momenta, shards, updates = [], [], [], []
    for u in units:
        p = new(S, t=torch.float32)
        fsdp.flatten_pad(u, params, p)
        masters.append(p)
        momenta.append(torch.zeros_like(p))
        shards.append(p.to(bf))
        updates.append(torch.zeros(S, dtype=bf, device=dev))
    flat = new(U)
    whole = [t.view(s) for t, s in zip(flat.split(units[0].numels), SHAPES)]
    gathered = [new(*s) for s in SHAPES]
    orth = [new(*SHAPES[0]), None, new(*SHAPES[2])]
    orth[1] = gathered[1]                         # the norm's weight steps along its momentum
    mats = [gathered[0], gathered[2]]
    work = new(fsdp.orthogonalize_workspace(mats), t=torch.uint8)
    scales = [max(1.0, s[0] / s[1]) ** 0.5 if len(s) == 2 else 1.0 for s in SHAPES]
    hp = fsdp.MuonHparams(lr=0.05, momentum=0.9, nesterov=True, weight_decay=0.01)
    batches = [torch.randn(ROWS, 256, device=dev).to(bf) for _ in range(2 * F)]
    target = 0.03 * torch.randn(256, 256, device=dev).to(bf)
    back = new(fsdp.rms_norm_backward_workspace(ROWS, 256), t=torch.uint8)
    total, normed, rstd, dx = new(ROWS, 256), new(ROWS, 256), new(ROWS, t=torch.float32), new(ROWS, 256)

    losses = []
    for _ in range(steps):
        fsdp.cast_unflatten(units[0], shards, whole)
        w1, wn, w2 = whole
        grads, loss = [], 0.0
        for r in range(F):
            x, res = batches[2 * r], batches[2 * r + 1]
            fsdp.rms_norm(x, wn, normed, residual=res, residual_out=total, rstd=rstd)
            a = normed @ w1.T
            h = torch.nn.functional.silu(a)
            err = (h @ w2.T).float() - (total @ target).float()
            loss += float(err.square().mean()) / F
            dy = (err * (2.0 / err.numel())).to(bf)
            row = torch.empty(U, dtype=bf, device=dev)
            g1, gn, g2 = (t.view(s) for t, s in zip(row.split(units[0].numels), SHAPES))
            torch.mm(dy.T, h, out=g2)
            sig = torch.sigmoid(a.float())
            da = ((dy @ w2).float() * sig * (1 + a.float() * (1 - sig))).to(bf)
            torch.mm(da.T, normed, out=g1)
            fsdp.rms_norm_backward(da @ w1, total, wn, rstd, dx, gn, back)
            grads.append(row)
        losses.append(loss)
        for u, m, upd in zip(units, momenta, updates):
            fsdp.reduce_momentum_shard(u, grads, m, upd, hp)
        fsdp.cast_unflatten(units[0], updates, gathered)
        fsdp.orthogonalize(mats, [orth[0], orth[2]], work)
        for u, p, w in zip(units, masters, shards):
            fsdp.muon_apply_shard(u, orth, scales, p, w, hp)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    for i, loss in enumerate(train(ap.parse_args().steps)):
        print(f"step {i}: loss {loss:.5f}")
