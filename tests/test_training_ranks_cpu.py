"""The balance loss of a batch split over ranks, on CPU: two gloo ranks add up
counts, tokens and prob_sum; the loss is the formula on the sums, and each
rank's gradient from the summed counts and tokens is its part of the whole
batch's."""

import os
import socket

import numpy as np
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import oracle

T, D, E, K, COEF, DLOSS = 61, 24, 6, 2, 0.3, 1.7
SPLIT = 40  # the ranks' shares are not of one size


def _batch():
    g = np.random.default_rng(5)
    z = g.standard_normal((T, E)) + g.standard_normal(E)
    p = np.exp(z) / np.exp(z).sum(1, keepdims=True)
    idx = np.argsort(-p, 1)[:, :K]
    mask = g.random(T) > 0.25
    return dict(x=g.standard_normal((T, D)), Wg=g.standard_normal((D, E)), scores=p.T.copy(),
                idx=idx, mask=mask)


def _gradients(b, rows, counts, tokens):
    dz = oracle.router_dlogits(len(b["idx"][rows]), E, idx=b["idx"][rows],
                               scores=b["scores"][:, rows], counts=counts, tokens=tokens,
                               coef=COEF, dloss=DLOSS, mask=b["mask"][rows])
    return oracle.route_backward(b["x"][rows], b["Wg"], dz, mask=b["mask"][rows])


def _worker(rank, world, port, results):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        b = _batch()
        rows = slice(0, SPLIT) if rank == 0 else slice(SPLIT, T)
        _, prob_sum, counts, n = oracle.balance_loss(b["scores"][:, rows], b["idx"][rows], E, COEF,
                                                     b["mask"][rows])
        sums = torch.from_numpy(np.concatenate([prob_sum, counts, [n]]).astype(np.float64))
        dist.all_reduce(sums)
        prob_sum, counts, n = sums[:E].numpy(), sums[E:2 * E].numpy(), int(sums[-1])
        loss = COEF * E * float((counts / (n * K) * prob_sum / n).sum())
        dx, dWg, dbias = _gradients(b, rows, counts, n)
        parts = torch.from_numpy(np.concatenate([dWg.ravel(), dbias]))
        dist.all_reduce(parts)
        results[rank] = (loss, dx, parts.numpy())
    finally:
        dist.barrier()
        dist.destroy_process_group()


def test_the_loss_and_its_gradient_of_a_split_batch():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    results = mp.get_context("spawn").Manager().dict()
    mp.start_processes(_worker, args=(2, port, results), nprocs=2, join=True, start_method="spawn")
    b = _batch()
    loss, _, counts, n = oracle.balance_loss(b["scores"], b["idx"], E, COEF, b["mask"])
    dx, dWg, dbias = _gradients(b, slice(0, T), counts, n)
    whole = np.concatenate([dWg.ravel(), dbias])
    # sums of at most T terms in 64 bits, in another order
    eps = T * 2.0 ** -52
    for rank in range(2):
        got_loss, _, got = results[rank]
        assert abs(got_loss - loss) <= eps * loss
        assert np.all(np.abs(got - whole) <= eps * np.abs(whole).max())
    got_dx = np.concatenate([results[0][1], results[1][1]])
    assert np.all(np.abs(got_dx - dx) <= eps * np.abs(dx).max())
