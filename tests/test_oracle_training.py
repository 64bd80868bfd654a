"""Pins of the training oracle: the generator's published known answers, and
every gradient against central differences of its forward formula (CPU)."""

import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_51_b200", "csrc")


@pytest.mark.parametrize("counter,key,want", [
    # the known answers that the generator's authors publish with it
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(int(w) for w in oracle.philox4x32_10(counter, key)) == want


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_kernels_generator_on_the_host(tmp_path):
    """philox.cuh compiled for the host gives the oracle's decisions, with
    counters, offsets and seeds past 32 bits."""
    src = tmp_path / "p.cpp"
    src.write_text(r"""
#include <cstdio>
#include <cstdlib>
#include "philox.cuh"
int main(int, char** v) {
  const uint64_t n = strtoull(v[1], 0, 0), off = strtoull(v[2], 0, 0), seed = strtoull(v[3], 0, 0);
  for (int i = 0; i < 64; ++i) {
    uint32_t w[4], keep = 0;
    moe::philox4x32_10(n + i, off, moe::philox_keys(seed), w);
    for (int j = 0; j < 8; ++j) keep |= (moe::dropout_kept(w, j, atoi(v[4])) ? 1u : 0u) << j;
    printf("%u ", keep);
  }
}
""")
    exe = tmp_path / "p"
    subprocess.run(["g++", "-std=c++17", "-D__host__=", "-D__device__=", "-D__forceinline__=inline",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True)
    for first, off, seed, p in [(0, 0, 0, 0.5), (2**32 - 20, 7, 2**63 + 5, 0.1),
                                (2**40 + 3, 2**62 + 1, 12345, 0.9)]:
        thr = oracle.dropout_threshold(p)
        got = subprocess.run([str(exe), str(first), str(off), str(seed), str(thr)],
                             capture_output=True, text=True, check=True).stdout.split()
        keep = oracle.dropout_keep(p, seed, off, 64, 8, first=first)
        want = (keep * (1 << np.arange(8))).sum(1)
        assert [int(g) for g in got] == want.tolist()


def test_keep_share():
    """The share of kept elements is 1 - p within five standard errors, at
    every place of an 8-element group."""
    T, d, p = 2000, 64, 0.1
    keep = oracle.dropout_keep(p, 11, 3, T, d).reshape(-1, 8)
    se = np.sqrt(p * (1 - p) / keep.shape[0])
    assert np.all(np.abs(keep.mean(0) - (1 - p)) <= 5 * se)
    assert not np.array_equal(keep, oracle.dropout_keep(p, 11, 4, T, d).reshape(-1, 8))


def _softmax(z):
    e = np.exp(z - z.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def _gates(z, idx, gating, s):
    if gating == "topk_softmax":
        return s * _softmax(np.take_along_axis(z, idx, 1))
    return s * np.take_along_axis(_softmax(z), idx, 1)


@pytest.mark.parametrize("gating,s,masked", [("topk_softmax", 1.0, False),
                                             ("topk_softmax", 2.5, True),
                                             ("softmax_topk", 1.0, True),
                                             ("softmax_topk", 4.0, False)])
def test_router_gradient_is_the_difference_quotient(gating, s, masked):
    """dx, dWg, dbias against central differences of sum(dgate * gate) +
    dloss * loss as functions of x, Wg and the bias (selection fixed)."""
    rng = np.random.default_rng(5)
    T, d, E, k, coef, dloss = 7, 8, 6, 3, 0.3, 1.7
    x, Wg, b = rng.standard_normal((T, d)), rng.standard_normal((d, E)) / 3, rng.standard_normal(E)
    mask = np.array([1, 1, 0, 1, 0, 1, 1], bool) if masked else None
    use = np.ones(T, bool) if mask is None else mask
    idx = np.argsort(-(x @ Wg + b), axis=1)[:, :k]
    up = rng.standard_normal((T, k))

    def f(x, Wg, b):
        z = x @ Wg + b
        loss, *_ = oracle.balance_loss(_softmax(z).T, idx, E, coef, mask)
        return float((up * _gates(z, idx, gating, s))[use].sum()) + dloss * loss

    z = x @ Wg + b
    p = _softmax(z).T
    _, _, counts, n = oracle.balance_loss(p, idx, E, coef, mask)
    dz = oracle.router_dlogits(T, E, idx, _gates(z, idx, gating, s), up, p, counts, n, coef, dloss,
                               mask, gating, s)
    got = oracle.route_backward(x, Wg, dz, mask=mask)
    h = 1e-5
    for arg, g in zip(range(3), got):
        args = [x, Wg, b]
        for at in np.ndindex(args[arg].shape):
            lo, hi = [v.copy() for v in args], [v.copy() for v in args]
            lo[arg][at] -= h
            hi[arg][at] += h
            # central differences: O(h^2) truncation, O(2^-52 / h) rounding
            assert abs((f(*hi) - f(*lo)) / (2 * h) - g[at]) < 1e-8


def test_combine_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(6)
    T, d, k, p = 5, 16, 2, 0.25
    pos = np.array([[0, 5], [1, -1], [-1, -1], [6, 2], [3, 7]])
    o, gate, dy = (rng.standard_normal(s) for s in ((9, d), (T, k), (T, d)))
    keep = oracle.dropout_keep(p, 1, 2, T, d)

    def f(o, gate):
        return float((dy * oracle.combine_dropout(o, pos, gate, keep, p)).sum())

    d_o, dgate = oracle.combine_dropout_backward(dy, o, pos, gate, keep, p)
    h = 1e-5
    for arg, g in ((0, d_o), (1, dgate)):
        args = [o, gate]
        for at in np.ndindex(args[arg].shape):
            lo, hi = [v.copy() for v in args], [v.copy() for v in args]
            lo[arg][at] -= h
            hi[arg][at] += h
            assert abs((f(*hi) - f(*lo)) / (2 * h) - g[at]) < 1e-8
    assert not d_o[[4, 8]].any() and not dgate[2].any() and dgate[1, 1] == 0


def test_even_use_gives_coef():
    """Uniform scores and evenly spread assignments: the loss is coef."""
    T, E, k = 12, 4, 2
    idx = np.stack([np.arange(T) % E, (np.arange(T) + 1) % E], 1)
    loss, prob_sum, counts, n = oracle.balance_loss(np.full((E, T), 1 / E), idx, E, 0.02)
    assert abs(loss - 0.02) < 1e-15 and n == T and counts.tolist() == [6] * 4
    assert np.allclose(prob_sum, T / E)
