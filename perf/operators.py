"""The training-side operators of the layer: what is timed, and their plain forms.

Four operators stand around the experts' products in a training step:

* ``balance``: the load-balancing loss of the router and the per-expert counts
  (``moe_balance_loss``);
* ``route_back``: the router's backward pass, from the gates' and the loss's
  gradients to x, W_g and the bias (``moe_route_backward``);
* ``combine``: the combine with dropout of the layer's output and the residual
  (``moe_combine_dropout``);
* ``combine_back``: its backward pass, to the expert outputs and the gates
  (``moe_combine_dropout_backward``).

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the
framework's entry points.
"""

import math

import numpy as np
import torch

own = False

COEF = 0.01      # weight of the balance loss
GATE_SCALE = 1.0
ALIGN = 128      # each expert's block of permuted rows starts on a multiple


# ------------------------------------------------------------------- cases
def listed():
    return [
        # A Switch-sized layer's batch: nothing but latency.
        dict(name="balance 256 of 4", op="balance", T=256, E=4, k=1, mask=False),
        # The Mixtral-shaped layer's batch.
        dict(name="balance 8192 of 8", op="balance", T=8192, E=8, k=2, mask=False),
        # A long fine-grained batch (many sequences at once), one token in six padding.
        dict(name="balance 100003 of 64", op="balance", T=100003, E=64, k=8, mask=True),
        # The Switch-sized fp32 layer's router: latency again.
        dict(name="route back 256x64", op="route_back", T=256, d=64, E=4, k=1, dtype="fp32",
             gating="topk_softmax", loss=True, gates=True, acc=False, mask=False),
        # A wide fp32 router, where the products run on fp32 FMA.
        dict(name="route back 4096x1024 fp32", op="route_back", T=4096, d=1024, E=8, k=2,
             dtype="fp32", gating="topk_softmax", loss=True, gates=True, acc=True, mask=False),
        # An odd batch, sizes off every tile, Switch gate order, no gradient from the loss.
        dict(name="route back 1001x1032", op="route_back", T=1001, d=1032, E=11, k=3, dtype="bf16",
             gating="softmax_topk", loss=False, gates=True, acc=False, mask=True),
        # The Mixtral-shaped router, on top of the experts' own gradient of x.
        dict(name="route back 8192x4096", op="route_back", T=8192, d=4096, E=8, k=2, dtype="bf16",
             gating="topk_softmax", loss=True, gates=True, acc=True, mask=False),
        # The fine-grained router: 64 experts, top 8, a padded batch.
        dict(name="route back 16384x2048", op="route_back", T=16384, d=2048, E=64, k=8,
             dtype="bf16", gating="softmax_topk", loss=True, gates=True, acc=False, mask=True),
        # A short fp32 batch with some slots dropped by capacity.
        dict(name="combine 33x264 fp32", op="combine", T=33, d=264, E=5, k=2, dtype="fp32",
             p=0.25, residual=True, cf=0.75),
        # The fine-grained layer's output: eight rows of o to a row of y.
        dict(name="combine 16384x2048 top-8", op="combine", T=16384, d=2048, E=64, k=8,
             dtype="bf16", p=0.1, residual=True, cf=0.0),
        # The Mixtral-shaped layer's backward pass.
        dict(name="combine back 8192x4096", op="combine_back", T=8192, d=4096, E=8, k=2,
             dtype="bf16", p=0.1, cf=0.0),
        # A layer with capacity and no dropout: the plain combine's backward pass.
        dict(name="combine back 16384x2048", op="combine_back", T=16384, d=2048, E=32, k=2,
             dtype="bf16", p=0.0, cf=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges: 1 to 131072 tokens for the loss, 1 to
    16384 tokens of 64 to 4096 elements for the others, 2 to 64 experts."""
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["balance", "route_back", "combine", "combine_back"])
        E = rng.choice([2, 4, 8, 8, 16, 32, 64, rng.randint(2, 64)])
        k = rng.randint(1, min(8, E))
        c = dict(op=op, T=_log_int(rng, 1, 131072 if op == "balance" else 16384), E=E, k=k)
        if op == "balance":
            c["mask"] = rng.random() < 0.5
        else:
            c["d"] = 8 * _log_int(rng, 8, 512)
            c["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        if op == "route_back":
            c["gating"] = rng.choice(["topk_softmax", "softmax_topk"])
            c["loss"] = rng.random() < 0.7
            c["gates"] = not c["loss"] or rng.random() < 0.7
            if c["gating"] == "topk_softmax" and k == 1:
                c["loss"] = True   # a single gate is 1 and has no gradient
            if k == E:
                c["gates"] = True  # every expert always taken: the loss has none
            c["acc"] = rng.random() < 0.5
            c["mask"] = rng.random() < 0.5
        elif op != "balance":
            c["p"] = rng.choice([0.0, 0.1, 0.1, round(rng.uniform(0.01, 0.9), 3)])
            c["cf"] = rng.choice([0.0, 0.0, 1.0, 0.5])
            if op == "combine":
                c["residual"] = rng.random() < 0.7
        if work(c)["bytes"] <= most:
            return c


def _kept(case):
    """Kept assignments: all, or what even queues of the capacity hold."""
    n = case["T"] * case["k"]
    if case["cf"] > 0:
        n = min(n, case["E"] * math.ceil(case["cf"] * n / case["E"]))
    return n


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "balance":
        # scores, indices and mask in; counts, sums, loss and the number of tokens out
        return {"bytes": 4 * T * E + 4 * T * k + (T if case["mask"] else 0) + 8 * E + 8,
                "flops": T * E}
    d, s = case["d"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route_back":
        rows = 3 if case["acc"] else 2  # x and dx, and what dx is added to
        scores = case["loss"] or case["gating"] == "softmax_topk"
        return {"bytes": rows * T * d * s + d * E * (s + 4) + 4 * E + (4 * T * E if scores else 0)
                + (12 * T * k if case["gates"] else 0) + (T if case["mask"] else 0),
                "flops": 4 * T * d * E}
    n = _kept(case)
    if case["op"] == "combine":
        return {"bytes": (n + T * (2 if case["residual"] else 1)) * d * s + 8 * T * k,
                "flops": 2 * n * d}
    return {"bytes": (2 * n + T) * d * s + 12 * T * k, "flops": 4 * n * d}


# ------------------------------------------------------------------ inputs
def _routing(case, gen, d=64):
    """Router inputs and what the forward pass made of them: the scores over
    all experts (expert-major), the selected experts and their gates."""
    T, E, k = case["T"], case["E"], case["k"]
    dev = "cuda"
    x = torch.randn((T, d), generator=gen, device=dev)
    Wg = torch.randn((d, E), generator=gen, device=dev) / math.sqrt(d)
    if case.get("dtype", "fp32") == "bf16":
        x, Wg = x.bfloat16(), Wg.bfloat16()
    bias = 0.0 if "cf" in case else 0.5  # with a capacity, queues of about the same length
    logits = x.float() @ Wg.float() + bias * torch.randn((E,), generator=gen, device=dev)
    top, idx = torch.topk(logits, k, dim=1)
    scores = torch.softmax(logits, dim=1)
    if case.get("gating", "topk_softmax") == "topk_softmax":
        gate = torch.softmax(top, dim=1)
    else:
        gate = scores.gather(1, idx)
    return x, Wg, scores.t().contiguous(), idx.int(), gate.contiguous()


def _mask(case, gen):
    if not case.get("mask"):
        return None
    mask = torch.rand((case["T"],), generator=gen, device="cuda") > 1 / 6
    mask[0] = True
    return mask


def _positions(idx, E, cf):
    """The row of every assignment in the per-expert blocks (-1: its expert's
    queue was full), and the rows that any routing of this size fits into."""
    T, k = idx.shape
    hot = torch.zeros((T, E), dtype=torch.int32, device=idx.device).scatter_(1, idx.long(), 1)
    rank = (torch.cumsum(hot, 0) - hot).gather(1, idx.long())
    counts = hot.sum(0)
    rows = T * k + E * (ALIGN - 1)
    if cf > 0:
        capacity = math.ceil(cf * T * k / E)
        counts = counts.clamp(max=capacity)
        rows = min(rows, E * (-(-capacity // ALIGN) * ALIGN))
    blocks = (counts + ALIGN - 1) // ALIGN * ALIGN
    offsets = torch.cumsum(blocks, 0) - blocks
    pos = torch.where(rank < counts[idx.long()], offsets[idx.long()] + rank, -1)
    return pos.int().contiguous(), -(-rows // ALIGN) * ALIGN


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, E, k = case["T"], case["E"], case["k"]
    st = dict(case=case)
    if case["op"] == "balance":
        _, _, st["scores"], st["idx"], _ = _routing(case, gen)
        st["mask"] = _mask(case, gen)
        return _buffers(st)
    d = case["d"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "route_back":
        st["x"], st["Wg"], st["scores"], st["idx"], st["gate"] = _routing(case, gen, d)
        mask = st["mask"] = _mask(case, gen)
        st["dgate"] = torch.randn((T, k), generator=gen, device="cuda") if case["gates"] else None
        st["counts"] = st["tokens"] = st["dloss"] = None
        if case["loss"]:  # what moe_balance_loss returned, and the loss's own gradient
            counted = st["idx"] if mask is None else st["idx"][mask]
            st["counts"] = torch.bincount(counted.flatten(), minlength=E).int()
            st["tokens"] = torch.full((1,), counted.shape[0], dtype=torch.int32, device="cuda")
            # the loss is a mean over the tokens: scaled to the gates' size
            st["dloss"] = torch.rand((1,), generator=gen, device="cuda") * T + 1
        st["dx_acc"] = None
        if case["acc"]:
            st["dx_acc"] = torch.randn((T, d), generator=gen, device="cuda").to(dt)
        return _buffers(st)
    _, _, _, st["idx"], st["gate"] = _routing(dict(case, dtype="fp32"), gen)
    st["pos"], rows = _positions(st["idx"], E, case["cf"])
    st["o"] = torch.randn((rows, d), generator=gen, device="cuda").to(dt)
    # the generator's seed and offset, in device memory
    st["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")
    st["residual"] = st["dy"] = None
    if case["op"] == "combine_back":
        st["dy"] = torch.randn((T, d), generator=gen, device="cuda").to(dt)
    elif case["residual"]:
        st["residual"] = torch.randn((T, d), generator=gen, device="cuda").to(dt)
    return _buffers(st)


def _buffers(st):
    """The output buffers and the workspace that a training loop keeps."""
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    dev = "cuda"
    if c["op"] == "balance":
        st["out"] = dict(loss=torch.zeros(1, device=dev), prob_sum=torch.zeros(E, device=dev),
                         counts=torch.zeros(E, dtype=torch.int32, device=dev),
                         tokens=torch.zeros(1, dtype=torch.int32, device=dev))
    elif c["op"] == "route_back":
        st["out"] = dict(dx=torch.zeros_like(st["x"]), dWg=torch.zeros((c["d"], E), device=dev),
                         dbias=torch.zeros(E, device=dev))
    elif c["op"] == "combine":
        st["out"] = dict(y=torch.zeros((T, c["d"]), dtype=st["o"].dtype, device=dev))
    else:
        # rows that no assignment owns keep these zeros
        st["out"] = dict(d_o=torch.zeros_like(st["o"]), dgate=torch.zeros((T, k), device=dev))
    st["ws"] = None
    return st


# --------------------------------------------------------- the plain forms
def _plain_balance(st):
    scores, idx, mask = st["scores"], st["idx"].long(), st["mask"]
    E, T = scores.shape
    k = idx.shape[1]
    counted = torch.ones((T,), dtype=torch.bool, device=idx.device) if mask is None else mask
    tokens = counted.sum()
    counts = torch.zeros((E,), dtype=torch.int64, device=idx.device)
    counts.scatter_add_(0, idx.flatten(), counted[:, None].expand(T, k).flatten().long())
    prob_sum = torch.where(counted, scores, 0.0).sum(1)
    n = tokens.clamp(min=1).float()
    loss = COEF * E * (counts.float() / (n * k) * (prob_sum / n)).sum()
    return dict(loss=loss[None], prob_sum=prob_sum, counts=counts.int(), tokens=tokens[None].int())


def _plain_route_back(st):
    c = st["case"]
    x, Wg, idx = st["x"], st["Wg"], st["idx"].long()
    p = st["scores"].t()
    dz = torch.zeros_like(p)
    if st["dgate"] is not None:
        part = st["gate"] * st["dgate"]
        total = part.sum(1, keepdim=True)
        if c["gating"] == "topk_softmax":
            dz = dz.scatter_add(1, idx, part - st["gate"] * total / GATE_SCALE)
        else:
            dz = dz.scatter_add(1, idx, part) - p * total
    if st["counts"] is not None:
        n = st["tokens"].clamp(min=1).float()
        f = st["counts"].float() / (n * c["k"])
        dz = dz + st["dloss"] * (COEF * c["E"] / n) * p * (f - (p * f).sum(1, keepdim=True))
    xf = x.float()
    if st["mask"] is not None:
        dz = torch.where(st["mask"][:, None], dz, 0.0)
        xf = torch.where(st["mask"][:, None], xf, 0.0)
    dx = dz @ Wg.float().t()
    if st["dx_acc"] is not None:
        dx = dx + st["dx_acc"].float()
    return dict(dx=dx.to(x.dtype), dWg=xf.t() @ dz, dbias=dz.sum(0))


def _plain_keep(p, rng, T, d):
    """Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
    3", 2011) on 32-bit words held in int64: key = seed, counter = (eight
    elements' number, offset); 16 bits an element, dropped below p * 2^16."""
    low = 0xFFFFFFFF
    n = torch.arange(T * d // 8, device=rng.device)
    seed, offset = rng[0], rng[1]
    k0, k1 = seed & low, (seed >> 32) & low
    c0, c1 = n & low, n >> 32
    c2, c3 = (offset & low).expand_as(n), ((offset >> 32) & low).expand_as(n)
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # low 64 bits, the sign bit one of them
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    lanes = torch.stack([words & 0xFFFF, words >> 16], 2).view(T, d)
    return lanes >= _threshold(p)


def _threshold(p):
    return min(int(p * 65536 + 0.5), 65535)


def _plain_combine(st):
    c = st["case"]
    pos, o = st["pos"].long(), st["o"]
    T, k = pos.shape
    rows = o[pos.clamp(min=0)].float()
    acc = (torch.where(pos >= 0, st["gate"], 0.0)[:, :, None] * rows).sum(1)
    if c["p"] > 0:
        keep = _plain_keep(c["p"], st["rng"], T, c["d"])
        acc = torch.where(keep, acc * (65536 / (65536 - _threshold(c["p"]))), 0.0)
    if st["residual"] is not None:
        acc = acc + st["residual"].float()
    return dict(y=acc.to(o.dtype))


def _plain_combine_back(st):
    c = st["case"]
    pos, o = st["pos"].long(), st["o"]
    T, k = pos.shape
    a = st["dy"].float()
    if c["p"] > 0:
        keep = _plain_keep(c["p"], st["rng"], T, c["d"])
        a = torch.where(keep, a * (65536 / (65536 - _threshold(c["p"]))), 0.0)
    kept = pos >= 0
    dgate = torch.where(kept, (a[:, None, :] * o[pos.clamp(min=0)].float()).sum(2), 0.0)
    d_o = torch.zeros_like(o)
    d_o[pos[kept]] = (st["gate"][:, :, None] * a[:, None, :])[kept].to(o.dtype)
    return dict(d_o=d_o, dgate=dgate)


# --------------------------------------------------- the framework's calls
def _moe():
    from mixture_experts_layer_51_b200 import moe
    return moe


def _own_balance(st):
    return _moe().moe_balance_loss(st["scores"], st["idx"], COEF, mask=st["mask"], ws=_ws(st),
                                   **st["out"])


def _own_route_back(st):
    return _moe().moe_route_backward(
        st["x"], st["Wg"], st["idx"], gate=st["gate"] if st["dgate"] is not None else None,
        dgate=st["dgate"], scores=st["scores"], counts=st["counts"], tokens=st["tokens"],
        coef=COEF, dloss=st["dloss"], mask=st["mask"], gating=st["case"]["gating"],
        gate_scale=GATE_SCALE, dx_acc=st["dx_acc"], ws=_ws(st), **st["out"])


def _own_combine(st):
    y = _moe().moe_combine_dropout(st["o"], st["pos"], st["gate"], p=st["case"]["p"], rng=st["rng"],
                                   residual=st["residual"], **st["out"])
    return dict(y=y)


def _own_combine_back(st):
    d_o, dgate = _moe().moe_combine_dropout_backward(
        st["dy"], st["o"], st["pos"], st["gate"], p=st["case"]["p"], rng=st["rng"], **st["out"])
    return dict(d_o=d_o, dgate=dgate)


def _ws(st):
    """The workspace, made at the first pass and kept with the state."""
    if st["ws"] is None:
        c, moe = st["case"], _moe()
        if c["op"] == "balance":
            need = moe.moe_balance_loss_workspace_bytes(c["T"], c["E"])
        else:
            need = moe.moe_route_backward_workspace_bytes(c["T"], c["d"], c["E"], st["x"].dtype)
        st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return st["ws"]


def run(state):
    op = state["case"]["op"]
    if own:
        calls = dict(balance=_own_balance, route_back=_own_route_back, combine=_own_combine,
                     combine_back=_own_combine_back)
    else:
        calls = dict(balance=_plain_balance, route_back=_plain_route_back, combine=_plain_combine,
                     combine_back=_plain_combine_back)
    return calls[op](state)


# ------------------------------------------------------- 64-bit references
def _exact_keep(p, seed, offset, T, d):
    """The same generator on numpy's unsigned words."""
    u32, u64 = np.uint32, np.uint64
    n = np.arange(T * d // 8, dtype=u64)
    ctr = [n.astype(u32), (n >> u64(32)).astype(u32),
           np.full(n.shape, offset & 0xFFFFFFFF, u32), np.full(n.shape, offset >> 32, u32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        lo = ctr[0].astype(u64) * u64(0xD2511F53)
        hi = ctr[2].astype(u64) * u64(0xCD9E8D57)
        ctr = [(hi >> u64(32)).astype(u32) ^ ctr[1] ^ u32(key[0]), hi.astype(u32),
               (lo >> u64(32)).astype(u32) ^ ctr[3] ^ u32(key[1]), lo.astype(u32)]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    lanes = np.ascontiguousarray(np.stack(ctr, 1)).view(np.uint16).reshape(T, d)
    return lanes >= _threshold(p)


def _scaled_keep(st):
    """m [T, d] in 64 bits: 0, or one over the share that is kept."""
    c = st["case"]
    if c["p"] == 0:
        return 1.0
    seed, offset = (int(v) for v in st["rng"].cpu())
    keep = torch.from_numpy(_exact_keep(c["p"], seed, offset, c["T"], c["d"])).cuda()
    return keep.double() / (1 - _threshold(c["p"]) / 65536)


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "balance":
        rows = slice(None) if st["mask"] is None else st["mask"]
        p, idx = st["scores"].to(f64)[:, rows], st["idx"][rows]
        n = p.shape[1]
        counts = (idx[:, :, None] == torch.arange(E, device="cuda")).sum((0, 1))
        prob_sum = p.sum(1)
        loss = COEF * E * torch.dot(counts.to(f64), prob_sum) / (n * n * k) if n else 0 * p.sum()
        return dict(loss=loss.reshape(1), prob_sum=prob_sum, counts=counts.int(),
                    tokens=torch.tensor([n], dtype=torch.int32))
    if case["op"] == "route_back":
        rows = torch.arange(T, device="cuda") if st["mask"] is None else st["mask"].nonzero()[:, 0]
        p = st["scores"].to(f64).t()[rows]
        dz = torch.zeros((T, E), dtype=f64, device="cuda")
        if st["dgate"] is not None:
            q, dq = st["gate"].to(f64)[rows], st["dgate"].to(f64)[rows]
            hot = torch.nn.functional.one_hot(st["idx"][rows].long(), E).to(f64)  # [rows, k, E]
            up = torch.einsum("tj,tje->te", dq, hot)                 # gradient of each expert's gate
            g = torch.einsum("tj,tje->te", q, hot)
            if case["gating"] == "topk_softmax":
                dz[rows] += g * up - g * (g * up).sum(1, keepdim=True) / GATE_SCALE
            else:
                dz[rows] += g * up - p * (g * up).sum(1, keepdim=True)
        if st["counts"] is not None and len(rows):
            n = float(st["tokens"])
            f = st["counts"].to(f64) / (n * k)
            dz[rows] += float(st["dloss"]) * COEF * E / n * (p * f - p * (p @ f)[:, None])
        x, dx = st["x"].to(f64), dz @ st["Wg"].to(f64).t()
        if st["dx_acc"] is not None:
            dx += st["dx_acc"].to(f64)
        return dict(dx=dx, dWg=x[rows].t() @ dz[rows], dbias=dz.sum(0))
    pos, gate, o, m = st["pos"].long(), st["gate"].to(f64), st["o"], _scaled_keep(st)
    if case["op"] == "combine":
        y = torch.zeros((T, case["d"]), dtype=f64, device="cuda")
        for j in range(k):
            t = (pos[:, j] >= 0).nonzero()[:, 0]
            y[t] += gate[t, j, None] * o[pos[t, j]].to(f64)
        y *= m
        if st["residual"] is not None:
            y += st["residual"].to(f64)
        return dict(y=y)
    a = st["dy"].to(f64) * m
    d_o = torch.zeros(o.shape, dtype=f64, device="cuda")
    dgate = torch.zeros((T, k), dtype=f64, device="cuda")
    for j in range(k):
        t = (pos[:, j] >= 0).nonzero()[:, 0]
        d_o[pos[t, j]] = gate[t, j, None] * a[t]
        dgate[t, j] = torch.einsum("tc,tc->t", a[t], o[pos[t, j]].to(f64))
    return dict(d_o=d_o, dgate=dgate)
