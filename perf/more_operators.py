"""Timed cases of routing limited to groups of experts and of products with 8-bit weights, with their plain forms.

Five operators, two cases or more each:

  route_groups   router logits -> ids, scores, counts, probability sums and balance loss, where only the experts
                 of the best groups can be chosen
  experts8       the expert layer on weights in 8 bits: E4M3 codes, one scale per 128 x 128 of a matrix; each
                 product's other operand is quantized per row and 128 of its reduction
  product8       rows times such weights: one matrix, or one per segment of the rows
  product8_grad  its gradients: rows and weights
  weights8       BF16 weights put into that form and expanded again

`run` computes the plain form with elementary torch operations, or, where `own` is true, calls the
package.  `exact` computes the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0                       # the largest E4M3 value
LEAST = 2.0 ** -100               # the least scale of a block of 128


def listed():
    return [
        # one token's routing in a decode step: 256 experts in 8 groups, 4 of them open
        dict(name="route_groups_t1_e256", op="route_groups", T=1, E=256, k=8, groups=8, top_groups=4, group_top=2,
             score="sigmoid", bias=True, mask=False, dtype="f32"),
        # a large training batch with padded rows, BF16 logits
        dict(name="route_groups_t16384_e256", op="route_groups", T=16384, E=256, k=8, groups=8, top_groups=4,
             group_top=2, score="sigmoid", bias=True, mask=True, dtype="bf16"),
        # decode of one token and of 32 tokens (the decode workloads' shape)
        dict(name="experts8_t1", op="experts8", T=1, d=2048, I=768, E=128, k=8),
        dict(name="experts8_t32", op="experts8", T=32, d=2048, I=768, E=128, k=8),
        # the prefill workload, and the large layer of the 8-bit workload
        dict(name="experts8_t8192", op="experts8", T=8192, d=2048, I=768, E=16, k=8),
        dict(name="experts8_t16384", op="experts8", T=16384, d=4096, I=2048, E=64, k=8),
        # one token through one matrix (a projection beside the experts), and a ragged batch
        dict(name="product8_r1", op="product8", R=1, N=4096, K=4096, E=1),
        dict(name="product8_r4099", op="product8", R=4099, N=4096, K=2048, E=1),
        # a training step's gradients: one matrix, and rows in the order of 16 experts of unequal load
        dict(name="product8_grad_r8192", op="product8_grad", R=8192, N=2048, K=2048, E=1),
        dict(name="product8_grad_r65536", op="product8_grad", R=65536, N=1536, K=2048, E=16),
        # weights of a tiny layer and of the prefill workload's layer
        dict(name="weights8_e8_d256", op="weights8", d=256, I=128, E=8),
        dict(name="weights8_e16_d2048", op="weights8", d=2048, I=768, E=16),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route_groups", "experts8", "experts8", "product8", "product8_grad", "weights8"])
    if op == "route_groups":
        groups = rng.choice([2, 4, 8, 8, 16, rng.randint(2, 16)])
        each = rng.choice([2, 4, 8, 16, 32, rng.randint(2, 64)])
        each = min(each, 256 // groups)
        top = rng.randint(1, groups)
        return dict(op=op, T=_between(rng, 1, 16384), E=groups * each, k=rng.randint(1, min(top * each, 16)),
                    groups=groups, top_groups=top, group_top=rng.choice([1, 2]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, mask=rng.random() < 0.5,
                    dtype=rng.choice(["f32", "bf16"]))
    if op in ("product8", "product8_grad"):
        N, K = BLOCK * _between(rng, 1, 32), BLOCK * _between(rng, 1, 32)
        E = rng.choice([1, 1, min(_between(rng, 2, 64), 2 ** 28 // (N * K))])
        return dict(op=op, R=_between(rng, 1, max(1, min(65536, 65536 * 1536 * 2048 // (N * K)))), N=N, K=K, E=E)
    d, I = BLOCK * _between(rng, 2, 32), BLOCK * _between(rng, 1, 16)
    if op == "weights8":
        return dict(op=op, d=d, I=I, E=_between(rng, 1, max(1, min(64, 16 * 768 * 2048 // (d * I)))))
    E = _between(rng, 4, max(5, min(256, 128 * 768 * 2048 // (d * I))))
    k = rng.randint(1, min(E, 8))
    rows = 256 if rng.random() < 0.4 else 65536          # decode, or any batch
    return dict(op=op, T=_between(rng, 1, max(1, min(rows // k, 8192 * 8 * 2048 * 2048 // (k * d * I)))), d=d, I=I, E=E,
                k=k)


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * std


def _distinct(g, T, E, k):
    """k distinct experts a token, as a router with unequal experts picks them."""
    keys = torch.rand(T, E, generator=g, device=DEV) + 0.5 * torch.rand(1, E, generator=g, device=DEV)
    return keys.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()


def _segments(g, R, E):
    """Starts of E segments of R rows, of unequal length, some empty."""
    share = torch.rand(E, generator=g, device=DEV) ** 2
    share[torch.rand(E, generator=g, device=DEV) < 0.1] = 0.0
    share[0] += 1e-3
    ends = (share.double().cumsum(0) / share.double().sum() * R).round().to(torch.int32)
    ends[-1] = R
    return torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), ends])


def _pow2(e):
    """2^e in 64 bits, exactly (a power function need not be)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _e4m3(q):
    """The nearest E4M3 values to q (64 bits), ties to even, in 32 bits (exact)."""
    _, e = torch.frexp(q)
    step = _pow2((e - 1).clamp(min=-6) - 3)
    return ((q / step).round() * step).clamp(-TOP, TOP).float()


def _scale8(top):
    """A block's scale, the quotient rounded once (a division by a number in 32 bits is a product here)."""
    return (top.double() / TOP).float().clamp(min=LEAST)


def _rows8(v):
    """Values of v [..., K] on the grid of 8 bits, a scale for each 128 of a row: (on the grid, scales), 32 bits."""
    b = v.float().unflatten(-1, (-1, BLOCK))
    s = _scale8(b.abs().amax(-1, keepdim=True))
    return _e4m3(b.double() / s.double()).flatten(-2), s.squeeze(-1)


def _squares8(w):
    """The same for one matrix w [N, K], a scale for each 128 x 128."""
    b = w.float().unflatten(-1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))            # [N / 128, 128, K / 128, 128]
    s = _scale8(b.abs().amax((1, 3), keepdim=True))
    return _e4m3(b.double() / s.double()).flatten(2, 3).flatten(0, 1), s[:, 0, :, 0]


def _weights8(g, E, N, K):
    """Weights as a program keeps them: E4M3 codes (uint8) [E, N, K] and scales f32 [E, N / 128, K / 128]."""
    codes = torch.empty(E, N, K, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, N // BLOCK, K // BLOCK, device=DEV)
    for e in range(E):
        v, s = _squares8(_randn(g, N, K, std=K ** -0.5).to(torch.bfloat16))
        codes[e] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[e] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    st = dict(case)
    if op == "route_groups":
        T, E = case["T"], case["E"]
        st["logits"] = (_randn(g, T, E) + _randn(g, 1, E, std=0.5)).to(_dtype(case["dtype"]))
        st["bias_t"] = _randn(g, E, std=0.05) if case["bias"] else None
        # a padded batch: about a tenth of the rows are no tokens
        st["mask_t"] = (torch.rand(T, generator=g, device=DEV) > 0.1) if case["mask"] else None
        st["coef"], st["scale"] = 0.01, (2.5 if case["score"] == "sigmoid" else 1.0)
        if own:
            from mixture_experts_routed_dispatch_amd import moe
            st["router"] = moe.Router(
                T, E, case["k"], score=moe.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                scale=st["scale"], balance_coef=st["coef"], groups=case["groups"], top_groups=case["top_groups"],
                group_top=case["group_top"])
    elif op == "experts8":
        T, d, I, E, k = (case[n] for n in "TdIEk")
        st["x"] = _randn(g, T, d).to(torch.bfloat16)
        st["ids"] = _distinct(g, T, E, k)
        p = (_randn(g, T, k)).exp()
        st["scores"] = (p / p.sum(1, keepdim=True)).contiguous()
        st["w13"], st["s13"] = _weights8(g, E, 2 * I, d)
        st["w2"], st["s2"] = _weights8(g, E, d, I)
        if own:
            from mixture_experts_routed_dispatch_amd import moe
            st["layer"] = moe.Layer(T, d, I, E, k, precision=moe.MOE_FP8_BLOCK128)
    elif op == "weights8":
        d, I, E = case["d"], case["I"], case["E"]
        st["w13"] = _randn(g, E, 2 * I, d, std=d ** -0.5).to(torch.bfloat16)
        st["w2"] = _randn(g, E, d, I, std=I ** -0.5).to(torch.bfloat16)
        if own:
            from mixture_experts_routed_dispatch_amd import moe
            st["layer"] = moe.Layer(1, d, I, E, 1, precision=moe.MOE_FP8_BLOCK128)
    else:
        R, N, K, E = (case[n] for n in "RNKE")
        st["x"] = _randn(g, R, K).to(torch.bfloat16)
        st["w"], st["s"] = _weights8(g, E, N, K)
        st["starts"] = _segments(g, R, E) if E > 1 else None
        if op == "product8_grad":
            st["dy"] = _randn(g, R, N, std=0.1).to(torch.bfloat16)
        if own:
            from mixture_experts_routed_dispatch_amd import moe
            st["product"] = moe.Product(R, N, K, E=E, training=op == "product8_grad")
    return st


# ------------------------------------------------------------------ plain forms

def _plain_route_groups(st):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    z = st["logits"].float()
    if st["score"] == "softmax":
        s = (z - z.amax(1, keepdim=True)).exp()
        s = p = s / s.sum(1, keepdim=True)
    else:
        s = 1 / (1 + (-z).exp())
        p = s / s.sum(1, keepdim=True)
    # what is ordered: scores with their bias in 64 bits (values next to a border), or the logits themselves
    z = z.double()
    if st["score"] == "softmax":
        key = (z - z.amax(1, keepdim=True)).exp()
        key = key / key.sum(1, keepdim=True)
    else:
        key = 1 / (1 + (-z).exp())
    if st["bias_t"] is not None:
        key = key + st["bias_t"].double()
    best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :st["group_top"]].sum(2)
    open_groups = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :st["top_groups"]]
    is_open = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, open_groups, True)
    order = key if st["bias_t"] is not None else z
    order = order.masked_fill(~is_open.repeat_interleave(E // G, 1), -math.inf)
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    live = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask_t"] is None else st["mask_t"]
    ids = torch.where(live[:, None], ids, torch.arange(k, device=DEV))
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * st["scale"] * live[:, None]
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    counts.scatter_add_(0, ids.flatten(), live.int()[:, None].expand(T, k).flatten())
    psum = (p.double() * live[:, None]).sum(0)
    n = live.sum().double().clamp(min=1)
    loss = st["coef"] * E / (k * n * n) * (counts.double() * psum).sum()
    return ids.to(torch.int32), w, counts, psum.float(), loss.float()


def _plain_matrix(codes, s):
    """One matrix' values in 32 bits."""
    v = codes.view(torch.float8_e4m3fn).float()
    return v * s.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)


def _plain_rows(v):
    """Rows as the product takes them: values in 8 bits times their scales, in 32 bits."""
    q, s = _rows8(v)
    return q * s.repeat_interleave(BLOCK, -1)


def _plain_experts8(st):
    T, d, I, k = st["T"], st["d"], st["I"], st["k"]
    x = _plain_rows(st["x"])
    flat = st["ids"].flatten()
    order = torch.sort(flat, stable=True).indices
    y = torch.zeros(T * k, d, device=DEV)
    counts = torch.zeros(st["E"], dtype=torch.int64, device=DEV).scatter_add_(0, flat.long(), torch.ones_like(flat).long())
    at = 0
    for e, n in enumerate(counts.tolist()):
        if n:
            rows = order[at:at + n]
            gu = x[rows // k] @ _plain_matrix(st["w13"][e], st["s13"][e]).T
            a = _plain_rows(gu[:, :I] / (1 + (-gu[:, :I]).exp()) * gu[:, I:])
            y[rows] = a @ _plain_matrix(st["w2"][e], st["s2"][e]).T
        at += n
    return (y.view(T, k, d) * st["scores"].unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _bounds(st):
    return [0, st["R"]] if st["starts"] is None else st["starts"].tolist()


def _plain_product8(st):
    x, at = _plain_rows(st["x"]), _bounds(st)
    y = [x[at[e]:at[e + 1]] @ _plain_matrix(st["w"][e], st["s"][e]).T for e in range(st["E"])]
    return torch.cat(y).to(torch.bfloat16)


def _columns8(v):
    """v [rows, N] along its rows: blocks of 32 rows (the last filled with zeros) and the smallest power of two as
    scale that keeps the block within the grid, in 32 bits."""
    n = v.shape[0]
    b = torch.nn.functional.pad(v.float(), (0, 0, 0, -n % 32)).unflatten(0, (-1, 32))
    top = b.abs().amax(1, keepdim=True)
    m, e = torch.frexp(top)                                   # top = m 2^e, m in [0.5, 1)
    s = torch.where(top > 0, e - 9 + (m > 0.875).int(), -127).clamp(-127, 127)    # smallest 2^s with top / 2^s <= 448
    q = _e4m3(b.double() * _pow2(-s))
    return (q.double() * _pow2(s)).float().flatten(0, 1)[:n]


def _plain_product8_grad(st):
    dy, at = _plain_rows(st["dy"]), _bounds(st)
    dx, dw = [], []
    for e in range(st["E"]):
        a, b = at[e], at[e + 1]
        dx.append((dy[a:b] @ _plain_matrix(st["w"][e], st["s"][e])).to(torch.bfloat16))
        dw.append((_columns8(st["dy"][a:b]).T @ _columns8(st["x"][a:b])).to(torch.bfloat16))
    return torch.cat(dx), torch.stack(dw)


def _plain_weights8(st):
    out = []
    for w in (st["w13"], st["w2"]):
        parts = []
        for m in w:
            v, s = _squares8(m)
            parts.append((v * s.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)).to(torch.bfloat16))
        out.append(torch.stack(parts))
    return tuple(out)


PLAIN = {"route_groups": _plain_route_groups, "experts8": _plain_experts8, "product8": _plain_product8,
         "product8_grad": _plain_product8_grad, "weights8": _plain_weights8}


# ------------------------------------------------------------------ the package's calls

def _own(st):
    op = st["op"]
    if op == "route_groups":
        return st["router"].forward(st["logits"], bias=st["bias_t"], mask=st["mask_t"])
    if op == "experts8":
        return st["layer"].forward(st["x"], st["ids"], st["scores"], st["w13"], st["w2"], st["s13"], st["s2"])
    if op == "product8":
        return st["product"].forward(st["x"], st["w"], st["s"], m_indptr=st["starts"])
    if op == "product8_grad":
        return st["product"].backward(st["dy"], st["x"], st["w"], st["s"], m_indptr=st["starts"])
    return st["layer"].expand_weights(*st["layer"].prepare_weights(st["w13"], st["w2"]))


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route_groups":
        T, E, k = case["T"], case["E"], case["k"]
        row = E * (4 if case["dtype"] == "f32" else 2)
        return {"bytes": T * row + 8 * T * k + 8 * E + (T if case["mask"] else 0) + (4 * E if case["bias"] else 0),
                "flops": 10 * T * E}
    if op in ("product8", "product8_grad"):
        R, N, K, E = (case[n] for n in "RNKE")
        met = E * (1 - (1 - 1 / E) ** R)                      # matrices that the rows meet, about
        if op == "product8":
            return {"bytes": int(2 * R * (N + K) + met * N * K), "flops": 2 * R * N * K}
        return {"bytes": int(2 * R * (N + 2 * K) + met * N * K + 2 * E * N * K), "flops": 4 * R * N * K}
    d, I, E = case["d"], case["I"], case["E"]
    each = 3 * I * d                                          # one expert's weights
    if op == "weights8":
        return {"bytes": E * each * (2 + 2 + 2), "flops": 4 * E * each}
    T, k = case["T"], case["k"]
    active = E * (1 - (1 - k / E) ** T)                       # experts that T tokens reach
    return {"bytes": int(active * each + 4 * T * d + 8 * T * k), "flops": 2 * T * k * each}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_route_groups(st):
    """ids and counts are checked as whole numbers; here the values."""
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    z = st["logits"].double()
    s = torch.softmax(z, 1) if st["score"] == "softmax" else torch.sigmoid(z)
    key = s if st["bias_t"] is None else s + st["bias_t"].double()
    of_group = key.view(T, G, E // G).topk(st["group_top"], dim=2).values.sum(2)
    shut = torch.ones(T, G, dtype=torch.bool, device=DEV)
    for _ in range(st["top_groups"]):
        # the largest that is left, the lowest index of several
        left = of_group.masked_fill(~shut, -math.inf)
        shut.scatter_(1, (left == left.amax(1, keepdim=True)).double().argmax(1, keepdim=True), False)
    left = (z if st["bias_t"] is None else key).masked_fill(shut.repeat_interleave(E // G, 1), -math.inf)
    live = st["mask_t"].double() if st["mask_t"] is not None else torch.ones(T, device=DEV, dtype=torch.float64)
    pick = torch.zeros_like(z)
    ws = []
    for _ in range(k):
        j = (left == left.amax(1, keepdim=True)).double().argmax(1, keepdim=True)
        ws.append(s.gather(1, j))
        pick.scatter_(1, j, 1.0)
        left.scatter_(1, j, -math.inf)
    w = torch.cat(ws, 1)
    w = w / w.sum(1, keepdim=True) * st["scale"] * live[:, None]
    p = s / s.sum(1, keepdim=True)
    counts, psum = (pick * live[:, None]).sum(0), (p * live[:, None]).sum(0)
    n = max(float(live.sum()), 1.0)
    return None, w, None, psum, st["coef"] * (counts * E / (k * n) * psum / n).sum()


def _grid64():
    """The E4M3 values from 0 up: 2^-9 steps to 2^-6, then eight to a power of two, to 448."""
    v = [i / 512 for i in range(8)] + [(8 + i) / 8 * 2.0 ** e for e in range(-6, 9) for i in range(8)]
    return torch.tensor(v[:-1], dtype=torch.float64, device=DEV)


def _nearest64(q):
    """The nearest values of the grid, ties to the even code."""
    grid = _grid64()
    mid = (grid[1:] + grid[:-1]) / 2
    a = q.abs()
    lo = torch.searchsorted(mid, a)                           # mid[lo - 1] < a <= mid[lo]
    tie = a == mid[lo.clamp(max=len(mid) - 1)]
    lo = lo + (tie & (lo % 2 == 1)).long()
    return grid[lo.clamp(max=len(grid) - 1)] * torch.sign(q)


def _block64(b, dims):
    """b on the grid with one scale (held in 32 bits) for the last axes `dims`, as values."""
    s = (b.abs().amax(dims, keepdim=True) / 448).float().double().clamp(min=2.0 ** -100)
    return _nearest64(b / s) * s


def _rows64(v):
    n = v.shape[-1] // 128
    return _block64(v.double().reshape(-1, n, 128), 2).reshape(v.shape)


def _matrix64(codes, s):
    grid = _grid64()
    c = codes.long()
    v = torch.where(c >= 128, -grid[(c & 127).clamp(max=126)], grid[(c & 127).clamp(max=126)])
    N, K = codes.shape
    return (v.view(N // 128, 128, K // 128, 128) * s.double()[:, None, :, None]).view(N, K)


def _exact_experts8(st):
    I = st["I"]
    y = torch.zeros(st["T"], st["d"], device=DEV, dtype=torch.float64)
    for e in st["ids"].unique().tolist():
        t, j = (st["ids"] == e).nonzero(as_tuple=True)
        gu = _rows64(st["x"][t]) @ _matrix64(st["w13"][e], st["s13"][e]).T
        a = _rows64(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
        y.index_add_(0, t, a @ _matrix64(st["w2"][e], st["s2"][e]).T * st["scores"][t, j].double()[:, None])
    return y


def _exact_product8(st):
    y = torch.zeros(st["R"], st["N"], device=DEV, dtype=torch.float64)
    at = _bounds(st)
    for e in range(st["E"]):
        y[at[e]:at[e + 1]] = _rows64(st["x"][at[e]:at[e + 1]]) @ _matrix64(st["w"][e], st["s"][e]).T
    return y


def _columns64(v):
    n, N = v.shape
    b = torch.zeros(-(-n // 32) * 32, N, dtype=torch.float64, device=DEV)
    b[:n] = v.double()
    b = b.view(-1, 32, N)
    top = b.abs().amax(1, keepdim=True)
    powers = torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=DEV)
    s = powers[torch.searchsorted(powers * 448, top).clamp(max=320)]     # the smallest with top / s <= 448
    return (_nearest64(b / s) * s).view(-1, N)[:n]


def _exact_product8_grad(st):
    R, N, K, E = (st[n] for n in "RNKE")
    at = _bounds(st)
    dx = torch.zeros(R, K, device=DEV, dtype=torch.float64)
    dw = torch.zeros(E, N, K, device=DEV, dtype=torch.float64)
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        dx[rows] = _rows64(st["dy"][rows]) @ _matrix64(st["w"][e], st["s"][e])
        dw[e] = _columns64(st["dy"][rows]).T @ _columns64(st["x"][rows])
    return dx, dw


def _exact_weights8(st):
    out = []
    for w in (st["w13"], st["w2"]):
        E, N, K = w.shape
        out.append(torch.stack([_block64(m.double().view(N // 128, 128, K // 128, 128), (1, 3)).view(N, K) for m in w]))
    return tuple(out)


EXACT = {"route_groups": _exact_route_groups, "experts8": _exact_experts8, "product8": _exact_product8,
         "product8_grad": _exact_product8_grad, "weights8": _exact_weights8}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
