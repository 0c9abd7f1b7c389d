"""Cases of the sorting gradients and of the 8-bit integer experts.

Four operators, each with its plain form in elementary torch operations:

* ``combine_grad``   the gradient of the weighted reduction ``out_t = sum_j w_tj y[p_tj]``: ``dy[p_tj] = w_tj dout_t``
                     (rows that no slot fills are zero) and ``dw_tj = <dout_t, y[p_tj]>``.
* ``dispatch_grad``  the gradient of sorting tokens by expert: ``dx_t = sum_j dx_perm[p_tj]``, plus an addend.
* ``ffn_int8``       gated expert FFN on sorted rows with 8-bit integer products: rows are quantised with one scale a
                     token (``q = rint(127 x / max|x|)``), weights carry one scale a channel, h = act(g) u is rounded to
                     bf16 and quantised the same way.
* ``routed_int8``    the routed experts from a routing decision to the output: sort and quantise the tokens, the 8-bit
                     experts, the weighted reduction back to token order.

``p`` is the row of a (token, slot) pair in expert order, -1 where a capacity dropped it.
"""

import math

import torch

own = False

SWIGLU, GEGLU = 0, 1


def listed():
    return [
        # one token of a small layer: launch latency
        dict(name="combine_grad_token", op="combine_grad", T=1, d=64, E=8, k=2, cf=0.0),
        # a batch with odd sizes and no capacity
        dict(name="combine_grad_odd", op="combine_grad", T=3001, d=784, E=33, k=5, cf=0.0),
        # a training batch of granular experts, capacity factor 1.25: rows past an expert's tokens hold nothing
        dict(name="combine_grad_granular", op="combine_grad", T=32768, d=768, E=192, k=4, cf=1.25),
        # one token
        dict(name="dispatch_grad_token", op="dispatch_grad", T=1, d=768, E=192, k=4, cf=0.0, dtype="bf16", add=False),
        # a training batch of granular experts, capacity factor 1.25
        dict(name="dispatch_grad_granular", op="dispatch_grad", T=32768, d=768, E=192, k=4, cf=1.25, dtype="bf16",
             add=False),
        # a wide layer, fp32 gradients added to what the rest of the layer sent back
        dict(name="dispatch_grad_wide", op="dispatch_grad", T=1500, d=7168, E=384, k=8, cf=0.0, dtype="fp32", add=True),
        # decode: 64 rows over the 48 experts that one of eight GPUs holds of a large pool; weight streaming
        dict(name="ffn_int8_decode", op="ffn_int8", R=64, d=7168, E=48, H=2048, act=SWIGLU),
        # prompt batch of granular experts
        dict(name="ffn_int8_granular", op="ffn_int8", R=131072, d=768, E=192, H=256, act=SWIGLU),
        # prompt batch of wide GeGLU experts
        dict(name="ffn_int8_geglu", op="ffn_int8", R=16384, d=768, E=32, H=4096, act=GEGLU),
        # a small layer: launch latency
        dict(name="routed_int8_tiny", op="routed_int8", T=256, d=64, E=8, k=2, H=128, act=SWIGLU, cf=0.0),
        # one token over a slice of a large pool
        dict(name="routed_int8_token", op="routed_int8", T=1, d=7168, E=48, k=8, H=2048, act=SWIGLU, cf=0.0),
        # a prompt batch of granular experts with the static-shape dispatch
        dict(name="routed_int8_granular", op="routed_int8", T=32768, d=768, E=192, k=4, H=256, act=SWIGLU, cf=1.25),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["combine_grad", "dispatch_grad", "ffn_int8", "routed_int8"])
    while True:
        d, E = _log(rng, 16, 7168, 16), _log(rng, 1, 384)
        k = rng.randint(1, min(E, 8))
        cf = rng.choice([0.0, 0.0, 1.0, 1.25])
        if op in ("combine_grad", "dispatch_grad"):
            T = _log(rng, 1, 32768)
            if T * k * d > 32768 * 4 * 768 or E * _cap(T, E, k, cf) * d > 32768 * 5 * 768:
                continue
            case = dict(op=op, T=T, d=d, E=E, k=k, cf=cf)
            if op == "dispatch_grad":
                case.update(dtype=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.5)
            return case
        H, act = _log(rng, 16, 4096, 16), rng.choice([SWIGLU, GEGLU])
        E = min(E, 192)
        k = min(k, E)
        if E * d * H > 48 * 7168 * 2048:
            continue
        if op == "ffn_int8":
            R = _log(rng, 1, 131072)
            if R * d * max(H, 64) > 131072 * 768 * 256 or R * max(d, 2 * H) > 131072 * 768:
                continue
            return dict(op=op, R=R, d=d, E=E, H=H, act=act)
        T = _log(rng, 1, 32768)
        if T * k * d * max(H, 64) > 131072 * 768 * 256 or T * k * max(d, 2 * H) > 131072 * 768:
            continue
        if E * _cap(T, E, k, cf) > 4 * T * k + 4 * E:
            continue
        return dict(op=op, T=T, d=d, E=E, k=k, H=H, act=act, cf=cf)


def _cap(T, E, k, cf):
    return math.ceil(cf * T * k / E)


def _routing(T, E, k, g, dev):
    """k distinct experts a token, and gates that sum to one."""
    z = torch.randn(T, E, generator=g, device=dev)
    v, idx = z.topk(k, dim=1)
    return idx.to(torch.int32), torch.softmax(v, dim=1)


def _sort(idx, E, cap):
    """Rows of the (token, slot) pairs in expert order, token order within an expert, ranks from cap on dropped:
    (p [T, k], rows filled of each expert [E], first row of each expert [E], number of rows)."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    order = torch.argsort(flat, stable=True)
    counts = torch.zeros(E, dtype=torch.long, device=idx.device).index_add_(0, flat, torch.ones_like(flat))
    start = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(n, device=idx.device) - start[flat[order]]
    if cap > 0:
        start = torch.arange(E, device=idx.device) * cap
        p = torch.where(rank < cap, start[flat] + rank, -1)
        return p.view(idx.shape).int(), counts.clamp(max=cap).int(), start.int(), E * cap
    return (start[flat] + rank).view(idx.shape).int(), counts.int(), start.int(), n


def _experts(case, g, dev):
    """8-bit weights [expert, out, in] and one fp32 scale a channel, such that a product keeps unit variance."""
    E, d, H = case["E"], case["d"], case["H"]

    def codes(*shape):
        return torch.randn(*shape, generator=g, device=dev).mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)

    def scales(n, fan_in):
        return (torch.rand(E, n, generator=g, device=dev) * 0.5 + 0.75) / (32.0 * math.sqrt(fan_in))

    return dict(w13=codes(E, 2 * H, d), s13=scales(2 * H, d), w2=codes(E, d, H), s2=scales(d, H))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = dict(case)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    if case["op"] == "ffn_int8":
        R, E = case["R"], case["E"]
        eid = torch.randint(0, E, (R,), generator=g, device=dev)
        rows = torch.bincount(eid, minlength=E)
        st.update(_experts(case, g, dev), x=normal(R, case["d"]), rows=rows.int(),
                  start=(torch.cumsum(rows, 0) - rows).int(), pad=int(rows.max()))
        return st
    T, d, E, k = case["T"], case["d"], case["E"], case["k"]
    st["cap"] = cap = _cap(T, E, k, case["cf"])
    idx, w = _routing(T, E, k, g, dev)
    st.update(idx=idx, w=w)
    if case["op"] == "routed_int8":
        rows = _sort(idx, E, cap)[1]
        st.update(_experts(case, g, dev), x=normal(T, d), pad=int(rows.max()))
        return st
    p, kept, _, R = _sort(idx, E, cap)
    st.update(p=p, kept=kept)
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    buf = normal(R, d, dtype=dtype)
    if cap > 0:  # rows that no slot fills hold whatever the memory held
        rank = torch.arange(R, device=dev) % cap
        buf[rank >= kept.long()[torch.arange(R, device=dev) // cap]] = float("nan")
    if case["op"] == "combine_grad":
        st.update(y=buf, dout=normal(T, d))
    else:
        st.update(dx_perm=buf, add=normal(T, d, dtype=dtype) if case["add"] else None)
    return st


# ------------------------------------------------------------------ plain forms (32-bit)


def _gather(rows, p):
    """rows[p] in fp32, zeros where p is -1."""
    return torch.where((p >= 0)[..., None], rows[p.clamp(min=0).long()].float(), 0.0)


def _plain_combine_grad(st):
    dout, p, R = st["dout"].float(), st["p"], st["y"].shape[0]
    dw = (_gather(st["y"], p) * dout[:, None]).sum(-1)
    dy = torch.zeros(R + 1, dout.shape[1], device=dout.device)
    dy[torch.where(p >= 0, p, R).long()] = st["w"][..., None] * dout[:, None]
    return dy[:R].to(torch.bfloat16), dw


def _plain_dispatch_grad(st):
    dx = _gather(st["dx_perm"], st["p"]).sum(1)
    if st["add"] is not None:
        dx = dx + st["add"].float()
    return dx.to(st["dx_perm"].dtype)


def _quantise(x):
    """Codes and scales of the rows of x (fp32): q = rint(x 127 / max|x|), s = max|x| / 127; zero rows have s = 0."""
    top = x.abs().amax(-1, keepdim=True)
    fine = top >= 2.0 ** -119
    # x and top hold bf16 values: x * 127 is exact, and no quotient but an exact tie lies next to a border
    q = torch.where(fine, torch.round(x * 127.0 / torch.where(fine, top, 1.0)), 0.0)
    return q, torch.where(fine, top / 127.0, 0.0)


def _plain_ffn(q, s, eid, rank, pad, st):
    """q [n, d] codes with scales s [n, 1] of rows that lie at place `rank` of expert eid's block of pad rows."""
    E, H = st["w13"].shape[0], st["w2"].shape[2]
    at = eid * pad + rank

    def product(rows, w):
        block = torch.zeros(E * pad, rows.shape[1], device=rows.device)
        block[at] = rows
        return torch.bmm(block.view(E, pad, -1), w.float().mT).view(E * pad, -1)[at]

    z = product(q, st["w13"]) * s * st["s13"][eid]
    a, u = z[:, :H], z[:, H:]
    if st["act"] == SWIGLU:
        a = a / (1.0 + torch.exp(-a))
    else:
        a = 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))
    hq, hs = _quantise((a * u).to(torch.bfloat16).float())
    return product(hq, st["w2"]) * hs * st["s2"][eid]


def _plain_ffn_int8(st):
    R, E = st["x"].shape[0], st["rows"].shape[0]
    eid = torch.repeat_interleave(torch.arange(E, device=st["x"].device), st["rows"].long(), output_size=R)
    rank = torch.arange(R, device=eid.device) - st["start"].long()[eid]
    return _plain_ffn(*_quantise(st["x"].float()), eid, rank, st["pad"], st).to(torch.bfloat16)


def _plain_routed_int8(st):
    E, cap, (T, k) = st["E"], st["cap"], st["idx"].shape
    p, _, start, _ = _sort(st["idx"], E, cap)
    eid = st["idx"].long()
    keep = p >= 0
    rank = torch.where(keep, p.long() - start.long()[eid], 0)
    q, s = _quantise(st["x"].float())
    # dropped pairs are computed at a place of their own behind the blocks and weigh nothing
    pad = st["pad"] + 1
    rank = torch.where(keep, rank, pad - 1).reshape(-1)
    q, s = q[:, None].expand(T, k, -1).reshape(T * k, -1), s[:, None].expand(T, k, 1).reshape(T * k, 1)
    y = _plain_ffn(q, s, eid.reshape(-1), rank, pad, st).to(torch.bfloat16).float().view(T, k, -1)
    return torch.where(keep[..., None], st["w"][..., None] * y, 0.0).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------ the framework's calls


def _own(st):
    import sparse_mixture_experts_expert_b200 as moe
    op = st["op"]
    if op in ("combine_grad", "dispatch_grad"):
        shape = moe.MoeShape(T=st["T"], d=st["d"], E=st["E"], k=st["k"], H=16, capacity=st["cap"])
        if op == "combine_grad":
            r = moe.moe_combine_backward(shape, st["dout"], st["y"], st["p"], st["w"], kept=st["kept"])
            return r["dy_perm"], r["dtopk_w"]
        return moe.moe_permute_backward(shape, st["dx_perm"], st["p"], add=st["add"], dtype=st["dx_perm"].dtype)
    if op == "ffn_int8":
        shape = moe.MoeShape(T=st["R"], d=st["d"], E=st["E"], k=1, H=st["H"], act=st["act"], wfmt=moe.WFMT_INT8)
        return moe.moe_expert_ffn(shape, st["x"], st["w13"], st["w2"], group_start=st["start"], group_rows=st["rows"],
                                  s13=st["s13"], s2=st["s2"])[1]
    shape = moe.MoeShape(T=st["T"], d=st["d"], E=st["E"], k=st["k"], H=st["H"], capacity=st["cap"], act=st["act"],
                         wfmt=moe.WFMT_INT8)
    r = moe.moe_permute_int8(shape, st["x"], st["idx"])
    y = moe.moe_expert_ffn_int8(shape, r["xq_perm"], r["xs_perm"], st["w13"], st["s13"], st["w2"], st["s2"],
                                group_start=r["offsets"], group_rows=r["kept"])
    return moe.moe_combine(shape, y, r["slot_pos"], st["w"])


def run(state):
    if own:
        return _own(state)
    return {"combine_grad": _plain_combine_grad, "dispatch_grad": _plain_dispatch_grad, "ffn_int8": _plain_ffn_int8,
            "routed_int8": _plain_routed_int8}[state["op"]](state)


def work(case):
    """Each input read once, each output written once; the weights of the experts that have rows."""
    d, E = case["d"], case["E"]
    if case["op"] in ("ffn_int8", "routed_int8"):
        H = case["H"]
        n = case["R"] if case["op"] == "ffn_int8" else case["T"] * case["k"]
        if case["op"] == "ffn_int8":
            hit = E * (1 - (1 - 1 / E) ** n)
            rows = 2 * n * d * 2
        else:
            hit = E * (1 - (1 - case["k"] / E) ** case["T"])
            rows = 2 * case["T"] * d * 2 + n * 8
        return {"bytes": int(hit * (3 * d * H + 4 * (2 * H + d)) + rows), "flops": 6 * n * d * H}
    T, k = case["T"], case["k"]
    b = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "combine_grad":
        R = E * _cap(T, E, k, case["cf"]) or T * k
        return {"bytes": T * d * 2 + min(R, T * k) * d * 2 + R * d * 2 + 12 * T * k, "flops": 3 * T * k * d}
    return {"bytes": T * k * d * b + 4 * T * k + (2 if case["add"] else 1) * T * d * b, "flops": T * k * d}


# ------------------------------------------------------------------ 64 bits, from the definitions


def _exact_codes(x):
    top = x.abs().max(dim=1).values
    zero = top < 2.0 ** -119
    q = torch.round((127 * x) / torch.where(zero, torch.ones_like(top), top)[:, None])
    q[zero] = 0
    return q, torch.where(zero, torch.zeros_like(top), top / 127)


def _exact_expert(x, st, e):
    """One expert on rows x (fp64), from codes to the unrounded output."""
    H = st["w2"].shape[2]
    q, s = _exact_codes(x)
    w13, w2 = st["w13"][e].double() * st["s13"][e].double()[:, None], st["w2"][e].double() * st["s2"][e].double()[:, None]
    xs = q * s[:, None]
    g, u = xs @ w13[:H].T, xs @ w13[H:].T
    phi = torch.sigmoid(g) if st["act"] == SWIGLU else 0.5 * torch.erfc(-g / math.sqrt(2.0))
    hq, hs = _exact_codes((g * phi * u).to(torch.bfloat16).double())
    return (hq * hs[:, None]) @ w2.T


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "ffn_int8":
        sizes = st["rows"].tolist()
        return torch.cat([_exact_expert(x.double(), st, e) for e, x in enumerate(st["x"].split(sizes))])
    w, E, cap = st["w"].double(), case["E"], st["cap"]
    if op == "routed_int8":
        out = torch.zeros(case["T"], case["d"], dtype=torch.float64, device=w.device)
        for e in range(E):
            t, j = torch.nonzero(st["idx"] == e, as_tuple=True)  # in token order
            if cap:
                t, j = t[:cap], j[:cap]
            if t.numel():
                out.index_add_(0, t, w[t, j][:, None] * _exact_expert(st["x"][t].double(), st, e))
        return out
    T, k, d = case["T"], case["k"], case["d"]
    p = st["p"].long()
    if op == "combine_grad":
        dy = torch.zeros(st["y"].shape, dtype=torch.float64, device=w.device)
        dw = torch.zeros(T, k, dtype=torch.float64, device=w.device)
        for j in range(k):
            t = torch.nonzero(p[:, j] >= 0)[:, 0]
            g = st["dout"][t].double()
            dy[p[t, j]] = w[t, j][:, None] * g
            dw[t, j] = torch.einsum("td,td->t", g, st["y"][p[t, j]].double())
        return dy, dw
    dx = torch.zeros(T, d, dtype=torch.float64, device=w.device) if st["add"] is None else st["add"].double()
    for j in range(k):
        t = torch.nonzero(p[:, j] >= 0)[:, 0]
        dx.index_add_(0, t, st["dx_perm"][p[t, j]].double())
    return dx
