"""Calls of the grouping that overlap (streams, host threads, captured graphs) count in scratch of their own."""

import threading

import numpy as np
import pytest
import torch

import oracle as O
import synth
from helpers import npi

pytestmark = pytest.mark.gpu
DEV = "cuda"

# two groupings that disagree everywhere: other experts, other numbers of chunks, one with a capacity
CASES = [(20000, 96, 4, 64, 0), (9000, 160, 8, 128, 300)]


def _problems(moe):
    out = []
    for i, (T, E, k, d, cap) in enumerate(CASES):
        idx = synth.draw_topk_idx(T, E, k, seed=i, skew=0.5)
        x = torch.randn(T, d, generator=torch.Generator().manual_seed(i)).bfloat16()
        out.append((moe.MoeShape(T=T, d=d, E=E, k=k, H=16, capacity=cap), x.to(DEV), idx.to(DEV),
                    O.permute(idx.numpy(), E, cap)))
    return out


def _check(shape, x, got, want):
    xp, slot, kept, offs = got
    assert (npi(slot) == want["slot_pos"]).all() and (npi(kept) == want["kept"]).all()
    assert (npi(offs) == want["offsets"]).all()
    src = want["row_src"]
    rows = torch.zeros_like(xp)
    rows[torch.from_numpy(src >= 0)] = x[torch.from_numpy(src[src >= 0] // shape.k).to(DEV)]
    assert torch.equal(xp, rows)


def test_dispatch_on_two_streams_at_a_time(lib):
    from sparse_mixture_experts_expert_b200.autograd import dispatch
    probs = _problems(lib)
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        for (s, x, idx, want), st in zip(probs, streams):
            with torch.cuda.stream(st):
                outs.append((s, x, dispatch(s, x, idx), want))
    torch.cuda.synchronize()
    for o in outs:
        _check(*o)


def test_dispatch_from_two_host_threads_on_one_stream(lib):
    from sparse_mixture_experts_expert_b200.autograd import dispatch
    probs = _problems(lib)
    outs = []

    def work(s, x, idx, want):
        for _ in range(20):
            outs.append((s, x, dispatch(s, x, idx), want))
    threads = [threading.Thread(target=work, args=p) for p in probs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(outs) == 40
    for o in outs:
        _check(*o)


def test_two_captured_dispatches_replayed_at_a_time(lib):
    from sparse_mixture_experts_expert_b200.autograd import dispatch
    probs = _problems(lib)
    graphs = []
    for s, x, idx, want in probs:
        dispatch(s, x, idx)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = dispatch(s, x, idx)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(8):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (s, x, idx, want), (_, out) in zip(probs, graphs):
        _check(s, x, out, want)


def test_whole_layers_on_two_streams_at_a_time(lib):
    """moe_forward and moe_route without ``ws`` too: the same bits as one after the other."""
    moe = lib
    probs = []
    for seed, name in ((0, "tiny"), (1, "small")):
        wl = synth.get_workload(name)
        inp = synth.make_inputs(wl, seed=seed, device=DEV)
        s = moe.MoeShape(T=wl.T, d=wl.d, E=wl.E, k=wl.k, H=wl.H, H_s=wl.H_s, act=wl.act)
        probs.append((s, inp))

    def run(s, inp):
        return moe.moe_forward(s, inp["x"], inp["w_router"], inp["w13"], inp["w2"], bias=inp["bias"],
                               w13_sh=inp.get("w13_sh"), w2_sh=inp.get("w2_sh"))
    want = [run(*p).clone() for p in probs]
    routes = [moe.moe_route(s, inp["x"], inp["w_router"], inp["bias"])["topk_idx"].clone() for s, inp in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        for p, w, r, st in zip(probs, want, routes, streams):
            with torch.cuda.stream(st):
                outs.append((run(*p), w))
                outs.append((moe.moe_route(p[0], p[1]["x"], p[1]["w_router"], p[1]["bias"])["topk_idx"], r))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)
    assert moe.moe_get_status()[0] == 0 and np.isfinite(want[0].float().cpu().numpy()).all()
