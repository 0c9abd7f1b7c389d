"""Expert parallelism with 8-bit integer experts on gloo ranks on CPU: the per-rank steps run on the float64 oracle, the
exchanges on torch.distributed.  Each rank must hand its own experts' codes and channel scales to the expert step, and
the shared expert's to the shared one: the output is the single-process layer's on the rank's tokens."""

import os

import numpy as np
import pytest
import torch.multiprocessing as mp

from test_ep_gloo import OracleOps, _free_port


class Int8OracleOps(OracleOps):
    def expert_ffn(self, shape, xg, w13, w2, hidden, group_start=None, group_rows=None, s13=None, s2=None, y=None):
        assert w13.shape[1] == 2 * hidden and s13.shape == w13.shape[:2] and s2.shape == w2.shape[:2]
        xg = xg.numpy()
        q, s = self.O.quantize_rows_int8(xg)
        yy = np.zeros((xg.shape[0], shape.d))
        groups = [(0, xg.shape[0])] if group_start is None else zip(group_start.tolist(), group_rows.tolist())
        for g, (a, n) in enumerate(groups):
            if n:
                yy[a:a + n] = self.O.expert_ffn_int8(q[a:a + n], s[a:a + n], w13[g].numpy(), s13[g].numpy(), w2[g].numpy(),
                                                     s2[g].numpy(), shape.act)[0]
        yy = self.torch.from_numpy(yy)
        return yy if y is None else y.copy_(yy)


def _problem(T, d, E, H, H_s):
    rng = np.random.default_rng(5)

    def experts(n, h):
        codes = lambda *sh: rng.integers(-127, 128, sh).astype(np.int8)  # noqa: E731
        scales = lambda m, fan: (rng.random((n, m)) + 0.5) / (64 * fan ** 0.5)  # noqa: E731
        return codes(n, 2 * h, d), scales(2 * h, d), codes(n, d, h), scales(d, h)
    return rng.standard_normal((T, d)), rng.standard_normal((E, d)) * 0.3, experts(E, H), experts(1, H_s)


def _worker(rank, world, port, case, cap, q):
    from datetime import timedelta

    import torch
    import torch.distributed as dist
    import oracle as O
    import sparse_mixture_experts_expert_b200 as moe
    from sparse_mixture_experts_expert_b200.ep import moe_forward_ep
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=timedelta(seconds=60))
    try:
        T, d, E, k, H, H_s, act = case
        x, w_r, routed, shared = _problem(T, d, E, H, H_s)
        toks = np.arange(rank, T, world)
        mine = slice(rank * E // world, (rank + 1) * E // world)
        f = lambda a: torch.from_numpy(np.ascontiguousarray(a))  # noqa: E731
        w13, s13, w2, s2 = (f(a[mine]) for a in routed)
        w13_sh, s13_sh, w2_sh, s2_sh = (f(a) for a in shared)
        shape = moe.MoeShape(T=len(toks), d=d, E=E, k=k, H=H, H_s=H_s, capacity=cap, act=act, wfmt=moe.WFMT_INT8)
        out, _, _ = moe_forward_ep(shape, f(x[toks]), f(w_r), w13, w2, s13_local=s13, s2_local=s2, w13_sh=w13_sh,
                                   s13_sh=s13_sh, w2_sh=w2_sh, s2_sh=s2_sh, ops=Int8OracleOps(O, torch))
        q.put((rank, toks, out.numpy()))
        dist.barrier()
    finally:
        dist.destroy_process_group()


def _layer(x, w_r, routed, shared, k, act, cap):
    """The layer on one process, token by token."""
    import oracle as O
    r = O.route(x, w_r, None, k, True)
    slot = O.permute(r["idx"], w_r.shape[0], cap)["slot_pos"]
    q, s = O.quantize_rows_int8(x)
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        ffn = lambda w, e: O.expert_ffn_int8(q[t:t + 1], s[t:t + 1], w[0][e], w[1][e], w[2][e], w[3][e], act)[0][0]  # noqa: E731
        out[t] = sum((r["w"][t, j] * ffn(routed, r["idx"][t, j]) for j in range(k) if slot[t, j] >= 0), ffn(shared, 0))
    return out, int((slot < 0).sum())


@pytest.mark.parametrize("world", [2, 4])
@pytest.mark.parametrize("cap", [0, 4])
def test_int8_experts_over_ranks_match_the_single_process_layer(world, cap):
    case = (38, 32, 8, 2, 16, 32, cap // 4)      # an uneven token split over four ranks
    T, d, E, k, H, H_s, act = case
    ctx = mp.get_context("spawn")
    q, port = ctx.Queue(), _free_port()
    procs = [ctx.Process(target=_worker, args=(r, world, port, case, cap, q)) for r in range(world)]
    for p in procs:
        p.start()
    got = [q.get(timeout=180) for _ in range(world)]
    for p in procs:
        p.join(120)
        assert p.exitcode == 0
    x, w_r, routed, shared = _problem(T, d, E, H, H_s)
    dropped = 0
    for rank, toks, out in got:
        want, n = _layer(x[toks], w_r, routed, shared, k, act, cap)
        dropped += n
        np.testing.assert_allclose(out, want, rtol=1e-10, atol=1e-12)
    assert (dropped > 0) == (cap > 0)
