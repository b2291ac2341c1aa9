"""A layer's MoE half run by its parts (residual and norm, the router's choice, rows sorted by expert, the experts' products, and
back onto the shared expert and the residual), for a window and for a prompt, against the window oracle: within the window's own
tolerance, 2e-3 of the rows' root mean square."""
import numpy as np
import pytest
import torch

import oracle
from slot_decode_window_gb300 import workloads as wlm
from tests.helpers import margin_accept, omoe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from slot_decode_window_gb300 import binding, build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()
    return binding


class Parts:
    """The calls of one MoE layer, over the residual stream x and the attention's output a."""

    def __init__(self, B, layer, max_rows):
        s = layer.spec
        self.norm = B.BlockNorm(s.hidden, before=True, eps=1e-6)
        self.sort = B.ExpertSort(s.n_experts, s.top_k, renorm=bool(s.renorm_topk))
        self.router_w, self.router_b = layer.router_w, layer.router_b
        self.up = B.Linear(layer.gate, up=layer.up, max_rows=max_rows * s.top_k)
        self.down = B.Linear(layer.down, max_rows=max_rows * s.top_k)
        self.shared = None
        if layer.shared_gate is not None:
            self.shared = (B.Linear(layer.shared_gate, up=layer.shared_up, max_rows=max_rows),
                           B.Linear(layer.shared_down, max_rows=max_rows))

    def forward(self, x, a):
        h, n = self.norm.forward(x, a)
        idx, w = self.sort.route(n @ self.router_w.T, bias=self.router_b)
        plan = self.sort.plan(idx)
        ys = self.down.forward(self.up.forward(self.sort.gather(plan, n), offsets=plan.offsets), offsets=plan.offsets)
        y = h
        if self.shared is not None:
            y = h + self.shared[1].forward(self.shared[0].forward(n))
        return idx, self.sort.combine(plan, ys, w=w, base=y)

    def sync(self):
        for l in (self.up, self.down) + (self.shared or ()):
            l.sync()


@pytest.mark.parametrize("T", [3, 8, 61])
def test_moe_half_by_its_parts(B, T):
    spec = wlm.MoESpec(256, 16, 4, 128, 128, 4, 32, renorm_topk=1)
    layer = wlm.make_moe_layer(spec, seed=0, cfg_id=71, device="cuda")
    om = omoe(layer)
    rng = np.random.default_rng(T)
    accept = margin_accept(om)
    x = np.zeros((T, 256), np.float32)
    a = np.zeros((T, 256), np.float32)
    for t in range(T):
        while True:
            x[t], a[t] = rng.standard_normal((2, 256))
            h = x[t].astype(np.float64) + a[t]
            if accept(oracle.rmsnorm(h).astype(np.float32)):
                break
    parts = Parts(B, layer, T)
    idx, y = parts.forward(torch.from_numpy(x).cuda(), torch.from_numpy(a).cuda())
    parts.sync()
    for t in range(T):
        h = x[t].astype(np.float64) + a[t]
        n = oracle.rmsnorm(h)
        m = oracle.moe_row(n, om)
        assert idx[t].tolist() == list(oracle.router(n, om.router_w, om.router_b, 4, True)[2])[:4]
        ref = m[0]
        assert np.abs(y[t].double().cpu().numpy() - h - ref).max() <= 2e-3 * np.sqrt(np.mean(ref * ref))


def test_a_window_gives_the_window_kernels_rows(B):
    """The same weights through strata_moe_window_forward and through the parts: routing equal, rows within the tolerance."""
    wl = wlm.WORKLOADS["tiny"]
    layer = wlm.make_moe_layer(wl.moe, seed=0, cfg_id=wl.cfg_id, device="cuda")
    win = B.Window(layer, max_rows=8)
    om = omoe(layer)
    x = torch.from_numpy(wlm.make_window(wl, 2, seed=0, window=0, accept_row=margin_accept(om))).cuda()
    want, rt = win.forward(x, routing=True)
    win.sync()
    sort = B.ExpertSort(wl.moe.n_experts, wl.moe.top_k)
    idx, w = sort.route(x @ layer.router_w.T, bias=layer.router_b)
    plan = sort.plan(idx)
    assert torch.equal(idx, rt["topk_idx"]) and torch.equal(plan.counts, rt["counts"]) and torch.equal(plan.offsets, rt["offsets"])
    assert torch.equal(plan.entries, rt["entries"]) and (w - rt["topk_w"]).abs().max() < 1e-5
    up, down = B.Linear(layer.gate, up=layer.up, max_rows=16), B.Linear(layer.down, max_rows=16)
    shared = B.Linear(layer.shared_down).forward(B.Linear(layer.shared_gate, up=layer.shared_up).forward(x))
    ys = down.forward(up.forward(sort.gather(plan, x), offsets=plan.offsets), offsets=plan.offsets)
    y = sort.combine(plan, ys, w=w, base=shared)
    assert (y - want).abs().max() <= 2e-3 * want.square().mean().sqrt()
    win.close()
