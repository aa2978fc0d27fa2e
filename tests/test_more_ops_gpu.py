"""One attention layer's training step through the operators as programs use
them together: norms and rotations, windowed attention with its largest logits,
both backward passes, the projections' gradients from 8-bit checkpoints,
clipping of them all into the step's bfloat16 buffers, the step and QK-Clip."""
import math

import numpy as np
import pytest
import torch

import rotate_ref
import window_ref
from test_attention_gpu import close, host
from test_checkpoint_gpu import check_grad, np64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


class Layer:
    lens, H, K, D, width, window, sinks = [90, 200, 14], 6, 2, 32, 128, 40, 3

    def __init__(self, mm, norm, seed=51):
        rng = np.random.default_rng([seed, norm])
        draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.mm, self.norm, self.T = mm, norm, sum(self.lens)
        self.heads = dict(q=self.H, k=self.K, v=self.K)
        self.W = {n: draw(h * self.D, self.width) * (0.1 if n == "v" else 0.4) for n, h in self.heads.items()}
        self.w = {n: 1 + 0.2 * draw(self.D) for n in "qk"} if norm else dict(q=None, k=None)
        self.x = draw(self.T, self.width).to(BF16)
        self.up = (1e-3 * draw(self.T, self.H, self.D)).to(BF16)
        self.packing = mm.muon_packing_create(self.lens)
        self.rotary = mm.MuonRotary(self.D, sections=[6, 5, 5], interleaved=norm)
        self.places = torch.randint(0, 4000, (3, self.T), device="cuda")
        self.rot = dict(positions=self.places, norm=norm, q_weight=self.w["q"], k_weight=self.w["k"])
        self.win = dict(window=self.window, sinks=self.sinks)

    def project(self, n):
        return (self.x.float() @ self.W[n].t()).to(BF16).view(self.T, self.heads[n], self.D)

    def forward(self, top):
        q, k, v = (self.project(n) for n in "qkv")
        qr, kr = self.mm.muon_qk_norm_rotate(q, k, self.packing, self.rotary, **self.rot)
        o, lse = self.mm.muon_attention(qr, kr, v, self.packing, max_logit=top, **self.win)
        return q, k, v, qr, kr, o, lse

    def backward(self, q, k, v, qr, kr, o, lse):
        dqr, dkr, dv = self.mm.muon_attention_backward(self.up, qr, kr, v, o, lse, self.packing, **self.win)
        dq, dk, dqw, dkw = self.mm.muon_qk_norm_rotate_backward(dqr, dkr, q, k, self.packing, self.rotary, **self.rot)
        return dqr, dkr, dv, dq, dk, dqw, dkw


@pytest.mark.parametrize("norm", [True, False])
def test_layer_step(mm, norm):
    print(f"[case] one layer's training step, norm {norm}", flush=True)
    L = Layer(mm, norm)
    T, scale = L.T, L.D ** -0.5
    saved = mm.muon_checkpoint_write([L.x])[0]
    top = torch.full((L.K,), -math.inf, device="cuda")
    q, k, v, qr, kr, o, lse = L.forward(top)
    dqr, dkr, dv, dq, dk, dqw, dkw = L.backward(q, k, v, qr, kr, o, lse)
    # each stage against its formula, from what it was given
    u = rotate_ref.angles(L.places.cpu().numpy(), L.rotary)
    for n, x, z, dz, dx, dw in (("q", q, qr, dqr, dq, dqw), ("k", k, kr, dkr, dk, dkw)):
        w = None if L.w[n] is None else np64(L.w[n])
        want, err = rotate_ref.forward(np64(x), u, L.rotary, norm, w, 1e-6)
        close(np64(z), want, err, n)
        want, want_w, err, err_w = rotate_ref.backward(np64(dz), np64(x), u, L.rotary, norm, w, 1e-6)
        close(np64(dx), want, err, "d" + n)
        if norm:
            close(np64(dw), want_w, err_w, f"d_{n}_weight")
    r = window_ref.forward(host(qr, T), host(kr, T), host(v, T), L.lens, scale, L.window, L.sinks)
    close(np64(o), r[0], r[3], "o")
    close(np64(lse), r[1], r[4], "lse")
    close(np64(top), r[2].reshape(L.K, -1).max(axis=1), r[5].reshape(L.K, -1).max(axis=1), "max_logit")
    r = window_ref.backward(np64(L.up), np64(qr), np64(kr), np64(v), np64(o), np64(lse), L.lens, scale, L.window, L.sinks)
    for name, got, want, err in zip(("dqr", "dkr", "dv"), (dqr, dkr, dv), r[:3], r[3:]):
        close(np64(got), want, err, name)
    # the gradients in float32, clipped together with the weights' into bfloat16
    sums = {n: torch.empty_like(L.W[n]) for n in L.W}
    mm.muon_checkpoint_grad([(d.view(T, -1), saved, sums[n]) for n, d in (("q", dq), ("k", dk), ("v", dv))])
    xh = np64(mm.muon_checkpoint_read([saved], dtype=F32)[0])
    for n, d in (("q", dq), ("k", dk), ("v", dv)):
        check_grad(d.view(T, -1), xh, sums[n])
    every = list(sums.values()) + ([dqw, dkw] if norm else [])
    G = [torch.empty(s.shape, dtype=BF16 if s.dim() == 2 else F32, device="cuda") for s in every]
    size = math.sqrt(sum(float((np64(s) ** 2).sum()) for s in every))
    limit = 0.37 * size
    got = mm.muon_grad_clip(every, limit, outs=G)
    assert abs(got.item() - size) <= 1e-12 * size
    for s, g in zip(every, G):
        want = np64(s) * (limit / size)
        assert (np.abs(np64(g) - want) <= (2.0 ** -8 if g.dtype == BF16 else 2.0 ** -23) * 1.001 * np.abs(want) + 1e-45).all()
    assert mm.muon_grad_norm(G).item() <= limit * (1 + 2.0 ** -8)
    # the step takes them: with mu 0 the momentum is the gradient
    before = {n: L.W[n].clone() for n in L.W}
    B = {n: torch.zeros_like(L.W[n]) for n in L.W}
    mm.muon_step([(L.W[n], g, B[n]) for n, g in zip("qkv", G)], mu=0.0, lr=0.0)
    assert all(torch.equal(B[n], g.float()) and torch.equal(L.W[n], before[n]) for n, g in zip("qkv", G))
    if norm:
        return
    # rotations keep logits linear in both projections: clipped, their largest is tau
    tau = 0.4 * top.min().item()
    mm.muon_qk_clip([(L.W["q"], L.D * L.H // L.K, top), (L.W["k"], L.D, top)], tau)
    after = torch.full((L.K,), -math.inf, device="cuda")
    L.forward(after)
    slack = scale * (np64(qr) ** 2).sum(axis=2).max() ** 0.5 * (np64(kr) ** 2).sum(axis=2).max() ** 0.5
    # q and k are rounded to bfloat16 before and after their rotation, on both sides
    assert (np.abs(np64(after) - tau) <= slack * tau / top.min().item() * 8 * 2.0 ** -8).all()


def test_layer_captured(mm):
    """The same calls in one graph, replayed with eager calls between."""
    print("[case] a captured layer", flush=True)
    L = Layer(mm, True)
    top = torch.full((L.K,), -math.inf, device="cuda")
    outs = [torch.empty(L.H * L.D, L.D, dtype=BF16, device="cuda"), torch.empty(L.D, device="cuda"),
            torch.empty(L.D, device="cuda")]

    def step():
        top.fill_(-math.inf)
        f = L.forward(top)
        b = L.backward(*f)
        flat = b[3].reshape(L.T, -1)[:L.H * L.D // 2, :2 * L.D].float().contiguous().view(-1)[:outs[0].numel()]
        grads = [flat.view_as(outs[0]), b[5], b[6]]
        norm = mm.muon_grad_clip(grads, 1e-4, outs=outs)
        return (*f, *b, norm)

    step()                                   # the projections' library calls set up before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        L.x.mul_(1.0 + 0.1 * i)
        L.up.mul_(1.0 - 0.1 * i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*held, top, *outs)]
        want = (*step(), top, *outs)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_at_once(mm):
    """Two streams through one packing, each with its own buffers, at the same time."""
    print("[case] two streams at once", flush=True)
    layers = [Layer(mm, True, seed=s) for s in (1, 2)]
    layers[1].packing = layers[0].packing
    tops = [torch.full((L.K,), -math.inf, device="cuda") for L in layers]
    want = []
    for L, top in zip(layers, tops):
        f = L.forward(top.clone())
        want.append((*f, *L.backward(*f)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [None, None]
    for _ in range(10):
        for i, (L, s) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(s):
                f = L.forward(tops[i].clone())
                got[i] = (*f, *L.backward(*f))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
