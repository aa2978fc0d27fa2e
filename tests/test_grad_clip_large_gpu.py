"""muon_grad_norm and muon_grad_clip on more gradients than the caches keep
(224 MiB), which are read and written past them, against float64 on the GPU."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}      # half a step, relative
TINY = {BF16: 2.0 ** -134, F32: 2.0 ** -150}   # half the smallest step
KEPT = 224 << 20


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


# how a call's bytes lie around what is kept: many tensors (several launches), one that holds the border in its
# middle, just above the border, and all of it in front of a last tensor that is kept whole
SIZES = {
    "many": [int(n) for n in np.random.default_rng(8).integers(0, 1100000, size=230)],
    "one": [77, 8192 * 15000 + 4321, 9],
    "border": [KEPT // 4, 5],
    "front": [8192 * 4000 + 1, 8191, (KEPT // 4) - 8191],
}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("types", [(F32, BF16), (BF16, F32), (F32,), (BF16,)], ids=["f32-bf16", "bf16-f32", "f32", "bf16"])
def test_more_than_the_caches(mm, name, shift, types):
    sizes = SIZES[name]
    if types == (BF16,):
        sizes = [2 * n for n in sizes]
    print(f"[case] {name} {types} shift {shift}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(shift)
    grads = []
    for i, n in enumerate(sizes):
        g = torch.randn(n + shift, generator=gen, device="cuda").mul_(1 + i % 3)
        grads.append(g.to(types[i % len(types)])[shift:])
    if len(types) == 1 or name == "many":
        assert sum(g.numel() * g.element_size() for g in grads) > KEPT
    # sums of n squares, on either side: n half steps of the sum
    total = sum(g.double().square().sum().item() for g in grads)
    norm, count = math.sqrt(total), sum(sizes)
    err = 2 * (count + 8) * 2.0 ** -53
    got = mm.muon_grad_norm(grads).item()
    assert abs(got - norm) <= norm * err
    factor = 0.5 / norm

    def check(x, y):
        want = x.double() * factor
        step = HALF[F32] + (HALF[y.dtype] * (1 + HALF[F32]) if y.dtype != F32 else 0.0)
        bound = want.abs() * (step + 2 * err) + TINY[F32] + TINY[y.dtype]
        assert bool(((y.double() - want).abs() <= bound).all())   # NaN where the call leaves an element out

    for outs in ((F32, BF16), (BF16, F32, F32, BF16)):
        to = [torch.full((g.numel() + 1 + shift,), math.nan, dtype=outs[(i + i // 2) % len(outs)], device="cuda")
              for i, g in enumerate(grads)]
        kept = [g.clone() for g in grads]
        views = [t[shift:-1] for t in to]
        assert mm.muon_grad_clip(grads, 0.5, outs=views).item() == got
        for x, y, old, whole in zip(grads, views, kept, to):
            check(x, y)
            assert torch.equal(x, old) and torch.isnan(whole[:shift]).all() and torch.isnan(whole[-1])
        del to, views, kept
    # below the limit: the values as they are, in the other type
    to = [torch.empty(g.shape, dtype=BF16 if g.dtype == F32 else F32, device="cuda") for g in grads]
    assert mm.muon_grad_clip(grads, 1e9, outs=to).item() == got
    assert all(torch.equal(y, x.to(y.dtype)) for x, y in zip(grads, to))
    kept = [g.clone() for g in grads]
    assert mm.muon_grad_clip(grads, 0.5).item() == got      # in place
    for x, y in zip(kept, grads):
        check(x, y)
    assert abs(mm.muon_grad_norm(grads).item() - 0.5) <= 0.5 * 2.0 ** -8
