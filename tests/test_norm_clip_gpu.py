"""QK-Clip of a layer whose queries and keys are normed on their way into
attention: what the README's example does with it."""
import math
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


def inputs(mm, heads=4, kv_heads=2, head_dim=128, T=300):
    gen = torch.Generator(device="cuda").manual_seed(5)

    def draw(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    q, k, v, do = (draw(T, h, head_dim).to(BF16) for h in (heads, kv_heads, kv_heads, heads))
    sums = [draw(64, 32), draw(7)]
    return dict(mm=mm, torch=torch, head_dim=head_dim, q=q, k=k, v=v, do=do, packing=mm.muon_packing_create([T - 37, 37]),
                pos=torch.randint(0, 1000, (3, T), generator=gen, device="cuda"), wq=8 + draw(head_dim), wk=8 + draw(head_dim),
                top=torch.full((heads,), -math.inf, device="cuda"), sums=sums,
                grads=[torch.empty_like(s, dtype=BF16) for s in sums])


def logits(n):
    """The largest logits of the example's forward pass, and how large a logit of its q and k could be."""
    rotary = n["mm"].MuonRotary(n["head_dim"], sections=[16, 24, 24])
    q, k = n["mm"].muon_qk_norm_rotate(n["q"], n["k"], n["packing"], rotary, positions=n["pos"], q_weight=n["wq"], k_weight=n["wk"])
    top = torch.full_like(n["top"], -math.inf)
    n["mm"].muon_attention(q, k, n["v"], n["packing"], max_logit=top, window=1024, sinks=4)
    sizes = [t.double().square().sum(dim=2).max().sqrt().item() for t in (q, k)]
    return top, sizes[0] * sizes[1] / math.sqrt(n["head_dim"])


def test_projections_do_not_matter(mm):
    """Why it is not W_q and W_k that are clipped there: a smaller projection gives the same logits."""
    print("[case] logits behind a norm", flush=True)
    n = inputs(mm)
    before, _ = logits(n)
    n["q"], n["k"] = n["q"] * 0.25, n["k"] * 0.25
    after, size = logits(n)
    # eps is 1e-6 of a mean square of 1 (then 1/16): 8e-6 each; the outputs may round to the next bfloat16
    assert ((after - before).abs() <= size * (2 * 2 * 2.0 ** -8 + 3.2e-5)).all()


def test_readme(mm):
    """The example with norms, run as it stands: the largest logit is tau at the next step."""
    print("[case] README", flush=True)
    with open(README) as f:
        examples = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "muon_qk_norm_rotate" in b]
    assert len(examples) == 1
    n = inputs(mm)
    before, size = logits(n)
    tau = 100.0
    assert before.max() > 1.5 * tau
    exec(examples[0], n)
    assert torch.equal(n["top"], before)
    after, _ = logits(n)
    # q and k are rounded to bfloat16 (2^-8 each) before and after, then float32
    assert abs(after.max().item() - tau) <= size * tau / before.max().item() * 4.1 * 2.0 ** -8
