"""How far the divergence's gradient reaches into a model with layers of 8-bit codes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from post_weight_quantization_02_amd import pipeline as P  # noqa: E402
from test_gpu_int8_modules import VOCAB, formula, linear, model_and_texts  # noqa: E402


@pytest.mark.parametrize("quantize", [P.quantize_model_int8, P.quantize_model_fp8])
def test_behind_the_last_coded_layer_and_no_further(quantize):
    """A norm and a head behind the blocks get the formula's gradients; a norm in front of a layer
    of codes is refused in the forward pass, before anything is lost."""
    blocks, xs, _ = model_and_texts()
    head, norm = linear(VOCAB, 64, 9), torch.nn.LayerNorm(64, device="cuda")
    ids, lp = P.top_logprobs(blocks, lambda h: head(norm(h)), xs[:1], 8)[0]
    quantize(blocks)
    for p in blocks[1].parameters():
        p.requires_grad_(False)

    def hidden():
        x = xs[0]
        for b in blocks:
            x = b(x)
        return x

    for p in blocks[0].parameters():
        p.requires_grad_(False)
    params = [*norm.parameters(), *(p.requires_grad_(True) for p in head.parameters())]
    x = hidden()
    assert not x.requires_grad
    got = torch.autograd.grad(P.distill_loss(head(norm(x)), ids, lp, 1.0, True).mean(), params)
    ref = torch.autograd.grad(formula(head(norm(x)).double(), ids, lp.double(), 1.0, True).mean(), params)
    for u, v in zip(got, ref):
        assert (u - v).norm() <= 1e-3 * v.norm() + 1e-7
    blocks[0].ln1.weight.requires_grad_(True)
    with pytest.raises(ValueError, match="no backward"):
        hidden()
    with torch.no_grad():
        assert torch.equal(hidden(), x)
