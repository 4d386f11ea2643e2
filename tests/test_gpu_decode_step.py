"""examples/decode_step.py on the GPU against the same block in float64, on the
weights that its codes stand for."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


def _blocks(x, T):
    return x if T is None else torch.einsum("...bi,boi->...bo", x.view(*x.shape[:-1], -1, T.shape[-1]),
                                            T).flatten(-2)


def _values(fmt, codes, scales, g):
    import mxfp4_activation_amd as wush

    return wush.dequant(fmt, codes, scales, g).double().cpu()


def _logits(block, tokens, ids, weights):
    """float64, with the experts chosen and weighted as the kernel did."""
    fmt = block.fmt
    x = block.embed[tokens].double().cpu()
    x = x + _blocks(x, _layout(block.proj_T)) @ _values(fmt, *block.proj).t()
    out = torch.zeros_like(x)
    for m in range(x.shape[0]):
        for e, w in zip(ids[m].tolist(), weights[m].double().tolist()):
            gs = [None if p.global_scale is None else p.global_scale[e : e + 1] for p in (block.gate_up, block.down)]
            gate, up = (_values(fmt, block.gate_up.codes[e], block.gate_up.scales[e], gs[0])
                        @ _blocks(x[m], _layout(block.gate_up.T))).chunk(2)
            h = torch.nn.functional.silu(gate) * up
            out[m] += w * (_values(fmt, block.down.codes[e], block.down.scales[e], gs[1])
                           @ _blocks(h, _layout(block.down.T[e])))
    return (x + out) @ _values(fmt, *block.head).t()


def _layout(T):
    return T.double().cpu()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "int4"])
def test_decode_step(fmt):
    from examples import decode_step as ex

    block = ex.Block(fmt, vocab=1000, hidden=256, experts=6, top_k=2, inner=96, seed=3)
    first = torch.tensor([5, 999, 0], device="cuda")
    ids, logprobs, entropies = ex.decode(block, first, 3)
    tokens = first
    for s in range(3):
        got, moe = block.logits(tokens)
        want = _logits(block, tokens, moe.ids.cpu(), moe.weights.cpu())
        # Six bf16 roundings (two results, two sums, transformed activations in two
        # planes not counted) of 2^-9 on the way to a logit, which sums 256 products:
        # their random parts stay below 2^-6 of the logits' spread.
        tol = 2.0**-6 * float(want.std()) * 4
        assert float((got.double().cpu() - want).abs().max()) <= tol
        lp = torch.log_softmax(want, dim=1)
        assert torch.allclose(logprobs[s].double().cpu(), lp.gather(1, ids[s].cpu()[:, None])[:, 0], rtol=0, atol=2 * tol)
        # The choice is the largest, or within the logits' error of it.
        assert torch.all(lp.gather(1, ids[s].cpu()[:, None])[:, 0] >= lp.max(dim=1).values - 2 * tol)
        assert torch.allclose(entropies[s].double().cpu(), -(lp.exp() * lp).sum(1), rtol=0, atol=4 * tol)
        tokens = ids[s]
    text = torch.cat([first[:1], ids[:, 0]])
    # Scored together or one by one: other shapes of workgroups, other orders of sums.
    assert torch.allclose(ex.score(block, text), logprobs[:, 0], rtol=0, atol=2 * tol)


def test_main_runs(capsys):
    from examples import decode_step as ex

    ids, _, _ = ex.main(["--vocab", "500", "--hidden", "128", "--inner", "64", "--experts", "4", "--top-k", "2",
                         "--batch", "2", "--steps", "2"])
    assert ids.shape == (2, 2) and "ms a step" in capsys.readouterr().out
