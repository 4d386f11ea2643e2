"""examples/attention_step.py on the GPU: every link of its steps against float64, on what
the link before it gave."""

import numpy as np
import pytest

from oracle import decode as ref
from oracle import kv4
from tests.decode_cases import values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


def _weights(w):
    codes, scales, g = w
    s = scales.view(torch.int16).cpu().numpy().view(np.uint16) if scales.dtype == torch.float16 else scales.cpu().numpy()
    return codes.cpu().numpy(), s, None if g is None else np.float32(g.reshape(-1)[0].item())


def _near(got, want, bound, dtype=torch.bfloat16):
    if dtype == torch.bfloat16:
        bound = bound + 2.0**-8 * (np.abs(want) + bound)
    off = np.abs(values(got) - want) - bound
    assert np.all(off <= 0), float(off.max())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "int4"])
def test_attention_step(fmt):
    from examples import attention_step as ex

    block = ex.Block(fmt, vocab=500, hidden=256, q_heads=4, heads=2, D=64, adapters=3, rank=8, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    prompts = [torch.randint(0, 500, (n,), generator=gen, device="cuda") for n in (70, 1, 33)]
    ids = torch.tensor([1, -1, 2], dtype=torch.int32, device="cuda")
    H = values(block.cache_T)
    qkv_w, out_w, head_w = _weights(block.qkv), _weights(block.out), _weights(block.head)
    A, B, scale = (values(t) for t in block.adapters)
    seen = []

    def look(n, call, step, cache, table, lengths, asked, said, logits, answer):
        x = values(block.embed[call["tokens"]])
        y, b = ref.linear(x, qkv_w[0], qkv_w[1], fmt, values(block.qkv_T), qkv_w[2], 2)
        d, c = ref.lora(x, A, B, scale, call["ids"].cpu().numpy())
        _near(step.qkv.reshape(len(x), -1), y + d, b + c + 2 * ref.U * (np.abs(y) + np.abs(d)))
        # The new tokens' codes, bit for bit.
        q, k, v = (values(t) for t in step.qkv.split([4, 2, 2], dim=1))
        g = None if cache.k_global is None else np.float32(cache.k_global.item())
        slots = call["slots"].cpu().numpy()
        kc, ks, vc, vs = (t.cpu().numpy() for t in cache[:4])
        if fmt == "int4":
            ks, vs = ks.view(np.uint16), vs.view(np.uint16)
        page = kc.shape[2]
        for rows, codes, scales in ((k, kc, ks), (v, vc, vs)):
            want_c, want_s = kv4.append(rows, fmt, H, g)
            assert np.array_equal(codes[slots // page, :, slots % page], want_c)
            assert np.array_equal(scales[slots // page, :, slots % page], want_s)
        # Attention over the whole cache, as it is.
        L, tab = lengths.cpu().numpy(), table.cpu().numpy()
        start = call["q_start"].cpu().numpy() if "q_start" in call else np.arange(len(L) + 1)
        for r in range(len(L)):
            lo, hi = start[r], start[r + 1]
            for h in range(2):
                part = lambda c: tuple(t[tab[r], h].reshape(-1, t.shape[-1])[: L[r]] for t in c)  # noqa: E731
                pos = np.repeat(L[r] - (hi - lo) + np.arange(hi - lo), 2)
                want, bound = kv4.attention(q[lo:hi, 2 * h : 2 * h + 2].reshape(-1, 64), part((kc, ks)), part((vc, vs)), fmt,
                                            pos, 64**-0.5, T=H[h], kg=g, vg=g)
                got = values(step.attention[lo:hi, 2 * h : 2 * h + 2]).reshape(-1, 64)
                assert np.all(np.abs(got - want) <= bound)
        rows = step.attention if "last" not in call else step.attention[call["last"]]
        y, b = ref.linear(values(rows).reshape(len(rows), -1), out_w[0], out_w[1], fmt, None, out_w[2], 2)
        # Two roundings to bf16: the projection's and the sum's.
        b = b + 2.0**-8 * (np.abs(y) + b)
        _near(step.hidden, values(step.x) + y, b)
        y, b = ref.linear(values(step.hidden), head_w[0], head_w[1], fmt, None, head_w[2], 3)
        _near(step.logits, y, b, torch.float32)
        R = len(L)
        want, bound = ref.adjust_logits(values(step.logits), asked.cpu().numpy(), said.cpu().numpy(), [np.float32(1.3)] * R,
                                        np.zeros(R), [float(np.float32(0.1))] * R, [[]] * R, [[]] * R, None)
        _near(logits, want, bound, torch.float32)
        best = values(logits)
        order = np.argsort(-best, axis=1, kind="stable")[:, :5]
        assert np.array_equal(answer.top_ids.cpu().numpy(), order)
        seen.append(n)

    tokens, logprobs = ex.decode(block, prompts, ids, 4, page=16, look=look)
    assert seen == [0, 1, 2, 3] and tokens.shape == (4, 3) and torch.all(logprobs < 0)


def test_main_runs(capsys):
    from examples import attention_step as ex

    tokens, _ = ex.main(["--vocab", "300", "--hidden", "128", "--q-heads", "4", "--heads", "2", "--width", "64", "--adapters", "2",
                         "--rank", "8", "--requests", "2", "--prompt", "20", "--steps", "3"])
    assert tokens.shape == (3, 2) and "ms a step" in capsys.readouterr().out
