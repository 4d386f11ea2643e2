"""Adapters and logits' adjustments where they can go wrong: captured graphs, other
streams, operands beyond 4 GiB, many tokens."""

import numpy as np
import pytest

from oracle import decode as ref
from tests.decode_cases import dev, values
from tests.test_gpu_adjust_logits import Case as Logits
from tests.test_gpu_lora import Case as Lora

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


def _captured(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


@pytest.mark.parametrize("M", [2, 30])
@pytest.mark.parametrize("T", [False, True])
def test_lora_graph_replays(M, T):
    import mxfp4_activation_amd as wush

    a = Lora("mxfp4", M, 300, 512, 16, 4, T=T).args()
    graph, out = _captured(lambda: wush.linear_w4_lora(**a))
    gen = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(4):
        a["ids"].copy_(torch.randint(-1, 4, (M,), generator=gen, device="cuda").int())
        a["x"].copy_(torch.randn(M, 512, generator=gen, device="cuda"))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        assert torch.equal(wush.linear_w4_lora(**a), replayed)


def test_adjust_graph_replays_and_feeds_logprobs():
    import mxfp4_activation_amd as wush

    c = Logits(3, 5001, "bf16", 40, 20, 5, True)
    kw, nothing = c.kwargs(), torch.full((3,), -1, device="cuda")
    logits = c.logits.clone()

    def call():
        return wush.token_logprobs(wush.adjust_logits(logits, **kw), nothing, top=4)

    graph, out = _captured(call)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(4):
        logits.copy_(4 * torch.randn(3, 5001, generator=gen, device="cuda"))
        kw["output"].copy_(torch.randint(0, 5001, kw["output"].shape, generator=gen, device="cuda").int())
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in out]
        for x, y in zip(call(), replayed):
            assert torch.equal(x, y)
    # A row that its mask leaves nothing of lists nothing.
    assert torch.all(replayed[2][0] == -1) and torch.all(torch.isneginf(replayed[3][0]))


def test_two_streams_at_once():
    import mxfp4_activation_amd as wush

    a, b = Lora("int4", 20, 400, 512, 32, 5, T=True).args(), Lora("nvfp4", 3, 1000, 256, 8, 2).args()
    c = Logits(9, 20000, "f32", 300, 200, 40, True)
    kw = c.kwargs()
    want = wush.linear_w4_lora(**a), wush.linear_w4_lora(**b), wush.adjust_logits(c.logits, **kw)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(6):
        for s, f in zip(streams, (lambda: wush.linear_w4_lora(**a), lambda: wush.linear_w4_lora(**b),
                                  lambda: wush.adjust_logits(c.logits, **kw))):
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 3])


def test_lora_many_tokens_and_adapters_beyond_4_gib():
    """600 tokens in chunks; of 70 adapters with 4.7 GB of B the last one."""
    import mxfp4_activation_amd as wush

    c = Lora("mxfp4", 600, 100, 64, 8, 6)
    want, bound = c.want(3)
    assert np.all(np.abs(values(wush.linear_w4_lora(**c.args(), out_dtype=torch.float32)) - want) <= bound)

    N, K, r, E = 65536, 64, 512, 70
    c = Lora("mxfp4", 10, N, K, r, 1)
    A = torch.zeros(E, r, K, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(E, N, r, dtype=torch.bfloat16, device="cuda")
    assert B.numel() * 2 > 4 << 30
    a = c.args()
    A[-1], B[-1] = a["adapters"].A[0], a["adapters"].B[0]
    scale = torch.ones(E, device="cuda")
    scale[-1] = a["adapters"].scale[0]
    for M in (10, 3):
        x = a["x"][:M]
        got = wush.linear_w4_lora("mxfp4", x, a["codes"], a["scales"], wush.LoraAdapters(A, B, scale),
                                  torch.full((M,), E - 1, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
        y, b0 = ref.linear(c.x[:M], c.codes, c.scales, "mxfp4", planes=3)
        d, b1 = ref.lora(c.x[:M], c.A, c.B, c.s, np.zeros(M, int))
        bound = b0 + b1 + 2 * ref.U * (np.abs(y) + np.abs(d))
        assert np.all(np.abs(values(got) - (y + d)) <= bound)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_beyond_4_gib(dtype):
    import mxfp4_activation_amd as wush

    V = 140001
    R = (5 << 30) // (V * torch.finfo(dtype).bits // 8)
    logits = torch.zeros(R, V, dtype=dtype, device="cuda")
    logits[:, 7] = 2.0
    rep = torch.full((R,), 4.0, device="cuda")
    bias_ids = torch.full((R, 1), V - 1, dtype=torch.int32, device="cuda")
    bias = torch.arange(R, device="cuda").float()[:, None] % 64 + 1
    seen = torch.full((R, 1), 7, dtype=torch.int32, device="cuda")
    out = wush.adjust_logits(logits, output=seen, repetition=rep, bias_ids=bias_ids, bias=bias, out=logits)
    assert torch.all(out[:, 7] == 0.5) and torch.equal(out[:, V - 1].float(), bias[:, 0])
    assert int((out[-1] != 0).sum()) == 2 and int((out[R // 2] != 0).sum()) == 2


def test_long_lists_and_many_biases():
    """Lists longer than what a workgroup asks for at first; one token very often."""
    c = Logits(2, 3000, "f32", 9000, 7001, 1500, False)
    c.output[:] = 11
    c.output[:, -1] = 2999
    c.freq = np.array([1e-3, -2e-4], np.float32)
    import mxfp4_activation_amd as wush

    c.check(values(wush.adjust_logits(c.logits, **c.kwargs())))
    c.bias_ids[:] = 5  # every bias at one token
    c.check(values(wush.adjust_logits(c.logits, **c.kwargs())))
