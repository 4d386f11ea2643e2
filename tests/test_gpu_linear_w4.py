"""GPU parity of the linear layer with 4-bit weights (wush_linear_w4).

* Exact cases: small integers times codes with power-of-two scales, every
  partial sum an fp32 number, must match bit for bit.  This pins the nibble
  order, the scale placement, ragged rows and partial K steps.
* General cases: within the oracle's bound (oracle.decode), plus 2^-8 |y| for a
  bf16 result.
"""

import numpy as np
import pytest

from oracle import decode
from tests import decode_cases as dc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import mxfp4_activation_amd as wush

    wush.load()
    yield


def _call(fmt, xbits, codes, scales, T=None, gs=None, out_dtype=None, **kw):
    import mxfp4_activation_amd as wush

    return wush.linear_w4(fmt, dc.dev_bf16(xbits), dc.dev(codes), dc.dev_scales(fmt, scales),
                          T=None if T is None else dc.dev_bf16(T),
                          global_scale=None if gs is None else torch.tensor([gs], dtype=torch.float32).cuda(),
                          out_dtype=out_dtype or torch.float32, **kw)


# (M, N, K): one element past and short of the 16-row tiles, the token tiles (16,
# 32, 64), the 128-element steps and the steps shared among the waves.
_SHAPES = [(1, 1, 32), (1, 16, 128), (2, 17, 160), (3, 33, 96), (5, 31, 1024), (16, 48, 1152), (17, 16, 256),
           (31, 50, 544), (32, 33, 2048), (33, 64, 224), (64, 40, 1312), (65, 15, 384), (130, 35, 416)]


@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("M,N,K", _SHAPES)
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_exact(fmt, M, N, K, transform):
    rng = np.random.default_rng(M * 1000 + N + K)
    if fmt == "nvfp4" and K % 64 == 32:
        K += 16  # half a group of 32
    G = decode.GROUP[fmt]
    codes, scales = dc.weights(rng, fmt, (N,), K, exact=True)
    x, xb = dc.bf16(rng.integers(-3, 4, size=(M, K)))
    T = Tb = None
    if transform:
        # Four entries of +-1 a row.
        T = np.zeros((K // G, G, G))
        at = rng.integers(0, G, size=(K // G, G, 4))
        np.put_along_axis(T, at, rng.choice([-1.0, 1.0], size=at.shape), 2)
        T, Tb = dc.bf16(T)
    gs = 0.5 if fmt == "nvfp4" else None
    want, _ = decode.linear(x, codes, scales, fmt, T, gs)
    got = _call(fmt, xb, codes, scales, Tb, gs)
    assert np.array_equal(dc.values(got), want)
    got16 = _call(fmt, xb, codes, scales, Tb, gs, torch.bfloat16)
    assert torch.equal(got16, got.to(torch.bfloat16))


# Many weight rows for the same token counts: the shapes of workgroups that serve
# those, each with a last workgroup that is not full.
_WIDE = [(3, 12400, 64), (6, 4700, 288), (13, 8200, 160), (12, 16500, 64), (16, 8200, 2080), (24, 8300, 96),
         (50, 4200, 160), (50, 16500, 64), (40, 33000, 32)]


@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("M,N,K", _WIDE)
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_exact_wide(fmt, M, N, K, transform):
    test_exact(fmt, M, N, K, transform)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 257, 2048), (4, 100, 5120), (20, 130, 1504), (64, 96, 1024)])
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_general(fmt, M, N, K, transform, out):
    rng = np.random.default_rng(7 + M + K)
    G = decode.GROUP[fmt]
    codes, scales = dc.weights(rng, fmt, (N,), K)
    x, xb = dc.bf16(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20.0, 1.0))
    T, Tb = dc.bf16(rng.standard_normal((K // G, G, G)) / G**0.5) if transform else (None, None)
    gs = float(np.float32(3.7e-5)) if fmt == "nvfp4" else None
    dt = torch.float32 if out == "f32" else torch.bfloat16
    want, bound = decode.linear(x, codes, scales, fmt, T, gs, planes=3 if out == "f32" else 2)
    if out == "bf16":
        bound = bound + 2.0**-8 * np.abs(want)
    err = np.abs(dc.values(_call(fmt, xb, codes, scales, Tb, gs, dt)) - want)
    assert np.all(err <= bound), np.max(err / bound)


def test_int4_lowest_code():
    """Code 8 is -8: no quantizer here writes it, but dequant reads it so."""
    codes = np.full((3, 64), 0x88, dtype=np.uint8)
    scales = np.full((3, 4), np.float16(0.25).view(np.uint16))
    x, xb = dc.bf16(np.ones((1, 128)))
    assert dc.values(_call("int4", xb, codes, scales)).tolist() == [[-256.0] * 3]


@pytest.mark.parametrize("code", [0, 1, 253])
def test_mxfp4_scale_extremes(code):
    """Codes of E8M0 at both ends: 2^-127 and 2^126 per element, in fp32."""
    codes = np.full((16, 64), 0x22, dtype=np.uint8)  # all 1.0
    scales = np.full((16, 4), code, dtype=np.uint8)
    x = np.zeros((2, 128))
    x[0, 5], x[1, 100] = 1.0, 0.5 if code > 200 else 2.0**30
    x, xb = dc.bf16(x)
    want, _ = decode.linear(x, codes, scales, "mxfp4")
    got = dc.values(_call("mxfp4", xb, codes, scales))
    # Below the smallest normal fp32 number the matrix cores may flush to zero.
    assert np.all(np.abs(got - want) <= 2.0**-126)


@pytest.mark.parametrize("transform", [False, True])
def test_row_stride_and_out(transform):
    rng = np.random.default_rng(11)
    M, N, K = 6, 40, 256
    codes, scales = dc.weights(rng, "mxfp4", (N,), K, exact=True)
    x, xb = dc.bf16(rng.integers(-3, 4, size=(M, K)))
    T = np.tile(np.eye(32), (K // 32, 1, 1))
    wide = dc.dev_bf16(np.pad(xb, ((0, 0), (8, 16))))[:, 8 : 8 + K]
    assert not wide.is_contiguous()
    import mxfp4_activation_amd as wush

    out = torch.full((M + 2, N), 7.0, device="cuda")
    got = wush.linear_w4("mxfp4", wide, dc.dev(codes), dc.dev(scales), T=dc.dev_bf16(dc.bf16(T)[1]) if transform else None,
                         out_dtype=torch.float32, out=out[1:-1])
    want, _ = decode.linear(x, codes, scales, "mxfp4")
    assert np.array_equal(dc.values(got), want)
    assert torch.all(out[0] == 7.0) and torch.all(out[-1] == 7.0)


def test_unaligned_scale_rows():
    """Rows of a stacked weight start at any byte of the scales."""
    rng = np.random.default_rng(12)
    K = 160
    codes, scales = dc.weights(rng, "mxfp4", (37,), K, exact=True)
    x, xb = dc.bf16(rng.integers(-3, 4, size=(2, K)))
    import mxfp4_activation_amd as wush

    dcodes, dscales = dc.dev(codes)[3:], dc.dev(scales)[3:]
    got = wush.linear_w4("mxfp4", dc.dev_bf16(xb), dcodes, dscales, out_dtype=torch.float32)
    assert np.array_equal(dc.values(got), decode.linear(x, codes[3:], scales[3:], "mxfp4")[0])


def test_weights_of_the_quantizer():
    """quantizer -> linear layer: the product of the dequantized values."""
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(13)
    N, K = 48, 512
    W, Wb = dc.bf16(rng.standard_normal((N, K)) * 0.02)
    x, xb = dc.bf16(rng.standard_normal((3, K)))
    for fmt in dc.FMTS:
        G = decode.GROUP[fmt]
        bank = wush.fixed_transforms("hadamard", K // G, G, "cuda")
        gs = wush.nvfp4_global_scale(dc.dev_bf16(Wb), bank) if fmt == "nvfp4" else None
        codes, scales = wush.quant(fmt, dc.dev_bf16(Wb), bank, global_scale=gs)
        got = wush.linear_w4(fmt, dc.dev_bf16(xb), codes, scales, T=bank, global_scale=gs, out_dtype=torch.float32)
        Wq = dc.values(wush.dequant(fmt, codes, scales, gs))
        xt, _ = decode.blocks(x, dc.values(bank))
        sc = scales.cpu().numpy()
        _, bound = decode.linear(x, codes.cpu().numpy(), sc.view(np.uint16) if fmt == "int4" else sc, fmt,
                                 dc.values(bank), None if gs is None else float(gs), planes=3)
        # dequant rounds the scale product once more.
        assert np.all(np.abs(dc.values(got) - xt @ Wq.T) <= bound + decode.U * (np.abs(xt) @ np.abs(Wq).T))
        # The block Hadamard transform is orthogonal: the result is near x W^T.
        assert np.linalg.norm(dc.values(got) - x @ W.T) < 0.2 * np.linalg.norm(x @ W.T)


def test_empty():
    import mxfp4_activation_amd as wush

    codes, scales = torch.zeros(8, 64, dtype=torch.uint8).cuda(), torch.zeros(8, 4, dtype=torch.uint8).cuda()
    x = torch.zeros(0, 128, dtype=torch.bfloat16).cuda()
    assert wush.linear_w4("mxfp4", x, codes, scales).shape == (0, 8)
    x = torch.zeros(2, 128, dtype=torch.bfloat16).cuda()
    assert wush.linear_w4("mxfp4", x, codes[:0], scales[:0]).shape == (2, 0)


def test_side_stream_and_graph_replay():
    import mxfp4_activation_amd as wush

    rng = np.random.default_rng(14)
    K, N, G = 1024, 80, 32
    codes, scales = dc.weights(rng, "int4", (N,), K)
    dcodes, dscales = dc.dev(codes), dc.dev_scales("int4", scales)
    T = dc.dev_bf16(dc.bf16(rng.standard_normal((K // G, G, G)) / 6)[1])
    xs = [dc.dev_bf16(dc.bf16(rng.standard_normal((4, K)))[1]) for _ in range(3)]
    eager = [wush.linear_w4("int4", x, dcodes, dscales, T=T) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = torch.empty_like(xs[0])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [wush.linear_w4("int4", v, dcodes, dscales, T=T) for v in xs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = wush.linear_w4("int4", x, dcodes, dscales, T=T)
    torch.cuda.synchronize()
    for a, b in zip(eager, again):
        assert torch.equal(a, b)
    for turn in range(3):
        x.copy_(xs[turn])
        graph.replay()
        assert torch.equal(y, eager[turn])
        torch.cuda.synchronize()


@pytest.mark.parametrize("transform", [False, True])
@pytest.mark.parametrize("M,K", [(3, 32), (4, 160), (7, 1056), (20, 160), (40, 2080)])
@pytest.mark.parametrize("fmt", dc.FMTS)
def test_not_finite_rows_stay_their_own(fmt, M, K, transform):
    """Rows with an infinity or a NaN anywhere, also where a step ends past K, have
    no finite result; every other row is exact."""
    rng = np.random.default_rng(M + K)
    G, N = decode.GROUP[fmt], 50
    codes, scales = dc.weights(rng, fmt, (N,), K, exact=True)
    x, xb = dc.bf16(rng.integers(-3, 4, size=(M, K)))
    T = np.tile(np.eye(G), (K // G, 1, 1))
    bad = {0: (0, 0x7F80), M // 2: (K - 1, 0xFF80), M - 1: (K // 2, 0x7FC0)}
    for row, (k, bits) in bad.items():
        xb[row, k] = bits
    gs = 1.0 if fmt == "nvfp4" else None
    want, _ = decode.linear(x, codes, scales, fmt, None, gs)
    got = dc.values(_call(fmt, xb, codes, scales, dc.bf16(T)[1] if transform else None, gs))
    keep = [m for m in range(M) if m not in bad]
    assert not np.isfinite(got[sorted(bad)]).any()
    assert np.array_equal(got[keep], want[keep])
