"""GPU: 8-bit coding of activations and weights, and the product of coded
operands, against the fp64 oracle (oracle.coded).

Tolerance of the product.  The 8-bit matrix instruction adds the products of 8
consecutive k on a fixed-point grid that starts 13 binary places below the
largest product's exponent (test_product_alignment_of_the_matrix_cores pins
this): each of the other 7 products loses less than 2^-13 of that largest one,
so a group is off by at most 7 * 2^-13 * max|x w| over its k.  The group sums
and the accumulation over K are float32: K * 2^-23 * sum|x w| at most (2^-23
per addition, whether it rounds or truncates).  The one rounding to bf16 adds
2^-8 |y|.  That bound takes every loss at its largest and of one sign; over a
whole output the losses cancel, so the norm of the error must also stay within
the bf16 rounding's own 2^-8 of the norm."""
import sys

import numpy as np
import pytest
import torch

from oracle import coded
from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def announce(msg):
    sys.__stderr__.write(f"[gpu] {msg}\n")
    sys.__stderr__.flush()


def np64(t):
    return t.detach().float().cpu().double().numpy()


def randn(seed, *shape, std=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def wide(seed, r, k):
    """Rows from tiny to huge, a hot channel, zero blocks."""
    x = randn(seed, r, k).float()
    x *= torch.logspace(-100, 100, r, base=2.0)[:, None]
    x[:, k // 3] *= 30
    x[r // 2, : min(k, 128)] = 0
    return x.to(torch.bfloat16)


def check_code(c, x, tall):
    vals, exps = coded.code(np64(x), tall)
    got = np64(c.codes)
    assert np.array_equal(np.isnan(got), np.isnan(vals))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(vals))
    assert np.array_equal(c.scales.cpu().numpy().astype(np.int64) - 127, exps)
    return coded.values(vals, exps, tall)


def same(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


@pytest.mark.parametrize("T,K", [(1, 8), (1, 1152), (3, 136), (16, 128), (17, 264), (77, 712), (130, 1000)])
def test_act_code_and_expand_are_exact(gpu_lib, T, K):
    x = wide(T + K, T, K)
    announce(f"encode act {T} x {K}")
    c = binding.encode_act(x.to(DEV))
    want = check_code(c, x, 1)
    same(np64(c.expand()), want)
    # padding: codes past K are zero, scales past T are 1
    kq = c.blocks * 128
    assert not c.buf[:T * kq].view(T, kq)[:, K:].any()
    run = -(-T // 16) * 16
    at = -(-T * kq // 256) * 256
    assert (c.buf[at:at + c.blocks * run].view(c.blocks, run)[:, T:] == 127).all()


@pytest.mark.parametrize("N,K", [(1, 8), (5, 1152), (128, 128), (129, 264), (300, 712), (513, 136)])
def test_weight_code_is_exact(gpu_lib, N, K):
    w = wide(N + K, N, K)
    announce(f"encode weight {N} x {K}")
    check_code(binding.encode_weight(w.to(DEV)), w, 128)


def test_extreme_and_non_finite_elements(gpu_lib):
    """bf16's largest and smallest magnitudes, ties, and blocks with infinities
    and NaN among finite values or alone."""
    x = torch.zeros(9, 264)
    x[0, :3] = torch.tensor([3.3895e38, -3.3895e38, 1.0])
    x[1, :3] = torch.tensor([2.0 ** -133, -2.0 ** -126, 2.0 ** -130])
    x[2, :8] = torch.tensor([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 0.0])
    x[3, :4] = torch.tensor([float("inf"), 5.0, float("nan"), -3.0])
    x[4, :130] = float("inf")
    x[5, 256:] = float("-inf")
    x[6, 128:256] = 449.0
    x[7, 100] = 450.0
    x = x.to(torch.bfloat16)
    announce("encode extremes")
    c = binding.encode_act(x.to(DEV))
    same(np64(c.expand()), check_code(c, x, 1))
    check_code(binding.encode_weight(x.to(DEV)), x, 128)


def test_every_bf16_value(gpu_lib):
    """All 65536 bf16 patterns, ordered so that each block holds near
    neighbours in magnitude (every mantissa at every exponent, each sign)."""
    bits = torch.arange(1 << 16, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.bfloat16).view(512, 128)
    announce("encode every bf16 value")
    c = binding.encode_act(x.to(DEV))
    same(np64(c.expand()), check_code(c, x, 1))


def group_max_sum(xv, wv):
    """sum over groups of 8 consecutive k of max|x w| in the group, [T, N]."""
    if xv.shape[1] >= 1 << 16:  # few rows and columns
        return (xv.abs()[:, None] * wv.abs()[None]).unflatten(-1, (-1, 8)).amax(-1).sum(-1)
    tops = torch.zeros(xv.shape[0], wv.shape[0], dtype=torch.float64, device=xv.device)
    for k in range(0, xv.shape[1], 8):
        top = torch.zeros_like(tops)
        for j in range(k, min(k + 8, xv.shape[1])):
            top = torch.maximum(top, xv[:, j, None].abs() * wv[None, :, j].abs())
        tops += top
    return tops


def check_product(y, xv, wv):
    """y against the fp64 product of the coded values (float64 arrays, or
    float64 tensors on the GPU)."""
    xv, wv = torch.as_tensor(xv, device=DEV), torch.as_tensor(wv, device=DEV)
    ref, mass = xv @ wv.t().contiguous(), xv.abs() @ wv.abs().t().contiguous()
    tol = 2.0 ** -8 * ref.abs() + 7 * 2.0 ** -13 * group_max_sum(xv, wv) + xv.shape[1] * 2.0 ** -23 * mass
    got = y.double()
    assert got.shape == ref.shape
    bad = torch.nonzero(~((got - ref).abs() <= tol))
    assert len(bad) == 0, (bad[:4], got[tuple(bad[0])].item(), ref[tuple(bad[0])].item())
    assert (got - ref).norm() <= 2.0 ** -8 * ref.norm()


def test_product_alignment_of_the_matrix_cores(gpu_lib):
    """Two products of 2^16 that cancel, and one of +-2^(16 - s): kept while
    s <= 13, and as a float32 sum keeps it (23 places) when it lies in another
    group of 8 k or another block."""
    def run(big, at, s, sign):
        x, w = torch.zeros(1, 384), torch.zeros(16, 384)
        for i, v in zip(big, (256.0, -256.0)):
            x[0, i], w[:, i] = v, 256.0
        a = (16 - s) // 2
        x[0, at], w[:, at] = sign * 2.0 ** a, 2.0 ** (16 - s - a)
        y = binding.coded_linear(binding.encode_weight(w.to(torch.bfloat16).to(DEV)), x.to(torch.bfloat16).to(DEV))
        return y[0, 0].item() / (sign * 2.0 ** (16 - s))
    announce("alignment")
    for sign in (1, -1):
        assert all(run((0, 1), 2, s, sign) == 1.0 for s in range(8, 14))
        assert all(run((0, 1), at, s, sign) == 1.0 for s in (14, 20, 23) for at in (8, 40, 127))
        assert all(run((0, 300), 130, s, sign) == 1.0 for s in range(8, 24))


SHAPES = [(1, 16, 8), (1, 1, 128), (1, 4096, 1152), (2, 33, 264), (5, 100, 136), (15, 257, 712), (16, 129, 5376),
          (17, 64, 128), (17, 1, 8), (33, 127, 264), (64, 128, 1152), (65, 130, 2048), (100, 1001, 712),
          (128, 256, 128), (129, 513, 1160), (257, 300, 904), (300, 2000, 1000), (513, 1030, 520)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_product_matches_oracle(gpu_lib, T, N, K):
    x, w = randn(T + N, T, K), randn(N + K, N, K, std=K ** -0.5)
    x[:, K // 2] *= 24
    announce(f"product {T} x {N} x {K}")
    wc = binding.encode_weight(w.to(DEV))
    code = binding.ActCode(T, K)
    code.buf.fill_(0xA5)
    y = binding.coded_linear(wc, x.to(DEV), code=code)
    xv = check_code(code, x, 1)
    wv = check_code(wc, w, 128)
    check_product(y, xv, wv)
    # the coded form of the call gives the same bits, and what encode_act writes
    again = binding.encode_act(x.to(DEV))
    assert torch.equal(again.codes.view(torch.uint8), code.codes.view(torch.uint8))
    assert torch.equal(again.scales, code.scales)
    assert torch.equal(binding.coded_linear(wc, again), y)


@pytest.mark.parametrize("T,N,K", [(20, 5376, 21504), (1, 1024, 21504), (600, 640, 8192)])
def test_long_k_splits(gpu_lib, T, N, K):
    """Long K over few output tiles (K slices summed by a second launch, or one
    workgroup's waves); the coded values are taken from the call's own operands,
    which the coding tests hold to the oracle."""
    x, w = randn(1, T, K).to(DEV), randn(2, N, K, std=K ** -0.5).to(DEV)
    announce(f"product {T} x {N} x {K}")
    wc, xc = binding.encode_weight(w), binding.encode_act(x)
    f = torch.exp2(wc.scales.double() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    check_product(binding.coded_linear(wc, xc), xc.expand().double(), wc.codes.double() * f)


@pytest.mark.parametrize("T,N,K", [(2000, 8100, 264), (2048, 8200, 264), (11000, 600, 264), (700, 4000, 136),
                                   (16, 8200, 8200), (5, 12300, 5464)])
def test_sizes_that_take_the_other_tiles(gpu_lib, T, N, K):
    """Enough output tiles for 256 x 256, 256 x 128 and pairs of 128 x 128
    workgroups, and few tokens over 64 M codes; ragged in every dimension.  The
    reference runs in float64 on the GPU on the call's own coded operands."""
    announce(f"product {T} x {N} x {K}")
    wc, xc = binding.encode_weight(randn(T, N, K, std=K ** -0.5).to(DEV)), binding.encode_act(randn(N, T, K).to(DEV))
    f = torch.exp2(wc.scales.double() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    check_product(binding.coded_linear(wc, xc), xc.expand().double(), wc.codes.double() * f)


@pytest.mark.parametrize("T,N,K", [(1 << 20, 9, 8), (2, 1 << 20, 8), (3, 1 << 20, 8), (40, 1 << 20, 8), (2, 16, 1 << 20),
                                   (7, 16, 1 << 20), (40, 16, 1 << 20)])
def test_largest_extents(gpu_lib, T, N, K):
    """Each dimension at the largest the library takes."""
    announce(f"product {T} x {N} x {K}")
    w, x = randn(N, N, K, std=K ** -0.5).to(DEV), randn(T, T, K).to(DEV)
    wc = binding.encode_weight(w)
    code = binding.ActCode(T, K)
    y = binding.coded_linear(wc, x, code=code)
    f = torch.exp2(wc.scales.double() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    xv, wv = code.expand().double(), wc.codes.double() * f
    # a code is within half a step of E4M3: 2^-4 of the value, or 2^-10 of the block's scale
    for v, src in ((xv, x), (wv, w)):
        step = 2.0 ** -4 * src.double().abs() + 2.0 ** -10 * 2.0 ** -8 * src.double().abs().max()
        assert ((v - src.double()).abs() <= step).all()
    check_product(y, xv, wv)


@pytest.mark.parametrize("N,K", [(200, 8192), (8200, 136)])
def test_more_than_2_31_elements(gpu_lib, N, K):
    """270000 tokens: x, then y, hold more than 2^31 elements, and their bytes
    pass 2^32; each run of rows against its own coded values."""
    T, run = 270000, 30000
    gen = torch.Generator(DEV).manual_seed(93)
    x = torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, run):
        x[i:i + run] = torch.randn(run, K, generator=gen, device=DEV)
    announce(f"product {T} x {N} x {K}")
    wc, code = binding.encode_weight(randn(94, N, K, std=K ** -0.5).to(DEV)), binding.ActCode(T, K)
    y = binding.coded_linear(wc, x, code=code)
    f = torch.exp2(wc.scales.double() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    wv = wc.codes.double() * f
    for i in range(0, T, run):
        part = binding.encode_act(x[i:i + run])
        assert torch.equal(code.codes[i:i + run].view(torch.uint8), part.codes.view(torch.uint8))
        assert torch.equal(code.scales[i:i + run], part.scales)
        for at in (i, i + run - 40):  # the first and the last 40 rows of the run
            check_product(y[at:at + 40], part.expand()[at - i:at - i + 40].double(), wv)


def test_a_weight_of_more_than_2_32_codes(gpu_lib):
    """550000 rows of 8192 codes: each run of rows against its own coding, and
    the products' first, middle and last columns against the coded values."""
    N, K, run = 550000, 8192, 12800  # whole blocks of rows, the last run short
    gen = torch.Generator(DEV).manual_seed(95)
    w = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, N, run):
        w[i:i + run] = torch.randn(w[i:i + run].shape, generator=gen, device=DEV) * K ** -0.5
    announce(f"code {N} x {K}")
    wc = binding.encode_weight(w)
    parts = {}
    for i in range(0, N, run):
        part = binding.encode_weight(w[i:i + run])
        assert torch.equal(wc.codes[i:i + run].view(torch.uint8), part.codes.view(torch.uint8))
        assert torch.equal(wc.scales[i // 128:i // 128 + part.scales.shape[0]], part.scales)
        if i in (0, N // 2 // run * run, N // run * run):
            parts[i] = part
    assert len(parts) == 3
    for T in (1, 12, 60):
        announce(f"product {T} x {N} x {K}")
        xc = binding.encode_act(randn(96, T, K).to(DEV))
        y, xv = binding.coded_linear(wc, xc), xc.expand().double()
        for i, part in parts.items():
            f = torch.exp2(part.scales.double() - 127).repeat_interleave(128, 0)[:part.N].repeat_interleave(128, 1)
            at = slice(part.N - 40, part.N)
            check_product(y[:, i:i + part.N][:, at], xv, (part.codes.double() * f)[at].contiguous())


def test_blocks_of_very_different_scale(gpu_lib):
    """Scales from 2^-60 to 2^60 along K, tokens and weight rows: each block's
    own two scales enter its products."""
    T, N, K = 40, 300, 640
    x, w = randn(3, T, K).float(), randn(4, N, K).float()
    x *= torch.logspace(-20, 20, T, base=2.0)[:, None]
    for b in range(5):
        x[:, b * 128:(b + 1) * 128] *= 2.0 ** (12 * b - 30)
        w[:, b * 128:(b + 1) * 128] *= 2.0 ** (30 - 12 * b)
    w[128:256] *= 2.0 ** 20
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    wc = binding.encode_weight(w.to(DEV))
    for t in (1, 16, T):
        announce(f"scales T={t}")
        y = binding.coded_linear(wc, x[:t].to(DEV))
        check_product(y, check_code(binding.encode_act(x[:t].to(DEV)), x[:t], 1), check_code(wc, w, 128))


@pytest.mark.parametrize("T", [4, 50])
def test_nan_stays_in_its_row_and_column(gpu_lib, T):
    N, K = 200, 264
    x, w = randn(5, T, K), randn(6, N, K)
    x[2, 260] = float("inf")
    w[130, 7] = float("nan")
    announce(f"nan T={T}")
    y = np64(binding.coded_linear(binding.encode_weight(w.to(DEV)), x.to(DEV)))
    nan = np.isnan(y)
    want = np.zeros_like(nan)
    want[2, :] = True
    want[:, 130] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("T", [3, 70])
def test_neighbouring_memory_is_left_alone(gpu_lib, T):
    """Rows behind the last token of y and the bytes behind the coded buffer
    keep their values; a y that starts at an odd element is written whole."""
    N, K = 131, 392
    x, w = randn(7, T, K).to(DEV), randn(8, N, K).to(DEV)
    wc = binding.encode_weight(w)
    need = binding.ActCode(T, K).buf.numel()
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    code = binding.ActCode(T, K, buf=buf)
    flat = torch.full((T * N + 2 * N + 1,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = flat[1:1 + T * N].view(T, N)
    announce(f"canaries T={T}")
    binding.coded_linear(wc, x, y=y, code=code)
    assert (buf[need:] == 0x5A).all()
    assert flat[0] == 7.0 and (flat[1 + T * N:] == 7.0).all()
    assert torch.equal(y, binding.coded_linear(wc, x))


def test_no_tokens(gpu_lib):
    wc = binding.encode_weight(randn(9, 64, 64).to(DEV))
    y = binding.coded_linear(wc, torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert y.shape == (0, 64)


def test_side_stream_and_graph_replays(gpu_lib):
    """A call on a side stream, and a captured call replayed on new inputs with
    eager work between the replays, give the eager call's bits."""
    N, K = 640, 4096
    wc = binding.encode_weight(randn(10, N, K, std=0.02).to(DEV))
    for T in (1, 40):
        xs = [randn(20 + i, T, K).to(DEV) for i in range(4)]
        want = [binding.coded_linear(wc, x) for x in xs]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        announce(f"side stream T={T}")
        got = binding.coded_linear(wc, xs[1], stream=side)
        side.synchronize()
        assert torch.equal(got, want[1])
        x = xs[0].clone()
        g = torch.cuda.CUDAGraph()
        announce(f"capture T={T}")
        with torch.cuda.graph(g):
            y = binding.coded_linear(wc, x)
        for i in (1, 2, 3, 0):
            x.copy_(xs[i])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i])
            assert torch.equal(binding.coded_linear(wc, xs[3 - i]), want[3 - i])


def test_two_calls_at_once(gpu_lib):
    """Two streams, one weight: each call's outputs are its own."""
    N, K, T = 1000, 2048, 96
    wc = binding.encode_weight(randn(11, N, K, std=0.02).to(DEV))
    xs = [randn(30 + i, T, K).to(DEV) for i in range(2)]
    want = [binding.coded_linear(wc, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    announce("two streams")
    for _ in range(8):
        for i in (0, 1):
            got[i].append(binding.coded_linear(wc, xs[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_binding_refusals(gpu_lib):
    wc = binding.encode_weight(randn(12, 64, 128).to(DEV))
    x = randn(13, 8, 128).to(DEV)
    E = binding.WlError
    with pytest.raises(E, match="contiguous"):
        binding.encode_act(randn(14, 128, 8).to(DEV).t())
    with pytest.raises(E, match="bfloat16"):
        binding.encode_act(x.float())
    with pytest.raises(E, match="WeightCode"):
        binding.coded_linear(binding.encode_act(x), x)
    with pytest.raises(E, match="x must be"):
        binding.coded_linear(wc, randn(15, 8, 136).to(DEV))
    with pytest.raises(E, match="coded as"):
        binding.coded_linear(wc, binding.encode_act(randn(15, 8, 136).to(DEV)))
    with pytest.raises(E, match="y must be"):
        binding.coded_linear(wc, x, y=torch.empty(8, 65, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(E, match="ActCode of"):
        binding.coded_linear(wc, x, code=binding.ActCode(9, 128))
    with pytest.raises(E, match="bytes"):
        binding.ActCode(9, 128, buf=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(E, match="ws must be"):
        binding.coded_linear(wc, x, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(E, match="expected|device tensor"):
        binding.coded_linear(wc, x, y=torch.empty(8, 64, dtype=torch.bfloat16))
