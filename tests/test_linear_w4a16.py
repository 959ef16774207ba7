"""linear_w4a16 and quantize_weight_w4a16 against the definition in float64.

Bound per output: the one rounding to 16 bits (half a step of y) plus the fp32
sums.  With A = sum_k |x_k| (|s q_k| + |o|), a sum of K terms in any order is
off by at most K u A, u = 2^-23 (a matrix unit may truncate where an adder
rounds); the scale's product and the joining of groups and slices add a few
more roundings: (K + 16) 2^-23 A."""

import pytest
import torch

import w4a4_hadamard_rotated_b200 as w4

DTYPES = [torch.bfloat16, torch.float16]


def make(M, K, N, group, dtype, offset, bias, seed=0):
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.int32).to(torch.uint8).view(torch.int8)
    scale = (torch.rand(N, K // group, generator=gen) * 0.02 + 0.001).to(dtype)
    off = (torch.randn(N, K // group, generator=gen) * 0.02).to(dtype) if offset else None
    x = torch.randn(M, K, generator=gen).to(dtype)
    b = torch.randn(N, generator=gen).to(dtype) if bias else None
    return x, codes, scale, off, b


def unpack(codes):
    c = codes.to(torch.int32)
    low, high = ((c & 15) ^ 8) - 8, c >> 4
    return torch.stack((low, high), 2).flatten(1).double()


def reference(x, codes, scale, off, b):
    q = unpack(codes)
    group = q.shape[1] // scale.shape[1]
    sq = q * scale.double().repeat_interleave(group, 1)
    o = off.double().repeat_interleave(group, 1) if off is not None else torch.zeros_like(sq)
    y = x.double() @ (sq + o).t()
    A = x.double().abs() @ (sq.abs() + o.abs()).t()
    if b is not None:
        y = y + b.double()
        A = A + b.double().abs()
    return y, A


def check(y, ref, A, K):
    dtype = y.dtype
    tol = torch.finfo(dtype).eps / 2 * (ref.abs() + (K + 16) * 2.0 ** -23 * A) + (K + 16) * 2.0 ** -23 * A + 2.0 ** -25
    bad = (y.double().cpu() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def on_gpu(*ts):
    return [t.cuda() if t is not None else None for t in ts]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,group,offset,bias", [
    (1, 32, 1, 32, False, False),            # the smallest
    (1, 64, 7, 32, True, True),
    (1, 128, 17, 128, False, True),
    (2, 96, 33, 32, True, False),            # K not a multiple of 64
    (3, 160, 130, 32, False, False),
    (1, 1984, 257, 64, True, True),          # ragged against any 128-column step
    (5, 3072, 129, 128, False, True),
    (7, 5120, 64, 64, True, False),
    (8, 12288, 40, 128, True, True),
    (9, 544, 100, 32, False, True),          # more than one block of eight rows
    (16, 13824, 72, 128, False, False),
    (17, 1024, 48, 64, True, True),
    (33, 320, 19, 64, False, True),
    (64, 2048, 50, 128, True, True),
    (1, 3072, 3072, 128, False, False),
    (1, 5120, 6000, 64, True, True),
    (1, 131072, 9, 128, True, False),        # the longest row
    (64, 131072, 3, 32, False, False),
])
def test_linear_matches_definition(cuda_lib, dtype, M, K, N, group, offset, bias):
    args = make(M, K, N, group, dtype, offset, bias, seed=M + K + N)
    x, codes, scale, off, b = on_gpu(*args)
    y = w4.linear_w4a16(x, codes, scale, offset=off, bias=b)
    assert y.shape == (M, N) and y.dtype == dtype
    check(y, *reference(*args), K)
    assert torch.equal(y, w4.linear_w4a16(x, codes, scale, offset=off, bias=b))   # deterministic


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 3, 16, 20])
def test_strided_rows_and_output(cuda_lib, dtype, M):
    """x a column slice of a wider buffer, y a slice of an oddly wide one: the
    padding keeps its values, the result equals the compact call's."""
    K, N = 640, 77
    x, codes, scale, off, b = on_gpu(*make(M, K, N, 64, dtype, True, True, seed=5))
    wide = torch.randn(M, K + 24, device="cuda").to(dtype)
    wide[:, 8:8 + K] = x
    out = torch.full((M, N + 3), 7.0, device="cuda", dtype=dtype)
    w4.linear_w4a16(wide[:, 8:8 + K], codes, scale, offset=off, bias=b, out=out[:, 1:1 + N])
    assert torch.equal(out[:, 1:1 + N], w4.linear_w4a16(x, codes, scale, offset=off, bias=b))
    assert (out[:, :1] == 7).all() and (out[:, 1 + N:] == 7).all()


@pytest.mark.gpu
def test_rows_do_not_reach_one_another(cuda_lib):
    """A NaN row and an infinite one leave the others as they are."""
    x, codes, scale, off, b = on_gpu(*make(11, 512, 90, 64, torch.bfloat16, True, True))
    y = w4.linear_w4a16(x, codes, scale, offset=off, bias=b)
    x2 = x.clone()
    x2[3] = float("nan")
    x2[9, 5] = float("inf")
    y2 = w4.linear_w4a16(x2, codes, scale, offset=off, bias=b)
    keep = [m for m in range(11) if m not in (3, 9)]
    assert torch.equal(y[keep], y2[keep])
    assert torch.isnan(y2[3]).all() and not torch.isfinite(y2[9]).any()


@pytest.mark.gpu
def test_empty_batch(cuda_lib):
    x, codes, scale, _, _ = on_gpu(*make(1, 64, 9, 32, torch.float16, False, False))
    assert w4.linear_w4a16(x[:0], codes, scale).shape == (0, 9)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("asymmetric", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (37, 256, 64), (130, 1024, 128), (9, 96, 32)])
def test_quantizer(cuda_lib, dtype, asymmetric, N, K, group):
    """Scales and offsets follow their formulas in fp32 (one rounding to 16
    bits each), and every code is a nearest one of the grid they span."""
    gen = torch.Generator().manual_seed(N + K)
    W = torch.randn(N, K + 4, generator=gen) * 0.02
    W[0, :group] = 0                                        # a group of zeros
    Wq, scale, offset = w4.quantize_weight_w4a16(W.cuda()[:, :K], group, dtype, asymmetric)
    w = W[:, :K].view(N, K // group, group)
    q = unpack(Wq.cpu()).view(N, K // group, group)
    if asymmetric:
        lo, hi = w.amin(2), w.amax(2)
        want = ((hi - lo) / 15).to(dtype)
        assert torch.equal(scale.cpu(), want)
        # 8 s + lo with one fp32 rounding: exact in fp64, then to fp32 and to 16 bits
        assert torch.equal(offset.cpu(), (8 * want.double() + lo.double()).float().to(dtype))
        o = offset.cpu().double()[:, :, None]
        assert q.min() >= -8 and q.max() <= 7
    else:
        assert offset is None
        assert torch.equal(scale.cpu(), (w.abs().amax(2) / 7).to(dtype))
        o = torch.zeros(())
        assert q.min() >= -7 and q.max() <= 7
    s = scale.cpu().double()[:, :, None]
    least = -8 if asymmetric else -7
    exact = torch.where(s > 0, (w.double() - o) / s.clamp(min=1e-300), torch.zeros(()).double()).clamp(least, 7)
    # the fp32 quotient is within 2^-23 (|w| + |o|) / s of the exact one, so a code may differ only that near a half
    slack = 2.0 ** -22 * (w.double().abs() + o.abs()) / s.clamp(min=1e-300) + 1e-12
    assert ((q - exact).abs() <= 0.5 + torch.where(s > 0, slack, torch.zeros(()).double())).all()
    assert (q[0, 0] == 0).all() or asymmetric and (scale[0, 0] == 0)


@pytest.mark.gpu
def test_quantized_product_is_near_the_full_one(cuda_lib):
    """Quantise, then multiply: the product with the dequantised weight, to the bound."""
    gen = torch.Generator().manual_seed(3)
    W = torch.randn(96, 512, generator=gen) * 0.02
    x = torch.randn(4, 512, generator=gen).to(torch.bfloat16)
    Wq, scale, offset = w4.quantize_weight_w4a16(W.cuda(), 64, torch.bfloat16, asymmetric=True)
    y = w4.linear_w4a16(x.cuda(), Wq, scale, offset=offset)
    check(y, *reference(x, Wq.cpu(), scale.cpu(), offset.cpu(), None), 512)


@pytest.mark.gpu
def test_graph_replay_and_other_stream(cuda_lib):
    """Captured twice and replayed on new inputs; run on a side stream."""
    x, codes, scale, off, b = on_gpu(*make(2, 1024, 300, 64, torch.bfloat16, True, True))
    x2 = torch.randn_like(x.float()).to(x.dtype)
    want, want2 = (w4.linear_w4a16(t, codes, scale, offset=off, bias=b) for t in (x, x2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = w4.linear_w4a16(x, codes, scale, offset=off, bias=b)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    buf = x.clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w4.linear_w4a16(buf, codes, scale, offset=off, bias=b))
        graphs.append(g)
    for g, o in zip(graphs, outs):
        buf.copy_(x2)
        g.replay()
        assert torch.equal(o, want2)
        buf.copy_(x)
        g.replay()
        assert torch.equal(o, want)


@pytest.mark.gpu
def test_binding_refusals(cuda_lib):
    x, codes, scale, off, b = on_gpu(*make(2, 128, 16, 32, torch.bfloat16, True, True))
    bad = [
        (TypeError, lambda: w4.linear_w4a16(x.float(), codes, scale)),
        (TypeError, lambda: w4.linear_w4a16(x, codes, scale.half())),
        (TypeError, lambda: w4.linear_w4a16(x, codes.view(torch.uint8), scale)),
        (ValueError, lambda: w4.linear_w4a16(x, codes[:, :32], scale)),
        (ValueError, lambda: w4.linear_w4a16(x, codes, scale[:8])),
        (ValueError, lambda: w4.linear_w4a16(x, codes, scale[:, :3])),
        (ValueError, lambda: w4.linear_w4a16(x, codes, scale, offset=off[:, :2])),
        (ValueError, lambda: w4.linear_w4a16(x, codes, scale, bias=b[:4])),
        (ValueError, lambda: w4.linear_w4a16(x[0], codes, scale)),
        (ValueError, lambda: w4.linear_w4a16(x.t().contiguous().t(), codes, scale)),
        (ValueError, lambda: w4.linear_w4a16(x, codes, scale, out=torch.empty(3, 16, device="cuda", dtype=x.dtype))),
        (w4.W4A4Error, lambda: w4.linear_w4a16(x, codes, scale[:, :1].contiguous().expand(16, 1).repeat(1, 8))),
        (w4.W4A4Error, lambda: w4.linear_w4a16(x.repeat(40, 1), codes, scale)),
        (ValueError, lambda: w4.quantize_weight_w4a16(torch.zeros(4, 128, device="cuda"), 48)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


@pytest.mark.gpu
def test_expired_waits_end_the_call(cuda_lib):
    """With a wait limit of a few nanoseconds the kernel gives up a wait that it
    has to wait for (data may be there already), reports it and leaves the
    context as it was; the next call is right."""
    cases = [on_gpu(*make(M, 5120, 4000, 64, torch.bfloat16, True, False)) for M in (1, 5, 16)]
    good = [w4.linear_w4a16(x, c, s, offset=o) for x, c, s, o, _ in cases]
    w4.debug_set_wait_limit(5)
    seen = set()
    try:
        for x, c, s, o, _ in cases * 5:
            w4.linear_w4a16(x, c, s, offset=o)
            seen.add(w4.last_device_error())
    finally:
        w4.debug_set_wait_limit(0)
    assert seen <= {0, 8}
    for (x, c, s, o, _), g in zip(cases, good):
        assert torch.equal(w4.linear_w4a16(x, c, s, offset=o), g)
    assert w4.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [9, 12, 16, 25])
@pytest.mark.parametrize("K,N", [(12288, 3001), (5120, 5000), (640, 9000), (9600, 33), (2080, 700)])
@pytest.mark.parametrize("group,offset", [(32, True), (32, False), (128, True)])
def test_every_split_of_more_rows(cuda_lib, M, K, N, group, offset):
    """More than eight rows: 32 rows and 12 warps a CTA, or 16 and 8."""
    if K % group:
        group = 32
    x, codes, scale, off, b = on_gpu(*make(M, K, N, group, torch.float16, offset, True, seed=N))
    y = w4.linear_w4a16(x, codes, scale, offset=off, bias=b)
    check(y, *[t.cpu() for t in reference(x, codes, scale, off, b)], K)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 3, 8])
@pytest.mark.parametrize("K,N", [(4096, 1000), (4096, 4090), (5120, 5000), (640, 9000), (1536, 2300), (9600, 33)])
@pytest.mark.parametrize("group,offset", [(32, True), (64, False), (128, True)])
def test_every_split_of_rows_and_warps(cuda_lib, M, K, N, group, offset):
    """Shapes that take 16 or 32 rows and 8 or 16 warps a CTA, several tiles and ragged ones."""
    args = make(M, K, N, group, torch.bfloat16, offset, True, seed=N)
    x, codes, scale, off, b = on_gpu(*args)
    y = w4.linear_w4a16(x, codes, scale, offset=off, bias=b)
    # the reference on the GPU, in float64
    check(y, *[t.cpu() for t in reference(x, codes, scale, off, b)], K)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 11])
def test_weights_past_32_bit_offsets(cuda_lib, M):
    """More than 2^31 bytes of codes: the last rows, and some before them."""
    K, N, tail = 1024, 2 ** 31 // 512 + 1003, 2000
    x, codes, scale, off, b = on_gpu(*make(M, K, tail, 128, torch.bfloat16, True, True))
    far = lambda t: torch.cat((torch.zeros(N - tail, *t.shape[1:], device="cuda", dtype=t.dtype), t))
    y = w4.linear_w4a16(x, far(codes), far(scale), offset=far(off), bias=far(b))
    check(y[:, -tail:], *[t.cpu() for t in reference(x, codes, scale, off, b)], K)
    assert (y[:, :-tail] == 0).all() and w4.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 16])
def test_expired_waits_are_reported(cuda_lib, M):
    """Weights of 77 MB that are not in L2: some warp has to wait for a stage,
    and with a limit of a few nanoseconds it gives up and says so. The call after it is right."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    K, N = 5120, 30000
    codes = torch.randint(-128, 128, (N, K // 2), generator=gen, device="cuda", dtype=torch.int8)
    scale = torch.full((N, K // 64), 0.01, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    good = w4.linear_w4a16(x, codes, scale)
    cold = torch.empty(2 ** 28, device="cuda", dtype=torch.uint8)
    w4.debug_set_wait_limit(5)
    try:
        for i in range(3):
            cold.fill_(i)
            torch.cuda.synchronize()
            w4.linear_w4a16(x, codes, scale)
            assert w4.last_device_error() == 8
    finally:
        w4.debug_set_wait_limit(0)
    assert torch.equal(w4.linear_w4a16(x, codes, scale), good) and w4.last_device_error() == 0


def slice_edges(K):
    """Columns beside the ends of the slices of k that 8, 12 and 16 warps take, in steps of 128."""
    units, cols = (K + 127) // 128, set()
    for warps in (8, 12, 16):
        for w in range(warps + 1):
            end = min(units * w // warps * 128, K)
            cols |= set(range(max(end - 32, 0), min(end + 32, K)))
    return sorted(cols)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 2, 5, 8, 16, 20])
@pytest.mark.parametrize("K,N", [(32, 5), (96, 33), (640, 9000), (1984, 257), (2080, 700), (4096, 1000), (5120, 5000),
                                 (9600, 33), (12288, 3001), (131072, 9)])
def test_whole_numbers_are_exact(cuda_lib, dtype, M, K, N):
    """Small whole x, scales 1/2, 1 and 2, offsets that are multiples of 1/2:
    every product and partial sum is a multiple of 1/2 below 2^23 (K (2 * 8 * 2 +
    2 * 2) <= 36 * 2^17 for the longest row), which fp32 holds, so the result is the exact sum
    rounded once. With x everywhere, with x beside the ends of the warps' slices
    only, and with x in the last 32 columns only: a column lost, read twice or
    met with another group's scale shows."""
    gen = torch.Generator(device="cuda").manual_seed(K + N + M)
    r = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=gen, device="cuda")
    codes = r(-128, 127, N, K // 2).to(torch.int8)
    bias = r(-8, 8, N).to(dtype)
    for group, offset in ((32, True), (32, False), (64, False), (64, True), (128, True), (128, False)):
        if K % group:
            continue
        scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")[r(0, 2, N, K // group)].to(dtype)
        off = (r(-4, 4, N, K // group) * 0.5).to(dtype) if offset else None
        w = unpack(codes) * scale.double().repeat_interleave(group, 1)
        if offset:
            w += off.double().repeat_interleave(group, 1)
        for where in (range(K), slice_edges(K), range(K - 32, K)):
            x = torch.zeros(M, K, device="cuda", dtype=dtype)
            at = torch.tensor(list(where), device="cuda")
            x[:, at] = r(-2, 2, M, len(at)).to(dtype)
            y = w4.linear_w4a16(x, codes, scale, offset=off, bias=bias)
            want = x.double() @ w.t() + bias.double()
            assert torch.equal(y, want.to(dtype)), (group, offset, len(at))
    assert w4.last_device_error() == 0
