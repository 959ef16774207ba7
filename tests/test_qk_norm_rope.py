"""qk_norm_rope against its definition in float64.

Bound per element: the one rounding to 16 bits (half a step), plus the fp32
steps.  With (a, b) the normed pair, the norm's sum of D <= 256 squares (a
tree of at most 16 roundings in any order here), its reciprocal root and two
products move a and b by at most 16 u each (u = 2^-24, halved by the root),
the angle's fraction of a turn rounded to fp32 moves cos and sin by at most
2 pi 2^-25 < 2^-22, sincospi by a few u more, the rotation's products and sum by 2 u:
together below 2^-20 (|a| + |b|)."""

import math

import pytest
import torch

import w4a4_hadamard_rotated_b200 as w4

DTYPES = [torch.bfloat16, torch.float16]


def reference(h, weight, eps, positions, freq, axis, interleaved):
    """(value, magnitude the bound is relative to), float64 on the CPU."""
    u = h.double().cpu()
    D = u.shape[2]
    if weight is not None:
        u = u / (u.square().mean(2, keepdim=True) + eps).sqrt() * weight.double().cpu()
    out, mag = u.clone(), u.abs()
    if positions is not None:
        p = positions.cpu().view(u.shape[0], -1).double()
        angle = p[:, axis.cpu().long()] * freq.cpu()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        half = freq.numel()
        first = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
        second = first + (1 if interleaved else half)
        a, b = u[..., first], u[..., second]
        out[..., first], out[..., second] = a * c - b * s, a * s + b * c
        mag[..., first] = mag[..., second] = a.abs() + b.abs()
    return out, mag


def check(got, ref):
    value, mag = ref
    eps = torch.finfo(got.dtype).eps
    tol = eps / 2 * value.abs() + 2.0 ** -20 * mag * (1 + eps) + 2.0 ** -25
    bad = (got.double().cpu() - value).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def make(T, Hq, Hk, D, dtype, seed=0, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    q, k = (r(T, Hq, D) * spread).to(dtype), (r(T, Hk, D) * spread).to(dtype)
    return q, k, (1 + 0.2 * r(D)).to(dtype), (1 + 0.2 * r(D)).to(dtype)


def places(T, axes, far, dtype=torch.int32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-far, far + 1, (T, axes), generator=gen, device="cuda", dtype=dtype)


CASES = [
    # T, Hq, Hk, D, axis dims, interleaved, farthest position
    (1, 1, 1, 8, (8,), True, 10),
    (1, 32, 8, 128, (128,), False, 200000),
    (2, 3, 1, 64, (24, 20, 20), True, 60),
    (3, 5, 5, 96, (48,), False, 5000),            # part of the head turns
    (5, 24, 24, 128, (16, 56, 56), True, 128),
    (7, 40, 40, 128, (44, 42, 42), True, 52),
    (9, 7, 7, 128, (44, 42, 42), False, 52),      # sections of axes on halves
    (33, 2, 1, 256, (256,), False, 1 << 20),
    (17, 1, 0, 16, (16,), False, 99),             # queries only
    (64, 9, 3, 40, (10, 30), True, 300),          # heads that fill no power of two
    (65, 6, 2, 200, (32, 32), False, 300),
    (129, 16, 2, 72, (6,), True, 1 << 24),        # far positions
    (301, 33, 11, 64, (32, 32), True, 180),
    (1000, 80, 10, 128, (64, 64), True, 180),
    (257, 100, 100, 64, (64,), False, 40000),
    (3, 700, 300, 64, (64,), True, 40000),        # many heads
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:4])))
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
def test_matches_definition(cuda_lib, dtype, case, norm):
    T, Hq, Hk, D, dims, inter, far = case
    q, k, qw, kw = make(T, Hq, Hk, D, dtype, seed=T + D)
    if not norm or Hk == 0:
        kw = None
    qw = qw if norm else None
    pos = places(T, len(dims), far)
    freq, axis = w4.rotary_frequencies(dims, theta=10000.0)
    qo, ko = w4.qk_norm_rope(q, k if Hk else None, qw, kw, pos, freq, axis, interleaved=inter)
    check(qo, reference(q, qw, 1e-6, pos, freq, axis, inter))
    if Hk:
        check(ko, reference(k, kw, 1e-6, pos, freq, axis, inter))
    else:
        assert ko is None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
def test_norm_alone_and_one_norm_only(cuda_lib, dtype):
    q, k, qw, kw = make(11, 6, 2, 128, dtype)
    qo, ko = w4.qk_norm_rope(q, k, qw, kw, eps=1e-5)
    check(qo, reference(q, qw, 1e-5, None, None, None, True))
    check(ko, reference(k, kw, 1e-5, None, None, None, True))
    qo, ko = w4.qk_norm_rope(q, k, q_weight=qw)
    check(qo, reference(q, qw, 1e-6, None, None, None, True))
    assert torch.equal(ko, k)                                # nothing to do: the same bits


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [True, False])
def test_strided_fused_buffer_and_in_place(cuda_lib, inter):
    """q and k out of one fused buffer and a head-major one; written in place;
    nothing else of the buffer changes."""
    T, Hq, Hk, D = 37, 6, 2, 128
    freq, axis = w4.rotary_frequencies((16, 56, 56))
    pos = places(T, 3, 90, dtype=torch.int64)
    _, _, qw, kw = make(1, 1, 1, D, torch.bfloat16)
    buf = torch.randn(T, (Hq + 2 * Hk) * D, device="cuda").to(torch.bfloat16)
    q, k = buf[:, :Hq * D].view(T, Hq, D), buf[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    want = w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis, interleaved=inter)
    check(want[0], reference(q, qw, 1e-6, pos, freq, axis, inter))
    major = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)          # [T, Hq, D] held head by head
    out = torch.empty_like(major)
    assert out.stride() == major.stride()
    got = w4.qk_norm_rope(major, k, qw, kw, pos, freq, axis, interleaved=inter, q_out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = buf[:, (Hq + Hk) * D:].clone()
    w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, (Hq + Hk) * D:], v)


@pytest.mark.gpu
def test_positions_of_every_kind(cuda_lib):
    """int32 and int64, one axis as [T], a strided [T, axes]; a far position in
    float64 turns; an axis number out of range is taken as the nearest axis."""
    T, D = 21, 64
    q, k, qw, kw = make(T, 2, 2, D, torch.float16)
    freq, axis = w4.rotary_frequencies((D,), theta=1e6)
    pos = places(T, 1, (1 << 31) - 1, dtype=torch.int64)
    a = w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis)
    check(a[0], reference(q, qw, 1e-6, pos, freq, axis, True))
    b = w4.qk_norm_rope(q, k, qw, kw, pos[:, 0].to(torch.int32), freq, axis)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = torch.zeros(T, 5, device="cuda", dtype=torch.int64)
    wide[:, 2:3] = pos
    c = w4.qk_norm_rope(q, k, qw, kw, wide[:, 2:3], freq, axis)
    assert torch.equal(a[0], c[0])
    d = w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis + 7)
    e = w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis - 3)
    assert torch.equal(a[0], d[0]) and torch.equal(a[0], e[0])


@pytest.mark.gpu
def test_values_at_the_edges(cuda_lib):
    """Zero heads stay zero; a NaN or infinite head reaches no other head;
    large fp16 heads do not overflow in the sum of squares."""
    q, k, qw, kw = make(3, 4, 4, 128, torch.float16)
    q[0, 0] = 0
    q[1, 1, 5] = float("nan")
    q[2, 2, 7] = float("inf")
    k[:] = 60000.0
    freq, axis = w4.rotary_frequencies((128,))
    pos = places(3, 1, 50)
    clean = q.clone()
    clean[1, 1], clean[2, 2] = 1, 1
    qo, ko = w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis)
    good, _ = w4.qk_norm_rope(clean, k, qw, kw, pos, freq, axis)
    assert (qo[0, 0] == 0).all() and torch.isnan(qo[1, 1]).all()
    same = torch.ones(3, 4, dtype=torch.bool)
    same[1, 1] = same[2, 2] = False
    assert torch.equal(qo[same.cuda()], good[same.cuda()])
    check(ko, reference(k, kw, 1e-6, pos, freq, axis, True))


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [True, False])
def test_what_does_not_turn_keeps_its_bits(cuda_lib, inter):
    """Without norms, elements past R are copied: negative zeros, NaN and
    infinities next to them included."""
    q, _, _, _ = make(4, 3, 1, 64, torch.bfloat16)
    q[:, :, 40], q[:, :, 43], q[:, :, 63] = -0.0, float("nan"), float("inf")
    freq, axis = w4.rotary_frequencies((32,))
    out, _ = w4.qk_norm_rope(q, None, None, None, places(4, 1, 9), freq, axis, interleaved=inter)
    assert torch.equal(out[:, :, 32:].contiguous().view(torch.int16), q[:, :, 32:].contiguous().view(torch.int16))
    check(out[:, :, :32], reference(q[:, :, :32], None, 0, places(4, 1, 9), freq, axis, inter))


@pytest.mark.gpu
def test_empty_graph_and_stream(cuda_lib):
    q, k, qw, kw = make(19, 8, 4, 128, torch.bfloat16)
    freq, axis = w4.rotary_frequencies((64, 64))
    pos = places(19, 2, 70)
    qo, ko = w4.qk_norm_rope(q[:0], k[:0], qw, kw, pos[:0], freq, axis)
    assert qo.shape == (0, 8, 128) and ko.shape == (0, 4, 128)
    want = w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0])
    buf = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go = w4.qk_norm_rope(buf, k, qw, kw, pos, freq, axis)
    buf.copy_(q)
    g.replay()
    assert torch.equal(go[0], want[0]) and torch.equal(go[1], want[1])


@pytest.mark.gpu
def test_binding_refusals(cuda_lib):
    q, k, qw, kw = make(4, 2, 2, 64, torch.bfloat16)
    freq, axis = w4.rotary_frequencies((64,))
    pos = places(4, 1, 5)
    bad = [
        (TypeError, lambda: w4.qk_norm_rope(q.float(), k)),
        (TypeError, lambda: w4.qk_norm_rope(q, k.half())),
        (TypeError, lambda: w4.qk_norm_rope(q, k, qw.half(), kw)),
        (TypeError, lambda: w4.qk_norm_rope(q, k, qw, kw, pos.float(), freq, axis)),
        (TypeError, lambda: w4.qk_norm_rope(q, k, qw, kw, pos, freq.float(), axis)),
        (TypeError, lambda: w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis.long())),
        (ValueError, lambda: w4.qk_norm_rope(q, k, qw, kw, pos)),
        (ValueError, lambda: w4.qk_norm_rope(q, k, qw, kw, pos[:3], freq, axis)),
        (ValueError, lambda: w4.qk_norm_rope(q, k[:3], qw, kw)),
        (ValueError, lambda: w4.qk_norm_rope(q, k, qw[:32], kw)),
        (ValueError, lambda: w4.qk_norm_rope(q[:, :, ::2], k)),
        (ValueError, lambda: w4.qk_norm_rope(q, None, qw, kw)),
        (ValueError, lambda: w4.qk_norm_rope(q, k, qw, kw, pos, freq, axis[:8])),
        (w4.W4A4Error, lambda: w4.qk_norm_rope(q[:, :, :20], k[:, :, :20])),
        (w4.W4A4Error, lambda: w4.qk_norm_rope(q, k, qw, kw, pos, freq[:12].clone(), axis[:12].clone(), interleaved=False)),
        (w4.W4A4Error, lambda: w4.qk_norm_rope(q, k, qw, kw, eps=math.nan)),
        (w4.W4A4Error, lambda: w4.qk_norm_rope(q[:1].expand(4, 2, 64), k)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [True, False])
def test_tokens_past_32_bit_offsets(cuda_lib, interleaved):
    """More than 2^31 elements of q, whose last tokens come out as in a small call."""
    T, H, D = 2 ** 31 // (8 * 64) + 77, 8, 64
    q = torch.empty(T, H, D, device="cuda", dtype=torch.bfloat16).normal_()
    _, _, w, _ = make(1, H, H, D, torch.bfloat16)
    freq, axis = w4.rotary_frequencies((D,))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    out, _ = w4.qk_norm_rope(q, None, w, None, pos, freq, axis, interleaved=interleaved)
    last = slice(T - 100, T)
    want, _ = w4.qk_norm_rope(q[last].clone(), None, w, None, pos[last].clone(), freq, axis, interleaved=interleaved)
    check(want, reference(q[last], w, 1e-6, pos[last], freq, axis, interleaved))
    assert torch.equal(out[last], want)
