"""attention against its definition in float64.

Bound per element of `out`, with p_j the exact weights of the keys a query
sees, L their number, S = scale max_j sum_d |q_d k_jd|:
  * scores: D products summed in fp32 (a matrix unit may truncate where an
    adder rounds: 2^-23 a step), the scale and the shift by the maximum:
    off by at most ds = (D + 8) 2^-23 S + 2^-20, the last term the
    exponential's own error; weights are off by 2 ds relative (numerator and sum);
  * weights rounded to 16 bits before they meet v: eps/2 relative, and in fp16
    below 2^-14 half a subnormal step, 2^-25 (the sum they are divided by is at least 1);
  * sums of L terms in fp32: L 2^-23 relative to sum_j p_j |v_j|;
  * the output's own rounding: eps/2.
lse: ds + L 2^-23 + 2^-20 (1 + |lse|)."""

import math

import pytest
import torch

import w4a4_hadamard_rotated_b200 as w4

DTYPES = [torch.bfloat16, torch.float16]


def cu(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def make(Tq, Tk, Hq, Hk, D, dtype, seed=0, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=gen, device="cuda") * spread).to(dtype)
    return r(Tq, Hq, D), r(Tk, Hk, D), r(Tk, Hk, D)


def check(out, lse, q, k, v, qs, ks, causal, scale=None):
    """Every row of the packed result against float64 (on the GPU, one
    sequence and head group at a time)."""
    Hq, D = q.shape[1:]
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    eps = torch.finfo(q.dtype).eps
    q0 = k0 = 0
    for n, m in zip(qs, ks):
        for h in range(Hq):
            qq, kk, vv = q[q0:q0 + n, h].double(), k[k0:k0 + m, h // G].double(), v[k0:k0 + m, h // G].double()
            o, z = out[q0:q0 + n, h].double(), lse[q0:q0 + n, h].double()
            seen = torch.ones(n, m, dtype=torch.bool, device="cuda")
            if causal:
                seen = torch.arange(m, device="cuda") <= torch.arange(n, device="cuda")[:, None] + (m - n)
            s = (qq @ kk.t() * scale).masked_fill(~seen, -math.inf)
            top = s.amax(1, keepdim=True) if m else torch.full((n, 1), -math.inf, device="cuda", dtype=torch.float64)
            p = (s - torch.where(top == -math.inf, 0.0, top)).exp()
            total = p.sum(1, keepdim=True)
            rows = (total > 0)[:, 0]
            assert (o[~rows] == 0).all() and (z[~rows] == -math.inf).all()
            if not rows.any():
                continue
            p = (p / total.clamp(min=1e-300))[rows]
            ref, A = p @ vv, p @ vv.abs()
            L = seen[rows].sum(1, keepdim=True).double()
            S = ((qq.abs() @ kk.abs().t()) * scale * seen).amax(1, keepdim=True)[rows]
            ds = (D + 8) * 2.0 ** -23 * S + 2.0 ** -20
            tol = eps / 2 * ref.abs() + (eps / 2 + 2 * ds + L * 2.0 ** -23) * A * (1 + eps) + 2.0 ** -25
            if q.dtype == torch.float16:
                tol = tol + 2.0 ** -25 * (seen[rows].double() @ vv.abs())
            bad = ~((o[rows] - ref).abs() <= tol)
            assert not bad.any(), (f"sequence {n}x{m} head {h}: {int(bad.sum())} of {bad.numel()} off, first at "
                                   f"{bad.nonzero()[0].tolist()}, worst {((o[rows] - ref).abs() / tol).max():.3g} of the bound")
            want = (top + total.log())[rows]
            off = (z[rows][:, None] - want).abs()
            assert (off <= ds + L * 2.0 ** -23 + 2.0 ** -20 * (1 + want.abs())).all(), f"lse of {n}x{m} head {h}: {off.max():.3g}"
        q0, k0 = q0 + n, k0 + m


def go(qs, ks, Hq, Hk, D, dtype, causal, seed=0, spread=1.0, scale=None):
    q, k, v = make(sum(qs), sum(ks), Hq, Hk, D, dtype, seed, spread)
    out, lse = w4.attention(q, k, v, cu(qs), cu(ks), causal=causal, scale=scale, return_lse=True)
    assert out.shape == q.shape and out.dtype == dtype
    check(out, lse, q, k, v, qs, ks, causal, scale)
    assert w4.last_device_error() == 0
    return q, k, v, out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("n", [1, 2, 31, 64, 127, 128, 129, 200, 255, 256, 257, 385, 513, 1000])
def test_one_prompt(cuda_lib, dtype, D, causal, n):
    go([n], [n], 2, 1, D, dtype, causal, seed=n)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (6, 2), (5, 1), (8, 1), (16, 2), (12, 3), (32, 1), (7, 7)])
def test_packed_prompts_and_heads(cuda_lib, D, causal, Hq, Hk):
    n = [300, 1, 0, 77, 128, 257, 33]
    go(n, n, Hq, Hk, D, torch.bfloat16, causal, seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("qs,ks", [
    ([1], [5000]),                                  # one token over a cache
    ([1, 1, 1, 1], [4097, 1, 300, 129]),
    ([3, 1, 2], [2000, 64, 5]),                     # a few tokens
    ([17, 130], [1000, 131]),                       # the tail of a prompt
    ([5, 200, 1], [3, 150, 0]),                     # more queries than keys: causal rows that see nothing
    ([4, 0, 6], [0, 9, 0]),                         # no keys; no queries
    ([1], [1]),
    ([300], [40]),
])
def test_lengths_of_queries_and_keys_differ(cuda_lib, dtype, causal, qs, ks):
    go(qs, ks, 8, 2, 128, dtype, causal, seed=sum(ks))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,D", [(32, 8, 128), (5, 5, 64), (25, 5, 128), (64, 1, 64)])
def test_single_tokens_over_long_caches(cuda_lib, Hq, Hk, D):
    ks = [20000, 1, 129, 8192, 777]
    go([1] * 5, ks, Hq, Hk, D, torch.bfloat16, True, seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float16, 64)], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("qs,ks,Hq,Hk", [
    ([300], [6000], 1, 1),                             # several query tiles and many chunks
    ([700, 1, 260], [3000, 900, 2100], 6, 2),
    ([130, 0, 5], [40, 3000, 7000], 5, 1),             # rows that see nothing, a sequence without queries
    ([2500], [2500], 1, 1),
])
def test_few_tiles_over_many_keys(cuda_lib, dtype, D, causal, qs, ks, Hq, Hk):
    go(qs, ks, Hq, Hk, D, dtype, causal, seed=sum(ks))


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ks,Hq,Hk", [
    ([1] * 40, [20000] + [100 + 7 * i for i in range(39)], 16, 4),   # one cache far longer than the rest
    ([1] * 64, [2000] * 64, 8, 1),                                   # a block walks over several places
    ([1, 0, 4, 2, 1] * 40, [300, 70, 1500, 0, 2600] * 40, 8, 1),
    ([3] * 20, [4100] * 20, 24, 1),                                  # a head set of 24
])
def test_decoded_batches(cuda_lib, qs, ks, Hq, Hk):
    go(qs, ks, Hq, Hk, 64 if Hk == 4 else 128, torch.bfloat16, True, seed=len(qs))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.float16, 128)], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hk", [(3, 1), (7, 1), (22, 2), (13, 1), (16, 1), (31, 1), (32, 1), (33, 1), (64, 1), (10, 2)])
def test_decoded_head_groups(cuda_lib, dtype, D, Hq, Hk):
    """Groups that fill 32 rows, leave some empty or do not fit them."""
    go([1, 2, 0, 1, 3], [700, 2000, 5, 0, 129], Hq, Hk, D, dtype, True, seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 70, 900])
def test_cache_past_32_bit_offsets(cuda_lib, n):
    """The last sequence's keys lie behind 2^31 elements (4 GB) of k and v."""
    ks, Hk, D = [2 ** 31 // (8 * 128) + 1000, 777], 8, 128
    q = make(1 + n, 1, 16, 1, D, torch.bfloat16)[0]
    k = torch.empty(sum(ks), Hk, D, device="cuda", dtype=torch.bfloat16).normal_()
    v = torch.empty_like(k).normal_()
    out, lse = w4.attention(q, k, v, cu([1, n]), cu(ks), causal=True, return_lse=True)
    check(out[1:], lse[1:], q[1:], k[ks[0]:], v[ks[0]:], [n], [ks[1]], True)
    assert torch.isfinite(out).all() and w4.last_device_error() == 0


@pytest.mark.gpu
def test_expired_waits_of_a_decoded_batch(cuda_lib):
    q, k, v = make(64, 64 * 2000, 8, 1, 128, torch.bfloat16)
    cq, ck = cu([1] * 64), cu([2000] * 64)
    good = w4.attention(q, k, v, cq, ck, causal=True)
    w4.debug_set_wait_limit(5)
    try:
        w4.attention(q, k, v, cq, ck, causal=True)
        assert w4.last_device_error() == 8
    finally:
        w4.debug_set_wait_limit(0)
    assert torch.equal(w4.attention(q, k, v, cq, ck, causal=True), good)
    assert w4.last_device_error() == 0


@pytest.mark.gpu
def test_many_short_sequences(cuda_lib):
    gen = torch.Generator().manual_seed(1)
    n = torch.randint(0, 40, (300,), generator=gen).tolist()
    go(n, n, 2, 2, 64, torch.float16, True)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [127, 128, 129, 1000])
def test_many_decoded_sequences(cuda_lib, B):
    """More sequences than a warp walks at a time, some without queries or keys."""
    gen = torch.Generator().manual_seed(B)
    qs = torch.randint(0, 3, (B,), generator=gen).tolist()
    ks = torch.randint(0, 200, (B,), generator=gen).tolist()
    q, k, v = make(sum(qs), sum(ks), 4, 2, 64, torch.bfloat16)
    out, lse = w4.attention(q, k, v, cu(qs), cu(ks), causal=True, return_lse=True)
    pick = [i for i in range(B) if i % 37 in (0, 5, 36) or i > B - 4]
    at_q, at_k = [0] + torch.tensor(qs).cumsum(0).tolist(), [0] + torch.tensor(ks).cumsum(0).tolist()
    rows = torch.cat([torch.arange(at_q[i], at_q[i + 1]) for i in pick]).cuda()
    keys = torch.cat([torch.arange(at_k[i], at_k[i + 1]) for i in pick]).cuda()
    check(out[rows], lse[rows], q[rows], k[keys], v[keys], [qs[i] for i in pick], [ks[i] for i in pick], True)
    assert torch.isfinite(out).all() and w4.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_long_prompt(cuda_lib, causal):
    go([4500], [4500], 2, 2, 128, torch.bfloat16, causal)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq,Hk", [
    ([1100], 40, 40),                       # two query tiles per block: more blocks than the GPU has SMs
    ([1025, 130, 1, 257, 0, 700], 40, 8),   # groups of five: 125 rows of a tile
    ([900, 300, 515], 48, 6),
])
def test_more_blocks_than_sms(cuda_lib, dtype, causal, D, n, Hq, Hk):
    go(n, n, Hq, Hk, D, dtype, causal, seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_more_blocks_than_sms_edges(cuda_lib, D):
    """The same kernel with what its last tiles must not read (NaN behind every
    sequence), queries that see nothing, sharp scores and keys that fall and rise."""
    qs, ks, Hq, Hk = [700, 900, 520], [650, 1200, 0], 32, 8
    go(qs, ks, Hq, Hk, D, torch.bfloat16, True, spread=4.0)
    q, k, v = make(sum(qs), sum(ks), Hq, Hk, D, torch.bfloat16)
    k *= torch.linspace(-6.0, 6.0, sum(ks), device="cuda")[:, None, None].to(k.dtype)
    out, lse = w4.attention(q, k, v, cu(qs), cu(ks), causal=True, return_lse=True)
    check(out, lse, q, k, v, qs, ks, True)
    bad = lambda t: torch.cat((t, torch.full((200, *t.shape[1:]), math.nan, device="cuda", dtype=t.dtype)))
    again = w4.attention(bad(q), bad(k), bad(v), cu(qs), cu(ks), causal=True)
    assert torch.equal(again[:sum(qs)], out)
    k[:650], v[:650] = math.nan, math.nan
    again = w4.attention(q, k, v, cu(qs), cu(ks), causal=True)
    assert torch.equal(again[700:], out[700:]) and torch.isnan(again[100:700]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("spread,scale", [(8.0, None), (0.01, None), (1.0, 1.0), (1.0, 1e-6), (3.0, 0.5)])
def test_sharp_and_flat_softmax(cuda_lib, spread, scale):
    """Scores of hundreds, where the running maximum moves by much from tile to
    tile, and scores that are all alike."""
    go([300], [700], 2, 2, 128, torch.bfloat16, False, spread=spread, scale=scale)
    go([300], [700], 2, 2, 64, torch.float16, True, spread=spread, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_running_maximum_moves_every_tile(cuda_lib, order):
    """Keys whose score grows (or falls) steadily along the sequence."""
    q, k, v = make(200, 1500, 2, 2, 128, torch.bfloat16)
    ramp = torch.linspace(0.0, 8.0, 1500, device="cuda")
    ramp = ramp if order == "rising" else ramp.flip(0)
    q[:] = 1
    k[:] = ramp[:, None, None].to(k.dtype)
    out, lse = w4.attention(q, k, v, return_lse=True)
    check(out, lse, q, k, v, [200], [1500], False)


@pytest.mark.gpu
def test_without_lengths_is_one_sequence(cuda_lib):
    q, k, v = make(333, 444, 4, 2, 128, torch.bfloat16)
    a = w4.attention(q, k, v)
    b = w4.attention(q, k, v, cu([333]), cu([444]))
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("D", [64, 128])
def test_strides(cuda_lib, D, causal):
    """q, k and v out of one fused buffer, held head by head, and an output
    that is a slice of a wider one."""
    T, Hq, Hk = 190, 6, 2
    buf = torch.randn(T, (Hq + 2 * Hk) * D, device="cuda").to(torch.bfloat16)
    q, k, v = (t.view(T, -1, D) for t in buf.split([Hq * D, Hk * D, Hk * D], 1))
    want, lse = w4.attention(q.contiguous(), k.contiguous(), v.contiguous(), causal=causal, return_lse=True)
    check(want, lse, q, k, v, [T], [T], causal)
    wide = torch.full((T, Hq + 3, D + 8), 5.0, device="cuda", dtype=torch.bfloat16)
    got = w4.attention(q, k, v, causal=causal, out=wide[:, 1:1 + Hq, :D])
    assert torch.equal(got, want)
    assert (wide[:, 0] == 5).all() and (wide[:, 1 + Hq:] == 5).all() and (wide[:, :, D:] == 5).all()
    major = [t.permute(1, 0, 2).contiguous().permute(1, 0, 2) for t in (q, k, v)]
    assert torch.equal(w4.attention(*major, causal=causal), want)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("qs,ks", [([100, 60, 130], [100, 60, 130]), ([1, 1, 1], [700, 130, 2000])])
def test_rows_outside_the_sequences(cuda_lib, causal, qs, ks):
    """Rows behind the last sequence keep what they hold, and what is there in
    q, k and v reaches nothing, NaN and infinities included; nor does one
    sequence reach another."""
    Hq, Hk, D = 4, 2, 128
    q, k, v = make(sum(qs), sum(ks), Hq, Hk, D, torch.bfloat16)
    want, wl = w4.attention(q, k, v, cu(qs), cu(ks), causal=causal, return_lse=True)
    pad = lambda t, fill: torch.cat((t, torch.full((37, *t.shape[1:]), fill, device="cuda", dtype=t.dtype)))
    q2, k2, v2 = pad(q, math.nan), pad(k, math.inf), pad(v, math.nan)
    out = torch.full_like(q2, 3.0)
    got, gl = w4.attention(q2, k2, v2, cu(qs), cu(ks), causal=causal, out=out, return_lse=True)
    assert torch.equal(got[:sum(qs)], want) and torch.equal(gl[:sum(qs)], wl)
    assert (got[sum(qs):] == 3).all()
    # the middle sequence all NaN: the others are as they were
    a, b = ks[0], ks[0] + ks[1]
    k3, v3 = k.clone(), v.clone()
    k3[a:b], v3[a:b] = math.nan, math.nan
    got = w4.attention(q, k3, v3, cu(qs), cu(ks), causal=causal)
    a, b = qs[0], qs[0] + qs[1]
    assert torch.equal(got[:a], want[:a]) and torch.equal(got[b:], want[b:])
    assert torch.isnan(got[a:b]).all()


@pytest.mark.gpu
def test_masked_keys_inside_a_sequence(cuda_lib):
    """Keys that the causal rule hides may be NaN or infinite."""
    q, k, v = make(300, 300, 2, 2, 128, torch.bfloat16)
    want = w4.attention(q, k, v, causal=True)
    k2 = k.clone()
    k2[150:] = math.nan
    got = w4.attention(q, k2, v, causal=True)
    assert torch.equal(got[:150], want[:150]) and torch.isnan(got[150:]).all()
    k2[150:] = math.inf
    got = w4.attention(q, k2, v, causal=True)
    assert torch.equal(got[:150], want[:150])


@pytest.mark.gpu
def test_nan_queries_stay_in_their_rows(cuda_lib):
    q, k, v = make(130, 300, 4, 2, 64, torch.float16)
    want = w4.attention(q, k, v)
    q2 = q.clone()
    q2[7, 1] = math.nan
    got = w4.attention(q2, k, v)
    keep = torch.ones(130, 4, dtype=torch.bool, device="cuda")
    keep[7, 1] = False
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[7, 1]).all()


@pytest.mark.gpu
def test_lengths_that_do_not_fit_stay_in_range(cuda_lib):
    """Lengths past the rows, falling ones and negative ones are clamped: rows
    that no sequence covers keep what they hold."""
    q, k, v = make(100, 100, 2, 2, 64, torch.bfloat16)
    bad = torch.tensor([0, 60, 40, 1000], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 2.0)
    w4.attention(q, k, v, bad, bad, out=out)
    first = w4.attention(q[:40], k[:60], v[:60])
    assert torch.isfinite(out).all() and torch.equal(out[:40], first)
    neg = torch.tensor([-5, 30, 30, -7], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 2.0)
    w4.attention(q, k, v, neg, neg, out=out)
    assert torch.equal(out[:30], w4.attention(q[:30], k[:30], v[:30])) and (out[30:] == 2).all()
    assert w4.last_device_error() == 0


@pytest.mark.gpu
def test_empty_calls(cuda_lib):
    q, k, v = make(5, 0, 2, 2, 64, torch.bfloat16)
    out, lse = w4.attention(q, k, v, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    q, k, v = make(0, 5, 2, 2, 64, torch.bfloat16)
    assert w4.attention(q, k, v).shape == (0, 2, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ks", [([1, 1], [3000, 500]), ([300, 40], [300, 40])])
def test_graphs_streams_and_repeats(cuda_lib, qs, ks):
    """Deterministic; on a side stream; two captured graphs replayed at once on
    their own streams with eager calls between; lengths that change on the
    device between replays."""
    q, k, v = make(sum(qs), sum(ks), 8, 2, 128, torch.bfloat16)
    q2 = make(sum(qs), 1, 8, 1, 128, torch.bfloat16, seed=9)[0]
    cq, ck = cu(qs), cu(ks)
    want, want2 = (w4.attention(t, k, v, cq, ck, causal=True) for t in (q, q2))
    assert torch.equal(want, w4.attention(q, k, v, cq, ck, causal=True))
    bufs = [q.clone(), q2.clone()]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w4.attention(b, k, v, cq, ck, causal=True))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = w4.attention(q, k, v, cq, ck, causal=True)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want2) and torch.equal(eager, want)
    # the same graph after the sequences' lengths changed in place
    shorter = cu([ks[0] - 100, ks[1]])
    ck.copy_(shorter)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], w4.attention(q, k, v, cq, shorter, causal=True))


@pytest.mark.gpu
def test_binding_refusals(cuda_lib):
    q, k, v = make(4, 6, 4, 2, 64, torch.bfloat16)
    c = cu([4])
    bad = [
        (TypeError, lambda: w4.attention(q.float(), k, v)),
        (TypeError, lambda: w4.attention(q, k.half(), v)),
        (TypeError, lambda: w4.attention(q, k, v, c.long(), c.long())),
        (ValueError, lambda: w4.attention(q, k, v[:5])),
        (ValueError, lambda: w4.attention(q, k, v, c)),
        (ValueError, lambda: w4.attention(q, k, v, c, torch.cat((c, c)))),
        (ValueError, lambda: w4.attention(q, k, v, c[:1], c[:1])),
        (ValueError, lambda: w4.attention(q[0], k, v)),
        (ValueError, lambda: w4.attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)),
        (ValueError, lambda: w4.attention(q, k, v, out=torch.empty(4, 4, 32, device="cuda", dtype=q.dtype))),
        (w4.W4A4Error, lambda: w4.attention(q[:, :3], k, v)),
        (w4.W4A4Error, lambda: w4.attention(q[..., :32], k[..., :32], v[..., :32])),
        (w4.W4A4Error, lambda: w4.attention(q, k, v, scale=0.0)),
        (w4.W4A4Error, lambda: w4.attention(q, k[:, :1].expand(6, 2, 64), v)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


@pytest.mark.gpu
def test_expired_waits_end_the_call(cuda_lib):
    """With a wait limit of a few nanoseconds the kernels give up, report it and
    leave the context as it was; the next call is right."""
    cases = [make(1100, 1100, 40, 40, 128, torch.bfloat16), make(300, 300, 4, 4, 64, torch.float16),
             make(1, 9000, 8, 2, 128, torch.bfloat16)]
    good = [w4.attention(*c, causal=True) for c in cases]
    w4.debug_set_wait_limit(5)
    try:
        for c in cases:
            w4.attention(*c, causal=True)
            assert w4.last_device_error() == 8
    finally:
        w4.debug_set_wait_limit(0)
    for c, g in zip(cases, good):
        assert torch.equal(w4.attention(*c, causal=True), g)
    assert w4.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float16, 64)], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("qs,ks,H", [
    ([590, 4, 3, 3], [8150, 20, 10, 12], 8),                                # one that has nearly all
    ([3, 3, 4, 590], [12, 10, 20, 8150], 8),
    ([1, 493, 0, 2, 1, 1, 1, 1], [5, 19950, 3, 0, 9, 11, 17, 5], 4),
    ([150, 150, 150, 150], [2048, 2048, 2048, 2048], 8),                    # alike: most blocks have no place
])
def test_split_batches(cuda_lib, dtype, D, causal, qs, ks, H):
    """Tiles of 128 rows whose keys are split, a block for every place there can be."""
    go(qs, ks, H, H, D, dtype, causal, seed=qs[0])
    assert sum(qs) > 32 * len(qs)


@pytest.mark.gpu
def test_batches_over_long_caches_take_little_memory(cuda_lib):
    """More queries a sequence than a tile of few holds, over long caches: beside
    the result the call takes 128 MB and a little."""
    q, k, v = make(64 * 39, 64 * 8192, 8, 1, 128, torch.bfloat16)
    c = [39] * 64, [8192] * 64
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out, lse = w4.attention(q, k, v, cu(c[0]), cu(c[1]), causal=True, return_lse=True)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= 140 * 2 ** 20
    check(out[-39:], lse[-39:], q[-39:], k[-8192:], v[-8192:], [39], [8192], True)
    assert w4.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("rows,keys,H", [(300, 4096, 2), (1, 4096, 2), (2600, 4096, 40), (200, 2 ** 17, 1), (40, 500, 3)])
@pytest.mark.parametrize("at", [0, 77, 130, -1])
def test_many_small_weights_beside_one_large(cuda_lib, dtype, rows, keys, H, at):
    """One key that takes nearly all of the softmax and has value 0, and keys
    17.6875 below it (2^-25.5 of its weight) with value 1: the result is their
    whole share.  Scores are one product and exact, as are the scale of 1 and
    18 ln 2's place in fp32 to 2^-24 relative: weights off by 2^-18 with the
    exponential's 2^-22; sums of L terms L 2^-23; weights rounded to 16 bits by
    half a step, eps/2, and in fp16 (which holds them times 2^11 or more) by at
    most 2^-36 of the largest each; the output by half a step, in fp16 2^-25 at least."""
    D = 64
    q = torch.zeros(rows, H, D, device="cuda", dtype=dtype)
    k = torch.zeros(keys, H, D, device="cuda", dtype=dtype)
    v = torch.ones(keys, H, D, device="cuda", dtype=dtype)
    q[..., 3] = 1
    k[..., 3] = 0.3125
    k[at, :, 3], v[at] = 18, 0
    out, lse = w4.attention(q, k, v, scale=1.0, return_lse=True)
    small = (keys - 1) * math.exp(-17.6875)
    want, eps = small / (1 + small), torch.finfo(dtype).eps
    tol = want * (eps + 2.0 ** -18 + keys * 2.0 ** -23) + 2.0 ** -25
    if dtype == torch.float16:
        tol += keys * 2.0 ** -36
    assert (out.double() - want).abs().max() <= tol
    assert (lse.double() - 18 - math.log1p(small)).abs().max() <= 19 * 2.0 ** -20 + keys * 2.0 ** -23


SENSITIVE = [
    ([700, 1, 260], [3000, 900, 2100], 6, 2),
    ([1] * 5, [20000, 1, 129, 8192, 777], 32, 8),
    ([1100], [1100], 40, 40),
    ([300], [6000], 1, 1),
    ([1, 0, 4, 2, 1] * 8, [300, 70, 1500, 0, 2600] * 8, 8, 1),
    ([1025, 130, 1, 257, 0, 700], [1025, 130, 1, 257, 0, 700], 40, 8),
    ([40, 33], [20000, 300], 8, 1),
    ([590, 4, 3, 3], [8150, 20, 10, 12], 8, 8),
    ([2, 300, 5], [127, 40, 256], 4, 2),
]


def seen_by(n, m, causal):
    """[n, m]: whether query i sees key j."""
    i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")
    return j <= i + (m - n) if causal else torch.ones(n, m, dtype=torch.bool, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("qs,ks,Hq,Hk", SENSITIVE)
def test_every_key_counts_once(cuda_lib, dtype, D, causal, qs, ks, Hq, Hk):
    """Queries of zeros: all weights are alike and exact, and so are their sums.
    The keys at the ends of tiles and sequences have value 1 in a column of their
    own or one that they share with a few, so the result is a small count over
    the number of keys seen: one lost or counted twice moves it by several
    percent, a bad bound of the keys moves lse.
    Bounds: the output's rounding, eps/2 (in fp16 2^-25 at least); the quotient
    and the join of chunks: some roundings, exponentials and logarithms of 2^-22
    to 2^-21 absolute, 2^-18 together, and 2^-19 (1 + |lse|) for lse."""
    rows = 30                                                    # behind the last sequence
    q = torch.zeros(sum(qs), Hq, D, device="cuda", dtype=dtype)
    k = make(1, sum(ks) + rows, 1, Hk, D, dtype)[1]
    v = torch.zeros(sum(ks) + rows, Hk, D, device="cuda", dtype=dtype)
    v[sum(ks):] = 1
    at = 0
    for m in ks:
        edge = [j for j in range(m) if j % 128 in (0, 1, 126, 127) or j >= m - 3]
        v[at + torch.tensor(edge, dtype=torch.long), :, torch.arange(len(edge)) % D] = 1
        at += m
    out, lse = w4.attention(q, k, v, cu(qs), cu(ks), causal=causal, return_lse=True)
    q0 = k0 = 0
    for n, m in zip(qs, ks):
        seen = seen_by(n, m, causal).double()
        total = seen.sum(1)
        want = (seen @ v[k0:k0 + m].double().flatten(1)).view(n, Hk, D) / total.clamp(min=1)[:, None, None]
        want = want.repeat_interleave(Hq // Hk, 1)
        tol = want * (torch.finfo(dtype).eps / 2 + 2.0 ** -18) + (2.0 ** -25 if dtype == torch.float16 else 0)
        assert ((out[q0:q0 + n].double() - want).abs() <= tol).all()
        z, off = total.log()[:, None], lse[q0:q0 + n].double()
        assert torch.where(z == -math.inf, off == z, (off - z).abs() <= 2.0 ** -19 * (1 + z.abs())).all()
        q0, k0 = q0 + n, k0 + m
    assert w4.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("qs,ks,Hq,Hk", SENSITIVE)
def test_one_key_takes_all(cuda_lib, dtype, D, causal, qs, ks, Hq, Hk):
    """Each key head of a sequence has one key whose score lies 100 or more above
    the others', at the edges of tiles, chunks and the sequence in turn: the
    result is its value, bit for bit (all other weights are nothing). Keys of the
    next sequence and those behind the last score higher still, so that one
    reached by mistake would take all."""
    rows, ends = 30, [0]
    for m in ks:
        ends.append(ends[-1] + m)
    gen = torch.Generator().manual_seed(sum(ks) + D)
    q = make(sum(qs), 1, Hq, 1, D, dtype)[0] * 0
    q[..., 5] = 1
    _, k, v = make(1, ends[-1] + rows, 1, Hk, D, dtype, seed=3)
    for turn in range(4):
        k[..., 5] = k[..., 5].clamp(-4, 4)
        k[ends[-1]:, :, 5] = 960
        where, score = {}, {}
        for b, m in enumerate(ks):
            edge = sorted({j for j in (0, 1, 127, 128, 129, 255, 256, m // 2, m - 129, m - 128, m - 127, m - 2, m - 1)
                           if 0 <= j < m})
            edge += [j for j in torch.randint(0, max(m // 128, 1), (4,), generator=gen).mul(128).tolist() if j < m]
            for h in range(Hk):
                if edge:
                    where[b, h] = edge[(h + 5 * b + turn * (Hk + 1)) % len(edge)]
                    score[b] = 128 + 16 * b
                    k[ends[b] + where[b, h], h, 5] = score[b]
        out, lse = w4.attention(q, k, v, cu(qs), cu(ks), causal=causal, scale=1.0, return_lse=True)
        q0 = 0
        for b, (n, m) in enumerate(zip(qs, ks)):
            for h in range(Hk):
                if (b, h) not in where or n == 0:
                    continue
                j, G = where[b, h], Hq // Hk
                rows_seeing = seen_by(n, m, causal)[:, j]
                got = out[q0:q0 + n, h * G:(h + 1) * G][rows_seeing]
                assert torch.equal(got, v[ends[b] + j, h].expand_as(got)), (turn, b, h, j)
                z = lse[q0:q0 + n, h * G:(h + 1) * G][rows_seeing].double()
                assert ((z - score[b]).abs() <= 2.0 ** -19 * (1 + score[b])).all()
            q0 += n
    assert w4.last_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,Hq,Hk", [(torch.bfloat16, 128, 32, 8), (torch.float16, 64, 8, 1)], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 7])
def test_caches_with_room_to_grow(cuda_lib, dtype, D, Hq, Hk, n):
    """One buffer of 5 caches of 3000 rows, of which some are filled: sequences
    without queries stand for the rest of each, whatever it holds. The same
    buffer and lengths that grow on the device, replayed from a graph."""
    B, room = 5, 3000
    used = [2999, 130, n, 3000, 1024]
    q, k, v = make(B * n, B * room, Hq, Hk, D, dtype)
    filled = torch.zeros(B, room, dtype=torch.bool, device="cuda")

    def lengths():
        at = [(room * b, room * b + m) for b, m in enumerate(used)]
        return torch.tensor([x for pair in at for x in pair] + [B * room], dtype=torch.int32, device="cuda")

    cq = torch.tensor([n * ((i + 1) // 2) for i in range(2 * B + 1)], dtype=torch.int32, device="cuda")
    ck = lengths()
    g = torch.cuda.CUDAGraph()
    w4.attention(q, k, v, cq, ck, causal=True)
    with torch.cuda.graph(g):
        out, lse = w4.attention(q, k, v, cq, ck, causal=True, return_lse=True)
    for _ in range(3):
        filled[:] = False
        for b, m in enumerate(used):
            filled[b, :m] = True
        rest = ~filled.view(-1)
        ck.copy_(lengths())
        k[rest], v[rest] = math.nan, math.inf
        g.replay()
        check(out, lse, q, k[~rest], v[~rest], [n] * B, used, True)
        assert torch.isfinite(out).all() and w4.last_device_error() == 0
        # each cache takes a token more, where it has room
        for b in range(B):
            if used[b] < room:
                k[room * b + used[b]], v[room * b + used[b]] = q[b, :Hk], 1
                used[b] += 1
