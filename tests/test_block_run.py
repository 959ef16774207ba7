"""The operators between a block's linears run as a block uses them: modulation
vectors from linear_w4a16, queries, keys and values from one shared W4A4
activation, qk_norm_rope, attention over packed sequences, the W4A4 output
linear.  Every stage is checked against its definition on the tensors that the
run itself hands to it, and the whole is replayed from a graph."""

import os
import subprocess
import sys

import pytest
import torch

import test_attention as ta
import test_linear_w4a16 as tl
import test_qk_norm_rope as tr
import w4a4_hadamard_rotated_b200 as w4

pytestmark = pytest.mark.gpu

D = 128


class Block:
    """Weights of a small block of `Hq` query and `Hk` key heads."""

    def __init__(self, Hq, Hk, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.Hq, self.Hk, self.width = Hq, Hk, Hq * D
        self.mod = w4.quantize_weight_w4a16(r(3 * self.width, self.width) * 0.02, 64, torch.bfloat16, asymmetric=True)
        self.mod_bias = (r(3 * self.width) * 0.1).to(torch.bfloat16)
        self.linears = {n: w4.quantize_weight(r(rows * D, self.width) * 0.02, 128)
                        for n, rows in (("q", Hq), ("k", Hk), ("v", Hk), ("out", Hq))}
        self.q_weight, self.k_weight = ((1 + 0.1 * r(D)).to(torch.bfloat16) for _ in range(2))
        self.freq, self.axis = w4.rotary_frequencies((16, 56, 56))

    def run(self, x, cond, positions, cu, causal=False):
        """(output, everything in between)"""
        shift, scale, gate = w4.linear_w4a16(cond, self.mod[0], self.mod[1], self.mod[2], self.mod_bias)[0].split(self.width)
        h = x * (1 + scale) + shift
        codes, s = w4.quantize_activation(h, 128)
        q, k, v = (w4.linear(codes, s, *self.linears[n]).view(x.shape[0], -1, D) for n in "qkv")
        qr, kr = w4.qk_norm_rope(q, k, self.q_weight, self.k_weight, positions, self.freq, self.axis)
        o, lse = w4.attention(qr, kr, v, cu, cu, causal=causal, return_lse=True)
        y = x + gate * w4.linear_fused(o.view(x.shape[0], self.width), *self.linears["out"])
        return y, (q, k, v, qr, kr, o, lse, torch.cat((shift, scale, gate))[None])


def make(block, grids, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lengths = [t * h * w for t, h, w in grids]
    x = torch.randn(sum(lengths), block.width, generator=gen, device="cuda").to(torch.bfloat16)
    cond = torch.randn(1, block.width, generator=gen, device="cuda").to(torch.bfloat16)
    positions = torch.cat([torch.cartesian_prod(*(torch.arange(n, device="cuda", dtype=torch.int32) for n in g))
                           for g in grids])
    return x, cond, positions, lengths


@pytest.mark.parametrize("Hq,Hk,causal", [(4, 4, False), (8, 2, True)])
def test_every_stage_of_a_block(cuda_lib, Hq, Hk, causal):
    block = Block(Hq, Hk)
    x, cond, positions, lengths = make(block, [(1, 16, 20), (3, 5, 7), (1, 1, 1), (2, 9, 11)])
    y, (q, k, v, qr, kr, o, lse, mod) = block.run(x, cond, positions, ta.cu(lengths), causal)
    cpu = [t.cpu() for t in (cond, *block.mod, block.mod_bias)]
    tl.check(mod, *tl.reference(*cpu), block.width)
    tr.check(qr, tr.reference(q, block.q_weight, 1e-6, positions, block.freq, block.axis, True))
    tr.check(kr, tr.reference(k, block.k_weight, 1e-6, positions, block.freq, block.axis, True))
    ta.check(o, lse, qr, kr, v, lengths, lengths, causal)
    assert torch.isfinite(y).all() and w4.last_device_error() == 0


def test_packed_images_equal_images_alone(cuda_lib):
    """Three images of different sizes in one call, and each by itself: the same bits."""
    block = Block(6, 6)
    grids = [(1, 24, 18), (1, 9, 31), (2, 12, 8)]
    x, cond, positions, lengths = make(block, grids)
    y, _ = block.run(x, cond, positions, ta.cu(lengths))
    at = 0
    for n in lengths:
        alone, _ = block.run(x[at:at + n], cond, positions[at:at + n], ta.cu([n]))
        assert torch.equal(y[at:at + n], alone)
        at += n


def test_block_replayed_from_graphs(cuda_lib):
    """Two blocks captured as graphs of their own, replayed on two streams at
    once with new inputs, against eager runs."""
    blocks = [Block(4, 4, seed=3), Block(8, 2, seed=4)]
    data = [make(b, [(1, 10, 15), (1, 7, 9)], seed=5) for b in blocks]
    cus = [ta.cu(d[3]) for d in data]
    fresh = [make(b, [(1, 10, 15), (1, 7, 9)], seed=6) for b in blocks]
    want = [b.run(f[0], f[1], d[2], c)[0] for b, f, d, c in zip(blocks, fresh, data, cus)]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for b, d, c, s in zip(blocks, data, cus, streams):
        # warm up on the stream it is captured on (the W4A4 linears keep a workspace for each)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            b.run(d[0], d[1], d[2], c)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(b.run(d[0], d[1], d[2], c)[0])
        graphs.append(g)
    for d, f in zip(data, fresh):
        d[0].copy_(f[0])
        d[1].copy_(f[1])
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert w4.last_device_error() == 0


def test_decoded_tokens_equal_the_prompt(cuda_lib):
    """A prompt at once, and its last tokens one by one over the cache of those
    before: the same attention to the kernels' bounds."""
    Hq, Hk, n = 8, 2, 700
    gen = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = r(n, Hq, D), r(n, Hk, D), r(n, Hk, D)
    freq, axis = w4.rotary_frequencies((D,), theta=1e6)
    pos = torch.arange(n, device="cuda")[:, None] + 90000
    qr, kr = w4.qk_norm_rope(q, k, positions=pos, freq=freq, axis=axis, interleaved=False)
    whole, lse = w4.attention(qr, kr, v, causal=True, return_lse=True)
    ta.check(whole, lse, qr, kr, v, [n], [n], True)
    for t in (n - 1, n - 2, 300, 0):
        q1, k1 = w4.qk_norm_rope(q[t:t + 1], k[t:t + 1], positions=pos[t:t + 1], freq=freq, axis=axis, interleaved=False)
        assert torch.equal(q1[0], qr[t]) and torch.equal(k1[0], kr[t])
        o, z = w4.attention(q1, kr[:t + 1], v[:t + 1], causal=True, return_lse=True)
        ta.check(o, z, q1, kr[:t + 1], v[:t + 1], [1], [t + 1], True)


def test_small_layers_between_attentions(cuda_lib):
    """Layers of a few rows (tensor memory of their own, the next kernel let in
    early) between attentions that take all of an SM's tensor memory and those
    that take half: a long chain without a gap, eager and replayed, ends and
    gives what each call gives alone."""
    block = Block(8, 8, seed=7)
    gen = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
    long = [r(2600, 40, d) for d in (64, D)]                    # two query tiles a block
    few = r(600, 2, 64)                                         # one, and chunks of keys
    x = r(16, block.width)

    def chain(times):
        outs = []
        for _ in range(times):
            for t in (*long, few):
                outs.append(w4.attention(t, t, t, causal=True))
                outs.append(w4.linear_fused(x, *block.linears["out"]))
        return outs

    want = []
    for t in (*long, few):
        want.append(w4.attention(t, t, t, causal=True))
        torch.cuda.synchronize()
        want.append(w4.linear_fused(x, *block.linears["out"]))
        torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(chain(20), want * 20))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(1)                                                # the layers' workspace of this stream
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        outs = chain(5)
    for _ in range(10):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want * 5)) and w4.last_device_error() == 0


FIRST_CALL = """
import sys
sys.path.insert(0, {root!r})
import torch
import w4a4_hadamard_rotated_b200 as w4

gen = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)
q, k, v, x = r(300, 8, 128), r(300, 2, 128), r(300, 2, 128), r(3, 256)
codes, scale = torch.randint(-128, 128, (500, 128), generator=gen, device="cuda", dtype=torch.int8), r(500, 4)
freq, axis = w4.rotary_frequencies((128,))
pos = torch.arange(300, device="cuda")
copies = [torch.empty_like(t) for t in (q, k, x)]
side = torch.cuda.Stream()
torch.cuda.synchronize()


def block():
    # copies and fills before each kernel, and a branch that joins
    for c, t in zip(copies, (q, k, x)):
        c.copy_(t)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = w4.linear_w4a16(copies[2], codes, scale)
    qr, kr = w4.qk_norm_rope(copies[0], copies[1], positions=pos, freq=freq, axis=axis)
    out = torch.empty_like(q)
    out.zero_()
    w4.attention(qr, kr, v, causal=True, out=out)
    torch.cuda.current_stream().wait_stream(side)
    o2 = w4.attention(qr[:3], kr, v)
    return y, qr, kr, out, o2


g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = block()
for c in copies:
    c.fill_(7)
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = block()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and w4.last_device_error() == 0
print("same")
"""


def test_first_calls_inside_a_capture(cuda_lib):
    """In a process that has not called the library yet: each entry's first
    call captured into a graph, behind copies, fills and a joined branch."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(w4.__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=root)], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
