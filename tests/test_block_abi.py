"""Refusals of the entries that run between a block's linears: invalid
arguments come back as status codes before any CUDA call, and the binding
refuses tensors the library cannot take."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import w4a4_hadamard_rotated_b200 as w4

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)          # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p((1 << 20) + 2)
BYTE = ctypes.c_void_p((1 << 20) + 1)

NULL_, SHAPE, GROUP, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 5, 9


@pytest.fixture(scope="module")
def lib():
    return w4.load_library()


QUANT = dict(W=FAKE, N=8, K=256, ldw=256, group=64, dtype=0, Wq=FAKE, scale=FAKE, offset=NULL, stream=NULL)


@pytest.mark.parametrize("change,status", [
    (dict(W=NULL), NULL_), (dict(Wq=NULL), NULL_), (dict(scale=NULL), NULL_), (dict(group=16), GROUP),
    (dict(group=256), GROUP), (dict(K=96, ldw=96), GROUP), (dict(K=48, ldw=48), SHAPE), (dict(N=0), SHAPE),
    (dict(K=262144, ldw=262144), SHAPE), (dict(ldw=255), SHAPE), (dict(ldw=258), ALIGN), (dict(W=ODD), ALIGN),
    (dict(Wq=ODD), ALIGN), (dict(scale=BYTE), ALIGN), (dict(offset=BYTE), ALIGN), (dict(dtype=2), ARG)])
def test_quantize_weight_w4a16_refuses(lib, change, status):
    assert lib.w4a4_quantize_weight_w4a16(*{**QUANT, **change}.values()) == status


LINEAR = dict(x=FAKE, ldx=256, Wq=FAKE, scale=FAKE, offset=NULL, group=64, bias=NULL, y=FAKE, ldy=9, M=3, N=9, K=256,
              dtype=0, stream=NULL)


@pytest.mark.parametrize("change,status", [
    (dict(x=NULL), NULL_), (dict(Wq=NULL), NULL_), (dict(scale=NULL), NULL_), (dict(y=NULL), NULL_),
    (dict(group=48), GROUP), (dict(K=96, ldx=96), GROUP), (dict(K=0), SHAPE), (dict(K=40), SHAPE), (dict(N=0), SHAPE),
    (dict(M=-1), SHAPE), (dict(M=65), SHAPE), (dict(ldx=248), SHAPE), (dict(ldy=8), SHAPE), (dict(ldx=260), ALIGN),
    (dict(x=ODD), ALIGN), (dict(Wq=ODD), ALIGN), (dict(y=BYTE), ALIGN), (dict(bias=BYTE), ALIGN), (dict(dtype=-1), ARG)])
def test_linear_w4a16_refuses(lib, change, status):
    assert lib.w4a4_linear_w4a16(*{**LINEAR, **change}.values()) == status


ROPE = dict(q=FAKE, qt=512, qh=128, Hq=4, k=FAKE, kt=256, kh=128, Hk=2, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, bits=32,
            pt=3, axes=3, freq=FAKE, axis=FAKE, R=128, interleaved=1, qo=FAKE, qot=512, qoh=128, ko=FAKE, kot=256,
            koh=128, T=5, D=128, dtype=0, stream=NULL)


@pytest.mark.parametrize("change,status", [
    (dict(q=NULL), NULL_), (dict(k=NULL), NULL_), (dict(ko=NULL), NULL_), (dict(qo=NULL), NULL_),
    (dict(freq=NULL), NULL_), (dict(axis=NULL), NULL_), (dict(T=-1), SHAPE), (dict(D=100), SHAPE),
    (dict(D=264), SHAPE), (dict(D=0), SHAPE), (dict(Hq=0), SHAPE), (dict(Hk=-1), SHAPE), (dict(Hq=4090, Hk=8), SHAPE),
    (dict(R=0), SHAPE), (dict(R=130), SHAPE), (dict(R=63), SHAPE), (dict(R=24, interleaved=0), SHAPE),
    (dict(axes=0), SHAPE), (dict(axes=9, pt=9), SHAPE), (dict(pt=2), SHAPE), (dict(qt=64), SHAPE), (dict(kh=64), SHAPE),
    (dict(qot=0), SHAPE), (dict(qt=516), ALIGN), (dict(qoh=132), ALIGN), (dict(q=ODD), ALIGN), (dict(kw=ODD), ALIGN),
    (dict(pos=ODD), ALIGN), (dict(bits=16), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(dtype=3), ARG)])
def test_qk_norm_rope_refuses(lib, change, status):
    assert lib.w4a4_qk_norm_rope(*{**ROPE, **change}.values()) == status


ATTN = dict(q=FAKE, qt=1024, qh=128, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, out=FAKE, ot=1024, oh=128, lse=FAKE,
            cuq=FAKE, cuk=FAKE, B=2, Tq=100, Tk=200, Hq=8, Hk=2, D=128, causal=1, scale=0.1, dtype=0, ws=NULL, wsb=0,
            stream=NULL)


@pytest.mark.parametrize("change,status", [
    (dict(q=NULL), NULL_), (dict(k=NULL), NULL_), (dict(v=NULL), NULL_), (dict(out=NULL), NULL_), (dict(cuq=NULL), NULL_),
    (dict(cuk=NULL), NULL_), (dict(cuq=NULL, cuk=NULL), NULL_), (dict(B=0), SHAPE), (dict(D=96), SHAPE),
    (dict(Hk=3), SHAPE), (dict(Hk=0), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=65536, Hk=1), SHAPE), (dict(Tq=-1), SHAPE),
    (dict(Tk=2 ** 31), SHAPE), (dict(kt=64), SHAPE), (dict(vh=0), SHAPE), (dict(ot=100), SHAPE), (dict(qt=1028), ALIGN),
    (dict(v=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(lse=ODD), ALIGN), (dict(cuq=ODD), ALIGN), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(dtype=2), ARG)])
def test_attention_refuses(lib, change, status):
    assert lib.w4a4_attention(*{**ATTN, **change}.values()) == status


@pytest.mark.parametrize("Tq,Tk,B,Hq,Hk,D", [
    (0, 10, 1, 8, 8, 128), (-1, 10, 1, 8, 8, 128), (1, -1, 1, 8, 8, 128), (1, 10, 0, 8, 8, 128), (1, 10, 1, 8, 3, 128),
    (1, 10, 1, 0, 1, 128), (1, 10, 1, 8, 0, 128), (1, 10, 1, 8, 8, 0), (2 ** 62, 2 ** 62, 1, 8, 8, 128),
    (1, 2 ** 62, 1, 8, 8, 128), (1, 2 ** 20, 2 ** 60, 8, 8, 128), (1, 2 ** 20, 2 ** 62, 2 ** 62, 1, 128),
    (1, 2 ** 20, 1, 8, 8, 2 ** 62)])
def test_attention_workspace_of_sizes_that_are_refused(lib, Tq, Tk, B, Hq, Hk, D):
    """Sizes past the limits, up to those whose products do not fit 64 bits."""
    assert lib.w4a4_attention_workspace_bytes(Tq, Tk, B, Hq, Hk, D) == 0


@pytest.mark.parametrize("Tq,Tk,B,Hq,Hk,D", [
    (1, 2 ** 30, 1, 8, 1, 128), (2 ** 24, 2 ** 30, 2 ** 24, 8, 1, 128), (2 ** 30, 2 ** 30, 1, 65535, 1, 64),
    (200 * 32, 200 * 2 ** 17, 200, 8, 8, 128), (1024, 1024 * 1000, 1024, 32, 8, 128)])
def test_attention_workspace_stays_small(lib, Tq, Tk, B, Hq, Hk, D):
    """Beside the keys, for a few queries a sequence: 128 MB and a little."""
    assert lib.w4a4_attention_workspace_bytes(Tq, Tk, B, Hq, Hk, D) <= 129 * 2 ** 20


def test_binding_refuses_host_tensors_and_other_types():
    h = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    calls = [
        lambda: w4.quantize_weight_w4a16(torch.zeros(8, 128)),
        lambda: w4.linear_w4a16(torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.int8),
                                torch.zeros(8, 1, dtype=torch.bfloat16)),
        lambda: w4.qk_norm_rope(h, h),
        lambda: w4.attention(h, h, h),
    ]
    for call in calls:
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_rotary_frequencies():
    freq, axis = w4.rotary_frequencies((4, 6), theta=100.0, device="cpu")
    assert freq.dtype == torch.float64 and axis.dtype == torch.int32
    assert axis.tolist() == [0, 0, 1, 1, 1]
    assert freq.tolist() == pytest.approx([1.0, 100.0 ** -0.5, 1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)], rel=1e-15)
    for bad in ((), (3,), (0, 4), (4, -2)):
        with pytest.raises(ValueError):
            w4.rotary_frequencies(bad)


@pytest.mark.parametrize("Tq,Tk,B,Hq,Hk,D", [
    (128 * 16, 128 * 32768, 128, 8, 1, 128), (128 * 128, 128 * 32768, 128, 1, 1, 128), (18 * 9, 18 * 16384, 18, 32, 8, 128),
    (64 * 39, 64 * 8192, 64, 8, 1, 128), (64 * 33, 64 * 4096, 64, 8, 1, 128), (32 * 64, 32 * 8192, 32, 8, 1, 64),
    (5 * 7, 5 * 2 ** 20, 5, 64, 8, 128), (2 ** 20, 2 ** 30, 2 ** 16, 1, 1, 128)])
def test_attention_workspace_of_batches_stays_small(lib, Tq, Tk, B, Hq, Hk, D):
    """The same for more queries a sequence than a tile of few holds."""
    assert lib.w4a4_attention_workspace_bytes(Tq, Tk, B, Hq, Hk, D) <= 129 * 2 ** 20


def run_copy(tmp_path, leave_out, code):
    """`code` in a fresh interpreter over a copy of the package without some of its files."""
    at = tmp_path / "w4a4_hadamard_rotated_b200"
    at.mkdir()
    here = os.path.dirname(w4.__file__)
    for name in ("__init__.py", "build.py", "libw4a4.so", "_binding.so"):
        if name not in leave_out:
            os.symlink(os.path.join(here, name), at / name)
    code = f"import sys; sys.path.insert(0, {str(tmp_path)!r})\nimport torch, w4a4_hadamard_rotated_b200 as w4\n" + code
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=tmp_path)


def test_layer_entries_do_not_need_the_extension(tmp_path):
    """libw4a4.so alone serves every entry but the three that the extension
    marshals, and those say what is missing."""
    r = run_copy(tmp_path, ["_binding.so"], """
assert w4.load_library().w4a4_version() >= 100
assert w4.linear_kernel(4096, 512, 512) == 0
h = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
for call in (lambda: w4.linear(h, h, h, h), lambda: w4.quantize_weight_w4a16(h)):
    try:
        call()
        raise SystemExit("taken")
    except TypeError:
        pass
for call in (lambda: w4.attention(h, h, h), lambda: w4.qk_norm_rope(h, h), lambda: w4.linear_w4a16(h, h, h)):
    for _ in range(2):
        try:
            call()
            raise SystemExit("taken")
        except RuntimeError as e:
            assert "_binding.so is missing" in str(e), e
""")
    assert r.returncode == 0, r.stdout + r.stderr


def test_extension_of_another_pytorch_or_python_is_not_loaded(tmp_path):
    r = run_copy(tmp_path, [], """
h = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
torch.__version__ = "1.0"
try:
    w4.attention(h, h, h)
    raise SystemExit("taken")
except RuntimeError as e:
    assert "not built for torch 1.0" in str(e), e
assert w4.load_library().w4a4_version() >= 100
""")
    assert r.returncode == 0, r.stdout + r.stderr


def test_extension_is_built_again_for_another_pytorch(monkeypatch):
    """By the build's rule of what is up to date; the compiler is not run."""
    from w4a4_hadamard_rotated_b200 import build
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "_up_to_date", lambda *_: True)     # by its time
    build.build_binding()
    assert not ran
    monkeypatch.setattr(torch, "__version__", "1.0")
    build.build_binding()
    assert len(ran) == 1 and any("torch 1.0" in a for a in ran[0])


def test_attention_of_too_many_sequences(lib):
    """The time to find a block's sequence grows with their number: 65536 at most."""
    most = {**ATTN, "B": 65536, "lse": ODD}                     # the lengths are taken, the next check is not
    assert lib.w4a4_attention(*most.values()) == ALIGN
    for B in (65537, 2 ** 20, 2 ** 24):
        assert lib.w4a4_attention(*{**ATTN, "B": B, "lse": ODD}.values()) == SHAPE
        assert lib.w4a4_attention_workspace_bytes(B, 2 ** 30, B, 8, 1, 128) == 0
