"""Refusals of the few-token product and of the products of 8-bit x, made on the host before any device call."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

from ring_allreduce_gradient_gb300 import binding as B
from ring_allreduce_gradient_gb300 import build as cuda_build
from ring_allreduce_gradient_gb300 import mx4, mx8

BASE = 0x7F0000000000
OK, INVALID, UNSUPPORTED, ALIAS = (B.DP_OK, B.DP_ERR_INVALID_ARG, B.DP_ERR_UNSUPPORTED,
                                   B.DP_ERR_ALIAS)
MX, NV = B.DP_MXFP4, B.DP_NVFP4


def fake(i, off=0):
    return BASE + (i << 26) + off


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return B.load()


def test_checks(lib):
    ws = [(fake(2 * k + 2), fake(2 * k + 3), None) for k in range(2)]

    def m(x=fake(0), M=4, D=64, ld=64, w=ws, K=2, Fs=32, fmt=MX, y=fake(20), dt=B.DP_BF16,
          work=None, wb=0):
        return B.dp_allgather_linear_w4(x, M, D, ld, w, K, Fs, fmt, y, dt, work, wb, stream=0,
                                        check=False)

    assert m(K=0) == INVALID and m(K=17) == INVALID
    assert m(M=-1) == INVALID and m(D=-32) == INVALID and m(Fs=-16) == INVALID
    assert m(ld=63) == INVALID and m(x=None) == INVALID and m(y=None) == INVALID
    assert m(w=[ws[0], (None, fake(5), None)]) == INVALID
    assert m(w=[ws[0], (fake(4), None, None)]) == INVALID
    assert m(w=[ws[0], (fake(4), fake(5), fake(9))]) == INVALID    # a tensor scale with mxfp4
    assert m(fmt=2) == UNSUPPORTED and m(dt=5) == UNSUPPORTED
    assert m(D=48, ld=48) == UNSUPPORTED and m(Fs=24) == UNSUPPORTED
    assert m(D=(1 << 30) + 32, ld=(1 << 30) + 32) == UNSUPPORTED
    assert m(M=65535 * 8 + 1) == UNSUPPORTED and m(K=16, w=ws * 8, Fs=0x8000000) == UNSUPPORTED
    assert m(x=fake(0, 1)) == UNSUPPORTED and m(y=fake(20, 1)) == UNSUPPORTED
    assert m(y=fake(20, 2), dt=B.DP_FP32) == UNSUPPORTED
    assert m(w=[(fake(2, 8), fake(3), None), ws[1]]) == UNSUPPORTED
    assert m(w=[(fake(2), fake(3, 4), None), ws[1]]) == UNSUPPORTED
    assert m(fmt=NV, w=[(fake(2), fake(3), fake(9, 2)), ws[1]]) == UNSUPPORTED
    assert m(y=fake(0)) == ALIAS and m(y=fake(2, 16)) == ALIAS and m(y=fake(5, 16)) == ALIAS
    assert m(fmt=NV, w=[(fake(2), fake(3), fake(20, 4)), ws[1]]) == ALIAS
    assert m(M=0, y=None) == OK and m(Fs=0, y=None) == OK
    # more than eight tokens are prepared in a workspace
    size = B.dp_allgather_linear_w4_workspace_size
    assert size(8, 64) == 0 and size(9, 0) == 0 and size(9, 64) == 9 * 256 + 9 * 4
    assert size(20, 160) == 20 * 512 + 20 * 4
    need = size(9, 64)
    assert m(M=9) == INVALID and m(M=9, work=fake(30), wb=need - 1) == INVALID
    assert m(M=9, work=fake(30, 8), wb=need) == UNSUPPORTED
    for at in (fake(0, 16), fake(20), fake(2), fake(5)):
        assert m(M=9, work=at, wb=need) == ALIAS
    assert m(M=9, fmt=NV, w=[(fake(2), fake(3), fake(30, 64)), ws[1]], work=fake(30),
             wb=need) == ALIAS
    n = ctypes.c_size_t(3)
    assert lib.dp_allgather_linear_w4_workspace_size(1, 1, None) == INVALID
    assert lib.dp_allgather_linear_w4_workspace_size(-1, 1, ctypes.byref(n)) == INVALID


def test_the_helper_checks():
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    q = mx4.Mx4Tensor(u8(16 * 32), u8(512), 16, 64, "mxfp4")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for args, err, word in [((x.float(), [q]), TypeError, "bf16"),
                            ((x, [q], torch.float16), TypeError, "dtype"),
                            ((x, []), ValueError, "at least one shard"),
                            ((x[:, :32], [q]), ValueError, "columns"),
                            ((x[0], [q]), ValueError, "need a matrix"),
                            ((x, [q]), B.DpError, "not the current CUDA device")]:
        with pytest.raises(err, match=word):
            mx4.linear_w4(*args)


def test_eight_bit_product_checks():
    ws = [(fake(2 * k + 2), fake(2 * k + 3), None) for k in range(2)]
    x = (fake(0), fake(1), None)

    def m(x=x, M=64, D=64, w=ws, K=2, Fs=32, y=fake(20), dt=B.DP_BF16):
        return B.dp_allgather_matmul_mx8(x, M, D, w, K, Fs, y, dt, stream=0, check=False)

    assert m(K=0) == INVALID and m(K=17) == INVALID and m(M=-1) == INVALID
    assert m(x=(None, fake(1), None)) == INVALID and m(x=(fake(0), None, None)) == INVALID
    assert m(x=(fake(0), fake(1), fake(9))) == INVALID and m(y=None) == INVALID
    assert m(w=[ws[0], (None, fake(5), None)]) == INVALID
    assert m(D=48) == UNSUPPORTED and m(Fs=24) == UNSUPPORTED and m(dt=5) == UNSUPPORTED
    assert m(x=(fake(0, 8), fake(1), None)) == UNSUPPORTED and m(y=fake(20, 4)) == UNSUPPORTED
    assert m(y=fake(0)) == ALIAS and m(y=fake(0, 64 * 64 - 16)) == ALIAS    # 8 bits: 64 x 64 bytes
    assert m(y=fake(1)) == ALIAS and m(y=fake(4, 512)) == ALIAS and m(y=fake(5)) == ALIAS
    assert m(M=0, y=None) == OK and m(Fs=0, y=None) == OK

    need = B.dp_allgather_linear_mx8_workspace_size(64, 64)
    assert need == 64 * 64 + 512

    def lin(x=fake(0), M=64, D=64, ld=64, xdt=B.DP_BF16, w=ws, Fs=32, y=fake(20), dt=B.DP_BF16,
            work=fake(30), wb=need):
        return B.dp_allgather_linear_mx8(x, M, D, ld, xdt, w, 2, Fs, y, dt, work, wb, stream=0,
                                         check=False)

    assert lin(work=None) == INVALID and lin(wb=need - 1) == INVALID and lin(M=-1) == INVALID
    assert lin(work=fake(30, 8)) == UNSUPPORTED and lin(D=48, ld=48) == UNSUPPORTED
    assert lin(work=fake(20)) == ALIAS and lin(work=fake(2)) == ALIAS and lin(work=fake(3)) == ALIAS
    assert lin(y=fake(0, 64)) == ALIAS


def test_the_eight_bit_helpers_check():
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    w = mx4.Mx4Tensor(u8(16 * 32), u8(512), 16, 64, "mxfp4")
    nv = mx4.Mx4Tensor(u8(16 * 32), u8(512), 16, 64, "nvfp4")
    q = mx8.Mx8Tensor(u8(4 * 64), u8(512), 4, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call, a in ((mx8.linear, x), (mx8.matmul, q)):
        for args, err, word in [((a, [w], torch.float16), TypeError, "dtype"),
                                ((a, []), ValueError, "at least one shard"),
                                ((a, [nv]), ValueError, "mxfp4"),
                                ((a, [w, nv]), ValueError, "one shape"),
                                ((a, [w]), B.DpError, "not the current CUDA device")]:
            with pytest.raises(err, match=word):
                call(*args)
    # 4-bit matrices where 8-bit ones belong, and the other way round: their buffers differ in size
    w8 = mx8.Mx8Tensor(u8(16 * 64), u8(512), 16, 64)
    for call in (lambda: mx8.matmul(w, [w]), lambda: mx8.dequantize(w), lambda: mx8.linear(x, [w8]),
                 lambda: mx4.matmul(q, [w]), lambda: mx4.matmul(w, [w8]),
                 lambda: mx8.matmul(q, [w8])):
        with pytest.raises(ValueError, match="mxfp"):
            call()
    for call in (lambda: mx4.dequantize(q), lambda: mx4.linear(x, [w8]), lambda: mx4.matmul(q, [w8]),
                 lambda: mx4.linear_w4(x, [w8])):
        with pytest.raises(KeyError, match="mxfp8"):
            call()
    with pytest.raises(TypeError, match="dtype"):
        mx8.linear(x.half(), [w])
    with pytest.raises(ValueError, match="columns"):
        mx8.linear(x[:, :32], [w])


def test_matrices_of_another_form_are_named():
    """An 8-bit matrix where a 4-bit one belongs is refused as other wrong values are, by name."""
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    q = mx8.Mx8Tensor(u8(16 * 64), u8(512), 16, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: mx4.dequantize(q), lambda: mx4.linear(x, [q]), lambda: mx4.matmul(q, [q]),
                 lambda: mx4.linear_w4(x, [q]), lambda: mx4.dequantize(q, stream=0),
                 lambda: mx4.matmul(q, [q], stream=0)):
        with pytest.raises(ValueError, match=r"^need an mxfp4 or nvfp4 matrix, not mxfp8: Mx8Tensor\(16 x 64"):
            call()


# Prints the few-token product's plan for each line "tokens D units mx nt ready".
PLANNER = r"""
#include "dp_w4_plan.h"
#include <cstdio>
int main() {
  int tokens, D, units, mx, nt, ready;
  while (std::scanf("%d %d %d %d %d %d", &tokens, &D, &units, &mx, &nt, &ready) == 6) {
    const w4::Plan p = w4::plan(tokens, D, units, mx, nt, ready);
    std::printf("%d %d %d %d %d %d %zu\n", p.split, p.split_bits, p.per, p.warps, p.slab, p.slabs,
                p.smem);
  }
}
"""


def test_the_plan_follows_from_the_sizes(tmp_path):
    """The order of the few-token product's sums is its plan's, which is made without a device:
    from the sizes.  Every plan covers d and the units, and stays within a CTA's means."""
    csrc = os.path.join(os.path.dirname(B.__file__), "csrc")
    (tmp_path / "p.cpp").write_text(PLANNER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", csrc,
                    str(tmp_path / "p.cpp"), "-o", str(tmp_path / "p")], check=True)
    rng = random.Random(5)
    cases = [(1, 4096, 128), (1, 8192, 2048), (8, 32, 4), (16, 8192, 2048), (32, 1 << 30, 4),
             (32, 8192, 1 << 26), (1, 1 << 30, 4), (8, 1 << 30, 4), (9, 16384, 4)]
    for _ in range(3000):
        cases.append((rng.choice([1, 2, 3, 5, 8, 9, 12, 16, 17, 31, 32]),
                      32 * int(2 ** rng.uniform(0, 12)), 4 * int(2 ** rng.uniform(0, 14))))
    lines = []
    for tokens, D, units in cases:
        nt = 1 if tokens <= 8 else 2 if tokens <= 16 else 4
        for mx in (0, 1):
            lines.append((tokens, D, units, mx, nt, int(tokens > 8)))
    out = subprocess.run([str(tmp_path / "p")], input="\n".join(" ".join(map(str, c)) for c in lines),
                         capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(lines)
    for (tokens, D, units, mx, nt, ready), o in zip(lines, out):
        split, bits, per, warps, slab, slabs, smem = map(int, o.split())
        steps = -(-D // 128)
        assert split == 1 << bits and warps == per * split and 1 <= warps <= 16
        assert split == 1 or (split <= steps and units * split <= 16 * 152)
        assert slab >= 1 and split * slabs * slab >= steps and (slabs - 1) * slab < -(-steps // split)
        assert warps * 32 >= split * tokens or not ready       # a lane copies a token's slab
        assert smem <= 220 << 10
        step = 32 * 64 + (128 if mx else 256)
        ring = warps * (2 if nt == 4 else 3) * step
        assert smem == ring + (2 if slabs > 1 else 1) * split * tokens * (slab * 256 + 64)
        if not ready and slabs > 1:
            assert slab >= 2                    # a slab of one step would not wait for the next
    with open(os.path.join(csrc, "dp_w4.cu")) as f:
        assert "sm_count" not in f.read()
