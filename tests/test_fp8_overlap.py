"""Outputs of the 8-bit layer's operators that lie over inputs or over each other are refused on the host, before anything is
enqueued; slices of the same rows are not (no GPU needed)."""
import os
import shutil
import subprocess

import pytest
import torch

import shape_driven_tile_gb300 as sdt
from shape_driven_tile_gb300 import fp8, rope

CSRC = os.path.join(os.path.dirname(os.path.abspath(sdt.__file__)), "csrc")
ARG = -10
BF16, F32, E4M3 = 1, 3, 4
T, W = 4, 256  # tokens and width; a row's bytes are 256 in fp8, 512 in 16 bits


def called(fn, pack, fields):
    rc = getattr(sdt.lib(), fn)(pack.pack(*fields.values()), None)
    return rc, sdt.lib().sdt_last_error().decode()


def refused(fn, pack, fields):
    rc, why = called(fn, pack, fields)
    return rc == ARG and "overlap" in why or rc == ARG and "lie apart" in why


def allowed(fn, pack, fields):
    """Past every check: the call then finds no GPU.  (With one, it would run on addresses that are none.)"""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    rc, why = called(fn, pack, fields)
    return rc == -4, why


def at(i):
    return 0x100000 * (i + 1)


QUANT = dict(x=at(0), gate=at(1), q=at(2), scales=at(3), tokens=T, width=W, x_row=W, gate_row=W, q_row=W, s_row=2, s_block=1, dtype=BF16,
             activation=1)
NORM = dict(x=at(0), weight=at(1), residual=at(2), out=at(3), q=at(4), scales=at(5), tokens=T, width=W, x_row=W, r_row=W, o_row=W, q_row=W,
            s_row=2, s_block=1, eps=1e-6, dtype=BF16, weight_dtype=F32)
GEMM = dict(a=at(0), a_scales=at(1), w=at(2), w_scales=at(3), c=at(4), M=T, N=64, K=W, lda=W, ldw=W, ldc=64, as_row=2, as_block=1, ws_row=2,
            ws_block=1, a_dtype=E4M3, w_dtype=E4M3, c_dtype=F32, tile=0, splits=0)
ROPE = dict(q=at(0), k=at(1), q_out=at(2), k_out=at(3), positions=at(4), turns=at(5), tokens=T, q_heads=4, k_heads=2, head_dim=64, rotary=64,
            q_token=256, q_head=64, k_token=128, k_head=64, qo_token=256, qo_head=64, ko_token=128, ko_head=64, magnitude=1.0, dtype=BF16,
            position_bytes=8, interleaved=0, inverse=0)
CALLS = {"gemm_fp8": (fp8._GEMM, GEMM, ("c",), dict(a=1024, a_scales=32, w=64 * 256, w_scales=8, c=1024)),
         "quant_fp8": (fp8._QUANT, QUANT, ("q", "scales"), dict(x=2048, gate=2048, q=1024, scales=32)),
         "rms_norm_fp8": (fp8._NORM, NORM, ("residual", "out", "q", "scales"),
                          dict(x=2048, weight=1024, residual=2048, out=2048, q=1024, scales=32)),
         "rope_qk": (rope._ROPE, ROPE, ("q_out", "k_out"), dict(q=2048, k=1024, q_out=2048, k_out=1024, positions=32, turns=256))}
PAIRS = [(fn, o, x) for fn, (_, _, outs, sizes) in CALLS.items() for o in outs for x in sizes if x != o and (fn, o, x) != ("rope_qk", "q_out", "q")
         and (fn, o, x) != ("rope_qk", "k_out", "k")]


@pytest.mark.parametrize("fn", CALLS)
def test_tensors_apart_are_taken(fn):
    pack, fields, _, _ = CALLS[fn]
    ok, why = allowed(fn, pack, fields)
    assert ok, why


@pytest.mark.parametrize("fn,out,other", PAIRS)
def test_an_output_over_another_tensor(fn, out, other):
    """The first and the last bytes in common; one step further they lie apart."""
    pack, fields, _, sizes = CALLS[fn]
    for shift in {0, (sizes[other] - 1) // 16 * 16}:  # the output starts at the other's first or last 16 bytes
        assert refused(fn, pack, {**fields, out: fields[other] + shift}), shift
    last = sizes[out] - 1 & ~15  # the other starts at the output's last 16 bytes
    assert refused(fn, pack, {**fields, out: fields[other] - last})
    for shift in (-(-sizes[other] // 16) * 16, -(-(-sizes[out] // 16) * 16)):
        ok, why = allowed(fn, pack, {**fields, out: fields[other] + shift})
        assert ok, (shift, why)


def test_slices_of_the_same_rows():
    row = 4096  # bytes
    quant = {**QUANT, "x": at(0), "gate": at(0) + 512, "q": at(0) + 1024, "scales": at(0) + 1280, "x_row": row // 2, "gate_row": row // 2,
             "q_row": row, "s_row": row // 4}
    assert allowed("quant_fp8", fp8._QUANT, quant)[0]
    for change in (dict(q=at(0) + 1016), dict(q=at(0) + 3848), dict(scales=at(0) + 1276), dict(scales=at(0) + 4092), dict(q_row=row + 8),
                   dict(q=at(0) + 3840 + 256, tokens=2, x=at(0) + row)):
        assert refused("quant_fp8", fp8._QUANT, {**quant, **change}), change
    norm = {**NORM, "x": at(0), "residual": at(0) + 512, "out": at(0) + 1024, "q": at(0) + 1536, "scales": at(0) + 1792, "x_row": row // 2,
            "r_row": row // 2, "o_row": row // 2, "q_row": row, "s_row": row // 4}
    assert allowed("rms_norm_fp8", fp8._NORM, norm)[0]
    for change in (dict(out=at(0) + 1024 - 16), dict(out=at(0)), dict(out=at(0) + 512), dict(residual=at(0) + 496), dict(r_row=W),
                   dict(scales=at(0) + 1788), dict(weight=at(0) + row + 1536)):
        assert refused("rms_norm_fp8", fp8._NORM, {**norm, **change}), change
    gemm = {**GEMM, "a": at(0), "c": at(0) + 256, "lda": row, "ldc": row // 4}
    assert allowed("gemm_fp8", fp8._GEMM, gemm)[0]
    for change in (dict(c=at(0) + 240), dict(c=at(0) + row - 240), dict(a_scales=at(0) + 2 * row + 508), dict(w_scales=at(0) + 256)):
        assert refused("gemm_fp8", fp8._GEMM, {**gemm, **change}), change


def test_slices_of_the_same_rows_turned():
    token = 2048  # elements; queries, keys, then room for both outputs
    sides = dict(q=at(0), k=at(0) + 512, q_out=at(0) + 768, k_out=at(0) + 1280, q_token=token, k_token=token, qo_token=token, ko_token=token)
    turned = {**ROPE, **sides}
    assert allowed("rope_qk", rope._ROPE, turned)[0]
    assert allowed("rope_qk", rope._ROPE, {**turned, "q_out": at(0), "k_out": at(0) + 512})[0]
    # heads outside tokens, next to one another
    assert allowed("rope_qk", rope._ROPE, {**ROPE, "q": at(0), "q_token": 128, "q_head": 2048, "q_out": at(0) + 128, "qo_token": 128, "qo_head": 2048})[0]
    for change in (dict(q_out=at(0) + 752), dict(k_out=at(0) + 1264), dict(k_out=at(0) + 768), dict(q_out=at(0) + 16), dict(k_out=at(0) + 256),
                   dict(q_out=at(0) + 512), dict(positions=at(0) + 800)):
        assert refused("rope_qk", rope._ROPE, {**turned, **change}), change
    assert refused("rope_qk", rope._ROPE, {**ROPE, "q": at(0), "q_token": 128, "q_head": 2048, "q_out": at(0) + 112, "qo_token": 128, "qo_head": 2048})


PROGRAM = r"""
#include "overlap.cuh"
#include <cstdio>
#include <random>
#include <set>
using namespace sdt;
int main() {
    std::mt19937 g(1);
    const auto r = [&](int lo, int hi) { return int(g() % (hi - lo + 1)) + lo; };
    long yes = 0;
    for (long n = 0; n < 100000; ++n) {
        Stretches s[2];
        std::set<uintptr_t> bytes[2];
        for (int k = 0; k < 2; ++k) {
            s[k] = {reinterpret_cast<void *>(uintptr_t(1000 + r(0, 60))), r(1, 4), r(0, 24), r(1, 4), r(0, 24), r(1, 6)};
            for (int i = 0; i < s[k].n0; ++i)
                for (int j = 0; j < s[k].n1; ++j)
                    for (int l = 0; l < s[k].len; ++l) bytes[k].insert(reinterpret_cast<uintptr_t>(s[k].p) + i * s[k].step0 + j * s[k].step1 + l);
        }
        bool want = false;
        for (uintptr_t x : bytes[0]) want = want || bytes[1].count(x);
        if (overlap(s[0], s[1]) != want || overlap(s[1], s[0]) != want) return 1;
        yes += want;
    }
    printf("%ld\n", yes);
}
"""


def test_strided_tensors_against_their_bytes(tmp_path):
    compiler = next((c for c in ("c++", "g++") if shutil.which(c)), None)
    if compiler is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run([compiler, "-O1", "-std=c++17", "-I", CSRC, str(tmp_path / "p.cpp"), "-o", str(tmp_path / "p")], check=True, capture_output=True)
    out = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True)
    assert out.returncode == 0 and 20000 < int(out.stdout) < 80000
