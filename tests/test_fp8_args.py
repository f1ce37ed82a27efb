"""What the 8-bit layer's operators refuse on the host, before anything is enqueued (no GPU needed)."""
import math
from fractions import Fraction

import pytest
import torch

import shape_driven_tile_gb300 as sdt
from shape_driven_tile_gb300 import fp8, rope

A = 0x10000  # an address that is aligned to everything; never followed
NULL, ALIGN, SHAPE, TILE, ARG = -1, -2, -3, -7, -10
F16, BF16, Q8, F32, E4M3, E5M2 = range(6)


def called(fn, pack, defaults, change):
    assert not set(change) - set(defaults)
    return getattr(sdt.lib(), fn)(pack.pack(*(0 if v is None else v for v in {**defaults, **change}.values())), None)


GEMM = dict(a=A, a_scales=A, w=A, w_scales=A, c=A, M=4, N=64, K=256, lda=256, ldw=256, ldc=64, as_row=2, as_block=1, ws_row=2,
            ws_block=1, a_dtype=E4M3, w_dtype=E4M3, c_dtype=BF16, tile=0, splits=0)
QUANT = dict(x=A, gate=0, q=A, scales=A, tokens=4, width=256, x_row=256, gate_row=256, q_row=256, s_row=2, s_block=1, dtype=BF16,
             activation=0)
NORM = dict(x=A, weight=A, residual=A, out=0, q=A, scales=A, tokens=4, width=256, x_row=256, r_row=256, o_row=256, q_row=256, s_row=2,
            s_block=1, eps=1e-6, dtype=BF16, weight_dtype=BF16)
ROPE = dict(q=A, k=2 * A, q_out=3 * A, k_out=4 * A, positions=A, turns=A, tokens=4, q_heads=4, k_heads=2, head_dim=64, rotary=64,
            q_token=256, q_head=64, k_token=128, k_head=64, qo_token=256, qo_head=64, ko_token=128, ko_head=64, magnitude=1.0,
            dtype=BF16, position_bytes=8, interleaved=0, inverse=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), SHAPE), (dict(N=-8), SHAPE), (dict(K=-1), SHAPE), (dict(M=2 ** 30 + 1), SHAPE), (dict(N=60), SHAPE),
    (dict(K=2 ** 31), SHAPE), (dict(a_dtype=BF16), ARG), (dict(w_dtype=Q8), ARG), (dict(c_dtype=Q8), ARG), (dict(c_dtype=E4M3), ARG),
    (dict(tile=1), TILE), (dict(tile=-16), TILE), (dict(splits=-1), ARG), (dict(splits=9), ARG), (dict(a=None), NULL),
    (dict(a_scales=None), NULL), (dict(w=None), NULL), (dict(w_scales=None), NULL), (dict(c=None), NULL), (dict(a=A + 8), ALIGN),
    (dict(w=A + 1), ALIGN), (dict(c=A + 8), ALIGN), (dict(a_scales=A + 2), ALIGN), (dict(w_scales=A + 1), ALIGN), (dict(lda=240), ARG),
    (dict(lda=264), ARG), (dict(ldw=128), ARG), (dict(ldw=257), ARG), (dict(ldc=56), ARG), (dict(ldc=68), ARG), (dict(as_row=-1), ARG),
    (dict(ws_block=-2), ARG), (dict(as_block=2 ** 33), ARG), (dict(lda=2 ** 33), ARG)])
def test_gemm(change, status):
    assert called("gemm_fp8", fp8._GEMM, GEMM, change) == status


@pytest.mark.parametrize("change", [dict(M=0, a=0, c=0), dict(N=0, w=0)])
def test_gemm_of_nothing(change):
    assert called("gemm_fp8", fp8._GEMM, GEMM, change) == 0


def test_null_calls():
    for fn in ("gemm_fp8", "quant_fp8", "rms_norm_fp8", "rope_qk"):
        assert getattr(sdt.lib(), fn)(None, None) == NULL


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), SHAPE), (dict(width=-8), SHAPE), (dict(width=252), SHAPE), (dict(width=65544), SHAPE), (dict(tokens=2 ** 28), SHAPE),
    (dict(dtype=F32), ARG), (dict(activation=3), ARG), (dict(activation=1), ARG), (dict(gate=A), ARG), (dict(x=None), NULL),
    (dict(q=None), NULL), (dict(scales=None), NULL), (dict(x=A + 8), ALIGN), (dict(gate=A + 8, activation=1), ALIGN), (dict(q=A + 4), ALIGN),
    (dict(scales=A + 2), ALIGN), (dict(x_row=260), ARG), (dict(x_row=-8), ARG), (dict(gate=A, activation=2, gate_row=4), ARG),
    (dict(q_row=248), ARG), (dict(q_row=260), ARG), (dict(s_row=-2), ARG), (dict(s_row=1), ARG), (dict(s_block=0), ARG),
    (dict(s_row=0), ARG), (dict(s_row=1, s_block=3), ARG)])
def test_quant(change, status):
    assert called("quant_fp8", fp8._QUANT, QUANT, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(width=32776), SHAPE), (dict(width=12), SHAPE), (dict(tokens=-1), SHAPE), (dict(dtype=F32), ARG), (dict(weight_dtype=F16), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(weight=None), NULL), (dict(x=None), NULL), (dict(weight=A + 4), ALIGN),
    (dict(residual=A + 2), ALIGN), (dict(out=A + 2), ALIGN), (dict(r_row=128), ARG), (dict(out=A, o_row=260), ARG), (dict(q_row=0), ARG),
    (dict(s_row=0), ARG)])
def test_norm(change, status):
    assert called("rms_norm_fp8", fp8._NORM, NORM, change) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F32), ARG), (dict(head_dim=63, rotary=62), SHAPE), (dict(rotary=66), SHAPE), (dict(rotary=63), SHAPE), (dict(rotary=-2), SHAPE),
    (dict(head_dim=2 ** 17), SHAPE), (dict(tokens=-1), SHAPE), (dict(q_heads=-1), SHAPE), (dict(k_heads=65536), SHAPE), (dict(tokens=2 ** 24), SHAPE),
    (dict(position_bytes=2), ARG), (dict(q=None), NULL), (dict(k_out=None), NULL), (dict(positions=None), NULL), (dict(turns=None), NULL),
    (dict(q=A + 1), ALIGN), (dict(positions=A + 4), ALIGN), (dict(turns=A + 4), ALIGN), (dict(q_token=-1), ARG), (dict(k_head=2 ** 41), ARG),
    (dict(qo_head=32), ARG), (dict(qo_token=64), ARG), (dict(ko_token=0), ARG), (dict(q_out=A + 128), ARG), (dict(q_out=A, qo_token=512), ARG), (dict(q_out=4 * A), ARG), (dict(q_out=2 * A), ARG),
    (dict(k_out=A), ARG)])
def test_rope(change, status):
    assert called("rope_qk", rope._ROPE, ROPE, change) == status


def test_the_binding_names_what_is_wrong():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, s = x.to(torch.float8_e4m3fn), torch.ones(4, 2)
    table = object()
    for call, error, words in [
            (lambda: sdt.gemm_fp8(q, s, q, s), ValueError, "a_scales|CUDA"), (lambda: sdt.gemm_fp8(x, s, q, s), TypeError, "a must be"),
            (lambda: sdt.gemm_fp8(None, s, q, s), TypeError, "a must be"), (lambda: sdt.gemm_fp8(q, s, q[:, :128], s), ValueError, "w must be|CUDA"),
            (lambda: sdt.quant_fp8(q), TypeError, "x must be"), (lambda: sdt.quant_fp8(x), ValueError, "CUDA"),
            (lambda: sdt.quant_fp8(x[0]), ValueError, "x must be"), (lambda: sdt.rms_norm_fp8(x, x), ValueError, "CUDA|weight"),
            (lambda: sdt.rms_norm_fp8([1], x), TypeError, "x must be"), (lambda: sdt.rope_qk(x, None, s, table), ValueError, "q must be"),
            (lambda: sdt.rope_qk("q", None, s, table), TypeError, "q must be")]:
        with pytest.raises(error, match=words):
            call()


@pytest.mark.parametrize("kw,words", [
    (dict(rotary=63), "even"), (dict(rotary=0), "even"), (dict(scaling="no"), "scaling"), (dict(base=1.0), "base"), (dict(base=math.inf), "base"),
    (dict(factor=0.5), "factor"), (dict(factor=math.nan), "factor"), (dict(scaling="ramp"), "original_length"),
    (dict(scaling="smooth", original_length=0), "original_length"), (dict(scaling="ramp", original_length=4096, low=32.0, high=1.0), "low"),
    (dict(scaling="base", rotary=2), "rotary")])
def test_frequencies_refused(kw, words):
    with pytest.raises(ValueError, match=words):
        sdt.rope_frequencies(**{"rotary": 64, **kw})


def test_tables_refused():
    for kw, words in [(dict(frequencies=[1.0]), "frequencies"), (dict(frequencies=[]), "frequencies"),
                      (dict(frequencies=[math.nan, 1.0]), "finite"), (dict(magnitude=math.inf), "magnitude"), (dict(magnitude=1e31), "magnitude")]:
        with pytest.raises(ValueError, match=words):
            sdt.RopeTable(4, device="cpu", **kw)
    with pytest.raises(TypeError, match="rotary"):
        sdt.RopeTable(4.0, device="cpu")
    with pytest.raises(TypeError, match="rotary"):
        sdt.RopeTable(4.0, frequencies=[1.0, 0.5], device="cpu")


def two_pi(bits):
    """2 pi * 2^bits to the nearest integer, by Machin's formula."""
    def arctan_inverse(n):
        total, term, k = Fraction(0), Fraction(1, n), 0
        while abs(term) > Fraction(1, 1 << (bits + 40)):
            total += term / (2 * k + 1) * (-1) ** k
            term, k = term / (n * n), k + 1
        return total
    return round(2 * 4 * (4 * arctan_inverse(5) - arctan_inverse(239)) * (1 << bits))


@pytest.mark.parametrize("f", [1.0, 0.5, 1e-5, 7.0, -0.25, 1e-300, 5e-324, 123456.789, 0.0, -1.0, 2 * math.pi])
def test_turns_are_the_frequency_to_64_bits(f):
    want = Fraction(f) * (1 << 400) / two_pi(400)
    off = (Fraction(rope._turns(f), 1 << 64) - want) % 1
    assert min(off, 1 - off) <= Fraction(1, 1 << 64)


def test_frequencies_of_the_scalings():
    own, one = sdt.rope_frequencies(128)
    assert one == 1.0 and own[0] == 1.0 and math.isclose(own[32], 0.01, rel_tol=1e-14) and len(own) == 64
    assert sdt.rope_frequencies(128, scaling="linear", factor=4.0)[0] == [f / 4 for f in own]
    based, _ = sdt.rope_frequencies(128, scaling="base", factor=4.0)
    assert based[0] == 1.0 and math.isclose(based[-1] * 4, own[-1], rel_tol=1e-12)  # the slowest pair is slowed by the factor
    for how in ("ramp", "smooth"):
        scaled, magnitude = sdt.rope_frequencies(128, scaling=how, factor=8.0, original_length=4096)
        ratio = [a / b for a, b in zip(scaled, own)]
        assert ratio[0] == 1.0 and math.isclose(ratio[-1], 1 / 8) and all(a >= b - 1e-12 for a, b in zip(ratio, ratio[1:]))
        assert any(1 / 8 < r < 1 for r in ratio) and math.isclose(magnitude, 1 + 0.1 * math.log(8) if how == "ramp" else 1.0)


@pytest.mark.parametrize("m", [1, 16, 17, 64, 100, 128, 129, 4096])
@pytest.mark.parametrize("n,k", [(8, 16), (4096, 14336), (12288, 4096), (248, 2000), (28672, 8192)])
def test_plans(m, n, k):
    tile, splits = sdt.gemm_fp8_plan(m, n, k)
    assert 1 <= splits <= min(8, -(-k // 128)) and (tile >= min(m, 64) or m > 64)


def test_plans_refused():
    for sms, error in ((0, sdt.SdtError), (65537, sdt.SdtError), (2 ** 31, ValueError), (1.5, TypeError)):
        with pytest.raises(error):
            sdt.gemm_fp8_plan(64, 128, 128, sms)
