"""Cases of the operators of a layer in 8 bits: what is measured, over which sizes.

A layer of a serving program calls, around the paged cache and its attention,

  rms_norm_fp8   the residual's addition, the norm, and its output in fp8 with a scale per 128;
  gemm_fp8       the projections: fp8 activations (a scale per token and 128) times fp8 weights
                 (a scale per 128 x 128);
  rope_qk        rotary positions of the new queries and keys, before the keys are appended;
  quant_fp8      fp8 of the attention's output, and of act(gate) * up between the feed-forward
                 block's two products.

``run`` computes each in plain torch operations in 32 bits (``own`` false) or with the
library's operators (``own`` true).  Sizes are generic serving shapes, and those of this
repository's benchmark (K = 4096, N = 12288 decode; the 4096 cube).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BLOCK = 128  # values per scale
E4M3_MAX = 448.0
TINY = 2.0 ** -100  # a block's scale is that of this largest value at least
LARGEST_GEMM = 2 * 8192 * 28672 * 8192  # flops of a drawn product
LARGEST_ROWS = 8192 * 14336  # values of a drawn norm, quantisation or rotation


def _gemm(name, **kw):
    case = dict(name=name, op="gemm", m=1, n=4096, k=4096, a="e4m3", out="bf16", scales="row")
    case.update(kw)
    return case


def _norm(name, **kw):
    case = dict(name=name, op="norm", tokens=1, width=4096, dtype="bf16", residual=True, also=False)
    case.update(kw)
    return case


def _quant(name, **kw):
    case = dict(name=name, op="quant", tokens=1, width=4096, dtype="bf16", gate="none")
    case.update(kw)
    return case


def _rope(name, **kw):
    case = dict(name=name, op="rope", tokens=1, q_heads=32, kv_heads=8, head_dim=128, rotary=128, pairs="half",
                longest=8192, scaling="none", dtype="bf16", inplace=True)
    case.update(kw)
    return case


def listed():
    return [
        # the fused projection of one new token: the weights' bytes are all there is
        _gemm("gemm-one-token", n=12288),
        # the projection back to the model's width in a decode step of a batch: few outputs, long sums
        _gemm("gemm-decode-48", m=48, n=4096, k=14336),
        # a chunk of prompts with decode tokens, ragged in every size; scales laid out block by block
        _gemm("gemm-chunk-ragged", m=333, n=5000, k=4208, out="fp16", scales="col"),
        # the benchmark's cube
        _gemm("gemm-4096-cube", m=4096, out="fp16"),
        # odd token count, wide-range activations, 32-bit results (scores, a router's logits)
        _gemm("gemm-e5m2-fp32", m=1021, n=2560, k=7168, a="e5m2", out="fp32"),
        # a long prompt through a wide feed-forward block: the largest
        _gemm("gemm-prompt-wide", m=8192, n=28672, k=8192),
        # the norm between two projections of one new token
        _norm("norm-one-token", tokens=1, width=4096),
        # a long prompt, the normalised values also in 16 bits; a last block of 64
        _norm("norm-prompt", tokens=8191, width=8128, also=True),
        # between the feed-forward products in a decode step
        _quant("quant-decode-gated", tokens=16, width=14336, gate="silu"),
        # the same in a prompt
        _quant("quant-prompt-gated", tokens=8192, width=14336, gate="gelu", dtype="fp16"),
        # a decode step of a full batch, in place in the fused projection's rows
        _rope("rope-decode", tokens=64, kv_heads=32),
        # a long context's chunk: interleaved pairs of part of each head, scaled frequencies
        _rope("rope-long-part", tokens=8191, q_heads=64, rotary=96, pairs="interleaved", longest=1048576,
              scaling="ramp", inplace=False),
    ]


def _logint(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "norm", "quant", "rope"])
    if op == "gemm":
        n, k = _logint(rng, 128, 28672, 8), _logint(rng, 128, 16384, rng.choice([16, 128]))
        m = _logint(rng, 1, min(8192, LARGEST_GEMM // (2 * n * k)))
        return dict(op="gemm", m=m, n=n, k=k, a=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    out=rng.choice(["bf16", "bf16", "fp16", "fp32"]), scales=rng.choice(["row", "col"]))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        head_dim = rng.choice([64, 80, 96, 128, 128, 256])
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
        kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16, 32])
        q_heads = kv_heads * rng.choice([g for g in (1, 2, 4, 5, 7, 8, 16) if kv_heads * g <= 128])
        tokens = _logint(rng, 1, min(16384, LARGEST_ROWS // ((q_heads + kv_heads) * head_dim)))
        return dict(op="rope", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, rotary=rotary,
                    pairs=rng.choice(["half", "half", "interleaved"]), longest=_logint(rng, 64, 1048576),
                    scaling=rng.choice(["none", "linear", "base", "ramp", "smooth"]), dtype=dtype,
                    inplace=rng.choice([True, False]))
    width = _logint(rng, 64, 16384, 8)
    tokens = _logint(rng, 1, min(16384, LARGEST_ROWS // width))
    if op == "norm":
        return dict(op="norm", tokens=tokens, width=width, dtype=dtype, residual=rng.choice([True, True, False]),
                    also=rng.choice([True, False, False]))
    return dict(op="quant", tokens=tokens, width=width, dtype=dtype, gate=rng.choice(["none", "silu", "gelu"]))


def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        return {"bytes": m * k + n * k + 4 * kb * (m + nb) + m * n * (4 if case["out"] == "fp32" else 2),
                "flops": 2.0 * m * n * k}
    if case["op"] == "rope":
        rows = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        # in place the rest of each head is not touched
        width = case["rotary"] if case["inplace"] else case["head_dim"]
        return {"bytes": rows * width * 4 + 8 * case["tokens"], "flops": 3.0 * rows * case["rotary"]}
    t, d = case["tokens"], case["width"]
    out = t * d + 4 * t * -(-d // BLOCK)
    if case["op"] == "norm":
        return {"bytes": out + 2 * t * d * (1 + 2 * case["residual"] + case["also"]) + 2 * d, "flops": 8.0 * t * d}
    return {"bytes": out + 2 * t * d * (1 if case["gate"] == "none" else 2), "flops": 4.0 * t * d}


# ---- inputs -------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _fp8(shape, g, name):
    """What quantised normal values look like: the largest of 128 near the type's largest."""
    top = 448.0 if name == "e4m3" else 57344.0
    return (torch.randn(shape, generator=g, device="cuda") * (top / 3.0)).clamp_(-top, top).to(DTYPES[name])


def _uniform(shape, g, lo, hi):
    return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g)


SCALING = {  # what a program that was trained on 4096 positions asks for
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, factor=8.0),
    "base": dict(base=10000.0, factor=8.0),
    "ramp": dict(base=10000.0, factor=40.0, original_length=4096, low=1.0, high=32.0),
    "smooth": dict(base=500000.0, factor=8.0, original_length=8192, low=1.0, high=4.0),
}


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case, op=case["op"])
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        s["a"], s["w"] = _fp8((m, k), g, case["a"]), _fp8((n, k), g, "e4m3")
        top = 448.0 if case["a"] == "e4m3" else 57344.0
        if case["scales"] == "row":
            s["a_scales"] = _uniform((m, kb), g, 2.0 / top, 5.0 / top)
        else:
            s["a_scales"] = _uniform((kb, m), g, 2.0 / top, 5.0 / top).t()
        s["w_scales"] = _uniform((nb, kb), g, 0.05 / 448, 0.2 / 448)
        return s
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "rope":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        # queries and keys as they leave the fused projection: slices of its rows
        rows = _randn((t, (hq + 2 * hk) * d), g, dtype)
        s["q"] = rows[:, : hq * d].unflatten(1, (hq, d))
        s["k"] = rows[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["positions"] = torch.randint(0, case["longest"], (t,), generator=g, device="cuda")
        freq, s["magnitude"] = _frequencies(case)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        if own:  # the frequencies' handle, which a program keeps with its model
            import shape_driven_tile_gb300 as sdt

            s["table"] = sdt.RopeTable(case["rotary"], interleaved=case["pairs"] == "interleaved",
                                       scaling=case["scaling"], **SCALING[case["scaling"]])
        return s
    t, d = case["tokens"], case["width"]
    if case["op"] == "norm":
        s["x"], s["weight"] = _randn((t, d), g, dtype), (1.0 + 0.2 * _randn((d,), g)).to(dtype)
        s["eps"] = 1e-5
        if case["residual"]:
            s["residual"] = (4.0 * _randn((t, d), g)).to(dtype)
        return s
    if case["gate"] == "none":
        s["x"] = _randn((t, d), g, dtype)
    else:  # both projections' outputs side by side, as one product writes them
        rows = _randn((t, 2 * d), g, dtype)
        s["gate"], s["x"] = rows[:, :d], rows[:, d:]
    return s


def _frequencies(case):
    """Radians per position of each rotated pair, and the factor on the rotated values."""
    r, how, p = case["rotary"], case["scaling"], SCALING[case["scaling"]]
    i = np.arange(0, r, 2, dtype=np.float64)
    factor = p.get("factor", 1.0)
    base = p["base"] * factor ** (r / (r - 2)) if how == "base" else p["base"]
    freq = base ** (-i / r)
    if how == "linear":
        freq = freq / factor
    if how in ("ramp", "smooth"):
        rotations = p["original_length"] * freq / (2 * math.pi)
        if how == "smooth":  # kept above `high` rotations over the original length, divided below `low`
            keep = np.clip((rotations - p["low"]) / (p["high"] - p["low"]), 0.0, 1.0)
        else:  # the same ends, blended over the pairs between them
            at = [r * math.log(p["original_length"] / (n * 2 * math.pi)) / (2 * math.log(p["base"]))
                  for n in (p["high"], p["low"])]
            first, last = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
            keep = 1.0 - np.clip((i / 2 - first) / max(last - first, 1e-3), 0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
    return freq, 0.1 * math.log(factor) + 1.0 if how == "ramp" else 1.0


# ---- the operators ------------------------------------------------------------------------


def _run_own(s):
    import shape_driven_tile_gb300 as sdt

    if s["op"] == "gemm":
        return sdt.gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], out_dtype=DTYPES[s["case"]["out"]])
    if s["op"] == "norm":
        also = torch.empty_like(s["x"]) if s["case"]["also"] else None
        q, scales = sdt.rms_norm_fp8(s["x"], s["weight"], s.get("residual"), eps=s["eps"], out=also)
        return dict(q=q, scales=scales, out=also, residual=s.get("residual"))
    if s["op"] == "quant":
        q, scales = sdt.quant_fp8(s["x"], s.get("gate"), activation=s["case"]["gate"] if "gate" in s else "silu")
        return dict(q=q, scales=scales)
    if s["case"]["inplace"]:
        return sdt.rope_qk(s["q"], s["k"], s["positions"], s["table"], q_out=s["q"], k_out=s["k"])
    return sdt.rope_qk(s["q"], s["k"], s["positions"], s["table"])


def _plain_gemm(s):
    def numbers(x, scales, rows):
        scales = scales.repeat_interleave(rows, 0)[: x.shape[0]] if rows > 1 else scales
        return x.float() * scales.repeat_interleave(BLOCK, 1)[:, : x.shape[1]]

    a, w = numbers(s["a"], s["a_scales"], 1), numbers(s["w"], s["w_scales"], BLOCK)
    return torch.matmul(a, w.t()).to(DTYPES[s["case"]["out"]])


def _plain_quantised(y):
    t, d = y.shape
    blocks = torch.nn.functional.pad(y, (0, -d % BLOCK)).unflatten(1, (-1, BLOCK))
    top = blocks.abs().amax(2).clamp(min=TINY)
    q = (blocks * (E4M3_MAX / top).unsqueeze(2)).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :d]
    return q.to(torch.float8_e4m3fn).contiguous(), top * (1.0 / E4M3_MAX)


def _plain_norm(s):
    x = s["x"]
    if "residual" in s:
        s["residual"].copy_(x.float() + s["residual"].float())
        x = s["residual"]
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    q, scales = _plain_quantised(y)
    return dict(q=q, scales=scales, out=y.to(s["x"].dtype) if s["case"]["also"] else None, residual=s.get("residual"))


def _plain_quant(s):
    y = s["x"].float()
    if "gate" in s:
        g = s["gate"].float()
        if s["case"]["gate"] == "silu":
            y = y * (g / (1.0 + torch.exp(-g)))
        else:
            y = y * (0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))))
    q, scales = _plain_quantised(y)
    return dict(q=q, scales=scales)


def _plain_rope(s):
    case = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"][None]  # far positions: 64 bits
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    r = case["rotary"]
    first = slice(0, r, 2) if case["pairs"] == "interleaved" else slice(0, r // 2)
    second = slice(1, r, 2) if case["pairs"] == "interleaved" else slice(r // 2, r)

    def turned(x):
        a, b = x[..., first].float(), x[..., second].float()
        to = x if case["inplace"] else x.clone(memory_format=torch.contiguous_format)
        to[..., first], to[..., second] = (a * cos - b * sin).to(x.dtype), (b * cos + a * sin).to(x.dtype)
        return to

    return turned(s["q"]), turned(s["k"])


def run(state):
    if own:
        return _run_own(state)
    return {"gemm": _plain_gemm, "norm": _plain_norm, "quant": _plain_quant, "rope": _plain_rope}[state["op"]](state)


# ---- the definition in 64 bits ------------------------------------------------------------


def _on_grid(v):
    """The nearest e4m3 numbers (ties to even) of values of at most 448."""
    step = torch.exp2(torch.frexp(v)[1].double().sub(1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _blocks(y):
    """(q, scales) of rows of 64-bit values."""
    q, scales = torch.empty_like(y), []
    for lo in range(0, y.shape[1], BLOCK):
        part = y[:, lo:lo + BLOCK]
        scale = part.abs().max(1).values.clamp(min=TINY) / E4M3_MAX
        q[:, lo:lo + BLOCK] = _on_grid(part / scale[:, None])
        scales.append(scale)
    return q, torch.stack(scales, 1)


def _in_rows(f, rows, *tensors):
    """f over a few rows at a time, its outputs joined."""
    parts = [f(*(None if t is None else t[lo:lo + rows] for t in tensors))
             for lo in range(0, tensors[0].shape[0], rows)]
    return [None if p[0] is None else torch.cat(p) for p in zip(*parts)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        out = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for j in range(s["a_scales"].shape[1]):
            part = slice(j * BLOCK, (j + 1) * BLOCK)
            w = s["w"][:, part].double()
            for i in range(s["w_scales"].shape[0]):
                w[i * BLOCK:(i + 1) * BLOCK] *= s["w_scales"][i, j].double()
            out.addmm_(s["a"][:, part].double() * s["a_scales"][:, j, None].double(), w.T)
        return out
    if case["op"] == "norm":
        w = s["weight"].double()

        def normed(x, r):
            held = None if r is None else (x.double() + r.double()).to(x.dtype)
            v = (x if r is None else held).double()
            y = w * v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + s["eps"])
            return *_blocks(y), y if case["also"] else None, None if held is None else held.double()

        q, scales, out, held = _in_rows(normed, 2048, s["x"], s.get("residual"))
        return dict(q=q, scales=scales, out=out, residual=held)
    if case["op"] == "quant":

        def gated(x, g):
            y = x.double()
            if g is not None:
                g = g.double()
                if case["gate"] == "silu":
                    y = y * g * torch.sigmoid(g)
                else:
                    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
                    y = y * g * torch.sigmoid(2 * inner)
            return _blocks(y)

        q, scales = _in_rows(gated, 2048, s["x"], s.get("gate"))
        return dict(q=q, scales=scales)
    freq, magnitude = _frequencies(case)
    half = case["rotary"] // 2
    outs = []
    for x in (s["q"], s["k"]):
        y = x.double()
        for j in range(half):
            angle = s["positions"].double() * float(freq[j])
            turn = torch.polar(torch.full_like(angle, magnitude), angle)[:, None]
            at = (2 * j, 2 * j + 1) if case["pairs"] == "interleaved" else (j, j + half)
            z = torch.complex(x[..., at[0]].double(), x[..., at[1]].double()) * turn
            y[..., at[0]], y[..., at[1]] = z.real, z.imag
        outs.append(y)
    return tuple(outs)
