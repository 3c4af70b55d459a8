"""Measured cases of the operators with which a decoder reads the encoder's output.

  linear_i8        y = epilogue((xq wq^T) sx sw + b): tokens quantised to 8-bit integers with a
                   scale each, times weights held as 8-bit integers with a scale per channel
  qk_norm_rope     RMS norm of every query and key head, then the rotation by position
  cross_attention  softmax(q k^T scale) v over the encoder's packed states, one segment of keys
                   per request, grouped key heads, an optional key mask

Each case is run in its plain form (elementary torch operations) or, with `own` set, by the calls
that a program makes of the library."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"bf16": 0, "f16": 1, "f32": 2}  # the library's element types
EPILOGUES = {"bf16": 0, "bf16_gelu": 1, "f32": 3}  # aut_linear's codes


def listed():
    return [
        # One decoder token's 2048-wide projection: a step of a single request, bound by latency.
        {"name": "i8_token", "op": "linear_i8", "M": 1, "K": 2048, "N": 2048, "x": "bf16", "y": "bf16"},
        # Keys and values of a 30 s clip (390 states, width 1024), from the encoder's fp32 output.
        {"name": "i8_clip_kv", "op": "linear_i8", "M": 390, "K": 1024, "N": 2048, "x": "f32", "y": "bf16"},
        # Keys and values of the 16-request batch (3253 states, width 2048).
        {"name": "i8_batch_kv", "op": "linear_i8", "M": 3253, "K": 2048, "N": 4096, "x": "f32", "y": "bf16"},
        # The encoder's own fc1 with GELU over a 20-minute recording (15600 tokens).
        {"name": "i8_long_fc1", "op": "linear_i8", "M": 15600, "K": 1280, "N": 5120, "x": "bf16", "y": "bf16_gelu"},
        # One decoder token: 16 query and 8 key heads of 128.
        {"name": "rope_token", "op": "qk_norm_rope", "Tq": 1, "Tk": 1, "heads_q": 16, "heads_kv": 8, "hd": 128, "rot": 128,
         "interleaved": False, "x": "bf16", "y": "bf16", "theta": 1e6, "pos0": 4000},
        # Prompts of the 16-request batch, whole-head rotation.
        {"name": "rope_batch", "op": "qk_norm_rope", "Tq": 3253, "Tk": 3253, "heads_q": 16, "heads_kv": 8, "hd": 128, "rot": 128,
         "interleaved": False, "x": "bf16", "y": "bf16", "theta": 1e6, "pos0": 0},
        # fp32 projections of a 20-minute recording, half of each head rotated in neighbouring pairs, far positions.
        {"name": "rope_long", "op": "qk_norm_rope", "Tq": 777, "Tk": 15600, "heads_q": 16, "heads_kv": 16, "hd": 64, "rot": 32,
         "interleaved": True, "x": "f32", "y": "bf16", "theta": 1e4, "pos0": 900000},
        # One token of one request on a 30 s clip's states.
        {"name": "xa_token", "op": "cross_attention", "seqs": 1, "q_min": 1, "q_max": 1, "k_min": 390, "k_max": 390, "heads_q": 16,
         "heads_kv": 16, "hd": 64, "dtype": "bf16", "mask": False, "lens": 0},
        # One token of one request on a 20-minute recording's states: the key axis has to be split.
        {"name": "xa_token_long", "op": "cross_attention", "seqs": 1, "q_min": 1, "q_max": 1, "k_min": 15600, "k_max": 15600,
         "heads_q": 16, "heads_kv": 8, "hd": 128, "dtype": "bf16", "mask": False, "lens": 0},
        # One token each of a 256-request batch of clips of half a second to a minute: bound by reading keys and values.
        {"name": "xa_step_batch", "op": "cross_attention", "seqs": 256, "q_min": 1, "q_max": 1, "k_min": 6, "k_max": 780,
         "heads_q": 16, "heads_kv": 8, "hd": 128, "dtype": "f16", "mask": False, "lens": 1},
        # Ragged prompts over ragged clips with silent stretches masked out, every query head with keys of its own.
        {"name": "xa_prompt_mask", "op": "cross_attention", "seqs": 16, "q_min": 5, "q_max": 448, "k_min": 13, "k_max": 1500,
         "heads_q": 20, "heads_kv": 20, "hd": 64, "dtype": "bf16", "mask": True, "lens": 2},
        # Long prompts over five-minute recordings: bound by the matrix products.
        {"name": "xa_prompt_long", "op": "cross_attention", "seqs": 16, "q_min": 300, "q_max": 500, "k_min": 3700, "k_max": 4000,
         "heads_q": 16, "heads_kv": 8, "hd": 128, "dtype": "bf16", "mask": False, "lens": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_i8", "qk_norm_rope", "cross_attention", "cross_attention"])
    if op == "linear_i8":
        M, K = _log(rng, 1, 15600), 16 * _log(rng, 4, 128)
        return {"op": op, "M": M, "K": K, "N": 16 * _log(rng, 4, min(256, int(9e10 / (16 * M * K)))),
                "x": rng.choice(["bf16", "f16", "f32"]), "y": rng.choice(["bf16", "bf16_gelu", "f32"])}
    heads_kv = rng.choice([1, 2, 4, 5, 8])
    heads_q = heads_kv * rng.choice([1, 2, 3, 4])
    if op == "qk_norm_rope":
        hd = rng.choice([64, 128])
        return {"op": op, "Tq": _log(rng, 1, 8000), "Tk": _log(rng, 1, 8000), "heads_q": heads_q, "heads_kv": heads_kv, "hd": hd,
                "rot": rng.choice([hd, hd // 2]), "interleaved": rng.random() < 0.5, "x": rng.choice(["bf16", "f16", "f32"]),
                "y": rng.choice(["bf16", "f16"]), "theta": rng.choice([1e4, 1e6]), "pos0": rng.choice([0, rng.randrange(1000000)])}
    case = {"op": op, "heads_q": heads_q, "heads_kv": heads_kv, "hd": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f16"]),
            "mask": rng.random() < 0.4, "lens": rng.randrange(1 << 30)}
    if rng.random() < 0.5:  # a decoding step
        case |= {"seqs": _log(rng, 1, 256), "q_min": 1, "q_max": 1}
        k_max = _log(rng, 16, min(15600, 60000 // case["seqs"]))
    else:  # prompts
        q_max = _log(rng, 2, 500)
        case |= {"seqs": _log(rng, 1, 16), "q_min": max(1, q_max // 3), "q_max": q_max}
        k_max = _log(rng, 16, min(4000, int(4e10 / (case["seqs"] * q_max * heads_q * case["hd"]))))
    return case | {"k_min": max(1, k_max // rng.choice([1, 2, 20])), "k_max": k_max}


def _lengths(case):
    """Query and key lengths of every request; uniform, and uniform in their logarithm."""
    rng = np.random.default_rng(case["lens"])
    q = rng.integers(case["q_min"], case["q_max"] + 1, size=case["seqs"])
    k = np.exp(rng.uniform(math.log(case["k_min"]), math.log(case["k_max"]), size=case["seqs"])).round().astype(np.int64)
    if case["seqs"] > 2 and case["k_max"] > 2 * case["k_min"]:
        k[1] = case["k_max"]
    return q, np.clip(k, case["k_min"], case["k_max"])


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    s = {"case": case}
    if case["op"] == "linear_i8":
        M, K, N = case["M"], case["K"], case["N"]
        # Activations whose rows differ in size and in which a few channels stand out.
        x = normal(M, K) * (0.3 + torch.rand(M, 1, generator=g, device="cuda"))
        x[:, :: max(1, K // 4)] *= 8
        s["x"] = x.to(DTYPES[case["x"]])
        w = normal(N, K) / math.sqrt(K)
        s["w_scale"] = w.abs().amax(1) / 127
        s["wq"] = (w / s["w_scale"][:, None]).round().to(torch.int8)
        s["bias"] = (normal(N) * 0.1).to(torch.bfloat16)
        s["xq"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
        s["x_scale"] = torch.empty(M, dtype=torch.float32, device="cuda")
        s["y"] = torch.empty(M, N, dtype=torch.float32 if case["y"] == "f32" else torch.bfloat16, device="cuda")
    elif case["op"] == "qk_norm_rope":
        hd, dt = case["hd"], DTYPES[case["x"]]
        for side, T, heads in (("q", case["Tq"], case["heads_q"]), ("k", case["Tk"], case["heads_kv"])):
            s[side] = normal(T, heads * hd, dtype=dt) * 2
            s[side + "_gamma"] = (1 + 0.2 * normal(hd)).to(torch.bfloat16)
            s[side + "_pos"] = torch.arange(T, dtype=torch.int32, device="cuda") + case["pos0"]
            s[side + "_out"] = torch.empty(T, heads * hd, dtype=DTYPES[case["y"]], device="cuda")
    else:
        ql, kl = _lengths(case)
        s["cu_q"], s["cu_k"] = _offsets(ql), _offsets(kl)
        s["q_lens"] = torch.from_numpy(ql).cuda()
        s["k_lens"] = torch.from_numpy(kl).cuda()
        Tq, Tk, hd, dt = int(s["cu_q"][-1]), int(s["cu_k"][-1]), case["hd"], DTYPES[case["dtype"]]
        s["q"] = normal(Tq, case["heads_q"] * hd, dtype=dt) * 1.5
        s["kv"] = normal(Tk, 2 * case["heads_kv"] * hd, dtype=dt)  # keys | values, as one projection leaves them
        s["mask"] = None
        if case["mask"]:  # silent stretches of about 20 states
            s["mask"] = (torch.rand(Tk // 20 + 1, generator=g, device="cuda") < 0.7).to(torch.uint8).repeat_interleave(20)[:Tk].contiguous()
        s["out"] = torch.empty(Tq, case["heads_q"] * hd, dtype=dt, device="cuda")
        s["ws"] = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


# ------------------------------------------------------------------ plain forms

def _plain_linear_i8(s):
    x = s["x"].float()
    scale = x.abs().amax(1) / 127
    q = (x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).round()
    y = (q @ s["wq"].float().t()) * scale[:, None] * s["w_scale"] + s["bias"].float()
    if s["case"]["y"] == "bf16_gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    return {"y": y.to(s["y"].dtype), "x_scale": scale}


def _plain_norm_rope(s, side, heads):
    c = s["case"]
    hd, half = c["hd"], c["rot"] // 2
    x = s[side].float().view(-1, heads, hd)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s[side + "_gamma"].float()
    # Angles of far positions need more than 24 bits.
    freq = torch.pow(torch.tensor(c["theta"], dtype=torch.float64, device="cuda"),
                     -torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = s[side + "_pos"].double()[:, None, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    r, rest = x[..., : c["rot"]], x[..., c["rot"]:]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], -1).flatten(-2) if c["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([r, rest], -1).reshape(-1, heads * hd).to(s[side + "_out"].dtype)


def _plain_qk_norm_rope(s):
    return {"q": _plain_norm_rope(s, "q", s["case"]["heads_q"]), "k": _plain_norm_rope(s, "k", s["case"]["heads_kv"])}


def _plain_cross_attention(s):
    c = s["case"]
    hk, g, hd = c["heads_kv"], c["heads_q"] // c["heads_kv"], c["hd"]

    def padded(t, lens, heads):  # packed rows -> [requests, longest, heads, hd], and which rows are real
        i = torch.arange(int(lens[1]), device="cuda")
        real = i < lens[0][:, None]
        at = ((lens[0].cumsum(0) - lens[0])[:, None] + i).clamp(max=t.shape[0] - 1)
        return t[at].float().view(*at.shape, heads, hd), real, at

    lens_q = (s["q_lens"], int(np.diff(s["cu_q"]).max()))
    lens_k = (s["k_lens"], int(np.diff(s["cu_k"]).max()))
    q, real_q, _ = padded(s["q"], lens_q, c["heads_q"])
    k, real_k, at = padded(s["kv"][:, : hk * hd], lens_k, hk)
    v, _, _ = padded(s["kv"][:, hk * hd:], lens_k, hk)
    seen = real_k if s["mask"] is None else real_k & (s["mask"][at] != 0)
    q = q.view(q.shape[0], q.shape[1], hk, g, hd).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, hk, g q, hd]
    p = (q @ k.permute(0, 2, 3, 1)) * (1 / math.sqrt(hd))
    p = p.masked_fill(~seen[:, None, None, :], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = (p - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, None, None], v, torch.zeros_like(v))
    o = (p @ v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(o.shape[0], hk, g, -1, hd).permute(0, 3, 1, 2, 4).flatten(2)  # [B, q, heads hd]
    return o[real_q].to(s["q"].dtype)


_plain = {"linear_i8": _plain_linear_i8, "qk_norm_rope": _plain_qk_norm_rope, "cross_attention": _plain_cross_attention}


# ------------------------------------------------------------- the library's calls

def _checked(status):
    if status != 0:
        raise RuntimeError("the library returned status %d" % status)


def _own_linear_i8(s):
    from audio_encoder_aut_b200 import _lib as A
    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    _checked(A.aut_quantize_rows(s["x"].data_ptr(), CODES[c["x"]], c["K"], c["M"], c["K"], s["xq"].data_ptr(), s["x_scale"].data_ptr(),
                                 stream))
    _checked(A.aut_linear_i8(s["xq"].data_ptr(), s["x_scale"].data_ptr(), s["wq"].data_ptr(), s["w_scale"].data_ptr(),
                             s["bias"].data_ptr(), s["y"].data_ptr(), c["M"], c["N"], c["K"], EPILOGUES[c["y"]], None, 0, 0, stream))
    return {"y": s["y"], "x_scale": s["x_scale"]}


def _own_qk_norm_rope(s):
    from audio_encoder_aut_b200 import _lib as A
    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    sides = [A.aut_head_rows(s[n].data_ptr(), heads * c["hd"], s[n + "_out"].data_ptr(), heads * c["hd"], s[n + "_gamma"].data_ptr(),
                             s[n + "_pos"].data_ptr(), T, heads)
             for n, T, heads in (("q", c["Tq"], c["heads_q"]), ("k", c["Tk"], c["heads_kv"]))]
    _checked(A.aut_qk_norm_rope(sides[0], sides[1], c["hd"], CODES[c["x"]], CODES[c["y"]], c["rot"], c["theta"], c["interleaved"], 1e-6,
                                stream))
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_cross_attention(s):
    from audio_encoder_aut_b200 import _lib as A
    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    hd, wide, kv = c["hd"], c["heads_q"] * c["hd"], s["kv"].data_ptr()
    _checked(A.aut_cross_attention(s["q"].data_ptr(), wide, kv, 2 * c["heads_kv"] * hd, kv + 2 * c["heads_kv"] * hd,
                                   2 * c["heads_kv"] * hd, s["out"].data_ptr(), wide, CODES[c["dtype"]], c["heads_q"], c["heads_kv"], hd,
                                   s["cu_q"], s["cu_k"], None if s["mask"] is None else s["mask"].data_ptr(), 1 / math.sqrt(hd),
                                   s["ws"].data_ptr(), s["ws"].numel(), None, 0, stream))
    return s["out"]


_own = {"linear_i8": _own_linear_i8, "qk_norm_rope": _own_qk_norm_rope, "cross_attention": _own_cross_attention}


# -------------------------------------------------------------------- what it takes

def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "linear_i8":
        M, K, N = case["M"], case["K"], case["N"]
        out = M * N * (4 if case["y"] == "f32" else 2)
        return {"bytes": M * K * size[case["x"]] + N * K + 4 * N + 2 * N + 4 * M + out, "flops": 2 * M * N * K}
    if case["op"] == "qk_norm_rope":
        n = (case["Tq"] * case["heads_q"] + case["Tk"] * case["heads_kv"]) * case["hd"]
        return {"bytes": n * (size[case["x"]] + size[case["y"]]) + 4 * (case["Tq"] + case["Tk"]) + 4 * case["hd"], "flops": 8 * n}
    ql, kl = _lengths(case)
    hd = case["hd"]
    return {"bytes": int(ql.sum()) * case["heads_q"] * hd * 4 + int(kl.sum()) * (case["heads_kv"] * hd * 4 + (1 if case["mask"] else 0)),
            "flops": 4 * int((ql * kl).sum()) * case["heads_q"] * hd}


# ------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear_i8":
        x = s["x"].to(torch.float64)
        peak = x.abs().max(dim=1).values
        steps = torch.round(x * (127 / peak.clamp(min=1e-300))[:, None])
        y = torch.mm(steps, (s["wq"].to(torch.float64) * s["w_scale"].to(torch.float64)[:, None]).T)
        y = torch.addcmul(s["bias"].to(torch.float64)[None], y, (peak / 127)[:, None])
        if case["y"] == "bf16_gelu":
            y = y * torch.special.ndtr(y)
        return {"y": y, "x_scale": peak / 127}
    if case["op"] == "qk_norm_rope":
        out = {}
        for n, heads in (("q", case["heads_q"]), ("k", case["heads_kv"])):
            x = s[n].to(torch.float64).reshape(-1, heads, case["hd"])
            x = x / (x.square().sum(-1, keepdim=True) / case["hd"] + 1e-6).sqrt() * s[n + "_gamma"].to(torch.float64)
            half = case["rot"] // 2
            y = x.clone()
            for i in range(half):  # one rotated pair at a time, as a complex number
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                turn = torch.polar(torch.ones_like(x[:, :1, 0]), s[n + "_pos"].to(torch.float64)[:, None] * case["theta"] ** (-i / half))
                z = torch.complex(x[..., a], x[..., b]) * turn
                y[..., a], y[..., b] = z.real, z.imag
            out[n] = y.reshape(-1, heads * case["hd"])
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    hd, hk, group = case["hd"], case["heads_kv"], case["heads_q"] // case["heads_kv"]
    for b in range(case["seqs"]):
        q0, q1, k0, k1 = (int(v) for v in (s["cu_q"][b], s["cu_q"][b + 1], s["cu_k"][b], s["cu_k"][b + 1]))
        rows = torch.arange(k0, k1, device="cuda")
        if s["mask"] is not None:
            rows = rows[s["mask"][k0:k1] != 0]
        if rows.numel() == 0:
            continue
        kv = s["kv"][rows].to(torch.float64).reshape(-1, 2, hk, hd)
        q = s["q"][q0:q1].to(torch.float64).reshape(-1, hk, group, hd)
        p = torch.softmax(torch.einsum("qhgd,khd->hgqk", q, kv[:, 0]) / math.sqrt(hd), -1)
        out[q0:q1] = torch.einsum("hgqk,khd->qhgd", p, kv[:, 1]).reshape(q1 - q0, -1)
    return out
