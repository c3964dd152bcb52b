"""What is measured of the operators around the decay linear attention: the attention itself (packed and
dense prompts, single tokens, gradients), the rotary positions of its q and k, and the root-mean-square
norm with the residual's addition ahead of its projections (16-bit, 8-bit and backward forms).

``run`` computes each operator in its plain form (``own`` false: elementary torch operations in 32 bits)
or with the framework's calls (``own`` true); ``exact`` computes it from its definition in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def _lengths(case):
    """Document lengths of a packed case: the listed text, or equal ones of a dense batch."""
    if "docs" in case:
        return [int(x) for x in case["docs"].split(",")]
    return [case["T"]] * case["B"]


def listed():
    return [
        # the long packed prompt of the framework's own prefill benchmark: four documents with states
        {"name": "attn_prompt_32k", "op": "prompt", "docs": "16749,4229,8077,3713", "H": 16, "Hk": 16, "d": 128,
         "dtype": "bf16", "decay": "retention"},
        # a server's mixed batch: a few dozen short and ragged prompts, one of them empty, shared k and v heads
        {"name": "attn_prompts_ragged", "op": "prompt",
         "docs": "1,63,64,65,0,511,17,1023,130,2,777,300,1,96,45,640,333,1200,28,5,250,700,191,7", "H": 16, "Hk": 4,
         "d": 64, "dtype": "bf16", "decay": "slopes"},
        # the smallest prompt of the framework's parity configuration, in fp32
        {"name": "attn_prompt_256_fp32", "op": "dense", "B": 1, "T": 256, "H": 2, "Hk": 2, "d": 64, "dtype": "fp32",
         "decay": "retention"},
        # one training step's gradients at the framework's training shape
        {"name": "attn_backward_train", "op": "backward", "B": 8, "T": 4096, "H": 32, "Hk": 32, "d": 128,
         "dtype": "bf16", "decay": "retention"},
        # gradients of a short odd batch in fp32 with shared k and v heads (a fine-tuning check)
        {"name": "attn_backward_odd_fp32", "op": "backward", "B": 2, "T": 1001, "H": 4, "Hk": 2, "d": 64,
         "dtype": "fp32", "decay": "slopes"},
        # the framework's decode workload: one token of 256 sequences
        {"name": "attn_decode_256", "op": "decode", "N": 256, "H": 16, "Hk": 16, "d": 128, "dtype": "bf16",
         "decay": "retention"},
        # one token of three sequences: latency
        {"name": "attn_decode_3", "op": "decode", "N": 3, "H": 8, "Hk": 2, "d": 128, "dtype": "bf16",
         "decay": "slopes"},
        # a long prompt's q and k inside the fused projection, whole heads, half layout, positions of a context
        # stretched four times to a million tokens
        {"name": "rotary_prompt_32k", "op": "rotary", "T": 32768, "Hq": 16, "Hk": 2, "d": 128, "r": 128,
         "interleaved": False, "inverse": False, "stretch": 4.0, "first": 1000000, "dtype": "bf16"},
        # decode rows: a quarter of each head, interleaved pairs, scattered positions, fp32
        {"name": "rotary_decode_256", "op": "rotary", "T": 256, "Hq": 24, "Hk": 2, "d": 256, "r": 64,
         "interleaved": True, "inverse": False, "stretch": 1.0, "first": -1, "dtype": "fp32"},
        # the norm ahead of a layer's projections for a long prompt, and its gradients
        {"name": "norm_prompt_32k", "op": "norm", "rows": 32768, "C": 2048, "dtype": "bf16", "out": "same"},
        # the same norm ahead of an 8-bit product, a scale for each 128 columns
        {"name": "norm_fp8_8k", "op": "norm", "rows": 8191, "C": 5120, "dtype": "bf16", "out": "fp8_128"},
        {"name": "norm_backward_16k", "op": "norm_backward", "rows": 16384, "C": 4096, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "dense", "backward", "decode", "rotary", "norm", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    decay = rng.choice(["retention", "slopes", "mixed"])
    d = rng.choice([64, 128])
    if op in ("prompt", "dense", "backward", "decode"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4]) if Hk <= 8 else Hk
        base = {"H": H, "Hk": Hk, "d": d, "dtype": dtype, "decay": decay}
        if op == "decode":
            return {"op": op, "N": _log_int(rng, 1, 4096 // H), **base}
        most = 16384 * 16 if op != "backward" else 8192 * 16
        if dtype == "fp32":
            most //= 4
        T = _log_int(rng, 1, most // H)
        if op == "prompt":
            n = rng.randint(1, 24)
            cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [T])]
            return {"op": op, "docs": ",".join(str(x) for x in lens), **base}
        B = rng.randint(1, 4)
        return {"op": op, "B": B, "T": max(1, T // B), **base}
    if op == "rotary":
        hd = rng.choice([64, 80, 96, 128, 256])
        r = rng.choice([hd, hd, hd // 2, hd // 4])
        Hq = rng.choice([1, 4, 8, 16, 24, 32])
        return {"op": op, "T": _log_int(rng, 1, 32768 * 16 * 128 // (Hq * hd)), "Hq": Hq, "Hk": rng.choice([1, 2, 4, 8]),
                "d": hd, "r": r, "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.3,
                "stretch": rng.choice([1.0, 4.0, 8.0]), "first": rng.choice([-1, 0, rng.randint(1, 1000000)]),
                "dtype": dtype}
    C = rng.choice([_log_int(rng, 1, 2048) * 8, 256, 1024, 2048, 4096, 5120, 8192])
    out = rng.choice(["same", "fp8_row", "fp8_128"])
    if out == "fp8_128":
        C = max(128, C // 128 * 128)
    rows = _log_int(rng, 1, 32768 * 2048 // C)
    case = {"op": op, "rows": rows, "C": C, "dtype": dtype}
    return {**case, "out": out} if op == "norm" else case


# ------------------------------------------------------------------------------------------ inputs
def _decay(kind, H):
    """Logarithms of the heads' decays: 1 - 2^-5 .. 1 - 2^-12 (retention), e^-(2^-8/H .. 2^-8) (slopes), or
    from forgetting within a few tokens to not forgetting at all (mixed)."""
    h = torch.arange(H, dtype=torch.float64)
    if kind == "slopes":
        g = -torch.exp2(-8.0 * (h + 1) / H)
    elif kind == "retention":
        g = torch.log1p(-torch.exp2(-5.0 - 7.0 * h / max(1, H - 1)))
    else:
        g = -torch.exp2(2.0 - 3.0 * h)
        g[-1] = 0.0
    return g.to(torch.float32)


def _inv_freq(r, stretch):
    """Angular frequencies 10^(-7 i / (r / 2)); stretched contexts divide the slow ones by `stretch` and leave
    the fast ones, with a linear ramp between (32 and 1 turns in 262144 positions)."""
    i = torch.arange(r // 2, dtype=torch.float64)
    f = 1e7 ** (-2.0 * i / r)
    if stretch > 1:
        turns = 262144 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / stretch * (1 - keep)
    return f.to(torch.float32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def rand(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op in ("prompt", "dense", "backward", "decode"):
        H, Hk, d = case["H"], case["Hk"], case["d"]
        s["log_decay"] = _decay(case["decay"], H).cuda()
        s["scale"] = d ** -0.5
        if op == "decode":
            N = case["N"]
            s.update(q=rand(N, H, d), k=rand(N, Hk, d), v=rand(N, Hk, d),
                     state=rand(N, H, d, d, dtype=torch.float32, std=0.5))
            return s
        lens = _lengths(case)
        lead = (1, sum(lens)) if op == "prompt" else (case["B"], case["T"])
        s.update(q=rand(*lead, H, d), k=rand(*lead, Hk, d), v=rand(*lead, Hk, d),
                 s0=rand(len(lens), H, d, d, dtype=torch.float32, std=0.5), ws={})
        s["lengths"] = lens
        if op == "prompt":
            ends = torch.tensor([0] + lens).cumsum(0)
            s["cu_seqlens"] = ends.to(torch.int32).cuda()
        if op == "backward":
            s.update(dy=rand(*lead, H, d), ds_final=rand(len(lens), H, d, d, dtype=torch.float32, std=0.1))
    elif op == "rotary":
        T, Hq, Hk, d = case["T"], case["Hq"], case["Hk"], case["d"]
        qkv = rand(T, (Hq + 2 * Hk) * d)
        s["q"] = qkv[:, : Hq * d].view(T, Hq, d)
        s["k"] = qkv[:, Hq * d: (Hq + Hk) * d].view(T, Hk, d)
        s["inv_freq"] = _inv_freq(case["r"], case["stretch"]).cuda()
        s["scale"] = 0.1 * math.log(case["stretch"]) + 1.0
        if case["first"] < 0:
            s["positions"] = torch.randint(0, 262144, (T,), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["positions"] = torch.arange(T, device="cuda", dtype=torch.int32) + case["first"]
    elif op == "norm":
        rows, C = case["rows"], case["C"]
        s.update(x=rand(rows, C), residual=rand(rows, C, std=3.0), w=rand(C, dtype=torch.float32, std=0.2))
    else:
        rows, C = case["rows"], case["C"]
        s.update(h=rand(rows, C, std=3.0), w=rand(C, dtype=torch.float32, std=0.2), d_o=rand(rows, C),
                 d_h=rand(rows, C), ws={})
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _cut(s):
    """Documents cut into chunks of CHUNK tokens from their own starts: every token's row (T past the end),
    and the chunks' documents, places and lengths."""
    lens = s["lengths"]
    n = torch.tensor(lens, device="cuda")
    per = (n + CHUNK - 1) // CHUNK
    total = sum((x + CHUNK - 1) // CHUNK for x in lens)
    doc = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), per, output_size=total)
    place = torch.arange(total, device="cuda") - (per.cumsum(0) - per)[doc]
    count = (n[doc] - place * CHUNK).clamp(max=CHUNK)
    at = torch.arange(CHUNK, device="cuda")
    row = ((n.cumsum(0) - n)[doc] + place * CHUNK)[:, None] + at
    row = torch.where(at < count[:, None], row, sum(lens))
    return row, doc, place, count, n


def _chunks(x, row, H):
    """[.., T, h, d] -> [H, chunks, CHUNK, d] in fp32, zero rows past a document's end."""
    x = x.reshape(-1, *x.shape[-2:]).float()
    x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[row]
    return x.permute(2, 0, 1, 3).repeat_interleave(H // x.shape[2], 0)


def _tokens(x, row, like):
    """Back from chunks to tokens; shared heads' parts are summed."""
    h = like.shape[-2]
    x = x.reshape(h, -1, *x.shape[1:]).sum(1).permute(1, 2, 0, 3)
    y = x.new_empty(like.numel() // (h * x.shape[-1]) + 1, h, x.shape[-1])
    y[row] = x
    return y[:-1].reshape(like.shape).to(like.dtype)


def _power(g, n):
    """e^(g n) where n >= 0, else 0: [H, *n.shape] in fp32 (exponents in 64 bits)."""
    e = g.double().view(-1, *[1] * n.dim()) * n.clamp(min=0).double()
    return torch.where(n >= 0, torch.exp(e), 0.0).float()


def _spread(weights, states):
    """sum over chunks: [H, a, b] weights, [H, b, d, d] states."""
    return (weights @ states.flatten(2)).unflatten(2, states.shape[2:])


def _attention(s, backward):
    H, g, scale = s["q"].shape[-2], s["log_decay"], s["scale"]
    row, doc, place, count, n = _cut(s)
    q, k, v = (_chunks(s[x], row, H) for x in "qkv")
    at = torch.arange(CHUNK, device="cuda")
    inside = _power(g, at[:, None] - at)[:, None]                       # e^(g (i - j)), i >= j
    to_end = _power(g, count[:, None] - 1 - at)[..., None]              # from a token to its chunk's end
    same = doc[:, None] == doc
    gap = (place[:, None] - place - 1) * CHUNK                          # from chunk c' end to chunk c start
    link = _power(g, torch.where(same, gap, -1))
    s0 = s["s0"].transpose(0, 1)
    start = place * CHUNK
    local = (k * to_end).transpose(-1, -2) @ v
    first = _spread(link, local) + _power(g, start)[..., None, None] * s0[:, doc]
    into = _power(g, at + 1)[:, None, :, None]                          # from a chunk's start to a token
    ends = start + count
    is_doc = torch.arange(len(s["lengths"]), device="cuda")[:, None] == doc
    if not backward:
        y = scale * (((q @ k.transpose(-1, -2)) * inside) @ v + into * (q @ first))
        last = _spread(_power(g, torch.where(is_doc, n[:, None] - ends, -1)), local)
        last = last + _power(g, n)[..., None, None] * s0
        return [_tokens(y, row, s["q"]), last.transpose(0, 1).contiguous()]
    dy = _chunks(s["dy"], row, H)
    dsf = s["ds_final"].transpose(0, 1)
    p = scale * (q @ k.transpose(-1, -2)) * inside
    dp = scale * (dy @ v.transpose(-1, -2)) * inside
    rlocal = scale * (q * into).transpose(-1, -2) @ dy
    rend = _spread(link.transpose(-1, -2), rlocal) + _power(g, n[doc] - ends)[..., None, None] * dsf[:, doc]
    dq = dp @ k + scale * into * (dy @ first.transpose(-1, -2))
    dk = dp.transpose(-1, -2) @ q + to_end * (v @ rend.transpose(-1, -2))
    dv = p.transpose(-1, -2) @ dy + to_end * (k @ rend)
    ds0 = _spread(_power(g, torch.where(is_doc, start, -1)), rlocal) + _power(g, n)[..., None, None] * dsf
    return [_tokens(dq, row, s["q"]), _tokens(dk, row, s["k"]), _tokens(dv, row, s["v"]),
            ds0.transpose(0, 1).contiguous()]


def _decode(s):
    H = s["q"].shape[1]
    q, k, v = (s[x].float().repeat_interleave(H // s[x].shape[1], 1) for x in "qkv")
    state = s["state"]
    state.mul_(torch.exp(s["log_decay"])[:, None, None]).add_(k[..., :, None] * v[..., None, :])
    y = s["scale"] * (state * q[..., :, None]).sum(-2)
    return [y.to(s["q"].dtype), state]


def _turn(x, pos, f, interleaved, inverse, scale):
    r = 2 * f.numel()
    ang = pos.double()[:, None] * f.double()
    c, t = (scale * torch.cos(ang)).float()[:, None], (scale * torch.sin(ang)).float()[:, None]
    t = -t if inverse else t
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., : r // 2], y[..., r // 2: r])
    u, w = a * c - b * t, b * c + a * t
    u = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([u, y[..., r:]], -1).to(x.dtype)


def _norm(s, out):
    dt = s["x"].dtype
    h = s["x"].float() + s["residual"].float()
    o = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * (1 + s["w"])
    if out == "same":
        return [o.to(dt), h.to(dt)]
    groups = o.unflatten(-1, (-1, 128 if out == "fp8_128" else o.shape[-1]))
    scales = groups.abs().amax(-1) / 448.0
    q = groups / torch.where(scales > 0, scales, 1.0)[..., None]
    return [q.clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn), scales, h.to(dt)]


def _norm_backward(s):
    h, do, gain = s["h"].float(), s["d_o"].float(), 1 + s["w"]
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    nrm, dn = h * r, do * gain
    dx = r * (dn - nrm * (dn * nrm).mean(-1, keepdim=True)) + s["d_h"].float()
    return [dx.to(s["h"].dtype), (do * nrm).sum(0)]


# ------------------------------------------------------------------------------------------ run
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op in ("prompt", "dense", "backward"):
        return _attention(s, op == "backward")
    if op == "decode":
        return _decode(s)
    if op == "rotary":
        a = (s["positions"], s["inv_freq"], case["interleaved"], case["inverse"], s["scale"])
        return [_turn(s["q"], *a), _turn(s["k"], *a)]
    return _norm(s, case["out"]) if op == "norm" else _norm_backward(s)


def _own(s, case, op):
    """The calls of the framework's user: workspaces are allocated once and kept."""
    from gated_deltanet_linear_eqs_b200 import api

    if op in ("prompt", "dense", "backward") and "t" not in s["ws"]:
        B, T = s["q"].shape[:2]
        H, d = case["H"], case["d"]
        size = api.gdn_linear_attn_workspace_bytes(B, T, H, case["Hk"], d, d, backward=op == "backward",
                                                   num_seqs=len(s["lengths"]) if op == "prompt" else 0)
        s["ws"]["t"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    if op == "prompt":
        return list(api.gdn_linear_attn_varlen(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"], s0=s["s0"],
                                               scale=s["scale"], ws=s["ws"]["t"]))
    if op == "dense":
        return list(api.gdn_linear_attn(s["q"], s["k"], s["v"], s["log_decay"], s0=s["s0"], scale=s["scale"],
                                        ws=s["ws"]["t"]))
    if op == "backward":
        o = api.gdn_linear_attn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["dy"], s0=s["s0"],
                                         ds_final=s["ds_final"], scale=s["scale"], ws=s["ws"]["t"])
        return [o["dq"], o["dk"], o["dv"], o["ds0"]]
    if op == "decode":
        y = api.gdn_linear_attn_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"])
        return [y, s["state"]]
    if op == "rotary":
        return list(api.gdn_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=case["interleaved"],
                                   inverse=case["inverse"], scale=s["scale"]))
    if op == "norm":
        if case["out"] == "same":
            return list(api.gdn_add_rmsnorm(s["x"], s["residual"], s["w"], eps=EPS))
        return list(api.gdn_add_rmsnorm_fp8(s["x"], s["residual"], s["w"], eps=EPS,
                                            group=128 if case["out"] == "fp8_128" else 0))
    if "t" not in s["ws"]:
        size = api.gdn_workspace_bytes(api._abi.GDN_OP_ADD_RMSNORM_BACKWARD, 1, case["rows"], 1, case["C"], case["C"])
        s["ws"]["t"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    o = api.gdn_add_rmsnorm_backward(s["h"], s["w"], s["d_o"], d_h=s["d_h"], eps=EPS, ws=s["ws"]["t"])
    return [o["dx"], o["dw"]]


# ------------------------------------------------------------------------------------------ work
def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("prompt", "dense", "backward", "decode"):
        H, Hk, d = case["H"], case["Hk"], case["d"]
        if op == "decode":
            N = case["N"]
            return {"bytes": N * (e * d * (2 * H + 2 * Hk) + 8 * H * d * d) + 4 * H, "flops": 5.0 * N * H * d * d}
        lens = _lengths(case)
        T, n = sum(lens), len(lens)
        # products of a 64-token chunked form: two masked d x 64 rows and two d x d ones a token and head
        one = T * H * (2 * 2 * d * CHUNK / 2 + 2 * 2 * d * d)
        if op == "backward":
            return {"bytes": e * T * d * (2 * H + 2 * Hk + H + 2 * Hk) + 3 * 4 * n * H * d * d,
                    "flops": T * H * (5 * 2 * d * CHUNK / 2 + 5 * 2 * d * d)}
        return {"bytes": e * T * d * (2 * H + 2 * Hk) + 2 * 4 * n * H * d * d, "flops": one}
    if op == "rotary":
        x = case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
        return {"bytes": 2 * e * x + 4 * case["T"] + 2 * case["r"], "flops": 3 * x}
    x = case["rows"] * case["C"]
    if op == "norm_backward":
        return {"bytes": 4 * e * x + 8 * case["C"], "flops": 10 * x}
    if case["out"] == "same":
        return {"bytes": 4 * e * x + 4 * case["C"], "flops": 6 * x}
    per = 128 if case["out"] == "fp8_128" else case["C"]
    return {"bytes": (3 * e + 1) * x + 4 * x // per + 4 * case["C"], "flops": 8 * x}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prompt", "dense", "backward"):
        return _exact_attention(s, case, op)
    if op == "decode":
        H = case["H"]
        q, k, v = (s[x].double().repeat_interleave(H // s[x].shape[1], 1) for x in "qkv")
        S = s["state"].double() * torch.exp(s["log_decay"].double())[:, None, None]
        S = S + torch.einsum("nhk,nhv->nhkv", k, v)
        return [s["scale"] * torch.einsum("nhkv,nhk->nhv", S, q), S]
    if op == "rotary":
        out = []
        for x in (s["q"].double(), s["k"].double()):
            r = case["r"]
            ang = torch.outer(s["positions"].double(), s["inv_freq"].double())
            z = s["scale"] * torch.polar(torch.ones_like(ang), -ang if case["inverse"] else ang)
            if case["interleaved"]:
                p = torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous())
                p = torch.view_as_real(p * z[:, None]).flatten(-2)
            else:
                p = torch.complex(x[..., : r // 2].contiguous(), x[..., r // 2: r].contiguous()) * z[:, None]
                p = torch.cat([p.real, p.imag], -1)
            out.append(torch.cat([p, x[..., r:]], -1))
        return out
    if op == "norm":
        h = s["x"].double() + s["residual"].double()
        o = h * (h.square().mean(-1, True) + EPS).rsqrt()
        o = o + o * s["w"].double()
        if case["out"] == "same":
            return [o, h]
        per = 128 if case["out"] == "fp8_128" else case["C"]
        top = o.reshape(case["rows"], -1, per).abs().max(-1).values
        return [_e4m3(o.reshape(case["rows"], -1, per) * 448 / top[..., None].clamp(min=1e-300)).reshape(o.shape),
                top / 448, h]
    h, do, w = s["h"].double(), s["d_o"].double(), s["w"].double()
    m = h.square().mean(-1, True) + EPS
    t = do * (1 + w)
    dx = t * m.rsqrt() - h * m.pow(-1.5) * (t * h).mean(-1, True) + s["d_h"].double()
    return [dx, torch.einsum("rc,rc->c", do, h * m.rsqrt())]


def _e4m3(x):
    """The nearest values of 1 + 4 + 3 bits (ties to even, subnormals of 2^-9)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_attention(s, case, op):
    """Token by token: S <- e^g S + k v^T, y = scale S^T q; the gradients by the adjoint recurrence."""
    H, d = case["H"], case["d"]
    lens = _lengths(case)
    top, n = max(lens), len(lens)
    if top * n * H * d * 8 * (8 if op == "backward" else 4) > 60e9:
        return None
    first = [sum(lens[:i]) for i in range(n)]

    def rows(x):
        """[n, top, H, d], zero past a document's end"""
        x = x.reshape(-1, *x.shape[-2:]).double()
        x = x.repeat_interleave(H // x.shape[1], 1)
        y = x.new_zeros(top, n, H, d)
        for i in range(n):
            y[: lens[i], i] = x[first[i]: first[i] + lens[i]]
        return y

    def packed(y, like):
        x = torch.cat([y[: lens[i], i] for i in range(n)])
        h = like.shape[-2]
        return x.reshape(-1, h, H // h, d).sum(2).reshape(like.shape)

    q, k, v = rows(s["q"]), rows(s["k"]), rows(s["v"])
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    on = torch.arange(top, device="cuda")[:, None] < torch.tensor(lens, device="cuda")
    factor = torch.where(on[:, :, None, None, None], lam, 1.0)           # [top, n, H, 1, 1]
    scale = s["scale"]
    S = s["s0"].double()
    if op != "backward":
        y = torch.empty_like(v)
        for t in range(top):
            S = torch.addcmul(S * factor[t], k[t][..., :, None], v[t][..., None, :])
            y[t] = (q[t][..., None, :] @ S)[..., 0, :]
        return [packed(scale * y, s["q"]), S]
    dy = rows(s["dy"])
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(top):
        S = torch.addcmul(S * factor[t], k[t][..., :, None], v[t][..., None, :])
        dq[t] = scale * (S @ dy[t][..., :, None])[..., 0]
    R = s["ds_final"].double()
    for t in range(top - 1, -1, -1):
        R = torch.addcmul(R, scale * q[t][..., :, None], dy[t][..., None, :])
        dk[t] = (R @ v[t][..., :, None])[..., 0]
        dv[t] = (k[t][..., None, :] @ R)[..., 0, :]
        R = R * factor[t]
    return [packed(dq, s["q"]), packed(dk, s["k"]), packed(dv, s["v"]), R]
