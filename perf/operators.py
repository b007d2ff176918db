"""What is measured of the expert and 8-bit-integer linear operators.

Three operators, each beside the plain form it is compared with:

* ``i8``: the linear layer whose weight is held in 8-bit integers with one scale
  per output channel; the call quantizes its tokens to 8-bit integers with one scale
  per token, multiplies in integers and adds the unmerged adapter branch;
* ``grouped``: the products of an expert layer: rows sorted by expert, device
  offsets, one stacked k-bit weight, one adapter per expert;
* ``grouped_bwd``: the gradients of ``grouped`` (input, A and B).

A case is a dict of sizes; ``prepare`` makes its inputs on the GPU from a seed.
"""
import math
import statistics

import numpy as np
import torch

own = False

BLOCK, GROUP = 64, 256


def listed():
    return [
        # one token through an attention projection, 8-bit weight, adapter: the decode loop's latency
        dict(name="i8_decode_m1_4096x4096_r16", op="i8", M=1, N=4096, K=4096, r=16, out="bf16"),
        # a small batch of sequences decoding through a large MLP projection: the weight's stream
        dict(name="i8_decode_m16_22016x8192", op="i8", M=16, N=22016, K=8192, r=0, out="bf16"),
        # a prompt through an MLP projection with its adapter
        dict(name="i8_prefill_m2048_11008x4096_r64", op="i8", M=2048, N=11008, K=4096, r=64, out="bf16"),
        # a ragged prompt, an output width that is odd, float32 outputs (logits)
        dict(name="i8_odd_m333_5003x4096_f32", op="i8", M=333, N=5003, K=4096, r=0, out="f32"),
        # one token routed to two of eight experts: the smallest expert call
        dict(name="grp_decode_t2_e8_4096x4096_b4_r16", op="grouped", T=2, E=8, N=4096, K=4096, bits=4, r=16, pad=0),
        # sixteen decoding tokens, two experts each, on MLP-sized experts
        dict(name="grp_decode_t32_e8_11008x4096_b4", op="grouped", T=32, E=8, N=11008, K=4096, bits=4, r=0, pad=0),
        # many small experts, a short ragged batch in a padded buffer, 2-bit codes
        dict(name="grp_mid_t777_e64_1408x2048_b2_r8", op="grouped", T=777, E=64, N=1408, K=2048, bits=2, r=8, pad=55),
        # a long batch on large experts
        dict(name="grp_prefill_t8192_e8_4096x4096_b4_r64", op="grouped", T=8192, E=8, N=4096, K=4096, bits=4, r=64,
             pad=0),
        # 8-bit experts, a batch of medium raggedness
        dict(name="grp_prefill_t4096_e16_2816x2048_b8_r16", op="grouped", T=4096, E=16, N=2816, K=2048, bits=8, r=16,
             pad=0),
        # adapter training of a long batch on large experts
        dict(name="bwd_t4096_e8_4096x4096_b4_r16", op="grouped_bwd", T=4096, E=8, N=4096, K=4096, bits=4, r=16, pad=0),
        # adapter training of many small experts, some without a row, 3-bit codes
        dict(name="bwd_t777_e64_1408x2048_b3_r8", op="grouped_bwd", T=777, E=64, N=1408, K=2048, bits=3, r=8, pad=0),
        # one short sequence: the smallest training step
        dict(name="bwd_t64_e8_1024x1024_b4_r16", op="grouped_bwd", T=64, E=8, N=1024, K=1024, bits=4, r=16, pad=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["i8", "grouped", "grouped_bwd"])
    if op == "i8":
        N, K = _log_int(rng, 512, 16384), 64 * _log_int(rng, 8, 128)
        M = _log_int(rng, 1, 2048)
        if M * N * K > 2048 * 11008 * 4096:
            M = 2048 * 11008 * 4096 // (N * K)
        return dict(op=op, M=M, N=N, K=K, r=rng.choice([0, 4, 16, 64]), out=rng.choice(["bf16", "f32"]))
    E = _log_int(rng, 4, 64)
    N, K = 8 * _log_int(rng, 64, 1024), 64 * _log_int(rng, 8, 128)
    while E * N * K > 8 * 11008 * 4096:
        E = max(2, E // 2)
        N, K = max(512, 8 * (N // 16)), max(512, 64 * (K // 96))
    T = _log_int(rng, 1, 8192 if op == "grouped" else 4096)
    top = 8192 * 4096 * 4096 if op == "grouped" else 4096 * 4096 * 4096
    T = max(1, min(T, top // (N * K)))
    return dict(op=op, T=T, E=E, N=N, K=K, bits=rng.choice([2, 3, 4, 4, 8]), r=rng.choice([4, 8, 16, 64]),
                pad=rng.choice([0, 0, 37]))


def _counts(case):
    """Rows of each expert, from the case alone: a skewed router, small calls leaving experts without rows."""
    E, T = case["E"], case["T"]
    rng = np.random.RandomState(E * 7919 + T)
    p = np.exp(0.5 * rng.randn(E))
    return rng.multinomial(T, p / p.sum()).astype(np.int64)


def work(case):
    r = case["r"]
    if case["op"] == "i8":
        M, N, K = case["M"], case["N"], case["K"]
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": N * K + 4 * N + 2 * M * K + out * M * N + 2 * r * (N + K),
                "flops": 2 * M * N * K + 2 * M * r * (N + K)}
    T, E, N, K, bits = case["T"], case["E"], case["N"], case["K"], case["bits"]
    live = int((_counts(case) > 0).sum())
    weight = live * N * K * (bits / 8 + 1 / 64 + 4 / (64 * 256)) + 2 * live * r * (N + K)
    if case["op"] == "grouped":
        return {"bytes": int(weight + 2 * T * (N + K) + 4 * (E + 1)), "flops": 2 * T * N * K + 2 * T * r * (N + K)}
    # dy and x in, dx out, float32 adapter gradients of every expert out
    return {"bytes": int(weight + 2 * T * (N + 2 * K) + 4 * E * r * (N + K) + 4 * (E + 1)),
            "flops": 2 * T * N * K + 6 * T * r * (N + K)}


# ---------------------------------------------------------------- inputs

def _levels(bits, device, dtype=torch.float32):
    """The normal-quantile codebook: Q((i + 1/2) / 2^b) over the largest of them, each rounded to float32."""
    n = 1 << bits
    q = [statistics.NormalDist().inv_cdf((i + 0.5) / n) for i in range(n // 2)]
    half = torch.tensor([v / -q[0] for v in q], dtype=torch.float64).to(torch.float32)
    return torch.cat([half, -half.flip(0)]).to(device=device, dtype=dtype)


def _pack(codes, bits):
    """Codes (one per element, blocks of 64) as the little-endian bit string of each block."""
    c = codes.reshape(-1, 8).to(torch.int64)
    if bits == 8:
        return codes.to(torch.uint8).reshape(-1)
    word = (c << (bits * torch.arange(8, device=c.device))).sum(1)
    return ((word[:, None] >> (8 * torch.arange(bits, device=c.device))) & 255).to(torch.uint8).reshape(-1)


def _stacked_weight(rows, cols, bits, g):
    """A normal weight in the blockwise format: packed codes, 8-bit absmax codes, float32 steps."""
    dev = g.device
    nblk = rows * cols // BLOCK
    lv = _levels(bits, dev)
    mid = (lv[1:] + lv[:-1]) / 2
    codes, absmax = [], []
    step = 1 << 18
    for b in range(0, nblk, step):
        w = torch.randn((min(step, nblk - b), BLOCK), generator=g, device=dev) * 0.02
        a = w.abs().amax(1)
        codes.append(_pack(torch.bucketize((w / a[:, None]).contiguous(), mid), bits))
        absmax.append(a)
    a = torch.cat(absmax)
    ngrp = -(-nblk // GROUP)
    padded = torch.zeros(ngrp * GROUP, device=dev)
    padded[:nblk] = a
    cst = padded.view(ngrp, GROUP).amax(1) / 255
    q8 = torch.round(padded.view(ngrp, GROUP) / cst[:, None]).clamp(0, 255).to(torch.uint8).reshape(-1)[:nblk]
    return torch.cat(codes), q8.contiguous(), cst


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


def _activations(g, rows, cols):
    """Token rows as a hidden layer has them: a magnitude per token and a few strong channels."""
    x = _randn(g, rows, cols) * torch.exp(0.3 * _randn(g, rows, 1))
    strong = torch.rand(cols, generator=g, device=g.device) < 0.002
    return (x * torch.where(strong, 12.0, 1.0)).to(torch.bfloat16)


def _adapter(g, E, N, K, r):
    if r == 0:
        return None, None
    lead = () if E is None else (E,)
    return ((_randn(g, *lead, r, K) / math.sqrt(K)).to(torch.bfloat16), (_randn(g, *lead, N, r) * 0.02).to(torch.bfloat16))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = dict(case=case)
    N, K, r = case["N"], case["K"], case["r"]
    s["scale"] = 16.0 / r if r else 0.0
    if case["op"] == "i8":
        s["x"] = _activations(g, case["M"], K)
        w = _randn(g, N, K) * 0.02 * torch.exp(0.2 * _randn(g, N, 1))
        s["w_scale"] = w.abs().amax(1) / 127
        s["w_q"] = torch.round(w / s["w_scale"][:, None]).clamp(-127, 127).to(torch.int8)
        s["A"], s["B"] = _adapter(g, None, N, K, r)
        s["dtype"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    else:
        E, T = case["E"], case["T"]
        rows = T + case["pad"]
        counts = _counts(case)[np.random.RandomState(int(seed) & 0x7FFFFFFF).permutation(E)]
        s["cap"] = int(counts.max())
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=dev)
        s["codes"], s["q8"], s["cst"] = _stacked_weight(E * N, K, case["bits"], g)
        s["A"], s["B"] = _adapter(g, E, N, K, r)
        s["x"] = _activations(g, rows, K)
        if case["op"] == "grouped":
            s["y"] = torch.zeros((rows, N), dtype=torch.bfloat16, device=dev)
        else:
            s["dy"] = (_randn(g, rows, N) * 0.01).to(torch.bfloat16)
            s["dx"] = torch.zeros((rows, K), dtype=torch.bfloat16, device=dev)
    if own:
        # the prepared call that a decode or training loop keeps
        from quantized_base_fine_amd import qlr
        if case["op"] == "i8":
            s["call"] = qlr.LinearI8Call(s["x"], qlr.I8Rows(N, K, s["w_q"], s["w_scale"]), s["A"], s["B"], s["scale"],
                                         out_dtype=s["dtype"])
        else:
            qw = qlr.QWeight(case["bits"], case["E"] * N, K, s["codes"], s["q8"], s["cst"])
            if case["op"] == "grouped":
                s["call"] = qlr.GroupedCall(s["x"], qw, s["offsets"], s["A"], s["B"], s["scale"], out=s["y"])
            else:
                s["call"] = qlr.GroupedBwdCall(s["dy"], s["x"], qw, s["offsets"], s["A"], s["B"], s["scale"], dx=s["dx"])
    return s


# ---------------------------------------------------------------- the plain forms

def _dequantized(s, dtype):
    """The stacked weight (E, N, K): fl32(level[code] * fl32(absmax code * step))."""
    c = s["case"]
    bits, dev = c["bits"], s["codes"].device
    if bits == 8:
        codes = s["codes"].to(torch.int32)
    else:
        by = s["codes"].view(-1, bits).to(torch.int32)
        word = (by << (8 * torch.arange(bits, device=dev, dtype=torch.int32))).sum(1, dtype=torch.int64)
        codes = ((word[:, None] >> (bits * torch.arange(8, device=dev))) & ((1 << bits) - 1)).to(torch.int32)
    nblk = s["q8"].numel()
    scale = s["q8"].float() * s["cst"].repeat_interleave(GROUP)[:nblk]
    w = _levels(bits, dev)[codes.reshape(-1)].view(nblk, BLOCK) * scale[:, None]
    return w.view(c["E"], c["N"], c["K"]).to(dtype)


def _slots(s):
    """Row numbers of the routed rows and the place of each in a table of `cap` rows per expert."""
    off = s["offsets"].long()
    row = torch.arange(s["case"]["T"], device=off.device)
    e = torch.searchsorted(off[1:], row, right=True)
    return row, e * s["cap"] + row - off[e]


def _spread(s, slots, v, dtype):
    """The routed rows of v as an (E, cap, columns) table, empty places zero."""
    t = torch.zeros((s["case"]["E"] * s["cap"], v.shape[1]), dtype=dtype, device=v.device)
    t[slots] = v[:s["case"]["T"]].to(dtype)
    return t.view(s["case"]["E"], s["cap"], v.shape[1])


def _i8_plain(s):
    x = s["x"].float()
    xs = x.abs().amax(1) / 127
    # the quotient in 64 bits: a value next to a rounding border keeps its side
    q = torch.round(x.double() / xs.double().clamp_min(1e-300)[:, None]).clamp(-127, 127).float()
    y = (q @ s["w_q"].float().t()) * xs[:, None] * s["w_scale"]
    if s["A"] is not None:
        y = y + s["scale"] * ((x @ s["A"].float().t()) @ s["B"].float().t())
    return y.to(s["dtype"])


def _grouped_plain(s):
    c = s["case"]
    row, slots = _slots(s)
    x = _spread(s, slots, s["x"], torch.float32)
    y = torch.bmm(x, _dequantized(s, torch.float32).transpose(1, 2).contiguous())
    if s["A"] is not None:
        t = torch.bmm(x, s["A"].float().transpose(1, 2).contiguous())
        y = y + s["scale"] * torch.bmm(t, s["B"].float().transpose(1, 2).contiguous())
    out = s["y"].clone()
    out[:c["T"]] = y.view(-1, c["N"])[slots].to(out.dtype)
    return out


def _grouped_bwd_plain(s):
    c = s["case"]
    row, slots = _slots(s)
    x, dy = _spread(s, slots, s["x"], torch.float32), _spread(s, slots, s["dy"], torch.float32)
    A, B = s["A"].float(), s["B"].float()
    u = torch.bmm(dy, B)
    t = torch.bmm(x, A.transpose(1, 2).contiguous())
    dx = torch.bmm(dy, _dequantized(s, torch.float32)) + s["scale"] * torch.bmm(u, A)
    dA = s["scale"] * torch.bmm(u.transpose(1, 2).contiguous(), x)
    dB = s["scale"] * torch.bmm(dy.transpose(1, 2).contiguous(), t)
    out = s["dx"].clone()
    out[:c["T"]] = dx.view(-1, c["K"])[slots].to(out.dtype)
    return {"dx": out, "dA": dA, "dB": dB}


def run(state):
    if own:
        if state["case"]["op"] == "grouped_bwd":
            dx, dA, dB = state["call"]()
            return {"dx": dx, "dA": dA, "dB": dB}
        return state["call"]()
    return {"i8": _i8_plain, "grouped": _grouped_plain, "grouped_bwd": _grouped_bwd_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definition in float64, expert by expert, on the inputs that prepare makes."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    sc = s["scale"]
    if case["op"] == "i8":
        x = s["x"].double()
        xs = (s["x"].float().abs().amax(1, keepdim=True) / 127).double()
        q = torch.where(xs > 0, torch.round(x / xs), torch.zeros_like(x)).clamp(-127, 127)
        y = torch.matmul(q * xs, (s["w_q"].double() * s["w_scale"].double()[:, None]).t().contiguous())
        if s["A"] is not None:
            y += sc * torch.matmul(torch.matmul(x, s["A"].double().t().contiguous()), s["B"].double().t().contiguous())
        return y
    off = s["offsets"].tolist()
    N, K = case["N"], case["K"]
    W = _dequantized(s, torch.float32)
    if case["op"] == "grouped":
        y = s["y"].double()
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if b > a:
                x = s["x"][a:b].double()
                y[a:b] = torch.matmul(x, W[e].double().t().contiguous())
                if s["A"] is not None:
                    y[a:b] += sc * torch.matmul(torch.matmul(x, s["A"][e].double().t().contiguous()),
                                                s["B"][e].double().t().contiguous())
        return y
    dx = s["dx"].double()
    dA = torch.zeros((case["E"], case["r"], K), dtype=torch.float64, device=dx.device)
    dB = torch.zeros((case["E"], N, case["r"]), dtype=torch.float64, device=dx.device)
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if b > a:
            x, dy, A, B = s["x"][a:b].double(), s["dy"][a:b].double(), s["A"][e].double(), s["B"][e].double()
            u, t = torch.matmul(dy, B), torch.matmul(x, A.t().contiguous())
            dx[a:b] = torch.matmul(dy, W[e].double()) + sc * torch.matmul(u, A)
            dA[e] = sc * torch.matmul(u.t().contiguous(), x)
            dB[e] = sc * torch.matmul(dy.t().contiguous(), t)
    return {"dx": dx, "dA": dA, "dB": dB}
