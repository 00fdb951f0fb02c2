"""Measured cases of the rotary-position and 8-bit key/value-cache operators.

The operators and what a user's program does with them:
  rope, rope_bwd   rotary positions with several axes (time, height, width) on the Q and K
                   that the projections return, written as [B, H, N, d] for routing and
                   attention; and the same for the gradients on their way back
  append           new keys and values into a paged e4m3 cache, one power-of-two scale per
                   page and head, the keys rotated on the way
  attend           attention of a few (one token) or many (a frame) new queries per sequence
                   over that cache

Head counts, latent grids, head dims and block sizes are those of the video, sweep and tiny
workloads (21 x 30 x 52 tokens, 40 heads, d 128, block 128; 16 x 32 x 64, 8 heads; 512 tokens,
d 64, block 64); ragged batches and odd sizes stand beside them.
"""
import math

import numpy as np
import torch

own = False

THETA = 10000.0
FRAME_H, FRAME_W = 30, 52          # tokens of one latent frame: 30 x 52
AXES = {64: (24, 20, 20), 128: (44, 42, 42)}   # channels of the head turned by time, height, width


def listed():
    return [
        # a short clip through a small model: launch latency counts
        dict(name="rope_tiny", op="rope", B=1, H=2, N=512, d=64, layout="bhnd", pairing="interleaved"),
        # one attention layer of the video model: projections' [B, N, H, d] in, [B, H, N, d] out
        dict(name="rope_video", op="rope", B=1, H=40, N=32760, d=128, layout="bnhd", pairing="interleaved"),
        # the gradients of a training step at the sweep's size, back into the projections' layout
        dict(name="rope_bwd_sweep", op="rope_bwd", B=1, H=8, N=32768, d=64, layout="bnhd", pairing="interleaved"),
        # an odd clip out of one fused projection, the two halves of the head turned against each other
        dict(name="rope_bwd_odd", op="rope_bwd", B=3, H=7, N=1571, d=128, layout="qkv", pairing="half"),
        # one new token per sequence of a small batch
        dict(name="append_token", op="append", B=8, H=40, T=1, start=9001, d=128, block=128, ragged=False, rope=True),
        # a ragged batch of chunks, some of them short, into pages of 64 tokens
        dict(name="append_ragged", op="append", B=5, H=8, T=333, start=2077, d=64, block=64, ragged=True, rope=True),
        # three latent frames of the video model at once
        dict(name="append_frames", op="append", B=1, H=40, T=4680, start=1560, d=128, block=128, ragged=False,
             rope=True),
        # one token against a short cache: launch latency counts
        dict(name="attend_token_tiny", op="attend", B=1, Hkv=8, G=1, M=1, len=509, d=64, block=64, causal=True,
             ragged=False),
        # one token per sequence of a ragged batch, long caches
        dict(name="attend_token_batch", op="attend", B=8, Hkv=40, G=1, M=1, len=16381, d=128, block=128, causal=True,
             ragged=False),
        # a few drafted tokens each, query heads sharing key heads, one sequence still empty
        dict(name="attend_few_shared", op="attend", B=4, Hkv=8, G=4, M=5, len=8111, d=128, block=64, causal=True,
             ragged=True),
        # a chunk of a prompt behind what is cached
        dict(name="attend_chunk", op="attend", B=2, Hkv=8, G=2, M=333, len=4099, d=64, block=128, causal=True,
             ragged=True),
        # a whole latent frame against the clip so far
        dict(name="attend_frame", op="attend", B=1, Hkv=40, G=1, M=1560, len=32760, d=128, block=128, causal=False,
             ragged=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "attend", "attend"])
    d = rng.choice([64, 128])
    if op in ("rope", "rope_bwd"):
        H = _log_int(rng, 1, 40)
        B = _log_int(rng, 1, 4)
        N = _log_int(rng, 1, min(32768, 40 * 32760 // (B * H)))
        return dict(op=op, B=B, H=H, N=N, d=d, layout=rng.choice(["bhnd", "bnhd", "qkv"]),
                    pairing=rng.choice(["interleaved", "half"]))
    block = rng.choice([64, 128])
    if op == "append":
        H = _log_int(rng, 1, 40)
        B = _log_int(rng, 1, 16)
        T = _log_int(rng, 1, min(4680, 40 * 4680 // (B * H)))
        return dict(op=op, B=B, H=H, T=T, start=_log_int(rng, 1, 8192) - 1, d=d, block=block,
                    ragged=rng.random() < 0.5, rope=rng.random() < 0.75)
    Hkv, G = _log_int(rng, 1, 40), rng.choice([1, 1, 2, 4, 8])
    B = _log_int(rng, 1, 16)
    M = _log_int(rng, 1, 2048)
    most = min(32768, 40 * 1560 * 32760 // (B * Hkv * G * M), 8 * 40 * 16384 // (B * Hkv))
    M = min(M, most)
    return dict(op=op, B=B, Hkv=Hkv, G=G, M=M, len=_log_int(rng, M, max(M, most)), d=d, block=block,
                causal=rng.random() < 0.6, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------- sizes that follow from a case


def _new_lens(c, most):
    """Valid new tokens of each sequence: all, or (ragged) fewer and fewer, the last sequence's none."""
    if not c["ragged"]:
        return [most] * c["B"]
    return [most - (most * b) // max(1, c["B"] - 1) if c["B"] > 1 else most for b in range(c["B"])]


def _starts(c):
    """Cached tokens of each sequence before an append: from `start` down to about a third of it."""
    return [c["start"] - (2 * c["start"] * b) // (3 * c["B"]) for b in range(c["B"])]


def _lens(c):
    """Cached tokens of each sequence, its new ones among them: from `len` down to about a quarter; with
    ragged batches of more than one sequence the last one has none."""
    new = _new_lens(c, c["M"])
    lens = [max(n, c["len"] - (3 * c["len"] * b) // (4 * c["B"])) for b, n in enumerate(new)]
    if c["ragged"] and c["B"] > 1:
        lens[-1] = 0
    return lens


def work(c):
    if c["op"] in ("rope", "rope_bwd"):
        n = 2 * c["B"] * c["H"] * c["N"] * c["d"]
        return {"bytes": 4 * n + 12 * c["B"] * c["N"], "flops": 3 * n}
    if c["op"] == "append":
        n = sum(_new_lens(c, c["T"])) * c["H"] * c["d"]
        return {"bytes": 2 * n * 3, "flops": (3 if c["rope"] else 0) * n + 2 * n}
    new, lens = _new_lens(c, c["M"]), _lens(c)
    Hq = c["Hkv"] * c["G"]
    keys = sum(sum(max(0, k - n + m + 1) for m in range(n)) if c["causal"] else n * k for n, k in zip(new, lens))
    rows = sum(new) * Hq
    return {"bytes": sum(lens) * c["Hkv"] * 2 * c["d"] + rows * (4 * c["d"] + 4), "flops": 4 * c["d"] * Hq * keys}


# ---------------------------------------------------------------- inputs


def _frequencies(d):
    """Per channel pair: angle per unit of position (fp64) and the axis whose position turns it."""
    f = [THETA ** (-2.0 * j / n) for n in AXES[d] for j in range(n // 2)]
    a = [i for i, n in enumerate(AXES[d]) for j in range(n // 2)]
    return np.array(f, dtype=np.float64), np.array(a, dtype=np.int32)


def _grid_positions(first, n):
    """(time, height, width) of tokens first .. first + n - 1 of a clip of 30 x 52 frames."""
    t = torch.arange(first, first + n, dtype=torch.int64, device="cuda")
    per = FRAME_H * FRAME_W
    return torch.stack([t // per, t % per // FRAME_W, t % FRAME_W], -1).to(torch.int32)


def _heads(g, B, H, n, d, layout):
    """Two bf16 tensors [B, H, n, d] in the layout the case names (views where it is another one)."""
    scale = 0.5 + 2.0 * torch.rand(2, H, 1, 1, generator=g, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    if layout == "bhnd":
        return [normal(B, H, n, d).mul_(s) for s in scale]
    if layout == "bnhd":
        return [normal(B, n, H, d).mul_(s.view(H, 1)).transpose(1, 2) for s in scale]
    x = normal(B, n, 3, H, d)
    return [x[:, :, i].mul_(scale[i].view(H, 1)).transpose(1, 2) for i in range(2)]


def _pool(g, pages, H, block, d):
    """Codes and scale exponents of a pool of pages as quantized normal values leave them."""
    def codes():
        x = torch.randn(pages, H, block, d, generator=g, device="cuda", dtype=torch.float16).mul_(80.0)
        return x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)

    def exps():
        return torch.randint(-7, -5, (pages, H), generator=g, device="cuda", dtype=torch.int32)

    return codes(), exps(), codes(), exps()


def _table(g, B, per_seq, spare):
    """A page table of B sequences, the pages of the pool in an arbitrary order; the pool's size; an unused page."""
    pages = B * per_seq + spare
    perm = torch.randperm(pages, generator=g, device="cuda")
    return perm[: B * per_seq].to(torch.int32).view(B, per_seq).contiguous(), pages, perm[-1]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(c)
    d = c["d"]
    s["inv_freq"], s["axis"] = _frequencies(d)
    s["freq_dev"] = torch.from_numpy(s["inv_freq"]).cuda()
    s["axis_dev"] = torch.from_numpy(s["axis"]).long().cuda()
    if c["op"] in ("rope", "rope_bwd"):
        s["Q"], s["K"] = _heads(g, c["B"], c["H"], c["N"], d, "bhnd" if c["op"] == "rope_bwd" else c["layout"])
        s["pos"] = _grid_positions(0, c["N"])
        if c["op"] == "rope_bwd" and c["layout"] != "bhnd":  # where the gradients go: the projections' layout
            n = 3 if c["layout"] == "qkv" else 2
            grads = torch.zeros(c["B"], c["N"], n, c["H"], d, dtype=torch.bfloat16, device="cuda")
            s["outs"] = [grads[:, :, i].transpose(1, 2) for i in range(2)]
        return s
    block = c["block"]
    if c["op"] == "append":
        starts, new = _starts(c), _new_lens(c, c["T"])
        per_seq = -(-(c["start"] + c["T"]) // block)
        s["table"], pages, s["unused"] = _table(g, c["B"], per_seq, 3)
        s["pool"] = _pool(g, pages, c["H"], block, d)
        s["K"], s["V"] = _heads(g, c["B"], c["H"], c["T"], d, "bnhd")
        s["start"] = _ints(starts)
        s["new"] = _ints(new) if c["ragged"] else None
        s["pos"] = torch.stack([_grid_positions(x, c["T"]) for x in starts]).contiguous() if c["rope"] else None
        return s
    per_seq = -(-c["len"] // block)
    s["table"], pages, _ = _table(g, c["B"], per_seq, 2)
    s["pool"] = _pool(g, pages, c["Hkv"], block, d)
    Hq = c["Hkv"] * c["G"]
    s["Q"] = torch.randn(c["B"], Hq, c["M"], d, generator=g, device="cuda", dtype=torch.bfloat16)
    s["lens"] = _ints(_lens(c))
    s["new"] = _ints(_new_lens(c, c["M"])) if c["ragged"] else None
    s["O"] = torch.zeros(c["B"], Hq, c["M"], d, dtype=torch.bfloat16, device="cuda")
    s["LSE"] = torch.zeros(c["B"], Hq, c["M"], dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- the operators


def run(s):
    if own:
        return _run_own(s)
    if s["op"] in ("rope", "rope_bwd"):
        back = s["op"] == "rope_bwd"
        outs = s.get("outs", [None, None])
        return [_plain_rope(x, s["pos"], s, back, o) for x, o in zip((s["Q"], s["K"]), outs)]
    return _plain_append(s) if s["op"] == "append" else _plain_attend(s)


def _run_own(s):
    import top_routed_block_b200 as fv
    if s["op"] in ("rope", "rope_bwd"):
        rope = fv.RopeAxes(s["inv_freq"], s["axis"], s["pairing"])
        outs = s.get("outs", (None, None))
        f = fv.fvattn_rope if s["op"] == "rope" else fv.fvattn_rope_bwd
        return list(f(s["Q"], s["K"], s["pos"], rope, out_q=outs[0], out_k=outs[1]))
    pages = fv.KvPages(*s["pool"])
    if s["op"] == "append":
        rope = fv.RopeAxes(s["inv_freq"], s["axis"], "interleaved") if s["rope"] else None
        fv.fvattn_cache_append(s["K"], s["V"], pages, s["table"], s["start"], new_lens=s["new"], positions=s["pos"],
                               rope=rope)
        return _pool_values(s["pool"])
    O, LSE, _ = fv.fvattn_cache_attend(s["Q"], pages, s["table"], s["lens"], new_lens=s["new"], causal=s["causal"],
                                       O=s["O"], LSE=s["LSE"])
    return [O, LSE]


def _pool_values(pool):
    """The pool as it stands: codes as the 8-bit numbers they are, and the scale exponents."""
    k, ke, v, ve = pool
    return [k.view(torch.float8_e4m3fn), ke, v.view(torch.float8_e4m3fn), ve]


def _turn(x, pos, s, pairing, back):
    """x fp32 [B, H, n, d] turned by pos int [n, axes] or [B, n, axes]; angles in 64 bits."""
    angle = pos.double()[..., s["axis_dev"]] * s["freq_dev"]
    cos, sin = angle.cos().float(), angle.sin().float()
    if pos.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    if back:
        sin = -sin
    if pairing == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_rope(x, pos, s, back, out):
    y = _turn(x.float(), pos, s, s["pairing"], back).to(torch.bfloat16)
    return y.contiguous() if out is None else out.copy_(y)


def _scale_need(amax):
    """The smallest e with amax 2^-e <= 448, from amax = m 2^x with m in [1/2, 1): 448 = 7/8 2^9."""
    m, x = torch.frexp(amax)
    return torch.where(m <= 0.875, x - 9, x - 8)


def _round_e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _place(s):
    """What goes into each slot of the pages that the new tokens reach: the new token's index [B, P, block],
    whether one goes there, whether an older token is there; and the pages [B, P] (where no new token
    goes, one that no sequence has and that keeps its contents)."""
    block, T = s["block"], s["T"]
    start = s["start"].long()
    n = s["new"].long() if s["new"] is not None else torch.full_like(start, T)
    first = start // block
    j = torch.arange((T + block - 2) // block + 1, device="cuda")
    at = (first[:, None] + j)[:, :, None] * block + torch.arange(block, device="cuda")
    token = at - start[:, None, None]
    is_new = (token >= 0) & (token < n[:, None, None])
    is_old = (token < 0) & is_new.any(-1, keepdim=True)
    page = s["table"].long().gather(1, (first[:, None] + j).clamp(max=s["table"].shape[1] - 1))
    page = torch.where(is_new.any(-1), page, s["unused"])
    return token.clamp(0, T - 1), is_new, is_old, page


def _plain_append(s):
    token, is_new, is_old, page = _place(s)
    B, P, block = token.shape
    K = s["K"].float()
    if s["rope"]:
        K = _turn(K, s["pos"], s, "interleaved", False)
    b = torch.arange(B, device="cuda")[:, None, None]
    touched = is_new.any(-1)[..., None]
    for x, codes, exps in ((K, s["pool"][0], s["pool"][1]), (s["V"].float(), s["pool"][2], s["pool"][3])):
        new = x.transpose(1, 2)[b, token].transpose(2, 3)                # [B, P, H, block, d]
        keep = is_new[:, :, None, :, None]
        amax = (new.abs() * keep).amax((-1, -2))                         # [B, P, H]
        e_old = exps[page]
        e = torch.where(is_old.any(-1)[..., None], torch.maximum(e_old, _scale_need(amax)), _scale_need(amax))
        old = codes[page].view(torch.float8_e4m3fn).float()              # the older tokens, on the page's new scale
        old = torch.ldexp(old, (e_old - e)[..., None, None])
        put = _round_e4m3(torch.where(keep, torch.ldexp(new, -e[..., None, None]), old)).view(torch.uint8)
        exps[page] = torch.where(touched, e, e_old)
        codes[page] = torch.where((is_new | is_old)[:, :, None, :, None], put, codes[page])
    return _pool_values(s["pool"])


def _cached(codes, exps, table):
    """fp32 values [B, H, L, d] of the pages a table names."""
    B, P = table.shape
    v = codes[table.long()].view(torch.float8_e4m3fn).float()
    v = torch.ldexp(v, exps[table.long()][..., None, None])
    return v.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(s):
    B, Hkv, G, M, d = s["B"], s["Hkv"], s["G"], s["M"], s["d"]
    K, V = (_cached(s["pool"][i], s["pool"][i + 1], s["table"]) for i in (0, 2))
    L = K.shape[2]
    lens = s["lens"].long()
    n = s["new"].long() if s["new"] is not None else torch.full_like(lens, M)
    m = torch.arange(M, device="cuda")
    u = torch.arange(L, device="cuda")
    limit = (lens - n)[:, None] + m + 1 if s["causal"] else lens[:, None].expand(B, M)
    seen = (u < limit[..., None]) & (u < lens[:, None, None])                        # [B, M, L]
    Q = s["Q"].float().view(B, Hkv, G, M, d)
    S = (Q.flatten(2, 3) @ K.transpose(-1, -2)).view(B, Hkv, G, M, L) * (1.0 / math.sqrt(d))
    S = S.masked_fill_(~seen[:, None, None], -math.inf)
    top = S.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    S = S.sub_(top).exp_()
    total = S.sum(-1, keepdim=True)
    V = V * (u < lens[:, None])[:, None, :, None]
    O = (S.flatten(2, 3) @ V).view(B, Hkv, G, M, d) / torch.where(total > 0, total, torch.ones_like(total))
    LSE = (top + total.log()).squeeze(-1)
    valid = (m < n[:, None])[:, None, :]
    s["O"].copy_(torch.where(valid[..., None], O.reshape(B, Hkv * G, M, d).to(torch.bfloat16), s["O"]))
    s["LSE"].copy_(torch.where(valid, LSE.reshape(B, Hkv * G, M), s["LSE"]))
    return [s["O"], s["LSE"]]


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_turn(x, pos, s, pairing, sign):
    """Each pair of channels as a complex number, times exp(i sign angle)."""
    d = x.shape[-1]
    f = torch.tensor(s["inv_freq"], dtype=torch.float64, device=x.device)
    theta = torch.stack([pos[..., int(a)].double() * f[i] for i, a in enumerate(s["axis"])], -1) * sign
    unit = torch.polar(torch.ones_like(theta), theta)
    unit = unit.unsqueeze(1) if pos.dim() == 3 else unit
    x = x.double()
    if pairing == "half":
        z = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous()) * unit
        return torch.cat([z.real, z.imag], -1)
    return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous()) * unit).flatten(-2)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("rope", "rope_bwd"):
        sign = -1.0 if c["op"] == "rope_bwd" else 1.0
        return [_exact_turn(x, s["pos"], s, c["pairing"], sign) for x in (s["Q"], s["K"])]
    return _exact_append(c, s) if c["op"] == "append" else _exact_attend(c, s)


def _exact_append(c, s):
    """Codes before their rounding: every value of a touched page over the page's scale, in 64 bits."""
    block, H = c["block"], c["H"]
    K = s["K"].double()
    if c["rope"]:
        K = _exact_turn(s["K"], s["pos"], s, "interleaved", 1.0)
    table, starts, new = s["table"].tolist(), s["start"].tolist(), _new_lens(c, c["T"])
    outs = []
    for x, codes, exps in ((K, s["pool"][0], s["pool"][1]), (s["V"].double(), s["pool"][2], s["pool"][3])):
        values = codes.view(torch.float8_e4m3fn).double()
        for b in range(c["B"]):
            t = 0
            while t < new[b]:
                page, slot = divmod(starts[b] + t, block)
                page = table[b][page]
                n = min(block - slot, new[b] - t)
                part = x[b, :, t: t + n]
                amax = part.abs().amax((-1, -2))
                need = torch.ceil(torch.log2(amax / 448.0))
                need -= (amax <= 448.0 * torch.exp2(need - 1.0)).double()  # the logarithm's own rounding
                need = need.to(torch.int32)
                e = torch.maximum(need, exps[page]) if slot else need
                values[page, :, :slot] *= torch.exp2((exps[page] - e).double())[:, None, None]
                values[page, :, slot: slot + n] = part * torch.exp2(-e.double())[:, None, None]
                t += n
        outs += [values, None]
    return outs


def _exact_attend(c, s):
    lens, new = _lens(c), _new_lens(c, c["M"])
    O, LSE = s["O"].double(), s["LSE"].double()
    k, ke, v, ve = s["pool"]
    for b in range(c["B"]):
        n, cached = new[b], lens[b]
        if not n:
            continue
        ids = s["table"][b].long()
        for h in range(c["Hkv"]):
            def values(codes, exps):
                x = codes[ids, h].view(torch.float8_e4m3fn).double() * torch.exp2(exps[ids, h].double())[:, None, None]
                return x.flatten(0, 1)[:cached]
            keys, vals = values(k, ke), values(v, ve)
            for q in range(h * c["G"], (h + 1) * c["G"]):
                x = s["Q"][b, q, :n].double() @ keys.T / math.sqrt(c["d"])
                if c["causal"]:
                    hide = torch.arange(cached, device="cuda") > torch.arange(n, device="cuda")[:, None] + cached - n
                    x = x.masked_fill(hide, -math.inf)
                LSE[b, q, :n] = torch.logsumexp(x, -1) if cached else -math.inf
                O[b, q, :n] = torch.softmax(x, -1) @ vals if cached else 0.0
    return [O, LSE]
